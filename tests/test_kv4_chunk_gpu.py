"""GPU parity of the 4-bit cache attention for many new rows per request (chunks of prompts and whole
prompts, in tiles of 128 rows) against its formula in 64 bits."""
import numpy as np
import pytest
import torch

from tests import block_reference as ref
from tests.gpu_common import qk  # noqa: F401
from tests.test_kv4_gpu import INDEX, Batch, bits, i32

pytestmark = pytest.mark.gpu


def chunks(qk, lens, rows, Hkv, G, D, page=16, **kw):  # noqa: F811
    """A batch that is worked on in tiles of 128 rows: its average request fills three quarters of one per
    kv head, and there are 96 of them or more."""
    c = Batch(qk, lens, rows, Hkv, D, page, **kw)
    average = G * -(-c.T // len(lens))
    assert average >= 96 and len(lens) * Hkv * -(-average // 128) >= 96
    return c


LENS = [300, 129, 64, 65, 700, 1, 128]
ROWS = [300, 100, 64, 65, 128, 1, 127]


@pytest.mark.parametrize("D,G,page", [(128, 2, 16), (64, 3, 48), (128, 5, 1024), (64, 1, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (5, 4), (64, 64), (100, 17), (300, 1), (100000, 3)])
def test_chunks_and_windows(qk, D, G, page, window, sinks):  # noqa: F811
    """Ragged chunks and whole prompts; rows of nobody stay as they were."""
    c = chunks(qk, LENS, ROWS, 16, G, D, page, seed=window + G, front=2, behind=3)
    q = c.q(16 * G)
    out = torch.full((c.T, 16 * G, D), 7.0, dtype=torch.bfloat16, device="cuda")
    qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu, window=window, sinks=sinks, out=out)
    c.check(q, out, window=window, sinks=sinks)
    assert (out[:2] == 7).all() and (out[c.first[-1]:] == 7).all()
    qk.qk_check_device_error()


@pytest.mark.parametrize("lens,rows,Hkv,G,D", [
    ([512] * 4, [512] * 4, 8, 4, 128),            # prompts: items of 1 to 8 blocks of keys, several to a block
    ([2000], [2000], 4, 3, 64),                   # one prompt, row tiles that end inside a token
    ([5000, 70], [600, 70], 8, 4, 128),           # a chunk behind a long cache
    ([9] * 1000, [9] * 1000, 1, 16, 64),          # more requests than threads
    ([40, 0, 1] * 300, [13, 0, 1] * 300, 2, 32, 128),
    ([700] + [0] * 6, [700] + [0] * 6, 16, 2, 128),  # all rows in one request
    ([20000, 30], [4, 30], 8, 64, 128),           # few tokens of many heads over a long cache
])
def test_spans_of_chunks(qk, lens, rows, Hkv, G, D):  # noqa: F811
    """Items cut between blocks; the same bits on a second run."""
    c = chunks(qk, lens, rows, Hkv, G, D, seed=len(lens))
    q = c.q(Hkv * G)
    out = qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu)
    c.check(q, out, requests=range(0, len(lens), max(1, len(lens) // 20)))
    for _ in range(3):
        again = qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu)
        assert torch.equal(bits(out), bits(again))
    qk.qk_check_device_error()


@pytest.mark.parametrize("seed", range(10))
def test_drawn_chunks(qk, seed):  # noqa: F811
    r = np.random.default_rng(700 + seed)
    B, D, page = int(r.integers(6, 12)), int(r.choice([64, 128])), int(r.choice([16, 32, 80, 256]))
    Hkv, G = 16, int(r.integers(1, 4))
    lens = np.exp(r.uniform(np.log(200), np.log(1500), B)).astype(int).tolist()
    rows = [int(r.integers(100, n + 1)) for n in lens]
    window, sinks = int(r.choice([0, r.integers(1, 1000)])), int(r.integers(0, 200))
    c = chunks(qk, lens, rows, Hkv, G, D, page, seed=seed, front=int(r.integers(0, 3)), behind=int(r.integers(0, 3)))
    qkv = c.randn(c.T, Hkv * G * D + 24).bfloat16()  # strided rows
    q = qkv[:, 8:8 + Hkv * G * D].unflatten(1, (Hkv * G, D))
    scale = float(r.choice([D ** -0.5, 0.0, 0.02, 1.0]))
    out = qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu, scale=scale, window=window, sinks=sinks)
    c.check(q, out, scale=scale, window=window, sinks=sinks)
    qk.qk_check_device_error()


def test_rows_in_front_of_the_first_token(qk):  # noqa: F811
    """More rows than tokens: the first ones, and an empty request's, are 0; without row bounds every
    request has T / B rows."""
    lens = [30, 0, 200, 100, 99, 5]
    c = chunks(qk, lens, [100] * 6, 16, 1, 64, seed=1)
    q = c.q(16)
    for cu in (c.cu, None):
        out = torch.full((c.T, 16, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        qk.qk_kv4_attention(q, c.cache, c.table, c.lens, cu, out=out)
        for b, n in enumerate(lens):
            m = min(n, 100)
            mine = out[100 * b:100 * b + 100]
            assert not mine[:100 - m].any(), b
            if m:
                k, v = ref.request_kv(c.cache, c.table[b], n, 64)
                want, tol = ref.attention(q[100 * b + 100 - m:100 * b + 100], k, v, 0.125, 0, 0)
                assert ((mine[100 - m:].double() - want).abs() <= tol).all(), b
    qk.qk_check_device_error()


@pytest.mark.parametrize("D", [64, 128])
def test_infinite_values_reach_the_rows_that_see_them(qk, D):  # noqa: F811
    """A token whose value group holds infinities: NaN in that group of the rows that see it, and nothing
    else, neither in the rows in front of it nor in the other group."""
    c = chunks(qk, [200] * 6, [200] * 6, 16, 1, D, seed=D)
    q = c.q(16)
    k, v = ref.request_kv(c.cache, c.table[0], 200, D)
    place = c.table[0, 4:5, None].clone()  # tokens 64 .. 79 of request 0, by a table of their page
    kk, vv = k[77:78].bfloat16(), v[77:78].bfloat16()
    vv[0, :, 3] = float("inf")
    qk.qk_kv4_append(kk, vv, c.cache, place, i32([14]))
    for window in (0, 20):
        out = qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu, window=window)
        k, v = ref.request_kv(c.cache, c.table[0], 200, D)
        sees = torch.zeros(200, dtype=torch.bool, device="cuda")
        sees[77:77 + (window or 200)] = True
        assert torch.isnan(out[:200][sees][..., :64]).all()
        want, tol = ref.attention(q[:200], k, v.nan_to_num(0, 0, 0), D ** -0.5, window, 0)
        good = (out[:200].double() - want).abs() <= tol
        assert good[~sees].all() and good[..., 64:].all()
        c.check(q, out, window=window, requests=[1, 5])
    qk.qk_check_device_error()


@pytest.mark.parametrize("D,G", [(64, 1), (128, 2)])
def test_value_scales_far_apart_in_chunks(qk, D, G):  # noqa: F811
    """Value scales over fp16's range in every order of size and score: every output within the rounding
    of its own sum P scale code (the bounds are those of the calls of few rows)."""
    g = torch.Generator(device="cuda").manual_seed(D + G)
    lens, rows = [500, 130, 333] * 2, [128, 130, 100] * 2
    n, bounds = sum(lens), np.concatenate([[0], np.cumsum(lens)])
    for trend in (-1, 0, 1, 2):
        c = chunks(qk, lens, rows, 16, G, D, seed=trend + 5, fill=False)
        at = torch.cat([torch.linspace(0, 1, m, device="cuda") for m in lens])
        if trend == 0:
            at = torch.rand(n, generator=g, device="cuda")
        if trend == 2:  # a first token of huge values, then tiny ones
            at = torch.where(at == 0, 1.0, 0.3)
        size = torch.exp2(-20 + 33 * (at if trend >= 0 else 1 - at))[:, None, None]
        v = (torch.randn(n, 16, D, generator=g, device="cuda") * size).bfloat16()
        v[5::7] = 0.0
        k = torch.randn(n, 16, D, generator=g, device="cuda").bfloat16()
        qk.qk_kv4_append(k, v, c.cache, c.table, c.lens, i32(bounds))
        for strength in (0.0, 1.0, 8.0):
            q = (c.randn(c.T, 16 * G, D) * strength).bfloat16()
            out = qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu)
            for b, m in enumerate(lens):
                kk, vv = ref.request_kv(c.cache, c.table[b], m, D)
                _, _, s, o = ref.quantize4(v[bounds[b]:bounds[b + 1]])
                reach = (15 * s + o.abs()).repeat_interleave(64, -1)  # of a key's codes and offset
                mine = q[c.first[b]:c.first[b + 1]]
                want, _ = ref.attention(mine, kk, vv, D ** -0.5, 0, 0)
                part, _ = ref.attention(mine, kk, reach, D ** -0.5, 0, 0)
                a = 3 * D ** -0.5 * mine.double().abs().sum(-1).amax() * kk.abs().amax()
                move = 2.0 ** -11 + m * 2.0 ** -30 + 2 * a * 2.0 ** -17 + 2.0 ** -20 + (m / 8 + 400) * 2.0 ** -23
                got = out[c.first[b]:c.first[b + 1]].double()
                assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + part * move).all(), (trend, strength, b)
    qk.qk_check_device_error()


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -30, 2.0 ** 30, 2.0 ** 100])
def test_query_sizes_of_chunks(qk, size):  # noqa: F811
    c = chunks(qk, [150] * 6, [100] * 6, 16, 1, 128)
    q = (c.randn(c.T, 16, 128) * size).bfloat16()
    scale = min(128 ** -0.5 / size, 2.0 ** 98)
    out = qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu, scale=scale)
    c.check(q, out, scale=scale)
    qk.qk_check_device_error()


@pytest.mark.parametrize("D", [64, 128])
def test_missing_pages_under_chunks(qk, D):  # noqa: F811
    """Pages that are not there: their keys are as if masked, and the call reports them; pages that no
    row's window holds may be gone."""
    n, rows = 1500, 128
    c = chunks(qk, [n] * 6, [rows] * 6, 16, 1, D, seed=D)
    q = c.q(16)
    gone = [0, 1, 5, 31, 32, 33, 60, 61, 62, 63]
    table = c.table.clone()
    table[0, gone] = i32([-1, c.P] * (len(gone) // 2))
    out = qk.qk_kv4_attention(q, c.cache, table, c.lens, c.cu)
    with pytest.raises(qk.QKError) as e:
        qk.qk_check_device_error()
    assert e.value.status == INDEX
    k, v = ref.request_kv(c.cache, c.table[0], n, D)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    for g in gone:
        keep[16 * g:16 * g + 16] = False
    want, tol = ref.attention(q[:rows], k[keep], v[keep], D ** -0.5, 0, 0)
    assert ((out[:rows].double() - want).abs() <= tol).all()
    c.check(q, out, requests=[1, 5])
    want = qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu, window=100, sinks=20)
    table = c.table.clone()
    table[:, 2:(n - rows - 100 + 1) // 16] = -1
    got = qk.qk_kv4_attention(q, c.cache, table, c.lens, c.cu, window=100, sinks=20)
    assert torch.equal(bits(got), bits(want))
    qk.qk_check_device_error()
    for lens in ([-5] + [n] * 5, [10 ** 9] + [n] * 5):
        out = qk.qk_kv4_attention(q, c.cache, c.table, i32(lens), c.cu)
        with pytest.raises(qk.QKError):
            qk.qk_check_device_error()
        c.check(q, out, requests=[3])
    for cu in ([0, 128, 0, 2, 3, 4, 5], [0, 128, 256, 9999, 9999, 9999, 9999], [-3, 1, 2, 4, 5, 6, 768]):
        qk.qk_kv4_attention(q, c.cache, c.table, c.lens, i32(cu))
        with pytest.raises(qk.QKError):
            qk.qk_check_device_error()


def test_no_rows_in_any_request(qk):  # noqa: F811
    c = chunks(qk, [50] * 6, [50] * 6, 16, 2, 128)
    q = c.q(32)
    out = torch.full_like(q, 7.0)
    qk.qk_kv4_attention(q, c.cache, c.table, c.lens, torch.zeros_like(c.cu), out=out)
    assert (out == 7).all()
    qk.qk_check_device_error()


def test_graph_of_chunks_with_new_lengths(qk):  # noqa: F811
    """A captured chunk and a captured single step that share a workspace, replayed in turn while lengths,
    row bounds and queries change; and two chunks in flight on two streams."""
    lens, rows = [700, 300, 128, 90, 200, 400], [128, 128, 128, 90, 100, 110]
    c = chunks(qk, lens, rows, 16, 1, 128, seed=3)
    q = c.q(16)
    ws = torch.empty(qk.qk_kv4_attention_workspace_size(128), dtype=torch.uint8, device="cuda")
    out, one = torch.empty_like(q), torch.empty_like(q[:6])
    now, cu = c.lens.clone(), c.cu.clone()
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        qk.qk_kv4_attention(q, c.cache, c.table, now, cu, out=out, workspace=ws)
        qk.qk_kv4_attention(q[:6], c.cache, c.table, now, out=one, workspace=ws)
    torch.cuda.current_stream().wait_stream(warm)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        qk.qk_kv4_attention(q, c.cache, c.table, now, cu, out=out, workspace=ws)
    with torch.cuda.graph(g2):
        qk.qk_kv4_attention(q[:6], c.cache, c.table, now, out=one, workspace=ws)
    for less in (0, 1, 60):
        c.lens_list = [n - less for n in lens]
        c.rows_list = [max(n - less, 0) for n in rows]
        c.first = np.concatenate([[0], np.cumsum(c.rows_list)])
        now.copy_(i32(c.lens_list))
        cu.copy_(i32(c.first))
        q.copy_(c.q(16))
        g1.replay()
        g2.replay()
        c.check(q, out)
        for b in range(6):
            k, v = ref.request_kv(c.cache, c.table[b], c.lens_list[b], 128)
            want, tol = ref.attention(q[b:b + 1], k, v, 128 ** -0.5, 0, 0)
            assert ((one[b:b + 1].double() - want).abs() <= tol).all()
    q2 = c.q(16)
    w1 = qk.qk_kv4_attention(q, c.cache, c.table, now, cu)
    w2 = qk.qk_kv4_attention(q2, c.cache, c.table, now, cu)
    mine = slice(0, int(c.first[-1]))
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        o1 = qk.qk_kv4_attention(q, c.cache, c.table, now, cu, stream=a, out=torch.empty_like(q))
        o2 = qk.qk_kv4_attention(q2, c.cache, c.table, now, cu, stream=b, out=torch.empty_like(q))
        torch.cuda.synchronize()
        assert torch.equal(bits(o1[mine]), bits(w1[mine])) and torch.equal(bits(o2[mine]), bits(w2[mine]))
    qk.qk_check_device_error()
