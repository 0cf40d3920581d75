"""GPU tests of the operators between two linears at the edges of their contracts: NaN rows, lengths and row
bounds out of range, queries and scores at the ends of their ranges, every key counted, calls beside other
threads and streams."""
import threading
import time

import numpy as np
import pytest
import torch

from tests import block_reference as ref
from tests.gpu_common import qk  # noqa: F401
from tests.test_kv4_gpu import INDEX, Batch, bits, i32

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


# -------------------------------------------------------------------------------------------------- norm

@pytest.mark.parametrize("M,K", [(5, 64), (5, 4096), (200, 5120), (400, 1024), (5, 16448)])
@pytest.mark.parametrize("where", ["all of x", "one of x", "beside zeros", "residual", "weight", "all of weight"])
def test_norm_of_nan(qk, M, K, where):  # noqa: F811
    """max |u| of a row with a NaN is NaN, and so is its scale, as the activation quantization's is: never a
    row of zeros.  The other rows are what they are without it."""
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    r = torch.randn(M, K, generator=g, device="cuda").bfloat16() if where == "residual" else None
    w = 1 + 0.1 * torch.randn(K, generator=g, device="cuda")
    clean = qk.qk_rmsnorm_quantize(x, w, r, with_xsum=True)
    x2, r2, w2 = x.clone(), None if r is None else r.clone(), w.clone()
    rows = [1, M - 2]
    if where == "all of x":
        x2[rows] = NAN
    elif where == "one of x":
        x2[1, 3], x2[M - 2, K - 1] = NAN, -NAN
    elif where == "beside zeros":
        x2[rows] = 0
        x2[rows, K // 2] = NAN
    elif where == "residual":
        r2[1, 0], r2[M - 2, K - 1] = INF, NAN
        x2[1, 0] = -INF
    else:
        w2[K - 5 if where == "weight" else slice(None)] = NAN
        rows = list(range(M))
    h, xq, sx, xsum = qk.qk_rmsnorm_quantize(x2, w2, r2, with_xsum=True)
    assert torch.isnan(sx[rows]).all()
    keep = [m for m in range(M) if m not in rows]
    for a, b in zip((xq, sx, xsum), clean[1:]):
        assert torch.equal(a[keep], b[keep])


# ------------------------------------------------------------------------------- lengths and row bounds

@pytest.mark.parametrize("rows", [[2, 1, 3], [100, 90, 120]])
def test_requests_out_of_range_are_skipped(qk, rows):  # noqa: F811
    """A request whose length or row bounds are out of range appends nothing, comes back as zeros and sees no
    key: none of its rows is taken for a row of another position."""
    D, Hkv = 64, 32
    c = Batch(qk, [300, 200, 260], rows, Hkv, D, 16, wide=2)
    most = c.table.shape[1] * c.page
    a, b, e, T = c.first[0], c.first[1], c.first[2], c.T
    q = c.q(Hkv)
    k, v = (c.randn(T, Hkv, D).bfloat16() for _ in range(2))
    cases = [(i32([300, 200, n]), c.cu, e, T) for n in (most + 1, most + rows[2], 2 ** 31 - 1, -1, -2 ** 31)]
    cases += [(c.lens, i32([a, b, e, T + n]), e, T) for n in (1, 50, 2 ** 30)]
    cases += [(c.lens, i32([-1, b, e, T]), a, b), (c.lens, i32([-2 ** 31, b, e, T]), a, b)]
    for lens, cu, at, end in cases:
        cache = c.cache.clone()
        qk.qk_kv4_append(k, v, cache, c.table, lens, cu)
        with pytest.raises(qk.QKError) as err:
            qk.qk_check_device_error()
        assert err.value.status == INDEX
        # only the other requests' tokens are written
        want = c.cache.clone()
        other = [i for i in range(3) if c.first[i] != at]
        for i in other:
            s = slice(c.first[i], c.first[i + 1])
            qk.qk_kv4_append(k[s].contiguous(), v[s].contiguous(), want,
                             c.table[i:i + 1].clone(), c.lens[i:i + 1].clone())
        qk.qk_check_device_error()
        assert torch.equal(cache, want)
        gk, gv = qk.qk_kv4_gather(want, c.table, lens, cu, T)
        out = torch.full_like(q, 7.0)
        qk.qk_kv4_attention(q, c.cache, c.table, lens, cu, out=out)
        with pytest.raises(qk.QKError) as err:
            qk.qk_check_device_error()
        assert err.value.status == INDEX
        assert not gk[at:end].any() and not gv[at:end].any() and not out[at:end].any()
        c.check(q, out, requests=other)
        for i in other:
            assert gk[c.first[i]:c.first[i + 1]].any()


# ------------------------------------------------------------------------------------- sizes of queries

# requests, rows of each: few rows; tiles of 128 rows (16 kv heads, 1 query head)
FEW, MANY = ([100, 17], [3, 1]), ([150] * 6, [100] * 6)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", [FEW, MANY])
@pytest.mark.parametrize("power", [104, 113, 117, 121, 124])
def test_largest_queries(qk, D, shape, power):  # noqa: F811
    """Rows up to the largest bf16 values, with the scale that brings the scores back (elements of 2^126 and
    more: neither the rows' sums nor the scores' factor may leave fp32 on the way)."""
    c = Batch(qk, *shape, 16, D, 16, seed=power)
    q = (c.randn(c.T, 16, D).clamp(-4, 4) * 2.0 ** power).bfloat16()
    q[:, 1] = q[:, 1].abs()  # (a row's sum: up to 2^130)
    scale = D ** -0.5 * 2.0 ** -power
    out = qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu, scale=scale)
    # the scale itself comes as fp32, below 2^-126 with fewer bits
    c.check(q, out, scale=float(np.float32(scale)))
    qk.qk_check_device_error()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", [FEW, MANY])
def test_scores_of_any_size(qk, D, shape):  # noqa: F811
    """Scores up to 2^26 (in units of log2) pick the key that is largest; a row with larger ones is NaN, and
    never the zeros of a row that sees nothing."""
    c = Batch(qk, *shape, 16, D, 16, fill=False)
    total = sum(c.lens_list)
    # key j of a request: -1 everywhere but in dim j % D, which is 1 (every value exact: offset -1, scale 2/15)
    at = torch.cat([torch.arange(n, device="cuda") for n in c.lens_list]) % D
    k = torch.full((total, 16, D), -1.0, device="cuda")
    k[torch.arange(total, device="cuda"), :, at] = 1.0
    v = torch.randn(total, 16, D, generator=c.g, device="cuda").bfloat16()
    qk.qk_kv4_append(k.bfloat16(), v, c.cache, c.table, c.lens, i32(np.concatenate([[0], np.cumsum(c.lens_list)])))
    qk.qk_check_device_error()
    # a query of one dim: a score of +q where the key's dim is that one, -q elsewhere
    dim = 3
    for power in (10, 20, 24, 25, 27, 40, 80, 120, 127):
        q = torch.zeros(c.T, 16, D, device="cuda")
        q[:, :, dim] = 1.0
        q[:, 1, dim] = 2.0 ** power  # (only this head's scores are large)
        out = qk.qk_kv4_attention(q.bfloat16(), c.cache, c.table, c.lens, c.cu, scale=1.0)
        qk.qk_check_device_error()
        for b, (n, L) in enumerate(zip(c.rows_list, c.lens_list)):
            kk, vv = ref.request_kv(c.cache, c.table[b], L, D)
            got = out[c.first[b]:c.first[b] + n].double()
            want, tol = ref.attention(torch.ones(n, 16, D, device="cuda") * (torch.arange(D, device="cuda") == dim),
                                      kk, vv, 1.0, 0, 0)
            rest = [h for h in range(16) if h != 1]
            assert ((got - want).abs() <= tol)[:, rest].all()
            if power >= 27:
                assert torch.isnan(got[:, 1]).all(), power
                continue
            # the keys of dim `dim` that a row sees, alike; a row that sees none: all of its keys alike
            key = torch.arange(L, device="cuda")
            see = key[None] <= torch.arange(L - n, L, device="cuda")[:, None]
            picked = see & (key % D == dim)[None]
            p = torch.where(picked.any(1, keepdim=True), picked, see).double()
            w = (p / p.sum(1, keepdim=True)) @ vv[:, 1]
            # bf16's rounding, and weight x scale in fp16: 15 scales are within twice the largest value
            bound = 2.0 ** -8 * w.abs() + (2.0 ** -11 + 2.0 ** -18) * 2 * vv.abs().amax()
            assert ((got[:, 1] - w).abs() <= bound).all(), power


# ---------------------------------------------------------------------------------------- every key counts

@pytest.mark.parametrize("lens,rows,Hkv,G,D", [
    ([20000], [1], 2, 4, 128),            # one request over every block
    ([20000], [1], 1, 12, 64),            # and with two row tiles to an item
    ([9000, 30, 14000], [1, 1, 1], 1, 8, 64),
    ([300], [300], 4, 4, 128),
    ([2100, 40], [700, 40], 2, 3, 64),
    ([777] * 40, [1] * 40, 8, 5, 128),
    ([3000] + [1, 17] * 60, [1] + [1, 1] * 60, 2, 8, 128),
    # in tiles of 128 rows
    ([2000], [2000], 4, 3, 64),
    ([5000, 70], [600, 70], 8, 4, 128),
    ([20000, 30], [4, 30], 8, 64, 128),
    ([700] + [0] * 6, [700] + [0] * 6, 16, 2, 128),
])
def test_every_record_counts(qk, lens, rows, Hkv, G, D):  # noqa: F811
    """Values of 15 in one dim each, which runs through the records, and 0 elsewhere: an output is a sum of
    weights without cancellation, so its bound is relative to it, and leaving out any record breaks it."""
    c = Batch(qk, lens, rows, Hkv, D, 32, fill=False, seed=len(lens))
    total = sum(lens)
    k = c.randn(total, Hkv, D).bfloat16()
    rec = torch.cat([torch.arange(n, device="cuda") // 16 for n in lens])
    v = torch.zeros(total, Hkv, D, device="cuda")
    v[torch.arange(total, device="cuda"), :, rec % D] = 15.0
    qk.qk_kv4_append(k, v.bfloat16(), c.cache, c.table, c.lens, i32(np.concatenate([[0], np.cumsum(lens)])))
    q = (c.randn(c.T, Hkv * G, D) * 0.3).bfloat16()
    out = qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu)
    qk.qk_check_device_error()
    for b in range(0, len(lens), max(1, len(lens) // 20)):
        n, L = rows[b], lens[b]
        if n == 0:
            continue
        kk, vv = ref.request_kv(c.cache, c.table[b], L, D)
        assert ((vv == 15) | (vv == 0)).all()  # scale 1, code 15; a group of zeros has scale 0
        qb = q[c.first[b]:c.first[b] + n]
        want, _ = ref.attention(qb, kk, vv, D ** -0.5, 0, 0)
        got = out[c.first[b]:c.first[b] + n].double()
        # all terms are >= 0 and each is off by relative amounts: half a step of bf16 2^-8; half a step 2^-11 of
        # fp16 in the weights; the scores' 2^-17 a (as in block_reference.attention; a: scale times the largest
        # sum |q| (|code scale| + |offset|), within 3 |k|), in the weights and in their sum; 2^x and the sum of
        # weights 2^-20; two fp32 roundings per 16 keys and 400 for the joins, above and below
        a = 3 * D ** -0.5 * (qb.double().abs().sum(-1).amax() * kk.abs().amax()).item()
        rel = 2.0 ** -8 + 2.0 ** -11 + 4 * a * 2.0 ** -17 + 2.0 ** -19 + 2 * (2 * (L / 16) + 400) * 2.0 ** -24
        assert rel < 0.011
        assert ((got - want).abs() <= rel * want).all(), b
        # without record r its dim keeps 1 - s / B of its sum B, and everything grows by 1 / (1 - s)
        x = torch.einsum("hd,jhd->hj", qb[-1].double(), kk.repeat_interleave(G, 1)) * D ** -0.5
        p = torch.softmax(x, 1)
        R = -(-L // 16)
        share = torch.zeros(Hkv * G, R, dtype=torch.float64, device="cuda")
        share.index_add_(1, torch.arange(L, device="cuda") // 16, p)
        dim = torch.zeros(Hkv * G, D, dtype=torch.float64, device="cuda")
        dim.index_add_(1, torch.arange(R, device="cuda") % D, share)
        if R > 1:
            left = (1 - share / dim[:, torch.arange(R, device="cuda") % D]) / (1 - share)
            other = 1 / (1 - share)  # (of a dim with other records only)
            assert (torch.maximum((left - 1).abs(), (other - 1).abs()) > 2 * rel).any(0).all(), b


# ------------------------------------------------------------------------------ other threads and streams

def step_calls(qk):  # noqa: F811
    """The calls of a step on small inputs, each returning its new outputs."""
    r = lambda *s: torch.randn(*s, device="cuda").bfloat16()  # noqa: E731
    x, q, k = r(4, 256), r(4, 8, 64), r(4, 2, 64)
    pos, table, lens = i32([0, 1, 2, 3]), i32([[0], [1], [2], [3]]), i32([1, 1, 1, 1])
    cache = torch.zeros(4, 2, 16, 72, dtype=torch.uint8, device="cuda")
    freq = qk.qk_rope_frequencies(64)
    out = torch.empty_like(q)
    ws = torch.empty(qk.qk_kv4_attention_workspace_size(64), dtype=torch.uint8, device="cuda")
    return {
        "norm": lambda **o: qk.qk_rmsnorm_quantize(x, None, x, with_xsum=True, **o),
        "rope": lambda **o: qk.qk_rope(q, k, pos, freq, **o),
        "append": lambda **o: qk.qk_kv4_append(k, k, cache, table, lens, **o),
        "gather": lambda **o: qk.qk_kv4_gather(cache, table, lens, None, 4, **o),
        "attention": lambda **o: qk.qk_kv4_attention(q, cache, table, lens, out=out, workspace=ws, **o),
    }


@pytest.mark.parametrize("name", ["norm", "rope", "append", "gather", "attention"])
def test_other_threads_run_while_a_call_waits(qk, name):  # noqa: F811
    """A call that waits for room in the launch queue does not hold the interpreter's lock."""
    call = step_calls(qk)[name]
    call()
    torch.cuda.synchronize()
    ticks, stop = [], threading.Event()

    def tick():
        while not stop.is_set():
            ticks.append(time.perf_counter())
            time.sleep(0.002)

    t = threading.Thread(target=tick)
    t.start()
    try:
        torch.cuda._sleep(800_000_000)  # 0.4 s and more, behind which the launches pile up
        longest = (0.0, 0.0, 0.0)
        for _ in range(4000):
            a = time.perf_counter()
            call()
            b = time.perf_counter()
            longest = max(longest, (b - a, a, b))
            if b - a > 0.1:
                break
    finally:
        torch.cuda.synchronize()
        stop.set()
        t.join()
    took, a, b = longest
    assert took > 0.1, "the queue was never full"
    inside = [a] + [x for x in ticks if a < x < b] + [b]
    assert max(y - x for x, y in zip(inside, inside[1:])) < took / 2
    qk.qk_check_device_error()


def test_new_outputs_on_another_stream(qk):  # noqa: F811
    """A call on a stream that is not the current one takes its new outputs from that stream's memory: what the
    current stream has queued may still read memory that is free to Python."""
    g = torch.Generator(device="cuda").manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    M, K, N = 512, 1024, 1024
    x, w = r(M, K).bfloat16(), r(N, K)
    q, k = r(M, 8, 64).bfloat16(), r(M, 2, 64).bfloat16()
    pos = torch.arange(M, dtype=torch.int32, device="cuda")
    table, lens = torch.arange(32, dtype=torch.int32, device="cuda").view(1, 32), i32([M])
    cache = torch.zeros(32, 2, 16, 72, dtype=torch.uint8, device="cuda")
    qk.qk_kv4_append(k, k, cache, table, lens)
    freq = qk.qk_rope_frequencies(64)
    W8, s8 = qk.qk_quantize_weights_int8(w)
    W4, s4, o4 = qk.qk_quantize_weights_int4(w)
    planes, _ = qk.qk_w4a8_prepare(W4, s4, o4)
    xq, sx, xsum = qk.qk_quantize_activations(x, with_xsum=True)
    bias, heads = r(N), r(1, 4, 128, 128).bfloat16()
    calls = {
        "weights8": lambda **o: qk.qk_quantize_weights_int8(w, **o),
        "weights4": lambda **o: qk.qk_quantize_weights_int4(w, **o),
        "activations": lambda **o: qk.qk_quantize_activations(x, with_xsum=True, **o),
        "w8a8": lambda **o: qk.qk_w8a8_linear(x, W8, s8, **o),
        "w8a8 fused": lambda **o: qk.qk_w8a8_linear(x, W8, s8, fused=True, **o),
        "w8a8 gated": lambda **o: qk.qk_w8a8_linear_gated(x, W8, s8, bias, bias, x, **o),
        "w8a8 gemm": lambda **o: qk.qk_w8a8_gemm(xq, sx, W8, s8, **o),
        "w8a8 noalloc": lambda **o: qk.qk_w8a8_linear_noalloc(x, W8, s8, **o),
        "w4a8": lambda **o: qk.qk_w4a8_linear(x, W4, s4, o4, **o),
        "w4a8 gemm": lambda **o: qk.qk_w4a8_gemm(xq, sx, xsum, W4, s4, o4, **o),
        "w4a8 prepare": lambda **o: qk.qk_w4a8_prepare(W4, s4, o4, **o)[0],
        "w4a8 prepared": lambda **o: qk.qk_w4a8_linear_prepared(x, W4, s4, o4, planes, **o),
        "w4a8 gemm prepared": lambda **o: qk.qk_w4a8_gemm_prepared(xq, sx, xsum, W4, s4, o4, planes, **o),
        "sage": lambda **o: qk.qk_sage_attention(heads, heads, heads, **o),
        "acc8": lambda **o: qk.qk_debug_w8a8_acc(xq, W8, **o),
        "acc4": lambda **o: qk.qk_debug_w4a8_group_acc(xq, W4, 0, 8, qk.QK_ROUTE_GEMM, **o),
        "norm": lambda **o: qk.qk_rmsnorm_quantize(x, None, x, with_xsum=True, **o),
        "frequencies": lambda **o: qk.qk_rope_frequencies(64, **o),
        "rope": lambda **o: qk.qk_rope(q, k, pos, freq, **o),
        "gather": lambda **o: qk.qk_kv4_gather(cache, table, lens, None, M, **o),
        "attention": lambda **o: qk.qk_kv4_attention(q, cache, table, lens, **o),
    }
    tensors = lambda out: [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]  # noqa: E731
    side = torch.cuda.Stream()
    for name, call in calls.items():
        for stream in (side, side.cuda_stream):
            want = tensors(call())
            torch.cuda.synchronize()
            torch.cuda.empty_cache()
            # memory of the sizes that the call may ask for, free to Python, read by the current stream later
            storages = {t.untyped_storage().data_ptr(): t.untyped_storage().nbytes() for t in want}
            side.wait_stream(torch.cuda.current_stream())
            old = [torch.full((n,), 77, dtype=torch.uint8, device="cuda") for n in storages.values() for _ in range(3)]
            old += [torch.full((t.nbytes,), 77, dtype=torch.uint8, device="cuda") for t in want]
            side.wait_stream(torch.cuda.current_stream())
            torch.cuda._sleep(20_000_000)
            late = [t.clone() for t in old]
            spans = [(t.data_ptr(), t.data_ptr() + t.nbytes) for t in old]
            del old
            got = tensors(call(stream=stream))
            for t in got:
                assert not any(a < t.data_ptr() + t.nbytes and t.data_ptr() < e for a, e in spans), name
            torch.cuda.synchronize()
            assert all((t == 77).all() for t in late), name
            if name != "w4a8 prepare":  # (planes that the weight does not need are not written)
                assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want)), name
            del got, late
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    qk.qk_check_device_error()


# --------------------------------------------------------------------------------------- one row, none

def test_an_empty_batch(qk):  # noqa: F811
    """No requests and no rows, with and without row bounds: nothing to do, and no refusal."""
    cache = torch.zeros(4, 2, 16, 72, dtype=torch.uint8, device="cuda")
    table = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    lens = torch.empty(0, dtype=torch.int32, device="cuda")
    k, q = (torch.empty(0, h, 64, dtype=torch.bfloat16, device="cuda") for h in (2, 8))
    for cu in (None, i32([0])):
        qk.qk_kv4_append(k, k, cache, table, lens, cu)
        assert qk.qk_kv4_attention(q, cache, table, lens, cu).shape == (0, 8, 64)
        assert [t.shape for t in qk.qk_kv4_gather(cache, table, lens, cu, 0)] == [(0, 2, 64)] * 2
    with pytest.raises(ValueError):  # rows of no request
        qk.qk_kv4_attention(torch.zeros(3, 8, 64, dtype=torch.bfloat16, device="cuda"), cache, table, lens)
    assert not cache.any()
    qk.qk_check_device_error()


@pytest.mark.parametrize("wide", [4, 2052, -3])
def test_the_stride_of_one_row(qk, wide):  # noqa: F811
    """A single row's distance to the next one means nothing, whatever its view says."""
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    odd = lambda t: t.as_strided(t.shape, (t.shape[1] * 64 + wide if wide > 0 else 5, 64, 1))  # noqa: E731
    q, k, v = r(1, 8, 64), r(1, 2, 64), r(1, 2, 64)
    pos, freq, table, lens = i32([7]), qk.qk_rope_frequencies(64), i32([[1]]), i32([1])
    caches = [torch.zeros(2, 2, 16, 72, dtype=torch.uint8, device="cuda") for _ in range(2)]
    want, got = [], []
    for view, cache, out in ((lambda t: t, caches[0], want), (odd, caches[1], got)):
        a, b = qk.qk_rope(view(q), view(k), pos, freq)
        qk.qk_kv4_append(view(b), view(v), cache, table, lens)
        out += [a, b, qk.qk_kv4_attention(view(a), cache, table, lens)]
        into = torch.empty_like(k), torch.empty_like(k)
        qk.qk_kv4_gather(cache, table, lens, None, 1, k=view(into[0]), v=view(into[1]))
        here = q.clone()
        qk.qk_rope(view(here), None, pos, freq, q_out=view(here))
        out += [*into, here]
    assert all(torch.equal(bits(x), bits(y)) for x, y in zip(want, got)) and torch.equal(*caches)
    qk.qk_check_device_error()
