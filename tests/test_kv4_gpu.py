"""GPU parity of the 4-bit paged cache and its attention against their formulas in 64 bits, and the
ways they are called: ragged and padded batches, bad indices, graphs, streams, a block's run."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests import block_reference as ref
from tests.gpu_common import qk  # noqa: F401

pytestmark = pytest.mark.gpu

INDEX = 8  # QK_ERR_INDEX


def bits(t):
    return t.contiguous().view(torch.int16)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Batch:
    """Requests of given lengths and new rows in a cache whose unused bytes (unused pages, tokens
    behind the lengths) hold NaN scales; `front`, `behind`: rows that belong to nobody."""

    def __init__(self, qk, lens, rows, Hkv, D, page, seed=0, front=0, behind=0, wide=0, fill=True):
        self.qk, self.Hkv, self.D, self.page = qk, Hkv, D, page
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        r = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        self.P = sum(need) + 3
        order = r.permutation(self.P)
        wide = max(max(need, default=1), 1) + wide
        table = np.full((len(lens), wide), -7, np.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.lens_list, self.rows_list = list(lens), list(rows)
        self.table, self.lens = i32(table), i32(lens)
        self.cu = i32(np.concatenate([[0], np.cumsum(rows)]) + front)
        self.first = front + np.concatenate([[0], np.cumsum(rows)])
        self.T = front + sum(rows) + behind
        self.cache = torch.full((self.P, Hkv, page, D + D // 8), 0xFF, dtype=torch.uint8, device="cuda")
        if fill:
            self.fill()

    def randn(self, *s):
        return torch.randn(*s, generator=self.g, device="cuda")

    def fill(self):
        """Every token of every request, appended."""
        total = sum(self.lens_list)
        if total == 0:
            return
        loud = 1 + 4 * (torch.rand(1, self.Hkv, self.D, generator=self.g, device="cuda") < 0.05)
        self.k = (self.randn(total, self.Hkv, self.D) * loud + self.randn(1, self.Hkv, self.D)).bfloat16()
        self.v = self.randn(total, self.Hkv, self.D).bfloat16()
        all_rows = i32(np.concatenate([[0], np.cumsum(self.lens_list)]))
        self.qk.qk_kv4_append(self.k, self.v, self.cache, self.table, self.lens, all_rows)

    def q(self, H):
        return (self.randn(self.T, H, self.D) * 1.5).bfloat16()

    def check(self, q, out, scale=None, window=0, sinks=0, requests=None):
        scale = self.D ** -0.5 if scale is None else scale
        for b in range(len(self.lens_list)) if requests is None else requests:
            n, L = self.rows_list[b], self.lens_list[b]
            if n == 0:
                continue
            k, v = ref.request_kv(self.cache, self.table[b], L, self.D)
            a, e = self.first[b], self.first[b] + n
            want, tol = ref.attention(q[a:e], k, v, scale, window, sinks)
            got = out[a:e].double()
            worst = ((got - want).abs() - tol).max().item()
            assert not torch.isnan(got).any() and worst <= 0, (b, worst)


# ------------------------------------------------------------------------------------------------- cache

@pytest.mark.parametrize("D,Hkv,page", [(128, 8, 16), (128, 3, 64), (64, 4, 32), (64, 1, 48), (128, 1, 1024)])
def test_append_and_gather(qk, D, Hkv, page):  # noqa: F811
    """Values come back as the 4-bit rule says, bit for bit; the record's bytes are the documented ones;
    no other byte changes."""
    lens, rows = [1, 16, 33, 17, 70, 5], [1, 4, 33, 0, 21, 5]
    c = Batch(qk, lens, rows, Hkv, D, page, seed=D + page, front=2, behind=3, wide=2, fill=False)
    qkv = c.randn(c.T, 2 * Hkv * D + 8).bfloat16()
    k, v = qkv[:, :Hkv * D].view(c.T, Hkv, D), qkv[:, Hkv * D:2 * Hkv * D].view(c.T, Hkv, D)
    k[3] = 0.75                    # constant groups: scale 0
    k[5, :, :64] = 0
    v[4, :, 0] = 300.0
    qk.qk_kv4_append(k, v, c.cache, c.table, c.lens, c.cu)
    ko = torch.full((c.T, Hkv, D), 9.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    qk.qk_kv4_gather(c.cache, c.table, c.lens, c.cu, c.T, k=ko, v=vo)
    qk.qk_check_device_error()
    mine = torch.zeros(c.T, dtype=torch.bool, device="cuda")
    mine[2:c.T - 3] = True
    for x, y in ((k, ko), (v, vo)):
        value = ref.quantize4(x)[0]
        want = value.to(torch.float32).to(torch.bfloat16)
        assert torch.equal(bits(y[mine]), bits(want[mine]))
        assert (y[~mine] == 9).all()
    # the documented bytes: decode the records of every request, and count what was touched
    touched = torch.zeros(c.P, Hkv, page, dtype=torch.bool, device="cuda")
    for b, (L, n) in enumerate(zip(lens, rows)):
        if n == 0:
            continue
        got = ref.request_kv(c.cache, c.table[b], L, D)
        for x, y in ((k, got[0]), (v, got[1])):
            assert torch.equal(y[L - n:], ref.quantize4(x[c.first[b]:c.first[b] + n])[0])
        p = torch.arange(L - n, L, device="cuda")
        touched[c.table[b].long()[p // page], :, p % page] = True
    kb, vb, shift = ref.record_places(D)
    rec = c.cache.view(-1, 18 * D)
    flags = touched.view(-1, 16)
    for byte in (kb, vb):
        nib = (rec[:, byte.cuda()] >> shift.cuda().to(torch.uint8)) & 15
        assert (nib[~flags] == 15).all()
    sc = rec[:, 16 * D:].view(-1, 2, 16, D // 16)
    assert (sc.transpose(1, 2)[~flags] == 0xFF).all()


def test_append_uniform_rows_and_long_requests(qk):  # noqa: F811
    """Without row bounds every request has T / B rows; a request over many blocks; 200 requests."""
    c = Batch(qk, [40] * 200, [3] * 200, 2, 64, 16, fill=False)
    k, v = c.randn(c.T, 2, 64).bfloat16(), c.randn(c.T, 2, 64).bfloat16()
    qk.qk_kv4_append(k, v, c.cache, c.table, c.lens)
    for got, x in zip(qk.qk_kv4_gather(c.cache, c.table, c.lens, None, c.T), (k, v)):
        assert torch.equal(bits(got), bits(ref.quantize4(x)[0].float().bfloat16()))
    c = Batch(qk, [5000, 0, 1, 2500], [5000, 0, 1, 2500], 1, 128, 32)
    for got, x in zip(qk.qk_kv4_gather(c.cache, c.table, c.lens, c.cu, c.T), (c.k, c.v)):
        assert torch.equal(bits(got), bits(ref.quantize4(x)[0].float().bfloat16()))
    qk.qk_check_device_error()


@pytest.mark.parametrize("B", [1, 31, 32, 33, 34, 1000, 1025])
def test_row_bounds_of_many_requests(qk, B):  # noqa: F811
    """The search over the row bounds, with empty requests among them."""
    rows = np.random.default_rng(B).integers(0, 3, B).tolist()
    rows[-1] = 1
    c = Batch(qk, [n + 1 for n in rows], rows, 1, 64, 16, seed=B, front=1, behind=2, fill=False)
    k, v = c.randn(c.T, 1, 64).bfloat16(), c.randn(c.T, 1, 64).bfloat16()
    qk.qk_kv4_append(k, v, c.cache, c.table, c.lens, c.cu)
    for b in range(B):
        if rows[b]:
            got = ref.request_kv(c.cache, c.table[b], rows[b] + 1, 64)[0][1:]
            assert torch.equal(got, ref.quantize4(k[c.first[b]:c.first[b + 1]])[0]), b
    qk.qk_check_device_error()


# --------------------------------------------------------------------------------------------- attention

LENS = [1, 15, 16, 17, 200, 0, 33, 1000, 64, 31]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,Hkv", [(1, 4), (2, 1), (3, 2), (4, 8), (5, 2), (7, 1), (8, 2), (12, 1), (16, 2), (20, 1), (32, 1)])
def test_decode_heads(qk, D, G, Hkv):  # noqa: F811
    """One row per request (none where the length is 0), every grouping of the heads."""
    c = Batch(qk, LENS, [min(1, n) for n in LENS], Hkv, D, 32, seed=G, front=1, behind=2)
    q = c.q(G * Hkv)
    out = torch.full((c.T, G * Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu, out=out)
    c.check(q, out)
    assert (out[0] == 7).all() and (out[c.first[-1]:] == 7).all()
    qk.qk_check_device_error()


@pytest.mark.parametrize("D,G,page", [(128, 4, 16), (64, 2, 64), (128, 1, 128), (64, 8, 48), (128, 3, 1024)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (5, 4), (16, 1), (40, 40), (300, 17), (100000, 3)])
def test_few_rows_and_windows(qk, D, G, page, window, sinks):  # noqa: F811
    """Several rows per request, whole prompts among them (rows == length)."""
    lens = [1, 7, 16, 45, 130, 700, 33, 260]
    rows = [1, 7, 3, 45, 9, 6, 1, 2]
    c = Batch(qk, lens, rows, 2, D, page, seed=window + G)
    q = c.q(2 * G)
    out = qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu, window=window, sinks=sinks)
    c.check(q, out, window=window, sinks=sinks)
    qk.qk_check_device_error()


@pytest.mark.parametrize("lens,rows,Hkv,G,D", [
    ([20000], [1], 2, 4, 128),            # one request over every block
    ([16], [1], 1, 1, 128),               # one record
    ([5000, 16, 16, 3000], [1, 1, 1, 1], 1, 8, 64),
    ([300], [300], 4, 4, 128),            # a prompt
    ([2100, 40], [700, 40], 2, 3, 64),    # a chunk of a prompt
    ([100] * 300, [1] * 300, 2, 2, 64),   # more requests than threads / 2
    ([40] * 700, [2] * 700, 1, 1, 128),   # more requests than threads
    ([777] * 40, [1] * 40, 8, 5, 128),
    ([40] * 600, [16] * 600, 1, 1, 128),  # two tiles of rows, several requests to a thread
    ([50] * 800, [12] * 800, 1, 2, 64),
    ([16] * 500, [1] * 500, 4, 8, 64),    # items of one record, many to a warp
    ([3000] + [0, 1, 17] * 60, [1] + [0, 1, 1] * 60, 2, 8, 128),
])
def test_spans(qk, lens, rows, Hkv, G, D):  # noqa: F811
    """Items cut within warps, blocks and between blocks; the same bits on a second run."""
    c = Batch(qk, lens, rows, Hkv, D, 16, seed=len(lens))
    q = c.q(Hkv * G)
    out = qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu)
    c.check(q, out, requests=range(0, len(lens), max(1, len(lens) // 40)))
    again = qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu)
    assert torch.equal(bits(out), bits(again))
    qk.qk_check_device_error()


@pytest.mark.parametrize("seed", range(12))
def test_drawn_batches(qk, seed):  # noqa: F811
    r = np.random.default_rng(100 + seed)
    B, D, page = int(r.integers(1, 30)), int(r.choice([64, 128])), int(r.choice([16, 32, 80, 256]))
    Hkv, G = int(r.choice([1, 2, 4])), int(r.integers(1, 18))
    lens = np.exp(r.uniform(0, np.log(3000), B)).astype(int).tolist()
    rows = [int(r.integers(0, min(n, 40) + 1)) for n in lens]
    rows[0] = 1
    window = int(r.choice([0, r.integers(1, 3000)]))
    sinks = int(r.integers(0, 200))
    c = Batch(qk, lens, rows, Hkv, D, page, seed=seed, front=int(r.integers(0, 3)), behind=int(r.integers(0, 3)))
    q = c.q(Hkv * G)
    scale = float(r.choice([D ** -0.5, 0.0, 0.02, 1.0]))
    out = qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu, scale=scale, window=window, sinks=sinks)
    c.check(q, out, scale=scale, window=window, sinks=sinks)
    qk.qk_check_device_error()


def test_rows_that_see_nothing(qk):  # noqa: F811
    """More rows than tokens: the rows in front of the first token, and an empty request's, are 0."""
    c = Batch(qk, [3, 0, 20], [5, 2, 20], 2, 64, 16)
    q = c.q(4)
    out = torch.full((c.T, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu, out=out)
    assert not out[:2].any() and not out[5:7].any()
    k, v = ref.request_kv(c.cache, c.table[0], 3, 64)
    want, tol = ref.attention(q[2:5], k, v, 0.125, 0, 0)
    assert ((out[2:5].double() - want).abs() <= tol).all()
    c.check(q, out, requests=[2])
    qk.qk_check_device_error()


def test_closed_forms(qk):  # noqa: F811
    """One key returns its value; scale 0 the mean; a window of 1 the row's own value; the sink case:
    a first key of almost all the weight and no value, the others' share keeps its precision."""
    c = Batch(qk, [1, 50], [1, 50], 1, 128, 16, seed=4)
    q = c.q(2)
    one = qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu, window=1)
    for b in range(2):
        _, v = ref.request_kv(c.cache, c.table[b], c.lens_list[b], 128)
        got = one[c.first[b]:c.first[b + 1]].double()
        assert ((got - v).abs() <= 2.0 ** -8 * v.abs() + 2.0 ** -14 * v.abs().max()).all()
    mean = qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu, scale=0.0)
    _, v = ref.request_kv(c.cache, c.table[1], 50, 128)
    want = v[:, 0].cumsum(0) / torch.arange(1, 51, device="cuda")[:, None]
    got = mean[1:51, 0].double()
    assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -14 * v.abs().max()).all()

    c = Batch(qk, [4000], [1], 1, 64, 16, fill=False)
    k, v = 0.1 * c.randn(4000, 1, 64), c.randn(4000, 1, 64)
    k[0], v[0] = 3.0, 0.0
    k[0, 0, 0] = 2.0
    qk.qk_kv4_append(k.bfloat16(), v.bfloat16(), c.cache, c.table, c.lens, i32([0, 4000]))
    q = torch.ones(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    out = qk.qk_kv4_attention(q, c.cache, c.table, c.lens)
    kk, vv = ref.request_kv(c.cache, c.table[0], 4000, 64)
    p = torch.softmax((kk[:, 0] @ q[0, 0].double()) / 8, 0)
    assert p[0] > 0.999
    want = p @ vv[:, 0]
    # relative to what the 3999 others add up to in absolute value, not to the largest value
    part = p @ vv[:, 0].abs()
    assert ((out[0, 0].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10 * part).all()


@pytest.mark.parametrize("D,G", [(64, 1), (128, 3), (128, 12)])
def test_value_scales_far_apart(qk, D, G):  # noqa: F811
    """Value scales over fp16's range (as far as the offsets are finite), in every order of size and score, heads of one key
    among them: every output within the rounding of its own sum P scale code."""
    g = torch.Generator(device="cuda").manual_seed(D + G)
    lens = [700, 90, 333]
    n = sum(lens)
    for trend in (-1, 0, 1, 2):
        c = Batch(qk, lens, [1, 2, 1], 2, D, 16, seed=trend + 5, fill=False)
        at = torch.cat([torch.linspace(0, 1, m, device="cuda") for m in lens])
        if trend == 0:
            at = torch.rand(n, generator=g, device="cuda")
        if trend == 2:  # a first token of huge values, then tiny ones
            at = torch.where(at == 0, 1.0, 0.3)
        size = torch.exp2(-20 + 33 * (at if trend >= 0 else 1 - at))[:, None, None]
        v = (torch.randn(n, 2, D, generator=g, device="cuda") * size).bfloat16()
        v[5::7] = 0.0
        k = torch.randn(n, 2, D, generator=g, device="cuda").bfloat16()
        qk.qk_kv4_append(k, v, c.cache, c.table, c.lens, i32([0, 700, 790, 1123]))
        for strength in (0.0, 1.0, 8.0):
            q = (c.randn(c.T, 2 * G, D) * strength).bfloat16()
            out = qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu)
            first = 0
            for b, m in enumerate(lens):
                kk, vv = ref.request_kv(c.cache, c.table[b], m, D)
                _, _, s, o = ref.quantize4(v[first:first + m])
                first += m
                reach = (15 * s + o.abs()).repeat_interleave(64, -1)  # of a key's codes and offset
                rows = q[c.first[b]:c.first[b + 1]]
                want, _ = ref.attention(rows, kk, vv, D ** -0.5, 0, 0)
                part, _ = ref.attention(rows, kk, reach, D ** -0.5, 0, 0)  # sum P (15 scale + |offset|)
                a = 3 * D ** -0.5 * rows.double().abs().sum(-1).amax() * kk.abs().amax()
                # P scale as fp16: 2^-11 of itself, or 2^-25 where the row's largest is at least 2^5: m
                # times 2^-30 of the largest; scores (2^-17 a each way), 2^x, fp32 sums as in ref.attention
                move = 2.0 ** -11 + m * 2.0 ** -30 + 2 * a * 2.0 ** -17 + 2.0 ** -20 + (m / 8 + 400) * 2.0 ** -23
                got = out[c.first[b]:c.first[b + 1]].double()
                assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + part * move).all(), (trend, strength, b)
    qk.qk_check_device_error()


def test_infinite_values_stay_in_their_group(qk):  # noqa: F811
    """A visible token whose value group holds infinities makes that group NaN, and nothing else."""
    c = Batch(qk, [300, 40], [1, 1], 1, 128, 16, seed=3)
    q = c.q(4)
    clean = qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu)
    x = c.randn(1, 1, 128).bfloat16()
    k, v = ref.request_kv(c.cache, c.table[0], 300, 128)
    place = c.table[0, 2:3, None].clone()  # token 37 of request 0, by a table of its own page
    kk = k[37:38].bfloat16()
    vv = v[37:38].bfloat16()
    vv[0, 0, 3] = float("inf")
    vv[0, 0, 64:] = x[0, 0, 64:]
    qk.qk_kv4_append(kk, vv, c.cache, place, i32([6]))
    out = qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu)
    assert torch.equal(bits(out[1]), bits(clean[1]))
    assert torch.isnan(out[0, :, :64]).all()
    k, v = ref.request_kv(c.cache, c.table[0], 300, 128)
    want, tol = ref.attention(q[:1], k, v.nan_to_num(0, 0, 0), 128 ** -0.5, 0, 0)
    assert ((out[0, :, 64:].double() - want[0, :, 64:]).abs() <= tol[0, :, 64:]).all()
    qk.qk_check_device_error()


@pytest.mark.parametrize("D,G", [(64, 2), (128, 4)])
@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -30, 1.0, 2.0 ** 30, 2.0 ** 100])
def test_query_sizes(qk, D, G, size):  # noqa: F811
    """Rows of any magnitude, with the scale that brings the scores back."""
    c = Batch(qk, [100, 17], [3, 1], 2, D, 16, seed=G)
    q = (c.randn(c.T, 2 * G, D) * size).bfloat16()
    scale = min(D ** -0.5 / size, 2.0 ** 98)
    out = qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu, scale=scale)
    c.check(q, out, scale=scale)
    qk.qk_check_device_error()


def test_strided_queries(qk):  # noqa: F811
    c = Batch(qk, [100, 37], [2, 3], 2, 64, 16)
    rows = c.randn(c.T, 6 * 64 + 40).bfloat16()
    q = rows[:, 8:8 + 4 * 64].unflatten(1, (4, 64))
    out = qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu)
    c.check(q, out)


def test_offsets_past_32_bits(qk):  # noqa: F811
    """A cache of over 4 GB whose last pages hold the request."""
    Hkv, D, page = 8, 128, 128
    P = (1 << 32) // (Hkv * page * 144) + 40
    cache = torch.empty(P, Hkv, page, 144, dtype=torch.uint8, device="cuda")
    assert cache.numel() > 1 << 32
    lens = [300, 129]
    g = torch.Generator(device="cuda").manual_seed(0)
    k = torch.randn(429, Hkv, D, generator=g, device="cuda").bfloat16()
    v = torch.randn(429, Hkv, D, generator=g, device="cuda").bfloat16()
    table = i32([[P - 1, 0, P - 3], [P - 4, P - 2, -1]])
    qk.qk_kv4_append(k, v, cache, table, i32(lens), i32([0, 300, 429]))
    got = qk.qk_kv4_gather(cache, table, i32(lens), i32([0, 300, 429]), 429)
    assert torch.equal(bits(got[0]), bits(ref.quantize4(k)[0].float().bfloat16()))
    assert torch.equal(bits(got[1]), bits(ref.quantize4(v)[0].float().bfloat16()))
    q = torch.randn(2, 32, D, generator=g, device="cuda").bfloat16()
    out = qk.qk_kv4_attention(q, cache, table, i32(lens))
    for b in range(2):
        kk, vv = ref.request_kv(cache, table[b], lens[b], D)
        want, tol = ref.attention(q[b:b + 1], kk, vv, D ** -0.5, 0, 0)
        assert ((out[b:b + 1].double() - want).abs() <= tol).all()
    del cache


# ------------------------------------------------------------------------------------------ bad indices

def test_bad_pages_and_lengths(qk):  # noqa: F811
    """What is out of range is skipped and reported; the other requests' results stand."""
    c = Batch(qk, [100, 40, 60], [1, 1, 2], 2, 64, 16, wide=1)
    q = c.q(4)
    good = qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu)
    qk.qk_check_device_error()
    before = c.cache.clone()
    for bad_id in (-1, c.P, 2 ** 31 - 1, -2 ** 31):
        table = c.table.clone()
        table[1, 2] = bad_id
        out = qk.qk_kv4_attention(q, c.cache, table, c.lens, c.cu)
        with pytest.raises(qk.QKError) as e:
            qk.qk_check_device_error()
        assert e.value.status == INDEX
        assert torch.equal(bits(out[0]), bits(good[0])) and torch.equal(bits(out[2:]), bits(good[2:]))
        # request 1 without its last 8 keys
        kk, vv = ref.request_kv(c.cache, c.table[1], 32, 64)
        want, tol = ref.attention(q[1:2], kk, vv, 0.125, 0, 0)
        assert ((out[1:2].double() - want).abs() <= tol).all()
        x = c.randn(c.T, 2, 64).bfloat16()
        cache = c.cache.clone()
        qk.qk_kv4_append(x, x, cache, table, c.lens, c.cu)
        k, _ = qk.qk_kv4_gather(cache, table, c.lens, c.cu, c.T)
        with pytest.raises(qk.QKError):
            qk.qk_check_device_error()
        assert not k[1].any() and k[0].any()
    assert torch.equal(c.cache, before)
    for lens in ([-5, 40, 60], [100, 40, 10 ** 9]):
        out = qk.qk_kv4_attention(q, c.cache, c.table, i32(lens), c.cu)
        with pytest.raises(qk.QKError):
            qk.qk_check_device_error()
        # (the others' lengths move where request 1 is cut, and with it the order of its sums)
        c.check(q, out, requests=[1])
    # row bounds that fall, or leave the rows
    for cu in ([0, 1, 0, 2], [0, 1, 2, 99], [-3, 1, 2, 4]):
        qk.qk_kv4_attention(q, c.cache, c.table, c.lens, i32(cu))
        with pytest.raises(qk.QKError):
            qk.qk_check_device_error()
    # appended rows in front of the first token
    x = c.randn(c.T, 2, 64).bfloat16()
    qk.qk_kv4_append(x, x, c.cache, c.table, i32([100, 40, 1]), c.cu)
    with pytest.raises(qk.QKError):
        qk.qk_check_device_error()
    qk.qk_check_device_error()


@pytest.mark.parametrize("D,G", [(128, 4), (64, 16)])
def test_missing_pages_of_a_long_request(qk, D, G):  # noqa: F811
    """Pages that are not there, first, last, next to each other and alone: their keys are as if
    masked, whatever the first page of the cache holds."""
    n, page = 9000, 16
    c = Batch(qk, [n, 40], [1, 1], 1, D, page, seed=D)
    q = c.q(G)
    gone = sorted({0, 1, 31, 32, 33, 100, 200, 201, 202, 203, 204, 205, 400, (n - 1) // page})
    table = c.table.clone()
    table[0, gone] = i32([-1, c.P] * (len(gone) // 2))
    out = qk.qk_kv4_attention(q, c.cache, table, c.lens, c.cu)
    with pytest.raises(qk.QKError) as e:
        qk.qk_check_device_error()
    assert e.value.status == INDEX
    k, v = ref.request_kv(c.cache, c.table[0], n, D)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    for g in gone:
        keep[page * g:page * g + page] = False
    want, tol = ref.attention(q[:1], k[keep], v[keep], D ** -0.5, 0, 0)
    assert ((out[:1].double() - want).abs() <= tol).all()
    c.check(q, out, requests=[1])


def test_freed_pages_behind_the_window(qk):  # noqa: F811
    """Pages that no row sees may be gone from the table."""
    c = Batch(qk, [500], [2], 2, 64, 16)
    q = c.q(4)
    want = qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu, window=64, sinks=4)
    table = c.table.clone()
    table[0, 1:(498 - 64 + 1) // 16] = -1
    out = qk.qk_kv4_attention(q, c.cache, table, c.lens, c.cu, window=64, sinks=4)
    assert torch.equal(bits(out), bits(want))
    qk.qk_check_device_error()


# --------------------------------------------------------------------------------- graphs, streams, runs

def test_graph_replays_with_new_lengths(qk):  # noqa: F811
    """append + attention captured once: lengths, rows and keys change under the same graph; two graphs
    that share a workspace, replayed in turn."""
    B, Hkv, D, page, wide = 6, 2, 128, 16, 20
    g = torch.Generator(device="cuda").manual_seed(8)
    cache = torch.full((B * wide, Hkv, page, 144), 0xFF, dtype=torch.uint8, device="cuda")
    table = torch.randperm(B * wide, generator=g, device="cuda").int().view(B, wide)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    q = torch.zeros(B, 8, D, dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros(2, B, Hkv, D, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(qk.qk_kv4_attention_workspace_size(D), dtype=torch.uint8, device="cuda")
    out, out2 = torch.empty_like(q), torch.empty_like(q)

    def step(o, window):
        qk.qk_kv4_append(kv[0], kv[1], cache, table, lens)
        qk.qk_kv4_attention(q, cache, table, lens, out=o, workspace=ws, window=window)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lens.fill_(1)
        step(out, 0)
    torch.cuda.current_stream().wait_stream(s)
    graph, graph2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out, 0)
    with torch.cuda.graph(graph2):
        step(out2, 30)
    host = torch.tensor([0, 10, 99, 200, 255, 16])
    for _ in range(5):
        host = host + torch.tensor([1, 1, 1, 1, 1, 1])
        lens.copy_(host.int())
        q.copy_(torch.randn(B, 8, D, generator=g, device="cuda").bfloat16())
        kv.copy_(torch.randn(2, B, Hkv, D, generator=g, device="cuda").bfloat16())
        # the tokens in front of the new one: written here, so that every key is real
        for b in range(B):
            n = int(host[b]) - 1
            if n:
                x = torch.randn(n, Hkv, D, generator=g, device="cuda").bfloat16()
                qk.qk_kv4_append(x, x.flip(0), cache, table[b:b + 1].contiguous(), i32([n]))
        graph.replay()
        graph2.replay()
        for o, window in ((out, 0), (out2, 30)):
            for b in range(B):
                kk, vv = ref.request_kv(cache, table[b], int(host[b]), D)
                want, tol = ref.attention(q[b:b + 1], kk, vv, D ** -0.5, window, 0)
                assert ((o[b:b + 1].double() - want).abs() <= tol).all()
    qk.qk_check_device_error()


def test_first_calls_inside_a_capture():
    """A process whose first calls of the library are captured: a step's five calls and the frequencies."""
    code = (
        "import torch\n"
        "from w4a8_quantized_gemm_token_b200 import binding as qk\n"
        "t = lambda v: torch.tensor(v, dtype=torch.int32, device='cuda')\n"
        "r = lambda *s: torch.randn(*s, device='cuda').bfloat16()\n"
        "x, q, k, v = r(4, 256), r(4, 8, 64), r(4, 2, 64), r(4, 2, 64)\n"
        "pos, table, lens = t([0, 1, 2, 3]), t([[0], [1], [2], [3]]), t([1, 1, 1, 1])\n"
        "cache = torch.zeros(4, 2, 16, 72, dtype=torch.uint8, device='cuda')\n"
        "g = torch.cuda.CUDAGraph()\n"
        "with torch.cuda.graph(g):\n"
        "    h, xq, sx, xsum = qk.qk_rmsnorm_quantize(x, None, x, with_xsum=True)\n"
        "    a, b = qk.qk_rope(q, k, pos, qk.qk_rope_frequencies(64))\n"
        "    qk.qk_kv4_append(b, v, cache, table, lens)\n"
        "    o = qk.qk_kv4_attention(a, cache, table, lens)\n"
        "    _, w = qk.qk_kv4_gather(cache, table, lens, None, 4)\n"
        "g.replay()\n"
        "qk.qk_check_device_error()\n"
        "assert torch.equal(h, x + x)\n"
        "d = (o.view(4, 2, 4, 64).float() - w[:, :, None].float()).abs()\n"
        "assert (d <= 2.0 ** -7 * w[:, :, None].float().abs() + 1e-3).all()\n"  # one key: two roundings to bf16
    )
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


def test_two_streams_at_once(qk):  # noqa: F811
    """Two calls in flight with workspaces of their own; no workspace given on another stream."""
    c = Batch(qk, [3000, 2000, 500], [1, 1, 1], 4, 128, 32)
    q1, q2 = c.q(16), c.q(16)
    want1 = qk.qk_kv4_attention(q1, c.cache, c.table, c.lens)
    want2 = qk.qk_kv4_attention(q2, c.cache, c.table, c.lens)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        o1 = qk.qk_kv4_attention(q1, c.cache, c.table, c.lens, stream=a, out=torch.empty_like(want1))
        o2 = qk.qk_kv4_attention(q2, c.cache, c.table, c.lens, stream=b, out=torch.empty_like(want2))
        torch.cuda.synchronize()
        assert torch.equal(bits(o1), bits(want1)) and torch.equal(bits(o2), bits(want2))
    qk.qk_check_device_error()


def test_refusals(qk):  # noqa: F811
    c = Batch(qk, [20, 20], [1, 1], 2, 64, 16)
    q = c.q(4)
    with pytest.raises(ValueError):
        qk.qk_kv4_attention(q, c.cache, c.table, c.lens[:1])
    with pytest.raises(ValueError):
        qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu[:2])
    with pytest.raises(ValueError):
        qk.qk_kv4_attention(q[:1], c.cache, c.table, c.lens)
    with pytest.raises(ValueError):
        qk.qk_kv4_attention(q[..., :32], c.cache, c.table, c.lens)
    with pytest.raises(TypeError):
        qk.qk_kv4_attention(q, c.cache, c.table.long(), c.lens)
    with pytest.raises(qk.QKError):
        qk.qk_kv4_attention(q[:, :3].contiguous(), c.cache, c.table, c.lens)
    with pytest.raises(qk.QKError):
        qk.qk_kv4_attention(q, c.cache, c.table, c.lens, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        qk.qk_kv4_append(q, q, c.cache, c.table, c.lens)
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert qk.qk_kv4_attention(e, c.cache, c.table, c.lens).shape == (0, 4, 64)
    qk.qk_check_device_error()


@pytest.mark.parametrize("tokens", [1, 3])
def test_decode_steps_of_a_block(qk, tokens):  # noqa: F811
    """The calls together, as a transformer block's decode step makes them: norm -> W4A8 projection ->
    rotary in place on the projection's rows -> append -> attention -> W8A8 projection -> norm; each
    against its formula on what the one before it gave."""
    B, K, H, Hkv, D = 5, 512, 8, 2, 64
    g = torch.Generator(device="cuda").manual_seed(tokens)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    Wqkv = qk.qk_quantize_weights_int4(rnd((H + 2 * Hkv) * D, K) * 0.05)
    Wo, so = qk.qk_quantize_weights_int8(rnd(K, H * D) * 0.05)
    w1, w2 = 1 + 0.1 * rnd(K), 1 + 0.1 * rnd(K)
    freq = qk.qk_rope_frequencies(D)
    wide = 8
    cache = torch.full((B * wide, Hkv, 16, D + D // 8), 0xFF, dtype=torch.uint8, device="cuda")
    table = torch.randperm(B * wide, generator=g, device="cuda").int().view(B, wide)
    host = torch.tensor([0, 3, 15, 16, 40])
    for b in range(B):
        if host[b]:
            x = rnd(int(host[b]), Hkv, D).bfloat16()
            qk.qk_kv4_append(x, x, cache, table[b:b + 1].contiguous(), host[b:b + 1].int().cuda())
    stream = rnd(B * tokens, K).bfloat16()
    update = rnd(B * tokens, K).bfloat16()
    for _ in range(4):
        host = host + tokens
        lens = host.int().cuda()
        pos = (host[:, None] - tokens + torch.arange(tokens)).flatten().int().cuda()
        before = stream.clone()
        _, xq, sx, xsum = qk.qk_rmsnorm_quantize(update, w1, stream, h=stream, with_xsum=True)
        hr, cr, _ = ref.rmsnorm_quantize(update, w1, before, 1e-6)
        assert torch.equal(bits(stream), bits(hr)) and torch.equal(xq, cr)
        rows = qk.qk_w4a8_gemm(xq, sx, xsum, *Wqkv)
        q = rows[:, :H * D].view(-1, H, D)
        k = rows[:, H * D:(H + Hkv) * D].view(-1, Hkv, D)
        v = rows[:, (H + Hkv) * D:].view(-1, Hkv, D)
        q0, k0 = q.clone(), k.clone()
        qk.qk_rope(q, k, pos, freq, q_out=q, k_out=k)
        for x0, x in ((q0, q), (k0, k)):
            want = ref.rope(x0, pos, freq, True, 1.0)
            norm = ref.rope(x0.abs(), torch.zeros_like(pos), torch.zeros_like(freq), True, 1.0)
            both = norm[..., :D // 2] + norm[..., D // 2:]
            tol = 2.0 ** -8 * want.abs() + torch.cat((both, both), -1) * 2.0 ** -21
            assert ((x.double() - want).abs() <= tol).all()
        qk.qk_kv4_append(k, v, cache, table, lens)
        out = qk.qk_kv4_attention(q, cache, table, lens)
        for b in range(B):
            kk, vv = ref.request_kv(cache, table[b], int(host[b]), D)
            a = slice(b * tokens, (b + 1) * tokens)
            assert torch.equal(kk[-tokens:], ref.quantize4(k[a])[0])
            want, tol = ref.attention(q[a], kk, vv, D ** -0.5, 0, 0)
            assert ((out[a].double() - want).abs() <= tol).all()
        update = qk.qk_w8a8_linear(out.view(B * tokens, H * D), Wo, so)
        assert torch.isfinite(update.float()).all()
    h, xq, _, _ = qk.qk_rmsnorm_quantize(update, w2, stream)
    hr, cr, _ = ref.rmsnorm_quantize(update, w2, stream, 1e-6)
    assert torch.equal(bits(h), bits(hr)) and torch.equal(xq, cr)
    qk.qk_check_device_error()


@pytest.mark.parametrize("rows", [1, 40])
def test_all_the_weight_on_a_value_of_scale_zero(qk, rows):  # noqa: F811
    """One key has all the weight but 2^-50, and a value group that is constant (scale 0): what the other
    keys add keeps its precision."""
    lens = [300] * 6
    c = Batch(qk, lens, [rows] * 6, 16, 64, 16, fill=False)
    k, v = 0.1 * c.randn(1800, 16, 64), c.randn(1800, 16, 64)
    k[5::300], v[5::300] = 4.5, 0.0
    k[5::300, :, 0] = 3.5
    k, v = k.bfloat16(), v.bfloat16()
    qk.qk_kv4_append(k, v, c.cache, c.table, c.lens, i32(list(range(0, 1801, 300))))
    q = torch.ones(c.T, 48, 64, dtype=torch.bfloat16, device="cuda")
    out = qk.qk_kv4_attention(q, c.cache, c.table, c.lens, c.cu)
    for b in range(6):
        kk, vv = ref.request_kv(c.cache, c.table[b], 300, 64)
        _, _, s, o = ref.quantize4(v[300 * b:300 * b + 300])
        mine = q[c.first[b]:c.first[b + 1]]
        want, _ = ref.attention(mine, kk, vv, 0.125, 0, 0)
        part, _ = ref.attention(mine, kk, (15 * s + o.abs()).repeat_interleave(64, -1), 0.125, 0, 0)
        assert 0 < part.max() < 2.0 ** -40
        a = 3 * 0.125 * 64 * kk.abs().amax()
        # as in test_value_scales_far_apart
        move = 2.0 ** -11 + 300 * 2.0 ** -30 + 2 * a * 2.0 ** -17 + 2.0 ** -20 + 440 * 2.0 ** -23
        got = out[c.first[b]:c.first[b + 1]].double()
        assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + part * move).all()
    qk.qk_check_device_error()
