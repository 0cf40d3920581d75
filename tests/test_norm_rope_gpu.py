"""GPU parity of the quantizing RMS norm and the rotary positions against their formulas in 64 bits."""
import math

import pytest
import torch

from tests import block_reference as ref
from tests.gpu_common import qk  # noqa: F401

pytestmark = pytest.mark.gpu


def bits(t):
    return t.contiguous().view(torch.int16)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def norm_inputs(M, K, seed, loud=True):
    g = gen(seed)
    x = torch.randn(M, K, generator=g, device="cuda") * 0.5
    r = torch.randn(M, K, generator=g, device="cuda")
    if loud:
        r = r * (1 + 19 * (torch.rand(K, generator=g, device="cuda") < 0.02))
    w = 1 + 0.2 * torch.randn(K, generator=g, device="cuda")
    return x.bfloat16(), r.bfloat16(), w


def check_norm(qk, x, r, w, eps, out, with_xsum):
    h, xq, sx, xsum = out
    M, K = x.shape
    hr, cr, sr = ref.rmsnorm_quantize(x, w, r, eps)
    if r is None:
        assert h is None
    else:
        assert torch.equal(bits(h), bits(hr))
    assert torch.equal(xq, cr)
    if with_xsum:
        assert torch.equal(xsum, cr.view(M, K // 64, 64).sum(2).to(torch.int32))
    # a thread adds at most 256 squares (64 up to 16384 elements) one by one, 13 more sums join
    # them; the root halves that; the scale itself has six roundings
    ulps = ((256 if K > 16384 else 64) + 14) / 2 + 6
    assert ((sx.double() - sr).abs() <= ulps * 2.0 ** -24 * sr).all()


@pytest.mark.parametrize("M,K", [(1, 32), (3, 64), (1, 4096), (2, 96), (149, 4096), (300, 96), (300, 288), (170, 608),
                                 (160, 1568), (17, 5120), (200, 5120), (151, 7168), (5, 8192), (160, 12288), (2, 12320),
                                 (3, 16384), (2, 16416), (150, 16448), (2, 65536)])
@pytest.mark.parametrize("residual,weight", [(True, True), (False, True), (True, False)])
def test_norm(qk, M, K, residual, weight):  # noqa: F811
    x, r, w = norm_inputs(M, K, M * 7 + K)
    r, w = (r if residual else None), (w if weight else None)
    sums = K % 64 == 0
    out = qk.qk_rmsnorm_quantize(x, w, r, eps=1e-5, with_xsum=sums)
    check_norm(qk, x, r, w, 1e-5, out, sums)


def test_norm_zero_rows_and_signs(qk):  # noqa: F811
    """A zero row: scale 1 and codes 0 (also where the residual cancels x); +-max codes +-127."""
    x, r, w = norm_inputs(6, 256, 3)
    x[1] = 0
    r[1] = 0
    r[3] = -x[3]
    w[5] = -w[5]
    out = qk.qk_rmsnorm_quantize(x, w, r, with_xsum=True)
    check_norm(qk, x, r, w, 1e-6, out, True)
    assert out[2][1] == 1 and out[2][3] == 1 and not out[1][1].any() and not out[1][3].any()
    live = [0, 2, 4, 5]
    assert (out[1][live].int().abs().amax(1) == 127).all()


@pytest.mark.parametrize("into", ["x", "residual"])
@pytest.mark.parametrize("M,K", [(9, 4096), (333, 5120), (2, 20480)])
def test_norm_in_place(qk, into, M, K):  # noqa: F811
    x, r, w = norm_inputs(M, K, 11)
    x2, r2 = x.clone(), r.clone()
    out = qk.qk_rmsnorm_quantize(x2, w, r2, h=x2 if into == "x" else r2, with_xsum=True)
    check_norm(qk, x, r, w, 1e-6, out, True)
    assert torch.equal(bits(r2 if into == "x" else x2), bits(r if into == "x" else x))


def test_norm_feeds_the_products(qk):  # noqa: F811
    """Its codes, scales and sums go into both products as the activation quantization's would."""
    x, r, w = norm_inputs(8, 512, 5)
    h, xq, sx, xsum = qk.qk_rmsnorm_quantize(x, w, r, with_xsum=True)
    W = torch.randn(256, 512, generator=gen(6), device="cuda") * 0.05
    Wq, sw = qk.qk_quantize_weights_int8(W)
    y = qk.qk_w8a8_gemm(xq, sx, Wq, sw)
    want = (xq.double() @ Wq.double().T) * sx.double()[:, None] * sw.double()
    # one rounding to bf16 (2^-8 relative) and fp32's evaluation of the dequantization (within 1/8 of it)
    assert ((y.double() - want).abs() <= 1.25 * 2.0 ** -8 * want.abs() + 1e-30).all()
    Wp, s, o = qk.qk_quantize_weights_int4(W)
    y = qk.qk_w4a8_gemm(xq, sx, xsum, Wp, s, o)
    codes = torch.stack((Wp & 15, Wp >> 4), -1).view(256, 8, 64).double()
    deq = (codes * s.double()[..., None] + o.double()[..., None]).view(256, 512)
    want = (xq.double() @ deq.T) * sx.double()[:, None]
    assert ((y.double() - want).abs() <= 1.25 * 2.0 ** -8 * want.abs() + 1e-30).all()


def rope_bound(x, positions, freq, half, amp):
    """Half a step of bf16, and the angle's fp32 (2^-25 turns) and the sine's and products' roundings."""
    want = ref.rope(x, positions, freq, half, amp)
    mag = ref.rope(x.abs(), torch.zeros_like(positions), torch.zeros_like(freq), half, 1.0)
    rot = 2 * freq.numel()
    both = mag.clone()
    if half:
        s = mag[..., :rot // 2] + mag[..., rot // 2:rot]
        both[..., :rot // 2], both[..., rot // 2:rot] = s, s
    else:
        s = mag[..., 0:rot:2] + mag[..., 1:rot:2]
        both[..., 0:rot:2], both[..., 1:rot:2] = s, s
    return want, 2.0 ** -8 * want.abs() + both * abs(amp) * (2 * math.pi * 2.0 ** -25 + 6 * 2.0 ** -24)


def check_rope(x, y, positions, freq, half, amp):
    want, tol = rope_bound(x, positions, freq, half, amp)
    rot = 2 * freq.numel()
    assert torch.equal(bits(y[..., rot:]), bits(x[..., rot:]))
    assert ((y.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("T,H,Hkv,D,rot", [(1, 1, 1, 8, 2), (1, 32, 8, 128, 128), (16, 5, 1, 64, 64), (7, 3, 3, 128, 32),
                                           (333, 2, 2, 64, 48), (5, 4, 2, 80, 40), (9, 2, 1, 128, 70), (3, 2, 1, 40, 34),
                                           (2000, 2, 1, 64, 16), (1, 2, 1, 1024, 1024), (4096, 1, 0, 64, 64)])
def test_rope(qk, T, H, Hkv, D, rot, half):  # noqa: F811
    g = gen(T + D + rot)
    rows = torch.randn(T, (H + 2 * Hkv) * D + 24, generator=g, device="cuda").bfloat16()
    q, k = rows[:, :H * D].view(T, H, D), rows[:, H * D:(H + Hkv) * D].view(T, Hkv, D)
    k = k if Hkv else None
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda", dtype=torch.int32)
    freq = qk.qk_rope_frequencies(rot)
    layout = qk.QK_ROPE_HALF if half else qk.QK_ROPE_INTERLEAVED
    before = rows.clone()
    qo, ko = qk.qk_rope(q, k, pos, freq, layout=layout, amplitude=1.25)
    check_rope(q, qo, pos, freq, half, 1.25)
    if Hkv:
        check_rope(k, ko, pos, freq, half, 1.25)
    assert torch.equal(bits(rows), bits(before))
    # in place, on the strided rows: the same bits, and nothing else of the rows changes
    qk.qk_rope(q, k, pos, freq, layout=layout, amplitude=1.25, q_out=q, k_out=k)
    assert torch.equal(bits(q), bits(qo)) and (not Hkv or torch.equal(bits(k), bits(ko)))
    assert torch.equal(bits(rows[:, (H + Hkv) * D:]), bits(before[:, (H + Hkv) * D:]))


def test_rope_positions_at_the_ends(qk):  # noqa: F811
    """Position 0 is the identity; the largest and negative ones keep their angle."""
    x = torch.randn(6, 2, 64, generator=gen(1), device="cuda").bfloat16()
    pos = torch.tensor([0, 1, 2 ** 31 - 1, -1, -2 ** 31, 10 ** 9], dtype=torch.int32, device="cuda")
    freq = qk.qk_rope_frequencies(64)
    y, _ = qk.qk_rope(x, None, pos, freq)
    assert torch.equal(bits(y[0]), bits(x[0]))
    check_rope(x, y, pos, freq, True, 1.0)


@pytest.mark.parametrize("mode,more", [(0, {}), (1, {"factor": 4.0}), (2, {"factor": 8.0}),
                                       (3, {"factor": 8.0, "trained": 8192.0, "slow": 1.0, "fast": 4.0})])
@pytest.mark.parametrize("rot", [2, 34, 128, 1024])
def test_rope_frequencies(qk, mode, more, rot):  # noqa: F811
    got = qk.qk_rope_frequencies(rot, 500000.0, mode, **more).cpu()
    want = ref.rope_frequencies(rot, 500000.0, mode, **more)
    assert ((got - want).abs() <= 1e-13 * want).all()


def test_refusals(qk):  # noqa: F811
    x, r, w = norm_inputs(4, 64, 1)
    with pytest.raises(ValueError):
        qk.qk_rmsnorm_quantize(x, w[:32])
    with pytest.raises(ValueError):
        qk.qk_rmsnorm_quantize(x, w, r[:2])
    with pytest.raises(ValueError):
        qk.qk_rmsnorm_quantize(x, w, h=r)
    with pytest.raises(ValueError):
        qk.qk_rmsnorm_quantize(x.t(), w[:4])
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos, freq = torch.zeros(4, dtype=torch.int32, device="cuda"), qk.qk_rope_frequencies(64)
    with pytest.raises(ValueError):
        qk.qk_rope(q, q[:2], pos, freq)
    with pytest.raises(ValueError):
        qk.qk_rope(q.transpose(0, 1), None, pos[:2], freq)
    with pytest.raises(TypeError):
        qk.qk_rope(q, None, pos.long(), freq)
    with pytest.raises(qk.QKError):
        qk.qk_rope(q, None, pos, qk.qk_rope_frequencies(66))


def test_empty(qk):  # noqa: F811
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    h, xq, sx, xsum = qk.qk_rmsnorm_quantize(e, None, e, with_xsum=True)
    assert xq.shape == (0, 64) and sx.shape == (0,) and xsum.shape == (0, 1) and h.shape == (0, 64)
    q, k = qk.qk_rope(e.view(0, 1, 64), None, torch.empty(0, dtype=torch.int32, device="cuda"),
                      qk.qk_rope_frequencies(64))
    assert q.shape == (0, 1, 64) and k is None
