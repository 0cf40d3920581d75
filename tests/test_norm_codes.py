"""The quantizing norm's codes beside the activation quantization's, on the same rows.

The norm multiplies by fl(127 fl(1 / U)), the activation quantization by fl(127 / U); u and U are bf16 here
(no residual, no weight).  Everything below is exact: fp32 operations in numpy, quotients of small whole numbers."""
import numpy as np
import pytest
import torch

F = np.float32


def pairs():
    """u <= U over every mantissa of both and the exponents whose codes are not all 0."""
    m = np.arange(128, 256, dtype=np.int64)
    U = np.repeat(m, 128 * 9)
    u = np.tile(np.repeat(m, 9), 128)
    down = np.tile(np.arange(9), 128 * 128)
    keep = u <= U << down
    return u[keep], U[keep], down[keep]


def codes(u, multiplier):
    return np.rint(F(u) * multiplier).astype(np.int64)


def test_codes_are_a_step_apart_only_halfway():
    """Both rules' codes are within 1/2 + 2^-15 of u 127 / U; where they differ, it is by one, around a value
    that close to halfway, and the distances of the two are alike within 2^-14."""
    u, U, down = pairs()
    x = u.astype(F) / F(2) ** down  # bf16 numbers, exact
    once, twice = F(127) / U.astype(F), F(127) * (F(1) / U.astype(F))
    a, b = codes(x, once), codes(x, twice)
    exact = 127.0 * u / (U * 2.0 ** down)  # 52 bits are enough: its error is 2^-46
    for c in (a, b):
        assert (np.abs(c - exact) <= 0.5 + 2.0 ** -15).all()
    differ = a != b
    assert differ.any() and (np.abs(a - b)[differ] == 1).all()
    assert (np.abs(exact - (a + b) / 2)[differ] <= 2.0 ** -15).all()
    # a bound of the multipliers: half a step, and one and a half
    assert (np.abs(once.astype(float) * U / 127 - 1) <= 2.0 ** -24).all()
    assert (np.abs(twice.astype(float) * U / 127 - 1) <= 2.0 ** -23).all()
    assert 0.2 < np.mean([F(127) / F(v) != F(127) * (F(1) / F(v)) for v in range(128, 256)]) < 0.3


@pytest.mark.gpu
def test_codes_beside_the_activation_quantization():
    """On the GPU: the same rows through both calls differ just where the two multipliers say, by one; +-U / 2
    is such a value."""
    from w4a8_quantized_gemm_token_b200 import binding as qk

    g = torch.Generator(device="cuda").manual_seed(2)
    M, K = 128, 4096
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    U = (128 + torch.arange(M, device="cuda")).float() / 16  # every mantissa, above all of x
    x[:, 0] = U.bfloat16()
    x[:, 1], x[:, 2] = (U / 2).bfloat16(), (-U / 2).bfloat16()
    norm, act = qk.qk_rmsnorm_quantize(x)[1].cpu().numpy(), qk.qk_quantize_activations(x)[0].cpu().numpy()
    x, U = x.float().cpu().numpy(), U.cpu().numpy()[:, None]
    assert np.array_equal(norm, codes(x, F(127) * (F(1) / U)))
    assert np.array_equal(act, codes(x, F(127) / U))
    differ = norm != act
    assert differ[:, 1].any() and np.abs(norm.astype(int) - act)[differ].max() == 1
