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
