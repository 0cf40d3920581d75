"""The norm, rotary and 4-bit cache calls on the CPU: argument checks, sizes, and the record's layout."""
import ctypes
import itertools

import pytest
import torch

from tests import block_reference as ref

FAKE = 1 << 20  # aligned, never dereferenced
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def qk():
    from w4a8_quantized_gemm_token_b200 import build

    build.build()
    from w4a8_quantized_gemm_token_b200 import binding

    return binding


def ready():
    """The status of a call whose arguments pass: the device check stops it here."""
    return 4


needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers: CPU only")


def norm(qk, x=FAKE, r=FAKE, M=4, K=64, w=FAKE, eps=1e-6, h=FAKE, xq=FAKE, sx=FAKE, xsum=None):
    return qk.lib.qk_rmsnorm_quantize(x, r, M, K, w, eps, h, xq, sx, xsum, None)


@needs_no_gpu
def test_norm_checks(qk):
    assert norm(qk) == ready() and norm(qk, r=None, h=None, w=None) == ready()
    assert norm(qk, M=0, x=None, r=None, h=None, xq=None, sx=None) == 0
    for bad in ({"x": None}, {"xq": None}, {"sx": None}, {"r": None}, {"h": None}, {"M": -1},
                {"eps": -1.0}, {"eps": NAN}, {"eps": INF}):
        assert norm(qk, **bad) == 1, bad
    for bad in ({"K": 16}, {"K": 48}, {"K": 65568}, {"K": 96, "xsum": FAKE}):
        assert norm(qk, **bad) == 2, bad
    assert norm(qk, K=96) == ready()
    for name in ("x", "r", "w", "h", "xq", "sx", "xsum"):
        assert norm(qk, **{name: FAKE + 8}) == 3, name


def rope(qk, q=FAKE, qs=512, qo=FAKE + (1 << 16), qos=512, H=4, k=FAKE, ks=256, ko=FAKE + (1 << 16),
         kos=256, Hkv=2, T=3, D=128, rot=128, layout=0, pos=FAKE, freq=FAKE, amp=1.0):
    return qk.lib.qk_rope(q, qs, qo, qos, H, k, ks, ko, kos, Hkv, T, D, rot, layout, pos, freq, amp, None)


@needs_no_gpu
def test_rope_checks(qk):
    assert rope(qk) == ready() and rope(qk, k=None, ko=None, ks=0, kos=0) == ready()
    assert rope(qk, T=0, q=None, qo=None, k=None, ko=None, pos=None, freq=None) == 0
    for bad in ({"q": None}, {"qo": None}, {"k": None}, {"ko": None}, {"pos": None}, {"freq": None},
                {"T": -1}, {"H": 0}, {"Hkv": 0}, {"layout": 2}, {"amp": NAN}, {"amp": INF},
                {"qo": FAKE, "qos": 1024}, {"ko": FAKE, "kos": 1024}):
        assert rope(qk, **bad) == 1, bad
    for bad in ({"rot": 0}, {"rot": 3}, {"rot": 130}, {"D": 12, "rot": 4}, {"D": 1032}, {"qs": 504},
                {"qos": 516}, {"ks": 248}, {"kos": 260}, {"H": 1 << 20, "qs": 1 << 30, "qos": 1 << 30}):
        assert rope(qk, **bad) == 2, bad
    for name in ("q", "qo", "k", "ko", "pos", "freq"):
        assert rope(qk, **{name: FAKE + 4}) == 3, name
    f = lambda rot=64, base=1e4, mode=0, factor=1.0, trained=0.0, slow=1.0, fast=32.0, out=FAKE: \
        qk.lib.qk_rope_frequencies(rot, base, mode, factor, trained, slow, fast, out, None)  # noqa: E731
    assert f() == ready() and f(mode=3, factor=8.0, trained=4096.0) == ready()
    for bad in ({"mode": 4}, {"mode": -1}, {"base": 1.0}, {"base": NAN}, {"mode": 1, "factor": 0.0},
                {"mode": 2, "factor": INF}, {"mode": 3, "trained": 0.0}, {"out": None},
                {"mode": 3, "trained": 1.0, "slow": 4.0, "fast": 4.0}):
        assert f(**bad) == 1, bad
    assert f(rot=0) == f(rot=7) == f(rot=1026) == 2 and f(out=FAKE + 8) == 3


def kv4(qk, call, **over):
    a = dict(k=FAKE, ks=1024, v=FAKE, vs=1024, T=6, Hkv=8, D=128, table=FAKE, B=3, wide=4, lens=FAKE,
             cu=FAKE, cache=FAKE, pages=9, page=32, H=32, scale=0.1, window=0, sinks=0, q=FAKE, qs=4096,
             out=FAKE, ws=None, wsb=0)
    a.update(over)
    if call == "append":
        return qk.lib.qk_kv4_append(a["k"], a["ks"], a["v"], a["vs"], a["T"], a["Hkv"], a["D"], a["table"], a["B"],
                                    a["wide"], a["lens"], a["cu"], a["cache"], a["pages"], a["page"], None)
    if call == "gather":
        return qk.lib.qk_kv4_gather(a["cache"], a["pages"], a["page"], a["Hkv"], a["D"], a["table"], a["B"], a["wide"],
                                    a["lens"], a["cu"], a["T"], a["k"], a["ks"], a["v"], a["vs"], None)
    return qk.lib.qk_kv4_attention(a["q"], a["qs"], a["T"], a["H"], a["Hkv"], a["D"], a["cache"], a["pages"], a["page"],
                                   a["table"], a["B"], a["wide"], a["lens"], a["cu"], a["scale"], a["window"],
                                   a["sinks"], a["out"], a["ws"], a["wsb"], None)


@needs_no_gpu
@pytest.mark.parametrize("call", ["append", "gather", "attention"])
def test_kv4_checks(qk, call):
    assert kv4(qk, call) == ready() and kv4(qk, call, cu=None) == ready()
    assert kv4(qk, call, T=0, k=None, v=None, q=None, table=None, lens=None, cu=None, cache=None) == 0
    for bad in ({"T": -1}, {"B": -1}, {"B": 0}, {"table": None}, {"lens": None}, {"cache": None},
                {"cu": None, "T": 7}, {"wide": -1}, {"pages": -1}):
        assert kv4(qk, call, **bad) == 1, bad
    for bad in ({"D": 96}, {"D": 256}, {"page": 8}, {"page": 24}, {"page": 1040}, {"Hkv": 0}, {"pages": 0},
                {"wide": 0}, {"wide": (1 << 25) + 1}, {"T": (1 << 30) + 1}, {"B": (1 << 30) + 1}):
        assert kv4(qk, call, **bad) == 2, bad
    for name in ("table", "lens", "cu", "cache"):
        assert kv4(qk, call, **{name: FAKE + 8}) == 3, name


@needs_no_gpu
def test_kv4_row_checks(qk):
    for call in ("append", "gather"):
        assert kv4(qk, call, ks=1016) == kv4(qk, call, vs=1028) == 2
        assert kv4(qk, call, k=None) == kv4(qk, call, v=None) == 1
        assert kv4(qk, call, k=FAKE + 2) == kv4(qk, call, v=FAKE + 8) == 3
    at = lambda **o: kv4(qk, "attention", **o)  # noqa: E731
    for bad in ({"scale": -1.0}, {"scale": NAN}, {"scale": INF}, {"window": -1}, {"sinks": -1}, {"q": None},
                {"out": None}):
        assert at(**bad) == 1, bad
    for bad in ({"H": 12}, {"H": 0}, {"qs": 4088}, {"qs": 4100}, {"window": (1 << 30) + 1},
                {"sinks": (1 << 30) + 1}, {"H": 1 << 20, "Hkv": 1, "qs": 1 << 27, "T": 3000}):
        assert at(**bad) == 2, bad
    assert at(q=FAKE + 8) == at(out=FAKE + 8) == 3
    need = qk.qk_kv4_attention_workspace_size(128)
    assert at(ws=FAKE, wsb=need - 1) == at(ws=FAKE + 16, wsb=need) == 5
    assert at(ws=FAKE, wsb=need) == ready()


def test_kv4_sizes(qk):
    assert qk.qk_kv4_cache_size(7, 3, 48, 128) == 7 * 3 * 48 * 144
    assert qk.qk_kv4_cache_size(7, 3, 48, 64) == 7 * 3 * 48 * 72
    for bad in ((0, 1, 16, 64), (1, 0, 16, 64), (1, 1, 8, 64), (1, 1, 16, 96), (1, 1, 2048, 64)):
        assert qk.qk_kv4_cache_size(*bad) == 0
    assert qk.qk_kv4_attention_workspace_size(128) > qk.qk_kv4_attention_workspace_size(64) > 0
    assert qk.qk_kv4_attention_workspace_size(96) == 0
    # records have 32-bit numbers
    assert qk.qk_kv4_cache_size((1 << 26) - 1, 64, 16, 64) == ((1 << 26) - 1) * 64 * 16 * 72
    assert qk.qk_kv4_cache_size(1 << 26, 64, 16, 64) == 0


@pytest.mark.parametrize("D", [64, 128])
def test_record_layout_is_a_bijection(D):
    """Every nibble of a record's code bytes belongs to one (K or V, token, dim)."""
    k, v, shift = ref.record_places(D)
    seen = set()
    for part in (k, v):
        for r, d in itertools.product(range(16), range(D)):
            seen.add((int(part[r, d]), int(shift[r, d])))
    assert seen == set(itertools.product(range(16 * D), (0, 4)))


def test_reference_quantize4_closed_forms():
    """A group on its own grid comes back as it is; a constant group has scale 0."""
    w = torch.arange(64).remainder(16).to(torch.float32).mul(0.25).sub(2).to(torch.bfloat16)[None]
    value, q, s, o = ref.quantize4(w)
    assert torch.equal(value, w.double()) and float(s) == 0.25 and float(o) == -2
    assert torch.equal(q[0], torch.arange(64).remainder(16).double())
    value, q, s, _ = ref.quantize4(torch.full((1, 64), 1.5, dtype=torch.bfloat16))
    assert float(s) == 0 and not q.any() and torch.equal(value, torch.full((1, 64), 1.5).double())


def test_binding_checks(qk):
    bf = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        qk.qk_rmsnorm_quantize(bf[0])
    with pytest.raises(TypeError):
        qk.qk_rmsnorm_quantize(bf[0].float())
    with pytest.raises(ValueError):
        qk.qk_rope(bf, None, torch.zeros(2, dtype=torch.int32), torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError):
        qk.qk_kv4_attention(bf, torch.zeros(1, 2, 16, 72, dtype=torch.uint8), torch.zeros(2, 1, dtype=torch.int32),
                            torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        qk.qk_kv4_append(bf, bf, torch.zeros(1, 4, 16, 72, dtype=torch.uint8), torch.zeros(2, 1, dtype=torch.int32),
                         torch.zeros(2, dtype=torch.int32))
    assert qk.qk_status_string(8).startswith("QK_ERR_INDEX")
    assert ctypes.sizeof(ctypes.c_int) == 4
