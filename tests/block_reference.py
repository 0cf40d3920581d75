"""64-bit references of the norm, the rotary positions and the 4-bit cache, written from their
formulas (include/qk.h) in torch; they run where their inputs are."""
import math

import torch

F64 = torch.float64


def r32(t):
    """Rounded to fp32 (an exact fp64 product of two fp32 numbers gives the fp32 product)."""
    return t.to(torch.float32).to(F64)


def rmsnorm_quantize(x, weight, residual, eps):
    h = x if residual is None else (x.to(F64) + residual.to(F64)).to(torch.float32).to(torch.bfloat16)
    h64 = h.to(F64)
    u = h64 if weight is None else r32(h64 * weight.to(F64))
    top = u.abs().amax(1)
    live = top > 0
    one = torch.ones_like(top)
    codes = (r32(u * r32(127.0 * r32(1.0 / torch.where(live, top, one)))[:, None])).round().clamp(-127, 127)
    rstd = 1.0 / torch.sqrt((h64 * h64).mean(1) + eps)
    sx = torch.where(live, top / 127.0 * rstd, one)
    return h, codes.to(torch.int8), sx


def rope_frequencies(rot, base, scaling, factor=1.0, trained=0.0, slow=1.0, fast=32.0):
    """scaling: 0 plain, 1 linear, 2 ntk, 3 by parts; turns per position."""
    out = []
    if scaling == 2 and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    for i in range(rot // 2):
        f = base ** (-2 * i / rot) / (2 * math.pi)
        if scaling == 1:
            f /= factor
        if scaling == 3:
            keep = min(1.0, max(0.0, (trained * f - slow) / (fast - slow)))
            f = f * keep + f / factor * (1 - keep)
        out.append(f)
    return torch.tensor(out, dtype=F64)


def rope(x, positions, freq, half, amplitude):
    """x [T, H, D] -> fp64"""
    y = x.to(F64).clone()
    rot = 2 * freq.numel()
    turns = positions.to(F64)[:, None] * freq
    angle = 2 * math.pi * (turns - turns.floor())
    c, s = (amplitude * angle.cos())[:, None], (amplitude * angle.sin())[:, None]
    ia = torch.arange(rot // 2, device=x.device) if half else torch.arange(0, rot, 2, device=x.device)
    ib = ia + rot // 2 if half else ia + 1
    a, b = x[..., ia].to(F64), x[..., ib].to(F64)
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


def quantize4(w):
    """w bf16 [..., D] -> the values of its 4-bit groups of 64, and (codes, scale, offset)"""
    x = w.to(F64).unflatten(-1, (-1, 64))
    lo, hi = x.amin(-1), x.amax(-1)
    s = r32(r32(hi - lo) / 15.0).to(torch.float32).to(torch.float16).to(F64)
    o = lo.to(torch.float32).to(torch.float16).to(F64)
    inv = r32(1.0 / torch.where(s > 0, s, torch.ones_like(s)))
    q = (r32(r32(x - o[..., None]) * inv[..., None])).round().clamp(0, 15)
    q = torch.where(s[..., None] > 0, q, torch.zeros_like(q))
    return (q * s[..., None] + o[..., None]).flatten(-2), q.flatten(-2), s, o


def record_places(D):
    """Byte in a record and shift of (token, dim), for K and V, by the documented layout."""
    NG = D // 64
    r = torch.arange(16)[:, None]
    d = torch.arange(D)[None, :]
    g, e = d // 64, d % 64
    k = ((r * 4 + e // 16) * NG + g) * 8 + (e % 16) // 8 * 4 + (e % 8) // 2
    v = 8 * D + (((r // 2) * 8 + e // 8) * NG + g) * 8 + (e % 8) // 4 * 4 + (r % 2) * 2 + (e % 4) // 2
    return k, v, (4 * (d % 2)).expand(16, D)


def decode_records(rec, D):
    """rec uint8 [n, 18 D] -> K, V values fp64 [n, 16, D]"""
    kb, vb, shift = (t.to(rec.device) for t in record_places(D))
    NG = D // 64
    sc = rec[:, 16 * D:].contiguous().view(torch.float16).to(F64).view(-1, 2, 16, NG, 2)
    out = []
    for i, byte in enumerate((kb, vb)):
        code = ((rec[:, byte].to(torch.int32) >> shift) & 15).to(F64)
        s = sc[:, i].repeat_interleave(64, 2)
        out.append(code * s[..., 0] + s[..., 1])
    return out


def request_kv(cache, table_row, length, D):
    """K, V values fp64 [length, Hkv, D] of one request"""
    P, Hkv, page, _ = cache.shape
    pages = table_row[:-(-length // page)].long()
    rec = cache[pages].view(len(pages), Hkv, page // 16, 18 * D).transpose(1, 2).reshape(-1, 18 * D)
    return [t.view(len(pages) * page // 16, Hkv, 16, D).transpose(1, 2).reshape(-1, Hkv, D)[:length]
            for t in decode_records(rec, D)]


def attention(q, k, v, scale, window, sinks):
    """q [n, H, D], k, v fp64 [L, Hkv, D] (the rows are the last n tokens) -> (out fp64, how far a
    result computed with fp32 scores and sums, and weight x scale rounded to fp16, may be from it)."""
    n, H, D = q.shape
    L, Hkv = k.shape[:2]
    G = H // Hkv
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    x = torch.einsum("ihd,jhd->hij", q.to(F64), kk) * scale
    pos = torch.arange(L - n, L, device=q.device)[:, None]
    key = torch.arange(L, device=q.device)[None, :]
    see = key <= pos
    if window:
        see = see & ((key > pos - window) | (key < sinks))
    x = x.masked_fill(~see, -math.inf)
    top = x.amax(-1, keepdim=True) if L else x.new_zeros(H, n, 1)
    p = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, torch.zeros_like(p))
    out = torch.einsum("hij,jhd->ihd", p, vv)
    if L == 0:
        return out, out
    # every key: |code scale| + |offset| <= spread (values and offset are within it)
    spread = 3 * vv.abs().amax((0, 2))[None, :, None] + 1e-30
    a = scale * torch.einsum("ihd,jhd->hij", q.to(F64).abs(), kk.abs()).masked_fill(~see, 0).amax(-1)
    a = 3 * a.T[..., None]  # bounds scale sum |q| (|code scale| + |offset|): 3 |k| as for the values
    # scores: 64 products and 4 group terms per sum, then one product: 2^-17 a; the weights move by
    # twice that and by 2^-20 (2^x, the sum of the weights).  weight x scale is rounded to fp16, half
    # a step 2^-11 of it: sum P scale code 2^-11 <= 2^-11 spread.  fp32 sums of P V: two roundings per
    # 16 keys and the join's
    move = 2 * a * 2.0 ** -17 + 2.0 ** -20 + 2.0 ** -11 + (2 * (L / 16) + 400) * 2.0 ** -23
    return out, 2.0 ** -8 * out.abs() + spread * move
