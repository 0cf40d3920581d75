"""The operators between two quantized linears of a transformer block, case by case: the RMS norm that
quantizes, rotary positions, and the 4-bit paged key/value cache with the attention that reads it.

``own`` chooses between the plain forms (elementary torch operations in 32 bits or more) and the calls of
``w4a8_quantized_gemm_token_b200.binding``.

The cache holds, per page and kv head, one record for every 16 tokens: K codes, V codes, K scales, V scales.
A group is 64 dims of one token's K (or V): value = code * scale + offset, scale and offset in fp16, codes
0..15.  With NG = D / 64 groups, the record's parts are
  K codes   u32 [row 16][t 4][group NG][j 2], nibble i of a word = dim 64 group + 16 t + 8 j + i
  V codes   u32 [pair 8][g 8][group NG][h 2], low half = token 2 pair, high half = token 2 pair + 1,
            nibble i of a half = dim 64 group + 8 g + 4 h + i
  K, V scales  fp16 [token 16][group NG][scale, offset]
"""
import math

import numpy as np
import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ------------------------------------------------------------------------------------------------ cases

def _norm(name, M, K, residual=True, weight=True, xsum=True):
    return {"name": name, "op": "norm", "M": M, "K": K, "residual": residual, "weight": weight, "xsum": xsum}


def _rope(name, T, H, Hkv, D, rot, layout, start, scaling="plain"):
    return {"name": name, "op": "rope", "T": T, "H": H, "Hkv": Hkv, "D": D, "rot": rot, "layout": layout,
            "start": start, "scaling": scaling}


def _append(name, B, new, ragged, past, Hkv, D, page):
    return {"name": name, "op": "append", "B": B, "new": new, "ragged": ragged, "past": past, "Hkv": Hkv,
            "D": D, "page": page}


def _attn(name, B, L, ragged, Tq, H, Hkv, D, page, window=0, sinks=0):
    return {"name": name, "op": "attn", "B": B, "L": L, "ragged": ragged, "Tq": Tq, "H": H, "Hkv": Hkv, "D": D,
            "page": page, "window": window, "sinks": sinks}


def listed():
    return [
        # one token's norm before the one-token GEMV (codes and group sums): pure latency
        _norm("norm_1x4096", 1, 4096),
        # a batch whose size is no multiple of anything, W8A8 (no group sums), rows longer than a warp holds
        _norm("norm_1111x5120", 1111, 5120, xsum=False),
        # a long prompt (or a diffusion transformer's token rows): memory-bound
        _norm("norm_16384x4096", 16384, 4096),
        # one decode step of 16 requests, grouped heads
        _rope("rope_16x32+8_half", 16, 32, 8, 128, 128, "half", 4000),
        # a long prompt, a quarter of the head rotated in pairs, positions far past the trained length
        _rope("rope_14040x40+8_pairs", 14040, 40, 8, 128, 32, "interleaved", 500000, "by_parts"),
        # one new token for each of 64 requests
        _append("append_64x1", 64, 1, False, 2000, 8, 128, 16),
        # ragged prompts written at once
        _append("append_8x2048_ragged", 8, 2048, True, 100, 8, 128, 64),
        # one request alone: the split along the cache is all the parallelism there is
        _attn("attn_1x4097", 1, 4097, False, 1, 32, 8, 128, 16),
        # an ordinary ragged batch, five query heads to a kv head
        _attn("attn_16x8192_ragged", 16, 8192, True, 1, 40, 8, 128, 64),
        # a few drafted tokens checked at once behind a sliding window with four first tokens kept, head dim 64
        _attn("attn_32x6000_window", 32, 6000, True, 4, 32, 8, 64, 32, 2048, 4),
        # a chunk of a prompt over its cache
        _attn("attn_4x2500_chunk200", 4, 2500, True, 200, 16, 16, 128, 16),
        # a full batch of long requests, eight query heads to a kv head: the cache stream
        _attn("attn_64x16384", 64, 16384, False, 1, 64, 8, 128, 128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "rope", "append", "attn", "attn"])
    if op == "norm":
        K = 32 * _log_int(rng, 8, 384)
        M = _log_int(rng, 1, min(16384, 16384 * 4096 // K))
        c = _norm("", M, K, rng.random() < 0.8, rng.random() < 0.9, K % 64 == 0 and rng.random() < 0.6)
    elif op == "rope":
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        H = Hkv * rng.randint(1, 5)
        T = _log_int(rng, 1, min(16384, 14040 * 48 * 128 // ((H + Hkv) * D)))
        rot = rng.choice([D, D, D // 2, D // 4, 2 * rng.randint(1, D // 2)])
        c = _rope("", T, H, Hkv, D, rot, rng.choice(["half", "interleaved"]), _log_int(rng, 1, 1000000),
                  rng.choice(["plain", "linear", "ntk", "by_parts"]))
    elif op == "append":
        B, Hkv, D = _log_int(rng, 1, 64), rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 128])
        new = _log_int(rng, 1, max(1, min(2048, 8 * 2048 * 8 * 128 // (B * Hkv * D))))
        c = _append("", B, new, rng.random() < 0.5, _log_int(rng, 1, 3000), Hkv, D, rng.choice([16, 32, 64, 128]))
    else:
        B, Hkv, D = _log_int(rng, 1, 64), rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 128])
        G = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
        L = _log_int(rng, 1, max(1, min(32768, 64 * 16384 * 8 * 128 // (B * Hkv * D))))
        most = max(1, min(L, 4 * 200 * 16 * 2500 // (B * Hkv * G * L)))
        Tq = rng.choice([1, 1, min(most, rng.randint(2, 8)), _log_int(rng, 1, most)])
        window = rng.choice([0, 0, _log_int(rng, 1, max(1, L))])
        c = _attn("", B, L, rng.random() < 0.6, Tq, Hkv * G, Hkv, D, rng.choice([16, 32, 64, 128]), window,
                  rng.choice([0, 4, rng.randint(1, 100)]) if window else 0)
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------- lengths, pages

def _lengths(case):
    """(tokens already there, new tokens) of each request, from the case alone."""
    B = case["B"]
    r = np.random.default_rng([B, case.get("L", 0), case.get("past", 0), case.get("Tq", 0), case.get("new", 0)])
    if case["op"] == "append":
        new, past = np.full(B, case["new"]), np.full(B, case["past"])
        if case["ragged"]:
            new, past = r.integers(1, case["new"] + 1, B), r.integers(0, case["past"] + 1, B)
            new[0] = case["new"]
        return past, new
    total, new = np.full(B, case["L"]), np.full(B, case["Tq"])
    if case["ragged"]:
        total = np.exp(r.uniform(np.log(max(1, case["L"] // 8)), np.log(case["L"] + 1), B)).astype(np.int64)
        total = np.clip(total, 1, case["L"])
        total[0] = case["L"]
        if case["Tq"] > 1:
            new = r.integers(1, case["Tq"] + 1, B)
            new[0] = case["Tq"]
        new = np.minimum(new, total)
    return total - new, new


def _pages(case, gen):
    """page table, lengths behind the new tokens, first row of each request's new tokens, pages in all"""
    past, new = _lengths(case)
    total, page = past + new, case["page"]
    wide = int(-(-total.max() // page))
    need = -(-total // page)
    count = int(need.sum()) + 5
    order = torch.randperm(count, generator=gen, device="cuda").cpu().numpy()
    table = np.full((case["B"], wide), -1, np.int32)
    at = 0
    for b in range(case["B"]):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return (torch.from_numpy(table).cuda(), torch.from_numpy(total.astype(np.int32)).cuda(),
            torch.from_numpy(cu).cuda(), count, wide, int(cu[-1]), int(new.max()))


# ------------------------------------------------------------------------------- the 4-bit rule and layout

def _quantize(w):
    """[..., D] fp32 -> codes (fp32 whole numbers) [..., D], scale and offset fp16 [..., NG]"""
    x = w.reshape(*w.shape[:-1], -1, 64)
    lo, hi = x.amin(-1), x.amax(-1)
    s, o = ((hi - lo) / 15.0).half(), lo.half()
    r = torch.where(s == 0, torch.zeros_like(lo), 1.0 / s.float())
    q = ((x - o.float()[..., None]) * r[..., None]).round().clamp(0, 15)
    return q.reshape(w.shape), s, o


def _unpack(rec, D):
    """records uint8 [n, 18 D] -> K codes, V codes [n, 16, D] uint8; K, V scales fp16 [n, 16, NG, 2]"""
    n, NG, half = rec.shape[0], D // 64, 8 * D
    kb = rec[:, :half]
    k = torch.stack((kb & 15, kb >> 4), -1).view(n, 16, 4, NG, 2, 8).permute(0, 1, 3, 2, 4, 5).reshape(n, 16, D)
    vb = rec[:, half:2 * half]
    v = torch.stack((vb & 15, vb >> 4), -1).view(n, 8, 8, NG, 2, 2, 4).permute(0, 1, 5, 3, 2, 4, 6).reshape(n, 16, D)
    sc = rec[:, 2 * half:].contiguous().view(torch.float16).view(n, 2, 16, NG, 2)
    return k, v, sc[:, 0], sc[:, 1]


def _pack(k, v, ks, vs):
    """the inverse of _unpack"""
    n, D = k.shape[0], k.shape[2]
    NG = D // 64
    kk = k.view(n, 16, NG, 4, 2, 8).permute(0, 1, 3, 2, 4, 5).reshape(n, 8 * D, 2)
    vv = v.view(n, 8, 2, NG, 8, 2, 4).permute(0, 1, 4, 3, 5, 2, 6).reshape(n, 8 * D, 2)
    sc = torch.stack((ks, vs), 1).reshape(n, -1).view(torch.uint8)
    return torch.cat((kk[..., 0] | kk[..., 1] << 4, vv[..., 0] | vv[..., 1] << 4, sc), 1)


def _fill(cache, gen, D):
    """A cache as a running server holds it: keys with a few strong channels, values near normal; pages in turn."""
    P, Hkv, page = cache.shape[:3]
    strong = 1.0 + 4.0 * (torch.rand(Hkv, 1, D, generator=gen, device="cuda") < 0.05)
    shift = torch.randn(Hkv, 1, D, generator=gen, device="cuda")
    step = max(1, (1 << 27) // (Hkv * page * D))
    for p in range(0, P, step):
        m = min(step, P - p)
        k = torch.randn(m, Hkv, page, D, generator=gen, device="cuda") * strong + shift
        v = torch.randn(m, Hkv, page, D, generator=gen, device="cuda")
        parts = []
        for w in (k, v):
            q, s, o = _quantize(w)
            parts.append((q.to(torch.uint8).view(-1, 16, D), torch.stack((s, o), -1).view(-1, 16, D // 64, 2)))
        cache[p:p + m] = _pack(parts[0][0], parts[1][0], parts[0][1], parts[1][1]).view(m, Hkv, page, -1)


# ---------------------------------------------------------------------------------------------- prepare

def _frequencies(case):
    """turns per position of every pair, in 64 bits"""
    rot, base, factor, trained = case["rot"], 10000.0, 8.0, 4096.0
    i = torch.arange(rot // 2, dtype=F64, device="cuda")
    if case["scaling"] == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] == "by_parts":
        keep = ((trained * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    return f / (2 * math.pi)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    op, s = case["op"], {"case": case}
    if op == "norm":
        M, K = case["M"], case["K"]
        loud = 1.0 + 19.0 * (torch.rand(K, generator=gen, device="cuda") < 0.01)  # a few large channels
        s["x"] = (randn(M, K) * 0.5).to(BF16)
        s["residual"] = (randn(M, K) * loud).to(BF16) if case["residual"] else None
        s["weight"] = 1.0 + 0.2 * randn(K) if case["weight"] else None
        return s
    D, Hkv = case["D"], case["Hkv"]
    if op == "rope":
        T, H = case["T"], case["H"]
        qkv = randn(T, (H + 2 * Hkv) * D).to(BF16)  # one projection's rows: q and k are strided views of it
        s["q"] = qkv[:, :H * D].view(T, H, D)
        s["k"] = qkv[:, H * D:(H + Hkv) * D].view(T, Hkv, D)
        s["positions"] = (case["start"] + torch.randperm(T, generator=gen, device="cuda")).to(torch.int32)
        s["freq"] = _frequencies(case)
        s["amplitude"] = 1.2 if case["scaling"] == "by_parts" else 1.0
        return s
    s["table"], s["lens"], s["cu"], count, s["wide"], T, s["most"] = _pages(case, gen)
    s["cache"] = torch.zeros(count, Hkv, case["page"], D + D // 8, dtype=torch.uint8, device="cuda")
    if op == "append":
        qkv = randn(T, 3 * Hkv * D).to(BF16)
        s["k"] = qkv[:, Hkv * D:2 * Hkv * D].view(T, Hkv, D)
        s["v"] = qkv[:, 2 * Hkv * D:].view(T, Hkv, D)
        return s
    _fill(s["cache"], gen, D)
    s["q"] = (randn(T, case["H"], D) * 1.5).to(BF16)
    return s


# ------------------------------------------------------------------------------------------ plain forms

def _plain_norm(s):
    x, w, h = s["x"], s["weight"], None
    if s["residual"] is not None:
        h = x = (x.float() + s["residual"].float()).to(BF16)
    u = x.float() if w is None else x.float() * w
    top = u.abs().amax(-1, keepdim=True)
    rstd = 1.0 / torch.sqrt((x.float() * x.float()).mean(-1, keepdim=True) + 1e-6)
    codes = (u * torch.where(top == 0, torch.zeros_like(top), 127.0 / top)).round().clamp(-127, 127)
    scale = torch.where(top == 0, torch.ones_like(top), top / 127.0 * rstd)
    sums = codes.view(x.shape[0], -1, 64).sum(-1).to(torch.int32) if s["case"]["xsum"] else None
    return {"h": h, "values": codes * scale, "scale": scale[:, 0], "sums": sums}


def _turn(x, c, s, rot, layout):
    y = x.float()
    a, b = (y[..., :rot // 2], y[..., rot // 2:rot]) if layout == "half" else (y[..., 0:rot:2], y[..., 1:rot:2])
    c, s = c[:, None, :], s[:, None, :]
    u, v = a * c - b * s, b * c + a * s
    y = torch.cat((u, v, y[..., rot:]) if layout == "half" else (torch.stack((u, v), -1).flatten(-2), y[..., rot:]), -1)
    return y.to(BF16)


def _plain_rope(s):
    case = s["case"]
    turns = s["positions"].double()[:, None] * s["freq"]
    angle = (turns - turns.floor()) * (2 * math.pi)
    c, n = (angle.cos() * s["amplitude"]).float(), (angle.sin() * s["amplitude"]).float()
    return [_turn(s["q"], c, n, case["rot"], case["layout"]), _turn(s["k"], c, n, case["rot"], case["layout"])]


def _places(s, T):
    """(request, position) of each new row"""
    row = torch.arange(T, device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), row, right=True)
    return b, s["lens"].long()[b] - (s["cu"].long()[b + 1] - row)


def _plain_append(s):
    case, cache, T = s["case"], s["cache"], s["k"].shape[0]
    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    NG = D // 64
    b, pos = _places(s, T)
    where = s["table"].long()[b, pos // page]
    off = pos % page
    raw = cache.view(cache.shape[0], Hkv, page // 16, 18 * D)
    tile, row = off // 16, off % 16
    heads = torch.arange(Hkv, device="cuda")
    at = lambda byte: (where[:, None, None], heads[None, :, None], tile[:, None, None], byte[:, None, :])  # noqa: E731
    (kq, ks, ko), (vq, vs, vo) = _quantize(s["k"].float()), _quantize(s["v"].float())
    kq = kq.to(torch.uint8).view(T, Hkv, NG, 4, 2, 8).permute(0, 1, 3, 2, 4, 5).reshape(T, Hkv, D // 2, 2)
    vq = vq.to(torch.uint8).view(T, Hkv, NG, 8, 2, 4).permute(0, 1, 3, 2, 4, 5).reshape(T, Hkv, D // 4, 2, 2)
    raw[at(row[:, None] * (D // 2) + torch.arange(D // 2, device="cuda"))] = kq[..., 0] | kq[..., 1] << 4
    word = (row // 2)[:, None] * D + (row % 2)[:, None] * 2 + 4 * torch.arange(D // 4, device="cuda")
    vb = vq[..., 0] | vq[..., 1] << 4
    raw[at(8 * D + word)] = vb[..., 0]
    raw[at(8 * D + word + 1)] = vb[..., 1]
    scale = row[:, None] * 4 * NG + torch.arange(4 * NG, device="cuda")
    raw[at(16 * D + scale)] = torch.stack((ks, ko), -1).reshape(T, Hkv, -1).view(torch.uint8)
    raw[at(16 * D + 64 * NG + scale)] = torch.stack((vs, vo), -1).reshape(T, Hkv, -1).view(torch.uint8)
    # read the new tokens back from the cache
    k, v, ks, vs = _unpack(raw[where, :, tile].reshape(T * Hkv, 18 * D), D)
    mine = (torch.arange(T * Hkv, device="cuda"), row.repeat_interleave(Hkv))
    spread = lambda q, sc: (q[mine].view(T, Hkv, NG, 64).float() * sc[mine].view(T, Hkv, NG, 2)[..., :1].float()  # noqa: E731
                            + sc[mine].view(T, Hkv, NG, 2)[..., 1:].float()).view(T, Hkv, D).to(BF16)
    return [spread(k, ks), spread(v, vs)]


def _plain_attn(s):
    case, cache, q = s["case"], s["cache"], s["q"]
    B, H, Hkv, D, page = case["B"], case["H"], case["Hkv"], case["D"], case["page"]
    G, NG, L, most, T = H // Hkv, D // 64, s["wide"] * case["page"], s["most"], q.shape[0]
    got = cache[s["table"].long().clamp(min=0)]  # [B, pages, Hkv, page, bytes]
    k, v, ks, vs = _unpack(got.view(-1, 18 * D), D)
    del got

    def spread(c, sc):
        w = c.view(-1, 16, NG, 64).float() * sc[..., :1].float() + sc[..., 1:].float()
        return w.view(B, s["wide"], Hkv, page, D).transpose(1, 2).reshape(B, Hkv, L, D)

    k, v = spread(k, ks), spread(v, vs)
    b, pos = _places(s, T)
    i = torch.arange(T, device="cuda") - s["cu"].long()[b]
    at = torch.full((B, most), -1, device="cuda", dtype=torch.long)
    at[b, i] = pos
    qq = torch.zeros(B, most, H, D, device="cuda")
    qq[b, i] = q.float()
    qq = qq.view(B, most, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, most * G, D)
    score = torch.matmul(qq, k.transpose(-1, -2)).view(B, Hkv, most, G, L) * D ** -0.5
    j = torch.arange(L, device="cuda")
    seen = j <= at[..., None]
    if case["window"]:
        seen = seen & ((j > at[..., None] - case["window"]) | (j < case["sinks"]))
    score = score.masked_fill(~seen[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    p = (p / p.sum(-1, keepdim=True).clamp(min=1e-30)).view(B, Hkv, most * G, L)
    o = torch.matmul(p, v).view(B, Hkv, most, G, D).permute(0, 2, 1, 3, 4).reshape(B, most, H, D)
    return o[b, i].to(BF16)


# -------------------------------------------------------------------------------------- the framework's

def _own(s):
    from w4a8_quantized_gemm_token_b200 import binding as qk

    case = s["case"]
    if case["op"] == "norm":
        h, codes, scale, sums = qk.qk_rmsnorm_quantize(s["x"], s["weight"], s["residual"], eps=1e-6,
                                                       with_xsum=case["xsum"])
        return {"h": h, "values": codes * scale[:, None], "scale": scale, "sums": sums}
    if case["op"] == "rope":
        layout = qk.QK_ROPE_HALF if case["layout"] == "half" else qk.QK_ROPE_INTERLEAVED
        return list(qk.qk_rope(s["q"], s["k"], s["positions"], s["freq"], layout=layout, amplitude=s["amplitude"]))
    if case["op"] == "append":
        qk.qk_kv4_append(s["k"], s["v"], s["cache"], s["table"], s["lens"], s["cu"])
        return list(qk.qk_kv4_gather(s["cache"], s["table"], s["lens"], s["cu"], s["k"].shape[0]))
    return qk.qk_kv4_attention(s["q"], s["cache"], s["table"], s["lens"], s["cu"], window=case["window"],
                               sinks=case["sinks"])


def run(s):
    if own:
        return _own(s)
    return {"norm": _plain_norm, "rope": _plain_rope, "append": _plain_append, "attn": _plain_attn}[s["case"]["op"]](s)


# ------------------------------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "norm":
        n = case["M"] * case["K"]
        return {"bytes": n * (7 if case["residual"] else 3) + 4 * case["M"] + (4 * case["K"] if case["weight"] else 0)
                + (n // 16 if case["xsum"] else 0), "flops": 8 * n}
    if op == "rope":
        n = case["T"] * (case["H"] + case["Hkv"])
        return {"bytes": n * case["D"] * 4 + 4 * case["T"] + 4 * case["rot"], "flops": 3 * n * case["rot"]}
    past, new = _lengths(case)
    D, Hkv = case["D"], case["Hkv"]
    if op == "append":  # rows read, records written, and read back into rows
        n = int(new.sum()) * Hkv
        return {"bytes": n * (2 * 4 * D + 2 * (D + D // 8)), "flops": 16 * n * D}
    tokens = pairs = 0
    for a, n in zip(past.tolist(), new.tolist()):
        w, k = case["window"] or a + n, case["sinks"]
        low = max(0, a + 1 - w)  # the first key that the first new token's window holds
        tokens += a + n - low + min(low, k)
        i = np.arange(a, a + n)
        first = np.maximum(0, i + 1 - w)
        pairs += int((i + 1 - first + np.minimum(first, k)).sum())
    return {"bytes": tokens * Hkv * (D + D // 8) + 4 * int(new.sum()) * case["H"] * D,
            "flops": 4 * pairs * case["H"] * D}


# ------------------------------------------------------------------------------------------------ exact

def exact(case, seed):
    """From the definitions, in 64 bits.  Codes are decided as the definition says: from products and
    quotients that are rounded to fp32 (or fp16) one by one."""
    s = prepare({**case}, seed)
    to32 = lambda t: t.to(F32).to(F64)  # noqa: E731
    if case["op"] == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = (h + s["residual"].double()).to(BF16).double()
        u = h if s["weight"] is None else to32(h * s["weight"].double())
        top = u.abs().max(dim=1).values
        live = top > 0
        factor = to32(127.0 / torch.where(live, top, torch.ones_like(top)))
        codes = torch.clamp(torch.round(to32(u * factor[:, None])), -127, 127)
        rms = torch.sqrt(torch.sum(h ** 2, dim=1) / case["K"] + 1e-6)
        scale = torch.where(live, top / (127.0 * rms), torch.ones_like(top))
        sums = codes.reshape(case["M"], case["K"] // 64, 64).sum(2).to(torch.int32) if case["xsum"] else None
        return {"h": h if s["residual"] is not None else None, "values": codes * scale[:, None], "scale": scale,
                "sums": sums}
    if case["op"] == "rope":
        out, rot = [], case["rot"]
        for x in (s["q"], s["k"]):
            y = x.double().clone()
            for i in range(rot // 2):
                m, n = (i, i + rot // 2) if case["layout"] == "half" else (2 * i, 2 * i + 1)
                turn = torch.remainder(s["positions"].double() * s["freq"][i], 1.0) * (2.0 * math.pi)
                z = torch.polar(torch.full_like(turn, float(s["amplitude"])), turn)[:, None]
                w = torch.complex(x[..., m].double(), x[..., n].double()) * z
                y[..., m], y[..., n] = w.real, w.imag
            out.append(y)
        return out
    D, Hkv, page = case["D"], case["Hkv"], case["page"]
    NG = D // 64
    if case["op"] == "append":
        out = []
        for x in (s["k"], s["v"]):
            y = torch.empty(x.shape, dtype=F64, device="cuda")
            for g in range(NG):
                w = x[..., 64 * g:64 * g + 64].double()
                low, high = w.min(-1, keepdim=True).values, w.max(-1, keepdim=True).values
                scale = to32(to32(high - low) / 15.0).to(torch.float16).double()
                base = low.to(torch.float16).double()
                inv = to32(1.0 / torch.where(scale > 0, scale, torch.ones_like(scale)))
                q = torch.clamp(torch.round(to32(to32(w - base) * inv)), 0, 15)
                y[..., 64 * g:64 * g + 64] = torch.where(scale > 0, q * scale, torch.zeros_like(q)) + base
            out.append(y)
        return out
    # byte and shift of every (token of a record, dim)
    d, r = torch.arange(D, device="cuda")[None, :], torch.arange(16, device="cuda")[:, None]
    g, e = d // 64, d % 64
    kbyte = r * (D // 2) + (e // 16) * 8 * NG + g * 8 + (e % 16) // 2
    vbyte = 8 * D + (r // 2) * D + (e // 8) * 8 * NG + g * 8 + ((e % 8) // 4) * 4 + (r % 2) * 2 + (e % 4) // 2
    shift = (d % 2) * 4
    G, out = case["H"] // Hkv, torch.zeros(s["q"].shape, dtype=F64, device="cuda")
    table, lens, cu = s["table"].cpu().numpy(), s["lens"].cpu().numpy(), s["cu"].cpu().numpy()
    for b in range(case["B"]):
        n, first = int(lens[b]), int(cu[b])
        new = int(cu[b + 1]) - first
        used = torch.from_numpy(table[b, :-(-n // page)].astype(np.int64)).cuda()
        rec = s["cache"][used].reshape(len(used), Hkv, page // 16, 18 * D)
        pos = torch.arange(n - new, n, device="cuda")
        key = torch.arange(len(used) * page, device="cuda")
        hidden = key[None, :] > pos[:, None]
        if case["window"]:
            hidden |= (key[None, :] <= pos[:, None] - case["window"]) & (key[None, :] >= case["sinks"])
        for h in range(Hkv):
            one = rec[:, h].reshape(-1, 18 * D)
            scales = one[:, 16 * D:].contiguous().view(torch.float16).double().reshape(-1, 2, 16, NG, 2)
            kv = []
            for which, byte in enumerate((kbyte, vbyte)):
                code = torch.bitwise_and(torch.bitwise_right_shift(one[:, byte], shift.to(torch.uint8)), 15).double()
                part = scales[:, which].repeat_interleave(64, dim=2)
                kv.append((code * part[..., 0] + part[..., 1]).reshape(-1, D))
            x = s["q"][first:first + new, h * G:h * G + G].double()
            a = torch.einsum("igd,jd->gij", x, kv[0]) / math.sqrt(D)
            a = torch.softmax(a.masked_fill(hidden, -math.inf), -1)
            out[first:first + new, h * G:h * G + G] = torch.einsum("gij,jd->igd", a, kv[1])
    return out
