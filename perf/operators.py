"""The operators around the attention kernels: what each computes in plain torch, and the calls a user makes.

Query / key norm with position rotation (forward and backward), the page plan of a paged key-value cache, the append
of keys and values to a cache held in 4 bits, attention over that cache, and its read-back as bf16.

The cache is uint8 [pages, H_kv, page_size / 16, 18 d]: one row of 18 d bytes holds 16 consecutive tokens of one head,
as e2m1 codes (two per byte, the even column in the low half) and one e4m3 scale per 16 columns:
  bytes 0 .. 8d      K codes, [key 16][d / 2]
  bytes 8d .. 16d    V codes, [t 2][g 8][c 4][p 2][d / 16]: key 8 t + 2 c + p, columns g d/8 .. (g + 1) d/8
  bytes 16d .. 17d   K scales, [key mod 8][column / 16][key / 8]
  bytes 17d .. 18d   V scales, [column / 16][c 4][t 2][p 2]
"""
import math
import random

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step of 48 requests: q and k are views of the fused projection's rows
        {"name": "norm_rope_decode", "op": "norm", "dir": "fwd", "B": 1, "N": 48, "H": 32, "Hkv": 8, "d": 128, "rot": 128,
         "inter": False, "wtype": "bf16", "packed": True, "maxpos": 32768},
        # prompts of a GPT layer, written in the attention kernels' [B, H, N, d] layout
        {"name": "norm_rope_prefill", "op": "norm", "dir": "fwd", "B": 4, "N": 1023, "H": 16, "Hkv": 16, "d": 64, "rot": 32,
         "inter": True, "wtype": "fp32", "packed": False, "maxpos": 4096},
        # the gradient of the long training sequence
        {"name": "norm_rope_bwd_long", "op": "norm", "dir": "bwd", "B": 1, "N": 16384, "H": 32, "Hkv": 8, "d": 128, "rot": 128,
         "inter": False, "wtype": "bf16", "packed": False, "maxpos": 16384},
        # one new token for each of 64 running requests
        {"name": "plan_decode", "op": "plan", "B": 64, "ctx": 8192, "new": 1, "page": 64},
        # many prompt chunks of uneven length, some requests with a history
        {"name": "plan_prefill", "op": "plan", "B": 333, "ctx": 3000, "new": 777, "page": 16},
        # one new token for each of 64 requests
        {"name": "append_decode", "op": "append", "T": 64, "Hkv": 8, "d": 128, "page": 64, "kg": 1.0, "vg": 1.0},
        # a long prompt
        {"name": "append_prefill", "op": "append", "T": 16385, "Hkv": 8, "d": 128, "page": 16, "kg": 1.0, "vg": 0.5},
        # one request, short history: latency
        {"name": "attn_one", "op": "attn", "B": 1, "ctx": 1000, "nq": 1, "H": 32, "Hkv": 8, "d": 128, "page": 64, "causal": True},
        # 48 running requests of uneven length
        {"name": "attn_batch", "op": "attn", "B": 48, "ctx": 8191, "nq": 1, "H": 32, "Hkv": 8, "d": 128, "page": 64, "causal": True},
        # two long requests, four proposed tokens each
        {"name": "attn_long", "op": "attn", "B": 2, "ctx": 131072, "nq": 4, "H": 16, "Hkv": 4, "d": 128, "page": 128, "causal": True},
        # the history of prompt chunks, read back for the packed attention
        {"name": "gather_chunk", "op": "gather", "B": 7, "ctx": 4097, "Hkv": 8, "d": 128, "page": 64, "kg": 1.0, "vg": 1.0},
        {"name": "gather_small", "op": "gather", "B": 3, "ctx": 300, "Hkv": 4, "d": 64, "page": 16, "kg": 2.0, "vg": 1.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "plan", "append", "attn", "attn", "attn", "gather"])
    d = rng.choice([16, 32, 64, 64, 128, 128])
    hkv = rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "norm":
        b = _log(rng, 1, 8)
        group = rng.choice([1, 2, 4, 5])
        n = _log(rng, 1, max(1, 40_000_000 // (b * hkv * (group + 1) * d)))
        n = min(n, 16384)
        packed = rng.random() < 0.5
        return {"op": "norm", "dir": rng.choice(["fwd", "bwd"]), "B": 1 if packed else b, "N": b * n if packed else n, "H": hkv * group,
                "Hkv": hkv, "d": d, "rot": rng.choice([d, max(16, d // 2)]), "inter": rng.random() < 0.5,
                "wtype": rng.choice(["bf16", "fp32"]), "packed": packed, "maxpos": max(b * n, 1024)}
    if op == "plan":
        return {"op": "plan", "B": _log(rng, 1, 600), "ctx": _log(rng, 1, 9000), "new": _log(rng, 1, 400), "page": page}
    if op == "append":
        return {"op": "append", "T": _log(rng, 1, 16000), "Hkv": hkv, "d": d, "page": page, "kg": rng.choice([0.25, 1.0, 2.0]),
                "vg": rng.choice([0.5, 1.0])}
    if op == "gather":
        return {"op": "gather", "B": _log(rng, 1, 16), "ctx": _log(rng, 1, 4000), "Hkv": hkv, "d": d, "page": page,
                "kg": rng.choice([1.0, 4.0]), "vg": rng.choice([0.5, 1.0])}
    b, nq, group = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 5]), rng.choice([1, 2, 4, 6, 8, 16])
    ctx = _log(rng, 1, min(100_000, 1_500_000 // (b * hkv * max(1, nq * group // 16))))
    return {"op": "attn", "B": b, "ctx": ctx, "nq": nq, "H": hkv * group, "Hkv": hkv, "d": d, "page": page, "causal": rng.random() < 0.8}


def _lengths(case, most):
    """The requests' lengths: from the case alone, uneven, the first at the maximum."""
    r = random.Random("%s %d %d" % (case["op"], case["B"], most))
    return [most] + [r.randint(max(1, most // 4), most) for _ in range(case["B"] - 1)]


def _plan_lengths(case):
    r = random.Random("plan %d %d %d" % (case["B"], case["ctx"], case["new"]))
    old = [r.choice([0, r.randint(0, case["ctx"])]) if case["new"] > 1 else r.randint(0, case["ctx"]) for _ in range(case["B"])]
    new = [r.randint(0, case["new"]) if case["new"] > 1 else 1 for _ in range(case["B"])]
    new[0] = case["new"]
    return old, new


def _pages(n, page):
    return -(-n // page)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _random_cache(g, pages, hkv, page, d):
    """A filled cache: codes as normal values scaled to a group's maximum have them, scales from 0.2 to 0.7."""
    shape = (pages, hkv, page // 16)
    # how often each magnitude occurs among normal values whose group's largest is 6
    often = np.array([0.10, 0.19, 0.17, 0.14, 0.17, 0.12, 0.07, 0.04])
    lut = np.repeat(np.arange(8), np.round(often * 128).astype(int))
    lut = np.resize(lut, 128)
    lut = torch.tensor(np.concatenate([lut, lut + 8]), dtype=torch.uint8, device="cuda")
    out = torch.empty(shape + (18 * d,), dtype=torch.uint8, device="cuda")
    for i in range(0, pages, 1024):  # in parts: the indices are eight times the bytes
        part = out[i:i + 1024]
        r = torch.randint(0, 256, (2,) + tuple(part.shape[:3]) + (16 * d,), generator=g, device="cuda", dtype=torch.uint8).int()
        part[..., :16 * d] = lut[r[0]] | (lut[r[1]] << 4)
        part[..., 16 * d:] = torch.randint(0x26, 0x34, tuple(part.shape[:3]) + (2 * d,), generator=g, device="cuda", dtype=torch.uint8)
    return out


def _paged(g, lens, case, spare=3):
    """A cache and the block table of requests whose pages are spread over it."""
    counts = [_pages(n, case["page"]) for n in lens]
    total = sum(counts) + spare
    order = torch.randperm(total, generator=g, device="cuda").int()
    width = max(max(counts), 1)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    order, at = order.cpu(), 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    return _random_cache(g, total, case["Hkv"], case["page"], case["d"]), table.cuda()


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    if case["op"] == "norm":
        b, n, h, hkv, d, rot = (case[k] for k in ("B", "N", "H", "Hkv", "d", "rot"))
        # the fused projection's output: a token's query, key and value heads side by side; some channels are larger
        qkv = randn(b, n, h + 2 * hkv, d) * (1 + 2 * (torch.rand(d, generator=g, device="cuda") > 0.95).float())
        qkv = qkv.to(torch.bfloat16)
        q, k = qkv[:, :, :h], qkv[:, :, h:h + hkv]
        if case["packed"]:
            s["q"], s["k"] = q[0], k[0]
            s["positions"] = torch.randint(0, case["maxpos"], (n,), generator=g, device="cuda", dtype=torch.int32)
        else:
            s["q"], s["k"] = q.transpose(1, 2), k.transpose(1, 2)
            s["positions"] = None
        wt = torch.bfloat16 if case["wtype"] == "bf16" else torch.float32
        s["wq"], s["wk"] = ((1 + 0.2 * randn(d)).to(wt) for _ in range(2))
        angle = torch.arange(case["maxpos"], device="cuda", dtype=torch.float64)[:, None] * (
            10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot))[None]
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        if case["dir"] == "bwd":  # as the attention's backward pass writes them
            s["dq"], s["dk"] = ((randn(*t.shape)).to(torch.bfloat16) for t in (s["q"], s["k"]))
    elif case["op"] == "plan":
        old, new = _plan_lengths(case)
        page = case["page"]
        width = max(_pages(o + n, page) for o, n in zip(old, new)) + 1
        need = sum(_pages(o + n, page) for o, n in zip(old, new))
        order = torch.randperm(need + 16, generator=g, device="cuda").int().cpu()
        table, at = torch.full((case["B"], width), -1, dtype=torch.int32), 0
        for b, o in enumerate(old):
            c = _pages(o, page)
            table[b, :c] = order[at:at + c]
            at += c
        s["old"], s["new"] = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (old, new))
        s["free"], s["table"] = order[at:].cuda(), table.cuda()
        s["most"] = sum(new) + 5  # rounded up, as a captured step's would be
    elif case["op"] == "append":
        t, hkv, d, page = (case[k] for k in ("T", "Hkv", "d", "page"))
        big = 1 + 3 * (torch.rand(d, generator=g, device="cuda") > 0.95).float()
        s["k"] = (randn(t, hkv, d) * big * case["kg"]).to(torch.bfloat16)
        s["v"] = (randn(t, hkv, d) * case["vg"]).to(torch.bfloat16)
        pages = _pages(t, page) + 2
        s["cache"] = torch.zeros((pages, hkv, page // 16, 18 * d), dtype=torch.uint8, device="cuda")
        s["slots"] = torch.randperm(pages * page, generator=g, device="cuda")[:t] if t < 1000 else torch.arange(t, device="cuda") + page
    else:
        lens = _lengths(case, case["ctx"])
        s["cache"], s["table"] = _paged(g, lens, case)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        if case["op"] == "gather":
            s["cu"] = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
            s["total"] = sum(lens)
        else:
            s["q"] = (randn(case["B"] * case["nq"], case["H"], case["d"]) * 1.5).to(torch.bfloat16)
            s["cu_q"] = None  # one token each
            if case["nq"] > 1:
                s["cu_q"] = torch.arange(0, case["B"] * case["nq"] + 1, case["nq"], dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    if own:
        import tiled_exact_attention_fa2_gb300 as fa2

        if case["op"] == "norm":
            if case["dir"] == "fwd":
                return fa2.fa2_qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["rope"], s["positions"], eps=1e-6, interleaved=case["inter"])
            return fa2.fa2_qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], s["rope"], s["positions"], eps=1e-6,
                                            interleaved=case["inter"])
        if case["op"] == "plan":
            p = fa2.fa2_page_plan(s["old"], s["new"], s["free"], s["table"], case["page"], s["most"])
            return [s["table"], p.lens, p.cu_new, p.cu_total, p.slots, p.positions, p.pages_needed]
        if case["op"] == "append":
            k, v = torch.empty_like(s["k"]), torch.empty_like(s["v"])
            fa2.fa2_kv4_append(s["k"], s["v"], s["cache"], s["slots"], k_scale=case["kg"], v_scale=case["vg"], k_out=k, v_out=v)
            return [k, v, s["cache"]]
        if case["op"] == "gather":
            return fa2.fa2_kv4_gather(s["cache"], s["table"], s["cu"], s["total"], k_scale=case["kg"], v_scale=case["vg"])
        return fa2.fa2_kv4_attn(s["q"], s["cache"], s["table"], s["lens"], cu_seqlens_q=s["cu_q"], max_seqlen_q=case["nq"], causal=case["causal"])
    return {"norm": _norm, "plan": _plan, "append": _append, "gather": _gather, "attn": _attn}[case["op"]](s)


# ------------------------------------------------------------------ plain forms
def _table_rows(s, n):
    at = s["positions"].long() if s["positions"] is not None else torch.arange(n, device="cuda")
    half = s["rope"].shape[1] // 2
    c, sn = s["rope"][at, :half], s["rope"][at, half:]
    return (c[:, None], sn[:, None]) if s["positions"] is not None else (c[None, None], sn[None, None])


def _rotate(y, c, sn, inter, back):
    half = c.shape[-1]
    a, b = (y[..., 0:2 * half:2], y[..., 1:2 * half:2]) if inter else (y[..., :half], y[..., half:2 * half])
    sn = -sn if back else sn
    p, q = a * c - b * sn, b * c + a * sn
    mixed = torch.stack([p, q], -1).flatten(-2) if inter else torch.cat([p, q], -1)
    return torch.cat([mixed, y[..., 2 * half:]], -1)


def _norm(s):
    case = s["case"]
    c, sn = _table_rows(s, case["N"])
    outs, grads = [], []
    names = (("q", "wq", "dq"), ("k", "wk", "dk"))
    one, two = (_norm_one(s, c, sn, *names[i]) for i in range(2))
    outs, grads = [one[0], two[0]], [one[1], two[1]]
    return outs if case["dir"] == "fwd" else outs + grads


def _norm_one(s, c, sn, x, w, dx):
    case = s["case"]
    x, w = s[x].float(), s[w].float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    if case["dir"] == "fwd":
        return _rotate(x * r * w, c, sn, case["inter"], False).to(torch.bfloat16).contiguous(), None
    gy = _rotate(s[dx].float(), c, sn, case["inter"], True)
    xn = x * r
    h = gy * w
    grad = r * (h - xn * (h * xn).mean(-1, keepdim=True))
    return grad.to(torch.bfloat16), (gy * xn).sum(tuple(range(x.dim() - 1)))


def _plan(s):
    page, old, new, table = s["case"]["page"], s["old"].long(), s["new"].long(), s["table"]
    zero = torch.zeros(1, dtype=torch.long, device="cuda")
    lens = old + new
    cu_new, cu_total = torch.cat([zero, new.cumsum(0)]), torch.cat([zero, lens.cumsum(0)])
    have, want = (old + page - 1) // page, (lens + page - 1) // page
    first = torch.cat([zero, (want - have).cumsum(0)])
    col = torch.arange(table.shape[1], device="cuda")[None]
    fresh = (col >= have[:, None]) & (col < want[:, None])
    at = (first[:-1, None] + col - have[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][at], table)
    t = torch.arange(s["most"], device="cuda")
    b = torch.searchsorted(cu_new[1:].contiguous(), t, right=True).clamp(max=old.numel() - 1)
    real = t < cu_new[-1]
    pos = torch.where(real, old[b] + t - cu_new[b], 0)
    slots = torch.where(real, table[b, pos // page].long() * page + pos % page, -1)
    i32 = torch.int32
    return [table, lens.to(i32), cu_new.to(i32), cu_total.to(i32), slots, pos.to(i32), first[-1:].to(i32)]


def _quantize(x, g):
    """Codes (0 to 15), scale bytes and the values they stand for, of [..., d] in groups of 16 columns."""
    y = (x.float() / g).unflatten(-1, (-1, 16))
    scale = (y.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = scale.float()[..., None]
    u = torch.where(sf > 0, y / sf, 0.0)
    a = u.abs()
    # round to the nearest of E2M1, ties to the even code
    mag = (a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int()
    code = mag + 8 * (torch.signbit(u)).int()
    value = torch.tensor(E2M1, device="cuda")[mag] * torch.where(torch.signbit(u), -1.0, 1.0) * sf * g
    return code.flatten(-2), scale.view(torch.uint8), value.flatten(-2).to(torch.bfloat16)


def _append(s):
    case, cache = s["case"], s["cache"]
    d, page = case["d"], case["page"]
    slot = s["slots"].long()
    at, key = slot // page, slot % page
    tile, key = key // 16, key % 16
    head = torch.arange(case["Hkv"], device="cuda")[None, :, None]
    at, tile, key = at[:, None, None], tile[:, None, None], key[:, None, None]
    kc, ks, kv = _quantize(s["k"], case["kg"])
    vc, vs, vv = _quantize(s["v"], case["vg"])
    byte = torch.arange(d // 2, device="cuda")[None, None]
    grp = torch.arange(d // 16, device="cuda")[None, None]
    t, c, p = key // 8, key % 8 // 2, key % 2
    piece = d // 16
    cache[at, head, tile, key * (d // 2) + byte] = (kc[..., 0::2] | kc[..., 1::2] << 4).to(torch.uint8)
    cache[at, head, tile, 8 * d + (((t * 8 + byte // piece) * 4 + c) * 2 + p) * piece + byte % piece] = (vc[..., 0::2] | vc[..., 1::2] << 4).to(torch.uint8)
    cache[at, head, tile, 16 * d + ((key % 8) * (d // 16) + grp) * 2 + t] = ks
    cache[at, head, tile, 17 * d + (grp * 4 + c) * 4 + t * 2 + p] = vs
    return [kv, vv, cache]


def _values(tiles, d):
    """fp32 K and V [..., 16, d] of tiles [..., 18 d]."""
    lead, ng = tiles.shape[:-1], d // 16
    lut = torch.tensor(E2M1, device="cuda")
    lut = torch.cat([lut, -lut])
    byte = torch.arange(256, device="cuda")
    pair = torch.stack([lut[byte % 16], lut[byte // 16]], -1)
    f8 = lambda x: x.contiguous().view(torch.float8_e4m3fn).float()  # noqa: E731
    n = len(lead)
    front = tuple(range(n))
    k = pair[tiles[..., :8 * d].int()].reshape(*lead, 16, ng, 16)
    ks = f8(tiles[..., 16 * d:17 * d]).reshape(*lead, 8, ng, 2).permute(*front, n + 2, n, n + 1).reshape(*lead, 16, ng, 1)
    v = pair[tiles[..., 8 * d:16 * d].int()].reshape(*lead, 2, 8, 4, 2, d // 8).permute(*front, n, n + 2, n + 3, n + 1, n + 4).reshape(*lead, 16, ng, 16)
    vs = f8(tiles[..., 17 * d:]).reshape(*lead, ng, 4, 2, 2).permute(*front, n + 2, n + 1, n + 3, n).reshape(*lead, 16, ng, 1)
    return (k * ks).reshape(*lead, 16, d), (v * vs).reshape(*lead, 16, d)


def _gather(s):
    case = s["case"]
    page, t = case["page"], torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(s["cu"][1:].contiguous(), t, right=True)
    pos = t - s["cu"][b]
    at = s["table"][b, pos // page].long()
    k, v = _values(s["cache"], case["d"])
    k, v = (x.flatten(2, 3)[at, :, pos % page] for x in (k, v))
    return [(k * case["kg"]).to(torch.bfloat16), (v * case["vg"]).to(torch.bfloat16)]


def _attn(s):
    case = s["case"]
    b, nq, h, hkv, d = (case[k] for k in ("B", "nq", "H", "Hkv", "d"))
    tiles = s["cache"][s["table"].clamp(min=0).long()]  # [B, pages, H_kv, page / 16, 18 d]
    k, v = _values(tiles, d)
    k, v = (x.flatten(3, 4).transpose(1, 2).flatten(2, 3) for x in (k, v))  # [B, H_kv, keys, d]
    q = s["q"].float().view(b, nq, hkv, h // hkv, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, nq * (h // hkv), d)
    key = torch.arange(k.shape[2], device="cuda")
    last = s["lens"][:, None].long() - 1 + torch.zeros(nq, device="cuda", dtype=torch.long)
    last = last - (nq - 1) + torch.arange(nq, device="cuda") if case["causal"] else last
    seen = key <= last[..., None]  # [B, nq, keys]
    seen = seen[:, None, :, None].expand(b, hkv, nq, h // hkv, key.numel()).reshape(b, hkv, nq * (h // hkv), -1)
    inside = (key < s["lens"][:, None])[:, None, :, None]
    x = torch.where(seen, (q @ torch.where(inside, k, 0.0).transpose(2, 3)) / math.sqrt(d), -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True)
    o = torch.where(total > 0, (e @ torch.where(inside, v, 0.0)) / total, 0.0)
    lse = (m + total.log()).squeeze(-1)
    o = o.view(b, hkv, nq, h // hkv, d).permute(0, 2, 1, 3, 4).reshape(b * nq, h, d)
    lse = lse.view(b, hkv, nq, h // hkv).permute(1, 3, 0, 2).reshape(h, b * nq)
    return [o.to(torch.bfloat16), lse]


# ------------------------------------------------------------------ bytes and operations
def work(case):
    op = case["op"]
    if op == "norm":
        rows = case["B"] * case["N"] * (case["H"] + case["Hkv"])
        tensors = 2 if case["dir"] == "fwd" else 3
        tokens = case["B"] * case["N"] if case["packed"] else case["N"]
        w = (2 if case["wtype"] == "bf16" else 4) * 2 * case["d"] + (0 if case["dir"] == "fwd" else 8 * case["d"])
        return {"bytes": rows * case["d"] * 2 * tensors + min(tokens, case["maxpos"]) * case["rot"] * 4 + w + (4 * tokens if case["packed"] else 0),
                "flops": rows * case["d"] * (8 if case["dir"] == "fwd" else 16)}
    if op == "plan":
        old, new = _plan_lengths(case)
        t, b = sum(new), case["B"]
        fresh = sum(_pages(o + n, case["page"]) - _pages(o, case["page"]) for o, n in zip(old, new))
        return {"bytes": 8 * b + 8 * fresh + 12 * (t + 5) + 12 * b + 12, "flops": 4 * t + 6 * b}
    if op == "append":
        n = case["T"] * case["Hkv"] * case["d"]
        # read 2 x 2 bytes, write the codes and scales (2 x 9/16) and the values (2 x 2)
        return {"bytes": n * 4 + n * 9 // 8 + n * 4 + 8 * case["T"], "flops": n * 2 * 4}
    lens = _lengths(case, case["ctx"])
    keys = sum(lens)
    held = keys * case["Hkv"] * case["d"] * 9 // 8
    if op == "gather":
        return {"bytes": held + keys * case["Hkv"] * case["d"] * 4, "flops": keys * case["Hkv"] * case["d"] * 2}
    rows = case["B"] * case["nq"] * case["H"]
    return {"bytes": held + rows * (case["d"] * 4 + 4), "flops": 4 * case["d"] * keys * case["nq"] * case["H"]}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "plan": _exact_plan, "append": _exact_append, "gather": _exact_gather, "attn": _exact_attn}[case["op"]](s)


def _exact_norm(s):
    """A rotation is multiplication by a complex number of modulus one; the gradient by the definition, row by row."""
    case = s["case"]
    half = case["rot"] // 2
    rope = s["rope"].double()
    turn = torch.complex(rope[:, :half], rope[:, half:])
    turn = turn[s["positions"].long()].unsqueeze(1) if case["packed"] else turn[:case["N"]]

    def spin(y, z):
        y = y.clone()
        a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["inter"] else (slice(0, half), slice(half, 2 * half))
        u = torch.complex(y[..., a].contiguous(), y[..., b].contiguous()) * z
        y[..., a], y[..., b] = u.real, u.imag
        return y

    first, second = [], []
    for x, w, dx in ((s["q"], s["wq"], s.get("dq")), (s["k"], s["wk"], s.get("dk"))):
        x, w = x.double(), w.double()
        rms = ((x ** 2).sum(-1, keepdim=True) / case["d"] + 1e-6).sqrt()
        if case["dir"] == "fwd":
            first.append(spin(w * x / rms, turn))
            continue
        back = spin(dx.double(), turn.conj())
        second.append((back * x / rms).flatten(0, -2).sum(0))
        along = (back * w * x).sum(-1, keepdim=True) / case["d"]
        first.append(back * w / rms - x * along / rms ** 3)
    return first + second


def _exact_plan(s):
    page, old, new = s["case"]["page"], s["old"].tolist(), s["new"].tolist()
    table, free = s["table"].cpu().clone(), s["free"].tolist()
    taken, slots, places, cu_new, cu_total = 0, [], [], [0], [0]
    for b, (o, n) in enumerate(zip(old, new)):
        for pos in range(o, o + n):
            if pos % page == 0:
                table[b, pos // page] = free[taken]
                taken += 1
            slots.append(int(table[b, pos // page]) * page + pos % page)
            places.append(pos)
        cu_new.append(cu_new[-1] + n)
        cu_total.append(cu_total[-1] + o + n)
    pad = s["most"] - len(slots)
    lens = torch.tensor([o + n for o, n in zip(old, new)], dtype=torch.int32)
    return [table, lens, torch.tensor(cu_new, dtype=torch.int32), torch.tensor(cu_total, dtype=torch.int32), torch.tensor(slots + [-1] * pad),
            torch.tensor(places + [0] * pad, dtype=torch.int32), torch.tensor([taken], dtype=torch.int32)]


def _exact_append(s):
    """Every scale and value by looking for the nearest one there is (of two as near, the one with the even code)."""
    small = [m * 2.0 ** -9 for m in range(8)]
    scales = np.array(small + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:119])  # codes 0 .. 126

    def nearest(x, there):
        hi = np.clip(np.searchsorted(there, x), 1, len(there) - 1)
        lo = hi - 1
        below, above = x - there[lo], there[hi] - x
        return np.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)

    def one(x, g):
        y = x.double().cpu().numpy().reshape(*x.shape[:-1], -1, 16) / g
        step = scales[nearest(np.abs(y).max(-1, keepdims=True) / 6, scales)]
        held = np.array(E2M1)
        u = np.divide(np.abs(y), step, out=np.zeros_like(y), where=step > 0)
        return torch.from_numpy((np.sign(y) * held[nearest(u, held)] * step * g).reshape(x.shape))

    return [one(s["k"], s["case"]["kg"]), one(s["v"], s["case"]["vg"]), None]


def _exact_tiles(tiles, d):
    """K and V of tiles [n, 18 d], column by column from the byte that holds each."""
    codes = np.array(list(E2M1) + [-x for x in E2M1])
    e, m = np.arange(256) >> 3 & 15, np.arange(256) & 7
    scale = np.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7), m * 2.0 ** -9) * np.where(np.arange(256) > 127, -1, 1)
    codes, scale = (torch.tensor(x, dtype=torch.float64, device=tiles.device) for x in (codes, scale))
    key, col = (x.to(tiles.device) for x in torch.meshgrid(torch.arange(16), torch.arange(d), indexing="ij"))
    t, c, p, per = key // 8, key % 8 // 2, key % 2, d // 8
    kb = key * (d // 2) + col // 2
    vb = 8 * d + ((t * 32 + (col // per) * 4 + c) * 2 + p) * (per // 2) + (col % per) // 2
    sk = 16 * d + (key % 8) * (d // 8) + (col // 16) * 2 + t
    sv = 17 * d + (col // 16) * 16 + c * 4 + t * 2 + p
    get = lambda code, sc: codes[(tiles[:, code].int() >> (4 * (col % 2))) & 15] * scale[tiles[:, sc].int()]  # noqa: E731
    return get(kb, sk), get(vb, sv)


def _exact_request(s, b, h):
    """K and V [len, d] of request b and head h."""
    case, n = s["case"], int(s["lens"][b])
    pages = s["table"][b, :_pages(n, case["page"])].long()
    tiles = s["cache"][pages, h].flatten(0, 1)
    return [x.flatten(0, 1)[:n] for x in _exact_tiles(tiles, case["d"])]


def _exact_gather(s):
    case = s["case"]
    got = [[_exact_request(s, b, h) for h in range(case["Hkv"])] for b in range(case["B"])]
    return [torch.cat([torch.stack([kv[i] for kv in heads], 1) for heads in got]) * g for i, g in enumerate((case["kg"], case["vg"]))]


def _exact_attn(s):
    case = s["case"]
    nq, h, hkv, d = (case[k] for k in ("nq", "H", "Hkv", "d"))
    o = torch.zeros((case["B"] * nq, h, d), dtype=torch.float64, device="cuda")
    lse = torch.full((h, case["B"] * nq), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        n = int(s["lens"][b])
        for j in range(hkv):
            k, v = _exact_request(s, b, j)
            heads = slice(j * (h // hkv), (j + 1) * (h // hkv))
            for i in range(nq):
                see = n - nq + i + 1 if case["causal"] else n
                if see > 0:
                    x = s["q"][b * nq + i, heads].double() @ k[:see].T * d ** -0.5
                    o[b * nq + i, heads] = torch.softmax(x, -1) @ v[:see]
                    lse[heads, b * nq + i] = torch.logsumexp(x, -1)
    return [o, lse]
