"""The paged cache in bf16 and e4m3, and the rotation's table, at the ends of their ranges."""
import math

import numpy as np
import pytest
import torch

import tiled_exact_attention_fa2_gb300 as fa2
from test_kv import bits, check_attention, filled, i32
from test_kv4 import check_attention as check4

# B, H, H_kv, d, keys, bound on the keys: the line, clusters of 8 and 2 CTAs and single CTAs, four, two and one warps a unit
FORMS = [(1, 4, 1, 128, 3000, None), (90, 4, 2, 64, 300, None), (1, 16, 1, 16, 20000, None), (1, 8, 1, 64, 2000, 2000), (20, 8, 2, 128, 1000, 1000),
         (100, 2, 1, 32, 700, 700), (100, 4, 2, 128, 900, 900), (100, 12, 4, 64, 600, 600), (350, 2, 2, 128, 500, 500), (350, 40, 2, 32, 200, 200)]


@pytest.mark.gpu
@pytest.mark.parametrize("scores", ["one late", "rising", "equal"])
@pytest.mark.parametrize("form", FORMS, ids=str)
def test_values_up_to_the_largest(form, scores):
    """bf16 values up to the largest there are, of one sign, so that O is as large; scores that lie some 10 nats (14.4
    doublings) above the first keys', of one key in the middle or of more and more, or all equal: O stays finite and
    right, since the sum of a weighted mean's weights is held at 1 at most.  A column is checked against its own largest
    value, so a small one beside it counts as much."""
    B, H, Hkv, d, n, bound = form
    rng = np.random.default_rng(n + d)
    lens = [n] + [int(x) for x in rng.integers(n // 2, n + 1, B - 1)]
    caches, table, kv = filled(rng, lens, Hkv, 16, d, torch.bfloat16, width=4096 if bound is None else 1)
    top = 2.0 ** np.linspace(-60, 127.99, d)
    for b, m in enumerate(lens):
        pos = np.arange(m)
        score = {"one late": 10.0 * (pos == m // 2), "rising": 10.0 * pos / m, "equal": 0.0 * pos}[scores]
        page, off = torch.from_numpy(table[b][pos // 16]).cuda(), torch.from_numpy(pos % 16).cuda()
        k = torch.zeros(m, Hkv, d)
        k[:, :, 0] = torch.from_numpy(score)[:, None]
        k[:, :, 1:] = 2.0 ** -4 * torch.from_numpy(rng.standard_normal((m, Hkv, d - 1)))
        v = torch.from_numpy(rng.uniform(0.5, 0.99, (m, Hkv, d)) * top).float()
        pair = []
        for cache, x in zip(caches, (k, v)):
            x = x.to(torch.bfloat16)
            bits(cache)[page, :, off] = bits(x).cuda()
            pair.append(x.double().numpy().transpose(1, 0, 2))
        kv[b] = tuple(pair)
    q = torch.from_numpy(rng.standard_normal((B, H, d)) * 2.0 ** -4)
    q[..., 0] = 1.0
    q = q.to(torch.bfloat16).cuda()
    fa2.fa2_device_status(reset=True)
    o, lse = fa2.fa2_kv_attn(q, *caches, i32(table), i32(lens), max_seqlen_k=bound, scale=1.0)
    assert fa2.fa2_device_status() == 0 and torch.all(torch.isfinite(o))
    some = sorted({0, 1 % B, B // 2, B - 1})
    scaled = [(k, v / top) for k, v in kv]
    for b in some:
        check_attention(o[b:b + 1].double() / torch.from_numpy(top).cuda(), lse[:, b:b + 1], [(0, 1)], q[b:b + 1].double().cpu().numpy(),
                        [scaled[b]], 1.0, True, H, torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("form", [f for f in FORMS if f[0] in (1, 90, 350)], ids=str)
@pytest.mark.parametrize("cache", ["bf16", "e4m3", "4 bit"])
def test_infinite_queries(form, cache):
    """Every key is positive in column 0 and of either sign elsewhere.  A query that is -inf there has no finite score,
    however large its other values are (its scores are -inf, not NaN): zeros and -inf.  +inf, or a NaN: NaN.  Rows beside
    them are right."""
    B, H, Hkv, d, n, bound = form
    rng = np.random.default_rng(n)
    lens = [n] + [int(x) for x in rng.integers(n // 2, n + 1, B - 1)]
    counts = [-(-m // 16) for m in lens]
    table = np.full((B, 4096 if bound is None else max(counts)), -1)
    order, at = rng.permutation(sum(counts)), 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    k, v = (torch.from_numpy(rng.standard_normal((at * 16, Hkv, d))).to(torch.bfloat16).cuda() for _ in range(2))
    k[..., 0] = 4 + k[..., 0].abs()
    slots = torch.arange(at * 16, device="cuda")
    if cache == "4 bit":
        held = fa2.fa2_kv4_cache(at, Hkv, 16, d)
        fa2.fa2_kv4_append(k, v, held, slots)
        call = lambda q: fa2.fa2_kv4_attn(q, held, i32(table), i32(lens), max_seqlen_k=bound)  # noqa: E731
    else:
        held = fa2.fa2_kv_cache(at, Hkv, 16, d, dtype=torch.bfloat16 if cache == "bf16" else torch.float8_e4m3fn)
        fa2.fa2_kv_append(k, v, *held, slots)
        call = lambda q: fa2.fa2_kv_attn(q, *held, i32(table), i32(lens), max_seqlen_k=bound)  # noqa: E731
    q = torch.from_numpy(rng.standard_normal((B, H, d))).to(torch.bfloat16).cuda()
    want_o, want_lse = call(q)
    odd = q.clone()
    odd[:, 0, 1:] *= 1e6
    odd[0, 0, 1:] = torch.where(odd[0, 0, 1:] < 0, -3e38, 3e38)
    odd[:, 0, 0] = -math.inf
    if H > 1:
        odd[:, 1, 0] = math.inf
    if H > 2:
        odd[:, 2, 1], odd[:, 2, 2] = math.nan, 3e38
    o, lse = call(odd)
    # A bf16 cache's products are summed as they are: where those of the finite values pass fp32's range (sum |q| |k| >=
    # 2^128, request 0 only: 1e6 times a normal number stays far below) their sum is an infinity itself, of either sign,
    # and the score may be NaN.  The other caches' sums are of q divided by a power of two.
    fits = torch.ones(B, dtype=torch.bool, device="cuda")
    if cache == "bf16":
        pages = torch.from_numpy(table[0, :counts[0]]).cuda()
        sums = odd[0, 0, 1:].double().abs() @ held[0][pages, 0].reshape(-1, d)[:n, 1:].double().abs().T
        fits[0] = bool(sums.max() < 2.0 ** 128)
    assert torch.all(o[fits, 0] == 0) and torch.all(lse[0, fits] == -math.inf)
    assert torch.all(torch.isnan(o[:, 1:3])) and torch.all(torch.isnan(lse[1:3]))
    # (not to the bit: the running maxima of a unit's rows are raised together, when one of them is passed, and with them
    # the weights' common factor; each of the two calls is held to the definition)
    o[:, :3], lse[:3] = want_o[:, :3], want_lse[:3]
    for b in (0, B - 1):
        pages, cu = i32(table[b:b + 1]), i32([0, lens[b]])
        got = fa2.fa2_kv4_gather(held, pages, cu, lens[b]) if cache == "4 bit" else fa2.fa2_kv_gather(*held, pages, cu, lens[b])
        kv = [tuple(x.double().cpu().numpy().transpose(1, 0, 2) for x in got)]
        for x, y in ((o, lse), (want_o, want_lse)):
            args = x[b:b + 1], y[:, b:b + 1], [(0, 1)], q[b:b + 1].double().cpu().numpy(), kv, d ** -0.5, True, H
            check4(*args) if cache == "4 bit" else check_attention(*args, held[0].dtype)


def test_table_amplitudes_that_fp32_has_no_digits_for():
    from tiled_exact_attention_fa2_gb300 import _build
    _build.build()
    lib = fa2.load_library()
    call = lambda amp: lib.fa2_rope_table(None, 0, 0, 32, 1e4, 1.0, 0.0, 1.0, 32.0, amp, None)  # noqa: E731
    for amp in (1e-39, 2.0 ** -127, 1e39, 1e-60):
        assert call(amp) == 5, amp
    for amp in (2.0 ** -126, 3.4e38):
        assert call(amp) == 0, amp


def near(column, rot, trained, width):
    """Borders of 1 +- width times the turns that a column makes, base 10^4."""
    turns = trained * 10000.0 ** (-2.0 * column / rot) / (2 * math.pi)
    return dict(low=turns * (1 - width), high=turns * (1 + width))


@pytest.mark.gpu
@pytest.mark.parametrize("first,n,rot,args", [
    (0, 5, 112, dict(base=1e-12)), (1000, 3000, 128, dict(base=1e-6)), (0, 300, 48, dict(base=3e-8, amplitude=2.0 ** -126)), (7, 1000, 96, dict(base=1e4, factor=1e-3)),
    ((1 << 31) - 50, 50, 112, dict(base=12.7)), (1 << 20, 99, 64, dict(base=1e4, factor=8.0, trained=8192, **near(10, 64, 8192, 2.0 ** -12))),
    (1 << 24, 77, 80, dict(base=1e4, factor=0.25, trained=100000, **near(3, 80, 100000, 2.0 ** -5))), (5, 64, 128, dict(base=1e4, amplitude=3e38))])
def test_table_within_the_stated_bound(first, n, rot, args):
    """The bound that the header states, for every base and factor: 2^-21 from fp32 (test_rope.py) and, a position, what
    fp64 leaves of theta'.  Its relative error: the power 1.04 2^-53 and its exponent's correction 2^-53, 1 - g, the
    quotient by the factor, the sum, the product, the quotient by 2 pi 2^-53 each and 2 pi itself 2^-54.5: 7.4 2^-53 <
    2^-50, times theta' <= max(1, 1 / base) max(1, 1 / factor).  Mixed columns: g is off by (4.4 high / (high - low) + 3)
    2^-53 more, where turns <= high: less than 15 2^-53 max(1, high / (high - low)) < 2^-49 of it, together."""
    import oracle.kv as ref

    call = dict(args)
    for a, b in (("trained", "trained_positions"), ("low", "low_turns"), ("high", "high_turns")):
        if a in call:
            call[b] = call.pop(a)
    got = fa2.fa2_rope_table(n, rot, first_position=first, **call).cpu().numpy().astype(np.longdouble)
    e = 2.0 ** -50 * max(1.0, 1 / args["base"]) * max(1.0, 1 / args.get("factor", 1.0))
    if "trained" in args:
        e *= 2 * max(1.0, args["high"] / (args["high"] - args["low"]))
    tol = (2.0 ** -21 + np.arange(first, first + n)[:, None] * e) * args.get("amplitude", 1.0)
    err = np.abs(got - ref.table(first, n, rot, **args))
    assert np.all(err <= tol), float((err / tol).max())


def queue_word(ws):
    """The queue's counter in a workspace of fa2_kv_attn: behind the two times 1440 counters of parts."""
    return ws[ws.numel() - -(-2881 * 8 // 256) * 256 + 2880 * 8:][:8].view(torch.int64)


@pytest.mark.gpu
def test_a_workspace_with_half_of_a_calls_number():
    """A workspace may hold anything: also a word whose upper 32 bits are those of the call's number.  (A captured call
    keeps its number, and the queue's word is left at it.)"""
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(1, 400, 120)]
    caches, table, kv = filled(rng, lens, 4, 16, 32, torch.bfloat16, width=4096)
    q = torch.from_numpy(rng.standard_normal((120, 4, 32))).to(torch.bfloat16).cuda()
    ws = torch.zeros(fa2.fa2_kv_attn_workspace_bytes(120, 4, 4, 1, 4096 * 16, 32), dtype=torch.uint8, device="cuda")
    t, n = i32(table), i32(lens)
    fa2.fa2_device_status(reset=True)
    want = fa2.fa2_kv_attn(q, *caches, t, n, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa2.fa2_kv_attn(q, *caches, t, n, workspace=ws)
    for low in (0, 1, 0x1234):
        graph.replay()
        word = queue_word(ws)
        word.copy_((word ^ (1 << 16)) | low)
        for x in got:
            x.fill_(9)
        graph.replay()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert fa2.fa2_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hkv", [(8300, 8), (33000, 4)])  # more than 65383 + 304 items; twice as many
def test_more_items_than_the_queue_counts(B, Hkv):
    """Items are then taken in runs: none is left out, a longer request among them is still cut; the same again from a
    captured call, whatever the workspace holds, and as with the warp form's bound."""
    d, P = 16, 16
    rng = np.random.default_rng(B)
    lens = [0 if i % 1000 == 7 else int(x) for i, x in enumerate(rng.integers(1, 33, B))]
    assert B * Hkv - Hkv * lens.count(0) > 65383 + 304
    lens[B // 2] = 20000
    g = torch.Generator("cuda").manual_seed(1)
    pages = 3000
    caches = fa2.fa2_kv_cache(pages, Hkv, P, d)
    for c in caches:
        c.copy_(torch.randn(c.shape, generator=g, device="cuda"))
    table = torch.randint(0, pages, (B, 20000 // P), generator=g, device="cuda", dtype=torch.int32)  # (requests share pages)
    q = torch.randn((B, Hkv, d), generator=g, device="cuda").to(torch.bfloat16)
    n = i32(lens)
    ws = torch.full((fa2.fa2_kv_attn_workspace_bytes(B, Hkv, Hkv, 1, 20000, d),), 0xFF, dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    fa2.fa2_device_status(reset=True)
    o, lse = torch.full_like(q, 9.0), torch.full((Hkv, B), 9.0, device="cuda")
    call = lambda: fa2.fa2_kv_attn(q, *caches, table, n, o=o, lse=lse, workspace=ws)  # noqa: E731
    call()
    assert not torch.any(lse == 9)
    first = o.clone(), lse.clone()
    some = sorted({0, 1, B // 2, B - 1} | {int(x) for x in rng.integers(0, B, 200)})
    for b in some:
        got = fa2.fa2_kv_gather(*caches, table[b:b + 1].contiguous(), i32([0, lens[b]]), lens[b])
        kv = tuple(x.double().cpu().numpy().transpose(1, 0, 2) for x in got)
        check_attention(o[b:b + 1], lse[:, b:b + 1], [(0, 1)], q[b:b + 1].double().cpu().numpy(), [kv], d ** -0.5, True, Hkv, torch.bfloat16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for fill in (0, 0x5A, None):
        if fill is not None:
            ws.fill_(fill)
        o.fill_(9), lse.fill_(9)
        graph.replay()
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    # Without the long request the warp form may take them: the same to two roundings of bf16 and twice check_attention's
    # bound, (2^-16 + 2 x) mass with scale sum |q| |k| < 2^4, so x < 2^-14 + 2^-20, and mass < 4: 2^-9.8.
    n[B // 2] = 32
    call()
    short = fa2.fa2_kv_attn(q, *caches, table, n, max_seqlen_k=32)
    assert torch.all((o.float() - short[0].float()).abs() <= 2.0 ** -7 * o.float().abs() + 2.0 ** -9)
    assert fa2.fa2_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float8_e4m3fn], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("B,H,Hkv,d,bound", [(100, 8, 2, 64, None), (2, 16, 1, 128, None), (100, 40, 2, 32, None), (3, 8, 2, 64, 40), (30, 8, 2, 128, 40),
                                             (100, 8, 2, 16, 40), (150, 15, 3, 64, 40), (400, 4, 2, 128, 40)])
def test_weights_keep_more_bits_than_one_16_bit_number(B, H, Hkv, d, bound, kind):
    """Few keys of scores near one another and values of either sign: outputs that nearly cancel show how the weights were
    rounded.  A weight is the sum of two numbers of 16 bits: 2^-16 relative, of either type (one fp16 number, 2^-11, leaves
    the bound four times over in one output of sixty).  Below fp16's normal numbers a weight is off by 2^-36 of the sum
    (test_kv.py), 40 of them by less than the 2^-19 that the bound has for the exponential."""
    rng = np.random.default_rng(B + d)
    lens = [int(x) for x in rng.integers(3, 41, B)]
    factors = (1.0, 1.0) if kind == torch.bfloat16 else (2.0 ** -6, 2.0 ** -6)
    caches, table, kv = filled(rng, lens, Hkv, 16, d, kind, factors, width=1 if bound else 4096, spread=0.5)
    q = torch.from_numpy(rng.standard_normal((B, H, d)) * 0.25).to(torch.bfloat16).cuda()
    fa2.fa2_device_status(reset=True)
    o, lse = fa2.fa2_kv_attn(q, *caches, i32(table), i32(lens), max_seqlen_k=bound, k_scale=factors[0], v_scale=factors[1])
    check_attention(o, lse, [(b, b + 1) for b in range(B)], q.double().cpu().numpy(), kv, d ** -0.5, True, H, torch.bfloat16)
    assert fa2.fa2_device_status() == 0
