"""The 4-bit paged cache: page plan, append, gather and attention.  Refusals and the definition on the CPU, the kernels on the GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle.kv4 as ref
import tiled_exact_attention_fa2_gb300 as fa2

A = 1 << 32  # fake device addresses, far apart; never dereferenced


@pytest.fixture(scope="module")
def lib():
    from tiled_exact_attention_fa2_gb300 import _build
    _build.build()
    return fa2.load_library()


# ---------------------------------------------------------------- CPU
@pytest.mark.parametrize("d", [16, 32, 64, 128])
def test_layout_uses_every_byte_once(d):
    key, col = np.meshgrid(np.arange(16), np.arange(d), indexing="ij")
    kb, vb, sh, ks, vs = ref.places(key, col, d)
    halves = np.concatenate([(kb * 8 + sh).ravel(), (vb * 8 + sh).ravel()])
    assert sorted(halves) == [8 * b + s for b in range(16 * d) for s in (0, 4)]
    scales = np.concatenate([ks[:, ::16].ravel(), vs[:, ::16].ravel()])
    assert sorted(scales) == list(range(16 * d, 18 * d))
    assert np.array_equal(ks, ks[:, col[0] // 16 * 16]) and np.array_equal(vs, vs[:, col[0] // 16 * 16])


def test_quantize_takes_the_nearest_value():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 32)) * np.exp(rng.standard_normal((50, 1)))
    code, scale, val = ref.quantize(x, 1.0)
    step = ref.E4M3[scale].repeat(16, 1)
    # e2m1 values are at most 2 apart (4 and 6), one step of half of it off at most; saturation costs at most the
    # scale's own rounding, 2^-4 of 6
    assert np.all(np.abs(val - x) <= step * 1.0 + 1e-12)
    sat = ref.quantize(np.r_[np.inf, np.full(15, 1.0)][None], 2.0)[2]
    assert sat[0, 0] == 448 * 6 * 2 and np.all(sat[0, 1:] == 0)
    assert np.isnan(ref.quantize(np.r_[np.nan, np.zeros(15)][None], 1.0)[2]).all()
    assert not ref.quantize(np.full((1, 16), 2.0 ** -12), 1.0)[2].any()


def append(lib, k=A, v=2 * A, cache=3 * A, slots=4 * A, ko=5 * A, vo=6 * A, T=8, Hkv=2, pages=4, P=16, d=64, ks=1.0, vs=1.0,
           stride=None, strides=None):
    s = None if strides is None else (ctypes.c_longlong * 4)(*strides)
    stride = Hkv * (P // 16) * 18 * d if stride is None else stride
    return lib.fa2_kv4_append(k, v, s, cache, stride, slots, ko, vo, T, Hkv, pages, P, d, ks, vs, None)


def gather(lib, cache=A, table=2 * A, cu=3 * A, k=4 * A, v=5 * A, B=2, Hkv=2, total=8, pages=4, P=16, W=2, tstride=None, d=64,
           ks=1.0, vs=1.0, stride=None):
    stride = Hkv * (P // 16) * 18 * d if stride is None else stride
    return lib.fa2_kv4_gather(cache, stride, table, W if tstride is None else tstride, cu, k, v, B, Hkv, total, pages, P, W, d, ks,
                              vs, None)


def attn(lib, q=A, cache=2 * A, table=3 * A, lens=4 * A, cu=5 * A, o=6 * A, lse=7 * A, B=2, H=4, Hkv=2, tq=8, mq=4, mk=1 << 30, pages=4,
         P=16, W=2, tstride=None, d=64, scale=0.1, ks=1.0, vs=1.0, ws=8 * A, wsb=1 << 30, stride=None):
    stride = Hkv * (P // 16) * 18 * d if stride is None else stride
    return lib.fa2_kv4_attn(q, cache, stride, table, W if tstride is None else tstride, lens, cu, o, lse, B, H, Hkv, tq, mq, mk, pages,
                            P, W, d, scale, ks, vs, 1, ws, wsb, None)


def plan(lib, p=None, B=4, F=3, W=5, tstride=None, P=16, T=10):
    p = p or [A * (i + 1) for i in range(10)]
    return lib.fa2_page_plan(*p, B, F, W, W if tstride is None else tstride, P, T, None)


def test_cache_refusals_are_the_same_everywhere(lib):
    assert append(lib, T=0) == 0 and gather(lib, total=0) == 0 and attn(lib, tq=0, mq=0) == 0
    for f in (append, gather, attn):
        for bad in (dict(pages=0), dict(P=8), dict(P=48), dict(P=256), dict(Hkv=0), dict(stride=100), dict(stride=1 << 50),
                    dict(stride=-4096), dict(stride=1 << 44, pages=5)):
            assert f(lib, **bad) == 2, (f.__name__, bad)
        for d in (0, 8, 48, 96, 256):
            assert f(lib, d=d) == 3
        assert f(lib, cache=None) == 1 and f(lib, cache=3 * A + 8) == 4 and f(lib, stride=2 * 18 * 64 + 8) == 4
        for s in (0.0, -1.0, 3.0, 0.3, float("nan"), float("inf"), 2.0 ** 65, 2.0 ** -65):
            assert f(lib, ks=s) == 5 and f(lib, vs=s) == 5, (f.__name__, s)
    assert fa2.fa2_kv4_page_bytes(8, 64, 128) == 8 * 4 * 18 * 128
    for bad in ((0, 64, 128), (8, 24, 128), (8, 64, 100)):
        assert fa2.fa2_kv4_page_bytes(*bad) == 0


def test_append_refusals(lib):
    for name in ("k", "v", "slots"):
        assert append(lib, **{name: None}) == 1
    assert append(lib, T=-1) == 2 and append(lib, strides=[-8, 64, 128, 64]) == 2
    assert append(lib, strides=[1 << 44, 64, 128, 64]) == 2 and append(lib, strides=[128, 64, 128, 1 << 60]) == 2
    for bad in (dict(k=A + 8), dict(vo=6 * A + 2), dict(slots=4 * A + 4), dict(strides=[132, 64, 128, 64])):
        assert append(lib, **bad) == 4, bad
    for bad in (dict(k=3 * A), dict(ko=A), dict(ko=3 * A), dict(vo=5 * A), dict(slots=3 * A + 64)):
        assert append(lib, **bad) == 9, bad


def test_gather_refusals(lib):
    for name in ("table", "cu", "k", "v"):
        assert gather(lib, **{name: None}) == 1
    for bad in (dict(B=0), dict(total=-1), dict(W=0), dict(tstride=1), dict(tstride=1 << 50)):
        assert gather(lib, **bad) == 2, bad
    for bad in (dict(k=4 * A + 2), dict(table=2 * A + 2), dict(cu=3 * A + 1)):
        assert gather(lib, **bad) == 4, bad
    for bad in (dict(k=A), dict(v=4 * A), dict(v=2 * A)):
        assert gather(lib, **bad) == 9, bad


def test_attention_refusals(lib):
    for name in ("q", "table", "lens", "o", "lse"):
        assert attn(lib, **{name: None}) == 1
    for bad in (dict(B=0), dict(H=0), dict(H=3), dict(tq=-1), dict(mq=0), dict(mq=9), dict(W=0), dict(tstride=1),
                dict(cu=None, tq=7), dict(tq=(1 << 30) + 1), dict(mk=0), dict(mk=-5), dict(tstride=1 << 50)):
        assert attn(lib, **bad) == 2, bad
    for s in (0.0, -0.1, float("nan"), float("inf")):
        assert attn(lib, scale=s) == 5
    for bad in (dict(q=A + 8), dict(o=6 * A + 2), dict(lse=7 * A + 2), dict(lens=4 * A + 1), dict(cu=5 * A + 2)):
        assert attn(lib, **bad) == 4, bad
    for bad in (dict(o=A), dict(o=2 * A), dict(lse=6 * A), dict(lse=4 * A)):
        assert attn(lib, **bad) == 9, bad
    # tables of more than 2048 keys: two launches and a workspace
    need = lib.fa2_kv4_attn_workspace_bytes(2, 4, 2, 4, 129 * 16, 64)
    assert need > 0 and attn(lib, W=129, ws=None) == 8 and attn(lib, W=129, ws=8 * A + 16) == 8
    assert attn(lib, W=129, wsb=need - 1) == 8 and attn(lib, W=129, ws=A) == 9 and attn(lib, W=129, ws=2 * A) == 9
    ws = lib.fa2_kv4_attn_workspace_bytes
    assert ws(76, 4, 2, 4, 32, 64) == 0 and ws(1, 4, 2, 4, 2048, 64) == 0
    assert ws(77, 4, 2, 4, 2048, 64) == 0 and ws(77, 4, 2, 4, 2049, 64) > 0  # more units than SMs
    assert ws(77, 4, 2, 8, 1024, 64) == 0 and ws(77, 4, 2, 8, 1025, 64) > 0  # of 16 rows
    assert ws(609, 4, 2, 4, 128, 64) == 0 and ws(609, 4, 2, 4, 127, 64) > 0 and ws(608, 4, 2, 4, 1, 64) == 0
    assert ws(76, 4, 2, 4, 54 * 152, 64) == 0 and ws(76, 4, 2, 4, 54 * 152 + 1, 64) > 0
    assert attn(lib, W=129, mk=2048, ws=None, o=A) == 9  # (a tight bound: no workspace asked for)
    for bad in ((0, 4, 2, 1, 99, 64), (1, 4, 3, 1, 99, 64), (1, 4, 2, 0, 99, 64), (1, 4, 2, 1, 0, 64), (1, 4, 2, 1, 99999, 60)):
        assert ws(*bad) == 0


def test_plan_refusals(lib):
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 8, 9):
        p = [A * (j + 1) for j in range(10)]
        p[i] = None
        assert plan(lib, p) == 1, i
    for bad in (dict(B=0), dict(B=16385), dict(F=-1), dict(W=0), dict(tstride=4), dict(tstride=1 << 50), dict(P=0), dict(P=20), dict(T=-1)):
        assert plan(lib, **bad) == 2, bad
    p = [A * (j + 1) for j in range(10)]
    p[7] += 4
    assert plan(lib, p) == 4
    for i, j in ((3, 0), (4, 1), (5, 4), (7, 8), (9, 2)):
        p = [A * (k + 1) for k in range(10)]
        p[i] = p[j]
        assert plan(lib, p) == 9, (i, j)


def test_python_refusals():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    c = torch.zeros(4, 2, 1, 18 * 64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        fa2.fa2_kv4_append(x, x, c, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        fa2.fa2_kv4_cache(4, 2, 24, 64)
    with pytest.raises(ValueError):
        fa2.fa2_page_plan(torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                          torch.zeros(1, 1, dtype=torch.int32), 16, 4)


# ---------------------------------------------------------------- GPU: page plan
def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def check_plan(cached, new, free, table, P, T):
    t = i32(table)
    p = fa2.fa2_page_plan(i32(cached), i32(new), i32(free), t, P, T)
    want = ref.plan(cached, new, free, table, P, T)
    for got, w, name in zip((t, p.lens, p.cu_new, p.cu_total, p.slots, p.positions, p.pages_needed), want,
                            ("table", "lens", "cu_new", "cu_total", "slots", "positions", "needed")):
        assert np.array_equal(got.cpu().numpy().ravel(), np.asarray(w).ravel()), name
    return p


@pytest.mark.gpu
@pytest.mark.parametrize("B,P,most_old,most_new", [(1, 16, 0, 1), (1, 128, 1000, 700), (31, 16, 100, 3), (64, 64, 4000, 1),
                                                   (600, 32, 300, 90), (513, 64, 65, 64), (5000, 16, 40, 20)])
def test_plan(B, P, most_old, most_new):
    rng = np.random.default_rng(B)
    cached, new = rng.integers(0, most_old + 1, B), rng.integers(0, most_new + 1, B)
    cached[rng.random(B) < 0.2] = 0
    new[rng.random(B) < 0.2] = 0
    cached[-1] = cached[-1] // P * P  # a page that is just full
    W = int(max(-(-(cached + new) // P))) + 1
    need = int(sum(-(-(cached + new) // P)))
    ids = rng.permutation(need + 3)
    table, at = np.full((B, W), -7), 0
    for b in range(B):
        n = -(-cached[b] // P)
        table[b, :n] = ids[at:at + n]
        at += n
    fa2.fa2_device_status(reset=True)
    T = int(new.sum())
    check_plan(cached, new, ids[at:], table, P, T + 4)
    check_plan(cached, new, ids[at:], table, P, T)
    assert fa2.fa2_device_status() == 0
    # too few free pages: -1, and the number that would do
    p = check_plan(cached, new, ids[at:at + max(0, (need - at) // 2)], table, P, T)
    assert int(p.pages_needed) == need - at
    assert fa2.fa2_device_status() == 0


@pytest.mark.gpu
def test_plan_impossible_requests_count_as_empty():
    fa2.fa2_device_status(reset=True)
    table = np.arange(12).reshape(4, 3)
    check_plan([5, -1, 10, 40], [3, 4, -2, 20], [100, 101, 102], table, 16, 12)
    assert fa2.fa2_device_status(reset=True) == 3
    check_plan([5, 0], [9, 9], [100, 101, 102], table[:2], 16, 12)  # more tokens than max_tokens
    assert fa2.fa2_device_status(reset=True) == 3
    big = 2 ** 31 - 16
    t = i32(np.zeros((3, 1)))
    p = fa2.fa2_page_plan(i32([big, big, 1]), i32([1, 1, 1]), i32([]), t, 128, 4)  # no room in the rows
    assert p.lens.tolist() == [0, 0, 2] and fa2.fa2_device_status(reset=True) == 3
    t = torch.zeros(2, 1 << 24, dtype=torch.int32, device="cuda")  # rows with room for 2^31 tokens
    p = fa2.fa2_page_plan(i32([1 << 30, (1 << 30) - 2]), i32([1, 0]), i32([5]), t, 128, 4)
    assert p.cu_total.tolist() == [0, (1 << 30) + 1, 2 ** 31 - 1] and p.slots.tolist() == [5 * 128, -1, -1, -1]
    assert fa2.fa2_device_status(reset=True) == 0
    p = fa2.fa2_page_plan(i32([1 << 30, (1 << 30) - 1]), i32([1, 0]), i32([5]), t, 128, 4)  # one more than 32 bits count
    assert p.cu_total.tolist() == [0, 0, 0] and p.lens.tolist() == [0, 0] and p.slots.tolist() == [-1] * 4
    assert int(p.pages_needed) == 0 and fa2.fa2_device_status(reset=True) == 3


@pytest.mark.gpu
def test_plan_captured_and_replayed_with_other_lengths():
    table = i32(np.full((3, 4), -1))
    cached, new, free = i32([0, 0, 0]), i32([0, 0, 0]), i32(np.arange(20, 32))
    p = fa2.fa2_page_plan(cached, new, free, table, 16, 40)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa2.fa2_page_plan(cached, new, free, table, 16, 40, plan=p)
    for lens in ([1, 17, 3], [16, 0, 20], [0, 0, 1]):
        table.fill_(-1)
        new.copy_(i32(lens))
        graph.replay()
        want = ref.plan([0, 0, 0], lens, list(range(20, 32)), np.full((3, 4), -1), 16, 40)
        assert np.array_equal(table.cpu().numpy(), want[0]) and p.slots.tolist() == want[4] and p.positions.tolist() == want[5]


# ---------------------------------------------------------------- GPU: append and gather
@pytest.mark.gpu
@pytest.mark.parametrize("d,P,Hkv,T,factors", [(16, 16, 1, 1, (1.0, 1.0)), (16, 64, 3, 70, (2.0, 0.5)), (32, 16, 2, 33, (1.0, 4.0)),
                                               (64, 32, 5, 100, (0.25, 1.0)), (128, 64, 8, 257, (1.0, 1.0)),
                                               (128, 128, 1, 300, (8.0, 2.0 ** -10))])
def test_append_stores_the_nearest_values(d, P, Hkv, T, factors):
    rng = np.random.default_rng(d + T)
    pages = -(-T // P) + 2
    slots = rng.permutation(pages * P)[:T]
    x = torch.from_numpy(rng.standard_normal((2, T, Hkv + 1, d)) * np.exp(rng.standard_normal((2, T, Hkv + 1, 1)))).to(torch.bfloat16)
    if T >= 33:  # special groups, at the head of every token's row
        x[0, 0, 0] = 0.0
        x[0, 1, 0] = -0.0
        x[0, 2, 0, 3] = float("inf")
        x[1, 3, 0, 5] = float("nan")
        x[0, 4, 0] = 1e-30
        x[1, 5, 0] = 3e38
        x[0, 6, 0, :16] = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 0])  # ties
        x[1, 7, 0, :16] = x[0, 6, 0, :16] * factors[1] * 0.875
        x[0, 8, 0] = 2.0 ** -10 * 6 * factors[0]      # a scale halfway between 0 and the least
        x[0, 9, 0] = 2.0 ** -9 * 1.5 * 6 * factors[0]
    k, v = x[0, :, :Hkv].cuda(), x[1, :, :Hkv].cuda()  # token stride (Hkv + 1) d
    if T == 1:
        k, v = k.contiguous(), v.contiguous()
    big = torch.randint(0, 255, (pages, 2, Hkv, P // 16, 18 * d), dtype=torch.uint8, device="cuda")  # two layers' pages in turn
    cache, other = big[:, 0], big[:, 1].clone()
    want = cache.cpu().numpy().copy()
    ko, vo = torch.empty(T, Hkv, d, dtype=torch.bfloat16, device="cuda"), torch.empty(T, Hkv, d, dtype=torch.bfloat16, device="cuda")
    fa2.fa2_kv4_append(k, v, cache, torch.from_numpy(slots).cuda(), *factors, k_out=ko, v_out=vo)
    k64, v64 = k.double().cpu().numpy(), v.double().cpu().numpy()
    for t in range(T):
        ref.store(want, int(slots[t]), k64[t], v64[t], *factors)
    # (a zero group's sign bits say nothing: codes of a scale 0 are stored as 0)
    assert np.array_equal(cache.cpu().numpy(), want)
    assert torch.equal(big[:, 1], other)
    for got, x64, f in ((ko, k64, factors[0]), (vo, v64, factors[1])):
        assert np.array_equal(got.double().cpu().numpy(), ref.quantize(x64, f)[2], equal_nan=True)
    # and back, as one sequence per token's page order
    inv = np.full(pages * P, -1)
    inv[slots] = np.arange(T)
    kk, vv = fa2.fa2_kv4_gather(cache, i32(np.arange(pages)[None]), i32([0, pages * P]), pages * P, *factors)
    at = torch.from_numpy(slots).cuda()
    assert torch.equal(kk[at].nan_to_num(7), ko.nan_to_num(7)) and torch.equal(vv[at].nan_to_num(7), vo.nan_to_num(7))


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hkv,d", [(5001, 8, 128), (9000, 20, 64), (70001, 1, 32)])
def test_append_many_tokens_and_back(T, Hkv, d):
    """Many tokens (two to a thread), heads beyond a CTA's 256 threads; what is stored is read back."""
    g = torch.Generator(device="cuda").manual_seed(T)
    k, v = (torch.randn(T, Hkv, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    pages = -(-T // 64) + 1
    cache = fa2.fa2_kv4_cache(pages, Hkv, 64, d)
    slots = torch.arange(T, device="cuda") + 64
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    fa2.fa2_kv4_append(k, v, cache, slots, k_out=ko, v_out=vo)
    some = torch.randint(0, T, (300,), generator=g, device="cuda")
    some[0] = T - 1
    for got, x in ((ko, k), (vo, v)):
        assert np.array_equal(got[some].double().cpu().numpy(), ref.quantize(x[some].double().cpu().numpy(), 1.0)[2])
    kk, vv = fa2.fa2_kv4_gather(cache, i32(np.arange(1, pages)[None]), i32([0, T]), T)
    assert torch.equal(kk, ko) and torch.equal(vv, vo)


@pytest.mark.gpu
def test_append_padding_and_bad_slots():
    fa2.fa2_device_status(reset=True)
    cache = fa2.fa2_kv4_cache(2, 2, 32, 64)
    cache.fill_(5)
    k = torch.randn(6, 2, 64, device="cuda").to(torch.bfloat16)
    slots = torch.tensor([-1, 3, -1, 40, -5, 63], device="cuda")
    fa2.fa2_kv4_append(k, k, cache, slots)
    assert fa2.fa2_device_status() == 0
    want = np.full(cache.shape, 5, np.uint8)
    for t in (1, 3, 5):
        ref.store(want, int(slots[t]), *[k[t].double().cpu().numpy()] * 2, 1.0, 1.0)
    assert np.array_equal(cache.cpu().numpy(), want)
    slots[0], slots[2] = 64, 1 << 40
    fa2.fa2_kv4_append(k, k, cache, slots)
    assert fa2.fa2_device_status(reset=True) == 5 and np.array_equal(cache.cpu().numpy(), want)


def filled(rng, lens, Hkv, P, d, junk=0xFF, spare=2, width=0):
    """A cache whose unwritten places hold `junk` (0xff: NaN scales), its table, and each request's K, V in fp64."""
    counts = [-(-n // P) for n in lens]
    pages = sum(counts) + spare
    ids, at = rng.permutation(pages), 0
    cache = np.full((pages, Hkv, P // 16, 18 * d), junk, np.uint8)
    table = np.full((len(lens), max(max(counts), 1) + width), -1)
    kv = []
    for b, n in enumerate(lens):
        table[b, :counts[b]] = ids[at:at + counts[b]]
        at += counts[b]
        k, v = rng.standard_normal((2, n, Hkv, d)) * np.exp(0.5 * rng.standard_normal((2, n, Hkv, 1)))
        for i in range(n):
            ref.store(cache, int(table[b, i // P]) * P + i % P, k[i], v[i], 1.0, 1.0)
        kv.append(ref.read(cache, table[b], n, 1.0, 1.0) if n else (np.zeros((Hkv, 0, d)),) * 2)
    return torch.from_numpy(cache).cuda(), table, kv


@pytest.mark.gpu
@pytest.mark.parametrize("d,P,Hkv", [(16, 32, 2), (32, 16, 3), (64, 128, 1), (128, 64, 2)])
def test_gather_ragged(d, P, Hkv):
    rng = np.random.default_rng(d)
    lens = [0, 1, 15, 16, 17, 0, 130, 33]
    cache, table, kv = filled(rng, lens, Hkv, P, d)
    cu = np.r_[0, np.cumsum(lens)]
    total = int(cu[-1])
    fa2.fa2_device_status(reset=True)
    k, v = (torch.full((total + 5, Hkv, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fa2.fa2_kv4_gather(cache, i32(table), i32(cu), total + 5, k=k, v=v)
    for got, i in ((k, 0), (v, 1)):
        want = np.concatenate([x[i].transpose(1, 0, 2) for x in kv])
        assert np.array_equal(got[:total].double().cpu().numpy(), want) and torch.all(got[total:] == 9)
    assert fa2.fa2_device_status() == 0
    # a page id that does not exist, a sequence longer than its row, offsets out of order
    bad = table.copy()
    bad[6, 0] = cache.shape[0]
    k.fill_(9)
    fa2.fa2_kv4_gather(cache, i32(bad), i32(cu), total, k=k[:total], v=v[:total])
    assert fa2.fa2_device_status(reset=True) == 5 and torch.all(k[int(cu[6]):int(cu[6]) + min(P, 130)] == 9)
    fa2.fa2_kv4_gather(cache, i32(table[:1, :1]), i32([0, P + 1]), P + 1)
    assert fa2.fa2_device_status(reset=True) in (3, 5)  # (row 0's only entry is -1 as well)
    fa2.fa2_kv4_gather(cache, i32(table[:2]), i32([4, 2, 3]), 4)
    assert fa2.fa2_device_status(reset=True) == 3


# ---------------------------------------------------------------- GPU: attention
def check_attention(o, lse, rows, q64, kv, scale, causal, H):
    """Each request's rows against the definition.  Bounds: the store rounds to bf16 (2^-8 relative); a weight is
    rounded to fp16 (2^-11) and its score is off by less than x = 2^-18 * scale * sum |q||k| (fp32 sums of exact
    products in the tensor core) plus 2^-20 for the exponential, in the numerator and in the sum.  A weight too small
    for fp16's normal numbers is off by 2^-25 absolute (half its subnormal spacing of 2^-24); weights are held 2^11
    times exp(s - m), m at most the row's maximum, so the sum they are divided by is at least 2^11: 2^-36 per key."""
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, (r0, r1) in enumerate(rows):
        if r0 == r1:
            continue
        want, wlse, mass, size = ref.attention(q64[r0:r1], *kv[b], scale, causal)
        x = 2.0 ** -18 * size + 2.0 ** -20
        none = ~np.isfinite(wlse)
        got_lse = lse[:, r0:r1]
        assert np.all(np.isneginf(got_lse[none]))
        assert np.all(np.abs(got_lse - np.where(none, 0, wlse))[~none] <= (x + 2.0 ** -20 * np.abs(np.where(none, 0, wlse)))[~none]), b
        tiny = 2.0 ** -36 * np.repeat(np.abs(kv[b][1]).sum(1), H // kv[b][1].shape[0], 0)
        tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2 * x.T[..., None]) * 1.01 * mass + tiny + 1e-30
        err = np.abs(o[r0:r1] - want)
        assert np.all(err <= tol), (b, float((err / tol).max()))


ATTN = [  # d, H, Hkv, P, lens, queries, causal
    (128, 1, 1, 16, [1], [1], True),
    (128, 8, 8, 64, [0, 1, 15, 16, 17, 64, 65, 300], [1] * 8, True),
    (128, 8, 1, 128, [1000, 129], [1, 1], True),
    (128, 16, 1, 32, [500, 31], [1, 1], True),
    (128, 12, 2, 16, [77, 200, 3], [5, 1, 5], True),
    (128, 4, 2, 64, [700, 40], [33, 40], True),
    (128, 4, 4, 16, [3, 0, 20], [7, 2, 20], True),      # more queries than keys: rows that see nothing
    (128, 6, 2, 32, [90, 33, 0], [3, 0, 2], False),
    (64, 8, 2, 16, [1, 14, 250, 0, 47], [1] * 5, True),
    (64, 15, 3, 64, [260, 65], [4, 9], True),
    (32, 4, 2, 32, [100, 17, 1], [2, 1, 3], True),
    (32, 8, 8, 128, [400], [1], False),
    (16, 2, 1, 16, [64, 5, 33], [1, 1, 1], True),
    (16, 6, 3, 64, [130, 2], [6, 5], True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True])  # room for at most 2048 / for more keys: one CTA per unit / the line
@pytest.mark.parametrize("case", ATTN, ids=str)
def test_attention(case, wide):
    d, H, Hkv, P, lens, nq, causal = case
    rng = np.random.default_rng(sum(lens) + d)
    cache, table, kv = filled(rng, lens, Hkv, P, d, width=8192 // P if wide else 1)
    cu = np.r_[0, np.cumsum(nq)]
    total = int(cu[-1])
    q = torch.from_numpy(rng.standard_normal((total + 3, H, d)) * 2).to(torch.bfloat16).cuda()
    o, lse = torch.full_like(q, 9.0), torch.full((H, total + 3), 9.0, device="cuda")
    fa2.fa2_device_status(reset=True)
    need = fa2.fa2_kv4_attn_workspace_bytes(len(lens), H, Hkv, max(nq), table.shape[1] * P, d)
    assert (need > 0) == wide
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda") if need else None
    fa2.fa2_kv4_attn(q, cache, i32(table), i32(lens), i32(cu), max(nq), o=o, lse=lse, workspace=ws, causal=causal)
    assert fa2.fa2_device_status() == 0
    assert torch.all(o[total:] == 9) and torch.all(lse[:, total:] == 9)  # rows behind the last request
    rows = [(int(cu[b]), int(cu[b + 1])) for b in range(len(lens))]
    check_attention(o, lse, rows, q.double().cpu().numpy(), kv, 1 / math.sqrt(d), causal, H)
    if wide:  # the same bound given: the other form, within the same tolerances
        short = fa2.fa2_kv4_attn(q, cache, i32(table), i32(lens), i32(cu), max(nq), max_seqlen_k=max(max(lens), 1), causal=causal)
        check_attention(*short, rows, q.double().cpu().numpy(), kv, 1 / math.sqrt(d), causal, H)
    o2, lse2 = fa2.fa2_kv4_attn(q, cache, i32(table), i32(lens), i32(cu), causal=causal)
    assert torch.equal(o2[:total], o[:total]) and torch.equal(lse2[:, :total], lse[:, :total])
    if len(set(nq)) == 1:
        o3, _ = fa2.fa2_kv4_attn(q[:total].contiguous(), cache, i32(table), i32(lens), causal=causal)
        assert torch.equal(o3, o[:total])


@pytest.mark.gpu
@pytest.mark.parametrize("B,n,H,Hkv,nq,d", [(3, 20011, 8, 2, 1, 128), (1, 40000, 16, 1, 2, 64), (90, 350, 4, 2, 1, 128),
                                            (2, 9000, 8, 1, 6, 128), (5, 2048, 8, 2, 3, 128), (19, 2000, 16, 8, 1, 64)])
def test_attention_long_and_shared_units(B, n, H, Hkv, nq, d):
    """Units cut over many spans, and many units in a span; scores that grow along the keys (late maxima)."""
    rng = np.random.default_rng(n)
    P = 64
    g = torch.Generator(device="cuda").manual_seed(n)
    lens = [n] + [int(x) for x in rng.integers(n // 3, n, B - 1)]
    counts = [-(-x // P) for x in lens]
    ids = torch.randperm(sum(counts) + 1, generator=g, device="cuda").int().cpu().numpy()
    table, at = np.full((B, max(counts)), -1), 0
    for b, c in enumerate(counts):
        table[b, :c] = ids[at:at + c]
        at += c
    cache = fa2.fa2_kv4_cache(sum(counts) + 1, Hkv, P, d)
    for b, x in enumerate(lens):
        ramp = torch.linspace(0.2, 2.0, x, device="cuda")[:, None, None]
        k = (torch.randn(x, Hkv, d, generator=g, device="cuda") * ramp).to(torch.bfloat16)
        v = torch.randn(x, Hkv, d, generator=g, device="cuda").to(torch.bfloat16)
        pos = torch.arange(x, device="cuda")
        slots = torch.from_numpy(table[b]).cuda()[pos // P].long() * P + pos % P
        fa2.fa2_kv4_append(k, v, cache, slots)
    q = (torch.randn(B * nq, H, d, generator=g, device="cuda") * 1.5).to(torch.bfloat16)
    o, lse = fa2.fa2_kv4_attn(q, cache, i32(table), i32(lens), max_seqlen_q=nq)
    some = sorted({0, B - 1, B // 2})
    host = cache.cpu().numpy()
    kv = {b: ref.read(host, table[b], lens[b], 1.0, 1.0) for b in some}
    for b in some:
        check_attention(o[b * nq:(b + 1) * nq], lse[:, b * nq:(b + 1) * nq], [(0, nq)], q[b * nq:(b + 1) * nq].double().cpu().numpy(),
                        [kv[b]], 1 / math.sqrt(d), True, H)
    assert fa2.fa2_device_status() == 0


@pytest.mark.gpu
def test_attention_scales_and_page_stride():
    rng = np.random.default_rng(5)
    cache, table, kv = filled(rng, [100, 37], 2, 32, 64)
    wide = torch.full((cache.shape[0], 3) + tuple(cache.shape[1:]), 0xFF, dtype=torch.uint8, device="cuda")
    wide[:, 1] = cache
    q = torch.from_numpy(rng.standard_normal((2, 4, 64))).to(torch.bfloat16).cuda()
    o, lse = fa2.fa2_kv4_attn(q, wide[:, 1], i32(table), i32([100, 37]), scale=0.05, k_scale=4.0, v_scale=0.5)
    kv = [(4.0 * k, 0.5 * v) for k, v in kv]
    check_attention(o, lse, [(0, 1), (1, 2)], q.double().cpu().numpy(), kv, 0.05, True, 4)


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [0, 128])
@pytest.mark.parametrize("d", [16, 64, 128])
def test_nan_reaches_only_the_rows_that_see_it(d, wide):
    """A NaN value or key at position 20 of 24 with 8 causal queries: the first four do not see it."""
    rng = np.random.default_rng(d)
    for where in ("v", "k"):
        cache, table, kv = filled(rng, [24, 24], 1, 16, d, width=wide)
        slot = int(table[0, 1]) * 16 + 4
        k, v = rng.standard_normal((2, 1, d))
        (v if where == "v" else k)[0, 3] = np.nan
        host = cache.cpu().numpy()
        ref.store(host, slot, k, v, 1.0, 1.0)
        cache = torch.from_numpy(host).cuda()
        kv = [ref.read(host, table[b], 24, 1.0, 1.0) for b in range(2)]
        q = torch.from_numpy(rng.standard_normal((16, 2, d))).to(torch.bfloat16).cuda()
        o, lse = fa2.fa2_kv4_attn(q, cache, i32(table), i32([24, 24]), max_seqlen_q=8)
        # queries 0 .. 3 of request 0 (positions 16 .. 19) and all of request 1
        q64 = q.double().cpu().numpy()
        want, wlse, mass, _ = ref.attention(q64[:8], *kv[0], 1 / math.sqrt(d), True)
        got = o[:8].double().cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(want)), where
        assert np.array_equal(np.isnan(lse[:, :8].cpu().numpy()), np.isnan(wlse))
        clean = [(kv[0][0][:, :20], kv[0][1][:, :20])]
        check_attention(o[:4], lse[:, :4], [(0, 4)], q64[:4], clean, 1 / math.sqrt(d), True, 2)
        check_attention(o[8:], lse[:, 8:], [(0, 8)], q64[8:], [kv[1]], 1 / math.sqrt(d), True, 2)


@pytest.mark.gpu
def test_large_queries_and_zero_rows():
    """Scores far apart (one key takes all), a query of zeros (uniform weights), queries near the ends of bf16's range."""
    rng = np.random.default_rng(8)
    cache, table, kv = filled(rng, [90], 1, 16, 64)
    q = torch.from_numpy(rng.standard_normal((1, 8, 64))).to(torch.bfloat16)
    q[0, 0] = 0
    q[0, 1] *= 100
    q[0, 2] *= 2.0 ** 100
    q[0, 3] *= 2.0 ** -120
    q[0, 4, 1:] = 0
    q[0, 5, 0] *= 2.0 ** 20  # one large column beside small ones
    scales = [0.125] * 2 + [2.0 ** -100] + [0.125] * 5
    for h in (0, 1, 3, 4, 5, 6, 7):
        o, lse = fa2.fa2_kv4_attn(q[:, h:h + 1].contiguous().cuda(), cache, i32(table), i32([90]), scale=scales[h])
        check_attention(o, lse, [(0, 1)], q[:, h:h + 1].double().numpy(), kv, scales[h], True, 1)
    o, lse = fa2.fa2_kv4_attn(q[:, 2:3].contiguous().cuda(), cache, i32(table), i32([90]), scale=2.0 ** -100)
    check_attention(o, lse, [(0, 1)], q[:, 2:3].double().numpy(), kv, 2.0 ** -100, True, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [0, 128])
def test_bad_lengths_and_pages_are_reported(wide):
    rng = np.random.default_rng(9)
    lens = [40, 50, 60]
    cache, table, kv = filled(rng, lens, 2, 16, 64, width=wide)
    q = torch.from_numpy(rng.standard_normal((3, 4, 64))).to(torch.bfloat16).cuda()
    q64 = q.double().cpu().numpy()
    fa2.fa2_device_status(reset=True)
    for bad in ([40, -1, 60], [40, 65 + 16 * wide, 60]):  # 4 (and `wide`) pages of 16 a row
        o, lse = torch.full_like(q, 9.0), torch.full((4, 3), 9.0, device="cuda")
        fa2.fa2_kv4_attn(q, cache, i32(table), i32(bad), o=o, lse=lse)
        assert fa2.fa2_device_status(reset=True) == 3
        assert torch.all(o[1] == 9) and torch.all(lse[:, 1] == 9)
        check_attention(o, lse, [(0, 1), (1, 1), (2, 3)], q64, kv, 0.125, True, 4)
    o = torch.full_like(q, 9.0)
    fa2.fa2_kv4_attn(q, cache, i32(table), i32(lens), o=o, max_seqlen_k=50)  # longer than the bound
    assert fa2.fa2_device_status(reset=True) == 3 and torch.all(o[2] == 9) and not torch.any(o[:2] == 9)
    # query offsets: backwards, past the end, longer than stated
    for cu in ([0, 2, 1, 3], [0, 1, 2, 5], [-1, 1, 2, 3], [0, 2, 3, 3]):
        o = torch.full_like(q, 9.0)
        fa2.fa2_kv4_attn(q, cache, i32(table), i32(lens), i32(cu), 1, o=o)
        assert fa2.fa2_device_status(reset=True) == 3, cu
    # a page id out of range: its 16 keys are left out
    t = table.copy()
    t[1, 2] = cache.shape[0]
    o, lse = fa2.fa2_kv4_attn(q, cache, i32(t), i32(lens))
    assert fa2.fa2_device_status(reset=True) == 5
    keep = np.r_[0:32, 48:50]
    kv[1] = tuple(x[:, keep] for x in kv[1])
    check_attention(o, lse, [(0, 1), (1, 2), (2, 3)], q64, kv, 0.125, True, 4)


@pytest.mark.gpu
def test_graphs_that_share_a_workspace_and_streams():
    rng = np.random.default_rng(10)
    lens = [300, 170]
    cache, table, kv = filled(rng, lens, 2, 16, 128)
    t, n = i32(table), i32(lens)
    qs = [torch.from_numpy(rng.standard_normal((2, 8, 128))).to(torch.bfloat16).cuda() for _ in range(2)]
    want = [fa2.fa2_kv4_attn(q, cache, t, n) for q in qs]
    t = torch.cat([t, torch.full((2, 128), -1, dtype=torch.int32, device="cuda")], 1)  # more than 2048 keys: needs a workspace
    want = [fa2.fa2_kv4_attn(q, cache, t, n) for q in qs]
    ws = torch.empty(fa2.fa2_kv4_attn_workspace_bytes(2, 8, 2, 1, t.shape[1] * 16, 128), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    graphs, outs = [], []
    for q in qs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(fa2.fa2_kv4_attn(q, cache, t, n, workspace=ws))
    for order in ((0, 1, 0), (1, 0, 1)):
        for o, lse in outs:
            o.zero_(), lse.zero_()
        for i in order:
            graphs[i].replay()
        for (o, lse), (wo, wl) in zip(outs, want):
            assert torch.equal(o, wo) and torch.equal(lse, wl)
    # other lengths in a captured step
    n.copy_(i32([17, 299]))
    t[:, :table.shape[1]] = i32(table[::-1].copy())
    graphs[0].replay()
    check_attention(*outs[0], [(0, 1), (1, 2)], qs[0].double().cpu().numpy(),
                    [tuple(x[:, :17] for x in kv[1]), tuple(x[:, :299] for x in kv[0])], 128 ** -0.5, True, 8)
    n.copy_(i32(lens))
    t[:, :table.shape[1]] = i32(table)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = fa2.fa2_kv4_attn(qs[0], cache, t, n, stream=side)
    b = fa2.fa2_kv4_attn(qs[1], cache, t, n)  # at the same time, each with a workspace of its own
    torch.cuda.current_stream().wait_stream(side)
    for got, w in ((a, want[0]), (b, want[1])):
        assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])


@pytest.mark.gpu
def test_empty_batch_and_foreign_stream_are_refused():
    cache = fa2.fa2_kv4_cache(2, 1, 16, 16)
    none, table = torch.zeros(0, dtype=torch.int32, device="cuda"), torch.zeros((0, 1), dtype=torch.int32, device="cuda")
    q = torch.zeros((0, 1, 16), dtype=torch.bfloat16, device="cuda")
    for call in (lambda: fa2.fa2_kv4_attn(q, cache, table, none),
                 lambda: fa2.fa2_kv4_attn(q, cache, table, none, i32([0]), 1),
                 lambda: fa2.fa2_kv4_gather(cache, table, i32([0]), 0),
                 lambda: fa2.fa2_page_plan(none, none, none, table, 16, 0)):
        with pytest.raises(fa2.FA2Error):
            call()
    with pytest.raises(ValueError):
        fa2._on(torch.cuda.current_device() + 1, torch.cuda.Stream())


@pytest.mark.gpu
def test_cache_past_32_bits():
    """Pages beyond 4 GB and slots beyond 2^31: what is written at the far end is read there by both readers."""
    P, d, T = 128, 16, 200
    pages = (1 << 24) + 3  # 39 GB
    cache = torch.empty((pages, 1, P // 16, 18 * d), dtype=torch.uint8, device="cuda")
    table = i32([[pages - 1, (1 << 24) - 1]])
    at = torch.arange(T, device="cuda")
    slots = table[0].long()[at // P] * P + at % P
    assert int(slots.max()) >= 1 << 31 and cache.numel() > 1 << 32
    near = fa2.fa2_kv4_cache(2, 1, P, d)
    k, v, q = (torch.randn(T, 1, d, device="cuda", generator=torch.Generator("cuda").manual_seed(i)).to(torch.bfloat16) for i in range(3))
    fa2.fa2_device_status(reset=True)
    plan = fa2.fa2_page_plan(i32([0]), i32([T]), table[0].contiguous(), table.clone().fill_(-1), P, T)
    assert torch.equal(plan.slots, slots)
    fa2.fa2_kv4_append(k, v, cache, slots)
    fa2.fa2_kv4_append(k, v, near, at)
    two = i32([[0, 1]])
    for a, b in zip(fa2.fa2_kv4_gather(cache, table, i32([0, T]), T), fa2.fa2_kv4_gather(near, two, i32([0, T]), T)):
        assert torch.equal(a, b)
    for bound in (T, 2 ** 20):  # (the table's room is the bound where it is less: the same form)
        got = fa2.fa2_kv4_attn(q[:4], cache, table, i32([T]), max_seqlen_k=bound)
        want = fa2.fa2_kv4_attn(q[:4], near, two, i32([T]), max_seqlen_k=bound)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # the line's form, which a wide table brings
    width = 64
    far, close = (torch.cat([t, t.new_zeros(1, width - 2)], 1) for t in (table, two))
    assert fa2.fa2_kv4_attn_workspace_bytes(1, 1, 1, 4, width * P, d) > 0
    got, want = fa2.fa2_kv4_attn(q[:4], cache, far, i32([T])), fa2.fa2_kv4_attn(q[:4], near, close, i32([T]))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert fa2.fa2_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("B,n,H,Hkv,nq,d,P", [(90, 350, 4, 2, 1, 128, 16), (23, 800, 16, 8, 1, 64, 64), (40, 70, 16, 4, 5, 32, 32),
                                              (17, 1000, 30, 10, 7, 128, 128), (160, 40, 1, 1, 2, 16, 16)])
def test_attention_more_units_than_sms(B, n, H, Hkv, nq, d, P):
    """Many units of short requests: a small CTA each, or (by the bound on the lengths alone) many units in a span."""
    rng = np.random.default_rng(n)
    lens = [n, 0, 1, 31, 33] + [int(x) for x in rng.integers(0, n, B - 5)]
    nqs = [nq] * (B - 3) + [0, 1, nq]
    cache, table, kv = filled(rng, lens, Hkv, P, d, width=4096 // P)
    cu = np.r_[0, np.cumsum(nqs)]
    total = int(cu[-1])
    q = torch.from_numpy(rng.standard_normal((total, H, d))).to(torch.bfloat16).cuda()
    rows = [(int(cu[b]), int(cu[b + 1])) for b in range(B)]
    fa2.fa2_device_status(reset=True)
    for bound in (n, None):
        assert (fa2.fa2_kv4_attn_workspace_bytes(B, H, Hkv, nq, bound or table.shape[1] * P, d) > 0) == (bound is None)
        for causal in (True, False):
            o, lse = fa2.fa2_kv4_attn(q, cache, i32(table), i32(lens), i32(cu), nq, max_seqlen_k=bound, causal=causal)
            check_attention(o, lse, rows, q.double().cpu().numpy(), kv, 1 / math.sqrt(d), causal, H)
            again = fa2.fa2_kv4_attn(q, cache, i32(table), i32(lens), i32(cu), nq, max_seqlen_k=bound, causal=causal)
            assert torch.equal(again[0], o) and torch.equal(again[1], lse)
    assert fa2.fa2_device_status() == 0
    # a length past the bound and a page that does not exist: reported, the other requests as before
    at = lens.index(max(lens[5:-3]), 5)
    o, lse = fa2.fa2_kv4_attn(q, cache, i32(table), i32(lens), i32(cu), nq, max_seqlen_k=n)
    bad = list(lens)
    bad[at] = n + 1
    o2, lse2 = torch.full_like(o, 9.0), torch.full_like(lse, 9.0)
    fa2.fa2_kv4_attn(q, cache, i32(table), i32(bad), i32(cu), nq, max_seqlen_k=n, o=o2, lse=lse2)
    assert fa2.fa2_device_status(reset=True) == 3
    mine = torch.zeros(total, dtype=torch.bool, device="cuda")
    mine[rows[at][0]:rows[at][1]] = True
    assert torch.all(o2[mine] == 9) and torch.all(lse2[:, mine] == 9)
    assert torch.equal(o2[~mine], o[~mine]) and torch.equal(lse2[:, ~mine], lse[:, ~mine])
    missing = table.copy()
    missing[at, 0] = cache.shape[0]
    o3, lse3 = fa2.fa2_kv4_attn(q, cache, i32(missing), i32(lens), i32(cu), nq, max_seqlen_k=n)
    assert fa2.fa2_device_status(reset=True) == 5
    assert torch.equal(o3[~mine], o[~mine]) and torch.equal(lse3[:, ~mine], lse[:, ~mine])


@pytest.mark.gpu
@pytest.mark.parametrize("B", [512, 513, 4096, 4097, 16384])
def test_plan_at_the_sizes_where_its_layout_changes(B):
    test_plan(B, 16, 40, 3)
    rng = np.random.default_rng(B)
    cached, new = rng.integers(0, 40, B), rng.integers(0, 4, B)
    bad = rng.choice(B, 7, replace=False)
    odd = cached.copy()
    odd[bad] = [-1, -2 ** 31, 2 ** 31 - 1, 65, 64, -5, 1000]
    cached[bad] = 0
    fewer, more = new.copy(), new.copy()
    fewer[bad], more[bad] = 0, 1
    free = i32(np.arange(4 * B))
    T = int(fewer.sum())
    fa2.fa2_device_status(reset=True)
    tables = [torch.full((B, 4), -7, dtype=torch.int32, device="cuda") for _ in range(2)]
    want = fa2.fa2_page_plan(i32(cached), i32(fewer), free, tables[0], 16, T)
    assert fa2.fa2_device_status() == 0
    got = fa2.fa2_page_plan(i32(odd), i32(more), free, tables[1], 16, T)
    assert fa2.fa2_device_status(reset=True) == 3
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(*tables)


@pytest.mark.gpu
@pytest.mark.parametrize("B,most,H,Hkv,d", [(40, 300, 4, 1, 128), (33, 77, 6, 2, 64), (70, 90, 3, 3, 16), (1100, 200, 2, 1, 32)])
def test_attention_ragged_queries(B, most, H, Hkv, d):
    """A few requests have most of the queries; offsets that do not begin at 0; a request that is left out."""
    rng = np.random.default_rng(B)
    nqs = rng.integers(0, 3, B)
    nqs[[0, B // 2, B - 1]] = [most // 2, most, 5]
    lens = rng.integers(0, 40 if B < 1000 else 5, B)
    lens[[0, B // 2, B - 1]] = [most, most + 100, 3]
    cache, table, kv = filled(rng, [int(x) for x in lens], Hkv, 16, d, width=64)
    cu = 4 + np.r_[0, np.cumsum(nqs)]
    total = int(cu[-1]) + 6
    q = torch.from_numpy(rng.standard_normal((total, H, d))).to(torch.bfloat16).cuda()
    rows = [(int(cu[b]), int(cu[b + 1])) for b in range(B)]
    fa2.fa2_device_status(reset=True)
    left = torch.ones(total, dtype=torch.bool, device="cuda")
    left[int(cu[0]):int(cu[-1])] = False
    for bound in (most + 100, 1 << 20):
        o, lse = torch.full_like(q, 9.0), torch.full((H, total), 9.0, device="cuda")
        tab = i32(table) if bound < 1 << 20 else torch.cat([i32(table), torch.zeros((B, 100), dtype=torch.int32, device="cuda")], 1)
        fa2.fa2_kv4_attn(q, cache, tab, i32(lens), i32(cu), most, max_seqlen_k=bound, o=o, lse=lse)
        assert (fa2.fa2_kv4_attn_workspace_bytes(B, H, Hkv, most, min(bound, tab.shape[1] * 16), d) > 0) == (bound == 1 << 20)
        assert fa2.fa2_device_status() == 0
        check_attention(o, lse, rows, q.double().cpu().numpy(), kv, 1 / math.sqrt(d), True, H)
        assert torch.all(o[left] == 9) and torch.all(lse[:, left] == 9)
        for at, bad_len in ((B // 2, -1), (1, 1 << 24)):
            bad = lens.copy()
            bad[at] = bad_len
            o2, lse2 = torch.full_like(q, 9.0), torch.full_like(lse, 9.0)
            fa2.fa2_kv4_attn(q, cache, tab, i32(bad), i32(cu), most, max_seqlen_k=bound, o=o2, lse=lse2)
            assert fa2.fa2_device_status(reset=True) == 3
            mine = left.clone()
            mine[rows[at][0]:rows[at][1]] = True
            assert torch.all(o2[mine] == 9)
            if bound < 1 << 20:
                assert torch.equal(o2[~mine], o[~mine]) and torch.equal(lse2[:, ~mine], lse[:, ~mine])
            else:  # (the line is cut elsewhere: sums in another order)
                others = [r if i != at else (0, 0) for i, r in enumerate(rows)]
                check_attention(o2, lse2, others, q.double().cpu().numpy(), kv, 1 / math.sqrt(d), True, H)
    # offsets that go down, and past the queries: nothing out of range is read or written
    for at, x in ((B // 3, total + 1000), (B // 2, -5)):
        wrong = cu.copy()
        wrong[at] = x
        o2, lse2 = torch.full_like(q, 9.0), torch.full_like(lse, 9.0)
        fa2.fa2_kv4_attn(q, cache, i32(table), i32(lens), i32(wrong), most, max_seqlen_k=most + 100, o=o2, lse=lse2)
        assert fa2.fa2_device_status(reset=True) == 3
        assert torch.all(o2[left] == 9)


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hkv,d", [(300, 12, 16), (100, 5, 16), (77, 33, 128), (65, 9, 32), (40, 20, 64), (1, 1, 16), (3001, 16, 32)])
def test_append_head_counts_that_do_not_fill_a_block(T, Hkv, d):
    test_append_many_tokens_and_back(T, Hkv, d)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,H,Hkv,nq,d", [([2048] * 19, 8, 8, 1, 64),    # every unit is one CTA's part of the line
                                             ([4096] * 19, 8, 4, 1, 32),    # two CTAs'
                                             ([2048] * 19, 128, 8, 1, 16),  # the same with 16 rows: parts that straddle
                                             ([60000], 4, 1, 1, 16), ([60000], 4, 1, 3, 16),
                                             ([30011, 5, 20000, 0, 9000], 2, 2, 1, 32),
                                             # few units, whose CTAs join their warps: all ends at CTAs' ends
                                             ([12288] * 19, 4, 1, 1, 16), ([9216] * 19, 16, 1, 1, 16),
                                             # a unit that is the share of one CTA of seven warps, behind a long one
                                             ([60032, 448], 2, 1, 1, 16), ([60032, 448], 16, 1, 1, 16),
                                             ([60000, 448, 0, 3], 1, 1, 1, 64), ([131072], 8, 1, 1, 128),
                                             ([20000, 130000], 24, 2, 1, 32)],
                         ids=lambda x: f"{len(x)}x{max(x)}" if isinstance(x, list) else str(x))
def test_attention_units_of_whole_ctas(lens, H, Hkv, nq, d):
    """Units that are long against a CTA's part of the line, whose warps join their results before the combine."""
    P, g = 128, torch.Generator(device="cuda").manual_seed(len(lens))
    counts = [-(-x // P) for x in lens]
    table, at = np.zeros((len(lens), max(max(counts), 16384 // P)), np.int64), 0
    cache = fa2.fa2_kv4_cache(sum(counts), Hkv, P, d)
    kv = []
    for b, x in enumerate(lens):
        table[b, :counts[b]] = np.arange(at, at + counts[b])
        at += counts[b]
        ramp = torch.linspace(0.2, 2.0, x, device="cuda")[:, None, None]
        k = (torch.randn(x, Hkv, d, generator=g, device="cuda") * ramp).to(torch.bfloat16)
        v = torch.randn(x, Hkv, d, generator=g, device="cuda").to(torch.bfloat16)
        ko, vo = torch.empty_like(k), torch.empty_like(v)
        pos = torch.arange(x, device="cuda")
        fa2.fa2_kv4_append(k, v, cache, i32(table[b]).long()[pos // P] * P + pos % P, k_out=ko, v_out=vo)
        kv.append([t.double().cpu().numpy().transpose(1, 0, 2) for t in (ko, vo)])
    q = torch.randn(len(lens) * nq, H, d, generator=g, device="cuda").to(torch.bfloat16)
    fa2.fa2_device_status(reset=True)
    assert fa2.fa2_kv4_attn_workspace_bytes(len(lens), H, Hkv, nq, table.shape[1] * P, d) > 0
    o, lse = fa2.fa2_kv4_attn(q, cache, i32(table), i32(lens))
    assert fa2.fa2_device_status() == 0
    rows = [(b * nq, (b + 1) * nq) for b in range(len(lens))]
    check_attention(o, lse, rows, q.double().cpu().numpy(), kv, 1 / math.sqrt(d), True, H)
    again = fa2.fa2_kv4_attn(q, cache, i32(table), i32(lens))
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,Hkv,nq,d,lens", [(1, 8, 1, 1, 128, [2048]), (1, 32, 8, 1, 64, [1100]), (3, 4, 2, 2, 32, [1500, 0, 33]),
                                               (4, 8, 8, 1, 16, [1, 31, 2047, 1025]), (2, 16, 1, 1, 128, [600, 2000]),
                                               (20, 4, 1, 3, 16, [1030] + list(range(0, 190, 10))),
                                               (8, 10, 5, 1, 32, [2000, 64, 0, 1, 500, 96, 7, 1999]),
                                               (6, 24, 2, 3, 64, [800, 700, 0, 5, 769, 32])])
def test_attention_units_of_clusters(B, H, Hkv, nq, d, lens):
    """Few units of one to two thousand keys: eight, four or two CTAs each, some with no key."""
    rng = np.random.default_rng(B)
    cache, table, kv = filled(rng, lens, Hkv, 32, d)
    q = torch.from_numpy(rng.standard_normal((B * nq, H, d)) * 2).to(torch.bfloat16).cuda()
    rows = [(b * nq, (b + 1) * nq) for b in range(B)]
    bound = max(max(lens), 769 if B == 6 else 1025)
    fa2.fa2_device_status(reset=True)
    assert fa2.fa2_kv4_attn_workspace_bytes(B, H, Hkv, nq, bound, d) == 0
    tab = torch.cat([i32(table), torch.zeros((B, 2), dtype=torch.int32, device="cuda")], 1)
    for causal in (True, False):
        o, lse = fa2.fa2_kv4_attn(q, cache, tab, i32(lens), max_seqlen_k=bound, causal=causal)
        check_attention(o, lse, rows, q.double().cpu().numpy(), kv, 1 / math.sqrt(d), causal, H)
        again = fa2.fa2_kv4_attn(q, cache, tab, i32(lens), max_seqlen_k=bound, causal=causal)
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)
    assert fa2.fa2_device_status() == 0
    bad = list(lens)
    bad[-1] = -1
    o2, lse2 = torch.full_like(o, 9.0), torch.full_like(lse, 9.0)
    fa2.fa2_kv4_attn(q, cache, tab, i32(bad), max_seqlen_k=bound, causal=False, o=o2, lse=lse2)
    assert fa2.fa2_device_status(reset=True) == 3
    at = rows[-1][0]
    assert torch.all(o2[at:] == 9) and torch.equal(o2[:at], o[:at]) and torch.equal(lse2[:, :at], lse[:, :at])
