"""The 4-bit paged cache where its calls meet what a caller gets wrong or leaves empty."""
import math

import numpy as np
import pytest
import torch

import tiled_exact_attention_fa2_gb300 as fa2
from test_kv4 import A, attn, check_attention, filled, i32


# ---------------------------------------------------------------- CPU
@pytest.fixture(scope="module")
def lib():
    from tiled_exact_attention_fa2_gb300 import _build
    _build.build()
    return fa2.load_library()


def test_no_queries_under_any_bound(lib):
    for cu in (5 * A, None):
        for mq in (0, 1, 7, 2 ** 31 - 1):
            assert attn(lib, tq=0, mq=mq, cu=cu) == 0
    assert attn(lib, tq=0, mq=-1) == 2 and attn(lib, tq=0, mq=1, B=0) == 2 and attn(lib, tq=0, mq=1, cache=None) == 1


def test_workspace_rule_as_documented(lib):
    """Which bounds need a workspace, which is not monotone in the bound, and one that is enough for all of them."""
    ws = lib.fa2_kv4_attn_workspace_bytes
    rng = np.random.default_rng(6)
    for _ in range(2000):
        B, Hkv, G, nq = (int(x) for x in np.exp(rng.uniform(0, np.log([400, 16, 16, 20]))))
        rows = G * nq
        units = B * Hkv * -(-rows // (16 if rows > 8 else 8))
        bound = int(np.exp(rng.uniform(0, np.log(20000))))
        if units <= 152:
            none = bound <= max(2048, 54 * units)
        else:
            none = bound <= (1024 if rows > 8 else 2048) and (units <= 1216 or bound >= 128)
        most = ws(B, G * Hkv, Hkv, nq, 1 << 30, 64)
        assert most > 0 and ws(B, G * Hkv, Hkv, nq, bound, 64) == (0 if none else most)
    # 2048 units: none needed under a bound of 2048 keys, but under one of 100
    long, short = dict(B=256, H=32, Hkv=8, tq=256, mq=1, W=128, mk=2048), dict(B=256, H=32, Hkv=8, tq=256, mq=1, W=128, mk=100)
    assert attn(lib, ws=None, o=A, **long) == 9 and attn(lib, ws=None, o=A, **short) == 8
    assert attn(lib, o=A, wsb=ws(256, 32, 8, 1, 1 << 30, 64), **short) == 9


# ---------------------------------------------------------------- GPU
@pytest.mark.gpu
def test_query_bounds_above_the_rows_there_are():
    """A step's rounded-up max_seqlen_q over fewer rows, and a step without any."""
    rng = np.random.default_rng(4)
    cache, table, kv = filled(rng, [40, 70], 2, 16, 64)
    t, lens = i32(table), i32([40, 70])
    q = torch.from_numpy(rng.standard_normal((5, 4, 64))).to(torch.bfloat16).cuda()
    fa2.fa2_device_status(reset=True)
    want = fa2.fa2_kv4_attn(q, cache, t, lens, i32([0, 2, 5]), 5)
    check_attention(*want, [(0, 2), (2, 5)], q.double().cpu().numpy(), kv, 0.125, True, 4)
    for bound in (8, 2 ** 31 - 1, 2 ** 40):
        got = fa2.fa2_kv4_attn(q, cache, t, lens, i32([0, 2, 5]), bound)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for bound in (0, 1, 8):
        o, lse = fa2.fa2_kv4_attn(q[:0], cache, t, lens, i32([0, 0, 0]), bound)
        assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
    assert fa2.fa2_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("B,most,H,Hkv,d", [(40, 300, 4, 1, 128), (70, 90, 3, 3, 16), (1100, 200, 2, 1, 32)])
def test_a_wrong_query_offset_costs_only_its_own_requests(B, most, H, Hkv, d):
    """Ragged queries: an offset far too small or too large takes the two requests it belongs to, and no other, in both
    forms of the kernel."""
    rng = np.random.default_rng(B)
    nqs = rng.integers(1, 3, B)
    nqs[[0, B // 2, B - 1]] = [most // 2, most, 5]
    lens = rng.integers(0, 40 if B < 1000 else 5, B)
    lens[[0, B // 2, B - 1]] = [most, most + 100, 3]
    cache, table, kv = filled(rng, [int(x) for x in lens], Hkv, 16, d, width=64)
    cu = np.r_[0, np.cumsum(nqs)]
    total = int(cu[-1])
    q = torch.from_numpy(rng.standard_normal((total, H, d))).to(torch.bfloat16).cuda()
    q64 = q.double().cpu().numpy()
    fa2.fa2_device_status(reset=True)
    for bound in (most + 100, 1 << 20):
        tab = i32(table) if bound < 1 << 20 else torch.cat([i32(table), torch.zeros((B, 100), dtype=torch.int32, device="cuda")], 1)
        # (the second request, one in the middle of the long ones', where a search would look first, the last but one)
        for at in (1, B // 3, B // 2 + 1, 8 * (B // 16), B - 1):
            for x in (-7, total + 1000):
                wrong = cu.copy()
                wrong[at] = x
                o, lse = torch.full_like(q, 9.0), torch.full((H, total), 9.0, device="cuda")
                fa2.fa2_kv4_attn(q, cache, tab, i32(lens), i32(wrong), most, max_seqlen_k=bound, o=o, lse=lse)
                assert fa2.fa2_device_status(reset=True) == 3
                gone = slice(int(cu[at - 1]), int(cu[at + 1]))
                assert torch.all(o[gone] == 9) and torch.all(lse[:, gone] == 9)
                rows = [(int(cu[b]), int(cu[b + 1])) if b not in (at - 1, at) else (0, 0) for b in range(B)]
                check_attention(o, lse, rows, q64, kv, 1 / math.sqrt(d), True, H)


@pytest.mark.gpu
@pytest.mark.parametrize("Hkv", [1, 4])
def test_a_wrong_query_offset_among_few_requests(Hkv):
    """The same where a unit has a full CTA, a cluster of them, or spans of the line that several warps join."""
    rng = np.random.default_rng(Hkv)
    B, H, d, most = 6, 2 * Hkv, 64, 40
    nqs, lens = [1, 1, most, 1, 1, 5], [33, 250, 290, 1, 70, 17]
    cache, table, kv = filled(rng, lens, Hkv, 16, d, width=8192 // 16)
    cu = np.r_[0, np.cumsum(nqs)]
    total = int(cu[-1])
    q = torch.from_numpy(rng.standard_normal((total, H, d))).to(torch.bfloat16).cuda()
    q64 = q.double().cpu().numpy()
    fa2.fa2_device_status(reset=True)
    for bound in (300, 900, 8192):
        assert (fa2.fa2_kv4_attn_workspace_bytes(B, H, Hkv, most, bound, d) > 0) == (bound == 8192)
        want = fa2.fa2_kv4_attn(q, cache, i32(table), i32(lens), i32(cu), most, max_seqlen_k=bound)
        assert fa2.fa2_device_status() == 0
        check_attention(*want, [(int(cu[b]), int(cu[b + 1])) for b in range(B)], q64, kv, 1 / math.sqrt(d), True, H)
        for at in range(B + 1):
            for x in (-7, total + 1000):
                wrong = cu.copy()
                wrong[at] = x
                o, lse = torch.full_like(q, 9.0), torch.full((H, total), 9.0, device="cuda")
                fa2.fa2_kv4_attn(q, cache, i32(table), i32(lens), i32(wrong), most, max_seqlen_k=bound, o=o, lse=lse)
                assert fa2.fa2_device_status(reset=True) == 3
                gone = slice(int(cu[max(at - 1, 0)]), int(cu[min(at + 1, B)]))
                assert torch.all(o[gone] == 9) and torch.all(lse[:, gone] == 9)
                rows = [(int(cu[b]), int(cu[b + 1])) if b not in (at - 1, at) else (0, 0) for b in range(B)]
                check_attention(o, lse, rows, q64, kv, 1 / math.sqrt(d), True, H)
        # requests 2 and 4 on the same rows (their keys differ: the rows hold the one's or the other's), 3 backwards
        twice = np.r_[cu[:4], cu[2], cu[3], total]
        o, lse = torch.full_like(q, 9.0), torch.full((H, total), 9.0, device="cuda")
        fa2.fa2_kv4_attn(q, cache, i32(table), i32(lens), i32(twice), most, max_seqlen_k=bound, o=o, lse=lse)
        assert fa2.fa2_device_status(reset=True) == 3
        check_attention(o, lse, [(0, 1), (1, 2)], q64, kv[:2], 1 / math.sqrt(d), True, H)
        check_attention(o, lse, [(int(cu[3]), total)], q64, kv[5:], 1 / math.sqrt(d), True, H)
        both = lse[:, 2:int(cu[3])]
        assert torch.all(torch.isfinite(both) & (both != 9))


@pytest.mark.gpu
def test_query_offsets_that_overlap():
    """Offsets that go up and down give the same rows to several requests, and a tile's number to several tiles: every
    request whose own offsets are in range is computed (here they all have the same keys, so it does not show which
    wrote a row last)."""
    rng = np.random.default_rng(3)
    B, H, Hkv, d, most = 48, 4, 1, 64, 64
    cache, table, kv = filled(rng, [90], Hkv, 16, d, width=64)
    cu = np.zeros(B + 1, np.int64)
    cu[1::2] = most  # requests 0, 2, ...: all 64 rows; 1, 3, ...: backwards
    q = torch.from_numpy(rng.standard_normal((most, H, d))).to(torch.bfloat16).cuda()
    fa2.fa2_device_status(reset=True)
    for width in (0, 100):
        tab = torch.cat([i32(table), torch.zeros((1, width), dtype=torch.int32, device="cuda")], 1).expand(B, -1).contiguous()
        o, lse = torch.full_like(q, 9.0), torch.full((H, most), 9.0, device="cuda")
        fa2.fa2_kv4_attn(q, cache, tab, i32([90] * B), i32(cu), most, o=o, lse=lse)
        assert fa2.fa2_device_status(reset=True) == 3
        check_attention(o, lse, [(0, most)], q.double().cpu().numpy(), kv, 1 / math.sqrt(d), True, H)


@pytest.mark.gpu
@pytest.mark.parametrize("d,Hkv", [(16, 3), (128, 2)])
def test_gather_behind_a_gap(d, Hkv):
    """Rows before the first sequence and behind the last keep what they hold, and are no error; nor is a smaller total."""
    rng = np.random.default_rng(d)
    lens = [0, 33, 0, 20]
    cache, table, kv = filled(rng, lens, Hkv, 16, d)
    cu = 37 + np.r_[0, np.cumsum(lens)]
    fa2.fa2_device_status(reset=True)
    for total in (int(cu[-1]) + 9, int(cu[-1]) - 5, 37, 20):
        k, v = (torch.full((total, Hkv, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        fa2.fa2_kv4_gather(cache, i32(table), i32(cu), total, k=k, v=v)
        assert fa2.fa2_device_status(reset=True) == 0
        for got, i in ((k, 0), (v, 1)):
            want = np.full((max(total, int(cu[-1])), Hkv, d), 9.0)
            want[37:int(cu[-1])] = np.concatenate([x[i].transpose(1, 0, 2) for x in kv])
            assert np.array_equal(got.double().cpu().numpy(), want[:total])


@pytest.mark.gpu
@pytest.mark.parametrize("B", [4, 700])
def test_gather_reports_offsets_out_of_order(B):
    """Wherever they are: rows can fall to a sequence whose own offsets are right and whose table row has room for them."""
    lens = [20] * B
    cache = fa2.fa2_kv4_cache(2 * B, 1, 16, 16)
    table = i32(np.arange(2 * B))[None].expand(B, -1).contiguous()
    cu = np.r_[0, np.cumsum(lens)]
    fa2.fa2_device_status(reset=True)
    fa2.fa2_kv4_gather(cache, table, i32(cu), int(cu[-1]))
    assert fa2.fa2_device_status(reset=True) == 0
    for at, x in ((0, -1), (1, 45), (B // 2, 10 ** 9), (B - 1, -2 ** 31), (B, 0), (B, -1), (2, int(cu[1]) - 1)):
        wrong = cu.copy()
        wrong[at] = x
        fa2.fa2_kv4_gather(cache, table, i32(wrong), int(cu[-1]))
        assert fa2.fa2_device_status(reset=True) == 3, (at, x)


@pytest.mark.gpu
@pytest.mark.parametrize("P", [16, 64])
def test_gather_stops_at_the_table_rows_end(P):
    """A sequence of one token more than its row's only (valid) page holds: its last row is left out, with status 3."""
    rng = np.random.default_rng(P)
    cache, table, kv = filled(rng, [P, P], 2, P, 32, spare=0)
    beyond = torch.cat([i32(table[:1]), i32(table[1:])], 1)  # (what lies behind the row is a valid page as well)
    fa2.fa2_device_status(reset=True)
    k, v = (torch.full((P + 1, 2, 32), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fa2.fa2_kv4_gather(cache, beyond[:, :1], i32([0, P + 1]), P + 1, k=k, v=v)
    assert fa2.fa2_device_status(reset=True) == 3
    for got, i in ((k, 0), (v, 1)):
        assert np.array_equal(got[:P].double().cpu().numpy(), kv[0][i].transpose(1, 0, 2)) and torch.all(got[P] == 9)
