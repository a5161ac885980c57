"""The paged cache in bf16 and e4m3, and the rotation's table, at the ends of their ranges."""
import math

import numpy as np
import pytest
import torch

import tiled_exact_attention_fa2_gb300 as fa2
from test_kv import bits, check_attention, filled, i32

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
