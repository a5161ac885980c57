"""The operators around the attention together, as a layer uses them: serving steps over the paged cache (plan, norm and
rotation, append, attention or gather), captured and replayed, and the training pass norm -> attention -> gradients."""
import math

import numpy as np
import pytest
import torch

import oracle
import oracle.kv4 as kv4
import oracle.norm_rope as nr
import tiled_exact_attention_fa2_gb300 as fa2
from parity_util import check_grad, check_lse, check_o
from test_kv4 import check_attention, i32
from test_norm_rope import table

pytestmark = pytest.mark.gpu


class Server:
    """A few requests of one layer: the GPU state a serving program keeps."""

    def __init__(self, B, H, Hkv, d, P, pages, seed):
        self.B, self.H, self.Hkv, self.d, self.P = B, H, Hkv, d, P
        self.g = torch.Generator().manual_seed(seed)
        self.w = [(1 + 0.2 * torch.randn(d, generator=self.g)).to(torch.bfloat16).cuda() for _ in range(2)]
        self.rope_np = table(4096, d)
        self.rope = torch.from_numpy(self.rope_np).cuda()
        self.cache = fa2.fa2_kv4_cache(pages, Hkv, P, d)
        self.cache.fill_(0xFF)
        self.free = list(np.random.default_rng(seed).permutation(pages))
        self.table = torch.full((B, 24), -1, dtype=torch.int32, device="cuda")
        self.lens = np.zeros(B, int)

    def qkv(self, tokens):
        return torch.randn(tokens, self.H + 2 * self.Hkv, self.d, generator=self.g).to(torch.bfloat16).cuda()

    def step(self, new, pad=3):
        """One step with new[b] tokens of request b; its plan, q, k, v, o, lse."""
        T = int(sum(new)) + pad
        qkv = self.qkv(T)
        plan = fa2.fa2_page_plan(i32(self.lens), i32(new), i32(self.free), self.table, self.P, T)
        H, Hkv = self.H, self.Hkv
        q, k = fa2.fa2_qk_norm_rope(qkv[:, :H], qkv[:, H:H + Hkv], *self.w, self.rope, plan.positions)
        ks, vs = torch.empty_like(k), torch.empty_like(k)
        fa2.fa2_kv4_append(k, qkv[:, H + Hkv:], self.cache, plan.slots, k_out=ks, v_out=vs)
        o, lse = fa2.fa2_kv4_attn(q, self.cache, self.table, plan.lens, plan.cu_new, max(new))
        self.free = self.free[int(plan.pages_needed):]
        old, self.lens = self.lens, self.lens + np.asarray(new)
        return plan, qkv, q, k, ks, vs, o, lse, old

    def held(self):
        host, t = self.cache.cpu().numpy(), self.table.cpu().numpy()
        return [kv4.read(host, t[b], self.lens[b], 1.0, 1.0) if self.lens[b] else (np.zeros((self.Hkv, 0, self.d)),) * 2
                for b in range(self.B)]


@pytest.mark.parametrize("H,Hkv,d,P", [(8, 2, 128, 16), (6, 6, 64, 64)])
def test_serving_steps(H, Hkv, d, P):
    s = Server(4, H, Hkv, d, P, 64, 1)
    stored = [([], []) for _ in range(4)]
    fa2.fa2_device_status(reset=True)
    for new in ([37, 0, 64, 5], [1, 1, 1, 1], [1, 20, 0, 1], [1, 1, 1, 1], [4, 4, 4, 4]):
        plan, qkv, q, k, ks, vs, o, lse, old = s.step(new)
        cu = plan.cu_new.tolist()
        for b in range(4):
            n = slice(cu[b], cu[b + 1])
            pos = np.arange(old[b], old[b] + new[b])
            cos, sin = (s.rope_np[pos][:, None, i].astype(np.float64) for i in (slice(0, d // 2), slice(d // 2, d)))
            for got, x, w in ((q, qkv[n, :H], s.w[0]), (k, qkv[n, H:H + Hkv], s.w[1])):
                want = nr.forward(x.double().cpu().numpy(), w.double().cpu().numpy(), cos, sin, 1e-6, False)
                # bf16 store, and the kernel's fp32 arithmetic
                assert np.all(np.abs(got[n].double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -16)
            stored[b][0].append(ks[n].double().cpu().numpy())
            stored[b][1].append(vs[n].double().cpu().numpy())
        held = s.held()
        for b in range(4):  # the cache holds what the append said it stored
            for i in range(2):
                assert np.array_equal(held[b][i].transpose(1, 0, 2), np.concatenate(stored[b][i]))
        check_attention(o, lse, [(cu[b], cu[b + 1]) for b in range(4)], q.double().cpu().numpy(), held, d ** -0.5, True, H)
        # the same queries through the packed attention on the gathered cache
        total = int(s.lens.sum())
        kk, vv = fa2.fa2_kv4_gather(s.cache, s.table, plan.cu_total, total)
        o2, lse2 = fa2.fa2_fwd_varlen(q[:cu[-1]].contiguous(), kk, vv, plan.cu_new, plan.cu_total, max(new), int(s.lens.max()))
        want_o, want_l = zip(*[kv4.attention(q[cu[b]:cu[b + 1]].double().cpu().numpy(), *held[b], d ** -0.5, True)[:2] for b in range(4)])
        check_o(o2.double().cpu().numpy(), np.concatenate(want_o))
        check_lse(lse2.double().cpu().numpy(), np.concatenate(want_l, 1))
    assert fa2.fa2_device_status() == 0


def test_decoding_step_captured_and_replayed():
    """One captured step serves growing requests: only the lengths, the free list and the projections change."""
    B, H, Hkv, d, P = 3, 8, 2, 128, 16
    s = Server(B, H, Hkv, d, P, 40, 2)
    s.step([30, 15, 48])
    cached, new, free = i32(s.lens), i32([1] * B), i32(s.free)
    qkv, T = s.qkv(B), B

    def run(plan=None):
        plan = fa2.fa2_page_plan(cached, new, free, s.table, P, T, plan=plan)
        q, k = fa2.fa2_qk_norm_rope(qkv[:, :H], qkv[:, H:H + Hkv], *s.w, s.rope, plan.positions)
        fa2.fa2_kv4_append(k, qkv[:, H + Hkv:], s.cache, plan.slots)
        return plan, q, fa2.fa2_kv4_attn(q, s.cache, s.table, plan.lens)

    before = s.cache.clone(), s.table.clone()
    run()
    s.cache.copy_(before[0]), s.table.copy_(before[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan, q, (o, lse) = run()
    for _ in range(20):
        qkv.copy_(s.qkv(B))
        graph.replay()
        s.lens = s.lens + 1
        check_attention(o, lse, [(b, b + 1) for b in range(B)], q.double().cpu().numpy(), s.held(), d ** -0.5, True, H)
        used = int(plan.pages_needed)
        free.copy_(torch.cat([free[used:], free[:used]]))
        cached.copy_(plan.lens)
    assert fa2.fa2_device_status() == 0


@pytest.mark.parametrize("B,H,Hkv,N,d,rot,inter", [(1, 2, 2, 70, 64, 32, True), (2, 4, 2, 130, 128, 128, False)])
def test_training_pass(B, H, Hkv, N, d, rot, inter):
    """norm + rotation -> attention -> both backward passes against fp64 throughout (bf16 between the steps; the
    attention's gradient bound holds for the whole)."""
    g = torch.Generator().manual_seed(N)
    x = torch.randn(B, N, H + Hkv, d, generator=g).to(torch.bfloat16).cuda()
    q, k = x[:, :, :H].transpose(1, 2), x[:, :, H:].transpose(1, 2)
    v, dO = (torch.randn(B, h, N, d, generator=g).to(torch.bfloat16).cuda() for h in (Hkv, H))
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g) for _ in range(2))
    tab = table(N, rot)
    rope = torch.from_numpy(tab).cuda()
    args = dict(q_weight=wq.cuda(), k_weight=wk.cuda(), rope=rope, interleaved=inter)
    qn, kn = fa2.fa2_qk_norm_rope(q, k, **args)
    o, lse = fa2.fa2_fwd_gqa(qn, kn, v)
    dqn, dkn, dv = fa2.fa2_bwd_gqa(qn, kn, v, o, dO, lse)
    grad = torch.zeros_like(x)
    dq, dk, dwq, dwk = fa2.fa2_qk_norm_rope_bwd(dqn, dkn, q, k, dq=grad[:, :, :H].transpose(1, 2), dk=grad[:, :, H:].transpose(1, 2),
                                                **args)
    cos, sin = (tab[:, i].astype(np.float64) for i in (slice(0, rot // 2), slice(rot // 2, rot)))
    q64, k64 = (t.double().cpu().numpy() for t in (q, k))
    w64 = [w.double().numpy() for w in (wq, wk)]
    a, b = (nr.forward(t, w, cos, sin, 1e-6, inter) for t, w in zip((q64, k64), w64))
    G = H // Hkv
    rep = lambda t: np.repeat(t, G, 1)  # noqa: E731
    r = oracle.attn_bwd(a, rep(b), rep(v.double().cpu().numpy()), dO.double().cpu().numpy(), 1 / math.sqrt(d), True)
    check_o(o.double().cpu().numpy(), r["O"])
    gk = r["dK"].reshape(B, Hkv, G, N, d).sum(2)
    for got, dw, gr, t, w, name in ((dq, dwq, r["dQ"], q64, w64[0], "dQ"), (dk, dwk, gk, k64, w64[1], "dK")):
        want, want_w, _, _ = nr.backward(gr, t, w, cos, sin, 1e-6, inter)
        check_grad(got.double().cpu().numpy(), want, name)
        check_grad(dw.double().cpu().numpy(), want_w, name + " weight")
    assert torch.equal(grad[:, :, :H].transpose(1, 2), dq) and fa2.fa2_device_status() == 0
