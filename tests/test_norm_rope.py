"""Per-head norm with position rotation: refusals and the definition's gradient on the CPU, the kernels on the GPU."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.norm_rope as ref
import tiled_exact_attention_fa2_gb300 as fa2

A = 1 << 22  # fake device addresses, far apart; never dereferenced


def table(n, rot, base=10000.0):
    """fp32 [n, rot]: cosines, then sines."""
    ang = np.arange(n)[:, None] * base ** (-np.arange(0, rot, 2) / max(rot, 1))[None]
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


# ---------------------------------------------------------------- CPU
@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_against_differences(interleaved):
    rng = np.random.default_rng(3)
    d, rot, eps, step = 32, 16, 1e-3, 1e-6
    x, g, w = rng.standard_normal((5, d)), rng.standard_normal((5, d)), 1 + 0.3 * rng.standard_normal(d)
    t = table(5, rot).astype(np.float64)
    cos, sin = t[:, :rot // 2], t[:, rot // 2:]
    dx, dw, _, _ = ref.backward(g, x, w, cos, sin, eps, interleaved)
    f = lambda x, w: (ref.forward(x, w, cos, sin, eps, interleaved) * g).sum()  # noqa: E731
    for i in range(5):
        for j in range(0, d, 5):
            e = np.zeros_like(x)
            e[i, j] = step
            # central differences: O(step^2) plus 2^-53 |f| / step, together below 1e-7
            assert abs((f(x + e, w) - f(x - e, w)) / (2 * step) - dx[i, j]) < 1e-7
    for j in range(d):
        e = np.zeros(d)
        e[j] = step
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * step) - dw[j]) < 1e-7


@pytest.fixture(scope="module")
def lib():
    from tiled_exact_attention_fa2_gb300 import _build
    _build.build()
    return fa2.load_library()


def fwd(lib, q=A, k=2 * A, wq=3 * A, wk=4 * A, w32=0, rope=5 * A, pos=6 * A, qo=7 * A, ko=8 * A, B=2, H=4, Hkv=2, N=16,
        d=64, rot=64, inter=0, maxpos=64, eps=1e-6, strides=None):
    s = None if strides is None else (ctypes.c_longlong * 12)(*strides)
    return lib.fa2_qk_norm_rope(q, k, wq, wk, w32, rope, pos, qo, ko, B, H, Hkv, N, d, rot, inter, maxpos, eps, s, None)


def test_forward_refusals(lib):
    assert fwd(lib, N=0) == 0
    for name in ("q", "k", "qo", "ko", "rope"):
        assert fwd(lib, **{name: None}) == 1, name
    for bad in (dict(B=0), dict(H=0), dict(N=-1), dict(Hkv=3), dict(Hkv=0), dict(rot=8), dict(rot=80), dict(rot=-16),
                dict(inter=2), dict(maxpos=0), dict(pos=None, N=65), dict(B=1 << 20, N=1 << 20)):
        assert fwd(lib, **bad) == 2, bad
    for d in (0, 8, 48, 256):
        assert fwd(lib, d=d) == 3
    for bad in (dict(q=A + 8), dict(ko=8 * A + 2), dict(rope=5 * A + 4), dict(pos=6 * A + 2), dict(wq=3 * A + 1),
                dict(w32=1, wk=4 * A + 2)):
        assert fwd(lib, **bad) == 4, bad
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert fwd(lib, eps=eps) == 5
    assert fwd(lib, qo=2 * A) == 9           # q_out over k
    assert fwd(lib, ko=7 * A + 64) == 9      # k_out over q_out
    assert fwd(lib, qo=5 * A) == 9           # q_out over the table
    assert fwd(lib, qo=A + 128) == 9         # half over q
    own = [4 * 16 * 64, 16 * 64, 64, 2 * 16 * 64, 16 * 64, 64]
    assert fwd(lib, strides=own + own, q=A + 4) == 4
    odd = own + own
    odd[2] = 65
    assert fwd(lib, strides=odd) == 4        # a stride that is not a multiple of 8
    neg = own + own
    neg[0] = -8
    assert fwd(lib, strides=neg) == 2
    far = own + own
    far[2] = 1 << 44
    assert fwd(lib, strides=far) == 2        # further than any memory reaches
    flat = own + own
    flat[7] = 0                              # q_out's heads on one another
    assert fwd(lib, strides=flat) == 9


def test_interleaved_output_views_pass_the_overlap_check(lib):
    """q_out and k_out as heads of one token-major buffer are apart, one head further on they are not.  (N = 0 launches
    nothing, so the check is reached through the refusal that follows it: a NULL last output of the backward call.)"""
    B, H, Hkv, N, d = 2, 4, 2, 16, 64
    row = (H + Hkv) * d
    view = lambda: [N * row, d, row]  # noqa: E731
    own = [H * N * d, N * d, d, Hkv * N * d, N * d, d]
    bad = (ctypes.c_longlong * 12)(*(own + view() + view()))
    # k_out starts inside q_out's heads: refused
    assert lib.fa2_qk_norm_rope(A, 2 * A, None, None, 0, None, None, 7 * A, 7 * A + (H - 1) * d * 2, B, H, Hkv, N, d, 0, 0, 0,
                                1e-6, bad, None) == 9


def bwd(lib, p=None, B=2, H=4, Hkv=2, N=16, d=64, ws=20 * A, wsb=1 << 24, eps=1e-6):
    p = p or [A * (i + 1) for i in range(12)]
    gq, gk, q, k, wq, wk, rope, pos, dq, dk, dwq, dwk = p
    return lib.fa2_qk_norm_rope_bwd(gq, gk, q, k, wq, wk, 0, rope, pos, dq, dk, dwq, dwk, B, H, Hkv, N, d, 64, 0, 64, eps, None,
                                    ws, wsb, None)


def test_overlap_check_accepts_views_that_are_apart(lib):
    """dq and dk as heads of one token-major buffer, reached through the refusal that follows the overlap check (8: no
    workspace): apart only where dk's heads begin behind dq's and end with the token's row."""
    B, H, Hkv, N, d = 2, 4, 2, 16, 64
    row = (H + Hkv) * d
    own = [[h * N * d, N * d, d] for h in (H, Hkv)]
    view = [N * row, d, row]
    for first, want in ((H * d, 8), ((H - 1) * d, 9), (H * d + 8, 9), (H * d - 8, 9), (0, 9), (row + H * d, 8)):
        s = (ctypes.c_longlong * 18)(*(own[0] + own[1] + own[0] + own[1] + view + view))
        p = [A * (i + 1) for i in range(12)]
        gq, gk, q, k, wq, wk, rope, pos, dq, dk, dwq, dwk = p
        assert lib.fa2_qk_norm_rope_bwd(gq, gk, q, k, wq, wk, 0, rope, pos, dq, dq + 2 * first, dwq, dwk, B, H, Hkv, N, d, 64, 0, 64,
                                        1e-6, s, None, 0, None) == want, first
    # the token's row of a padded buffer, [heads of q, 64 columns unused, heads of k]
    wide = [N * (row + 64), d, row + 64]
    s = (ctypes.c_longlong * 18)(*(own[0] + own[1] + own[0] + own[1] + wide + wide))
    assert lib.fa2_qk_norm_rope_bwd(gq, gk, q, k, wq, wk, 0, rope, pos, dq, dq + 2 * (H * d + 64), dwq, dwk, B, H, Hkv, N, d, 64, 0, 64,
                                    1e-6, s, None, 0, None) == 8


def test_backward_refusals(lib):
    p = [A * (i + 1) for i in range(12)]
    for i in (0, 1, 2, 3, 6, 8, 9):
        x = list(p)
        x[i] = None
        assert bwd(lib, x) == 1, i
    assert bwd(lib, B=0) == 2 and bwd(lib, d=20) == 3 and bwd(lib, eps=0.0) == 5
    assert bwd(lib, ws=None) == 8 and bwd(lib, ws=20 * A + 16) == 8 and bwd(lib, wsb=100) == 8
    need = lib.fa2_qk_norm_rope_bwd_workspace_bytes(64)
    assert need > 0 and lib.fa2_qk_norm_rope_bwd_workspace_bytes(48) == 0
    assert bwd(lib, wsb=need - 1) == 8
    for i, j in ((8, 3), (9, 8), (10, 2), (10, 11), (11, 6)):  # dq over k, dk over dq, dwq over q, dwq = dwk, dwk over rope
        x = list(p)
        x[i] = x[j]
        assert bwd(lib, x) == 9, (i, j)
    assert bwd(lib, ws=A) == 9
    x = list(p)
    x[10] = 11 * A + 2
    assert bwd(lib, x) == 4


def test_python_refusals():
    x = torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa2.fa2_qk_norm_rope(x, x)  # not on the GPU


# ---------------------------------------------------------------- GPU
def inputs(B, H, Hkv, N, d, layout, seed, scale=1.0):
    """q, k on the GPU in a layout, and their fp64 values as [B, heads, N, d]."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(B, N, H + 2 * Hkv, d, generator=g) * scale).to(torch.bfloat16).cuda()
    q, k = x[:, :, :H], x[:, :, H:H + Hkv]
    if layout == "bhnd":
        q, k = (t.transpose(1, 2).contiguous() for t in (q, k))
    elif layout == "fused":
        q, k = (t.transpose(1, 2) for t in (q, k))
    else:
        q, k = q[0], k[0]  # packed views, B = 1
    four = lambda t: t.double().cpu().numpy() if t.dim() == 4 else t.transpose(0, 1)[None].double().cpu().numpy()  # noqa: E731
    return q, k, four(q), four(k), four


CASES = [  # B, H, Hkv, N, d, rot, interleaved, weights, layout
    (1, 1, 1, 1, 16, 16, False, "bf16", "packed"),
    (2, 2, 1, 3, 16, 16, True, "fp32", "bhnd"),
    (1, 4, 4, 65, 32, 16, False, "fp32", "fused"),
    (3, 6, 2, 17, 32, 32, True, "bf16", "fused"),
    (2, 5, 5, 33, 64, 48, False, "bf16", "bhnd"),
    (2, 16, 4, 129, 64, 32, True, "fp32", "fused"),
    (1, 8, 2, 200, 128, 128, False, "bf16", "packed"),
    (2, 3, 1, 77, 128, 96, False, "none", "bhnd"),
    (1, 32, 8, 1, 128, 128, True, "bf16", "packed"),
    (5, 4, 2, 1, 128, 64, False, "fp32", "fused"),
    (1, 2, 2, 50, 64, 0, False, "fp32", "bhnd"),
    (1, 7, 1, 40000, 32, 32, False, "bf16", "packed"),  # four heads a group, a last group that is not full
    (2, 18, 6, 2000, 128, 128, False, "bf16", "fused"),
]


def setup(case, seed):
    B, H, Hkv, N, d, rot, inter, wt, layout = case
    q, k, q64, k64, four = inputs(B, H, Hkv, N, d, layout, seed)
    rng = np.random.default_rng(seed)
    if wt == "none":
        wq = wk = None
        w64 = [np.ones(d)] * 2
    else:
        t = torch.bfloat16 if wt == "bf16" else torch.float32
        wq, wk = (torch.from_numpy(1 + 0.3 * rng.standard_normal(d)).to(t).cuda() for _ in range(2))
        w64 = [w.double().cpu().numpy() for w in (wq, wk)]
    maxpos = 4 * N + 5
    rope = pos = None
    cos = sin = np.zeros((1, 1, 1, 0))
    if rot:
        tab = table(maxpos, rot)
        rope = torch.from_numpy(tab).cuda()
        if layout == "bhnd":
            p64 = np.broadcast_to(np.arange(N), (B, N))
        else:
            p64 = rng.integers(0, maxpos, (B, N))
            p64[-1, -1] = maxpos - 1
            pos = torch.from_numpy(p64.astype(np.int32)).cuda()
            pos = pos[0] if layout == "packed" else pos
        cos, sin = (tab[p64][:, None, :, s].astype(np.float64) for s in (slice(0, rot // 2), slice(rot // 2, rot)))
    return q, k, q64, k64, four, wq, wk, w64, rope, pos, cos, sin, inter


# The kernel's fp32 arithmetic: the row's sum, its root and three products are
# off by less than 2^-20 relative in all, the rotation adds two such terms; the
# store rounds to bf16 (2^-8 relative).
def close(got, want, size, what):
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * size
    err = np.abs(got - want)
    assert np.all(err <= tol), f"{what}: {np.max(err - tol):.3e} over the bound"


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case):
    q, k, q64, k64, four, wq, wk, w64, rope, pos, cos, sin, inter = setup(case, 11)
    qo, ko = fa2.fa2_qk_norm_rope(q, k, wq, wk, rope, pos, eps=1e-5, interleaved=inter)
    assert qo.is_contiguous() and qo.shape == q.shape and ko.shape == k.shape
    for got, x, w in ((qo, q64, w64[0]), (ko, k64, w64[1])):
        want = ref.forward(x, w, cos, sin, 1e-5, inter)
        close(four(got), want, np.abs(want).max(-1, keepdims=True), "out")
    assert fa2.fa2_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case):
    q, k, q64, k64, four, wq, wk, w64, rope, pos, cos, sin, inter = setup(case, 12)
    g = torch.Generator().manual_seed(1)
    gq, gk = (torch.randn(t.shape, generator=g).to(torch.bfloat16).cuda() for t in (q, k))
    dq, dk, dwq, dwk = fa2.fa2_qk_norm_rope_bwd(gq, gk, q, k, wq, wk, rope, pos, eps=1e-5, interleaved=inter)
    again = fa2.fa2_qk_norm_rope_bwd(gq, gk, q, k, wq, wk, rope, pos, eps=1e-5, interleaved=inter)
    for got, dw, gr, x, w in ((dq, dwq, four(gq), q64, w64[0]), (dk, dwk, four(gk), k64, w64[1])):
        dx64, dw64, size, mass = ref.backward(gr, x, w, cos, sin, 1e-5, inter)
        close(four(got), dx64, size, "dx")
        if wq is None:
            assert dw is None
        else:
            # at most 256 additions in a row (lanes, then CTAs, then slots), each 2^-24 of the sum of magnitudes, and
            # 2^-20 for the terms
            assert np.all(np.abs(dw.double().cpu().numpy() - dw64) <= (2.0 ** -16 + 2.0 ** -20) * mass + 1e-30)
    for a, b in zip((dq, dk, dwq, dwk), again):
        assert a is None or torch.equal(a, b)
    assert fa2.fa2_device_status() == 0


@pytest.mark.gpu
def test_in_place_and_into_views():
    """Outputs over their inputs, and as heads of one fused buffer whose other heads stay as they are."""
    case = (2, 4, 2, 40, 64, 64, False, "bf16", "fused")
    q, k, q64, k64, four, wq, wk, w64, rope, pos, cos, sin, inter = setup(case, 13)
    want = fa2.fa2_qk_norm_rope(q, k, wq, wk, rope, pos)
    buf = torch.full((2, 40, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    qo, ko = buf[:, :, :4].transpose(1, 2), buf[:, :, 4:6].transpose(1, 2)
    fa2.fa2_qk_norm_rope(q, k, wq, wk, rope, pos, q_out=qo, k_out=ko)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1]) and torch.all(buf[:, :, 6:] == 7)
    g = torch.randn(2, 40, 6, 64, device="cuda").to(torch.bfloat16)
    gq, gk = g[:, :, :4].transpose(1, 2), g[:, :, 4:].transpose(1, 2)
    wantb = fa2.fa2_qk_norm_rope_bwd(gq, gk, q, k, wq, wk, rope, pos)
    got = fa2.fa2_qk_norm_rope_bwd(gq, gk, q, k, wq, wk, rope, pos, dq=gq, dk=gk)
    for a, b in zip(got, wantb):
        assert torch.equal(a, b)
    fa2.fa2_qk_norm_rope(q, k, wq, wk, rope, pos, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


@pytest.mark.gpu
def test_no_tokens():
    q, k = (torch.empty(0, h, 64, dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    w = torch.ones(64, device="cuda")
    rope = torch.zeros(4, 64, device="cuda")
    qo, ko = fa2.fa2_qk_norm_rope(q, k, w, w, rope)
    assert qo.shape == q.shape
    _, _, dwq, dwk = fa2.fa2_qk_norm_rope_bwd(qo, ko, q, k, w, w, rope)
    assert not dwq.any() and not dwk.any()


@pytest.mark.gpu
def test_position_out_of_range_is_reported():
    case = (1, 2, 1, 6, 64, 64, False, "fp32", "packed")
    q, k, _, _, _, wq, wk, _, rope, pos, _, _, _ = setup(case, 14)
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    want, _ = fa2.fa2_qk_norm_rope(q, k, wq, wk, rope, pos)
    bad = pos.clone()
    bad[2], bad[4] = -1, rope.shape[0]
    qo, ko = torch.full_like(want, 9), torch.full((6, 1, 64), 9, dtype=torch.bfloat16, device="cuda")
    assert fa2.fa2_device_status(reset=True) == 0
    fa2.fa2_qk_norm_rope(q, k, wq, wk, rope, bad, q_out=qo, k_out=ko)
    assert fa2.fa2_device_status(reset=True) == 5 and fa2.fa2_device_status() == 0
    keep = [0, 1, 3, 5]
    assert torch.equal(qo[keep], want[keep]) and torch.all(qo[[2, 4]] == 9) and torch.all(ko[[2, 4]] == 9)


@pytest.mark.gpu
def test_nonfinite_values_stay_in_their_row():
    case = (1, 2, 1, 8, 64, 32, False, "fp32", "packed")
    q, k, _, _, _, wq, wk, _, rope, pos, _, _, _ = setup(case, 15)
    want, _ = fa2.fa2_qk_norm_rope(q, k, wq, wk, rope, pos)
    q2 = q.clone()
    q2[3, 1, 5], q2[5, 0, 60] = float("nan"), float("inf")
    got, _ = fa2.fa2_qk_norm_rope(q2, k, wq, wk, rope, pos)
    assert torch.isnan(got[3, 1]).all()
    rows = torch.ones(8, 2, dtype=torch.bool)
    rows[3, 1] = rows[5, 0] = False
    assert torch.equal(got[rows], want[rows])


@pytest.mark.gpu
def test_other_stream_and_graph():
    case = (1, 8, 2, 64, 128, 128, False, "bf16", "packed")
    q, k, _, _, _, wq, wk, _, rope, pos, _, _, _ = setup(case, 16)
    want = fa2.fa2_qk_norm_rope(q, k, wq, wk, rope, pos)
    gq, gk = torch.randn_like(want[0]), torch.randn_like(want[1])
    wantb = fa2.fa2_qk_norm_rope_bwd(gq, gk, q, k, wq, wk, rope, pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fa2.fa2_qk_norm_rope(q, k, wq, wk, rope, pos, stream=side)
    gotb = fa2.fa2_qk_norm_rope_bwd(gq, gk, q, k, wq, wk, rope, pos, stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got + gotb, want + wantb):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa2.fa2_qk_norm_rope(q, k, wq, wk, rope, pos)
        gotb = fa2.fa2_qk_norm_rope_bwd(gq, gk, q, k, wq, wk, rope, pos)
    for _ in range(2):
        for t in got + gotb:
            t.zero_()
        graph.replay()
        for a, b in zip(got + gotb, want + wantb):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_strides_past_32_bits():
    """Rows more than 2^31 elements apart give what their contiguous copies give."""
    B, H, N, d, far = 2, 2, 5, 64, (1 << 31) + 512
    buf = torch.empty(2 * far, dtype=torch.bfloat16, device="cuda")
    q, k, out_q, out_k = (buf.as_strided((B, H, N, d), (far, d, 4 * H * d, 1), i * H * d) for i in range(4))
    q.copy_(torch.randn(B, H, N, d, device="cuda"))
    k.copy_(torch.randn(B, H, N, d, device="cuda"))
    w, rope = torch.rand(d, device="cuda") + 0.5, torch.randn(N, d, device="cuda")
    want = fa2.fa2_qk_norm_rope(q.contiguous(), k.contiguous(), w, w, rope)
    fa2.fa2_qk_norm_rope(q, k, w, w, rope, q_out=out_q, k_out=out_k)
    assert torch.equal(out_q, want[0]) and torch.equal(out_k, want[1])
    grads = fa2.fa2_qk_norm_rope_bwd(out_q.contiguous(), out_k.contiguous(), q.contiguous(), k.contiguous(), w, w, rope)
    got = fa2.fa2_qk_norm_rope_bwd(out_q, out_k, q, k, w, w, rope, dq=out_q, dk=out_k)
    assert all(torch.equal(a, b) for a, b in zip(got, grads))


@pytest.mark.gpu
@pytest.mark.parametrize("case", [(1, 8, 8, 7301, 128, 128, False, "bf16", "packed"),   # eight heads a group
                                  (2, 39, 39, 3001, 32, 16, False, "fp32", "fused"),    # and a last group of seven
                                  (2, 16, 8, 5000, 64, 64, False, "none", "bhnd")], ids=str)
def test_forward_many_tokens(case):
    q, k, q64, k64, four, wq, wk, w64, rope, pos, cos, sin, inter = setup(case, 13)
    qo, ko = fa2.fa2_qk_norm_rope(q, k, wq, wk, rope, pos, eps=1e-5)
    for got, x, w in ((qo, q64, w64[0]), (ko, k64, w64[1])):
        want = ref.forward(x, w, cos, sin, 1e-5, inter)
        close(four(got), want, np.abs(want).max(-1, keepdims=True), "out")
    a, b = q.clone() if q.is_contiguous() else q, k.clone() if k.is_contiguous() else k
    fa2.fa2_qk_norm_rope(a, b, wq, wk, rope, pos, eps=1e-5, q_out=a, k_out=b)  # in place
    assert torch.equal(a, qo) and torch.equal(b, ko) and fa2.fa2_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("case", [(1, 4, 1, 3001, 32, 32, False, "bf16", "packed"), (2, 2, 2, 1500, 128, 96, True, "fp32", "fused"),
                                  (3, 2, 1, 700, 64, 32, False, "fp32", "bhnd"), (1, 5, 1, 9001, 16, 16, True, "bf16", "packed"),
                                  (1, 1, 1, 9000, 128, 128, False, "bf16", "packed")], ids=str)
def test_few_heads(case):
    """Groups of two heads, and groups with rows missing, over many tokens."""
    test_forward(case)
    test_backward(case)
