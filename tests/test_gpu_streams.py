"""Calls on a stream that is not torch's current one (GPU only): what they allocate is that stream's."""
import pytest
import torch

import tiled_exact_attention_fa2_gb300 as fa2

pytestmark = pytest.mark.gpu


def calls():
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v, dO = r(1, 4, 200, 128), r(1, 4, 200, 128), r(1, 4, 200, 128), r(1, 4, 200, 128)
    kg, vg = k[:, :2].contiguous(), v[:, :2].contiguous()
    o, lse = fa2.fa2_fwd(q, k, v)
    og, lseg = fa2.fa2_fwd_gqa(q, kg, vg)
    packed = [x[0].transpose(0, 1).contiguous() for x in (q, k, v, dO)]
    cu = torch.tensor([0, 70, 200], dtype=torch.int32, device="cuda")
    op, lsep = fa2.fa2_fwd_varlen(*packed[:3], cu, cu, 130, 130)
    ws = torch.empty(fa2.fa2_fwd_workspace_bytes(1, 4, 200, 128), dtype=torch.uint8, device="cuda")
    wsb = torch.empty(fa2.fa2_bwd_workspace_bytes(1, 4, 200, 128), dtype=torch.uint8, device="cuda")
    one = q[:, :, :1].contiguous()
    long = r(1, 2, 4000, 128)
    return {
        "fwd": lambda s: fa2.fa2_fwd(q, k, v, stream=s),
        "fwd positional": lambda s: fa2.fa2_fwd(q, k, v, None, None, None, True, s),
        "fwd_ws": lambda s: fa2.fa2_fwd_ws(q, k, v, ws, stream=s),
        "fwd_gqa": lambda s: fa2.fa2_fwd_gqa(q, kg, vg, stream=s),
        "fwd_splitkv": lambda s: fa2.fa2_fwd_splitkv(one, long, long, stream=s),
        "fwd_varlen": lambda s: fa2.fa2_fwd_varlen(*packed[:3], cu, cu, 130, 130, stream=s),
        "bwd": lambda s: fa2.fa2_bwd(q, k, v, o, dO, lse, stream=s)[1:],  # (dQ's sums vary in order)
        "bwd_ws": lambda s: fa2.fa2_bwd_ws(q, k, v, o, dO, lse, wsb, stream=s)[1:],
        "bwd_gqa": lambda s: fa2.fa2_bwd_gqa(q, kg, vg, og, dO, lseg, stream=s)[1:],
        "bwd_varlen": lambda s: fa2.fa2_bwd_varlen(*packed[:3], op, packed[3], lsep, cu, cu, 130, 130, stream=s)[1:],
        "bwd_noalloc": lambda s: fa2.fa2_bwd_noalloc(q, k, v, o, dO, lse, stream=s)[1:],
        "bwd_deterministic": lambda s: fa2.fa2_bwd_deterministic(q, k, v, o, dO, lse, stream=s),
    }


def test_what_a_call_allocates_belongs_to_its_stream(monkeypatch):
    """Memory of the current stream would be handed to other work there while the given stream still uses it: scratch as
    soon as the call returns, outputs if the block was free with work of the current stream still to come."""
    made = []
    for name in ("empty", "empty_like"):
        real = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, real=real, **kw: made.append(torch.cuda.current_stream().cuda_stream) or real(*a, **kw))
    side = torch.cuda.Stream()
    for name, call in calls().items():
        want = call(None)
        for given in (side, side.cuda_stream):
            torch.cuda.synchronize()
            before = torch.cuda.current_stream()
            made.clear()
            got = call(given)
            assert made and set(made) == {side.cuda_stream}, name
            assert torch.cuda.current_stream() == before
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), name
    host = {x: torch.randn(1, 2, 128, 64).to(torch.bfloat16) for x in ("q", "k", "v", "dO", "o", "dq", "dk", "dv")}
    host["lse"] = torch.empty(1, 2, 128)
    made.clear()
    fa2.fa2_step_from_host(host, stream=side)
    torch.cuda.synchronize()
    assert set(made) == {side.cuda_stream}
    assert fa2.fa2_device_status(reset=True) == 0


def test_a_stream_of_another_device_is_refused():
    with pytest.raises(ValueError):
        fa2._stream(torch.cuda.Stream(), torch.device("cuda", torch.cuda.current_device() + 1))


def test_default_stream_by_its_handles():
    """0 and cudaStreamLegacy (1) are torch's default stream; neither is one of torch's own numbers."""
    dev, default = torch.cuda.current_device(), torch.cuda.default_stream()
    q = torch.randn(1, 2, 64, 64, device="cuda").to(torch.bfloat16)
    want = fa2.fa2_qk_norm_rope(q, q.clone())
    with torch.cuda.stream(torch.cuda.Stream()):
        for handle in (0, 1, default):
            with fa2._on(dev, handle):
                assert torch.cuda.current_stream() == default
            torch.cuda.synchronize()
            got = fa2.fa2_qk_norm_rope(q, q.clone(), stream=handle)
            torch.cuda.synchronize()
            assert torch.equal(got[0], want[0])
    per_thread = fa2._on(dev, 2)
    with per_thread:
        assert torch.cuda.current_stream().cuda_stream == 2
