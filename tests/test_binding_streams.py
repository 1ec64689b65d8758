"""Where the binding allocates what a call on another stream needs and was not given: on that stream, since memory of the
current one may still be in use by work queued there, and may be handed out there again while the call runs."""
import contextlib

import pytest
import torch

import moe_dispatch_expert_amd as mk

BF16 = torch.bfloat16
X = torch.zeros(4, 256, dtype=BF16)
W = torch.zeros(8, 64, 256, dtype=BF16)
DOWN = torch.zeros(8, 256, 32, dtype=BF16)
WR = torch.zeros(256, 8)
IDS, GATES = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
OFFSETS = torch.zeros(9, dtype=torch.int32)

CALLS = {
    "mk_route_topk": lambda s: mk.mk_route_topk(X, WR, 2, stream=s),
    "mk_dispatch_gemm": lambda s: mk.mk_dispatch_gemm(X, W, 2, w_router=WR, stream=s),
    "mk_combine": lambda s: mk.mk_combine(X, IDS, GATES, stream=s),
    "mk_swiglu": lambda s: mk.mk_swiglu(X, stream=s),
    "mk_grouped_gemm": lambda s: mk.mk_grouped_gemm(X, OFFSETS, W, stream=s),
    "mk_grouped_gemm_swiglu": lambda s: mk.mk_grouped_gemm_swiglu(X, OFFSETS, W, stream=s),
    "mk_add_rmsnorm": lambda s: mk.mk_add_rmsnorm(X, torch.ones(256, dtype=BF16), X, q8=True, stream=s),
    "mk_moe_layer": lambda s: mk.mk_moe_layer(X, W, DOWN, 2, w_router=WR, stream=s),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_allocations_are_made_on_the_calls_stream(name, monkeypatch):
    """On the CPU: the calls refuse these tensors, after they have allocated what they were not given."""
    inside, made = [], []
    other = object()

    @contextlib.contextmanager
    def stream_context(s):
        assert s is other
        inside.append(s)
        yield
        inside.pop()

    def watch(fn):
        def call(*args, **kw):
            made.append(bool(inside))
            return fn(*args, **kw)
        return call

    monkeypatch.setattr(torch.cuda, "stream", stream_context)
    for n in ("empty", "empty_like", "zeros"):
        monkeypatch.setattr(torch, n, watch(getattr(torch, n)))
    with pytest.raises(ValueError):
        CALLS[name](other)
    assert made and all(made), made
    made.clear()
    with pytest.raises(ValueError):
        CALLS[name](None)
    assert made and not any(made), made


def _pool_of(t):
    """The stream whose memory a tensor's storage is."""
    at = t.untyped_storage().data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in any segment")


@pytest.mark.gpu
def test_outputs_and_workspaces_are_the_streams_memory():
    side = torch.cuda.Stream()
    g = torch.Generator().manual_seed(1)
    x = torch.randn(40, 256, generator=g).to(BF16).cuda()
    w = (torch.randn(8, 256, 256, generator=g) / 16).to(BF16).cuda()
    dn = (torch.randn(8, 256, 128, generator=g) / 11).to(BF16).cuda()
    offsets = torch.tensor([0] + [40] * 8, dtype=torch.int32, device="cuda")
    wr, gamma = (torch.randn(256, 8, generator=g) / 16).cuda(), torch.ones(256, dtype=BF16, device="cuda")

    def chain(s):
        n = mk.mk_add_rmsnorm(x, gamma, x, q8=True, stream=s)
        layer = mk.mk_moe_layer(n["y"], w, dn, 2, w_router=wr, stream=s)
        ids, gates = mk.mk_route_topk(n["y"], wr, 2, stream=s)
        p = mk.mk_dispatch_gemm(n["y"], w, 2, w_router=wr, swiglu=True, stream=s)
        z = mk.mk_grouped_gemm(p["y_perm"], p["expert_offsets"], dn, stream=s)
        y = mk.mk_combine(z, p["slot_of"], p["topk_w"], stream=s)
        h = mk.mk_grouped_gemm_swiglu(x, offsets, w, stream=s)
        a = mk.mk_swiglu(x, stream=s)
        own = [*n.values(), layer["out"], layer["workspace"], ids, gates, z, y, h, a]
        return own + [p[k] for k in ("slot_of", "expert_offsets", "topk_w", "workspace")], \
            [n["y"], layer["out"], ids, gates, y, h, a]

    want = chain(None)[1]
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    own, got = chain(side)
    for t in own:
        assert _pool_of(t) == side.cuda_stream, t.shape
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_many_calls_on_another_stream_without_a_workspace():
    """Each call's workspace and outputs are dropped while it runs, and the current stream allocates and writes meanwhile."""
    side = torch.cuda.Stream()
    g = torch.Generator().manual_seed(2)
    x = torch.randn(64, 512, generator=g).to(BF16).cuda()
    w = (torch.randn(16, 256, 512, generator=g) / 22).to(BF16).cuda()
    dn = (torch.randn(16, 512, 128, generator=g) / 11).to(BF16).cuda()
    wr = (torch.randn(512, 16, generator=g) / 22).cuda()
    want = mk.mk_moe_layer(x, w, dn, 4, w_router=wr)["out"]
    size = mk.mk_moe_layer_workspace_bytes(64, 512, 16, 4, 0, 16, 128)
    torch.cuda.synchronize()
    outs = []
    for _ in range(50):
        outs.append(mk.mk_moe_layer(x, w, dn, 4, w_router=wr, stream=side)["out"])
        torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


@pytest.mark.gpu
def test_captured_on_a_forked_stream():
    """A capture whose calls run on a second stream and allocate for themselves, replayed between eager calls."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(40, 256, generator=g).to(BF16).cuda()
    w = (torch.randn(8, 256, 256, generator=g) / 16).to(BF16).cuda()
    dn = (torch.randn(8, 256, 128, generator=g) / 11).to(BF16).cuda()
    wr, gamma = (torch.randn(256, 8, generator=g) / 16).cuda(), torch.ones(256, dtype=BF16, device="cuda")
    side = torch.cuda.Stream()

    def step(s):
        n = mk.mk_add_rmsnorm(x, gamma, stream=s)["y"]
        return mk.mk_moe_layer(n, w, dn, 2, w_router=wr, stream=s)["out"]

    step(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        out = step(side)
        torch.cuda.current_stream().wait_stream(side)
    for i in range(4):
        x.mul_(1.25)
        out.zero_()
        graph.replay()
        want = step(None)
        assert torch.equal(out, want), i
        torch.cuda.synchronize()
