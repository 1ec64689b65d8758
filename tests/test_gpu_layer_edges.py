"""The few-token MoE layer at the ends of its range: the largest expert and choice counts, every row count and tile
width, both sides of its selection's switches, and weights past 32-bit offsets.  References and tolerances as in
test_gpu_layer.py."""
import math

import pytest
import torch

import moe_dispatch_expert_amd as mk
from test_gpu_layer import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q8", [False, True])
def test_most_tokens_experts_and_choices(q8):
    c = Case(128, 128, 1024, 32, 1024, 16, q8=q8)
    out = c.choices()
    r = c.call(out=out)
    ids, w = mk.mk_route_topk(c.gpu["x"], c.gpu["wr"], c.k, None)
    assert torch.equal(out["topk_ids"], ids) and torch.equal(out["topk_w"], w)
    c.check(r["out"], ids, w)


# (T, k, E): up to 8 and more tokens, up to 32 and more choices, up to 64, 256 and more experts
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("T,k,E", [(8, 4, 64), (8, 5, 64), (9, 3, 64), (11, 3, 16), (16, 2, 8), (17, 2, 8), (1, 32, 256),
                                   (2, 17, 65), (8, 4, 257), (9, 4, 257), (1, 1, 1), (128, 1, 1)])
def test_selection_switches(T, k, E, q8):
    c = Case(T, 256, E, k, E, 32, q8=q8, bias=True)
    out = c.choices()
    r = c.call(out=out)
    ids, w = mk.mk_route_topk(c.gpu["x"], c.gpu["wr"], c.k, c.gpu["bias"])
    assert torch.equal(out["topk_ids"], ids) and torch.equal(out["topk_w"], w)
    c.check(r["out"], ids, w)


# shapes whose tasks take one or two, and four weight tiles: few columns, many features, many columns
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("d,F", [(256, 48), (128, 16384), (32768, 80)])
@pytest.mark.parametrize("rows", [(1, 128), (8, 9), (16, 17), (32, 33), (41, 48), (49, 56), (64, 65), (31, 127)])
def test_rows_of_an_expert(d, F, rows, q8):
    """Two experts with the given numbers of rows, on the last tokens and on the first."""
    c = Case(128, d, 4, 2, 4, F, q8=q8)
    ids = torch.full((128, 2), -1, dtype=torch.int32)
    ids[128 - rows[0]:, 0] = 1
    ids[:rows[1], 1] = 3
    gates = torch.rand(128, 2, generator=torch.Generator().manual_seed(3)) + 0.1
    c.check(c.call(ids, gates)["out"], ids, gates)


@pytest.mark.parametrize("q8", [False, True])
def test_experts_past_32_bit_offsets(q8):
    """The last of many large experts gives the bits of the same weights in a call of one expert."""
    d, F, E = 8192, 4096, 72 if q8 else 40
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(3, d, generator=g, device="cuda", dtype=torch.bfloat16)
    gu = (torch.randn(1, 2 * F, d, generator=g, device="cuda") / math.sqrt(d))
    dn = (torch.randn(1, d, F, generator=g, device="cuda") / math.sqrt(F))
    one = torch.zeros(3, 1, dtype=torch.int32, device="cuda")
    gates = torch.full((3, 1), 0.5, device="cuda")
    kind = torch.float8_e4m3fn if q8 else torch.bfloat16
    gu, dn = (gu * (64 if q8 else 1)).to(kind), (dn * (64 if q8 else 1)).to(kind)

    def last(v):   # the other experts are not read; zeros keep them defined
        many = torch.zeros((E,) + v.shape[1:], dtype=torch.uint8 if q8 else v.dtype, device="cuda")
        many = many.view(v.dtype) if q8 else many
        many[E - 1].copy_(v[0])
        return many

    assert gu.numel() * E * gu.element_size() > 2 ** 32
    if q8:
        xq, xs = x.float().to(kind), torch.ones(3, d // 128, device="cuda")
        gs, ds = (torch.full((E, n, m), 1 / 64, device="cuda") for n, m in ((2 * F // 128, d // 128), (d // 128, F // 128)))
        want = mk.mk_moe_layer_q8(xq, xs, gu, gs[:1], dn, ds[:1], 1, topk_ids_in=one, topk_w_in=gates)["out"]
        got = mk.mk_moe_layer_q8(xq, xs, last(gu), gs, last(dn), ds, 1, topk_ids_in=one + E - 1, topk_w_in=gates)["out"]
    else:
        want = mk.mk_moe_layer(x, gu, dn, 1, topk_ids_in=one, topk_w_in=gates)["out"]
        got = mk.mk_moe_layer(x, last(gu), last(dn), 1, topk_ids_in=one + E - 1, topk_w_in=gates)["out"]
    assert torch.equal(got, want) and want.abs().max() > 0.01


@pytest.mark.parametrize("q8", [False, True])
def test_choices_written_over_those_given(q8):
    """The given ids and gates may be the outputs' tensors: they keep their values."""
    c = Case(40, 256, 16, 4, 16, 64, q8=q8)
    ids, gates = c.random_choices(9)
    want = c.call(ids, gates)["out"]
    di, dg = ids.cuda(), gates.cuda()
    kw = dict(topk_ids_in=di, topk_w_in=dg, E=c.E, out={"topk_ids": di, "topk_w": dg})
    G = c.gpu
    if q8:
        got = mk.mk_moe_layer_q8(G["xq"], G["xs"], G["gq"], G["gs"], G["dq"], G["ds"], c.k, **kw)["out"]
    else:
        got = mk.mk_moe_layer(G["x"], G["gu"], G["dn"], c.k, **kw)["out"]
    assert torch.equal(got, want) and torch.equal(di.cpu(), ids) and torch.equal(dg.cpu(), gates)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("T,k", [(1, 2), (2, 8), (8, 4)])
def test_few_choices_replayed(T, k, q8):
    """A captured call of a few choices, replayed with other choices, none at all, and fewer valid tokens, between eager
    calls of its own workspace: every result is the eager one's, bit for bit."""
    c = Case(T, 512, 16, k, 16, 80, q8=q8)
    ids, gates = c.random_choices(1)
    G = c.gpu
    di, dg = ids.cuda(), gates.cuda()
    valid = torch.tensor([T], dtype=torch.int32, device="cuda")
    ws = torch.full((mk.mk_moe_layer_workspace_bytes(T, 512, 16, k, 0, 16, 80),), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.empty(T, 512, dtype=torch.bfloat16, device="cuda")

    def call(dst, w):
        kw = dict(topk_ids_in=di, topk_w_in=dg, E=16, t_valid=valid, workspace=w, out={"out": dst})
        if q8:
            mk.mk_moe_layer_q8(G["xq"], G["xs"], G["gq"], G["gs"], G["dq"], G["ds"], k, **kw)
        else:
            mk.mk_moe_layer(G["x"], G["gu"], G["dn"], k, **kw)

    call(out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, ws)
    for step in range(8):
        new, _ = c.random_choices(10 + step)
        if step % 4 == 2:
            new.fill_(-1)
        n = max(T - step % 3, 0)
        di.copy_(new)
        valid.fill_(n)
        out.fill_(7.0)
        eager = torch.full_like(out, 7.0)
        graph.replay()
        call(eager, None if step % 2 else ws)
        graph.replay()
        assert torch.equal(out, eager), step
        assert (out[n:] == 7.0).all()
        if step % 4 == 2:
            assert (out[:n] == 0).all()
        elif n:
            c.check(out, torch.where(torch.arange(T)[:, None] < n, new, -1), gates, rows=slice(0, n))
