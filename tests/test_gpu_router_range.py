"""mk_route_topk of more tokens than one launch's grid holds (2^32 work items): the last tokens' ids, gates and logits bit for
bit as in a call of their own."""
import gc

import pytest
import torch

import moe_dispatch_expert_amd as mk

pytestmark = pytest.mark.gpu


# a token takes 64 work items of the selection, and 16 per 8 experts of the router
@pytest.mark.parametrize("T,E", [((1 << 26) + 3, 2), ((1 << 25) + 70, 64)])
def test_routing_of_more_tokens_than_a_grid(T, E):
    d, k = 128, 2
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    wr = torch.randn(d, E, generator=g, device="cuda") / d ** 0.5
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -7.0, device="cuda")
    ws = torch.empty(mk.mk_route_topk_workspace_bytes(T, E), dtype=torch.uint8, device="cuda")
    ws[-(1 << 30):].zero_()
    mk.mk_route_topk(x, wr, k, topk_ids=ids, topk_w=w, workspace=ws)
    for at in (0, T // 2, T - 1000):
        part = slice(at, at + 1000)
        want_ids, want_w = mk.mk_route_topk(x[part].clone(), wr, k)
        assert torch.equal(ids[part], want_ids), at
        assert torch.equal(w[part].view(torch.int32), want_w.view(torch.int32)), at
    assert int(ids.min()) >= 0 and int(ids.max()) < E
    del x, ids, w, ws
    gc.collect()
    torch.cuda.empty_cache()
