"""Calls of the few-token layer that run at the same time on streams of their own, each with its own workspace: the forms
that add the rows up inside the down kernel (few choices) beside those that do not, in both weight types."""
import pytest
import torch

import moe_dispatch_expert_amd as mk
from test_gpu_layer import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q8", [False, True])
def test_few_and_many_choices_at_once(q8):
    shapes = [(1, 2), (4, 8), (8, 4), (8, 8), (96, 4)]
    cases = [Case(T, 1024, 32, k, 32, 208, q8, seed=T) for T, k in shapes]
    want = [c.call()["out"] for c in cases]
    streams = [torch.cuda.Stream() for _ in shapes]
    wss = [torch.full((mk.mk_moe_layer_workspace_bytes(T, 1024, 32, k, 0, 32, 208),), 0xC3, dtype=torch.uint8,
                      device="cuda") for T, k in shapes]
    outs = [[torch.zeros_like(w) for _ in range(20)] for w in want]
    torch.cuda.synchronize()
    for i in range(20):
        for c, s, ws, o in zip(cases, streams, wss, outs):
            c.call(out={"out": o[i]}, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for w, o, shape in zip(want, outs, shapes):
        for i in range(20):
            assert torch.equal(o[i].view(torch.int16), w.view(torch.int16)), (shape, i)
