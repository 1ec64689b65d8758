"""The few-token layer where the experts of one call have very different numbers of rows, so that a workgroup goes from one
row form of its kernels to another: against the fp64 layer, and bit for bit against the same tokens a few at a time."""
import pytest
import torch

from test_gpu_layer import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("F", [16, 272])      # one step of K for the four waves, and several
@pytest.mark.parametrize("rows", [(65, 20), (40, 5), (5, 40), (8, 40), (96, 33), (70, 1), (16, 64)])
def test_forms_of_different_rows_in_one_workgroup(rows, F, q8):
    """d = 32768: two experts' down products are two whole rounds of four-tile tasks, one of each expert a workgroup."""
    c = Case(128, 32768, 2, 2, 2, F, q8=q8)
    ids = torch.full((128, 2), -1, dtype=torch.int32)
    ids[128 - rows[0]:, 0] = 0
    ids[:rows[1], 1] = 1
    gates = torch.rand(128, 2, generator=torch.Generator().manual_seed(4)) + 0.1
    first = c.call(ids, gates)["out"]
    c.check(first, ids, gates)
    for at in range(0, 128, 16):
        part = torch.arange(at, at + 16)
        alone = c.call(ids, gates, rows=part.cuda())["out"]
        assert torch.equal(alone.view(torch.int16), first[at:at + 16].view(torch.int16)), at
    for _ in range(3):
        again = c.call(ids, gates)["out"]
        assert torch.equal(again.view(torch.int16), first.view(torch.int16))
