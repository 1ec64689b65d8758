"""Ids that a token is given several times, through the few-token layer's two ways of building its rows."""
import pytest
import torch

from test_gpu_layer import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("k", [3, 4, 8])
def test_repeated_ids_have_the_same_bits_in_every_batch(k, q8):
    """The gates of an id given three times or more add up in the order of the choices, in a call of a few choices (one
    token at a time) as in one of many (all tokens at once)."""
    c = Case(64, 256, 16, k, 16, 64, q8)
    ids, gates = c.random_choices(13)
    for j in range(2, k):
        ids[:, j] = ids[:, 0]
    ids[::2, 1] = ids[::2, 0]
    # the last gate takes the others' sum back but for 2^-10 of it: another order of the fp32 sum would move what is left by
    # about 2^-14 of itself, which one in 2^6 of a row's 256 bf16 outputs shows
    gates[:, k - 1] = -gates[:, :k - 1].sum(1) * (1 - 2.0 ** -10)
    whole = c.call(ids, gates)["out"]
    c.check(whole, ids, gates)
    for t in range(64):
        one = c.call(ids, gates, rows=torch.tensor([t], device="cuda"))["out"]
        assert torch.equal(one[0].view(torch.int16), whole[t].view(torch.int16)), t


@pytest.mark.parametrize("q8", [False, True])
def test_the_order_of_repeated_gates(q8):
    """2^24, 1 and 1 in this order add up to 2^24 in fp32 (1 + 1 first would give 2^24 + 2); with -2^24 as the fourth the
    sum is 0 (else 2)."""
    c = Case(40, 256, 8, 4, 8, 32, q8)
    ids = torch.full((40, 4), 5, dtype=torch.int32)
    gates = torch.tensor([2.0 ** 24, 1.0, 1.0, -2.0 ** 24]).repeat(40, 1)
    assert (c.call(ids, gates)["out"] == 0).all()
    one = c.call(ids, gates, rows=torch.tensor([3], device="cuda"))["out"]
    assert (one == 0).all()
