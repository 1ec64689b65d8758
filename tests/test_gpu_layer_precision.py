"""What the few-token layer keeps of its intermediate: whatever the size of gates and activations, and in every row form,
task shape and tail of its kernels, only the output's rounding to bf16 shows."""
import math

import pytest
import torch

import layer_bound
import layer_ref
from test_gpu_layer import Case

pytestmark = pytest.mark.gpu


def _check(c, out, ids, gates, rows, what=""):
    want, bound = layer_bound.layer(c.x64, c.gu64, c.dn64, ids.long().cpu(), gates.cpu(), c.q8, c.e_begin)
    got = out.cpu().double()
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, first {torch.nonzero(bad)[0]}"
    # Rounding to bf16 is off by at most 2^-8 of a value, 2^-8 / sqrt(3) in the mean square at worst, and here by
    # `rounding`.  What is kept of h adds 2^-11 |h| at most, an eighth of that at the worst place of a binade and 1.6 percent
    # in the sum of squares; another few percent are the chance of `rows` outputs' sums of squares.
    got, want = got[rows], want[rows]
    rounding = (want.to(torch.bfloat16).double() - want).norm()
    assert want.norm() > 0 and rounding <= 2.0 ** -8 / math.sqrt(3) * want.norm()
    assert (got - want).norm() <= 1.1 * rounding, (what, float((got - want).norm() / rounding))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("gate,act", [(0, 0), (-10, 0), (-20, 0), (-40, 0), (10, 0), (0, -10), (0, -20), (0, 8), (-10, -10),
                                      (20, 8)])
def test_error_is_one_rounding_at_any_scale(gate, act, q8):
    """Gates scaled by 2^gate, activations by 2^act (the intermediate by 2^gate, and by 2^act to 4^act)."""
    c = Case(64, 1024, 16, 4, 16, 512, q8)
    if q8:
        c.gpu["xs"].mul_(2.0 ** act)
        c.x64 = c.x64 * 2.0 ** act
    else:
        c.gpu["x"].mul_(2.0 ** act)
        c.x64 = c.x64 * 2.0 ** act
    ids, gates = c.random_choices(21)
    gates = gates * 2.0 ** gate
    _check(c, c.call(ids, gates)["out"], ids, gates, slice(None))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("spread", [0, 24])
@pytest.mark.parametrize("rows", [1, 7, 8, 12, 16, 17, 32, 33, 48, 49, 64, 100])
@pytest.mark.parametrize("d,F", [(1024, 176), (1024, 512), (32768, 80), (128, 16384)])   # tails; few and many tasks
def test_error_is_one_rounding_in_every_row_form(d, F, rows, spread, q8):
    """One expert's rows; the activations of neighbouring features up to 2^spread apart (the up rows' sizes)."""
    c = Case(rows, d, 2, 1, 2, F, q8)
    if spread:
        # feature f's up row times 2^-(f % 5) spread / 4: exact in bf16, and in 8 bits by new codes of the same values
        scale = 2.0 ** -((torch.arange(F) % 5) * (spread // 4)).double()
        c.gu64[:, F:] *= scale[None, :, None]
        if q8:
            q, s = layer_ref.blocks_q8(c.gu64[:, F:].float())
            c.gu64[:, F:] = layer_ref.blocks_values(q, s)
            nf = -(-F // 128)
            c.gpu["gq"].view(torch.uint8)[:, F:] = q.view(torch.uint8).cuda()
            c.gpu["gs"][:, nf:] = s.cuda()
        else:
            c.gpu["gu"][:, F:] = c.gu64[:, F:].to(torch.bfloat16).cuda()
    ids = torch.full((rows, 1), 1, dtype=torch.int32)
    gates = torch.rand(rows, 1, generator=torch.Generator().manual_seed(6)) * 0.01 + 0.001
    _check(c, c.call(ids, gates)["out"], ids, gates, slice(None))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("T,d,E,k,F", [(1, 2048, 64, 6, 176), (2, 512, 16, 8, 512), (8, 1024, 32, 4, 144), (13, 512, 8, 2, 80)])
def test_error_is_one_rounding_routed_inside(T, d, E, k, F, q8):
    """The forms for few tokens, with the softmax's gates of many experts."""
    c = Case(T, d, E, k, E, F, q8)
    o = c.call(out=c.choices())
    _check(c, o["out"], o["topk_ids"], o["topk_w"], slice(None))


def test_infinite_and_largest_intermediates_stay_in_their_token():
    """8-bit weights: a token whose intermediate overflows shares its groups of features with nobody."""
    c = Case(24, 512, 4, 1, 4, 256, True)
    ids, gates = c.random_choices(3)
    clean = c.call(ids, gates)["out"]
    big = gates.clone()
    big[5] = float("inf")
    big[9] = 3.0e38
    out = c.call(ids, big)["out"]
    keep = [t for t in range(24) if t not in (5, 9)]
    assert torch.equal(out[keep].view(torch.int16), clean[keep].view(torch.int16))
    assert not torch.isfinite(out[5].float()).any()
