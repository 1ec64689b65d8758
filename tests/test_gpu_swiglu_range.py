"""mk_swiglu_i8 over the whole range of gates: where e^-g leaves fp32's range, where h = silu(g) u does, and rows that are zeros or
not finite.

h is computed to 2^-20, relative, on a value and on its row's maximum (see test_gpu_grouped_i8.py), as long as the maximum m is
at least 2^-119, so that m / 127 has all its bits: codes lie within 1/2 + 127 * 2^-19 of 127 h / m, 127 scale within 2^-19 m of m.
A value below 2^-126 is off by up to 2^-149, which is 2^-30 of such an m at most and so within the same bound."""
import pytest
import torch

import moe_dispatch_expert_amd as mk

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _exact(gu):
    a, u = gu.double().chunk(2, dim=1)
    # silu(a) = a e^a / (1 + e^a) below 0: e^a of 64 bits reaches to e^-745
    e = torch.exp(-a.abs())
    return torch.where(a < 0, a * e, a) / (1 + e) * u


def _check(gu):
    F = gu.shape[1] // 2
    got = mk.mk_swiglu_i8(gu.cuda())
    h = _exact(gu)
    m = h.abs().amax(dim=1)
    assert ((m >= 2.0 ** -119) & (m < 2.0 ** 128)).all()
    q, s = got["q"].cpu().double(), got["scale"].cpu().double()
    assert ((127 * s - m).abs() <= 2.0 ** -19 * m).all()
    assert ((q - 127 * h / m[:, None]).abs() <= 0.5 + 127 * 2.0 ** -19).all()
    assert q.shape == (gu.shape[0], F) and (q.abs().amax(dim=1) == 127).all()


@pytest.mark.parametrize("F", [8, 272, 2056, 16384])
@pytest.mark.parametrize("lo,hi,exponents", [
    (-100.0, -60.0, (60, 127)), (-90.0, -86.0, (20, 126)), (-140.0, -90.0, (100, 126)), (60.0, 140.0, (-100, 100)),
    (-200.0, 200.0, (-60, 100)), (-81.0, -79.0, (0, 60)),
])
def test_gates_far_from_zero(F, lo, hi, exponents):
    """Values of u across a power of two a row, so that a row's h lie close together."""
    g = torch.Generator().manual_seed(F + int(lo))
    rows = 40
    gate = lo + (hi - lo) * torch.rand(rows, 1, generator=g) + 0.5 * torch.rand(rows, F, generator=g)
    power = torch.randint(*exponents, (rows, 1), generator=g).double()
    u = ((1 + torch.rand(rows, F, generator=g)).double() * 2.0 ** power).float()
    u[:, ::3] *= -1
    gu = torch.cat([gate, u], dim=1).to(BF)
    h = _exact(gu).abs().amax(dim=1)
    gu = gu[(h >= 2.0 ** -119) & (h < 2.0 ** 128)].contiguous()
    assert len(gu) >= 10
    _check(gu)


def test_every_gate_below_minus_60():
    """Each bf16 gate from -60 down to -210 in a row of its own, u the largest power of two and one between."""
    gate = torch.arange(0xC270, 0xC352, dtype=torch.int32).to(torch.int16).view(BF)
    gu = torch.zeros(len(gate), 16, dtype=BF)
    gu[:, 0], gu[:, 8] = gate, 2.0 ** 127
    gu[:, 1], gu[:, 9] = gate, -1.6e38
    h = _exact(gu).abs().amax(dim=1)
    keep = h >= 2.0 ** -119
    assert keep.sum() > 190 and (_exact(gu) != 0).any(dim=1).all()
    _check(gu[keep].contiguous())


def test_far_gates_beside_ordinary_ones():
    """What is far below its row's maximum has code 0, and ordinary values keep the codes that they have alone."""
    g = torch.Generator().manual_seed(1)
    gu = (2 * torch.randn(30, 2 * 704, generator=g)).to(BF)
    alone = mk.mk_swiglu_i8(gu.cuda())
    far = gu.clone()
    far[:, 5:704:7] = torch.tensor([-81.0, -88.5, -95.0, -110.0, -400.0, -1e30, torch.finfo(BF).min]).to(BF).repeat(15)[:100]
    near = torch.ones(704, dtype=torch.bool)
    near[5:704:7] = False
    keep = _exact(gu)[:, near].abs().amax(1) == _exact(gu).abs().amax(1)   # the maximum is still there
    got = mk.mk_swiglu_i8(far.cuda())
    assert keep.sum() > 10
    assert torch.equal(got["scale"].cpu()[keep], alone["scale"].cpu()[keep])
    assert torch.equal(got["q"].cpu()[keep][:, near], alone["q"].cpu()[keep][:, near])
    assert (got["q"].cpu()[keep][:, ~near] == 0).all()


def test_rows_of_zeros_and_what_is_not_finite():
    inf, nan = float("inf"), float("nan")
    gu = torch.randn(12, 32, generator=torch.Generator().manual_seed(2)).to(BF)
    gu[1, :16] = 0.0                       # gates of zero
    gu[2, 16:] = -0.0                      # values of zero
    gu[3, :16] = torch.finfo(BF).min       # e^g u is below everything
    gu[4, 3], gu[5, 3], gu[6, 3] = nan, -inf, inf
    gu[7, 19], gu[8, 19] = nan, inf
    gu[9, 3], gu[9, 19] = -100.0, inf
    gu[10, 3], gu[10, 19] = 1e30, 1e30     # a product past fp32
    got = mk.mk_swiglu_i8(gu.cuda())
    q, s = got["q"].cpu(), got["scale"].cpu()
    for r in (1, 2, 3):
        assert (q[r] == 0).all() and s[r] == 0, r
    for r in (4, 5, 6, 7, 8, 9, 10):
        assert (q[r] == 0).all() and s[r].isnan(), r
    _check(gu[[0, 11]])


@pytest.mark.parametrize("F", [8, 704])
def test_gradient_of_gates_far_below_zero(F):
    """mk_swiglu_backward where s = 1 / (1 + e^-g) is below fp32's range and the gradients are not: dg = dh u s (1 + g (1 - s)), du =
    dh g s within 2^-20 for the operations (see test_gpu_ffn_backward.py) and a bf16 rounding; what is below 2^-126 may be flushed."""
    g = torch.Generator().manual_seed(F)
    rows = 160
    gate = (-75.0 - torch.arange(rows) * 0.9)[:, None] + 0.5 * torch.rand(rows, F, generator=g)
    lift = ((-gate[:, :1]).double() * 1.4427 / 2).floor()   # dh and u each make up for half of e^g
    u = (torch.randn(rows, F, generator=g).double() * 2.0 ** lift.clamp(max=120)).to(BF)
    dh = (torch.randn(rows, F, generator=g).double() * 2.0 ** lift.clamp(max=120)).to(BF)
    gate = gate.to(BF)
    gate[0, :4] = torch.tensor([-80.0, -80.5, -1e30, torch.finfo(BF).min]).to(BF)
    got = mk.mk_swiglu_backward(torch.cat([gate, u], 1).cuda(), dh.cuda())["dgate_up"].cpu().double()
    a, U, d = gate.double(), u.double(), dh.double()
    e = torch.exp(a)
    s, s1 = e / (1 + e), 1 / (1 + e)
    dg, du = d * U * s * (1 + a * s1), d * a * s
    assert (dg[1:].abs() > 2.0 ** -100).all() and (dg.abs() < 2.0 ** 127).all()
    assert ((got[:, :F] - dg).abs() <= (2.0 ** -8 + 2.0 ** -19) * dg.abs() + 2.0 ** -126).all()
    assert ((got[:, F:] - du).abs() <= (2.0 ** -8 + 2.0 ** -20) * du.abs() + 2.0 ** -126).all()
    h = mk.mk_swiglu(torch.cat([gate, u], 1).cuda())
    both = mk.mk_swiglu_backward(torch.cat([gate, u], 1).cuda(), dh.cuda(), h=True)
    assert torch.equal(both["h"], h) and torch.equal(both["dgate_up"].cpu().double(), got)
