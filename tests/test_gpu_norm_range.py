"""mk_add_rmsnorm at the ends of its range: more rows than one launch's grid holds, and eps = 0.  Formula and tolerances as in
test_gpu_norm.py."""
import pytest
import torch

import moe_dispatch_expert_amd as mk
from test_gpu_norm import _check, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,d,q8", [((1 << 24) + 3, 8, False), ((1 << 23) + 5, 128, True)])
def test_norm_of_more_rows_than_a_grid(T, d, q8):
    """2^24 workgroups of 256 threads are more work items than one launch takes."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    gamma = (1 + 0.2 * torch.randn(d, generator=torch.Generator().manual_seed(2))).to(torch.bfloat16)
    r = x.flip(0).contiguous()
    out = mk.mk_add_rmsnorm(x, gamma.cuda(), r, q8=q8)
    for at in (0, (1 << 22) - 8, (1 << 22), (1 << 23) - 100, T - 1000):
        rows = slice(at, at + 1000)
        part = {n: v[rows] if v.dtype != torch.float8_e4m3fn else v.view(torch.uint8)[rows].view(v.dtype)
                for n, v in out.items()}
        _check(part, x[rows].cpu(), r[rows].cpu(), gamma)
    # every row: its y has a mean square of about gamma's
    y = out["y"].float()
    ms = (y / gamma.cuda().float()).square().mean(1)
    assert ((ms - 1).abs() < 0.02).all()


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("d", [8, 1024, 16384])
def test_norm_of_tiny_rows_without_eps(d, residual):
    """Squares that fp32 cannot hold: with eps = 0 (or as tiny) the formula's values are still of ordinary size."""
    x, r, gamma = _inputs(6, d, residual, 12)
    scale = torch.tensor([0, -40, -66, -80, -110, -120])[:, None].double()
    x = (x.double() * 2.0 ** scale).to(torch.bfloat16)
    r = None if r is None else (r.double() * 2.0 ** scale).to(torch.bfloat16)
    dx, dr = x.cuda(), None if r is None else r.cuda()
    for eps in (0.0, 1e-38, 1e-30):
        out = mk.mk_add_rmsnorm(dx, gamma.cuda(), dr, eps=eps, q8=d % 128 == 0)
        _check(out, x, r, gamma, eps=float(torch.tensor(eps, dtype=torch.float32)))


def test_norm_of_zero_rows_without_eps():
    """0 / 0 in the formula: NaN in that row only."""
    x, _, gamma = _inputs(3, 256, False, 13)
    x[1] = 0
    y = mk.mk_add_rmsnorm(x.cuda(), gamma.cuda(), eps=0.0)["y"].float().cpu()
    assert torch.isnan(y[1]).all() and torch.isfinite(y[[0, 2]]).all()
    y = mk.mk_add_rmsnorm(x.cuda(), gamma.cuda(), eps=1e-38)["y"].float().cpu()
    assert (y[1] == 0).all()
