"""mk_add_rmsnorm against its formula in fp64 on the CPU.

Tolerances (u = 2^-24, the relative rounding error of fp32):
  residual  one fp32 addition and one bf16 rounding: (2^-8 + u) |h|.
  y         the sum of squares adds at most 8 + 4 + 6 + 16 positive fp32 terms on top of each other per path, so it is
            off by at most 36 u relative; mean, eps, square root, reciprocal and two products add at most 8 u:
            below 2^-18 with the square root's halving left out.  With the bf16 rounding: (2^-8 + 2^-18) |y|.
  q8_scale  a maximum of such y, one division: 2^-17 relative.
  q8        against y / s with the s the GPU returned: e4m3's half step (2^-4 relative, 2^-10 absolute below 2^-6),
            with 2^-17 relative on the value before it.
"""
import numpy as np
import pytest
import torch

import moe_dispatch_expert_amd as mk

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _inputs(T, d, residual, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, d, generator=g).to(torch.bfloat16)
    r = (2 * torch.randn(T, d, generator=g)).to(torch.bfloat16) if residual else None
    gamma = (1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16)
    return x, r, gamma


def _ref(x, r, gamma, eps=EPS):
    h = x.double() if r is None else x.double() + r.double()
    y = h * gamma.double() / torch.sqrt((h * h).mean(dim=1, keepdim=True) + eps)
    return h, y


def _check(out, x, r, gamma, eps=EPS):
    h, y = _ref(x, r, gamma, eps)
    if "residual" in out:
        got = out["residual"].cpu().double()
        assert ((got - h).abs() <= (2.0 ** -8 + 2.0 ** -24) * h.abs()).all()
    if "y" in out:
        got = out["y"].cpu().double()
        assert ((got - y).abs() <= (2.0 ** -8 + 2.0 ** -18) * y.abs() + 2.0 ** -133).all()
    if "q8" in out:
        T, d = x.shape
        s = out["q8_scale"].cpu().double()
        s_ref = y.view(T, d // 128, 128).abs().amax(dim=2).clamp_min(2.0 ** -40) / 448.0
        assert ((s - s_ref).abs() <= 2.0 ** -17 * s_ref).all()
        v = y / s.repeat_interleave(128, dim=1)
        got = out["q8"].cpu().double()
        tol = torch.maximum(2.0 ** -4 * v.abs(), torch.tensor(2.0 ** -10, dtype=torch.float64)) + 2.0 ** -17 * v.abs()
        assert ((got - v).abs() <= tol).all()


def _dev(*ts):
    return [None if t is None else t.cuda() for t in ts]


@pytest.mark.parametrize("T,d,residual,bf16,q8", [
    (1, 8, False, True, False),
    (1, 128, True, True, True),
    (1, 7168, True, True, True),
    (2, 2048, False, True, False),
    (3, 2056, True, True, False),      # one piece past 256 threads
    (5, 4104, True, True, False),      # one piece past 512
    (37, 2048, True, False, True),
    (129, 512, True, True, True),
    (67, 1000, True, True, False),
    (300, 4096, False, True, True),
    (1000, 7168, True, True, True),
    (9, 8192, True, True, True),
    (4, 8200, False, True, False),     # one piece past 1024 threads
    (3, 16384, True, True, True),
    (2, 16512, True, True, True),
    (2, 32768, True, True, True),
    (4111, 640, True, True, True),
    (2500, 1032, True, True, False),
])
def test_norm_matches_formula(T, d, residual, bf16, q8):
    x, r, gamma = _inputs(T, d, residual, T + d)
    dx, dr, dg = _dev(x, r, gamma)
    out = mk.mk_add_rmsnorm(dx, dg, dr, eps=EPS, bf16=bf16, q8=q8)
    assert set(out) == ({"residual"} if residual else set()) | ({"y"} if bf16 else set()) | \
        ({"q8", "q8_scale"} if q8 else set())
    torch.cuda.synchronize()
    assert torch.equal(dx.cpu(), x)
    _check(out, x, r, gamma)


def test_norm_in_place_gives_the_same_bits():
    x, r, gamma = _inputs(77, 4096, True, 5)
    dx, dr, dg = _dev(x, r, gamma)
    want = mk.mk_add_rmsnorm(dx, dg, dr, q8=True)
    got = mk.mk_add_rmsnorm(dx, dg, dr, q8=True, out={"residual": dr, "y": dx})   # h over the residual, y over x
    assert got["residual"] is dr and got["y"] is dx
    for n in want:
        assert torch.equal(want[n].view(torch.uint8), got[n].view(torch.uint8)), n


def test_norm_rows_do_not_depend_on_the_batch():
    """A row's bits are the same alone, in a small batch and in a large one."""
    x, r, gamma = _inputs(3000, 2048, True, 6)
    dx, dr, dg = _dev(x, r, gamma)
    big = mk.mk_add_rmsnorm(dx, dg, dr, q8=True)
    for a, b in ((0, 1), (7, 20), (1500, 1900)):
        part = mk.mk_add_rmsnorm(dx[a:b], dg, dr[a:b], q8=True)
        for n in part:
            assert torch.equal(part[n].view(torch.uint8), big[n][a:b].view(torch.uint8)), n


def test_norm_extreme_rows():
    """Zero rows, rows of tiny and of large values, and rows holding a NaN or an infinity, which must not touch
    their neighbours."""
    T, d = 8, 512
    x, _, gamma = _inputs(T, d, False, 7)
    x[1] = 0
    x[2] = (x[2].float() * 2.0 ** -60).to(torch.bfloat16)
    x[3] = (x[3].float() * 2.0 ** 50).to(torch.bfloat16)
    x[4, 100] = float("nan")
    x[6, 5] = float("inf")
    dx, dg = _dev(x, gamma)
    out = mk.mk_add_rmsnorm(dx, dg, q8=True)
    fine = [0, 1, 2, 3, 5, 7]
    _check({n: v.view(torch.uint8)[fine].view(v.dtype) for n, v in out.items()}, x[fine], None, gamma)
    assert (out["y"][1] == 0).all() and (out["q8"][1].float() == 0).all()
    assert (out["q8_scale"][1].cpu() == torch.tensor(2.0 ** -40, dtype=torch.float32) / 448.0).all()
    assert torch.isnan(out["y"][4].float()).all() and torch.isnan(out["q8"][4].float()).all()
    y6, q6 = out["y"][6].float(), out["q8"][6].float()      # inf * (1 / inf) in its own column, 0 elsewhere
    assert torch.isnan(y6[5]) and torch.isnan(q6[5])
    assert (y6[torch.arange(d, device=y6.device) != 5] == 0).all()


def test_norm_zero_rows_is_a_no_op():
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    out = mk.mk_add_rmsnorm(x, torch.ones(256, dtype=torch.bfloat16, device="cuda"), x.clone(), q8=True)
    assert out["y"].shape == (0, 256) and out["q8_scale"].shape == (0, 2)


def test_norm_offsets_past_32_bits():
    """More than 2^31 elements (and more than 2^32 bytes) before the last rows."""
    T, d = 270000, 8192
    rows = [0, 1, T // 2, T - 2, T - 1]
    x, _, gamma = _inputs(len(rows), d, False, 8)
    dx = torch.empty(T, d, dtype=torch.bfloat16, device="cuda").zero_()
    for i, t in enumerate(rows):
        dx[t].copy_(x[i])
    out = mk.mk_add_rmsnorm(dx, gamma.cuda(), q8=True, out={"y": dx})
    at = torch.tensor(rows, device="cuda")
    _check({"y": out["y"][at], "q8": out["q8"].view(torch.uint8)[at].view(torch.float8_e4m3fn),
            "q8_scale": out["q8_scale"][at]}, x, None, gamma)


def test_norm_captured_and_on_another_stream():
    x, r, gamma = _inputs(64, 7168, True, 9)
    dx, dr, dg = _dev(x, r, gamma)
    want = mk.mk_add_rmsnorm(dx, dg, dr, q8=True)
    out = {n: torch.empty_like(v) for n, v in want.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mk.mk_add_rmsnorm(dx, dg, dr, q8=True, out=out, stream=side)
    side.synchronize()
    for n in want:
        assert torch.equal(want[n].view(torch.uint8), out[n].view(torch.uint8)), n
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mk.mk_add_rmsnorm(dx, dg, dr, q8=True, out=out)
    for i in range(4):
        x2 = (x.float() * (i + 1)).to(torch.bfloat16)
        dx.copy_(x2)
        for v in out.values():
            v.view(torch.uint8).zero_()
        g.replay()
        torch.cuda.synchronize()
        _check(out, x2, r, gamma)
        eager = mk.mk_add_rmsnorm(dx, dg, dr, q8=True)
        for n in eager:
            assert torch.equal(eager[n].view(torch.uint8), out[n].view(torch.uint8)), n


def test_norm_binding_refusals():
    x, r, gamma = _dev(*_inputs(4, 256, True, 10))
    for bad in (dict(x=x.float()), dict(gamma=gamma[:128]), dict(residual=r[:3]), dict(x=x.t().contiguous().t()),
                dict(residual=r.cpu()), dict(out={"y": torch.empty_like(x)[:, :128]}),
                dict(out={"y": torch.empty(4, 256, device="cuda")})):
        kw = dict(dict(x=x, gamma=gamma, residual=r), **bad)
        with pytest.raises(ValueError):
            mk.mk_add_rmsnorm(kw["x"], kw["gamma"], kw["residual"], q8=True, out=kw.get("out"))
    odd = torch.empty(4 * 256 + 8, dtype=torch.bfloat16, device="cuda")[4:4 + 1024].view(4, 256)   # 8-byte aligned
    with pytest.raises(mk.MkError) as e:
        mk.mk_add_rmsnorm(odd, gamma)
    assert e.value.status == mk.MK_EINVAL
    with pytest.raises(mk.MkError):
        mk.mk_add_rmsnorm(x, gamma, r, out={"residual": x, "y": x})
    assert np.isfinite(mk.mk_add_rmsnorm(x, gamma, r)["y"].float().cpu().numpy()).all()
