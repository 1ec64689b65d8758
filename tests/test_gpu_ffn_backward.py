"""mk_combine_backward and mk_swiglu_backward against their formulas, and the whole backward pass of the expert FFN.

Tolerances: a row of the combine's gradient is one fp32 product rounded to bf16, compared bit for bit.  A gate's gradient is
a sum of N exact products: a thread adds 8 per piece of 2048 columns, then a tree of 6 + 2 and one addition per 8192
columns, so (N / 256 + N / 8192 + 12) 2^-24 of sum |terms| covers it.  The SwiGLU's gradient evaluates e^-|g| (2 ulp) and at
most 8 more operations in fp32: below 2^-20 of |dh u| s (1 + |g| (1 - s)) (|dh g s| for the other half), then a bf16
rounding of 2^-8 of the value; results below 2^-126 may be flushed."""
import pytest
import torch

import grouped_ref as ref
import moe_dispatch_expert_amd as mk

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _slots(g, T, k, rows, none=0.3):
    """Distinct slots of [0, rows) for some of the choices, -1 or values outside for the others."""
    n = T * k
    pick = torch.randperm(max(rows, n), generator=g)[:n].to(torch.int32)
    pick[pick >= rows] = -1
    pick[torch.rand(n, generator=g) < none] = -1
    return pick.view(T, k)


@pytest.mark.parametrize("T,k,N,rows", [
    (1, 1, 8, 1), (1, 8, 7168, 8), (37, 6, 2048, 222), (37, 6, 2056, 300), (5, 32, 4104, 100), (64, 2, 8192, 128),
    (9, 3, 8200, 20), (3, 2, 32768, 6), (1000, 4, 72, 4000), (130, 7, 512, 200), (4, 2, 64, 0),
])
@pytest.mark.parametrize("gates", [True, False])
def test_combine_backward(T, k, N, rows, gates):
    g = torch.Generator().manual_seed(T + N)
    dout, y = torch.randn(T, N, generator=g).to(BF), torch.randn(rows, N, generator=g).to(BF)
    w, slot = torch.rand(T, k, generator=g), _slots(g, T, k, rows)
    if T > 3:
        slot[1, 0], slot[2, 0] = rows, 2 ** 31 - 1   # outside
    out = {"dy_perm": torch.full((rows, N), 9.0, dtype=BF, device="cuda")}
    got = mk.mk_combine_backward(dout.cuda(), y.cuda(), slot.cuda(), w.cuda(), gates=gates, out=out)
    want = torch.full((rows, N), 9.0, dtype=BF)
    dw, size = torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            s = int(slot[t, j])
            if 0 <= s < rows:
                want[s] = (w[t, j] * dout[t].float()).to(BF)
                terms = dout[t].double() * y[s].double()
                dw[t, j], size[t, j] = terms.sum(), terms.abs().sum()
    assert torch.equal(got["dy_perm"].cpu(), want)
    assert ("dtopk_w" in got) == gates
    if gates:
        assert ((got["dtopk_w"].cpu().double() - dw).abs() <= (N / 256 + N / 8192 + 12) * 2.0 ** -24 * size).all()


def test_combine_backward_in_place_and_repeated_slots():
    """dy in the place of y_perm, with a token that names a slot twice (its gates add up, its gradients are equal)."""
    g = torch.Generator().manual_seed(4)
    T, k, N = 6, 4, 2560
    dout, y = ref.whole(g, T, N), ref.whole(g, T * k, N)
    w = torch.randint(1, 9, (T, k), generator=g) / 8.0
    slot = torch.arange(T * k, dtype=torch.int32).view(T, k)
    slot[2, 3], slot[2, 1], slot[4, 0] = slot[2, 0], slot[2, 0], slot[4, 3]
    d = y.cuda()
    got = mk.mk_combine_backward(dout.cuda(), d, slot.cuda(), w.cuda(), out={"dy_perm": d})
    want = y.clone()
    for t in range(T):
        for j in range(k):
            want[slot[t, j]] = (w[t][slot[t] == slot[t, j]].sum() * dout[t].float()).to(BF)
            assert got["dtopk_w"][t, j] == (dout[t].double() * y[slot[t, j]].double()).sum()
    assert torch.equal(d.cpu(), want)


@pytest.mark.parametrize("rows,F", [(1, 8), (221, 1408), (3, 14336), (1000, 72), (65, 272), (4000, 256)])
@pytest.mark.parametrize("in_place", [False, True])
def test_swiglu_backward(rows, F, in_place):
    g = torch.Generator().manual_seed(rows + F)
    gu, dh = (3 * torch.randn(rows, 2 * F, generator=g)).to(BF), torch.randn(rows, F, generator=g).to(BF)
    edge = torch.tensor([0.0, -0.0, 88.0, -88.0, -120.0, 1e30, -1e30, -1.2785])
    gu[0, :8] = edge.to(BF)
    d_gu, d_dh = gu.cuda(), dh.cuda()
    h = mk.mk_swiglu(d_gu)
    out = {"dgate_up": d_gu, "h": d_dh} if in_place else None
    got = mk.mk_swiglu_backward(d_gu, d_dh, h=True, out=out)
    assert torch.equal(got["h"], h)
    a, u, d = gu[:, :F].double(), gu[:, F:].double(), dh.double()
    s, s1 = torch.sigmoid(a), torch.sigmoid(-a)
    dg, du = d * u * s * (1 + a * s1), d * a * s
    r = got["dgate_up"].cpu().double()
    size = (d * u).abs() * s * (1 + a.abs() * s1)
    assert ((r[:, :F] - dg).abs() <= 2.0 ** -20 * size + 2.0 ** -8 * dg.abs() + 2.0 ** -126).all()
    assert ((r[:, F:] - du).abs() <= (2.0 ** -8 + 2.0 ** -20) * du.abs() + 2.0 ** -126).all()


def test_swiglu_backward_is_the_gradient():
    """Against differences of silu(g) u in 64 bits: step 2^-12, so 2^-24 |h'''| / 6 < 2^-24 from the derivative."""
    g = torch.Generator().manual_seed(8)
    gu, dh = (2 * torch.randn(50, 128, generator=g)).to(BF), torch.randn(50, 64, generator=g).to(BF)
    got = mk.mk_swiglu_backward(gu.cuda(), dh.cuda())["dgate_up"].cpu().double()
    a, u, d, step = gu[:, :64].double(), gu[:, 64:].double(), dh.double(), 2.0 ** -12

    def h(a, u):
        return a * torch.sigmoid(a) * u

    dg = d * (h(a + step, u) - h(a - step, u)) / (2 * step)
    du = d * (h(a, u + step) - h(a, u - step)) / (2 * step)
    assert ((got[:, :64] - dg).abs() <= 2.0 ** -8 * dg.abs() + 2.0 ** -18 * (d * u).abs()).all()
    assert ((got[:, 64:] - du).abs() <= 2.0 ** -8 * du.abs() + 2.0 ** -18 * d.abs()).all()


def test_swiglu_backward_leaves_rows_behind_the_valid_ones():
    g = torch.Generator().manual_seed(9)
    gu, dh = torch.randn(20, 128, generator=g).to(BF).cuda(), torch.randn(20, 64, generator=g).to(BF).cuda()
    full = mk.mk_swiglu_backward(gu, dh, h=True)
    counts = torch.tensor([0, 3, 20, -5, 100, 13], dtype=torch.int32, device="cuda")
    for i, n in enumerate((0, 3, 20, 0, 20, 13)):
        out = {"dgate_up": torch.full_like(gu, 7.0), "h": torch.full_like(dh, 7.0)}
        mk.mk_swiglu_backward(gu, dh, h=True, rows_valid=counts[i:i + 1], out=out)
        for name in out:
            assert torch.equal(out[name][:n], full[name][:n]) and (out[name][n:] == 7.0).all()


def _forward_backward(x, w1, w2, wr, dout, k, F):
    """A training step's expert FFN through the library: outputs, then every gradient."""
    p = mk.mk_dispatch_gemm(x, w1, k, w_router=wr)
    off, rt = p["expert_offsets"], p["row_token"]
    h = mk.mk_swiglu(p["y_perm"])
    z = mk.mk_grouped_gemm(h, off, w2)
    out = mk.mk_combine(z, p["slot_of"], p["topk_w"])
    b = mk.mk_combine_backward(dout, z, p["slot_of"], p["topk_w"])
    dh = mk.mk_grouped_gemm_dgrad(b["dy_perm"], off, w2)
    s = mk.mk_swiglu_backward(p["y_perm"], dh, h=True, rows_valid=off[w1.shape[0]:])
    dw2 = mk.mk_grouped_gemm_wgrad(b["dy_perm"], s["h"], off)
    dw1 = mk.mk_grouped_gemm_wgrad(s["dgate_up"], x, off, row_token=rt)
    da = mk.mk_grouped_gemm_dgrad(s["dgate_up"], off, w1)
    dx = mk.mk_combine(da, p["slot_of"], torch.ones_like(p["topk_w"]))
    return {"out": out, "dgates": b["dtopk_w"], "dw1": dw1, "dw2": dw2, "dx": dx, "ids": p["topk_ids"],
            "gates": p["topk_w"]}


def test_backward_pass_of_the_expert_ffn():
    """Every gradient of the chain against 64-bit differentiation of  sum(dout * out)  at the same routing.  Between input and
    gradient lie at most 8 bf16 roundings of 2^-8 each, on quantities whose relative errors the chain carries on with
    factors of about one: each gradient is within 16 * 2^-8 of the exact one in norm."""
    g = torch.Generator().manual_seed(12)
    T, d, E, k, F = 200, 256, 6, 2, 136
    x, dout = torch.randn(T, d, generator=g).to(BF), torch.randn(T, d, generator=g).to(BF)
    w1 = (torch.randn(E, 2 * F, d, generator=g) / 16).to(BF)
    w2 = (torch.randn(E, d, F, generator=g) / 12).to(BF)
    # grouped products contract over multiples of 128 in the forward direction
    w2 = torch.nn.functional.pad(w2, (0, 256 - F))
    w1 = torch.cat([torch.nn.functional.pad(w1[:, :F], (0, 0, 0, 256 - F)),
                    torch.nn.functional.pad(w1[:, F:], (0, 0, 0, 256 - F))], dim=1).contiguous()
    wr = torch.randn(d, E, generator=g) / 16
    wr[:, 3] = -10 * x.float().mean(0)   # an expert with hardly a row
    got = _forward_backward(*(t.cuda() for t in (x, w1, w2, wr, dout)), k, 256)
    ids, gates = got["ids"].cpu().long(), got["gates"].cpu().double().requires_grad_()
    X, W1, W2 = (t.double().requires_grad_() for t in (x, w1, w2))
    out = torch.zeros(T, d, dtype=torch.float64)
    for j in range(k):
        gu = torch.bmm(W1[ids[:, j]], X[:, :, None])[:, :, 0]
        h = torch.nn.functional.silu(gu[:, :256]) * gu[:, 256:]
        out = out + gates[:, j, None] * torch.bmm(W2[ids[:, j]], h[:, :, None])[:, :, 0]
    (out * dout.double()).sum().backward()
    for name, want in (("out", out.detach()), ("dgates", gates.grad), ("dw1", W1.grad), ("dw2", W2.grad),
                       ("dx", X.grad)):
        err = (got[name].cpu().double() - want).norm() / want.norm()
        assert err <= 16 * 2.0 ** -8, (name, float(err))
    for e in range(E):   # experts without rows have no gradient
        if not (ids == e).any():
            assert (got["dw1"][e] == 0).all() and (got["dw2"][e] == 0).all()


def test_captured_backward_pass():
    """The backward pass in a graph, replayed with other inputs between eager passes."""
    g = torch.Generator().manual_seed(13)
    T, d, E, k, F = 96, 128, 8, 2, 128
    x, dout = torch.randn(T, d, generator=g).to(BF).cuda(), torch.randn(T, d, generator=g).to(BF).cuda()
    w1 = (torch.randn(E, 2 * F, d, generator=g) / 11).to(BF).cuda()
    w2 = (torch.randn(E, d, F, generator=g) / 11).to(BF).cuda()
    ids = torch.rand(T, E, generator=g).topk(k, 1).indices.to(torch.int32).cuda()
    gates = torch.rand(T, k, generator=g).cuda()
    gu = torch.randn(T * k, 2 * F, generator=g).to(BF).cuda()

    def step():
        lay = mk.mk_expert_layout(ids, E)
        off, rt = lay["expert_offsets"], lay["row_token"]
        h = mk.mk_swiglu(gu)
        z = mk.mk_grouped_gemm(h, off, w2)
        b = mk.mk_combine_backward(dout, z, lay["slot_of"], gates)
        dh = mk.mk_grouped_gemm_dgrad(b["dy_perm"], off, w2)
        s = mk.mk_swiglu_backward(gu, dh, h=True, rows_valid=off[E:])
        dw2 = mk.mk_grouped_gemm_wgrad(b["dy_perm"], s["h"], off)
        dw1 = mk.mk_grouped_gemm_wgrad(s["dgate_up"], x, off, row_token=rt, dtype=BF)
        q = mk.mk_quant_i8(x)
        wq = mk.mk_quant_i8(w1.view(-1, d))
        y = mk.mk_grouped_gemm_i8(q["q"], q["scale"], off, wq["q"].view(w1.shape), wq["scale"].view(E, 2 * F),
                                  row_token=rt)
        return [b["dtopk_w"], dh, s["dgate_up"], dw2, dw1, y, mk.mk_swiglu_i8(y)["q"]]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        ids.copy_(torch.rand(T, E, generator=g).topk(k, 1).indices.to(torch.int32))
        x.copy_(torch.randn(T, d, generator=g).to(BF))
        dout.mul_(1.25)
        for o in out:
            o.zero_()
        graph.replay()
        for a, b in zip(out, step()):
            assert torch.equal(a, b), i
        torch.cuda.synchronize()


def test_calls_on_another_stream():
    """Each call's outputs are dropped while it runs, and the current stream allocates and writes meanwhile."""
    g = torch.Generator().manual_seed(14)
    side = torch.cuda.Stream()
    off = torch.tensor([0, 100, 100, 250], dtype=torch.int32, device="cuda")
    dy, a = torch.randn(250, 272, generator=g).to(BF).cuda(), torch.randn(250, 136, generator=g).to(BF).cuda()
    w, half = torch.randn(3, 272, 136, generator=g).to(BF).cuda(), torch.randn(250, 136, generator=g).to(BF).cuda()

    def chain(s):
        da = mk.mk_grouped_gemm_dgrad(dy, off, w, stream=s)
        dw = mk.mk_grouped_gemm_wgrad(dy, da, off, stream=s)
        q = mk.mk_quant_i8(da, stream=s)
        return [da, dw, q["q"], q["scale"], mk.mk_swiglu_i8(dy, stream=s)["q"],
                mk.mk_swiglu_backward(dy, half, stream=s)["dgate_up"]]

    want = chain(None)
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(20):
        got.append(chain(side))
        torch.full((1 << 16,), float("nan"), device="cuda")
    torch.cuda.current_stream().wait_stream(side)
    for outs in got:
        for x, y in zip(outs, want):
            assert torch.equal(x, y)
