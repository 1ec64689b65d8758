"""mk_moe_layer and mk_moe_layer_q8 against the layer in fp64 (tests/layer_ref.py, which derives the tolerances), and
their routing bit for bit against mk_route_topk."""
import math

import pytest
import torch

import layer_ref as ref
import moe_dispatch_expert_amd as mk

pytestmark = pytest.mark.gpu


class Case:
    """Seeded CPU inputs and their device copies."""

    def __init__(self, T, d, E, k, E_local, F, q8=False, e_begin=0, bias=False, seed=0):
        g = torch.Generator().manual_seed(1000 * seed + T * 31 + d + 7 * F + E)
        self.T, self.d, self.E, self.k, self.E_local, self.F, self.q8, self.e_begin = T, d, E, k, E_local, F, q8, e_begin
        self.x = torch.randn(T, d, generator=g).to(torch.bfloat16)
        self.wr = torch.randn(d, E, generator=g) / math.sqrt(d)
        self.bias = torch.randn(E, generator=g) if bias else None
        self.gu = (torch.randn(E_local, 2 * F, d, generator=g) / math.sqrt(d)).to(torch.bfloat16)
        self.dn = (torch.randn(E_local, d, F, generator=g) / math.sqrt(F)).to(torch.bfloat16)
        if q8:
            self.xq, self.xs = ref.rows_q8(self.x)
            gq, gs = ref.blocks_q8(self.gu[:, :F])
            uq, us = ref.blocks_q8(self.gu[:, F:])
            self.gq = torch.cat([gq.view(torch.uint8), uq.view(torch.uint8)], 1).view(torch.float8_e4m3fn)
            self.gs = torch.cat([gs, us], 1).contiguous()
            self.dq, self.ds = ref.blocks_q8(self.dn)
            self.x64 = ref.rows_values(self.xq, self.xs)
            self.gu64 = torch.cat([ref.blocks_values(gq, gs), ref.blocks_values(uq, us)], 1)
            self.dn64 = ref.blocks_values(self.dq, self.ds)
        else:
            self.x64, self.gu64, self.dn64 = self.x.double(), self.gu.double(), self.dn.double()
        self.gpu = {n: v.cuda() for n, v in vars(self).items() if isinstance(v, torch.Tensor) and v.dtype != torch.float64}

    def call(self, ids=None, gates=None, rows=None, **kw):
        G = self.gpu
        cut = (lambda v: v) if rows is None else (lambda v: v[rows].contiguous())
        if ids is None:
            kw.update(w_router=G["wr"], bias=G.get("bias"))
        else:
            kw.update(topk_ids_in=cut(ids.cuda()), topk_w_in=cut(gates.cuda()), E=self.E)
        kw.setdefault("e_begin", self.e_begin)
        if self.q8:
            return mk.mk_moe_layer_q8(cut(G["xq"].view(torch.uint8)).view(torch.float8_e4m3fn), cut(G["xs"]), G["gq"],
                                      G["gs"], G["dq"], G["ds"], self.k, x=cut(G["x"]) if ids is None else None, **kw)
        return mk.mk_moe_layer(cut(G["x"]), G["gu"], G["dn"], self.k, **kw)

    def choices(self):
        """Buffers for the choices, filled with a pattern."""
        return {"topk_ids": torch.full((self.T, self.k), -7, dtype=torch.int32, device="cuda"),
                "topk_w": torch.full((self.T, self.k), -7.0, device="cuda")}

    def random_choices(self, seed, lo=None, hi=None):
        g = torch.Generator().manual_seed(seed)
        lo, hi = (0, self.E) if lo is None else (lo, hi)
        ids = torch.stack([torch.randperm(hi - lo, generator=g)[:self.k] + lo for _ in range(self.T)]).to(torch.int32)
        return ids, torch.rand(self.T, self.k, generator=g) + 0.1

    def check(self, out, ids, gates, rows=slice(None), what=""):
        want, bound = ref.layer(self.x64, self.gu64, self.dn64, ids.long().cpu(), gates.cpu(), self.e_begin)
        got = out.cpu().double()[rows]
        want, bound = want[rows], bound[rows]
        bad = ~((got - want).abs() <= bound)
        assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, first {torch.nonzero(bad)[0]}"
        # two independent bf16 roundings: at most 2^-8 / sqrt(3) rms each, together below 2^-8 in the 2-norm
        n = want.norm()
        if n > 0 and want.numel() >= 1024:
            assert (got - want).norm() <= 2.0 ** -8 * n, what


ROUTED = [
    # T, d, E, k, E_local, F, e_begin, bias
    (1, 128, 1, 1, 1, 8, 0, False),
    (1, 512, 8, 2, 8, 512, 0, False),
    (1, 2048, 64, 6, 64, 176, 0, True),
    (2, 256, 8, 2, 8, 24, 0, False),
    (3, 384, 65, 3, 65, 40, 0, True),          # E % 4 != 0, K split of 12 steps over 4 waves
    (5, 640, 60, 4, 60, 136, 0, False),        # E not a multiple of 32
    (8, 896, 256, 8, 32, 64, 224, True),       # last experts of a share
    (8, 7168, 256, 8, 16, 48, 16, False),      # the longest staged router segment
    (7, 8192, 40, 2, 4, 16, 3, False),         # a router segment in two chunks
    (4, 256, 300, 8, 300, 16, 0, False),       # more experts than the up kernel selects from
    (6, 128, 1024, 32, 1024, 8, 0, True),
    (9, 512, 8, 2, 8, 512, 0, False),          # one token past the vector router
    (16, 1024, 64, 6, 64, 88, 0, True),
    (17, 512, 64, 6, 64, 200, 0, False),       # two weight tiles per task, F % 16 != 0
    (33, 512, 8, 2, 8, 264, 0, False),
    (50, 256, 4, 3, 4, 96, 0, False),          # more than 32 rows per expert
    (128, 512, 16, 8, 8, 72, 4, False),        # 64 rows per expert
    (128, 256, 4, 4, 4, 40, 0, False),         # every token at every expert
    (128, 1024, 256, 8, 32, 128, 0, True),
    (100, 384, 1024, 32, 200, 16, 700, False),
]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("T,d,E,k,E_local,F,e_begin,bias", ROUTED)
def test_layer_routed_inside(T, d, E, k, E_local, F, e_begin, bias, q8):
    if q8:
        F = -(-F // 16) * 16
    c = Case(T, d, E, k, E_local, F, q8, e_begin, bias)
    o = c.call(out=c.choices())
    ids, w = mk.mk_route_topk(c.gpu["x"], c.gpu["wr"], k, c.gpu.get("bias"))
    assert torch.equal(o["topk_ids"], ids)
    assert torch.equal(o["topk_w"].view(torch.int32), w.view(torch.int32))
    c.check(o["out"], ids, w)


GIVEN = [
    (1, 256, 8, 2, 8, 64, 0), (3, 128, 16, 4, 4, 24, 8), (8, 512, 256, 8, 32, 128, 0), (16, 256, 8, 8, 8, 72, 0),
    (40, 384, 12, 3, 12, 56, 0), (127, 256, 6, 5, 6, 88, 0), (128, 128, 64, 2, 64, 16, 0),
]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("T,d,E,k,E_local,F,e_begin", GIVEN)
def test_layer_given_choices(T, d, E, k, E_local, F, e_begin, q8):
    """Ids from the caller: distinct ones, padding and out-of-range ids, and ids given twice."""
    if q8:
        F = -(-F // 16) * 16
    c = Case(T, d, E, k, E_local, F, q8, e_begin)
    ids, gates = c.random_choices(1)
    o = c.call(ids, gates, out=c.choices())
    assert torch.equal(o["topk_ids"].cpu(), ids) and torch.equal(o["topk_w"].cpu(), gates)
    c.check(o["out"], ids, gates, what="distinct")
    ids[::3, 0] = -1
    ids[1::4] = torch.iinfo(torch.int32).min
    ids[2::5, -1] = E + 1000000
    ids[0] = torch.iinfo(torch.int32).max
    o = c.call(ids, gates)
    c.check(o["out"], ids, gates, what="padding")
    assert (o["out"][0] == 0).all()
    if k > 1:
        ids, gates = c.random_choices(2)
        ids[:, k - 1] = ids[:, 0]
        if k > 3:
            ids[::2, 1] = ids[::2, 0]
        c.check(c.call(ids, gates)["out"], ids, gates, what="repeated")


@pytest.mark.parametrize("q8", [False, True])
def test_layer_no_local_choice(q8):
    c = Case(20, 256, 64, 4, 8, 32, q8, e_begin=16)
    ids, gates = c.random_choices(3, 32, 64)
    out = torch.full((20, 256), 5.0, dtype=torch.bfloat16, device="cuda")
    c.call(ids, gates, out={"out": out})
    assert (out == 0).all()


@pytest.mark.parametrize("q8", [False, True])
def test_layer_rows_do_not_depend_on_the_batch(q8):
    """A token's result has the same bits alone and in batches of any size (the router's two forms, both task shapes,
    every number of token tiles)."""
    c = Case(128, 512, 16, 4, 16, 176, q8)
    whole = c.call(out=c.choices())
    for rows in ([0], [127], list(range(8)), list(range(3, 12)), list(range(16)), list(range(60, 100))):
        part = c.call(rows=torch.tensor(rows, device="cuda"),
                      out={"topk_ids": torch.empty(len(rows), 4, dtype=torch.int32, device="cuda")})
        assert torch.equal(part["topk_ids"], whole["topk_ids"][rows])
        assert torch.equal(part["out"].view(torch.int16), whole["out"][rows].view(torch.int16)), rows


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("T", [5, 40])
def test_layer_valid_tokens(T, q8):
    """t_valid: the first tokens as in a call of that many, the rest of every output untouched, also past the ends."""
    c = Case(T, 256, 32, 3, 32, 48, q8)
    ids, gates = c.random_choices(4)
    for given in (False, True):
        kw = dict(ids=ids, gates=gates) if given else {}
        whole = c.call(out=c.choices(), **kw)
        for n in (0, 1, T - 1, T, T + 9, -3):
            m = max(0, min(T, n))
            o = dict(c.choices(), out=torch.full((T, 256), 3.0, dtype=torch.bfloat16, device="cuda"))
            c.call(out=o, t_valid=torch.tensor([n], dtype=torch.int32, device="cuda"), **kw)
            for name, fill in (("out", 3.0), ("topk_ids", -7), ("topk_w", -7.0)):
                assert torch.equal(o[name][:m], whole[name][:m]), (n, name)
                assert (o[name][m:] == fill).all(), (n, name)


@pytest.mark.parametrize("q8", [False, True])
def test_layer_nonfinite_values_stay_where_they_are(q8):
    """A NaN or infinity in one token, in an expert nobody chose and in memory behind the inputs reaches no other row."""
    c = Case(24, 256, 16, 2, 16, 40 if not q8 else 48, q8)
    ids, gates = c.random_choices(5, 0, 15)
    clean = c.call(ids, gates)["out"]
    G = c.gpu
    if q8:
        G["xs"][7] = float("nan")
        G["gs"][15], G["ds"][15] = float("inf"), float("nan")
    else:
        G["x"][7, 3] = float("nan")
        G["gu"][15], G["dn"][15] = float("inf"), float("nan")
    ws = torch.full((mk.mk_moe_layer_workspace_bytes(24, 256, 16, 2, 0, 16, c.F),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    out = c.call(ids, gates, workspace=ws)["out"]
    keep = [t for t in range(24) if t != 7]
    assert torch.equal(out[keep], clean[keep])
    assert torch.isnan(out[7].float()).all()


@pytest.mark.parametrize("q8", [False, True])
def test_layer_in_place_and_on_another_stream(q8):
    c = Case(12, 512, 8, 2, 8, 64, q8)
    want = c.call()["out"]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(want)
    c.call(out={"out": out}, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    x = c.gpu["x"]
    c.call(out={"out": x})
    assert torch.equal(x, want)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("T", [6, 48])
def test_layer_captured(T, q8):
    """A captured call replayed with other tokens, other weights of the router and another number of valid tokens, eager
    calls of the same workspace in between; two graphs sharing one workspace, replayed in turn."""
    c = Case(T, 512, 64, 4, 64, 80, q8)
    ws = torch.empty(mk.mk_moe_layer_workspace_bytes(T, 512, 64, 4, 0, 64, 80), dtype=torch.uint8, device="cuda")
    n = torch.tensor([T], dtype=torch.int32, device="cuda")
    o1, o2 = torch.zeros(T, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, 512, dtype=torch.bfloat16, device="cuda")
    ids, gates = c.random_choices(6)
    ids, gates = ids.cuda(), gates.cuda()
    c.call(out={"out": o1}, workspace=ws)   # once before the capture
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        c.call(out={"out": o1}, workspace=ws, t_valid=n)
    with torch.cuda.graph(g2):
        c.call(ids, gates, out={"out": o2}, workspace=ws)
    name = "xs" if q8 else "x"
    for i in range(5):
        c.gpu[name].mul_(1.0 + 0.25 * i)
        c.gpu["wr"].copy_(c.gpu["wr"].roll(1, dims=1))
        n.fill_(T - i)
        o1.zero_()
        o2.zero_()
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        e1 = c.call(workspace=ws)["out"]
        e2 = c.call(ids, gates, workspace=ws)["out"]
        assert torch.equal(o1[:T - i], e1[:T - i]) and (o1[T - i:] == 0).all()
        assert torch.equal(o2, e2)


def test_layer_two_calls_at_once():
    """Two streams with a workspace each."""
    c = Case(64, 1024, 64, 4, 64, 176)
    want = c.call()["out"]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    wss = [torch.empty(mk.mk_moe_layer_workspace_bytes(64, 1024, 64, 4, 0, 64, 176), dtype=torch.uint8, device="cuda")
           for _ in streams]
    outs = [torch.empty_like(want) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, ws, o in zip(streams, wss, outs):
            c.call(out={"out": o}, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


@pytest.mark.parametrize("T", [4, 96])
def test_layer_step_with_the_norms(T):
    """A decode step as used: norm (bf16 for the router, e4m3 for the experts), the 8-bit layer, and the next norm, which
    adds the layer's output to the residual stream; against the same step from the formulas."""
    d, E, k, F = 512, 32, 4, 144
    c = Case(T, d, E, k, E, F, True)
    g = torch.Generator().manual_seed(11)
    res = torch.randn(T, d, generator=g).to(torch.bfloat16)
    gamma = (1 + 0.1 * torch.randn(d, generator=g)).to(torch.bfloat16)
    G = c.gpu
    n1 = mk.mk_add_rmsnorm(G["x"], gamma.cuda(), res.cuda(), q8=True)
    o = mk.mk_moe_layer_q8(n1["q8"], n1["q8_scale"], G["gq"], G["gs"], G["dq"], G["ds"], k, x=n1["y"],
                           w_router=G["wr"], out=c.choices())
    n2 = mk.mk_add_rmsnorm(o["out"], gamma.cuda(), n1["residual"], out={"residual": n1["residual"]})
    # the layer from the norm's own outputs (each of which the norm's tests hold to its formula)
    c.x64 = ref.rows_values(n1["q8"].cpu(), n1["q8_scale"].cpu())
    c.check(o["out"], o["topk_ids"], o["topk_w"])
    h1 = (c.x.double() + res.double()).to(torch.bfloat16)
    want, bound = ref.layer(c.x64, c.gu64, c.dn64, o["topk_ids"].long().cpu(), o["topk_w"].cpu())
    h = h1.double() + want
    assert ((n2["residual"].cpu().double() - h).abs() <= bound + 2.0 ** -8 * (h.abs() + bound) + 2.0 ** -20).all()


def test_layer_agrees_with_the_dispatch_chain():
    """The dispatch with SwiGLU, the down-projection and the combine give the same layer with three more roundings
    (g, u and the expert outputs to bf16): within 2^-8 of each other per rounding, 4 x 2^-8 in the 2-norm."""
    c = Case(64, 1024, 16, 4, 16, 256)
    G = c.gpu
    o = c.call(out=c.choices())
    p = mk.mk_dispatch_gemm(G["x"], G["gu"], 4, w_router=G["wr"], swiglu=True)
    z = mk.mk_grouped_gemm(p["y_perm"], p["expert_offsets"], G["dn"])
    y = mk.mk_combine(z, p["slot_of"], p["topk_w"])
    assert torch.equal(o["topk_ids"], p["topk_ids"]) and torch.equal(o["topk_w"], p["topk_w"])
    a, b = o["out"].double(), y.double()
    assert (a - b).norm() <= 4 * 2.0 ** -8 * b.norm()


def test_layer_zero_tokens():
    c = Case(1, 256, 8, 2, 8, 16)
    G = c.gpu
    o = mk.mk_moe_layer(G["x"][:0], G["gu"], G["dn"], 2, w_router=G["wr"])
    assert o["out"].shape == (0, 256)


def test_layer_binding_refusals():
    c = Case(4, 256, 8, 2, 8, 16)
    G = c.gpu
    ids, gates = (v.cuda() for v in c.random_choices(7))
    ok = dict(x=G["x"], gu=G["gu"], dn=G["dn"], k=2, kw=dict(w_router=G["wr"]))

    def call(**ch):
        v = dict(ok, **ch)
        return mk.mk_moe_layer(v["x"], v["gu"], v["dn"], v["k"], **v["kw"])

    call()
    for ch in (dict(x=G["x"].float()), dict(x=G["x"].cpu()), dict(dn=G["dn"][:, :, :8]), dict(gu=G["gu"].half()),
               dict(kw=dict(w_router=G["wr"].t().contiguous().t())), dict(kw=dict(w_router=G["wr"].bfloat16())),
               dict(kw=dict(topk_ids_in=ids.long(), topk_w_in=gates, E=8)),
               dict(kw=dict(topk_ids_in=ids, topk_w_in=gates[:, :1], E=8)),
               dict(kw=dict(w_router=G["wr"], t_valid=torch.tensor([3], device="cuda"))),
               dict(kw=dict(w_router=G["wr"], out={"out": torch.empty(4, 256, device="cuda")}))):
        with pytest.raises(ValueError):
            call(**ch)
    for ch, st in ((dict(kw=dict(topk_ids_in=ids, E=8)), mk.MK_EINVAL), (dict(kw={}), mk.MK_EINVAL),
                   (dict(kw=dict(w_router=G["wr"], workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))),
                    mk.MK_EWORKSPACE)):
        with pytest.raises(mk.MkError) as err:
            call(**ch)
        assert err.value.status == st
    with pytest.raises(mk.MkError) as err:
        mk.mk_moe_layer(torch.zeros(129, 256, dtype=torch.bfloat16, device="cuda"), G["gu"], G["dn"], 2,
                        w_router=G["wr"])
    assert err.value.status == mk.MK_EUNSUPPORTED


@pytest.mark.parametrize("q8", [False, True])
def test_layer_error_is_one_rounding(q8):
    """The intermediate keeps more bits than the output: the layer's error is that of rounding the output to bf16 alone.
    Rounding moves a value by at most 2^-8 of it and, spread evenly over a binade's step, by 2^-8 / sqrt(3) in the mean
    square at worst (values just above a power of two); an intermediate of 8 bits would add as much again."""
    c = Case(64, 1024, 16, 4, 16, 512, q8)
    o = c.call(out=c.choices())
    want, _ = ref.layer(c.x64, c.gu64, c.dn64, o["topk_ids"].long().cpu(), o["topk_w"].cpu())
    got = o["out"].cpu().double()
    rounding = (want.to(torch.bfloat16).double() - want).norm()
    assert rounding <= 2.0 ** -8 / math.sqrt(3) * want.norm()
    # 65536 outputs: the two sums of squares of one rounding agree to a few in a thousand; the kept bits add at most
    # 2^-11 against 2^-9 of a step, 3% in the sum of squares
    assert (got - want).norm() <= 1.1 * rounding
