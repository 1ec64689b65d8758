"""The experts' products in every tile form, at more tiles than there are workgroups, and several of them at once.

A form is chosen from the number of tiles and 256 workgroups, so each shape below says which it reaches.  Whole numbers and
8-bit codes have exact sums (see test_gpu_grouped_grad.py and test_gpu_grouped_i8.py), so outputs are compared bit for bit."""
import pytest
import torch

import grouped_ref as ref
import moe_dispatch_expert_amd as mk

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

# rows of each expert, contraction, columns of the output
ROWS = [
    ([700, 836] * 8, 136, 2120, "48 tall tiles: 256 wide, half a round of halves, the last 72 columns; short ones 128 wide"),
    ([700, 836] * 8, 200, 2296, "48 tall tiles of 9 x 256 columns, the last of them ragged, all whole"),
    ([256] * 70, 64, 1288, "70 tall tiles of 5 x 256 columns, the last 94 as halves, and 8 columns, no short ones"),
    ([256] * 40, 64, 1144, "40 tall tiles, all 128 wide"),
    ([300, 200] * 11, 264, 2760, "22 tall tiles of 11 x 256 columns, whole"),
    ([300, 200] * 12, 264, 2760, "24 tall tiles of 11 x 256 columns, the last 8 in eighths"),
    ([300, 200] * 12, 72, 2696, "24 tall tiles of 11 x 256 columns, the last 8 in eighths, of which some have no columns"),
    ([250] * 8, 328, 1240, "40 tall tiles in quarters"),
    ([300, 20] * 4, 520, 136, "4 tall tiles in eighths, a quarter of which have no columns; short ones 64 wide"),
    ([20] * 64, 80, 2040, "64 short tiles of at most 32 rows, 256 wide"),
    ([33, 20] * 32, 80, 2040, "64 short tiles of at most 128 rows, 256 wide"),
    ([25] * 44, 144, 2048, "44 short tiles of at most 32 rows, 128 wide"),
    ([100] * 44, 144, 2040, "44 short tiles of at most 128 rows, 128 wide"),
    ([20] * 30, 144, 72, "few short tiles of at most 32 rows: 64 wide"),
    ([128] * 30, 144, 72, "few short tiles of 128 rows: 64 wide"),
    ([513, 1] * 30, 16, 1032, "tall and short ones, less than a slab of contraction"),
]


def _id(v):
    return v.replace(" ", "_") if isinstance(v, str) else ""


@pytest.mark.parametrize("counts,L,C,what", ROWS, ids=_id)
def test_dgrad(counts, L, C, what):
    g = torch.Generator().manual_seed(L + C)
    R, E, off = sum(counts), len(counts), ref.offsets_of(counts)
    dy, w = ref.whole(g, R, L), ref.whole(g, E, L, C)
    got = mk.mk_grouped_gemm_dgrad(dy.cuda(), off.cuda(), w.cuda())
    assert torch.equal(got.cpu(), ref.dgrad(dy, off, w).to(BF))


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,L,C,what", ROWS, ids=_id)
def test_i8(counts, L, C, what, gather):
    L = (L + 15) // 16 * 16
    g = torch.Generator().manual_seed(L + C)
    R, E, off = sum(counts), len(counts), ref.offsets_of(counts)
    T = 333 if gather else R
    a, s = torch.randint(-128, 128, (T, L), generator=g).to(torch.int8), torch.rand(T, generator=g) + 0.1
    w, ws = torch.randint(-128, 128, (E, C, L), generator=g).to(torch.int8), torch.rand(E, C, generator=g) + 0.1
    rt = torch.randint(-4, T + 4, (R,), generator=g, dtype=torch.int32) if gather else None
    got = mk.mk_grouped_gemm_i8(a.cuda(), s.cuda(), off.cuda(), w.cuda(), ws.cuda(),
                                row_token=None if rt is None else rt.cuda())
    assert torch.equal(got.cpu(), ref.i8(a, s, off, w, ws, rt))


# rows of each expert, K, N, around where the stream of the weights for few rows begins and ends (at most 512 rows, 16 to an
# expert that has any), its widths, and a contraction that leaves some of its waves nothing
FEW = [
    ([16] * 32, 272, 1032, "512 rows"),
    ([16] * 31 + [17], 272, 1032, "513 rows"),
    ([16], 2064, 8192, "16 rows of an expert, 32 columns a task"),
    ([16], 2064, 8200, "16 rows of an expert, 16 columns a task"),
    ([17], 2064, 520, "17 rows of an expert"),
    ([31, 1], 1040, 520, "16 rows an expert on the mean"),
    ([512], 128, 72, "512 rows of one expert"),
    ([60, 0, 1, 1, 1], 176, 264, "more rows of one expert than a pass takes"),
    ([1] * 512, 64, 40, "512 experts of a row"),
    ([0, 2, 0] * 20, 16, 16, "one piece of contraction"),
    ([5, 3], 1008, 24, "waves with less than a slab"),
    ([9, 1, 2], 16400, 8, "a long contraction, 8 columns"),
]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,K,N,what", FEW, ids=_id)
def test_i8_of_few_rows(counts, K, N, what, gather):
    test_i8(counts, K, N, what, gather)


# rows of each expert, K, N: tasks of full and half tiles in several rounds, from both ends
GRADIENTS = [
    ([3, 90, 0, 131] * 10, 520, 1400, "720 tasks of 40 experts, a sixth of them half tiles"),
    ([64, 33, 65, 0, 1], 520, 1000, "120 tasks, all of half tiles"),
    ([300, 70, 5], 264, 2600, "126 tasks, all of half tiles"),
    ([64, 33, 65, 1] * 16, 264, 1280, "640 tasks, full tiles only"),
    ([40, 0, 7] * 100, 776, 128, "1200 tasks of half tiles only"),
    ([2000, 5, 700, 1] * 4, 1032, 1160, "400 tasks of very different lengths"),
]


@pytest.mark.parametrize("form", ["fp32", "bf16", "accumulate", "gather", "gather_accumulate"])
@pytest.mark.parametrize("counts,K,N,what", GRADIENTS, ids=_id)
def test_wgrad(counts, K, N, what, form):
    g = torch.Generator().manual_seed(K + N)
    R, E, off = sum(counts), len(counts), ref.offsets_of(counts)
    T = 77 if form.startswith("gather") else R
    dy, a = ref.whole(g, R, N), ref.whole(g, T, K)
    rt = torch.randint(-2, T + 2, (R,), generator=g, dtype=torch.int32) if form.startswith("gather") else None
    want, out, dtype = ref.wgrad(dy, a, off, rt), None, BF if form == "bf16" else torch.float32
    if form.endswith("accumulate"):
        base = torch.randint(-1000, 1000, (E, N, K), generator=g).float()
        want, out = want + base.double(), base.cuda()
    got = mk.mk_grouped_gemm_wgrad(dy.cuda(), a.cuda(), off.cuda(), row_token=None if rt is None else rt.cuda(),
                                   dtype=dtype, out=out, accumulate=out is not None)
    assert torch.equal(got.cpu(), want.to(dtype))


def test_offsets_past_the_last_one_are_cut_to_it():
    """Offsets that go back at the end: what lies past the last one belongs to nobody, however few rows are left."""
    g = torch.Generator().manual_seed(1)
    given, cut = torch.tensor([0, 2000, 900, 10], dtype=torch.int32), torch.tensor([0, 10, 10, 10], dtype=torch.int32)
    dy, a, w = ref.whole(g, 2000, 72), ref.whole(g, 2000, 48), ref.whole(g, 3, 72, 48)
    out = torch.full((2000, 48), 7.0, dtype=BF, device="cuda")
    mk.mk_grouped_gemm_dgrad(dy.cuda(), given.cuda(), w.cuda(), out=out)
    assert torch.equal(out[:10].cpu(), ref.dgrad(dy, cut, w)[:10].to(BF)) and (out[10:] == 7.0).all()
    got = mk.mk_grouped_gemm_wgrad(dy.cuda(), a.cuda(), given.cuda())
    assert torch.equal(got.cpu(), ref.wgrad(dy, a, cut).float())
    codes, s = torch.randint(-128, 128, (2000, 48), generator=g).to(torch.int8), torch.rand(2000, generator=g)
    w, ws = torch.randint(-128, 128, (3, 40, 48), generator=g).to(torch.int8), torch.rand(3, 40, generator=g)
    for rt in (None, torch.randint(0, 2000, (2000,), generator=g, dtype=torch.int32)):
        out = torch.full((2000, 40), 7.0, dtype=BF, device="cuda")
        mk.mk_grouped_gemm_i8(codes.cuda(), s.cuda(), given.cuda(), w.cuda(), ws.cuda(),
                              row_token=None if rt is None else rt.cuda(), out=out)
        assert torch.equal(out[:10].cpu(), ref.i8(codes, s, cut, w, ws, rt)[:10]) and (out[10:] == 7.0).all()


def test_no_tokens_to_read():
    """Rows that would read tokens, of which there are none: zeros, or nothing added."""
    off, rt = torch.tensor([0, 40, 300], dtype=torch.int32).cuda(), torch.zeros(300, dtype=torch.int32).cuda()
    dy, none = torch.ones(300, 136, dtype=BF, device="cuda"), torch.empty(0, 264, dtype=BF, device="cuda")
    assert (mk.mk_grouped_gemm_wgrad(dy, none, off, row_token=rt) == 0).all()
    out = torch.full((2, 136, 264), 3.0, device="cuda")
    mk.mk_grouped_gemm_wgrad(dy, none, off, row_token=rt, out=out, accumulate=True)
    assert (out == 3.0).all()


def test_a_row_of_dgrad_has_the_same_bits_in_any_batch():
    g = torch.Generator().manual_seed(2)
    dy, w = torch.randn(1600, 520, generator=g).to(BF).cuda(), torch.randn(2, 520, 264, generator=g).to(BF).cuda()
    whole = mk.mk_grouped_gemm_dgrad(dy, torch.tensor([0, 800, 1600], dtype=torch.int32, device="cuda"), w)
    for r0, r1 in ((0, 1), (10, 50), (790, 800), (800, 940), (1000, 1600)):
        off = torch.tensor([0, r1 - r0, r1 - r0] if r0 < 800 else [0, 0, r1 - r0], dtype=torch.int32, device="cuda")
        assert torch.equal(mk.mk_grouped_gemm_dgrad(dy[r0:r1], off, w), whole[r0:r1])


def _i8_ffn(x, ids, gates, w1, s1, w2, s2, **kw):
    E, F = w1.shape[0], w2.shape[2]
    lay = mk.mk_expert_layout(ids, E, **kw)
    off, rt = lay["expert_offsets"], lay["row_token"]
    x8 = mk.mk_quant_i8(x, **kw)
    gu = mk.mk_grouped_gemm_i8(x8["q"], x8["scale"], off, w1, s1, row_token=rt, **kw)
    h8 = mk.mk_swiglu_i8(gu, rows_valid=off[E:], **kw)
    z = mk.mk_grouped_gemm_i8(h8["q"], h8["scale"], off, w2, s2, **kw)
    return {**lay, "xq": x8["q"], "xs": x8["scale"], "gu": gu, "hq": h8["q"], "hs": h8["scale"], "z": z,
            "out": mk.mk_combine(z, lay["slot_of"], gates, **kw)}


def _i8_layer(g, T, d, E, k, F):
    x, gates = torch.randn(T, d, generator=g).to(BF), torch.rand(T, k, generator=g)
    ids = torch.rand(T, E + 3, generator=g).topk(k, 1).indices.to(torch.int32)   # some of them not local
    w1, w2 = (torch.randint(-127, 128, s, generator=g).to(torch.int8) for s in ((E, 2 * F, d), (E, d, F)))
    s1, s2 = torch.rand(E, 2 * F, generator=g) * 2e-3 + 1e-4, torch.rand(E, d, generator=g) * 2e-3 + 1e-4
    return x, ids, gates, w1, s1, w2, s2


@pytest.mark.parametrize("T,d,E,k,F", [(1, 256, 8, 2, 272), (40, 128, 16, 4, 176), (700, 256, 6, 3, 400)])
def test_8_bit_ffn(T, d, E, k, F):
    """The 8-bit expert FFN as it is used, each step against its definition on what the step before gave; the whole within
    the errors of two 8-bit roundings of an unrounded FFN with the same weights."""
    args = _i8_layer(torch.Generator().manual_seed(T), T, d, E, k, F)
    x, ids, gates, w1, s1, w2, s2 = args
    got = {n: t.cpu() for n, t in _i8_ffn(*(t.cuda() for t in args)).items()}
    off, slot, token = ref.layout(ids, 0, E)
    R = int(off[-1])
    assert torch.equal(got["expert_offsets"], off) and torch.equal(got["slot_of"], slot)
    assert torch.equal(got["row_token"][:R], token)
    m = x.double().abs().amax(1)
    assert torch.equal(got["xq"].double(), torch.round(127 * x.double() / m[:, None])) and torch.equal(got["xs"], m.float() / 127)
    assert torch.equal(got["gu"][:R], ref.i8(got["xq"], got["xs"], off, w1, s1, token))
    a, u = got["gu"][:R, :F].double(), got["gu"][:R, F:].double()
    h = a * torch.sigmoid(a) * u
    hm = h.abs().amax(1)
    assert ((got["hq"][:R].double() - 127 * h / hm[:, None]).abs() <= 0.5 + 127 * 2.0 ** -19).all()
    assert torch.equal(got["z"][:R], ref.i8(got["hq"][:R], got["hs"][:R], off, w2, s2))
    want, size = torch.zeros(T, d, dtype=torch.float64), torch.zeros(T, d, dtype=torch.float64)
    whole = torch.zeros(T, d, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            if slot[t, j] >= 0:
                z = got["z"][slot[t, j]].double() * gates[t, j].double()
                want[t] += z
                size[t] += z.abs()
                e = int(ids[t, j])
                v = w1[e].double() @ x[t].double() * s1[e]
                whole[t] += gates[t, j].double() * (w2[e].double() @ (torch.nn.functional.silu(v[:F]) * v[F:]) * s2[e])
    # at most k additions and products in fp32, one rounding to bf16
    assert ((got["out"].double() - want).abs() <= 2 * k * 2.0 ** -24 * size + 2.0 ** -8 * want.abs()).all()
    # Codes are off by at most half a step, max / 254, so an input's error is within sqrt(d) max / (254 |x|) of it in norm:
    # below 4.2 / 254 for normal values of this width, and at most 8 / 254 for products of two; x acts through both halves
    # of the gate, with a slope of at most 1.1 each.
    assert (got["out"].double() - whole).norm() <= (2.2 * 4.2 + 8) / 254 * whole.norm()


def test_two_streams_at_once():
    """The same operators on two streams with inputs of their own, while each other's calls are on their way."""
    g = torch.Generator().manual_seed(3)
    layers = [[t.cuda() for t in _i8_layer(g, T, 256, 8, 2, 304)] for T in (300, 37)]
    grads = []
    for counts in ([700, 20, 0, 90] * 4, [33] * 40):
        R = sum(counts)
        grads.append([t.cuda() for t in (ref.whole(g, R, 520), ref.whole(g, R, 264), ref.whole(g, len(counts), 520, 264),
                                         ref.offsets_of(counts))])

    def run(i, s=None):
        dy, a, w, off = grads[i]
        o = _i8_ffn(*layers[i], stream=s)
        return [o["out"], o["expert_offsets"], mk.mk_grouped_gemm_dgrad(dy, off, w, stream=s),
                mk.mk_grouped_gemm_wgrad(dy, a, off, stream=s), mk.mk_grouped_gemm_wgrad(dy, a, off, dtype=BF, stream=s)]

    want = [run(0), run(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[run(i, streams[i]) for i in (0, 1)] for _ in range(12)]
    torch.cuda.synchronize()
    for pair in got:
        for outs, ws in zip(pair, want):
            for o, w in zip(outs, ws):
                assert torch.equal(o, w)


def test_captured_accumulation():
    """A graph that adds a weights' gradient and runs the 8-bit FFN, replayed on other rows and another number of them."""
    g = torch.Generator().manual_seed(4)
    E, N, K = 12, 264, 136
    counts = [[30, 0, 200, 5, 1, 0, 17, 300, 2, 2, 2, 41], [0] * 11 + [600], [50] * 12]
    dy, a = ref.whole(g, 600, N).cuda(), ref.whole(g, 600, K).cuda()
    off = ref.offsets_of(counts[0]).cuda()
    out, want = torch.zeros(E, N, K, device="cuda"), torch.zeros(E, N, K, device="cuda")
    layer = [t.cuda() for t in _i8_layer(g, 30, 128, 8, 2, 144)]

    def step(into):
        mk.mk_grouped_gemm_wgrad(dy, a, off, out=into, accumulate=True)
        return _i8_ffn(*layer)["out"]

    step(out)
    torch.cuda.synchronize()
    out.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(out)
    for i in range(5):
        off.copy_(ref.offsets_of(counts[i % 3]))
        dy.copy_(ref.whole(g, 600, N))
        layer[0].copy_(torch.randn(30, 128, generator=g).to(BF))
        layer[1].copy_(torch.rand(30, 11, generator=g).topk(2, 1).indices.to(torch.int32))
        graph.replay()
        assert torch.equal(y, step(want)), i
        assert torch.equal(out, want), i
        torch.cuda.synchronize()
