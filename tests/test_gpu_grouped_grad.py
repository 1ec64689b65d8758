"""mk_grouped_gemm_dgrad and mk_grouped_gemm_wgrad against their sums in 64 bits.

On whole numbers of at most 4 in size, with at most 2^20 terms, every partial sum is exact in fp32, so the outputs are the
exact sums rounded once: compared bit for bit.  On other values (products of bf16 are exact in fp32): a matrix
instruction adds at most 32 products to its accumulator and L / 16 of them follow one another, each addition off by at most
2^-23 of what it holds, so a sum is within (L / 16 + 34) 2^-23 sum |terms| of the exact one, and a bf16 output rounds by
2^-8 of its value at most."""
import pytest
import torch

import grouped_ref as ref
import moe_dispatch_expert_amd as mk

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

# rows of each expert, K, N: tile edges on either side, empty experts, single rows, sizes that are odd multiples of 8
SHAPES = [
    ([1], 8, 8),
    ([0, 1, 0], 64, 64),
    ([3, 0, 5, 1], 72, 136),
    ([31, 32, 33], 128, 64),
    ([63, 64, 65, 0], 256, 192),
    ([127, 128, 129], 264, 248),
    ([255, 0, 256, 257], 512, 328),
    ([0, 0, 0, 0, 0], 256, 256),
    ([700], 1000, 1032),
    ([513, 2, 190], 704, 1408),
    ([1, 2, 3, 4, 5, 6, 7, 8, 9, 10] * 6, 320, 56),
    ([1100, 20], 136, 2048),
    ([40] * 16, 2048, 24),
    ([2, 0, 300, 0, 1], 16, 4096),
]


def _id(v):
    return "x".join(map(str, v)) if isinstance(v, list) and len(v) < 6 else None


@pytest.mark.parametrize("counts,K,N", SHAPES, ids=_id)
def test_dgrad_is_exact_on_whole_numbers(counts, K, N):
    g = torch.Generator().manual_seed(K + N)
    R, E = sum(counts), len(counts)
    extra = 5   # rows behind the last expert's
    dy, w = ref.whole(g, R + extra, N), ref.whole(g, E, N, K)
    dy[R:] = float("nan")
    off = ref.offsets_of(counts)
    out = torch.full((R + extra, K), 7.0, dtype=BF, device="cuda")
    got = mk.mk_grouped_gemm_dgrad(dy.cuda(), off.cuda(), w.cuda(), out=out)
    assert got is out
    assert torch.equal(got[:R].cpu(), ref.dgrad(dy, off, w)[:R].to(BF))
    assert (got[R:] == 7.0).all()


@pytest.mark.parametrize("counts,K,N", SHAPES, ids=_id)
@pytest.mark.parametrize("form", ["fp32", "bf16", "accumulate", "gather", "gather_accumulate"])
def test_wgrad_is_exact_on_whole_numbers(counts, K, N, form):
    g = torch.Generator().manual_seed(K * 3 + N)
    R, E = sum(counts), len(counts)
    extra = 3
    off = ref.offsets_of(counts)
    dy = ref.whole(g, R + extra, N)
    dy[R:] = float("nan")
    rt = None
    if form.startswith("gather"):
        T = max(2, R // 2)
        a = ref.whole(g, T, K)
        rt = torch.randint(0, T, (R + extra,), generator=g, dtype=torch.int32)
        rt[R:] = 2 ** 30
    else:
        a = ref.whole(g, R + extra, K)
        a[R:] = float("inf")
    want = ref.wgrad(dy, a, off, rt)
    out, dtype = None, torch.bfloat16 if form == "bf16" else torch.float32
    if form.endswith("accumulate"):
        base = torch.randint(-1000, 1000, (E, N, K), generator=g).float()
        want, out = want + base.double(), base.cuda()
    got = mk.mk_grouped_gemm_wgrad(dy.cuda(), a.cuda(), off.cuda(), row_token=None if rt is None else rt.cuda(),
                                   dtype=dtype, out=out, accumulate=out is not None)
    assert torch.equal(got.cpu(), want.to(dtype))


@pytest.mark.parametrize("counts,K,N", [([200, 3, 77], 264, 520), ([1024, 0, 300], 512, 1408), ([90] * 5, 136, 72)])
def test_sums_of_random_values(counts, K, N):
    g = torch.Generator().manual_seed(11)
    R, E = sum(counts), len(counts)
    off = ref.offsets_of(counts)
    dy, a = torch.randn(R, N, generator=g).to(BF), torch.randn(R, K, generator=g).to(BF)
    w = torch.randn(E, N, K, generator=g).to(BF)
    d = [t.cuda() for t in (dy, a, w, off)]

    def check(got, want, size, L, half):
        tol = (L / 16 + 34) * 2.0 ** -23 * size + half * want.abs()
        assert ((got.cpu().double() - want).abs() <= tol).all()

    check(mk.mk_grouped_gemm_dgrad(d[0], d[3], d[2]), ref.dgrad(dy, off, w), ref.dgrad(dy.abs(), off, w.abs()), N,
          2.0 ** -8)
    want, size = ref.wgrad(dy, a, off), ref.wgrad(dy.abs(), a.abs(), off)
    check(mk.mk_grouped_gemm_wgrad(d[0], d[1], d[3]), want, size, max(counts), 0.0)
    check(mk.mk_grouped_gemm_wgrad(d[0], d[1], d[3], dtype=BF), want, size, max(counts), 2.0 ** -8)
    base = torch.randn(E, N, K, generator=g)
    got = mk.mk_grouped_gemm_wgrad(d[0], d[1], d[3], out=base.cuda(), accumulate=True)
    check(got, want + base.double(), size + base.abs().double(), max(counts), 2.0 ** -24)


def test_gradients_are_those_of_the_product():
    """<c, y(a + h da, W + h dW) - y(a - h da, W - h dW)> / 2h of the sum's definition in 64 bits against the kernels'
    gradients along (da, dW), within their roundings."""
    g = torch.Generator().manual_seed(5)
    counts, K, N = [40, 0, 25], 128, 96
    R, E, off = sum(counts), len(counts), ref.offsets_of(counts)
    a, w, c = (torch.randn(*s, generator=g).to(BF) for s in ((R, K), (E, N, K), (R, N)))
    da, dw = torch.randn(R, K, generator=g).double(), torch.randn(E, N, K, generator=g).double()

    def y(a, w):
        return torch.cat([a[off[e]:off[e + 1]] @ w[e].t() for e in range(E)])

    h = 2.0 ** -10
    diff = (c.double() * (y(a.double() + h * da, w.double() + h * dw) - y(a.double() - h * da, w.double() - h * dw))
            ).sum() / (2 * h)
    ga = mk.mk_grouped_gemm_dgrad(c.cuda(), off.cuda(), w.cuda()).cpu().double()
    gw = mk.mk_grouped_gemm_wgrad(c.cuda(), a.cuda(), off.cuda(), dtype=BF).cpu().double()
    got = (ga * da).sum() + (gw * dw).sum()
    # the product is bilinear, so the difference is exact; each gradient rounds by 2^-8 and its fp32 sums by 2^-16 more
    tol = (2.0 ** -8 + 2.0 ** -16) * ((ga * da).abs().sum() + (gw * dw).abs().sum())
    assert abs(got - diff) <= tol


def test_infinities_and_nan_stay_in_their_rows():
    """A row of dy with a NaN or an infinity reaches its own row of da, and its expert's dW, alone."""
    g = torch.Generator().manual_seed(6)
    counts, K, N = [70, 41, 30], 136, 200   # N: a ragged last slab, whose tail lies in the next row
    off = ref.offsets_of(counts)
    dy, a, w = ref.whole(g, 141, N), ref.whole(g, 141, K), ref.whole(g, 3, N, K)
    bad = dy.clone()
    bad[70, 0], bad[110, N - 1] = float("nan"), float("inf")   # first and last row of expert 1
    got, want = (mk.mk_grouped_gemm_dgrad(t.cuda(), off.cuda(), w.cuda()).cpu() for t in (bad, dy))
    rows = torch.ones(141, dtype=torch.bool)
    rows[[70, 110]] = False
    assert torch.equal(got[rows], want[rows]) and not got[~rows].isfinite().any()
    bad_a = a.clone()
    bad_a[69, K - 1], bad_a[111, 0] = float("nan"), float("inf")   # the rows on either side of expert 1
    got, want = (mk.mk_grouped_gemm_wgrad(dy.cuda(), t.cuda(), off.cuda()).cpu() for t in (bad_a, a))
    assert torch.equal(got[1], want[1])
    assert torch.equal(got[0][:, :K - 1], want[0][:, :K - 1]) and torch.equal(got[2][:, 1:], want[2][:, 1:])


def test_offsets_past_the_rows_are_cut_and_foreign_tokens_read_zeros():
    g = torch.Generator().manual_seed(7)
    K, N = 64, 72
    dy, a, w = ref.whole(g, 50, N), ref.whole(g, 50, K), ref.whole(g, 3, N, K)
    off, cut = torch.tensor([0, 20, 60, 90], dtype=torch.int32), torch.tensor([0, 20, 50, 50], dtype=torch.int32)
    assert torch.equal(mk.mk_grouped_gemm_dgrad(dy.cuda(), off.cuda(), w.cuda()).cpu(), ref.dgrad(dy, cut, w).to(BF))
    rt = torch.randint(-20, 70, (50,), generator=g, dtype=torch.int32)
    rt[0], rt[1], rt[2] = -2 ** 31, 2 ** 31 - 1, 50
    got = mk.mk_grouped_gemm_wgrad(dy.cuda(), a.cuda(), off.cuda(), row_token=rt.cuda())
    assert torch.equal(got.cpu(), ref.wgrad(dy, a, cut, rt).float())


def test_no_rows():
    w = torch.zeros(3, 64, 32, dtype=BF, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    none = torch.zeros(0, 64, dtype=BF, device="cuda"), torch.zeros(0, 32, dtype=BF, device="cuda")
    assert mk.mk_grouped_gemm_dgrad(none[0], off, w).shape == (0, 32)
    out = torch.full((3, 64, 32), 5.0, device="cuda")
    mk.mk_grouped_gemm_wgrad(*none, off, out=out, accumulate=True)
    assert (out == 5.0).all()
    mk.mk_grouped_gemm_wgrad(*none, off, out=out)
    assert (out == 0.0).all()


def test_many_experts():
    """As many experts as there may be, most of them with nothing, and rows with a row offset past 2^31 bytes."""
    g = torch.Generator().manual_seed(8)
    E, K, N = 1024, 16, 24
    counts = [int(c) for c in torch.randint(0, 3, (E,), generator=g)]
    counts[17], counts[1023] = 600, 130
    off, R = ref.offsets_of(counts), sum(counts)
    dy, a, w = ref.whole(g, R, N), ref.whole(g, R, K), ref.whole(g, E, N, K)
    d = [t.cuda() for t in (dy, a, off, w)]
    assert torch.equal(mk.mk_grouped_gemm_dgrad(d[0], d[2], d[3]).cpu(), ref.dgrad(dy, off, w).to(BF))
    assert torch.equal(mk.mk_grouped_gemm_wgrad(d[0], d[1], d[2]).cpu(), ref.wgrad(dy, a, off).float())


def test_offsets_past_32_bits():
    """The last expert's rows lie behind 4 GiB of other rows, its matrix behind 4 GiB of other matrices."""
    K, N = 8192, 8
    R0 = (1 << 32) // (2 * K) + 100        # rows of K before them
    g = torch.Generator().manual_seed(9)
    dy = torch.zeros(R0 + 40, N, dtype=BF, device="cuda")
    a = torch.zeros(R0 + 40, K, dtype=BF, device="cuda")
    dy[R0:], a[R0:] = ref.whole(g, 40, N).cuda(), ref.whole(g, 40, K).cuda()
    off = torch.tensor([0, R0, R0 + 40], dtype=torch.int32, device="cuda")
    got = mk.mk_grouped_gemm_wgrad(dy, a, off)
    want = ref.wgrad(dy[R0:].cpu(), a[R0:].cpu(), torch.tensor([0, 40]))
    assert torch.equal(got[1].cpu(), want[0].float()) and (got[0] == 0).all()
    w = ref.whole(g, 2, N, K)
    da = mk.mk_grouped_gemm_dgrad(dy, off, w.cuda())
    assert torch.equal(da[R0:].cpu(), ref.dgrad(dy[R0:].cpu(), torch.tensor([0, 40]), w[1:]).to(BF))
    del a, da
    n = 65536
    w = torch.zeros(5, n, K, dtype=BF, device="cuda")   # 1 GiB an expert
    w[4] = ref.whole(g, n, 8).cuda().repeat(1, K // 8)
    dy = ref.whole(g, 30, n)
    off = torch.tensor([0, 0, 0, 0, 0, 30], dtype=torch.int32)
    got = mk.mk_grouped_gemm_dgrad(dy.cuda(), off.cuda(), w)
    want = (dy.cuda().float() @ w[4, :, :8].float()).to(BF).repeat(1, K // 8)
    assert torch.equal(got, want)
