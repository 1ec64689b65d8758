"""mk_quant_i8, mk_swiglu_i8 and mk_grouped_gemm_i8.

The product's sum is exact and its three roundings (to fp32, two scalings, to bf16) are the definition's, so it is
compared bit for bit; so are mk_quant_i8's codes (see there: the quotient of two bf16 values times 127 is a tie only where
it is one exactly) and scales (one fp32 division).  mk_swiglu_i8 evaluates e^-g and four more operations in fp32, below
2^-20 relative together, on a value and on its row's maximum: codes lie within 1/2 + 127 * 2^-19 of 127 h / max|h|."""
import numpy as np
import pytest
import torch

import grouped_ref as ref
import moe_dispatch_expert_amd as mk

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _codes(g, *shape):
    return torch.randint(-128, 128, shape, generator=g).to(torch.int8)


def _scales(g, *shape):
    return torch.rand(*shape, generator=g) * 0.01 + 0.001


SHAPES = [   # rows of each expert, K, N
    ([1], 16, 8),
    ([1], 4096, 512),
    ([0, 1, 0], 128, 64),
    ([3, 0, 5, 1], 144, 136),
    ([7, 8, 9, 15, 16, 17], 256, 72),
    ([31, 32, 33], 128, 64),
    ([63, 64, 65, 0], 512, 192),
    ([127, 128, 129], 528, 248),
    ([255, 0, 256, 257], 1024, 328),
    ([0, 0, 0], 256, 256),
    ([700], 1008, 1032),
    ([513, 2, 190], 1408, 704),
    ([1, 2, 3, 4, 5, 6, 7, 8, 9, 10] * 6, 320, 56),
    ([20, 1100], 2048, 136),
    ([40] * 16, 48, 1024),
    ([6], 14336, 520),
    ([300], 112, 2056),
]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,K,N", SHAPES, ids=lambda v: "x".join(map(str, v[:6])) if isinstance(v, list) else None)
def test_product_bit_for_bit(counts, K, N, gather):
    g = torch.Generator().manual_seed(K + 7 * N)
    R, E, extra = sum(counts), len(counts), 4
    off = ref.offsets_of(counts)
    T = max(2, R // 2) if gather else R + extra
    a, s = _codes(g, T, K), _scales(g, T)
    rt = torch.randint(0, T, (R + extra,), generator=g, dtype=torch.int32) if gather else None
    w, ws = _codes(g, E, N, K), _scales(g, E, N)
    out = torch.full((R + extra, N), 3.0, dtype=BF, device="cuda")
    got = mk.mk_grouped_gemm_i8(a.cuda(), s.cuda(), off.cuda(), w.cuda(), ws.cuda(),
                                row_token=None if rt is None else rt.cuda(), out=out)
    want = ref.i8(a, s, off, w, ws, rt)
    assert torch.equal(got[:R].cpu(), want[:R])
    assert (got[R:] == 3.0).all()


def test_largest_sums():
    """131056 products of -128 and -128 fill 31 bits."""
    K = 131056
    a, w = torch.full((3, K), -128, dtype=torch.int8), torch.full((1, 16, K), -128, dtype=torch.int8)
    w[0, 1] = 127
    s, ws, off = torch.ones(3), torch.ones(1, 16), torch.tensor([0, 3], dtype=torch.int32)
    got = mk.mk_grouped_gemm_i8(a.cuda(), s.cuda(), off.cuda(), w.cuda(), ws.cuda())
    assert torch.equal(got.cpu(), ref.i8(a, s, off, w, ws))


def test_rows_have_the_same_bits_in_any_batch():
    g = torch.Generator().manual_seed(3)
    K, N = 1040, 264
    a, s, w, ws = _codes(g, 600, K), _scales(g, 600), _codes(g, 2, N, K), _scales(g, 2, N)
    d = [t.cuda() for t in (a, s, w, ws)]
    whole = mk.mk_grouped_gemm_i8(d[0], d[1], torch.tensor([0, 300, 600], dtype=torch.int32, device="cuda"), d[2], d[3])
    for r0, r1 in ((0, 1), (10, 40), (299, 300), (300, 370)):
        e = r0 // 300
        off = torch.tensor([0, r1 - r0, r1 - r0] if e == 0 else [0, 0, r1 - r0], dtype=torch.int32, device="cuda")
        part = mk.mk_grouped_gemm_i8(d[0][r0:r1], d[1][r0:r1].clone(), off, d[2], d[3])   # (16-byte aligned)
        assert torch.equal(part, whole[r0:r1])


def test_foreign_tokens_give_zeros_and_offsets_past_the_rows_are_cut():
    g = torch.Generator().manual_seed(4)
    a, s, w, ws = _codes(g, 9, 64), _scales(g, 9), _codes(g, 3, 72, 64), _scales(g, 3, 72)
    rt = torch.randint(-3, 12, (50,), generator=g, dtype=torch.int32)
    rt[0], rt[1], rt[2] = -2 ** 31, 2 ** 31 - 1, 9
    off, cut = torch.tensor([0, 20, 60, 90], dtype=torch.int32), torch.tensor([0, 20, 50, 50], dtype=torch.int32)
    got = mk.mk_grouped_gemm_i8(a.cuda(), s.cuda(), off.cuda(), w.cuda(), ws.cuda(), row_token=rt.cuda())
    assert torch.equal(got.cpu(), ref.i8(a, s, cut, w, ws, rt))
    assert mk.mk_grouped_gemm_i8(a[:0].cuda(), s[:0].cuda(), off.cuda(), w.cuda(), ws.cuda()).shape == (0, 72)
    got = mk.mk_grouped_gemm_i8(a[:0].cuda(), s[:0].cuda(), off.cuda(), w.cuda(), ws.cuda(), row_token=rt.cuda())
    assert (got == 0).all()


def test_scales_that_are_not_finite_stay_in_their_rows_and_columns():
    g = torch.Generator().manual_seed(5)
    a, s, w, ws = _codes(g, 40, 128), _scales(g, 40), _codes(g, 1, 64, 128), _scales(g, 1, 64)
    off = torch.tensor([0, 40], dtype=torch.int32)
    want = ref.i8(a, s, off, w, ws)
    s[7], s[39], ws[0, 5] = float("nan"), float("inf"), float("nan")
    got = mk.mk_grouped_gemm_i8(a.cuda(), s.cuda(), off.cuda(), w.cuda(), ws.cuda()).cpu()
    ok = torch.ones(40, 64, dtype=torch.bool)
    ok[7], ok[39], ok[:, 5] = False, False, False
    assert torch.equal(got[ok], want[ok]) and got[7].isnan().all() and got[:, 5].isnan().all()


def test_many_experts():
    g = torch.Generator().manual_seed(6)
    E, K, N = 1024, 32, 24
    counts = [int(c) for c in torch.randint(0, 3, (E,), generator=g)]
    counts[17], counts[1023] = 600, 130
    off, R = ref.offsets_of(counts), sum(counts)
    a, s, w, ws = _codes(g, R, K), _scales(g, R), _codes(g, E, N, K), _scales(g, E, N)
    got = mk.mk_grouped_gemm_i8(*(t.cuda() for t in (a, s, off, w, ws)))
    assert torch.equal(got.cpu(), ref.i8(a, s, off, w, ws))


def test_offsets_past_32_bits():
    """The last expert's matrix lies behind 5 GiB of others; the last expert's rows behind 4 GiB of other rows."""
    g = torch.Generator().manual_seed(7)
    E, K, N = 5, 65536, 20480
    w = torch.zeros(E, N, K, dtype=torch.int8, device="cuda")
    w[4] = _codes(g, N, 16).cuda().repeat(1, K // 16)
    a, s, ws = _codes(g, 70, 16).repeat(1, K // 16), _scales(g, 70), _scales(g, E, N)
    off = torch.tensor([0, 0, 0, 0, 0, 70], dtype=torch.int32)
    got = mk.mk_grouped_gemm_i8(a.cuda(), s.cuda(), off.cuda(), w, ws.cuda())
    dots = a[:, :16].double() @ w[4, :, :16].cpu().double().t() * (K // 16)
    assert torch.equal(got.cpu(), (dots.float() * ws[4] * s[:, None]).to(BF))
    del w
    N, R0 = 8, (1 << 32) // K + 50
    w, ws = _codes(g, 2, N, 16).repeat(1, 1, K // 16), _scales(g, 2, N)
    big = torch.zeros(R0 + 70, K, dtype=torch.int8, device="cuda")
    big[R0:] = a.cuda()
    s = _scales(g, R0 + 70)
    off = torch.tensor([0, R0, R0 + 70], dtype=torch.int32)
    got = mk.mk_grouped_gemm_i8(big, s.cuda(), off.cuda(), w.cuda(), ws.cuda())
    dots = a[:, :16].double() @ w[1, :, :16].double().t() * (K // 16)
    assert torch.equal(got[R0:].cpu(), (dots.float() * ws[1] * s[R0:, None]).to(BF)) and (got[:R0] == 0).all()


# ------------------------------------------------------------------------------------------------ rows of codes

WIDTHS = [(1, 8), (5, 64), (37, 2048), (3, 2056), (2, 4104), (9, 7168), (4, 8200), (3, 16384), (2, 16392), (2, 32768),
          (1000, 704)]


def _exact_codes(x):
    x = x.double()
    m = x.abs().amax(dim=1, keepdim=True)
    q = torch.from_numpy(np.rint((127.0 * x / torch.where(m > 0, m, 1.0)).numpy()))
    return q, m.flatten().float() / 127.0


@pytest.mark.parametrize("rows,d", WIDTHS)
def test_codes_are_those_of_real_numbers(rows, d):
    g = torch.Generator().manual_seed(rows + d)
    x = torch.randn(rows, d, generator=g).to(BF)
    x[0, 0] = 4.0
    x[0, 1:] = torch.randn(d - 1, generator=g).to(BF) * 0.25   # many ties at 63.5 below:
    x[0, d // 2:] = 2.0
    got = mk.mk_quant_i8(x.cuda())
    q, s = _exact_codes(x)
    assert torch.equal(got["q"].cpu().double(), q) and torch.equal(got["scale"].cpu(), s)


def test_codes_of_every_pair_of_significands():
    """Every bf16 significand against every maximum: all ties and near ties there are."""
    m = torch.arange(128, 256).float()
    x = torch.cat([torch.arange(0, 256), torch.arange(0, 256) * -0.5, torch.arange(128, 256) * 2.0 ** -9]).to(BF)
    rows = torch.where(x[None, :].float().abs() <= m[:, None], x[None, :].float(), 0.0)
    rows = torch.cat([m[:, None].expand(-1, 8), rows], dim=1).to(BF).contiguous()
    got = mk.mk_quant_i8(rows.cuda())
    q, s = _exact_codes(rows)
    assert torch.equal(got["q"].cpu().double(), q) and torch.equal(got["scale"].cpu(), s)


def test_rows_of_zeros_extremes_and_what_is_not_finite():
    d = 64
    x = torch.randn(9, d, generator=torch.Generator().manual_seed(1)).to(BF)
    x[1] = 0.0
    x[2, 5] = float("nan")
    x[3, 63] = float("-inf")
    x[4] *= 2.0 ** 125
    x[5] = 0.0
    x[5, 7] = -2.0 ** -133            # the smallest bf16
    x[6] *= 2.0 ** -110
    x[7] = 0.0
    x[7, 0], x[7, 1] = torch.finfo(BF).max, torch.finfo(BF).min
    got = mk.mk_quant_i8(x.cuda())
    q, s = got["q"].cpu(), got["scale"].cpu()
    fine = [0, 4, 6, 7, 8]
    wq, ws = _exact_codes(x[fine])
    assert torch.equal(q[fine].double(), wq) and torch.equal(s[fine], ws)
    assert (q[1] == 0).all() and s[1] == 0
    assert (q[2] == 0).all() and s[2].isnan() and (q[3] == 0).all() and s[3].isnan()
    assert q[5, 7] == -127 and (q[5] != 0).sum() == 1


@pytest.mark.parametrize("rows,F", WIDTHS)
def test_swiglu_codes(rows, F):
    g = torch.Generator().manual_seed(rows + 3 * F)
    gu = (2 * torch.randn(rows, 2 * F, generator=g)).to(BF)
    got = mk.mk_swiglu_i8(gu.cuda())
    a, u = gu[:, :F].double(), gu[:, F:].double()
    h = a * torch.sigmoid(a) * u
    m = h.abs().amax(dim=1)
    assert ((got["scale"].cpu().double() * 127 - m).abs() <= 2.0 ** -19 * m).all()
    assert ((got["q"].cpu().double() - 127 * h / m[:, None]).abs() <= 0.5 + 127 * 2.0 ** -19).all()
    assert (got["q"].cpu().abs().amax(dim=1) == 127).all()


@pytest.mark.parametrize("swiglu", [False, True])
def test_rows_behind_the_valid_ones_stay(swiglu):
    g = torch.Generator().manual_seed(2)
    x = torch.randn(20, 128, generator=g).to(BF).cuda()
    f = mk.mk_swiglu_i8 if swiglu else mk.mk_quant_i8
    full = f(x)
    counts = torch.tensor([0, 3, 20, -5, 100, 13], dtype=torch.int32, device="cuda")
    for i, n in enumerate((0, 3, 20, 0, 20, 13)):   # the word is 4-byte aligned
        out = {"q": torch.full_like(full["q"], 99), "scale": torch.full_like(full["scale"], -1.0)}
        f(x, rows_valid=counts[i:i + 1], out=out)
        assert torch.equal(out["q"][:n], full["q"][:n]) and torch.equal(out["scale"][:n], full["scale"][:n])
        assert (out["q"][n:] == 99).all() and (out["scale"][n:] == -1.0).all()
