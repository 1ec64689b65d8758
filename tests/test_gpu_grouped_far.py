"""Rows read in place from far inside a matrix of tokens, and outputs that are dropped while the call that writes them is queued."""
import pytest
import torch

import grouped_ref as ref
import moe_dispatch_expert_amd as mk

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _tokens(g, rows, T):
    """Tokens of the whole matrix, with the first and last ones and those around its middle."""
    rt = torch.randint(0, T, (rows,), generator=g, dtype=torch.int32)
    rt[:6] = torch.tensor([0, T - 1, T // 2 - 1, T // 2, T // 2 + 1, T - 2], dtype=torch.int32)
    return rt


@pytest.mark.parametrize("form", ["fp32", "bf16", "accumulate"])
def test_weights_gradient_of_tokens_past_2_gib(form):
    """As many bytes of tokens as the call takes (4 GiB less a row): offsets of the gather use all 32 bits."""
    g = torch.Generator().manual_seed(1)
    K, N = 8192, 72
    T = (2 ** 32 - 512) // (2 * K)
    a = torch.randint(-4, 5, (T, K), dtype=torch.int8, device="cuda").to(BF)
    assert a.nbytes > 2 ** 32 - 32768
    off, rt = ref.offsets_of([70, 0, 131]), _tokens(g, 201, T)
    dy = ref.whole(g, 201, N)
    rows = a[rt.cuda().long()]
    base = torch.full((3, N, K), 5.0, device="cuda") if form == "accumulate" else None
    got = mk.mk_grouped_gemm_wgrad(dy.cuda(), a, off.cuda(), row_token=rt.cuda(), out=base, accumulate=base is not None,
                                   dtype=BF if form == "bf16" else torch.float32)
    want = ref.wgrad(dy, rows.cpu(), off) + (5.0 if base is not None else 0.0)
    assert torch.equal(got.cpu(), want.to(got.dtype))


@pytest.mark.parametrize("counts", [[5, 0, 16], [300, 20, 263], [600]], ids=["stream", "tiles", "one_expert"])
def test_8_bit_product_of_tokens_past_2_gib(counts):
    g = torch.Generator().manual_seed(2)
    K, N, R, E = 65536, 40, sum(counts), len(counts)
    T = (2 ** 32 - 512) // K
    a = torch.randint(-128, 128, (T, K), dtype=torch.int8, device="cuda")
    s = torch.rand(T, generator=g) + 0.1
    w, ws = torch.randint(-128, 128, (E, N, K), generator=g).to(torch.int8), torch.rand(E, N, generator=g) + 0.1
    off, rt = ref.offsets_of(counts), _tokens(g, R, T)
    got = mk.mk_grouped_gemm_i8(a, s.cuda(), off.cuda(), w.cuda(), ws.cuda(), row_token=rt.cuda())
    assert torch.equal(got.cpu(), ref.i8(a[rt.cuda().long()].cpu(), s[rt.long()], off, w, ws))


def test_outputs_dropped_while_their_calls_are_queued():
    """Calls on a busy stream whose outputs nobody holds: copies are made on that stream, and what the current stream allocates and
    writes meanwhile stays as it is, though the calls run after that."""
    g = torch.Generator().manual_seed(3)
    side = torch.cuda.Stream()
    T, k, E, d, F = 250, 2, 6, 272, 136
    ids = torch.rand(T, E, generator=g).topk(k, 1).indices.to(torch.int32).cuda()
    gates = torch.rand(T, k, generator=g).cuda()
    dout, z = torch.randn(T, d, generator=g).to(BF).cuda(), torch.randn(T * k, d, generator=g).to(BF).cuda()
    gu, w = torch.randn(T * k, 2 * F, generator=g).to(BF).cuda(), torch.randn(E, d, F, generator=g).to(BF).cuda()
    q8 = torch.randint(-127, 128, (E, 64, d), generator=g).to(torch.int8).cuda()
    s8 = torch.rand(E, 64, generator=g).cuda()
    slow = torch.randn(4096, 4096, device="cuda")

    def chain(s):
        lay = mk.mk_expert_layout(ids, E, stream=s)
        off = lay["expert_offsets"]
        b = mk.mk_combine_backward(dout, z, lay["slot_of"], gates, stream=s)
        dh = mk.mk_grouped_gemm_dgrad(b["dy_perm"], off, w, stream=s)
        sb = mk.mk_swiglu_backward(gu, dh, h=True, stream=s)
        dw = mk.mk_grouped_gemm_wgrad(b["dy_perm"], sb["h"], off, stream=s)
        q = mk.mk_quant_i8(dout, stream=s)
        y = mk.mk_grouped_gemm_i8(q["q"], q["scale"], off, q8, s8, row_token=lay["row_token"], stream=s)
        h8 = mk.mk_swiglu_i8(gu, stream=s)
        return [lay["slot_of"], b["dtopk_w"], dh, sb["dgate_up"], dw, y, h8["q"], h8["scale"]]

    want = chain(None)
    kept = [[torch.empty_like(t) for t in want] for _ in range(8)]
    meanwhile = []
    torch.cuda.synchronize()
    for to in kept:
        with torch.cuda.stream(side):
            for _ in range(4):   # some milliseconds, so that all of the calls below are queued behind them
                slow @ slow
        outs = chain(side)
        with torch.cuda.stream(side):
            for a, b in zip(to, outs):
                a.copy_(b)
        sizes = [(t.numel() * t.element_size() + 3) // 4 for t in outs]
        del outs
        for n in sizes + [T * k * d // 2, 256]:
            meanwhile.append(torch.full((n,), 7.0, device="cuda"))
    torch.cuda.synchronize()
    assert all((t == 7.0).all() for t in meanwhile)
    for outs in kept:
        for x, y in zip(outs, want):
            assert torch.equal(x, y)
