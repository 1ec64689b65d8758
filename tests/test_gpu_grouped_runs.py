"""The gathered 8-bit product where a workgroup goes through several tiles of one run, each with tokens of its own."""
import pytest
import torch

import grouped_ref as ref
import moe_dispatch_expert_amd as mk

pytestmark = pytest.mark.gpu


# rows of each expert, K, N: more than twice as many tiles of a form as a card has workgroups (256)
@pytest.mark.parametrize("counts,K,N", [
    ([256] * 70, 64, 2048),                     # 256 x 256
    ([256] * 80, 64, 1160),                     # 256 x 256, the last 136 columns too
    ([256] * 600, 48, 128),                     # 256 x 128
    ([100, 120] * 40, 64, 2048),                # 128 rows, short tiles
    ([20] * 300, 64, 1024),                     # 32 rows, short tiles
], ids=lambda v: None if not isinstance(v, list) else f"{len(v)}x{v[0]}")
def test_rows_read_in_place_are_those_of_their_tile(counts, K, N):
    """Against the same rows laid out one after the other, and some of them against the definition."""
    g = torch.Generator().manual_seed(K + N + len(counts))
    R, E, T, off = sum(counts), len(counts), 4099, ref.offsets_of(counts)
    a, s = torch.randint(-128, 128, (T, K), generator=g).to(torch.int8), torch.rand(T, generator=g) + 0.1
    w, ws = torch.randint(-128, 128, (E, N, K), generator=g).to(torch.int8), torch.rand(E, N, generator=g) + 0.1
    rt = torch.randint(0, T, (R,), generator=g, dtype=torch.int32)
    d = [t.cuda() for t in (a, s, off, w, ws, rt)]
    at = d[5].long()
    want = mk.mk_grouped_gemm_i8(d[0][at], d[1][at], *d[2:5])
    for _ in range(5):
        assert torch.equal(mk.mk_grouped_gemm_i8(*d[:5], row_token=d[5]), want)
    last = counts[-1]
    t = rt[R - last:]
    part = ref.i8(a[t.long()], s[t.long()], torch.tensor([0, last], dtype=torch.int32), w[E - 1:], ws[E - 1:])
    assert torch.equal(want[R - last:].cpu(), part)


# rows of the experts, K, N: where the stream of the weights for few rows ends, at uneven counts
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,K,N", [
    ([1, 0, 481] + [1] * 30, 272, 1408),        # the most rows of one expert: tiles
    ([1, 0, 100] + [1] * 30, 272, 2816),        # seven passes of one expert: the stream
    ([17] * 16 + [2] * 16, 144, 2816),          # two passes of many: tiles
    ([17] * 4 + [2] * 28, 144, 2816),           # of few: the stream
    ([64], 1040, 4088),                         # four passes of one expert's narrow tiles
    ([65], 1040, 4088),
    ([33, 1], 400, 4096),
    ([40] * 8, 400, 504),
], ids=lambda v: None if not isinstance(v, list) else f"{len(v)}x{max(v)}")
def test_uneven_counts_of_few_rows(counts, K, N, gather):
    g = torch.Generator().manual_seed(K + N + len(counts))
    R, E, off = sum(counts), len(counts), ref.offsets_of(counts)
    T = 77 if gather else R
    a, s = torch.randint(-128, 128, (T, K), generator=g).to(torch.int8), torch.rand(T, generator=g) + 0.1
    w, ws = torch.randint(-128, 128, (E, N, K), generator=g).to(torch.int8), torch.rand(E, N, generator=g) + 0.1
    rt = torch.randint(-4, T + 4, (R,), generator=g, dtype=torch.int32) if gather else None
    got = mk.mk_grouped_gemm_i8(*(t.cuda() for t in (a, s, off, w, ws)), row_token=None if rt is None else rt.cuda())
    assert torch.equal(got.cpu(), ref.i8(a, s, off, w, ws, rt))
