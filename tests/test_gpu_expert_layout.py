"""mk_expert_layout against a sort of the choices, and against the dispatch's own layout."""
import pytest
import torch

import grouped_ref as ref
import moe_dispatch_expert_amd as mk

pytestmark = pytest.mark.gpu


def _check(ids, e_begin, E_local):
    T, k = ids.shape
    out = {"row_token": torch.full((T * k,), -7, dtype=torch.int32, device="cuda")}
    got = mk.mk_expert_layout(ids.cuda(), E_local, e_begin, out=out)
    off, slot, rt = ref.layout(ids, e_begin, E_local)
    R = len(rt)
    assert torch.equal(got["expert_offsets"].cpu(), off)
    assert torch.equal(got["slot_of"].cpu(), slot)
    assert torch.equal(got["row_token"][:R].cpu(), rt) and (got["row_token"][R:] == -7).all()


@pytest.mark.parametrize("T,k,E,e_begin,E_local", [
    (1, 1, 1, 0, 1), (1, 8, 256, 0, 256), (0, 2, 8, 0, 8), (63, 2, 8, 0, 8), (65, 3, 7, 2, 4), (128, 8, 256, 224, 32),
    (341, 3, 64, 0, 64), (342, 3, 64, 0, 64), (1024, 1, 1024, 0, 1024), (1025, 1, 1024, 5, 1000), (700, 32, 65, 0, 65),
    (5000, 6, 64, 0, 64), (20011, 7, 300, 100, 150), (70000, 4, 2, 0, 2),
])
def test_layout_matches_a_sort(T, k, E, e_begin, E_local):
    g = torch.Generator().manual_seed(T + k + E)
    _check(torch.randint(0, E, (T, k), generator=g, dtype=torch.int32), e_begin, E_local)   # repeated ids among them


def test_foreign_and_extreme_ids():
    g = torch.Generator().manual_seed(1)
    ids = torch.randint(-3, 12, (300, 5), generator=g, dtype=torch.int32)
    ids[0] = torch.tensor([-2 ** 31, 2 ** 31 - 1, 0, -1, 8], dtype=torch.int32)
    _check(ids, 0, 8)
    _check(ids, 3, 2)
    _check(torch.full((90, 4), -1, dtype=torch.int32), 0, 8)
    _check(torch.full((2000, 4), 5, dtype=torch.int32), 0, 8)
    ids[1] = 2 ** 31 - 1
    _check(ids, 2 ** 31 - 2, 8)


def test_same_layout_as_the_dispatch():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(500, 128, generator=g).to(torch.bfloat16).cuda()
    w = torch.randn(20, 64, 128, generator=g).to(torch.bfloat16).cuda()
    wr = torch.randn(128, 40, generator=g).cuda()
    d = mk.mk_dispatch_gemm(x, w, 6, w_router=wr, E=40, e_begin=10)
    got = mk.mk_expert_layout(d["topk_ids"], 20, 10)
    R = int(d["expert_offsets"][-1])
    for name in ("expert_offsets", "slot_of"):
        assert torch.equal(got[name], d[name]), name
    assert torch.equal(got["row_token"][:R], d["row_token"][:R])


def test_many_choices():
    """More choices than the chunks' smallest size covers: 2^21 choices in 128 chunks of 16384."""
    g = torch.Generator().manual_seed(3)
    T, k, E = 1 << 18, 8, 200
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    got = mk.mk_expert_layout(ids.cuda(), 100, 50)
    e = ids.flatten().long() - 50
    e = torch.where((e >= 0) & (e < 100), e, 100)
    order = torch.sort(e, stable=True).indices
    counts = torch.bincount(e, minlength=101)[:100]
    R = int(counts.sum())
    slot = torch.full((T * k,), -1, dtype=torch.int32)
    slot[order[:R]] = torch.arange(R, dtype=torch.int32)
    assert torch.equal(got["expert_offsets"].cpu(), ref.offsets_of(counts.tolist()))
    assert torch.equal(got["slot_of"].cpu().flatten(), slot)
    assert torch.equal(got["row_token"][:R].cpu(), (order[:R] // k).to(torch.int32))
