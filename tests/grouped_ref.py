"""Definitions of the experts' products backward and in 8-bit integers, in 64 bits on the CPU, and layouts to test on."""
import torch


def offsets_of(counts):
    return torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32)


def whole(g, *shape, most=4):
    """Small whole numbers in bf16: sums of their products are exact in fp32, so one rounding remains."""
    return torch.randint(-most, most + 1, shape, generator=g).to(torch.bfloat16)


def dgrad(dy, offsets, w):
    da = torch.zeros(dy.shape[0], w.shape[2], dtype=torch.float64)
    for e in range(w.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        da[lo:hi] = dy[lo:hi].double() @ w[e].double()
    return da


def wgrad(dy, a, offsets, row_token=None):
    E = offsets.shape[0] - 1
    if row_token is not None:
        ok = (row_token >= 0) & (row_token < a.shape[0])
        rows = torch.zeros(dy.shape[0], a.shape[1], dtype=torch.float64)
        rows[ok] = a[row_token[ok].long()].double()
    else:
        rows = a.double()
    dw = torch.zeros(E, dy.shape[1], a.shape[1], dtype=torch.float64)
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        dw[e] = dy[lo:hi].double().t() @ rows[lo:hi]
    return dw


def i8(a, a_scale, offsets, w, w_scale, row_token=None):
    """The rounding steps of mk_grouped_gemm_i8: the exact sum to fp32, times w_scale, times a_scale, to bf16."""
    rows = a.shape[0] if row_token is None else row_token.shape[0]
    t = torch.arange(rows) if row_token is None else row_token.long()
    ok = (t >= 0) & (t < a.shape[0])
    t = torch.where(ok, t, 0)
    codes = a[t].double() * ok[:, None]
    scale = torch.where(ok, a_scale[t], torch.zeros(()))
    y = torch.zeros(rows, w.shape[1], dtype=torch.bfloat16)
    for e in range(w.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        y[lo:hi] = ((codes[lo:hi] @ w[e].double().t()).float() * w_scale[e] * scale[lo:hi, None]).to(torch.bfloat16)
    return y


def layout(ids, e_begin, E_local):
    """Offsets, slots and rows' tokens by sorting (expert, position) pairs."""
    T, k = ids.shape
    pairs = sorted((int(ids[t, j]) - e_begin, t * k + j) for t in range(T) for j in range(k)
                   if 0 <= int(ids[t, j]) - e_begin < E_local)
    slot = torch.full((T * k,), -1, dtype=torch.int32)
    counts = [0] * E_local
    for r, (e, i) in enumerate(pairs):
        slot[i] = r
        counts[e] += 1
    return offsets_of(counts), slot.view(T, k), torch.tensor([i // k for _, i in pairs], dtype=torch.int32)
