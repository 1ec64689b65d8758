"""The few-token MoE layer in fp64 on the CPU, with a bound that counts what the kernels keep of the intermediate
h = w silu(g) u, so that a lost second part of h shows in every shape.

u = 2^-24.  The fp32 sums as in layer_ref.py: p <= 40 + d / 32 additions on a path of the gate|up products and
p <= 40 + F / 32 + hits of the down products; |silu'| < 1.1, silu, the products with u and w: 2^-18 relative.
What is kept of h:
  bf16 weights  hi = bf16(h), |h - hi| <= 2^-8 |h|, and bf16(h - hi), which is off by at most 2^-8 of that: 2^-16 |h|.
  8-bit weights an fp16 of h scaled by a power of two of its 8 features, brought to that of the largest in a block of 128
                before the product: 2^-11 |h|, or half of fp16's smallest step where the block's largest is at least 2^14,
                twice (stored, and brought to the block's scale): 2 x 2^-25 / 2^14 = 2^-38 max|h| of the row.
and 2^-124 where the parts leave the formats' smallest values.  The output is rounded to bf16 once: 2^-8 |out|.
"""
import torch

U = 2.0 ** -24
BF16 = 2.0 ** -8


def layer(x, w_gu, w_dn, ids, gates, q8, e_begin=0):
    """(out, bound) of fp64 activations x [T, d] and weights [E_local, 2F, d], [E_local, d, F]; ids, gates [T, k]."""
    T, d = x.shape
    E_local, F2, _ = w_gu.shape
    F = F2 // 2
    out = torch.zeros(T, d, dtype=torch.float64)
    err = torch.zeros(T, d, dtype=torch.float64)
    mag = torch.zeros(T, d, dtype=torch.float64)
    p1 = 40 + d / 32
    hits = 0
    for e in range(E_local):
        w = (gates.double() * (ids == e + e_begin)).sum(dim=1)
        t = torch.nonzero((ids == e + e_begin).any(dim=1)).flatten()
        if len(t) == 0:
            continue
        hits += 1
        a = x[t] @ w_gu[e].T
        ea = p1 * U * (x[t].abs() @ w_gu[e].abs().T)
        g, u = a[:, :F], a[:, F:]
        act = g * torch.sigmoid(g)
        h = w[t, None] * act * u
        eh = w[t, None].abs() * (1.1 * ea[:, :F] * u.abs() + act.abs() * ea[:, F:] + 1.1 * ea[:, :F] * ea[:, F:])
        most = h.abs() + eh
        kept = 2.0 ** -11 * most + 2.0 ** -38 * most.amax(1, keepdim=True) if q8 else 2.0 ** -16 * most
        eh = eh + kept + 2.0 ** -18 * most + 2.0 ** -124
        out[t] += h @ w_dn[e].T
        err[t] += eh @ w_dn[e].abs().T
        mag[t] += most @ w_dn[e].abs().T
    err = err + (40 + F / 32 + hits) * U * mag
    return out, err + BF16 * (out.abs() + err) + 2.0 ** -133
