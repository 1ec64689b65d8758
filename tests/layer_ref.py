"""The few-token MoE layer in fp64 on the CPU, with a bound on what fp32 sums and the two bf16 roundings may move it by.

u = 2^-24.  A dot product of n terms summed in fp32 along paths of at most p additions is off by at most
p u sum|a_i b_i|.  The gate|up products add 32 terms inside a matrix instruction, d / 128 instructions per wave (or
128-column blocks with two more roundings each, scale products and joins) and four waves: p <= 40 + d / 32.  The down
products likewise, once more per expert: p <= 40 + F / 32 + hits.  silu has |silu'| < 1.1 and is computed to 2^-20.
h = w silu(g) u is rounded to bf16 (2^-8 relative), and so is the output.
"""
import torch

U = 2.0 ** -24
BF16 = 2.0 ** -8


def layer(x, w_gu, w_dn, ids, gates, e_begin=0):
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
        eh = eh + (BF16 + 2.0 ** -18) * (h.abs() + eh) + 2.0 ** -133
        out[t] += h @ w_dn[e].T
        err[t] += eh @ w_dn[e].abs().T
        mag[t] += (h.abs() + eh) @ w_dn[e].abs().T
    err = err + (40 + F / 32 + hits) * U * mag
    return out, err + BF16 * (out.abs() + err) + 2.0 ** -133


def rows_q8(v):
    """e4m3 codes and fp32 scales of rows, one scale per 128 columns."""
    T, d = v.shape
    g = v.float().view(T, d // 128, 128)
    s = g.abs().amax(dim=2).clamp_min(2.0 ** -40) / 448.0
    return (g / s[:, :, None]).view(T, d).to(torch.float8_e4m3fn), s


def blocks_q8(w):
    """e4m3 codes and fp32 scales of matrices [E, R, C], one scale per 128 x 128 block."""
    E, R, C = w.shape
    nr, nc = -(-R // 128), -(-C // 128)
    p = torch.zeros(E, nr * 128, nc * 128)
    p[:, :R, :C] = w.float()
    b = p.view(E, nr, 128, nc, 128)
    s = b.abs().amax(dim=(2, 4)).clamp_min(2.0 ** -40) / 448.0
    q = (b / s[:, :, None, :, None]).view(E, nr * 128, nc * 128)[:, :R, :C].contiguous()
    return q.to(torch.float8_e4m3fn), s.contiguous()


def rows_values(q, s):
    return q.double() * s.double().repeat_interleave(128, dim=1)


def blocks_values(q, s):
    v = s.double().repeat_interleave(128, dim=1)[:, :q.shape[1]]
    return q.double() * v.repeat_interleave(128, dim=2)[:, :, :q.shape[2]]
