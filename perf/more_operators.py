"""What is measured of the experts' products backward and in 8-bit integers: the gradients of the combine
(mk_combine_backward), the SwiGLU (mk_swiglu_backward) and the grouped product (mk_grouped_gemm_dgrad,
mk_grouped_gemm_wgrad), the grouped product of 8-bit integers (mk_quant_i8, mk_grouped_gemm_i8) and the expert FFN made
of it (mk_expert_layout, mk_swiglu_i8).

`run` computes an operator in elementary torch operations where `own` is false, and through the library's binding
where it is true.  Definitions (over real numbers; each operator's output is rounded once, and what a chain hands from
one operator to the next is that rounded output):

  layout            row slot(t, j) of choice (t, j): the choices sorted by expert, then by token; other choices -1
  combine           out[t] = sum_j w[t, j] * y[slot(t, j)];  backward:  dy[slot(t, j)] = w[t, j] * dout[t],
                    dw[t, j] = sum_n dout[t, n] * y[slot(t, j), n],  0 where the choice has no slot
  SwiGLU            h = silu(g) * u;  backward:  dg = dh * u * s * (1 + g * (1 - s)),  du = dh * g * s,  s = sigmoid(g)
  grouped product   y[r] = W[e] . a[r] for the rows r of expert e;  backward:  da[r] = W[e]^T . dy[r],
                    dW[e] = sum over e's rows of dy[r] a[r]^T  (added to what is there, where a case accumulates)
  8-bit rows        scale = max|x| / 127 per row,  q = round(127 * x / max|x|)  (ties to even)
  8-bit product     y[r, n] = scale[r] * wscale[e, n] * sum_i q[r, i] * wq[e, n, i], in bf16
"""
import math

import torch

own = False


# ------------------------------------------------------------------------------------------------ cases

def _combine(name, T, N, E, k, E_local):
    return {"name": name, "op": "combine_backward", "T": T, "N": N, "E": E, "k": k, "E_local": E_local}


def _swiglu(name, rows, F, h):
    return {"name": name, "op": "swiglu_backward", "rows": rows, "F": F, "h": h}


def _grad(name, op, T, k, E, K, N, zipf=False, gather=False, accumulate=False, bf16=True):
    return {"name": name, "op": op, "T": T, "k": k, "E": E, "K": K, "N": N, "zipf": zipf, "gather": gather,
            "accumulate": accumulate, "bf16": bf16}


def _i8(name, T, k, E, K, N):
    return {"name": name, "op": "i8", "T": T, "k": k, "E": E, "K": K, "N": N, "zipf": False}


def _ffn(name, T, k, E, E_local, d, F, zipf=False):
    return {"name": name, "op": "i8_ffn", "T": T, "k": k, "E": E, "E_local": E_local, "d": d, "F": F, "zipf": zipf}


def listed():
    return [
        # the backward pass of the combine: an odd batch over fine-grained experts, where the launch counts ...
        _combine("combine_odd", 37, 2048, 64, 6, 64),
        # ... and every token of the wide expert-parallel workload, whose choices are mostly on other GPUs
        _combine("combine_wide", 16384, 7168, 256, 8, 32),
        # the SwiGLU's: the rows of that odd batch, and all rows of the Mixtral-shaped workload with h made again for the
        # down-projection's gradient
        _swiglu("swiglu_odd", 221, 1408, False),
        _swiglu("swiglu_mixtral", 8192, 14336, True),
        # gradient of the rows through the grouped product: a few rows over many experts (bound by their weights), and
        # the Mixtral-shaped workload
        _grad("dgrad_odd", "dgrad", 37, 6, 64, 2048, 1408),
        _grad("dgrad_mixtral", "dgrad", 4096, 2, 8, 4096, 14336),
        # gradient of the experts' weights: skewed popularity with idle experts, rows read in place, added to the fp32
        # gradients of an earlier micro-batch; and the Mixtral-shaped workload
        _grad("wgrad_skewed", "wgrad", 8192, 6, 64, 2048, 1408, zipf=True, gather=True, accumulate=True, bf16=False),
        _grad("wgrad_mixtral", "wgrad", 4096, 2, 8, 4096, 14336),
        # 8-bit product: one token through one matrix, and a Mixtral-shaped prefill
        _i8("i8_token", 1, 1, 1, 4096, 14336),
        _i8("i8_mixtral", 4096, 2, 8, 4096, 14336),
        # the 8-bit expert FFN from given ids: one GPU's share of a decode step, and a skewed batch
        _ffn("i8_ffn_decode", 128, 8, 256, 32, 7168, 2048),
        _ffn("i8_ffn_skewed", 8192, 6, 64, 64, 2048, 1408, zipf=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["combine_backward", "swiglu_backward", "dgrad", "dgrad", "wgrad", "wgrad", "i8", "i8", "i8_ffn",
                     "i8_ffn"])
    E = rng.choice([1, 2, 7, 8, 16, 60, 64, 65, 128, 256])
    k = rng.randint(1, min(8, E))
    if op == "combine_backward":
        E_local = max(1, E // rng.choice([1, 1, 2, 8]))
        T = _log_int(rng, 1, 16384)
        most = 131072 * 2048 // max(1, T * min(k, E_local))
        return {"op": op, "T": T, "N": 8 * _log_int(rng, 8, max(9, min(896, most // 8))), "E": E, "k": k, "E_local": E_local}
    if op == "swiglu_backward":
        return {"op": op, "rows": _log_int(rng, 1, 8192), "F": 8 * _log_int(rng, 8, 1792), "h": rng.random() < 0.5}
    if op == "i8_ffn":
        E_local = max(1, E // rng.choice([1, 1, 2, 8]))
        T, d = _log_int(rng, 1, 8192), 128 * _log_int(rng, 2, 56)
        F = 16 * _log_int(rng, 4, 896)
        E_local = max(1, min(E_local, int(1.4e9 // (3 * F * d))))
        while T > 1 and 6 * T * k * F * d > 8.5e11:
            T //= 2
        return {"op": op, "T": T, "k": k, "E": E, "E_local": E_local, "d": d, "F": F, "zipf": rng.random() < 0.4}
    T = _log_int(rng, 1, 8192)
    step = 16 if op == "i8" else 8
    K, N = step * _log_int(rng, 64 // step, 7168 // step), 8 * _log_int(rng, 8, 1792)
    if E * K * N > 470e6:
        E = max(1, int(470e6 // (K * N)))
        k = min(k, E)
    while T > 1 and 2 * T * k * K * N > 9.6e11:
        T //= 2
    case = {"op": op, "T": T, "k": k, "E": E, "K": K, "N": N, "zipf": rng.random() < 0.4}
    if op != "i8":
        case.update(gather=False, accumulate=False, bf16=True)
    if op == "wgrad":
        kind = rng.randint(0, 2)
        case.update(gather=rng.random() < 0.5, accumulate=kind == 2, bf16=kind == 0)
    return case


# ------------------------------------------------------------------------------------------------ inputs

def _randn(g, *shape, dtype=torch.bfloat16, scale=1.0):
    out = torch.empty(*shape, dtype=dtype, device=g.device)
    out.normal_(generator=g)
    return out.mul_(scale) if scale != 1.0 else out


def _routing(g, T, k, E, zipf):
    """ids [T, k] of T tokens' k choices (distinct, best first) and their gates, from logits of unit scale, with the
    popularity of a rank-Zipf(1.2) bias where asked for."""
    logits = torch.empty(T, E, device=g.device).normal_(generator=g)
    if zipf:
        p = torch.arange(1, E + 1, device=g.device, dtype=torch.float32) ** -1.2
        logits += torch.log2(p / p.sum())
    top = logits.topk(k, dim=1)
    return top.indices.to(torch.int32), torch.exp(top.values - torch.logsumexp(logits, 1, keepdim=True))


def _layout(ids, E_local):
    """Offsets, slots and rows' tokens of the local choices, as the dispatch leaves them, and the number of rows."""
    T, k = ids.shape
    e = ids.long().flatten()
    e = torch.where(e < E_local, e, E_local)
    order = torch.sort(e, stable=True).indices
    counts = torch.bincount(e, minlength=E_local + 1)[:E_local]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    R = int(offsets[-1])
    slot = torch.full((T * k,), -1, dtype=torch.int32, device=ids.device)
    slot[order[:R]] = torch.arange(R, dtype=torch.int32, device=ids.device)
    return offsets, slot.view(T, k), (order[:R] // k).to(torch.int32), R


def _row_buffer(case):
    """Rows of the buffers that a program with part of the experts keeps: the choices it expects and 12 deviations."""
    T, k, E, E_local = case["T"], case["k"], case["E"], case["E_local"]
    mean = T * k * E_local / E
    return min(T * min(k, E_local), int(mean + 12.0 * math.sqrt(mean)) + 16)


def _quant_weights(g, E, N, K):
    """8-bit codes [E, N, K] and scales [E, N] of experts' matrices of unit gain, one expert at a time."""
    codes = torch.empty(E, N, K, dtype=torch.int8, device=g.device)
    scales = torch.empty(E, N, device=g.device)
    for e in range(E):
        w = torch.empty(N, K, device=g.device).normal_(generator=g).mul_(1.0 / math.sqrt(K))
        m = w.abs().amax(dim=1)
        scales[e] = m / 127.0
        codes[e] = torch.round(w * (127.0 / m)[:, None]).to(torch.int8)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 6151 + 29)
    st = {"case": dict(case)}
    op = case["op"]
    if op == "swiglu_backward":
        st["gate_up"] = _randn(g, case["rows"], 2 * case["F"])
        st["dh"] = _randn(g, case["rows"], case["F"], scale=0.1)
        return st
    T, k, E = case["T"], case["k"], case["E"]
    ids, gates = _routing(g, T, k, E, case.get("zipf", False))
    if op == "i8_ffn":
        d, F, E_local = case["d"], case["F"], case["E_local"]
        st["ids"], st["gates"] = ids, gates
        st["x"] = _randn(g, T, d)
        st["gate_up"], st["gate_up_scale"] = _quant_weights(g, E_local, 2 * F, d)
        st["down"], st["down_scale"] = _quant_weights(g, E_local, d, F)
        # rows' tokens past the last row stay as they were
        st["row_token"] = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
        return st
    if op == "combine_backward":
        _, st["slot_of"], _, R = _layout(ids, case["E_local"])
        rows = _row_buffer(case)
        st["slot_of"][st["slot_of"] >= rows] = -1
        st["gates"] = gates
        st["dout"] = _randn(g, T, case["N"])
        st["y"] = _randn(g, rows, case["N"])
        st["dy"] = torch.zeros(rows, case["N"], dtype=torch.bfloat16, device="cuda")
        return st
    K, N = case["K"], case["N"]
    st["offsets"], _, st["row_token"], R = _layout(ids, E)
    if op == "i8":
        st["x"] = _randn(g, T, K)
        st["w"], st["w_scale"] = _quant_weights(g, E, N, K)
        return st
    st["dy"] = _randn(g, R, N)
    if op == "dgrad":
        st["w"] = _randn(g, E, N, K, scale=1.0 / math.sqrt(K))
        return st
    st["a"] = _randn(g, T if case["gather"] else R, K)
    if case["accumulate"]:   # the fp32 gradients of earlier micro-batches, which the call adds to
        st["dw"] = torch.empty(E, N, K, device="cuda").normal_(generator=g).mul_(20.0)
    return st


# ------------------------------------------------------------------------------------------------ the plain forms

def _plain_combine_backward(st):
    slot = st["slot_of"].long()
    T, k = slot.shape
    dout, y = st["dout"].float(), st["y"]
    dy = st["dy"]   # rows without a choice stay as they were
    dw = torch.zeros(T, k, device=y.device)
    for j in range(k):
        t = torch.nonzero(slot[:, j] >= 0).flatten()
        r = slot[t, j]
        dy[r] = (dout[t] * st["gates"][t, j, None]).to(torch.bfloat16)
        dw[t, j] = (dout[t] * y[r].float()).sum(dim=1)
    return {"dy_perm": dy, "dtopk_w": dw}


def _plain_swiglu(gate_up):
    g, u = gate_up.float().chunk(2, dim=1)
    return g / (1.0 + torch.exp(-g)) * u


def _plain_swiglu_backward(st):
    g, u = st["gate_up"].float().chunk(2, dim=1)
    dh = st["dh"].float()
    s = 1.0 / (1.0 + torch.exp(-g))
    out = {"dgate_up": torch.cat([dh * u * (s * (1.0 + g * (1.0 - s))), dh * (g * s)], dim=1).to(torch.bfloat16)}
    if st["case"]["h"]:
        out["h"] = _plain_swiglu(st["gate_up"]).to(torch.bfloat16)
    return out


def _plain_dgrad(st):
    at = st["offsets"].tolist()
    da = torch.empty(st["dy"].shape[0], st["case"]["K"], dtype=torch.bfloat16, device="cuda")
    for e in range(st["case"]["E"]):
        if at[e + 1] > at[e]:
            da[at[e]:at[e + 1]] = (st["dy"][at[e]:at[e + 1]].float() @ st["w"][e].float()).to(torch.bfloat16)
    return {"da": da}


def _plain_wgrad(st):
    c = st["case"]
    at = st["offsets"].tolist()
    a = st["a"][st["row_token"].long()] if c["gather"] else st["a"]
    dw = torch.empty(c["E"], c["N"], c["K"], dtype=torch.bfloat16 if c["bf16"] else torch.float32, device="cuda")
    for e in range(c["E"]):
        rows = slice(at[e], at[e + 1])
        dw[e] = st["dy"][rows].float().t() @ a[rows].float()
    if c["accumulate"]:
        st["dw"] += dw
        dw = st["dw"]
    return {"dw": dw}


def _plain_quant(x):
    """Codes (as fp32 whole numbers) and scales of rows."""
    x = x.float()
    m = x.abs().amax(dim=1, keepdim=True)
    q = torch.where(m > 0, torch.round(127.0 * x / m.clamp_min(1e-38)), torch.zeros_like(x))
    return q, m.flatten() / 127.0


def _plain_i8(q, scale, offsets, w, w_scale, row_token):
    at = offsets.tolist()
    y = torch.empty(row_token.shape[0], w.shape[1], dtype=torch.bfloat16, device="cuda")
    for e in range(w.shape[0]):
        t = row_token[at[e]:at[e + 1]].long()
        if len(t):
            y[at[e]:at[e + 1]] = ((q[t] @ w[e].float().t()) * scale[t, None] * w_scale[e]).to(torch.bfloat16)
    return y


def _plain_i8_ffn(st):
    c = st["case"]
    offsets, slot_of, row_token, R = _layout(st["ids"], c["E_local"])
    q, s = _plain_quant(st["x"])
    gate_up = _plain_i8(q, s, offsets, st["gate_up"], st["gate_up_scale"], row_token)
    q, s = _plain_quant(_plain_swiglu(gate_up))
    z = _plain_i8(q, s, offsets, st["down"], st["down_scale"], torch.arange(R, device="cuda")).float()
    out = torch.zeros(c["T"], c["d"], device="cuda")
    for j in range(c["k"]):
        t = torch.nonzero(slot_of[:, j] >= 0).flatten()
        out[t] += st["gates"][t, j, None] * z[slot_of[t, j].long()]
    st["row_token"][:R] = row_token
    return {"out": out.to(torch.bfloat16), "expert_offsets": offsets, "slot_of": slot_of, "row_token": st["row_token"]}


# ------------------------------------------------------------------------------------------------ the library's calls

def _own(st):
    import moe_dispatch_expert_amd as mk
    c = st["case"]
    op = c["op"]
    if op == "combine_backward":
        return mk.mk_combine_backward(st["dout"], st["y"], st["slot_of"], st["gates"], out={"dy_perm": st["dy"]})
    if op == "swiglu_backward":
        return mk.mk_swiglu_backward(st["gate_up"], st["dh"], h=c["h"])
    if op == "dgrad":
        return {"da": mk.mk_grouped_gemm_dgrad(st["dy"], st["offsets"], st["w"])}
    if op == "wgrad":
        return {"dw": mk.mk_grouped_gemm_wgrad(st["dy"], st["a"], st["offsets"],
                                               row_token=st["row_token"] if c["gather"] else None,
                                               dtype=torch.bfloat16 if c["bf16"] else torch.float32,
                                               out=st.get("dw"), accumulate=c["accumulate"])}
    if op == "i8":
        a = mk.mk_quant_i8(st["x"])
        return {"y": mk.mk_grouped_gemm_i8(a["q"], a["scale"], st["offsets"], st["w"], st["w_scale"],
                                           row_token=st["row_token"])}
    lay = mk.mk_expert_layout(st["ids"], c["E_local"], out={"row_token": st["row_token"]})
    rows = lay["expert_offsets"][c["E_local"]:]   # how many of the T * k rows are in use, on the device
    a = mk.mk_quant_i8(st["x"])
    gate_up = mk.mk_grouped_gemm_i8(a["q"], a["scale"], lay["expert_offsets"], st["gate_up"], st["gate_up_scale"],
                                    row_token=lay["row_token"])
    h = mk.mk_swiglu_i8(gate_up, rows_valid=rows)
    z = mk.mk_grouped_gemm_i8(h["q"], h["scale"], lay["expert_offsets"], st["down"], st["down_scale"])
    return {"out": mk.mk_combine(z, lay["slot_of"], st["gates"]), "expert_offsets": lay["expert_offsets"],
            "slot_of": lay["slot_of"], "row_token": lay["row_token"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "combine_backward":
        return _plain_combine_backward(state)
    if op == "swiglu_backward":
        return _plain_swiglu_backward(state)
    if op == "dgrad":
        return _plain_dgrad(state)
    if op == "wgrad":
        return _plain_wgrad(state)
    if op == "i8":
        q, s = _plain_quant(state["x"])
        return {"y": _plain_i8(q, s, state["offsets"], state["w"], state["w_scale"], state["row_token"])}
    return _plain_i8_ffn(state)


# ------------------------------------------------------------------------------------------------ what a pass needs

def _rows_and_hits(case, E_local):
    """Rows of local experts and experts with rows, for one fixed draw of the inputs' routing."""
    g = torch.Generator().manual_seed(1)
    ids, _ = _routing(g, case["T"], case["k"], case["E"], case.get("zipf", False))
    local = ids[ids < E_local]
    return local.numel(), len(torch.unique(local))


def work(case):
    op = case["op"]
    if op == "swiglu_backward":
        n = case["rows"] * case["F"]
        return {"bytes": (10 + (2 if case["h"] else 0)) * n, "flops": (14 if case["h"] else 11) * n}
    T, k = case["T"], case["k"]
    if op == "combine_backward":
        R, _ = _rows_and_hits(case, case["E_local"])
        N = case["N"]
        return {"bytes": 2 * T * N + 4 * R * N + 12 * T * k, "flops": 3 * R * N}
    if op == "i8_ffn":
        R, hit = _rows_and_hits(case, case["E_local"])
        d, F = case["d"], case["F"]
        weights = hit * (3 * F * d + 4 * (2 * F + d))
        return {"bytes": weights + 4 * T * d + 16 * T * k, "flops": 6 * R * F * d}
    R, hit = _rows_and_hits(case, case["E"])
    K, N, E = case["K"], case["N"], case["E"]
    flops = 2 * R * K * N
    if op == "i8":
        return {"bytes": 2 * T * K + hit * (K * N + 4 * N) + 2 * R * N + 4 * R, "flops": flops}
    if op == "dgrad":
        return {"bytes": 2 * (R * N + hit * K * N + R * K), "flops": flops}
    each = 2 if case["bf16"] else 4
    written = E * K * N * each if not case["accumulate"] else 2 * hit * K * N * each
    return {"bytes": 2 * R * N + 2 * (T if case["gather"] else R) * K + written, "flops": flops}


# ------------------------------------------------------------------------------------------------ 64 bits

def _exact_product(codes, scale, offsets, w, w_scale):
    """sum over an expert's columns of codes, in 64 bits; codes [R, K], scale [R]."""
    R = codes.shape[0]
    y = torch.zeros(R, w.shape[1], dtype=torch.float64, device=codes.device)
    for e in range(w.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            y[lo:hi] = torch.matmul(codes[lo:hi], w[e].to(torch.float64).T)
            y[lo:hi] *= scale[lo:hi].unsqueeze(1) * w_scale[e].to(torch.float64)
    return y


def _exact_codes(v):
    """Codes and scales of rows of 64-bit values."""
    big = v.abs().max(dim=1).values
    codes = (127 * v / torch.where(big == 0, torch.ones_like(big), big).unsqueeze(1)).round()
    return codes, big / 127


def exact(case, seed):
    """The definitions in 64 bits; what one operator of a chain hands to the next is rounded as that operator's output."""
    st = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "swiglu_backward":
        F = case["F"]
        g, u, dh = st["gate_up"][:, :F].to(f64), st["gate_up"][:, F:].to(f64), st["dh"].to(f64)
        s = torch.sigmoid(g)
        d = torch.empty(case["rows"], 2 * F, dtype=f64, device=g.device)
        d[:, :F] = dh * u * (s + g * s * torch.sigmoid(-g))
        d[:, F:] = dh * g * s
        return {"dgate_up": d, "h": g * s * u} if case["h"] else {"dgate_up": d}
    if op == "combine_backward":
        T, k = st["slot_of"].shape
        pairs = torch.nonzero(st["slot_of"] >= 0)
        t, j = pairs[:, 0], pairs[:, 1]
        slots = st["slot_of"][t, j].long()
        dy = torch.zeros(st["y"].shape, dtype=f64, device=t.device)
        dw = torch.zeros(T, k, dtype=f64, device=t.device)
        for i in range(0, len(t), 16384):   # a block of choices at a time
            ti, ji, si = t[i:i + 16384], j[i:i + 16384], slots[i:i + 16384]
            rows = st["dout"][ti].to(f64)
            dy.index_copy_(0, si, rows * st["gates"][ti, ji].to(f64).unsqueeze(1))
            dw[ti, ji] = (rows * st["y"][si].to(f64)).sum(1)
        return {"dy_perm": dy, "dtopk_w": dw}
    if op == "dgrad":
        da = torch.zeros(st["dy"].shape[0], case["K"], dtype=f64, device="cuda")
        for e in range(case["E"]):
            lo, hi = int(st["offsets"][e]), int(st["offsets"][e + 1])
            da[lo:hi] = torch.matmul(st["dy"][lo:hi].to(f64), st["w"][e].to(f64))
        return {"da": da}
    if op == "wgrad":
        dw = torch.zeros(case["E"], case["N"], case["K"], dtype=f64, device="cuda")
        for e in range(case["E"]):
            lo, hi = int(st["offsets"][e]), int(st["offsets"][e + 1])
            a = st["a"].index_select(0, st["row_token"][lo:hi].long()) if case["gather"] else st["a"][lo:hi]
            dw[e] = torch.matmul(st["dy"][lo:hi].to(f64).T, a.to(f64))
        if case["accumulate"]:
            dw += st["dw"].to(f64)
        return {"dw": dw}
    if op == "i8":
        codes, scale = _exact_codes(st["x"].to(f64))
        t = st["row_token"].long()
        return {"y": _exact_product(codes[t], scale[t], st["offsets"], st["w"], st["w_scale"])}
    T, k, F, E_local = case["T"], case["k"], case["F"], case["E_local"]
    ids = st["ids"].long()
    slot_of = torch.full((T, k), -1, dtype=torch.int32, device=ids.device)
    row_token = torch.full((T * k,), -1, dtype=torch.int32, device=ids.device)
    offsets, gates = [0], []
    for e in range(E_local):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        at = torch.arange(offsets[-1], offsets[-1] + len(t), dtype=torch.int32, device=ids.device)
        slot_of[t, j] = at
        row_token[at.long()] = t.to(torch.int32)
        gates.append(st["gates"][t, j].to(f64))
        offsets.append(offsets[-1] + len(t))
    t = row_token[:offsets[-1]].long()
    codes, scale = _exact_codes(st["x"].to(f64))
    gu = _exact_product(codes[t], scale[t], offsets, st["gate_up"], st["gate_up_scale"]).to(torch.bfloat16).to(f64)
    codes, scale = _exact_codes(gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:])
    z = _exact_product(codes, scale, offsets, st["down"], st["down_scale"]).to(torch.bfloat16).to(f64)
    out = torch.zeros(T, case["d"], dtype=f64, device=ids.device)
    out.index_add_(0, t, z * torch.cat(gates).unsqueeze(1))
    return {"out": out, "expert_offsets": torch.tensor(offsets, dtype=torch.int32, device=ids.device),
            "slot_of": slot_of, "row_token": row_token}
