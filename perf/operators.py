"""What is measured of the operators around the expert FFN of a few tokens: residual addition with RMS norm
(mk_add_rmsnorm, with and without an 8-bit output) and the whole MoE layer for at most 128 tokens, router to
combined rows, with bf16 weights (mk_moe_layer) and with 8-bit activations and weights (mk_moe_layer_q8).

`run` computes an operator in elementary torch operations where `own` is false, and through the library's binding
where it is true.  Definitions (sums and products over real numbers, each output rounded once):

  add + norm   h = x + residual;  y = h * gamma / sqrt(mean(h^2) + eps);  the 8-bit form per group of 128 columns:
               s = max(max|y|, 2^-40) / 448,  q = e4m3(y / s)
  MoE layer    logits = x . Wr (+ bias);  the k largest, ties to the lowest expert id;  gate = softmax over all
               experts at the chosen ones;  out[t] = sum over t's local choices e of
               gate * W_down[e] . (silu(W_gate[e] . x) * (W_up[e] . x))
  8-bit form   x = q_x * s_x (one scale per token and 128 columns), W = q_w * s_w (one scale per 128 x 128 block of
               the gate, up and down matrices); the router reads the bf16 x that q_x was made from
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
GROUP = 128            # columns per scale of 8-bit activations, rows and columns per scale of 8-bit weights
FP8_MAX = 448.0        # largest e4m3 value
AMAX_FLOOR = 2.0 ** -40
TIE_MARGIN = 1e-5      # see _make_x


# ------------------------------------------------------------------------------------------------ cases

def _norm(name, T, d, residual, bf16, q8):
    return {"name": name, "op": "norm", "T": T, "d": d, "residual": residual, "bf16": bf16, "q8": q8}


def _layer(name, op, T, d, E, k, E_local, F, route, zipf=False):
    return {"name": name, "op": op, "T": T, "d": d, "E": E, "k": k, "E_local": E_local, "F": F, "route": route,
            "zipf": zipf}


def listed():
    return [
        # the norm in front of the layer: one token of a decode step, bf16 for the router and e4m3 for the experts
        _norm("norm_token", 1, 7168, True, True, True),
        # an odd batch in front of a bf16 layer, nothing to add (the first layer)
        _norm("norm_odd", 37, 2048, False, True, False),
        # a prefill of the Mixtral-shaped workload
        _norm("norm_prefill", 4096, 4096, True, True, False),
        # every token of the wide expert-parallel workload, both outputs
        _norm("norm_wide_q8", 16384, 7168, True, True, True),
        # the smallest layer: one token of the tiny workload, where launches and waits count
        _layer("layer_tiny_token", "layer", 1, 512, 8, 2, 8, 512, True),
        # one token through Mixtral-shaped experts: two of eight experts' weights
        _layer("layer_mixtral_token", "layer", 1, 4096, 8, 2, 8, 14336, True),
        # an odd batch through fine-grained experts with skewed popularity
        _layer("layer_skewed_odd", "layer", 13, 2048, 64, 6, 64, 1408, True, True),
        # one GPU's share of a decode step, routed by the sources, most choices elsewhere
        _layer("layer_share_routed", "layer", 8, 7168, 256, 8, 32, 2048, False),
        # the decode-shaped workload: 128 tokens, every local expert hit
        _layer("layer_decode", "layer", 128, 7168, 256, 8, 32, 2048, True),
        # the 8-bit forms: one token over fine-grained experts, a batch over Mixtral-shaped ones, and the decode-shaped
        # workload
        _layer("q8_fine_token", "layer_q8", 1, 2048, 64, 6, 64, 1408, True),
        _layer("q8_mixtral_batch", "layer_q8", 24, 4096, 8, 2, 8, 14336, False),
        _layer("q8_decode", "layer_q8", 128, 7168, 256, 8, 32, 2048, True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "layer", "layer", "layer", "layer_q8", "layer_q8"])
    if op == "norm":
        q8 = rng.random() < 0.5
        d = 128 * _log_int(rng, 2, 56) if q8 else 8 * _log_int(rng, 16, 896)
        bf16 = not q8 or rng.random() < 0.7
        return {"op": "norm", "T": _log_int(rng, 1, 16384), "d": d, "residual": rng.random() < 0.7, "bf16": bf16,
                "q8": q8}
    d = 128 * _log_int(rng, 4, 56)
    E = rng.choice([8, 16, 60, 64, 65, 128, 256])
    k = rng.randint(1, 8)
    share = rng.choice([1, 1, 2, 8])
    E_local = max(1, E // share)
    step = 8 if op == "layer" else 16
    F = step * _log_int(rng, 64 // step, 14336 // step)
    most = 2.8e9 if op == "layer" else 1.4e9   # bytes of all local experts: the largest listed case's
    each = 3 * F * d * (2 if op == "layer" else 1)
    E_local = max(1, min(E_local, int(most // each)))
    T = _log_int(rng, 1, 128)
    return {"op": op, "T": T, "d": d, "E": E, "k": k, "E_local": E_local, "F": F, "route": rng.random() < 0.7,
            "zipf": rng.random() < 0.3}


# ------------------------------------------------------------------------------------------------ inputs

def _zipf_bias(E):
    """log2 of rank-Zipf(1.2) expert popularity."""
    p = np.arange(1, E + 1, dtype=np.float64) ** -1.2
    return torch.from_numpy(np.log2(p / p.sum()).astype(np.float32))


def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    out = torch.empty(*shape, dtype=dtype, device=g.device)
    out.normal_(generator=g)
    return out.mul_(scale) if scale != 1.0 else out


def _make_x(g, case, wr, bias):
    """Activations as a norm leaves them (unit scale).  A token whose k + 1 largest logits are not TIE_MARGIN apart is
    passed over: which of two experts comes first would there depend on the order of an fp32 sum."""
    T, k = case["T"], case["k"]
    pool = _randn(g, T + 64, case["d"], dtype=torch.bfloat16)
    if wr is None:
        return pool[:T].contiguous()
    logits = pool.double() @ wr.double()
    if bias is not None:
        logits = logits + bias.double()
    top = logits.topk(min(k + 1, case["E"]), dim=1).values
    gap = (top[:, :-1] - top[:, 1:]).min(dim=1).values if top.shape[1] > 1 else torch.ones(T + 64, device=g.device)
    return pool[torch.nonzero(gap > TIE_MARGIN).flatten()[:T]].contiguous()


def _quant_rows(y):
    """e4m3 codes and scales of rows, one scale per 128 columns (inputs of the 8-bit layer)."""
    T, d = y.shape
    g = y.float().view(T, d // GROUP, GROUP)
    s = g.abs().amax(dim=2).clamp_min(AMAX_FLOOR) / FP8_MAX
    return (g / s[:, :, None]).view(T, d).to(torch.float8_e4m3fn), s.contiguous()


def _quant_blocks(w):
    """e4m3 codes [E, R, C] and scales [E, ceil(R / 128), ceil(C / 128)] of expert matrices."""
    E, R, C = w.shape
    nr, nc = -(-R // GROUP), -(-C // GROUP)
    codes = torch.empty(E, R, C, dtype=torch.float8_e4m3fn, device=w.device)
    scales = torch.empty(E, nr, nc, device=w.device)
    for e in range(E):
        p = torch.zeros(nr * GROUP, nc * GROUP, device=w.device)
        p[:R, :C] = w[e].float()
        b = p.view(nr, GROUP, nc, GROUP)
        s = b.abs().amax(dim=(1, 3)).clamp_min(AMAX_FLOOR) / FP8_MAX
        scales[e] = s
        codes[e] = (b / s[:, None, :, None]).view(nr * GROUP, nc * GROUP)[:R, :C].to(torch.float8_e4m3fn)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    T, d = case["T"], case["d"]
    st = {"case": dict(case)}
    if case["op"] == "norm":
        st["x"] = _randn(g, T, d, dtype=torch.bfloat16)
        st["residual"] = _randn(g, T, d, dtype=torch.bfloat16, scale=2.0) if case["residual"] else None
        st["gamma"] = (1.0 + 0.2 * _randn(g, d)).to(torch.bfloat16)
        return st
    E, k, E_local, F = case["E"], case["k"], case["E_local"], case["F"]
    wr = _randn(g, d, E, scale=1.0 / math.sqrt(d))
    bias = _zipf_bias(E).cuda() if case["zipf"] else None
    st["x"] = _make_x(g, case, wr, bias)
    st["w_router"], st["bias"], st["ids"], st["gates"] = wr, bias, None, None
    if not case["route"]:   # routed by the sources, gates scaled to a sum of one over the k choices
        logits = st["x"].double() @ wr.double() + (0.0 if bias is None else bias.double())
        top = logits.topk(k, dim=1)
        st["ids"] = top.indices.to(torch.int32)
        st["gates"] = torch.softmax(top.values, dim=1).float()
    gate_up = torch.empty(E_local, 2 * F, d, dtype=torch.bfloat16, device="cuda")
    down = torch.empty(E_local, d, F, dtype=torch.bfloat16, device="cuda")
    gate_up.normal_(generator=g).mul_(1.0 / math.sqrt(d))
    down.normal_(generator=g).mul_(1.0 / math.sqrt(F))
    if case["op"] == "layer":
        st["gate_up"], st["down"] = gate_up, down
    else:
        st["x_q8"], st["x_scale"] = _quant_rows(st["x"])
        # the gate and the up matrix have block scales of their own: [E_local, 2 ceil(F / 128), d / 128]
        gq, gs = _quant_blocks(gate_up[:, :F])
        uq, us = _quant_blocks(gate_up[:, F:])
        st["gate_up"] = torch.cat([gq.view(torch.uint8), uq.view(torch.uint8)], dim=1).view(torch.float8_e4m3fn)
        st["gate_up_scale"] = torch.cat([gs, us], dim=1).contiguous()
        st["down"], st["down_scale"] = _quant_blocks(down)
    if own:   # the workspace that a serving program keeps
        import moe_dispatch_expert_amd as mk
        st["workspace"] = torch.zeros(mk.mk_moe_layer_workspace_bytes(T, d, E, k, 0, E_local, F), dtype=torch.uint8,
                                      device="cuda")
    return st


# ------------------------------------------------------------------------------------------------ the plain forms

def _plain_norm(st):
    c = st["case"]
    h = st["x"].float()
    if c["residual"]:
        h = h + st["residual"].float()
    y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS) * st["gamma"].float()
    out = {}
    if c["residual"]:
        out["residual"] = h.to(torch.bfloat16)
    if c["bf16"]:
        out["y"] = y.to(torch.bfloat16)
    if c["q8"]:
        groups = y.view(c["T"], c["d"] // GROUP, GROUP)
        s = groups.abs().amax(dim=2).clamp_min(AMAX_FLOOR) / FP8_MAX
        out["q8"] = (groups / s[:, :, None]).view(c["T"], c["d"]).to(torch.float8_e4m3fn)
        out["q8_scale"] = s
    return out


def _block_values(codes, scales):
    """fp32 values of e4m3 matrices with one scale per 128 x 128 block."""
    s = scales.repeat_interleave(GROUP, dim=1)[:, :codes.shape[1]]
    return codes.float() * s.repeat_interleave(GROUP, dim=2)[:, :, :codes.shape[2]]


def _plain_layer(st):
    c = st["case"]
    T, d, E, k, E_local, F = (c[n] for n in ("T", "d", "E", "k", "E_local", "F"))
    if c["route"]:
        # 64 bits: an expert next to the k-th place must not change sides
        logits = st["x"].double() @ st["w_router"].double()
        if st["bias"] is not None:
            logits = logits + st["bias"].double()
        order = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
        p = torch.exp(logits - logits.amax(dim=1, keepdim=True))
        gates = (p.gather(1, order) / p.sum(dim=1, keepdim=True)).float()
        ids = order.to(torch.int32)
    else:
        ids, gates = st["ids"], st["gates"]
    # gate of every (token, local expert) pair, 0 where the token did not choose it
    local = torch.arange(E_local, device=ids.device, dtype=torch.int32)
    dense = (gates[:, :, None] * (ids[:, :, None] == local)).sum(dim=1)
    if c["op"] == "layer":
        x, gate_up, down = st["x"].float(), st["gate_up"].float(), st["down"].float()
    else:
        x = st["x_q8"].float() * st["x_scale"].repeat_interleave(GROUP, dim=1)
        nb = -(-F // GROUP)
        gate_up = torch.cat([_block_values(st["gate_up"][:, :F], st["gate_up_scale"][:, :nb]),
                             _block_values(st["gate_up"][:, F:], st["gate_up_scale"][:, nb:])], dim=1)
        down = _block_values(st["down"], st["down_scale"])
    gu = (x @ gate_up.view(E_local * 2 * F, d).t()).view(T, E_local, 2 * F)
    gate, up = gu[:, :, :F], gu[:, :, F:]
    h = gate / (1.0 + torch.exp(-gate)) * up * dense[:, :, None]
    y = torch.bmm(h.transpose(0, 1).contiguous(), down.transpose(1, 2).contiguous()).sum(dim=0)
    return {"out": y.to(torch.bfloat16)}


# ------------------------------------------------------------------------------------------------ the library's calls

def _own_norm(st):
    import moe_dispatch_expert_amd as mk
    c = st["case"]
    return mk.mk_add_rmsnorm(st["x"], st["gamma"], st["residual"], eps=EPS, bf16=c["bf16"], q8=c["q8"])


def _own_layer(st):
    import moe_dispatch_expert_amd as mk
    c = st["case"]
    routing = {"w_router": st["w_router"], "bias": st["bias"]} if c["route"] else \
        {"topk_ids_in": st["ids"], "topk_w_in": st["gates"], "E": c["E"]}
    if c["op"] == "layer":
        o = mk.mk_moe_layer(st["x"], st["gate_up"], st["down"], c["k"], workspace=st["workspace"], **routing)
    else:
        if c["route"]:
            routing["x"] = st["x"]
        o = mk.mk_moe_layer_q8(st["x_q8"], st["x_scale"], st["gate_up"], st["gate_up_scale"], st["down"],
                               st["down_scale"], c["k"], workspace=st["workspace"], **routing)
    return {"out": o["out"]}


def run(state):
    if state["case"]["op"] == "norm":
        return _own_norm(state) if own else _plain_norm(state)
    return _own_layer(state) if own else _plain_layer(state)


# ------------------------------------------------------------------------------------------------ what a pass needs

def _hit_experts(case):
    """Local experts that T tokens of random routing choose (one fixed draw of logits of the inputs' distribution)."""
    z = np.random.RandomState(1).randn(case["T"], case["E"])
    if case["zipf"]:
        z = z + _zipf_bias(case["E"]).numpy()
    chosen = np.argsort(-z, axis=1)[:, :case["k"]]
    local = chosen[chosen < case["E_local"]]
    return len(np.unique(local)), local.size


def work(case):
    T, d = case["T"], case["d"]
    if case["op"] == "norm":
        n = T * d
        b = 2 * n + (4 * n if case["residual"] else 0) + (2 * n if case["bf16"] else 0) + 2 * d
        if case["q8"]:
            b += n + 4 * n // GROUP
        return {"bytes": b, "flops": 5 * n}
    hit, rows = _hit_experts(case)
    F, E, k = case["F"], case["E"], case["k"]
    w = 3 * F * d
    if case["op"] == "layer":
        b = hit * 2 * w + 2 * T * d
    else:
        b = hit * (w + 4 * w // GROUP ** 2) + T * d + 4 * T * d // GROUP + (2 * T * d if case["route"] else 0)
    b += 2 * T * d + (0 if case["route"] else 8 * T * k)
    fl = 2 * rows * w
    if case["route"]:
        b += 4 * d * E
        fl += 2 * T * d * E
    return {"bytes": b, "flops": fl}


# ------------------------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The definitions in 64 bits, expert by expert.  An 8-bit output is given before its rounding to 8 bits."""
    st = prepare(case, seed)
    if case["op"] == "norm":
        h = st["x"].to(torch.float64)
        if st["residual"] is not None:
            h += st["residual"].to(torch.float64)
        out = {"residual": h.clone()} if case["residual"] else {}
        y = h / (h.pow(2).sum(1, keepdim=True) / case["d"] + EPS).sqrt() * st["gamma"].to(torch.float64)
        if case["bf16"]:
            out["y"] = y
        if case["q8"]:
            blocks = y.unflatten(1, (-1, GROUP))
            s = torch.maximum(blocks.abs().max(2).values, torch.tensor(AMAX_FLOOR, device=y.device)) / FP8_MAX
            out["q8"] = (blocks / s.unsqueeze(2)).flatten(1)
            out["q8_scale"] = s
        return out
    T, d, k, F = case["T"], case["d"], case["k"], case["F"]
    if case["route"]:
        z = torch.matmul(st["x"].to(torch.float64), st["w_router"].to(torch.float64))
        z = z if st["bias"] is None else z + st["bias"].to(torch.float64)
        top = z.topk(k, dim=1)
        ids, gates = top.indices, torch.exp(top.values - torch.logsumexp(z, dim=1, keepdim=True))
    else:
        ids, gates = st["ids"].long(), st["gates"].to(torch.float64)

    def spread(scale, axis, size):
        return torch.repeat_interleave(scale.to(torch.float64), GROUP, axis).narrow(axis, 0, size)

    x = st["x"].to(torch.float64)
    if case["op"] != "layer":
        x = st["x_q8"].to(torch.float64) * spread(st["x_scale"], 1, d)
    y = torch.zeros(T, d, dtype=torch.float64, device=x.device)
    for e in range(case["E_local"]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not len(t):
            continue
        gu, dn = st["gate_up"][e].to(torch.float64), st["down"][e].to(torch.float64)
        if case["op"] != "layer":
            blocks = st["gate_up_scale"].shape[1] // 2
            gs, us = st["gate_up_scale"][e, :blocks], st["gate_up_scale"][e, blocks:]
            gu[:F] *= spread(spread(gs, 0, F), 1, d)
            gu[F:] *= spread(spread(us, 0, F), 1, d)
            dn *= spread(spread(st["down_scale"][e], 0, d), 1, F)
        a = torch.matmul(x[t], gu.T)
        h = a[:, :F] * torch.sigmoid(a[:, :F]) * a[:, F:]
        y.index_add_(0, t, gates[t, j].unsqueeze(1) * torch.matmul(h, dn.T))
    return {"out": y}
