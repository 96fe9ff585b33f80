"""Cases, plain forms and 64-bit definitions of the few-token operators.

Three operators that a decode step calls between the library's GEMMs:

  quantize  4-bit codes, group scales (and zero points) of a [K, N] bf16 weight
  product   y = epilogue(x · dequant(codes, scales, zeros)), x of 1 to 64 tokens
  moe       a mixture-of-experts layer for 1 to 64 tokens: router product,
            softmax, top-k, gated up projection, down projection, weighted sum,
            with experts in bf16 or in 4 bits

Layouts follow the library: activations [tokens, K], weights [K, N] row-major
(experts [E, K, N]), scales [ceil(K / group), N]; two columns share a byte, the
even one in its low half; a fused gate+up weight alternates 32 gate columns and
32 up columns.
"""
import math

import torch

own = False

DEV = "cuda"


# --- cases ----------------------------------------------------------------------

def _product(name, T, K, N, group, zeros, epi):
    return {"name": name, "op": "product", "T": T, "K": K, "N": N, "group": group, "zeros": zeros, "epi": epi}


def _moe(name, T, H, I, E, k, weights, act, group=0, zeros=False, normalize=True):
    return {"name": name, "op": "moe", "T": T, "H": H, "I": I, "E": E, "k": k, "weights": weights, "act": act,
            "group": group, "zeros": zeros, "normalize": normalize}


def _quantize(name, K, N, group, zeros):
    return {"name": name, "op": "quantize", "K": K, "N": N, "group": group, "zeros": zeros}


def listed():
    return [
        # one token through an attention output projection: a few microseconds, latency counts
        _product("product_t1_4096x4096", 1, 4096, 4096, 128, False, "none"),
        # one token through the widest projection of the decode workload, zero points, memory-bound
        _product("product_t1_8192x28672_zeros", 1, 8192, 28672, 128, True, "none"),
        # a small batch through a fused gate+up projection, fine groups
        _product("product_t16_4096x28672_swiglu", 16, 4096, 28672, 64, True, "swiglu"),
        # ragged everything: odd N, K no multiple of a tile, five tokens, smallest groups, bias and GELU
        _product("product_t5_1000x1001_gelu", 5, 1000, 1001, 32, True, "gelu"),
        # the most tokens, a long reduction, residual added in the epilogue
        _product("product_t64_14336x4096_residual", 64, 14336, 4096, 128, False, "bias_residual"),
        # one token, many small experts: eight of them read, launch and routing latency count
        _moe("moe_t1_e64k8_2048x1024", 1, 2048, 1024, 64, 8, "bf16", "swiglu"),
        # one token, few large experts (hidden 4096, FFN 14336): memory-bound
        _moe("moe_t1_e8k2_4096x14336", 1, 4096, 14336, 8, 2, "bf16", "swiglu"),
        # the most tokens over many experts, nearly all of them read
        _moe("moe_t64_e32k4_4096x2048", 64, 4096, 2048, 32, 4, "bf16", "swiglu"),
        # a small batch over 4-bit experts with zero points
        _moe("moe_t16_e64k8_4096x2048_q", 16, 4096, 2048, 64, 8, "wq", "swiglu", 128, True),
        # ragged sizes, an odd expert count, probabilities not renormalised
        _moe("moe_t7_e13k3_1000x224_gelu", 7, 1000, 224, 13, 3, "bf16", "geglu", normalize=False),
        # a projection's weight quantised at load time, one scale a group
        _quantize("quantize_1024x4096", 1024, 4096, 128, False),
        # the decode workload's weight, with zero points
        _quantize("quantize_8192x28672_zeros", 8192, 28672, 64, True),
    ]


def _size(rng, lo, hi, step, odd=0.25, odd_step=8):
    """A size spread over its logarithm: a multiple of `step`, at times only of `odd_step`."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    q = odd_step if rng.random() < odd else step
    v = max(q, int(round(v / q)) * q)
    return v + q if v == 3072 else v


def _tokens(rng):
    return max(1, min(64, int(round(math.exp(rng.uniform(0.0, math.log(64.0)))))))


def draw(rng):
    op = rng.choice(["product", "product", "product", "moe", "moe", "moe", "quantize"])
    group = rng.choice([32, 64, 128, 256])
    zeros = rng.random() < 0.5
    if op == "product":
        epi = rng.choice(["none", "bias", "relu", "gelu", "bias_residual", "reglu", "geglu", "swiglu"])
        T = _tokens(rng)
        K = _size(rng, 512, 14336, 64)
        N = _size(rng, 512, 28672, 64, 0.4, 1)
        while K * N > 8192 * 28672 or T * K * N > 64 * 14336 * 4096:
            N = N * 3 // 4
        if epi in ("reglu", "geglu", "swiglu"):
            N = max(64, N // 64 * 64)
        while 3072 in (N, N // 2):
            N -= 64
        return {"op": "product", "T": T, "K": K, "N": N, "group": group, "zeros": zeros, "epi": epi}
    if op == "moe":
        E = rng.choice([4, 8, 13, 16, 32, 64, 128])
        k = rng.randint(1, min(8, E))
        H = _size(rng, 256, 4096, 64)
        I = _size(rng, 128, 14336, 64, 0.25, 32)
        T = _tokens(rng)
        while E * H * I > 32 * 4096 * 2048 or T * k * H * I > 64 * 4 * 4096 * 2048:
            I = max(32, I // 64 * 32)
        while 3072 in (I, 2 * I):
            I += 32
        weights = rng.choice(["bf16", "wq"])
        return {"op": "moe", "T": T, "H": H, "I": I, "E": E, "k": k, "weights": weights,
                "act": rng.choice(["reglu", "geglu", "swiglu"]), "group": group if weights == "wq" else 0,
                "zeros": zeros and weights == "wq", "normalize": rng.random() < 0.7}
    return {"op": "quantize", "K": _size(rng, 256, 8192, 64), "N": _size(rng, 512, 28672, 64, 0.4, 1), "group": group,
            "zeros": zeros}


# --- inputs ---------------------------------------------------------------------

def _normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32) * scale).bfloat16()


def _weight(g, E, K, N):
    """[E, K, N] bf16 with the spread of a trained projection, one expert at a time."""
    w = torch.empty(E, K, N, device=DEV, dtype=torch.bfloat16)
    for e in range(E):
        w[e] = _normal(g, K, N, scale=K ** -0.5)
    return w


def _codes(g, E, K, N, group, zeros):
    """4-bit codes with group scales and zero points, as a quantised checkpoint holds them."""
    ng = -(-K // group)
    codes = torch.randint(0, 256, (E, K, (N + 1) // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.rand(E, ng, N, generator=g, device=DEV) * 0.5 + 0.75
    scales = (s * (K ** -0.5 / 4.6)).bfloat16()
    z = torch.randint(5, 11, (E, ng, N), generator=g, device=DEV, dtype=torch.uint8) if zeros else None
    return codes, scales, z


def _glu(epi):
    return epi in ("reglu", "geglu", "swiglu")


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)
    if case["op"] == "quantize":
        s["W"] = _weight(g, 1, case["K"], case["N"])[0]
        return s
    T = case["T"]
    if case["op"] == "product":
        K, N = case["K"], case["N"]
        s["x"] = _normal(g, T, K)
        s["codes"], s["scales"], s["z"] = (None if v is None else v[0]
                                           for v in _codes(g, 1, K, N, case["group"], case["zeros"]))
        s["bias"] = None if case["epi"] == "none" else _normal(g, N, scale=0.1)
        out = N // 2 if _glu(case["epi"]) else N
        s["R"] = _normal(g, T, out) if case["epi"] == "bias_residual" else None
        if own:
            import autotuning_tcgen05_tmem_gb300 as lib
            s["packed"] = lib.wq_pack(s["codes"], s["scales"], s["z"], N, case["group"], gated=_glu(case["epi"]))
            s["plan"] = lib.wq_plan(K, N, group=case["group"], zeros=case["zeros"], epi=case["epi"])
            s["y"] = torch.empty(T, out, device=DEV, dtype=torch.bfloat16)
        return s
    H, I, E, k = case["H"], case["I"], case["E"], case["k"]
    s["x"] = _normal(g, T, H)
    s["router"] = _normal(g, H, E, scale=H ** -0.5)
    if case["weights"] == "bf16":
        s["gate_up"], s["down"] = _weight(g, E, H, 2 * I), _weight(g, E, I, H)
    else:
        s["gate_up"] = _codes(g, E, H, 2 * I, case["group"], case["zeros"])
        s["down"] = _codes(g, E, I, H, case["group"], case["zeros"])
    if own:
        import autotuning_tcgen05_tmem_gb300 as lib
        if case["weights"] == "wq":
            s["gate_up"] = lib.wq_pack(*s["gate_up"], 2 * I, case["group"], gated=True)
            s["down"] = lib.wq_pack(*s["down"], H, case["group"])
        s["plan"] = lib.moe_plan(H, I, E, k, act=case["act"], weights=case["weights"], group=case["group"],
                                 zeros=case["zeros"], normalize=case["normalize"])
        s["y"] = torch.empty(T, H, device=DEV, dtype=torch.bfloat16)
        s["ids"] = torch.empty(T, k, device=DEV, dtype=torch.int32)
        s["w"] = torch.empty(T, k, device=DEV, dtype=torch.float32)
    return s


# --- plain forms ----------------------------------------------------------------

def _dequant(codes, scales, zeros, N, group):
    """[..., K, N] fp32 weights: (code - zero) · scale."""
    K = codes.shape[-2]
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)[..., :N].float()
    of = torch.arange(K, device=codes.device) // group
    z = 8.0 if zeros is None else zeros.float()[..., of, :]
    return (q - z) * scales.float()[..., of, :]


def _act(v, name):
    if name in ("relu", "reglu"):
        return v.clamp_min(0.0)
    if name in ("gelu", "geglu"):
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if name == "swiglu":
        return v / (1.0 + torch.exp(-v))
    return v


def _gated(v, name):
    """act(gate) · up of [..., N] whose columns alternate 32 gate and 32 up."""
    b = v.unflatten(-1, (-1, 2, 32))
    return (_act(b[..., 0, :], name) * b[..., 1, :]).flatten(-2)


def _plain_quantize(s):
    K, N, G = s["K"], s["N"], s["group"]
    ng = -(-K // G)
    w = s["W"].float()
    pad = torch.cat((w, w[-1:].expand(ng * G - K, N))).view(ng, G, N)   # the last row again: no new extreme
    if s["zeros"]:
        lo, hi = pad.amin(1).clamp_max(0.0), pad.amax(1).clamp_min(0.0)
        scale = ((hi - lo) * (1.0 / 15.0)).bfloat16().float()
        scale = torch.where(scale == 0, 1.0, scale)
        zero = torch.round(-lo / scale).clamp(0.0, 15.0)
    else:
        scale = (pad.abs().amax(1) * (1.0 / 7.0)).bfloat16().float()
        scale = torch.where(scale == 0, 1.0, scale)
        zero = torch.full_like(scale, 8.0)
    q = (torch.round(pad / scale[:, None]) + zero[:, None]).clamp(0.0, 15.0).view(ng * G, N)[:K].to(torch.uint8)
    if N % 2:
        q = torch.cat((q, torch.zeros_like(q[:, :1])), dim=1)
    codes = q[:, 0::2] | (q[:, 1::2] << 4)
    return {"codes": codes, "scales": scale.bfloat16(), "zeros": zero.to(torch.uint8) if s["zeros"] else None}


def _plain_product(s):
    v = s["x"].float() @ _dequant(s["codes"], s["scales"], s["z"], s["N"], s["group"])
    if s["bias"] is not None:
        v = v + s["bias"].float()
    v = _gated(v, s["epi"]) if _glu(s["epi"]) else _act(v, s["epi"])
    if s["R"] is not None:
        v = v + s["R"].float()
    return v.bfloat16()


def _experts(w, N, group, ids):
    """fp32 weights of the experts `ids` (all of them where it is None)."""
    if isinstance(w, tuple):
        codes, scales, zeros = w if ids is None else (None if t is None else t[ids] for t in w)
        return _dequant(codes, scales, zeros, N, group)
    return (w if ids is None else w[ids]).float()


def _plain_moe(s):
    T, H, I, E, k = s["T"], s["H"], s["I"], s["E"], s["k"]
    x = s["x"].float()
    logits = x @ s["router"].float()
    top, ids = torch.sort(logits, dim=-1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    e = torch.exp(top - top[:, :1])
    w = e / (e.sum(-1, keepdim=True) if s["normalize"] else torch.exp(logits - top[:, :1]).sum(-1, keepdim=True))
    if T * k <= E:      # few rows: one product for each token and each of its experts
        at = ids.reshape(-1)
        h = _gated(x.repeat_interleave(k, 0)[:, None] @ _experts(s["gate_up"], 2 * I, s["group"], at), s["act"])
        o = (h @ _experts(s["down"], H, s["group"], at)).view(T, k, H)
        y = (o * w[..., None]).sum(1)
    else:               # every expert on every token, weighted by zero where it was not chosen
        h = _gated(x[None] @ _experts(s["gate_up"], 2 * I, s["group"], None), s["act"])
        o = h @ _experts(s["down"], H, s["group"], None)
        m = torch.zeros(T, E, device=x.device).scatter_(1, ids, w)
        y = (o * m.t()[..., None]).sum(0)
    return {"y": y.bfloat16(), "ids": ids.int(), "weights": w}


def run(state):
    s = state
    if not own:
        return {"quantize": _plain_quantize, "product": _plain_product, "moe": _plain_moe}[s["op"]](s)
    import autotuning_tcgen05_tmem_gb300 as lib
    if s["op"] == "quantize":
        codes, scales, zeros = lib.wq_quantize(s["W"], group=s["group"], zeros=s["zeros"])
        return {"codes": codes, "scales": scales, "zeros": zeros}
    if s["op"] == "product":
        s["plan"].run(s["x"], s["packed"], s["bias"], s["y"], residual=s["R"])
        return s["y"]
    s["plan"].run(s["x"], s["router"], s["gate_up"], s["down"], s["y"], ids=s["ids"], weights=s["w"])
    return {"y": s["y"], "ids": s["ids"], "weights": s["w"]}


# --- what a pass cannot do without ----------------------------------------------

def _weight_bytes(K, N, group, zeros):
    return K * N / 2 + -(-K // group) * N * (3 if zeros else 2)


def work(case):
    if case["op"] == "quantize":
        K, N = case["K"], case["N"]
        return {"bytes": 2 * K * N + _weight_bytes(K, N, case["group"], case["zeros"]), "flops": 4 * K * N}
    T = case["T"]
    if case["op"] == "product":
        K, N = case["K"], case["N"]
        out = N // 2 if _glu(case["epi"]) else N
        b = _weight_bytes(K, N, case["group"], case["zeros"]) + 2 * T * (K + out)
        b += 0 if case["epi"] == "none" else 2 * N
        b += 2 * T * out if case["epi"] == "bias_residual" else 0
        return {"bytes": b, "flops": 2 * T * K * N}
    H, I, E, k = case["H"], case["I"], case["E"], case["k"]
    active = E * (1.0 - (1.0 - k / E) ** T)      # distinct experts that T tokens choose, on average
    if case["weights"] == "bf16":
        each = 2 * 3 * H * I
    else:
        each = _weight_bytes(H, 2 * I, case["group"], case["zeros"]) + _weight_bytes(I, H, case["group"], case["zeros"])
    return {"bytes": active * each + 2 * H * E + 4 * T * H + 8 * T * k, "flops": 2 * T * H * E + 6 * T * k * H * I}


# --- the definitions in 64 bits -------------------------------------------------

def _exact_weight(w, e, N, group):
    """Expert e's [K, N] weight in 64 bits."""
    if not isinstance(w, tuple):
        return w[e].double()
    codes, scales, zeros = w
    c = codes[e].to(torch.int16)
    K = c.shape[0]
    full = torch.empty(K, 2 * c.shape[1], device=c.device, dtype=torch.float64)
    full[:, 0::2] = (c % 16).double()
    full[:, 1::2] = (c // 16).double()
    full = full[:, :N].contiguous()
    for g0 in range(0, K, group):
        rows = slice(g0, min(K, g0 + group))
        full[rows] -= 8.0 if zeros is None else zeros[e, g0 // group].double()
        full[rows] *= scales[e, g0 // group].double()
    return full


def _exact_act(v, name):
    if name in ("relu", "reglu"):
        return torch.where(v > 0, v, torch.zeros_like(v))
    if name in ("gelu", "geglu"):
        return v * torch.special.ndtr(v)
    if name == "swiglu":
        return v * torch.sigmoid(v)
    return v


def _exact_gated(v, name):
    cols = torch.arange(v.shape[-1] // 2, device=v.device)
    gate = 64 * (cols // 32) + cols % 32
    return _exact_act(v[:, gate], name) * v[:, gate + 32]


def _exact_product(s):
    codes, scales = s["codes"][None], s["scales"][None]
    zeros = None if s["z"] is None else s["z"][None]
    N = s["N"]
    parts = []
    for c0 in range(0, N, 4096):                  # a band of columns at a time
        c1 = min(N, c0 + 4096)
        w = (codes[:, :, c0 // 2:(c1 + 1) // 2], scales[:, :, c0:c1], None if zeros is None else zeros[:, :, c0:c1])
        parts.append(s["x"].double() @ _exact_weight(w, 0, c1 - c0, s["group"]))
    v = torch.cat(parts, dim=1)
    if s["bias"] is not None:
        v = v + s["bias"].double()
    v = _exact_gated(v, s["epi"]) if _glu(s["epi"]) else _exact_act(v, s["epi"])
    return v if s["R"] is None else v + s["R"].double()


def _exact_moe(s):
    T, H, I, E, k = s["T"], s["H"], s["I"], s["E"], s["k"]
    x = s["x"].double()
    logits = x @ s["router"].double()
    p = torch.softmax(logits, dim=-1)
    left = logits.clone()
    ids = torch.empty(T, k, device=x.device, dtype=torch.int64)
    for j in range(k):                            # the largest that is left, the lowest index among equals
        best = left.amax(-1, keepdim=True)
        ids[:, j] = (left == best).int().argmax(-1)
        left.scatter_(1, ids[:, j:j + 1], -math.inf)
    w = p.gather(1, ids)
    if s["normalize"]:
        w = w / w.sum(-1, keepdim=True)
    y = torch.zeros(T, H, device=x.device, dtype=torch.float64)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if len(t) == 0:
            continue
        h = _exact_gated(x[t] @ _exact_weight(s["gate_up"], e, 2 * I, s["group"]), s["act"])
        y[t] += w[t, j][:, None] * (h @ _exact_weight(s["down"], e, H, s["group"]))
    return {"y": y, "ids": ids.int(), "weights": w}


def _exact_quantize(s):
    """Scales and zero points; the codes follow from the rounded scales and have no 64-bit value of their own."""
    K, N, G = s["K"], s["N"], s["group"]
    scales = torch.empty(-(-K // G), N, device=DEV, dtype=torch.float64)
    for i in range(scales.shape[0]):
        w = s["W"][i * G:(i + 1) * G].double()
        if s["zeros"]:
            scales[i] = (w.amax(0).clamp_min(0) - w.amin(0).clamp_max(0)) / 15.0
        else:
            scales[i] = w.abs().amax(0) / 7.0
    return {"codes": None, "scales": torch.where(scales == 0, torch.ones_like(scales), scales), "zeros": None}


def exact(case, seed):
    global own
    was, own = own, False                          # the inputs as they are, without the library's layouts
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"quantize": _exact_quantize, "product": _exact_product, "moe": _exact_moe}[case["op"]](s)
