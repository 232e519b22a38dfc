"""Cases and plain forms of the microscaled 4-bit and expert-routing operators.

Four operators of a weight-only 4-bit serving path:

  quantize  values -> 4-bit floating point (E2M1) with one power-of-two scale
            (E8M0) per 32 values along K, and the values it stands for
  matmul    y = x . W^T with such weights; x in 16 bits, or quantized the same
            way on its way in (act "mx4")
  route     router logits -> chosen experts, their weights, and the (token,
            choice) pairs grouped by expert
  experts   the block behind the router: routing, gate and up products, SiLU,
            down product, weighted sum per token

``run`` computes them in elementary torch operations, or through the package
where ``own`` is true. ``exact`` evaluates the definitions in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
# the magnitudes of the eight E2M1 codes; bit 3 of a code is the sign
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = 32


# ---- cases ---------------------------------------------------------------------

def _quantize(rows, K, dtype, rule):
    return {"op": "quantize", "rows": rows, "K": K, "dtype": dtype, "rule": rule}


def _matmul(M, N, K, dtype, act="same"):
    return {"op": "matmul", "M": M, "N": N, "K": K, "dtype": dtype, "act": act}


def _route(T, E, k, dtype, score, groups=1, top_groups=1, padded=0):
    return {"op": "route", "T": T, "E": E, "k": k, "dtype": dtype, "score": score, "groups": groups,
            "top_groups": top_groups, "padded": padded}


def _experts(T, E, k, D, F, dtype):
    return {"op": "experts", "T": T, "E": E, "k": k, "D": D, "F": F, "dtype": dtype}


def listed():
    return [
        # one token's activations before a 4-bit product: latency only
        dict(_quantize(1, 4096, "bf16", "floor"), name="quantize_token"),
        # a ragged prompt's activations in front of a down projection, scales that never clip
        dict(_quantize(1023, 14336, "fp16", "ceil"), name="quantize_prompt"),
        # the weights of a large up projection, offline, as a checkpoint holds them
        dict(_quantize(28672, 8192, "fp32", "floor"), name="quantize_weights"),
        # one token through a small projection: latency counts
        dict(_matmul(1, 1024, 1024, "fp16"), name="matmul_small"),
        # one token through an up projection: the weights' bytes bound it
        dict(_matmul(1, 14336, 4096, "bf16"), name="matmul_token"),
        # a decoding batch of odd size through a down projection
        dict(_matmul(33, 4096, 14336, "fp16"), name="matmul_batch"),
        # a ragged prompt through an up projection
        dict(_matmul(2047, 14336, 4096, "bf16"), name="matmul_prompt"),
        # a long prompt with 4-bit activations through a large up projection: the largest product
        dict(_matmul(4096, 28672, 8192, "bf16", "mx4"), name="matmul_mx4_prompt"),
        # one token's router
        dict(_route(1, 64, 8, "bf16", "softmax"), name="route_token"),
        # a padded prompt's router: sigmoid scores, a balance bias, 8 groups of which 4 are kept
        dict(_route(8191, 256, 8, "fp32", "sigmoid", 8, 4, 250), name="route_prompt"),
        # one token through its 4 of 32 experts
        dict(_experts(1, 32, 4, 4096, 1024, "bf16"), name="experts_token"),
        # a ragged prompt over 64 experts
        dict(_experts(4095, 64, 6, 4096, 1024, "bf16"), name="experts_prompt"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A K: a power of two between the bounds, or an odd number of blocks of 32."""
    n = _log(rng, lo, hi)
    if rng.random() < 0.4:
        return 1 << max(lo.bit_length() - 1, min(n.bit_length(), hi.bit_length() - 1))
    return BLOCK * (n // BLOCK | 1)


def draw(rng):
    op = rng.choice(["quantize", "matmul", "matmul", "route", "experts"])
    if op == "quantize":
        K = _width(rng, 1024, 14336)
        rows = min(_log(rng, 1, 28672), 28672 * 8192 // K)
        return _quantize(rows, K, rng.choice(["bf16", "fp16", "fp32"]), rng.choice(["floor", "ceil"]))
    if op == "matmul":
        M, N, K = _log(rng, 1, 4096), _log(rng, 1024, 28672) | 1, _width(rng, 1024, 14336)
        N = min(N, 28672 * 8192 // K | 1)
        return _matmul(M, N, K, rng.choice(["bf16", "fp16"]), rng.choice(["same", "same", "mx4"]))
    if op == "route":
        T = _log(rng, 1, 8191)
        if rng.random() < 0.5:
            return _route(T, rng.choice([8, 32, 60, 64, 128]), rng.choice([1, 2, 4, 6, 8]),
                          rng.choice(["bf16", "fp16", "fp32"]), "softmax", padded=T // 20)
        groups = rng.choice([1, 4, 8])
        E = groups * rng.choice([16, 24, 32])
        return _route(T, E, rng.choice([4, 6, 8]), rng.choice(["bf16", "fp32"]), "sigmoid", groups,
                      max(1, groups // 2), T // 20)
    E = rng.choice([8, 16, 32, 60, 64])
    return _experts(_log(rng, 1, 4095), E, rng.choice([1, 2, 4, 6]), _width(rng, 1024, 4096),
                    _width(rng, 512, 1024), rng.choice(["bf16", "fp16"]))


def work(case):
    c = case
    b = BYTES[c["dtype"]]
    per = 0.5 + 1.0 / BLOCK                       # bytes of a 4-bit value with its share of the scale
    if c["op"] == "quantize":
        n = c["rows"] * c["K"]
        return {"bytes": n * (2 * b + per), "flops": 2.0 * n}
    if c["op"] == "matmul":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": N * K * per + (M * K + M * N) * b, "flops": 2.0 * M * N * K}
    T, E, k = c["T"], c["E"], c["k"]
    route = T * E * b + 12.0 * T * k + 4 * (E + 1)
    if c["op"] == "route":
        return {"bytes": route + (4 * E if c["score"] == "sigmoid" else 0), "flops": 4.0 * T * E}
    D, F = c["D"], c["F"]
    # experts that at least one of T * k pairs reaches, were they spread evenly
    live = E * (1.0 - (1.0 - 1.0 / E) ** (T * k)) if T > 1 else k
    return {"bytes": route + live * 3 * D * F * per + 2.0 * T * D * b, "flops": 6.0 * T * k * D * F}


# ---- inputs --------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _activations(g, rows, K, dtype):
    """Normal values with a few loud channels, as a transformer block's inputs have."""
    x = torch.randn(rows, K, generator=g, device=DEV)
    loud = torch.rand(K, generator=g, device=DEV) < 0.004
    return torch.where(loud, x * 12.0, x).to(dtype)


def _weights(g, rows, K):
    return torch.randn(rows, K, generator=g, device=DEV) * 0.02


def _packed(codes, scales):
    """The handle a user's program keeps of its weights."""
    import weight_only_lut_amd as lutq
    return lutq.mx_pack(codes, scales)


def prepare(case, seed):
    c, g = case, _gen(seed)
    dt = DTYPES[c["dtype"]]
    st = {"case": c}
    if c["op"] == "quantize":
        st["x"] = (_weights if dt == torch.float32 else lambda g, r, K: _activations(g, r, K, dt))(g, c["rows"], c["K"])
    elif c["op"] == "matmul":
        st["x"] = _activations(g, c["M"], c["K"], dt)
        st["w"] = _quantized(_weights(g, c["N"], c["K"]), "floor")
        if own:
            st["packed"] = _packed(*st["w"])
    else:
        T, E = c["T"], c["E"]
        # some experts are liked more than others, by most tokens
        logits = torch.randn(T, E, generator=g, device=DEV) + 0.5 * torch.randn(E, generator=g, device=DEV)
        if c["op"] == "route":
            st["bias"] = None
            if c["score"] == "sigmoid":
                st["bias"] = 0.1 * torch.randn(E, generator=g, device=DEV)
            if c["padded"]:
                logits[torch.randperm(T, generator=g, device=DEV)[:c["padded"]]] = float("-inf")
            st["logits"] = logits.to(dt)
        else:
            D, F = c["D"], c["F"]
            st["logits"] = logits.to(dt)
            st["x"] = _activations(g, T, D, dt)
            q = _quantized(_weights(g, E * 2 * F, D), "floor")
            st["gate_up"] = tuple(t.view(E, 2 * F, -1) for t in q)
            q = _quantized(_weights(g, E * D, F), "floor")
            st["down"] = tuple(t.view(E, D, -1) for t in q)
            if own:
                st["packed"] = _packed(*st["gate_up"]), _packed(*st["down"])
    return st


# ---- plain forms ---------------------------------------------------------------

def _quantized(x, rule):
    """uint8 codes [rows, K / 2] (even k in the low nibble) and E8M0 scales [rows, K / 32]."""
    v = x.float().view(x.shape[0], -1, BLOCK)
    top = v.abs().amax(-1)
    bits = top.view(torch.int32)
    e = (bits >> 23) - 2                                  # floor(log2 max) less that of 6
    if rule == "ceil":
        e = e + ((bits & 0x7FFFFF) > 0x400000).int()      # above 6 times the scale: the next power of two
    bad = ~torch.isfinite(top)
    e = e.clamp(0, 254)
    v = v * torch.exp2((127 - e).float()).unsqueeze(-1)
    a = v.abs()
    code = (a > 0.25).to(torch.uint8)                     # the level, halfway cases to the even code
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code += torch.signbit(v).to(torch.uint8) * 8
    code = torch.where(bad.unsqueeze(-1), torch.zeros_like(code), code).view(x.shape[0], -1)
    return code[:, 0::2] | (code[:, 1::2] << 4), torch.where(bad, 255, e).to(torch.uint8)


def _values(codes, scales, dtype=torch.float32):
    """The values codes and scales stand for."""
    level = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    pair = torch.stack((level.repeat(16), level.repeat_interleave(16)), -1)   # of a byte: low, high nibble
    s = torch.exp2(scales.float() - 127.0)
    s = torch.where(scales == 255, float("nan"), s)
    v = pair[codes.int()].view(*scales.shape, BLOCK)
    return (v * s.unsqueeze(-1)).view(*codes.shape[:-1], -1).to(dtype)


def _routed(c, logits, bias):
    """ids and weights [T, k] of the chosen experts; id -1 and weight 0 where nothing is left to choose."""
    l = logits.float()
    T, E = l.shape
    k, G = c["k"], c.get("groups", 1)
    if c.get("score", "softmax") == "softmax":
        key = l                                           # the score rises with the logit
    else:
        score = 1.0 / (1.0 + torch.exp(-l))
        key = torch.where(torch.isneginf(l), float("-inf"), score + bias)
    if G > 1:
        per = key.view(T, G, E // G)
        gs = torch.sort(per, dim=-1, descending=True, stable=True)[0][..., :2]
        gs = gs[..., 0] + gs[..., 1]
        kept = torch.sort(gs, dim=-1, descending=True, stable=True)[1][:, :c["top_groups"]]
        mask = (kept.unsqueeze(-1) == torch.arange(G, device=l.device)).any(1)
        key = torch.where(mask.unsqueeze(-1), per, float("-inf")).view(T, E)
    ids = torch.sort(key, dim=-1, descending=True, stable=True)[1][:, :k]
    live = torch.gather(key, 1, ids) > float("-inf")
    if c.get("score", "softmax") == "softmax":
        chosen = torch.gather(l, 1, ids)
        w = torch.exp(chosen - chosen[:, :1])
        w = torch.where(live, w, 0.0)
        w = w / w.sum(-1, keepdim=True)
    else:
        w = torch.where(live, torch.gather(score, 1, ids), 0.0)
        w = w / (w.sum(-1, keepdim=True) + 1e-20) * 2.5
    return torch.where(live, ids, -1).int(), torch.where(live, w, 0.0)


def _grouped(ids, E):
    """offsets [E + 1] of each expert's pairs in order [T * k], the pairs t * k + j by expert; -1 past the last."""
    flat = ids.reshape(-1)
    by = torch.where(flat < 0, E, flat)
    order = torch.sort(by, stable=True)[1].int()
    ends = torch.searchsorted(by.sort()[0].contiguous(), torch.arange(E + 1, device=ids.device, dtype=by.dtype))
    order = torch.where(torch.arange(order.numel(), device=ids.device) < ends[E], order, -1)
    return ends.int(), order


def _experts_plain(c, st):
    E, k, D, F = c["E"], c["k"], c["D"], c["F"]
    ids, w = _routed(c, st["logits"], None)
    offsets, order = _grouped(ids, E)
    pair = order.long()
    expert = ids.reshape(-1)[pair].long()
    room = int((offsets[1:] - offsets[:-1]).max())        # rows of the fullest expert
    at = expert * room + torch.arange(pair.numel(), device=ids.device) - offsets[expert]
    xs = torch.zeros(E * room, D, device=ids.device)
    xs[at] = st["x"].float()[pair // k]
    if c["T"] * k < E:                                    # few pairs: only their experts' weights
        xs, at = xs[at].view(-1, 1, D), torch.arange(pair.numel(), device=ids.device)
        gu, dn = [tuple(t[expert] for t in st[n]) for n in ("gate_up", "down")]
    else:
        xs, gu, dn = xs.view(E, room, D), st["gate_up"], st["down"]
    h = torch.bmm(xs, _values(*gu).transpose(1, 2).contiguous())
    h = h[..., :F] / (1.0 + torch.exp(-h[..., :F])) * h[..., F:]
    y = torch.bmm(h, _values(*dn).transpose(1, 2).contiguous()).view(-1, D)[at]
    y = y * w.reshape(-1)[pair].unsqueeze(-1)
    out = torch.empty_like(y)
    out[pair] = y                                         # back in the order of the tokens
    return ids, w, out.view(c["T"], k, D).sum(1).to(st["x"].dtype)


def run(state):
    c = state["case"]
    if own:
        return _run_own(c, state)
    if c["op"] == "quantize":
        return _values(*_quantized(state["x"], c["rule"]), state["x"].dtype)
    if c["op"] == "matmul":
        x = state["x"].float()
        if c["act"] == "mx4":
            x = _values(*_quantized(state["x"], "floor"))
        return (x @ _values(*state["w"]).T).to(state["x"].dtype)
    if c["op"] == "route":
        ids, w = _routed(c, state["logits"], state["bias"])
        return (ids, w) + _grouped(ids, c["E"])
    return _experts_plain(c, state)


def _run_own(c, state):
    import weight_only_lut_amd as lutq
    if c["op"] == "quantize":
        codes, scales = lutq.mx_quantize(state["x"], rule=c["rule"])
        return lutq.mx_dequantize(codes, scales, state["x"].dtype)
    if c["op"] == "matmul":
        if c["act"] == "mx4":
            return lutq.mx_matmul(lutq.mx_quantize(state["x"]), state["packed"], dtype=state["x"].dtype)
        return lutq.mx_matmul(state["x"], state["packed"])
    if c["op"] == "route":
        if c["score"] == "softmax":
            r = lutq.moe_route(state["logits"], c["k"])
        else:
            r = lutq.moe_route(state["logits"], c["k"], score="sigmoid", bias=state["bias"], groups=c["groups"],
                               top_groups=c["top_groups"], group_best=2, scale=2.5)
        return r.ids, r.weights, r.offsets, r.order
    r = lutq.moe_route(state["logits"], c["k"])
    return r.ids, r.weights, lutq.moe_mlp(state["x"], *state["packed"], r)


# ---- the definitions in 64 bits --------------------------------------------------

def _exact_rounded(x, rule):
    """The 4-bit values of x as fp64: the nearest level times the block's scale, found by distance."""
    v = x.double().view(x.shape[0], -1, BLOCK)
    top = v.abs().amax(-1)
    e = torch.frexp(top)[1].double() - 1.0 - 2.0
    s = torch.exp2(e.clamp(-127.0, 127.0))
    if rule == "ceil":
        s = torch.where(top > 6.0 * s, 2.0 * s, s)
    s = torch.where(top == 0, 1.0, s).unsqueeze(-1)
    q = v.abs() / s
    even = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    mid = (even[1:] + even[:-1]) / 2
    hi = torch.bucketize(q, mid, right=True)              # halfway cases up ...
    lo = torch.bucketize(q, mid, right=False)             # ... and down
    return (even[torch.where(hi % 2 == 0, hi, lo)].copysign(v) * s).view(x.shape)


def _exact_values(codes, scales):
    level = torch.tensor(LEVELS, dtype=torch.float64, device=codes.device)
    n = torch.stack((codes % 16, codes // 16), -1).view(*codes.shape[:-1], -1).long()
    v = torch.where(n >= 8, -level[n % 8], level[n % 8])
    return torch.ldexp(v, scales.repeat_interleave(BLOCK, -1).int() - 127)


def _exact_routed(c, logits, bias):
    l = logits.double()
    T, E = l.shape
    p = torch.sigmoid(l) if c.get("score", "softmax") == "sigmoid" else torch.softmax(l, -1)
    key = l if bias is None else torch.where(torch.isinf(l), l, p + bias.double())
    G = c.get("groups", 1)
    if G > 1:
        best = key.view(T, G, -1).topk(2, -1)[0].sum(-1).topk(c["top_groups"], -1)[1]
        out = torch.ones(T, G, dtype=torch.bool, device=l.device).scatter_(1, best, False)
        key = key.masked_fill(out.repeat_interleave(E // G, 1), float("-inf"))
    top, ids = key.topk(c["k"], -1)
    w = p.gather(1, ids).masked_fill(torch.isneginf(top), 0.0)
    w = w.nan_to_num(0.0) / (w.nan_to_num(0.0).sum(-1, keepdim=True) + 1e-300)
    return ids, w * (2.5 if bias is not None else 1.0)


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "quantize":
        return _exact_rounded(st["x"], c["rule"])
    if c["op"] == "matmul":
        x = _exact_rounded(st["x"], "floor") if c["act"] == "mx4" else st["x"].double()
        return x @ _exact_values(*st["w"]).T
    ids, w = _exact_routed(c, st["logits"], st.get("bias"))
    if c["op"] == "route":
        return None, w, None, None
    y = torch.zeros(c["T"], c["D"], dtype=torch.float64, device=ids.device)
    for e in range(c["E"]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            g, u = (st["x"][t].double() @ _exact_values(st["gate_up"][0][e], st["gate_up"][1][e]).T).chunk(2, -1)
            h = g * torch.sigmoid(g) * u
            y[t] += w[t, j].unsqueeze(-1) * (h @ _exact_values(st["down"][0][e], st["down"][1][e]).T)
    return None, w, y
