"""The operators around the recalibrated expert backward that one training step of an MoE layer
needs, as cases that can be timed and compared: the plain form of each operator in elementary
torch operations, and the calls of this package that compute the same.

  route      top-K routing of a token block: indices, routing weights, per-expert counts, the sum
             of the router's probabilities, the balance loss and the z-loss
  route_bwd  the gradients back to the logits: the routing weights' own gradient (a dot product of
             the output's cotangent with each routed expert's output row), then the router's
  norm       h = x + residual and RMS norm of h, with an 8-bit output and its scales where asked
  norm_bwd   its gradients
  adamw      one AdamW step over many tensors at once, moments in 32 bits or in 8

Layer sizes are those of workloads/configs.py.
"""

import math

import torch

own = False

F8 = torch.float8_e4m3fn
F8_MAX = 448.0        # largest e4m3 value
F8_STEP = 2.0 ** -9   # smallest positive e4m3 value
AMAX_MIN = 2.0 ** -100  # group maxima are floored here, so that no scale is zero
BLOCK = 256           # values under one scale of the 8-bit moments
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4, "f8": 1}
EPS = 1e-6            # of the norm
BETA1, BETA2, ADAM_EPS, LR, DECAY = 0.9, 0.95, 1e-8, 3e-4, 0.1
BALANCE, ZLOSS = 1e-2, 1e-3


def listed():
    return [
        # one token of a decoding user, routed alone: no losses, latency only
        {"name": "route_one_token", "op": "route", "T": 1, "E": 128, "K": 8, "dtype": "f32",
         "renorm": True, "stats": False, "pad": 0.0, "off": 0.0},
        # the full micro-batch of the 128-expert layer, 4 x 8192 tokens
        {"name": "route_t32k_e128", "op": "route", "T": 32768, "E": 128, "K": 8, "dtype": "bf16",
         "renorm": False, "stats": True, "pad": 0.0, "off": 0.0},
        # 256 experts, some of them switched off, padded sequences, an odd number of tokens
        {"name": "route_t5003_e256_padded", "op": "route", "T": 5003, "E": 256, "K": 8,
         "dtype": "f32", "renorm": True, "stats": True, "pad": 0.15, "off": 0.1},
        # the wide layer's backward: 16,384 tokens, model dimension 4096
        {"name": "route_bwd_t16k_d4096", "op": "route_bwd", "T": 16384, "E": 128, "K": 8,
         "D": 4096, "dtype": "bf16", "renorm": False, "pad": 0.0, "off": 0.0},
        # a short padded block of the 256-expert layer
        {"name": "route_bwd_t777_e256_padded", "op": "route_bwd", "T": 777, "E": 256, "K": 8,
         "D": 2048, "dtype": "bf16", "renorm": True, "pad": 0.15, "off": 0.1},
        # four decoding users: sum, norm and the 8-bit rows, latency only
        {"name": "norm_t4_d4096_q8", "op": "norm", "T": 4, "D": 4096, "dtype": "bf16",
         "residual": True, "q_cols": 128, "gap": 0},
        # the full micro-batch of a training step, 8-bit rows with a scale for 128 columns
        {"name": "norm_t32k_d2048_q8", "op": "norm", "T": 32768, "D": 2048, "dtype": "bf16",
         "residual": True, "q_cols": 128, "gap": 0},
        # the wide layer's norm in the backward pass, the residual stream's gradient added
        {"name": "norm_bwd_t16k_d4096", "op": "norm_bwd", "T": 16384, "D": 4096, "dtype": "bf16",
         "grad": "f32", "residual": True},
        # an odd, short block of a 32-bit layer
        {"name": "norm_bwd_t1021_d2040_f32", "op": "norm_bwd", "T": 1021, "D": 2040,
         "dtype": "f32", "grad": "f32", "residual": False},
        # every expert weight of the 128-expert layer (604 million), 32-bit moments
        {"name": "adamw_layer_f32", "op": "adamw", "tensors": 3, "largest": 128 * 2048 * 768,
         "smallest": 128 * 2048 * 768, "param": "bf16", "grad": "f32", "master": True,
         "state": "f32"},
        # the same with 8-bit moments
        {"name": "adamw_layer_f8", "op": "adamw", "tensors": 3, "largest": 128 * 2048 * 768,
         "smallest": 128 * 2048 * 768, "param": "bf16", "grad": "f32", "master": True,
         "state": "f8"},
        # norm weights, biases and router weights of many layers: many short, odd tensors
        {"name": "adamw_97_small", "op": "adamw", "tensors": 97, "largest": 2048 * 128,
         "smallest": 17, "param": "f32", "grad": "f32", "master": False, "state": "f32"},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route_bwd", "norm", "norm_bwd", "adamw"])
    if op in ("route", "route_bwd"):
        E = _log_uniform(rng, 4, 512)
        K = rng.randint(1, min(8, E))
        T = _log_uniform(rng, 1, 32768 if op == "route" else 16384)
        while T * E > 32768 * 128:
            T = max(1, T // 2)
        case = {"op": op, "T": T, "E": E, "K": K, "dtype": rng.choice(["bf16", "f32"]),
                "renorm": rng.random() < 0.5, "pad": rng.choice([0.0, 0.2]),
                "off": rng.choice([0.0, 0.1])}
        if op == "route":
            return {**case, "stats": rng.random() < 0.75}
        D = 8 * _log_uniform(rng, 4, 512)
        while D * T * K * BYTES[case["dtype"]] > 16384 * 8 * 4096 * 2:
            D = max(8, D // 16 * 8)
        return {**case, "D": D}
    if op in ("norm", "norm_bwd"):
        D = 8 * _log_uniform(rng, 4, 1024)
        T = _log_uniform(rng, 1, 32768)
        while T * D > 32768 * 2048:
            T = max(1, T // 2)
        case = {"op": op, "T": T, "D": D, "dtype": rng.choice(["bf16", "f32"]),
                "residual": rng.random() < 0.7}
        if op == "norm":
            return {**case, "q_cols": rng.choice([-1, -1, 0, 32, 64, 128]),
                    "gap": rng.choice([0, 0, 64])}
        return {**case, "grad": rng.choice(["f32", "bf16"])}
    count = _log_uniform(rng, 1, 200)
    total = _log_uniform(rng, 1000, 300_000_000)
    largest = max(1, total // count)
    param = rng.choice(["bf16", "f32"])
    return {"op": op, "tensors": count, "largest": largest,
            "smallest": _log_uniform(rng, 1, largest), "param": param,
            "grad": rng.choice(["f32", "bf16"]), "master": param == "bf16" and rng.random() < 0.7,
            "state": rng.choice(["f32", "f8"])}


# -- inputs -----------------------------------------------------------------------------------
def _sizes(case):
    """Lengths of the tensors of an optimizer case: from the largest to the smallest, evenly on a
    logarithmic scale, and where each begins in the flat buffers (on a whole block)."""
    n, hi, lo = case["tensors"], case["largest"], case["smallest"]
    sizes = [max(1, int(round(hi * (lo / hi) ** (i / max(1, n - 1))))) for i in range(n)]
    starts, at = [], 0
    for s in sizes:
        starts.append(at)
        at += -(-s // BLOCK) * BLOCK
    return sizes, starts, at


def _quantise_blocks(v, low):
    """e4m3 codes and scales of the 256-blocks of v; `low`: positive values stay positive."""
    b = v.view(-1, BLOCK)
    amax = b.abs().amax(1).clamp_min(AMAX_MIN)
    s = b * (F8_MAX / amax)[:, None]
    if low:
        s = torch.where(b > 0, s.clamp_min(F8_STEP), s)
    return s.to(F8).view(-1), amax / F8_MAX


def _route_inputs(case, gen):
    T, E = case["T"], case["E"]
    dev = "cuda"
    e = torch.arange(E, device=dev, dtype=torch.float32)
    x = torch.randn(T, E, generator=gen, device=dev) - 1.2 * torch.log(e + 1)
    if case["off"]:
        # experts that a token may not use; every 61st token may use none
        closed = torch.rand(T, E, generator=gen, device=dev) < case["off"]
        closed |= (torch.arange(T, device=dev) % 61 == 60)[:, None]
        x = x.masked_fill(closed, -math.inf)
    mask = None
    if case["pad"]:
        mask = (torch.rand(T, generator=gen, device=dev) >= case["pad"]).to(torch.uint8)
    return x.to(DT[case["dtype"]]), mask


def prepare(case, seed):
    dev, op = "cuda", case["op"]
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    s = {"case": case}
    if own:
        import demand_side_expert_gb300 as lib
    if op in ("route", "route_bwd"):
        T, E, K = case["T"], case["E"], case["K"]
        s["logits"], s["mask"] = _route_inputs(case, gen)
        if own:
            s["router"] = lib.Router(T, E, K, case["dtype"], renorm=case["renorm"],
                                     balance_coef=BALANCE, z_coef=ZLOSS)
        if op == "route_bwd":
            D, dt = case["D"], DT[case["dtype"]]
            fwd = _plain_route({**s, "case": {**case, "stats": True}})
            s["topk_idx"], s["counts"] = fwd["topk_idx"], fwd["counts"]
            # each pair's row among the experts' outputs: pairs sorted by expert
            order = torch.sort(s["topk_idx"].view(-1), stable=True).indices
            s["inv"] = torch.empty(T * K, dtype=torch.int32, device=dev)
            s["inv"][order] = torch.arange(T * K, dtype=torch.int32, device=dev)
            s["g"] = (randn(T, D) * torch.exp(0.5 * randn(T, 1))).to(dt)
            s["y"] = torch.empty(T * K, D, dtype=dt, device=dev).normal_(generator=gen)
            s["dloss"] = torch.ones(2, device=dev)
            if own:
                s["router"].topk_idx.copy_(s["topk_idx"])
                s["router"].counts.copy_(s["counts"])
                s["shape"] = lib.lrm.make_shape(T, D, D, E, K, lib.dtype_code(case["dtype"]))
                s["ws_bytes"] = lib.lrm.lrm_workspace_bytes(s["shape"])
                s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device=dev)
                lib.lrm.lrm_clear_device_error(s["ws"], s["ws_bytes"])
                s["dalpha"] = torch.empty(T, K, device=dev)
                s["lrm"] = lib.lrm
        return s
    if op in ("norm", "norm_bwd"):
        T, D, dt = case["T"], case["D"], DT[case["dtype"]]
        s["w"] = (1 + 0.1 * randn(D)).to(dt)
        # a residual stream has columns of very different size
        cols = torch.exp(0.7 * randn(D))
        if op == "norm":
            gap = case["gap"]
            s["x"] = (randn(T, D + gap) * 0.5).to(dt)[:, :D]
            s["res"] = (randn(T, D) * cols).to(dt) if case["residual"] else None
            if own:
                q = None if case["q_cols"] < 0 else case["q_cols"]
                s["norm"] = lib.AddRMSNorm(T, D, case["dtype"], eps=EPS, q_cols=q)
            return s
        gt = DT[case["grad"]]
        s["h"] = (randn(T, D) * cols).to(dt)
        s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
        s["dy"] = (randn(T, D) * 1e-2).to(gt)
        s["dh"] = (randn(T, D) * 1e-2).to(gt) if case["residual"] else None
        if own:
            s["norm"] = lib.AddRMSNorm(T, D, case["dtype"], eps=EPS, grad_dtype=case["grad"])
            s["norm"].rstd.copy_(s["rstd"])
        return s
    # adamw
    sizes, starts, total = _sizes(case)
    live = torch.zeros(total, dtype=torch.bool, device=dev)
    for a, n in zip(starts, sizes):
        live[a:a + n] = True

    def flat(scale):
        return torch.randn(total, generator=gen, device=dev).mul_(scale).mul_(live)

    master = flat(0.02)
    s["param"] = master.to(DT[case["param"]])
    s["grad"] = flat(1e-3).to(DT[case["grad"]])
    m, r = flat(3e-4), flat(1e-3).abs_()
    s["master"] = master if case["master"] else None
    s["step"] = 100
    if case["state"] == "f8":
        s["m"], s["m_scale"] = _quantise_blocks(m, False)
        s["v"], s["v_scale"] = _quantise_blocks(r, True)
    else:
        s["m"], s["v"] = m, r.square_()
    # tensors of up to 4096 values (norm weights, biases) are not decayed
    decay = [DECAY if n > 4096 else 0.0 for n in sizes]
    s["decay"] = decay[0] if len(set(decay)) == 1 else torch.repeat_interleave(
        torch.tensor(decay, device=dev),
        torch.tensor([-(-n // BLOCK) * BLOCK for n in sizes], device=dev))
    if own:
        opt = lib.AdamW([s["param"][a:a + n] for a, n in zip(starts, sizes)],
                        [s["grad"][a:a + n] for a, n in zip(starts, sizes)],
                        lr=LR, betas=(BETA1, BETA2), eps=ADAM_EPS, weight_decay=decay,
                        state=case["state"], master=case["master"])
        opt.load_state_dict({"step": s["step"], "master": s["master"], "m": s["m"], "v": s["v"],
                             "m_scale": s.get("m_scale"), "v_scale": s.get("v_scale")})
        s["opt"] = opt
    return s


# -- plain forms ------------------------------------------------------------------------------
def _usable(x, mask):
    """Tokens that take part: not padding, and with at least one expert open."""
    some = (x > -math.inf).any(1) | torch.isnan(x).any(1)
    return some if mask is None else some & (mask != 0)


def _softmax(x, use):
    top = torch.where(use, x.amax(1), torch.zeros_like(x[:, 0]))[:, None]
    ex = torch.where(use[:, None], torch.exp(x - top), torch.zeros_like(x))
    total = torch.where(use, ex.sum(1), torch.ones_like(top[:, 0]))[:, None]
    return ex / total, (top + torch.log(total))[:, 0]


def _plain_route(s):
    c = s["case"]
    x = s["logits"].float()
    use = _usable(x, s["mask"])
    rank = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
    idx = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :c["K"]]
    p, lse = _softmax(x, use)
    alpha = p.gather(1, idx)
    if c["renorm"]:
        total = alpha.sum(1, keepdim=True)
        alpha = alpha / torch.where(total == 0, torch.ones_like(total), total)
    out = {"topk_idx": idx.to(torch.int32), "alpha": alpha}
    if c["stats"]:
        chosen = torch.zeros_like(x, dtype=torch.int32).scatter_(1, idx, 1) * use[:, None]
        counts, psum, n = chosen.sum(0).to(torch.int32), p.sum(0), use.sum().clamp_min(1)
        balance = BALANCE * c["E"] * (counts * psum).sum() / (n.float().square() * c["K"])
        z = ZLOSS * lse.square().sum() / n
        out |= {"counts": counts, "prob_sum": psum, "loss": torch.stack([balance, z])}
    return out


def _plain_route_bwd(s):
    c = s["case"]
    x, idx = s["logits"].float(), s["topk_idx"].long()
    rows = s["y"][s["inv"].long()].view(c["T"], c["K"], c["D"]).float()
    dalpha = (rows * s["g"].float()[:, None, :]).sum(2)
    use = _usable(x, s["mask"])
    p, lse = _softmax(x, use)
    n = use.sum().clamp_min(1).float()
    chosen = p.gather(1, idx)
    if c["renorm"]:
        total = chosen.sum(1, keepdim=True)
        a = chosen / torch.where(total == 0, torch.ones_like(total), total)
        at = a * (dalpha - (a * dalpha).sum(1, keepdim=True))
        dx = torch.zeros_like(x).scatter_(1, idx, at)
    else:
        dp = torch.zeros_like(x).scatter_(1, idx, dalpha)
        dx = p * (dp - (p * dp).sum(1, keepdim=True))
    cost = s["dloss"][0] * BALANCE * c["E"] * s["counts"].float() / (n * n * c["K"])
    dx = dx + p * (cost - (p * cost).sum(1, keepdim=True))
    dx = dx + p * (s["dloss"][1] * 2 * ZLOSS * lse / n)[:, None]
    dx = torch.where(use[:, None], dx, torch.zeros_like(dx))
    return {"dalpha": dalpha, "dlogits": dx.to(s["logits"].dtype)}


def _quantise_rows(y, cols):
    T, D = y.shape
    cols = cols or D
    groups = -(-D // cols)
    g = torch.nn.functional.pad(y, (0, groups * cols - D)).view(T, groups, cols)
    amax = g.abs().amax(2).clamp_min(AMAX_MIN)
    q = (g * (F8_MAX / amax)[:, :, None]).view(T, groups * cols)[:, :D]
    return q.to(F8).contiguous(), amax / F8_MAX


def _plain_norm(s):
    c = s["case"]
    h = s["x"].float()
    if c["residual"]:
        h = h + s["res"].float()
    rstd = torch.rsqrt(h.square().mean(1) + EPS)
    y = h * rstd[:, None] * s["w"].float()
    out = {"rstd": rstd}
    if c["residual"]:
        out["h"] = h.to(s["x"].dtype)
    if c["q_cols"] < 0:
        out["y"] = y.to(s["x"].dtype)
    else:
        out["q"], out["q_scale"] = _quantise_rows(y, c["q_cols"])
    return out


def _plain_norm_bwd(s):
    h, dy, rstd = s["h"].float(), s["dy"].float(), s["rstd"][:, None]
    xhat = h * rstd
    wdy = dy * s["w"].float()
    dx = rstd * (wdy - xhat * (wdy * xhat).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["dy"].dtype), "dw": (dy * xhat).sum(0)}


def _spread(scale):
    return scale.repeat_interleave(BLOCK)


def _plain_adamw(s):
    c = s["case"]
    s["step"] += 1
    bc1, bc2 = 1 - BETA1 ** s["step"], 1 - BETA2 ** s["step"]
    g = s["grad"].float()
    held = s["master"] if c["master"] else s["param"]
    p = held.float()
    if c["state"] == "f8":
        m = s["m"].float() * _spread(s["m_scale"])
        v = (s["v"].float() * _spread(s["v_scale"])).square()
    else:
        m, v = s["m"], s["v"]
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    r = torch.sqrt(v)
    p = p * (1 - LR * s["decay"]) - (m / (r * (1 / math.sqrt(bc2)) + ADAM_EPS)) * (LR / bc1)
    held.copy_(p)
    if c["master"]:
        s["param"].copy_(p)
    if c["state"] == "f8":
        s["m"], s["m_scale"] = _quantise_blocks(m, False)
        s["v"], s["v_scale"] = _quantise_blocks(r, True)
    else:
        s["m"], s["v"] = m, v
    return {k: s[k] for k in ("param", "master", "m", "v", "m_scale", "v_scale")
            if s.get(k) is not None}


_PLAIN = {"route": _plain_route, "route_bwd": _plain_route_bwd, "norm": _plain_norm,
          "norm_bwd": _plain_norm_bwd, "adamw": _plain_adamw}


# -- one pass ---------------------------------------------------------------------------------
def run(state):
    s = state
    if not own:
        return _PLAIN[s["case"]["op"]](s)
    c = s["case"]
    op = c["op"]
    if op == "route":
        r = s["router"]
        r.route(s["logits"], mask=s["mask"], stats=c["stats"])
        if not c["stats"]:
            return {"topk_idx": r.topk_idx, "alpha": r.alpha}
        return {"topk_idx": r.topk_idx, "alpha": r.alpha, "counts": r.counts,
                "prob_sum": r.prob_sum, "loss": r.loss}
    if op == "route_bwd":
        s["lrm"].lrm_gate_grad(s["shape"], s["g"], s["y"], s["inv"], s["dalpha"], s["ws"],
                               s["ws_bytes"])
        s["router"].backward(s["logits"], s["dalpha"], mask=s["mask"], dloss=s["dloss"])
        return {"dalpha": s["dalpha"], "dlogits": s["router"].dlogits}
    if op == "norm":
        n = s["norm"]
        n.forward(s["x"], s["w"], residual=s["res"])
        out = {"rstd": n.rstd}
        if c["residual"]:
            out["h"] = n.h
        if c["q_cols"] < 0:
            out["y"] = n.y
        else:
            out["q"], out["q_scale"] = n.q, n.q_scale
        return out
    if op == "norm_bwd":
        n = s["norm"]
        n.backward(s["dy"], s["w"], dh=s["dh"], h=s["h"])
        return {"dx": n.dx, "dw": n.dw}
    opt = s["opt"]
    opt.step()
    out = {"param": s["param"], "m": opt.m, "v": opt.v}
    if c["master"]:
        out["master"] = opt.master
    if c["state"] == "f8":
        out |= {"m_scale": opt.m_scale, "v_scale": opt.v_scale}
    return out


def work(case):
    op = case["op"]
    if op in ("route", "route_bwd"):
        T, E, K = case["T"], case["E"], case["K"]
        b = BYTES[case["dtype"]]
        mask = T if case["pad"] else 0
        if op == "route":
            # logits once; an index and a weight for each pair; the statistics
            stats = 8 * E + 8 if case["stats"] else 0
            return {"bytes": T * E * b + mask + 8 * T * K + stats, "flops": 4 * T * E}
        D = case["D"]
        # output rows, cotangent, logits and their gradient, indices, inverse, dalpha
        return {"bytes": T * K * D * b + T * D * b + 2 * T * E * b + mask + 12 * T * K + 4 * E,
                "flops": 2 * T * K * D + 10 * T * E}
    if op in ("norm", "norm_bwd"):
        T, D, b = case["T"], case["D"], BYTES[case["dtype"]]
        if op == "norm":
            rows = b + (2 * b if case["residual"] else 0)
            if case["q_cols"] < 0:
                extra = T * D * b
            else:
                extra = T * D + 4 * T * -(-D // (case["q_cols"] or D))
            return {"bytes": T * D * rows + extra + D * b + 4 * T, "flops": 6 * T * D}
        g = BYTES[case["grad"]]
        rows = b + 2 * g + (g if case["residual"] else 0)
        return {"bytes": T * D * rows + D * (b + 4) + 4 * T, "flops": 9 * T * D}
    n = sum(_sizes(case)[0])
    # gradient in; parameter, master copy and both moments in and out (the parameter beside a
    # master copy is only written)
    moments = 2 * 2 * (1 + 4 / BLOCK) if case["state"] == "f8" else 16
    p = BYTES[case["param"]]
    held = 8 + p if case["master"] else 2 * p
    return {"bytes": n * (BYTES[case["grad"]] + held + moments), "flops": 16 * n}


# -- the same in 64 bits ----------------------------------------------------------------------
def _exact_router(case, x, mask):
    """Probabilities, log-sums, weights (differentiable in x) and the tokens that take part."""
    T, K = case["T"], case["K"]
    open_ = ~torch.isneginf(x.detach())
    use = open_.any(1)
    if mask is not None:
        use = use & mask.bool()
    safe = torch.where(use[:, None], x, torch.zeros_like(x))
    lse = torch.logsumexp(safe, 1)
    logp = safe - lse[:, None]
    p = torch.exp(logp) * use[:, None]
    # position of every expert in its token's order: how many come before it
    key = x.detach()
    idx = torch.argsort(-key, dim=1, stable=True)[:, :K]
    a = p.gather(1, idx)
    if case["renorm"]:
        a = torch.where(use[:, None], a / torch.where(use, a.sum(1), torch.ones(
            T, dtype=a.dtype, device=a.device))[:, None], torch.zeros_like(a))
    n = max(1, int(use.sum()))
    counts = torch.bincount(idx[use].reshape(-1), minlength=case["E"])
    balance = BALANCE * case["E"] * ((counts.double() / (n * K)) * (p.sum(0) / n)).sum()
    z = ZLOSS * torch.where(use, lse, torch.zeros_like(lse)).square().sum() / n
    return idx, a, counts, p, balance, z


def _e4m3(v):
    return v.float().to(F8).double()


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "route":
        idx, a, counts, p, balance, z = _exact_router(case, s["logits"].double(), s["mask"])
        out = {"topk_idx": idx.to(torch.int32), "alpha": a}
        if case["stats"]:
            out |= {"counts": counts.to(torch.int32), "prob_sum": p.sum(0),
                    "loss": torch.stack([balance, z])}
        return out
    if op == "route_bwd":
        T, K = case["T"], case["K"]
        at = s["inv"].long().view(T, K)
        g = s["g"].double()
        dalpha = torch.stack([(s["y"][at[:, k]].double() * g).sum(1) for k in range(K)], 1)
        x = s["logits"].double().requires_grad_(True)
        _, a, _, _, balance, z = _exact_router(case, x, s["mask"])
        total = (a * dalpha).sum() + s["dloss"][0].double() * balance
        total = total + s["dloss"][1].double() * z
        total.backward()
        return {"dalpha": dalpha, "dlogits": x.grad}
    if op == "norm":
        T, D = case["T"], case["D"]
        h = s["x"].double() + (s["res"].double() if case["residual"] else 0.0)
        ms = (h * h).sum(1) / D + EPS
        y = h / torch.sqrt(ms)[:, None] * s["w"].double()[None, :]
        out = {"rstd": 1 / torch.sqrt(ms)}
        if case["residual"]:
            out["h"] = h
        if case["q_cols"] < 0:
            out["y"] = y
            return out
        cols = case["q_cols"] or D
        q, scales = torch.empty_like(y), []
        for lo in range(0, D, cols):
            part = y[:, lo:lo + cols]
            scale = part.abs().max(1).values.clamp_min(AMAX_MIN) / F8_MAX
            q[:, lo:lo + cols] = _e4m3(part / scale[:, None])
            scales.append(scale)
        out["q"], out["q_scale"] = q, torch.stack(scales, 1)
        return out
    if op == "norm_bwd":
        # the gradients as functions of the given h and 1/rms: the row's own dot products
        h, dy, rs = s["h"].double(), s["dy"].double(), s["rstd"].double()
        w = s["w"].double()
        dot = torch.einsum("td,td,d->t", h, dy, w)
        dx = dy * w * rs[:, None] - h * (dot * rs ** 3 / case["D"])[:, None]
        if s["dh"] is not None:
            dx = dx + s["dh"].double()
        return {"dx": dx, "dw": torch.einsum("td,td,t->d", h, dy, rs)}
    out, piece = {}, 1 << 25
    t = s["step"] + 1
    total = s["grad"].numel()
    parts = {}
    for lo in range(0, total, piece):
        sl, bl = slice(lo, min(total, lo + piece)), slice(lo // BLOCK, -(-(lo + piece) // BLOCK))
        g = s["grad"][sl].double()
        p = (s["master"] if case["master"] else s["param"])[sl].double()
        m, v = s["m"][sl].double(), s["v"][sl].double()
        if case["state"] == "f8":
            m = (m.view(-1, BLOCK) * s["m_scale"][bl].double()[:, None]).view(-1)
            v = (v.view(-1, BLOCK) * s["v_scale"][bl].double()[:, None]).view(-1) ** 2
        m = BETA1 * m + (1 - BETA1) * g
        v = BETA2 * v + (1 - BETA2) * g ** 2
        mhat, vhat = m / (1 - BETA1 ** t), v / (1 - BETA2 ** t)
        decay = s["decay"] if isinstance(s["decay"], float) else s["decay"][sl].double()
        p = p - LR * (mhat / (vhat.sqrt() + ADAM_EPS) + decay * p)
        got = {"param": p}
        if case["master"]:
            got["master"] = p
        if case["state"] == "f8":
            for name, w, low in (("m", m, 0.0), ("v", v.sqrt(), F8_STEP)):
                w = w.view(-1, BLOCK)
                scale = w.abs().max(1).values.clamp_min(AMAX_MIN) / F8_MAX
                u = w / scale[:, None]
                got[name] = _e4m3(torch.where(w > 0, u.clamp_min(low), u)).view(-1)
                got[name + "_scale"] = scale
        else:
            got["m"], got["v"] = m, v
        for k, val in got.items():
            parts.setdefault(k, []).append(val)
    for k, vals in parts.items():
        out[k] = vals[0] if len(vals) == 1 else torch.cat(vals)
    return out
