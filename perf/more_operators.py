"""Operators of a training step under tight memory, as cases that can be timed and compared: the
plain form of each in elementary torch operations, and the calls of this package that compute the
same.

  route      routing with sigmoid or softmax scores, a selection bias, and groups of experts of
             which only the best are open to a token: indices, weights, counts, the scores' sums and
             the balance loss; the bias's step towards even loads
  route_bwd  its gradient to the logits
  save       the experts' saved state [a | b] in 8 bits with a scale for `cols` columns, and
             |phi|^2 of every pair
  load       its use in the backward pass: the pairs' scores, then the retained rows' gradient
             rows, [a | b] and phi (and the layer's input rows, where those are held in 8 bits too)
  norm       norm behind a block, gate, scaled residual and the norm in front of the next block
  norm_bwd   its gradients

Layer sizes are those of workloads/configs.py.
"""

import math

import torch

own = False

F8 = torch.float8_e4m3fn
F8_MAX = 448.0          # largest e4m3 value
AMAX_MIN = 2.0 ** -100  # group maxima are floored here, so that no scale is zero
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
EPS = 1e-6              # of the norms
BALANCE = 1e-2
SCALE = 2.5             # of the routing weights
RATE = 1e-3             # of the bias's steps
RES_SCALE = 0.8


def listed():
    return [
        # one token of a decoding user, routed alone over 8 groups: latency only
        {"name": "route_one_token", "op": "route", "T": 1, "E": 256, "groups": 8, "top_groups": 4,
         "group_top": 2, "K": 8, "dtype": "f32", "score": "sigmoid", "bias": True, "renorm": True,
         "stats": False, "pad": 0.0, "off": 0.0},
        # the full micro-batch of the 256-expert layer, 4 x 8192 tokens
        {"name": "route_t32k_e256_g8", "op": "route", "T": 32768, "E": 256, "groups": 8,
         "top_groups": 4, "group_top": 2, "K": 8, "dtype": "f32", "score": "sigmoid", "bias": True,
         "renorm": True, "stats": True, "pad": 0.0, "off": 0.0},
        # an odd number of tokens, padded sequences, experts switched off, softmax over 4 groups
        {"name": "route_t5003_e128_padded", "op": "route", "T": 5003, "E": 128, "groups": 4,
         "top_groups": 2, "group_top": 1, "K": 8, "dtype": "bf16", "score": "softmax",
         "bias": False, "renorm": False, "stats": True, "pad": 0.15, "off": 0.1},
        # the full micro-batch's gradient
        {"name": "route_bwd_t32k_e256_g8", "op": "route_bwd", "T": 32768, "E": 256, "groups": 8,
         "top_groups": 4, "group_top": 2, "K": 8, "dtype": "f32", "score": "sigmoid", "bias": True,
         "renorm": True, "pad": 0.0, "off": 0.0},
        # a short block of one sequence on a 512-column expert
        {"name": "save_t777_h512", "op": "save", "T": 777, "K": 8, "H": 512, "cols": 64,
         "dtype": "bf16"},
        # every pair of the full micro-batch of the 128-expert layer
        {"name": "save_t32k_h768", "op": "save", "T": 32768, "K": 8, "H": 768, "cols": 128,
         "dtype": "bf16"},
        # the wide layer's backward at half retention, its input read in place
        {"name": "load_t16k_d4096_h1408", "op": "load", "T": 16384, "D": 4096, "H": 1408, "E": 128,
         "K": 8, "cols": 128, "dtype": "bf16", "num": 1, "den": 2, "x8": False},
        # a short odd block, its input in 8 bits
        {"name": "load_t1021_d2048_h192", "op": "load", "T": 1021, "D": 2048, "H": 192, "E": 24,
         "K": 2, "cols": 64, "dtype": "bf16", "num": 3, "den": 5, "x8": True},
        # four decoding users: both norms, a gate for each user, 8-bit rows
        {"name": "norm_t4_d4096_q8", "op": "norm", "T": 4, "D": 4096, "dtype": "bf16",
         "block": "f32", "post": True, "gate": "token", "q_cols": 128},
        # the wide layer, the experts' float32 output, a gate for each column
        {"name": "norm_t16k_d4096", "op": "norm", "T": 16384, "D": 4096, "dtype": "bf16",
         "block": "f32", "post": True, "gate": "column", "q_cols": -1},
        # its gradients, the residual stream's in float32
        {"name": "norm_bwd_t16k_d4096", "op": "norm_bwd", "T": 16384, "D": 4096, "dtype": "bf16",
         "block": "f32", "grad": "f32", "post": True, "gate": "column", "stream": True},
        # an odd, short block of a 32-bit layer
        {"name": "norm_bwd_t1021_d2040_f32", "op": "norm_bwd", "T": 1021, "D": 2040,
         "dtype": "f32", "block": "f32", "grad": "f32", "post": True, "gate": "token",
         "stream": False},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route_bwd", "save", "load", "norm", "norm_bwd"])
    if op in ("route", "route_bwd"):
        groups = rng.choice([1, 2, 4, 8, 8, 16])
        size = rng.choice([32, 16, _log_uniform(rng, 2, 64)])
        while groups * size > 512:
            size //= 2
        top = rng.randint(1, groups)
        K = rng.randint(1, min(8, top * size))
        T = _log_uniform(rng, 1, 32768)
        while T * groups * size > 32768 * 256:
            T = max(1, T // 2)
        case = {"op": op, "T": T, "E": groups * size, "groups": groups, "top_groups": top,
                "group_top": rng.choice([1, 2]), "K": K, "dtype": rng.choice(["bf16", "f32"]),
                "score": rng.choice(["sigmoid", "sigmoid", "softmax"]),
                "bias": rng.random() < 0.7, "renorm": rng.random() < 0.6,
                "pad": rng.choice([0.0, 0.2]), "off": rng.choice([0.0, 0.1])}
        return {**case, "stats": rng.random() < 0.75} if op == "route" else case
    if op in ("save", "load"):
        K = rng.randint(1, 8)
        H = 8 * _log_uniform(rng, 2, 192)
        T = _log_uniform(rng, 1, 32768)
        case = {"op": op, "T": T, "K": K, "H": H, "cols": rng.choice([32, 64, 128]),
                "dtype": rng.choice(["bf16", "bf16", "f32"])}
        b = BYTES[case["dtype"]]
        if op == "save":
            while case["T"] * K * H * b > 32768 * 8 * 768 * 2:
                case["T"] = max(1, case["T"] // 2)
            return case
        E = _log_uniform(rng, max(K, 4), 256)
        D = 8 * _log_uniform(rng, 4, 512)
        num, den = rng.choice([(1, 4), (1, 2), (3, 5), (1, 1)])
        while case["T"] * K * (D + 3 * H) * b * num // den > 16384 * 4 * (4096 + 3 * 1408) * 2:
            case["T"] = max(1, case["T"] // 2)
        return {**case, "E": E, "D": D, "num": num, "den": den, "x8": rng.random() < 0.4}
    D = 8 * _log_uniform(rng, 4, 1024)
    T = _log_uniform(rng, 1, 32768)
    while T * D > 16384 * 4096:
        T = max(1, T // 2)
    case = {"op": op, "T": T, "D": D, "dtype": rng.choice(["bf16", "bf16", "f32"]),
            "block": rng.choice(["f32", "same"]), "post": rng.random() < 0.7,
            "gate": rng.choice(["none", "column", "token"])}
    if case["block"] == "same":
        case["block"] = case["dtype"]
    if op == "norm":
        return {**case, "q_cols": rng.choice([-1, -1, 0, 32, 64, 128])}
    return {**case, "grad": rng.choice(["f32", "bf16"]), "stream": rng.random() < 0.7}


# -- inputs -----------------------------------------------------------------------------------
def _logits(case, gen):
    T, E = case["T"], case["E"]
    dev = "cuda"
    e = torch.arange(E, device=dev, dtype=torch.float32)
    # some experts are liked more than others, wherever their group is
    x = torch.randn(T, E, generator=gen, device=dev) - 0.6 * torch.log(e * 37 % E + 1)
    if case["off"]:
        # experts that a token may not use; every 61st token may use none
        closed = torch.rand(T, E, generator=gen, device=dev) < case["off"]
        closed |= (torch.arange(T, device=dev) % 61 == 60)[:, None]
        x = x.masked_fill(closed, -math.inf)
    mask = None
    if case["pad"]:
        mask = (torch.rand(T, generator=gen, device=dev) >= case["pad"]).to(torch.uint8)
    return x.to(DT[case["dtype"]]), mask


def _dispatch(case, gen):
    """A routed token block and its retained pairs: perm, inv, off, alpha, keep, sel_off, sel_pos."""
    T, E, K = case["T"], case["E"], case["K"]
    dev, N = "cuda", case["T"] * case["K"]
    e = torch.arange(E, device=dev, dtype=torch.float32)
    x = torch.randn(T, E, generator=gen, device=dev) - 1.2 * torch.log(e + 1)
    w, idx = torch.sort(x, dim=1, descending=True)
    s = {"alpha": torch.exp(w[:, :K] - torch.logsumexp(x, 1, keepdim=True)).contiguous()}
    flat = idx[:, :K].reshape(-1)
    perm = torch.sort(flat, stable=True).indices
    inv = torch.empty(N, dtype=torch.int64, device=dev)
    inv[perm] = torch.arange(N, device=dev)
    counts = torch.bincount(flat, minlength=E)
    # each expert's share, the parts of a pair that are lost going to the largest of them
    M = -(-N * case["num"] // case["den"])
    quota, rest = counts * case["num"] // case["den"], counts * case["num"] % case["den"]
    largest = torch.sort(rest, descending=True, stable=True).indices
    quota[largest] += (torch.arange(E, device=dev) < M - quota.sum()).to(quota.dtype)
    # the retained pairs of an expert: those with the largest of some scores
    expert = flat[perm]
    order = torch.sort(torch.rand(N, generator=gen, device=dev), descending=True).indices
    order = order[torch.sort(expert[order], stable=True).indices]
    off = torch.cumsum(counts, 0) - counts
    rank = torch.arange(N, device=dev) - off[expert]
    keep = torch.zeros(N, dtype=torch.bool, device=dev)
    keep[order] = rank < quota[expert]
    s["perm"], s["inv"] = perm.to(torch.int32), inv.to(torch.int32)
    s["keep"] = keep.to(torch.uint8)
    s["sel_off"] = torch.cat([quota.new_zeros(1), torch.cumsum(quota, 0)]).to(torch.int32)
    s["rows"] = M
    s["sel_pos"] = torch.zeros(N, dtype=torch.int32, device=dev)
    s["sel_pos"][:M] = torch.nonzero(keep).view(-1).to(torch.int32)
    return s


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
        s["logits"], s["mask"] = _logits(case, gen)
        # what many steps of RATE have added up to
        bias = torch.randint(-60, 61, (E,), generator=gen, device=dev) * RATE
        s["bias"] = bias if case["bias"] else None
        if own:
            s["router"] = lib.GroupRouter(
                T, E, K, case["dtype"], score=case["score"], groups=case["groups"],
                top_groups=case["top_groups"], group_top=case["group_top"],
                renorm=case["renorm"], scale=SCALE, balance_coef=BALANCE)
        if op == "route_bwd":
            fwd = _plain_route({**s, "case": {**case, "stats": True, "bias": False}})
            s["topk_idx"], s["counts"] = fwd["topk_idx"], fwd["counts"]
            s["dalpha"] = randn(T, K)
            s["dloss"] = torch.ones(1, device=dev)
            if own:
                s["router"].topk_idx.copy_(s["topk_idx"])
                s["router"].counts.copy_(s["counts"])
        return s
    if op in ("save", "load"):
        T, K, H, dt = case["T"], case["K"], case["H"], DT[case["dtype"]]
        ab = torch.empty(T * K, 2 * H, device=dev).normal_(generator=gen)
        # pairs of very different size
        ab *= torch.exp(0.5 * randn(T * K, 1))
        ab = ab.to(dt)
        if op == "save":
            s["ab"] = ab
            if own:
                s["packed"] = lib.PackedState(T, K, H, case["dtype"], cols=case["cols"])
            return s
        D, E = case["D"], case["E"]
        s |= _plain_save({"case": case, "ab": ab})
        s |= _dispatch(case, gen)
        s["g"] = (randn(T, D) * torch.exp(0.5 * randn(T, 1))).to(dt)
        s["x"] = s["x_scale"] = None
        if case["x8"]:
            s["x"], s["x_scale"] = _quantise(randn(T, D), 128)
        if own:
            s["packed"] = lib.PackedState(T, K, H, case["dtype"], cols=case["cols"])
            s["packed"].q.copy_(s["q"])
            s["packed"].scale.copy_(s["scale"])
            s["packed"].phi_sq.copy_(s["phi_sq"])
            s["lrm"] = lib.lrm
            s["shape"] = lib.lrm.make_shape(T, D, H, E, K, lib.dtype_code(case["dtype"]))
            s["ws_bytes"] = lib.lrm.lrm_workspace_bytes(s["shape"])
            s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device=dev)
            lib.lrm.lrm_clear_device_error(s["ws"], s["ws_bytes"])
            N = T * K
            s["score"] = torch.empty(N, device=dev)
            s["tok_c"] = torch.empty(N, dtype=torch.int32, device=dev)
            s["row_of_pos"] = torch.empty(N, dtype=torch.int32, device=dev)
            for name, cols in (("dy_c", D), ("ab_c", 2 * H), ("phi_c", H)):
                s[name] = torch.empty(N, cols, dtype=dt, device=dev)
            s["x_c"] = torch.empty(N, D, dtype=dt, device=dev) if case["x8"] else None
        return s
    T, D, dt, bt = case["T"], case["D"], DT[case["dtype"]], DT[case["block"]]
    s["w"] = (1 + 0.1 * randn(D)).to(dt)
    s["w_post"] = (1 + 0.1 * randn(D)).to(dt) if case["post"] else None
    s["gate"] = None
    if case["gate"] != "none":
        n = D if case["gate"] == "column" else T
        s["gate"] = (0.5 + 0.3 * randn(n)).to(dt)
    # a residual stream has columns of very different size
    cols = torch.exp(0.7 * randn(D))
    s["block"] = (randn(T, D) * 0.3).to(bt)
    s["res"] = (randn(T, D) * cols).to(dt)
    if own:
        q = None if case.get("q_cols", -1) < 0 else case["q_cols"]
        s["norm"] = lib.BlockNorm(T, D, case["dtype"], block_dtype=case["block"],
                                  gate=None if case["gate"] == "none" else case["gate"],
                                  post=case["post"], residual_scale=RES_SCALE, eps=EPS, q_cols=q,
                                  grad_dtype=case.get("grad", "f32"))
    if op == "norm_bwd":
        gt = DT[case["grad"]]
        fwd = _plain_norm({**s, "case": {**case, "q_cols": -1}})
        s["h"], s["rstd"] = fwd["h"], fwd["rstd"]
        s["block_rstd"] = fwd.get("block_rstd")
        s["dy"] = (randn(T, D) * 1e-2).to(gt)
        s["dh"] = (randn(T, D) * 1e-2).to(gt) if case["stream"] else None
        if own:
            s["norm"].rstd.copy_(s["rstd"])
            if case["post"]:
                s["norm"].block_rstd.copy_(s["block_rstd"])
    return s


# -- plain forms ------------------------------------------------------------------------------
def _scores(x, score, use):
    """Scores in 64 bits (which of two near ones is larger decides a choice), 0 for tokens that
    take no part."""
    if score == "sigmoid":
        s = 1 / (1 + torch.exp(-x))
    else:
        top = torch.where(use, x.amax(1), torch.zeros_like(x[:, 0]))[:, None]
        ex = torch.exp(x - top)
        total = ex.sum(1, keepdim=True)
        s = ex / torch.where(total == 0, torch.ones_like(total), total)
    return torch.where(use[:, None], s, torch.zeros_like(s))


def _usable(x, mask):
    """Tokens that take part: not padding, and with at least one expert open."""
    some = (x > -math.inf).any(1)
    return some if mask is None else some & (mask != 0)


def _plain_route(s):
    c = s["case"]
    T, E, G, K = c["T"], c["E"], c["groups"], c["K"]
    x = s["logits"].double()
    use = _usable(x, s["mask"])
    some = (x > -math.inf).any(1)
    score = _scores(x, c["score"], some)
    key = score if s["bias"] is None else score + s["bias"].double()
    shut = x == -math.inf
    if G > 1:
        top = torch.sort(key.masked_fill(shut, -math.inf).view(T, G, E // G), dim=2,
                         descending=True).values[:, :, :c["group_top"]]
        rank = torch.where(top == -math.inf, torch.zeros_like(top), top).sum(2)
        rank = rank.masked_fill(shut.view(T, G, E // G).all(2), -math.inf)
        order = torch.sort(rank, dim=1, descending=True, stable=True).indices
        kept = torch.zeros(T, G, dtype=torch.bool, device=x.device)
        kept.scatter_(1, order[:, :c["top_groups"]], True)
        kept = kept[:, :, None].expand(T, G, E // G).reshape(T, E)
    else:
        kept = torch.ones_like(shut)
    # without a bias a larger logit is a larger score
    key = x if s["bias"] is None else key.masked_fill(shut, -math.inf)
    first = torch.sort(key, dim=1, descending=True, stable=True).indices
    first = first.gather(1, torch.sort((~kept).gather(1, first).to(torch.uint8), dim=1,
                                       stable=True).indices)
    idx = first[:, :K]
    a = score.gather(1, idx)
    if c["renorm"]:
        total = a.sum(1, keepdim=True)
        a = a / torch.where(total == 0, torch.ones_like(total), total)
    a = torch.where(use[:, None], a * SCALE, torch.zeros_like(a))
    out = {"topk_idx": idx.to(torch.int32), "alpha": a.float()}
    if c["stats"]:
        chosen = torch.zeros_like(x, dtype=torch.int32).scatter_(1, idx, 1) * use[:, None]
        counts, n = chosen.sum(0).to(torch.int32), use.sum().clamp_min(1)
        p = torch.where(use[:, None], score, torch.zeros_like(score)).float()
        total = p.sum(1, keepdim=True)
        psum = (p / torch.where(total == 0, torch.ones_like(total), total)).sum(0)
        out |= {"counts": counts, "prob_sum": psum,
                "loss": (BALANCE * E * (counts * psum).sum() / (n.float().square() * K))[None]}
        if c["bias"]:
            lack = counts.sum().long() - E * counts.long()
            out["bias"] = s["bias"] + RATE * torch.sign(lack).float()
    return out


def _plain_route_bwd(s):
    c = s["case"]
    x, idx, E, K = s["logits"].float(), s["topk_idx"].long(), c["E"], c["K"]
    use = _usable(x, s["mask"])
    p = _scores(s["logits"].double(), c["score"], use).float()
    n = use.sum().clamp_min(1).float()
    chosen, da = p.gather(1, idx), s["dalpha"] * SCALE
    if c["renorm"]:
        total = chosen.sum(1, keepdim=True)
        total = torch.where(total == 0, torch.ones_like(total), total)
        da = (da - (chosen * da).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(x).scatter_(1, idx, da)
    total = p.sum(1, keepdim=True)
    total = torch.where(total == 0, torch.ones_like(total), total)
    cost = s["dloss"][0] * BALANCE * E * s["counts"].float() / (n * n * K)
    ds = ds + (cost - (p * cost).sum(1, keepdim=True) / total) / total
    if c["score"] == "sigmoid":
        less = _scores(-s["logits"].double(), "sigmoid", use).float()
        dx = ds * p * less
    else:
        dx = p * (ds - (p * ds).sum(1, keepdim=True))
    return {"dlogits": torch.where(use[:, None], dx, torch.zeros_like(dx)).to(s["logits"].dtype)}


def _quantise(v, cols):
    """e4m3 codes and scales of each `cols` columns of the rows of v (0: of a row)."""
    rows, width = v.shape
    cols = cols or width
    groups = -(-width // cols)
    b = torch.nn.functional.pad(v, (0, groups * cols - width)).view(rows, groups, cols)
    amax = b.abs().amax(2).clamp_min(AMAX_MIN)
    q = (b * F8_MAX / amax[:, :, None]).view(rows, groups * cols)[:, :width]
    return q.to(F8).contiguous(), amax / F8_MAX


def _decode(q, scale, cols):
    return q.float() * scale.repeat_interleave(cols, 1)[:, :q.shape[1]]


def _phi(a, b):
    return a / (1 + torch.exp(-a)) * b


def _plain_save(s):
    c = s["case"]
    H, cols = c["H"], c["cols"]
    a, b = s["ab"][:, :H].float(), s["ab"][:, H:].float()
    (qa, sa), (qb, sb) = _quantise(a, cols), _quantise(b, cols)
    return {"q": torch.cat([qa.view(torch.uint8), qb.view(torch.uint8)], 1).view(F8),
            "scale": torch.cat([sa, sb], 1), "phi_sq": _phi(a, b).square().sum(1)}


def _plain_load(s):
    c = s["case"]
    T, K, H, cols, dt = c["T"], c["K"], c["H"], c["cols"], DT[c["dtype"]]
    M, N, G = s["rows"], c["T"] * c["K"], s["scale"].shape[1] // 2
    norm = s["g"].float().square().sum(1)
    pair = s["perm"].long()
    score = s["alpha"].view(-1)[pair].square() * norm[pair // K] * s["phi_sq"]
    pos = s["sel_pos"][:M].long()
    u = pair[pos]
    t = u // K
    dy = s["g"][t].float() * s["alpha"].view(-1)[u][:, None]
    q, sc = s["q"].view(torch.uint8)[pos].view(F8), s["scale"][pos]
    a, b = _decode(q[:, :H], sc[:, :G], cols), _decode(q[:, H:], sc[:, G:], cols)
    row = torch.full((N,), -1, dtype=torch.int32, device="cuda")
    row[pos] = torch.arange(M, dtype=torch.int32, device="cuda")
    out = {"score": score, "dy_c": dy.to(dt), "ab_c": torch.cat([a, b], 1).to(dt),
           "phi_c": _phi(a, b).to(dt), "tok_c": t.to(torch.int32), "row_of_pos": row}
    if c["x8"]:
        out["x_c"] = _decode(s["x"].view(torch.uint8)[t].view(F8), s["x_scale"][t], 128).to(dt)
    return out


def _gate(s):
    if s["gate"] is None:
        return 1.0
    g = s["gate"].float()
    return g[:, None] if s["case"]["gate"] == "token" else g


def _plain_norm(s):
    c = s["case"]
    u, out = s["block"].float(), {}
    if c["post"]:
        rs = torch.rsqrt(u.square().mean(1) + EPS)
        u = u * rs[:, None] * s["w_post"].float()
        out["block_rstd"] = rs
    h = RES_SCALE * s["res"].float() + _gate(s) * u
    rstd = torch.rsqrt(h.square().mean(1) + EPS)
    y = h * rstd[:, None] * s["w"].float()
    out |= {"h": h.to(s["res"].dtype), "rstd": rstd}
    if c["q_cols"] < 0:
        out["y"] = y.to(s["res"].dtype)
    else:
        out["q"], out["q_scale"] = _quantise(y, c["q_cols"])
    return out


def _plain_norm_bwd(s):
    c = s["case"]
    h, dy, rstd = s["h"].float(), s["dy"].float(), s["rstd"][:, None]
    xhat = h * rstd
    wdy = dy * s["w"].float()
    dh = rstd * (wdy - xhat * (wdy * xhat).mean(1, keepdim=True))
    if s["dh"] is not None:
        dh = dh + s["dh"].float()
    out = {"dres": (RES_SCALE * dh).to(s["dy"].dtype), "dw": (dy * xhat).sum(0)}
    o = s["block"].float()
    if c["post"]:
        o = o * s["block_rstd"][:, None]
    u = o * s["w_post"].float() if c["post"] else o
    if s["gate"] is not None:
        out["dgate"] = (dh * u).sum(1 if c["gate"] == "token" else 0)
    du = dh * _gate(s)
    if c["post"]:
        out["dw_post"] = (du * o).sum(0)
        du = du * s["w_post"].float()
        du = s["block_rstd"][:, None] * (du - o * (du * o).mean(1, keepdim=True))
    out["dblock"] = du.to(s["res"].dtype)
    return out


_PLAIN = {"route": _plain_route, "route_bwd": _plain_route_bwd, "save": _plain_save,
          "load": _plain_load, "norm": _plain_norm, "norm_bwd": _plain_norm_bwd}


# -- one pass ---------------------------------------------------------------------------------
def run(state):
    s = state
    if not own:
        return _PLAIN[s["case"]["op"]](s)
    c = s["case"]
    op = c["op"]
    if op == "route":
        r = s["router"]
        r.route(s["logits"], bias=s["bias"], mask=s["mask"], stats=c["stats"])
        out = {"topk_idx": r.topk_idx, "alpha": r.alpha}
        if c["stats"]:
            out |= {"counts": r.counts, "prob_sum": r.prob_sum, "loss": r.loss}
            if c["bias"]:
                out["bias"] = r.next_bias(s["bias"], RATE)
        return out
    if op == "route_bwd":
        r = s["router"]
        r.backward(s["logits"], s["dalpha"], mask=s["mask"], dloss=s["dloss"])
        return {"dlogits": r.dlogits}
    if op == "save":
        p = s["packed"]
        p.pack(s["ab"])
        return {"q": p.q, "scale": p.scale, "phi_sq": p.phi_sq}
    if op == "load":
        L, p = s["lrm"], s["packed"].desc
        L.lrm_score_packed(s["shape"], p, s["g"], s["alpha"], s["inv"], s["score"], s["ws"],
                           s["ws_bytes"])
        L.lrm_compact_packed(s["shape"], p, s["perm"], s["keep"], s["sel_off"], s["sel_pos"],
                             s["alpha"], s["x"], s["x_scale"], 128, s["g"], s["dy_c"], s["x_c"],
                             s["ab_c"], s["phi_c"], s["tok_c"], s["row_of_pos"], s["ws"],
                             s["ws_bytes"])
        M = s["rows"]  # the buffers hold every pair, the retained rows come first
        out = {k: s[k][:M] for k in ("dy_c", "ab_c", "phi_c", "tok_c")}
        out |= {"score": s["score"], "row_of_pos": s["row_of_pos"]}
        if c["x8"]:
            out["x_c"] = s["x_c"][:M]
        return out
    n = s["norm"]
    if op == "norm":
        n.forward(s["block"], s["res"], s["w"], w_post=s["w_post"], gate=s["gate"])
        out = {"h": n.h, "rstd": n.rstd}
        if c["post"]:
            out["block_rstd"] = n.block_rstd
        if c["q_cols"] < 0:
            out["y"] = n.y
        else:
            out["q"], out["q_scale"] = n.q, n.q_scale
        return out
    n.backward(s["dy"], s["block"], s["w"], w_post=s["w_post"], gate=s["gate"], dh=s["dh"],
               h=s["h"])
    out = {"dres": n.dres, "dblock": n.dblock, "dw": n.dw}
    if c["post"]:
        out["dw_post"] = n.dw_post
    if c["gate"] != "none":
        out["dgate"] = n.dgate
    return out


def work(case):
    op = case["op"]
    if op in ("route", "route_bwd"):
        T, E, K = case["T"], case["E"], case["K"]
        b = BYTES[case["dtype"]]
        mask = T if case["pad"] else 0
        if op == "route":
            # logits once, the bias; an index and a weight for each pair; the statistics
            extra = 4 * E if case["bias"] else 0
            if case["stats"]:
                extra += 8 * E + 4 + (4 * E if case["bias"] else 0)
            return {"bytes": T * E * b + mask + 8 * T * K + extra, "flops": 6 * T * E}
        return {"bytes": 2 * T * E * b + mask + 8 * T * K + 4 * E, "flops": 12 * T * E}
    if op in ("save", "load"):
        N, K, H, b = case["T"] * case["K"], case["K"], case["H"], BYTES[case["dtype"]]
        groups = -(-H // case["cols"])
        if op == "save":
            return {"bytes": N * (2 * H * b + 2 * H + 8 * groups + 4), "flops": 14 * N * H}
        T, D = case["T"], case["D"]
        M = -(-N * case["num"] // case["den"])
        # cotangent, pair data; codes and scales of the retained rows; scores, rows and maps
        read = T * D * b + N * 17 + M * (2 * H + 8 * groups + 4)
        write = N * 8 + M * ((D + 3 * H) * b + 4)
        if case["x8"]:
            read, write = read + T * (D + 4 * -(-D // 128)), write + M * D * b
        return {"bytes": read + write, "flops": 2 * T * D + M * (D + 8 * H)}
    T, D = case["T"], case["D"]
    b, o = BYTES[case["dtype"]], BYTES[case["block"]]
    gate = {"none": 0, "column": D, "token": T}[case["gate"]]
    vectors = D * b * (2 if case["post"] else 1) + gate * b + 4 * T * (2 if case["post"] else 1)
    if op == "norm":
        if case["q_cols"] < 0:
            y = T * D * b
        else:
            y = T * D + 4 * T * -(-D // (case["q_cols"] or D))
        return {"bytes": T * D * (o + 2 * b) + y + vectors, "flops": 12 * T * D}
    g = BYTES[case["grad"]]
    rows = o + b + 2 * g + b + (g if case["stream"] else 0)
    sums = 4 * (D * (2 if case["post"] else 1) + gate)
    return {"bytes": T * D * rows + vectors + sums, "flops": 24 * T * D}


# -- the same in 64 bits ----------------------------------------------------------------------
def _exact_router(case, x, bias, mask, idx=None):
    """Choices, weights (differentiable in x), counts, the scores' sums and the balance loss."""
    T, E, G, K = case["T"], case["E"], case["groups"], case["K"]
    v = x.detach()
    open_ = ~torch.isneginf(v)
    some = open_.any(1)
    use = some if mask is None else some & mask.bool()
    safe = torch.where(some[:, None], x, torch.zeros_like(x))
    if case["score"] == "softmax":
        score = torch.softmax(safe, 1)
    else:
        score = torch.sigmoid(safe)
    score = score * some[:, None]
    if idx is None:
        key = score.detach() if bias is None else score.detach() + bias.double()
        low = torch.full_like(key, -math.inf)
        key = torch.where(open_, key, low)
        blocks = key.view(T, G, E // G)
        best = blocks.amax(2)
        if case["group_top"] == 2 and E > G:
            second = torch.kthvalue(-blocks, 2, dim=2).values.neg()
            best = best + torch.where(torch.isneginf(second), torch.zeros_like(second), second)
        # a group's place: how many others come before it
        g = torch.arange(G, device=x.device)
        mine, other = best[:, :, None], best[:, None, :]
        before = (other > mine) | ((other == mine) & (g[None, :] < g[:, None])[None])
        kept = (before.sum(2) < case["top_groups"]).repeat_interleave(E // G, 1)
        key = torch.where(open_, v if bias is None else key, low)
        # experts of other groups come last, behind the closed ones of the kept
        place = torch.argsort(-key, dim=1, stable=True)
        late = (~kept).gather(1, place).long() * E + torch.arange(E, device=x.device)
        idx = place.gather(1, torch.argsort(late, dim=1))[:, :K]
    a = score.gather(1, idx)
    if case["renorm"]:
        total = a.sum(1, keepdim=True)
        a = a / torch.where(total > 0, total, torch.ones_like(total))
    a = SCALE * a * use[:, None]
    n = max(1, int(use.sum()))
    counts = torch.bincount(idx[use].reshape(-1), minlength=E)
    total = score.sum(1, keepdim=True)
    share = score / torch.where(total > 0, total, torch.ones_like(total)) * use[:, None]
    loss = BALANCE * E * ((counts.double() / (n * K)) * (share.sum(0) / n)).sum()
    return idx, a, counts, share.sum(0), loss


def _exact_codes(v, cols):
    q, scales = torch.empty_like(v), []
    for lo in range(0, v.shape[1], cols):
        part = v[:, lo:lo + cols]
        scale = part.abs().max(1).values.clamp_min(AMAX_MIN) / F8_MAX
        q[:, lo:lo + cols] = (part / scale[:, None]).float().to(F8).double()
        scales.append(scale)
    return q, torch.stack(scales, 1)


def _exact_norm(case, s, block, res, w, w_post, gate):
    u, rs = block, None
    if case["post"]:
        rs = 1 / torch.sqrt((block * block).sum(1) / case["D"] + EPS)
        u = block * rs[:, None] * w_post[None, :]
    if gate is not None:
        u = u * (gate[:, None] if case["gate"] == "token" else gate[None, :])
    h = RES_SCALE * res + u
    rstd = 1 / torch.sqrt((h * h).sum(1) / case["D"] + EPS)
    return rs, h, rstd, h * rstd[:, None] * w[None, :]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "route":
        idx, a, counts, psum, loss = _exact_router(case, s["logits"].double(), s["bias"], s["mask"])
        out = {"topk_idx": idx.to(torch.int32), "alpha": a}
        if case["stats"]:
            out |= {"counts": counts.to(torch.int32), "prob_sum": psum, "loss": loss[None]}
            if case["bias"]:
                mean = counts.double().mean()
                up, down = counts.double() < mean, counts.double() > mean
                out["bias"] = s["bias"].double() + RATE * (up.double() - down.double())
        return out
    if op == "route_bwd":
        x = s["logits"].double().requires_grad_(True)
        _, a, _, _, loss = _exact_router(case, x, None, s["mask"], idx=s["topk_idx"].long())
        total = (a * s["dalpha"].double()).sum() + s["dloss"][0].double() * loss
        total.backward()
        return {"dlogits": x.grad}
    if op == "save":
        H = case["H"]
        ab = s["ab"]
        qa, sa = _exact_codes(ab[:, :H].double(), case["cols"])
        qb, sb = _exact_codes(ab[:, H:].double(), case["cols"])
        sq = []
        for part in ab.split(1 << 16):
            phi = torch.nn.functional.silu(part[:, :H].double()) * part[:, H:].double()
            sq.append((phi * phi).sum(1))
        return {"q": torch.cat([qa, qb], 1), "scale": torch.cat([sa, sb], 1),
                "phi_sq": torch.cat(sq)}
    if op == "load":
        K, H, M, N = case["K"], case["H"], s["rows"], case["T"] * case["K"]
        alpha, g = s["alpha"].double().view(-1), s["g"].double()
        norm = torch.einsum("td,td->t", g, g)
        by_pair = alpha ** 2 * norm.repeat_interleave(K)
        score = torch.empty(N, dtype=torch.float64, device="cuda")
        score[s["inv"].long()] = by_pair
        score *= s["phi_sq"].double()
        pos = torch.nonzero(s["keep"]).view(-1)
        u = s["perm"][pos].long()
        t = torch.div(u, K, rounding_mode="floor")
        col = torch.arange(H, device="cuda") // case["cols"]
        G = s["scale"].shape[1] // 2
        sc = s["scale"].double()
        a = s["q"][:, :H].float().double()[pos] * sc[:, :G][:, col][pos]
        b = s["q"][:, H:].float().double()[pos] * sc[:, G:][:, col][pos]
        row = torch.full((N,), -1, dtype=torch.int32, device="cuda")
        row[pos] = torch.arange(M, dtype=torch.int32, device="cuda")
        out = {"score": score, "dy_c": alpha[u][:, None] * g[t], "ab_c": torch.cat([a, b], 1),
               "phi_c": torch.nn.functional.silu(a) * b, "tok_c": t.to(torch.int32),
               "row_of_pos": row}
        if case["x8"]:
            wide = torch.arange(case["D"], device="cuda") // 128
            x = s["x"].float().double() * s["x_scale"].double()[:, wide]
            out["x_c"] = x[t]
        return out
    names = ["block", "res", "w", "w_post", "gate"]
    v = {k: None if s[k] is None else s[k].double() for k in names}
    if op == "norm":
        rs, h, rstd, y = _exact_norm(case, s, *(v[k] for k in names))
        out = {"h": h, "rstd": rstd}
        if case["post"]:
            out["block_rstd"] = rs
        if case["q_cols"] < 0:
            out["y"] = y
        else:
            out["q"], out["q_scale"] = _exact_codes(y, case["q_cols"] or case["D"])
        return out
    # the gradients as functions of the given h and the two given 1/rms
    D, h, dy, rstd, w = case["D"], s["h"].double(), s["dy"].double(), s["rstd"].double(), v["w"]
    dot = torch.einsum("td,td,d->t", h, dy, w)
    dh = dy * w * rstd[:, None] - h * (dot * rstd ** 3 / D)[:, None]
    if s["dh"] is not None:
        dh = dh + s["dh"].double()
    out = {"dres": RES_SCALE * dh, "dw": torch.einsum("td,td,t->d", h, dy, rstd)}
    block, rs = v["block"], s["block_rstd"].double() if case["post"] else None
    post = rs[:, None] * v["w_post"][None, :] if case["post"] else 1.0
    gate = 1.0
    if v["gate"] is not None:
        gate = v["gate"][:, None] if case["gate"] == "token" else v["gate"][None, :]
        out["dgate"] = (dh * block * post).sum(1 if case["gate"] == "token" else 0)
    if case["post"]:
        out["dw_post"] = (dh * gate * block * rs[:, None]).sum(0)
        dot = (dh * gate * block * v["w_post"]).sum(1)
        out["dblock"] = dh * gate * post - block * (dot * rs ** 3 / D)[:, None]
    else:
        out["dblock"] = dh * gate
    return out
