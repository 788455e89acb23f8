"""More operators around the expert layer, as measured cases.

  route      moe_route_scores: top-k experts of every token by softmax or
             sigmoid scores, with a bias that only the choice sees, groups of
             experts of which a few are kept, and weights that are
             renormalised and scaled.
  route_grad moe_route_scores_backward: the gradient of the router's logits
             through those weights.
  linear     moe_int8_linear: rows of bf16, quantised inside with one scale per
             row, times 8-bit integer weights with one scale per output channel.
  experts    moe_int8_experts: the expert MLPs (gate/up product, SwiGLU, down
             product) of routed, expert-sorted tokens on such weights.
  norm       moe_combine_norm: the end of an expert block: weighted top-k sum,
             the shared expert with its gate, a norm of the sum, the scaled
             residual addition and the next block's norm.
  norm_grad  moe_combine_norm_backward: the gradients of all of its inputs.

`own = False` computes each from elementary torch operations; `own = True`
calls the library.
"""
import math

import torch

own = False

DEV = "cuda"
I8_MAX = 127.0
TINY = 2.0 ** -100  # smallest magnitude that sets a row's scale


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one decoded token's routing, 8 groups of 32 experts of which 4 are kept: latency counts
        {"name": "route t1 e256", "op": "route", "T": 1, "E": 256, "k": 8, "score": "sigmoid", "bias": True, "G": 8,
         "KG": 4, "top": 2, "renorm": True, "scale": 2.5, "off": 0},
        # the same router over a long prompt, with a few experts switched off
        {"name": "route t16384 e256", "op": "route", "T": 16384, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "G": 8, "KG": 4, "top": 2, "renorm": True, "scale": 2.5, "off": 3},
        # a small padded training batch, softmax over all experts without renormalising: a dense gradient
        {"name": "route_grad t500 e64", "op": "route_grad", "T": 500, "E": 64, "k": 6, "score": "softmax",
         "renorm": False, "scale": 1.0, "masked": True},
        # a large training batch, sigmoid scores renormalised
        {"name": "route_grad t32768 e256", "op": "route_grad", "T": 32768, "E": 256, "k": 8, "score": "sigmoid",
         "renorm": True, "scale": 2.5, "masked": False},
        # an odd decode batch through a gate/up-sized projection
        {"name": "linear m33 2816x4096", "op": "linear", "M": 33, "N": 2816, "K": 4096},
        # a prompt of 8192 tokens through a gate/up-sized projection
        {"name": "linear m8192 4096x7168", "op": "linear", "M": 8192, "N": 4096, "K": 7168},
        # one decoded token through its 8 of 256 experts
        {"name": "experts t1 e256", "op": "experts", "T": 1, "H": 7168, "I": 2048, "E": 256, "k": 8, "skew": 0.0},
        # a prompt of 8192 tokens
        {"name": "experts t8192 e256", "op": "experts", "T": 8192, "H": 7168, "I": 2048, "E": 256, "k": 8, "skew": 0.25},
        # the end of an expert block for one decoded token
        {"name": "norm t1 h7168", "op": "norm", "T": 1, "H": 7168, "k": 8, "shared": True, "gate": False, "post": False,
         "next": True, "residual": True, "scale": 1.0},
        # for a prompt of 8192 tokens, with a gated shared expert and norms on both sides
        {"name": "norm t8192 h7168", "op": "norm", "T": 8192, "H": 7168, "k": 8, "shared": True, "gate": True,
         "post": True, "next": True, "residual": True, "scale": 0.5},
        # the gradients of an odd training batch on a smaller layer without a norm of the sum
        {"name": "norm_grad t333 h4096", "op": "norm_grad", "T": 333, "H": 4096, "k": 6, "shared": True, "gate": True,
         "post": False, "next": True, "residual": True, "scale": 1.0},
        # and those of a large one with everything
        {"name": "norm_grad t8192 h7168", "op": "norm_grad", "T": 8192, "H": 7168, "k": 8, "shared": True, "gate": True,
         "post": True, "next": True, "residual": True, "scale": 0.5},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "linear", "experts", "norm", "norm_grad"])
    if op == "route" or op == "route_grad":
        G, per = rng.choice([(1, _log_int(rng, 4, 512)), (4, rng.randint(2, 40)), (8, 32), (8, 20), (16, 16), (6, 10)])
        E = G * per
        KG = rng.randint(max(1, G // 4), G)
        T = _log_int(rng, 1, (16384 if op == "route" else 32768) * 256 // max(E, 256))
        case = {"op": op, "T": T, "E": E, "k": rng.randint(1, min(KG * per, 10)),
                "score": rng.choice(["softmax", "sigmoid"]), "renorm": rng.random() < 0.7,
                "scale": rng.choice([1.0, 2.5, 0.75])}
        if op == "route_grad":
            return {**case, "masked": rng.random() < 0.5}
        return {**case, "bias": rng.random() < 0.7, "G": G, "KG": KG, "top": rng.choice([1, 2]),
                "off": rng.choice([0, 0, 1, 2])}
    if op == "linear":
        return {"op": op, "M": _log_int(rng, 1, 8192), "N": _log_int(rng, 64, 4096), "K": 16 * _log_int(rng, 8, 448)}
    if op == "experts":
        H, I, E, k = rng.choice([(7168, 2048, 32, 8), (4096, 1408, 64, 6), (2048, 1024, 128, 8), (1024, 512, 16, 2),
                                 (2048, 768, 60, 4)])
        return {"op": op, "T": _log_int(rng, 1, 4096), "H": H, "I": I, "E": E, "k": k,
                "skew": round(rng.uniform(0.0, 1.0), 2)}
    H, k = 8 * _log_int(rng, 16, 896), rng.choice([0, 1, 2, 4, 6, 8, 10])
    shared = k == 0 or rng.random() < 0.6
    return {"op": op, "T": _log_int(rng, 1, min(16384, 8192 * 9 * 7168 // (H * (k + 1)))), "H": H, "k": k,
            "shared": shared, "gate": shared and rng.random() < 0.5, "post": rng.random() < 0.5,
            "next": rng.random() < 0.7, "residual": k > 0 or rng.random() < 0.7, "scale": rng.choice([1.0, 0.5, 0.22])}


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _hidden(T, K, g):
    """Hidden states: N(0, 1) with a hundredth of the channels ten times as large."""
    wide = 1.0 + 9.0 * (torch.rand(K, generator=g, device=DEV) < 0.01).float()
    return (torch.randn(T, K, generator=g, device=DEV) * wide).to(torch.bfloat16)


def _weights(count, N, K, g):
    """Codes and scales of weights of about N(0, 0.02): a channel's codes fill the range up to about 4 sigma."""
    w = torch.randn(count, N, K, generator=g, device=DEV, dtype=torch.bfloat16)
    codes = w.mul_(30.0).clamp_(-127.0, 127.0).round_().to(torch.int8)
    return codes, 7e-4 * (0.5 + torch.rand(count, N, generator=g, device=DEV))


def _logits(T, E, spread, g):
    return torch.randn(T, E, generator=g, device=DEV) + spread * torch.randn(E, generator=g, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case)
    bf16 = torch.bfloat16
    if op in ("route", "route_grad"):
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = 2.0 * _logits(T, E, 0.5, g)
        s["topk_ids"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
        if op == "route":
            s["bias_e"] = 0.1 * torch.randn(E, generator=g, device=DEV) if case["bias"] else None
            if case["off"]:  # experts that are switched off for all tokens
                s["logits"][:, torch.randperm(E, generator=g, device=DEV)[:min(case["off"], E - k)]] = -math.inf
            s["topk_w"] = torch.empty(T, k, device=DEV)
        else:
            s["topk_ids"] = torch.topk(s["logits"], k, dim=1).indices.to(torch.int32)
            s["d_topk_w"] = torch.randn(T, k, generator=g, device=DEV) / T
            s["mask"] = (torch.rand(T, generator=g, device=DEV) < 0.8).to(torch.uint8) if case["masked"] else None
            s["d_logits"] = torch.empty(T, E, device=DEV)
    elif op == "linear":
        codes, scales = _weights(1, case["N"], case["K"], g)
        s.update(codes=codes[0], scales=scales[0], x=_hidden(case["M"], case["K"], g),
                 out=torch.empty(case["M"], case["N"], dtype=bf16, device=DEV))
    elif op == "experts":
        T, H, I, E, k = (case[n] for n in "THIEk")
        flat = torch.topk(_logits(T, E, case["skew"], g), k, dim=1).indices.reshape(-1)
        counts = torch.bincount(flat, minlength=E)
        offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
        offsets[1:] = torch.cumsum(counts, 0)
        s["w13"], s["s13"] = _weights(E, 2 * I, H, g)
        s["w2"], s["s2"] = _weights(E, H, I, g)
        s.update(x=_hidden(T, H, g), offsets=offsets, sorted_pairs=torch.argsort(flat, stable=True).to(torch.int32),
                 max_rows=int(counts.max()), out=torch.empty(T * k, H, dtype=bf16, device=DEV))
    else:
        T, H, k = case["T"], case["H"], case["k"]
        s["y"] = torch.randn(T * k, H, generator=g, device=DEV, dtype=bf16) if k else None
        s["topk_w"] = torch.softmax(torch.randn(T, k, generator=g, device=DEV), dim=1) if k else None
        s["shared_x"] = torch.randn(T, H, generator=g, device=DEV, dtype=bf16) if case["shared"] else None
        s["gate_t"] = torch.sigmoid(torch.randn(T, generator=g, device=DEV)) if case["gate"] else None
        s["post_w"] = (1.0 + 0.2 * torch.randn(H, generator=g, device=DEV)).to(bf16) if case["post"] else None
        s["next_w"] = (1.0 + 0.2 * torch.randn(H, generator=g, device=DEV)).to(bf16) if case["next"] else None
        # the residual stream: a few channels far above the rest
        s["res"] = _hidden(T, H, g) if case["residual"] else None
        s["eps"] = 1e-6
        if op == "norm":
            s["out"] = torch.empty(T, H, dtype=bf16, device=DEV)
            s["normed"] = torch.empty(T, H, dtype=bf16, device=DEV) if case["next"] else None
        else:
            s["out"] = _hidden(T, H, g)  # what the forward pass left
            s["d_out"] = torch.randn(T, H, generator=g, device=DEV, dtype=bf16)
            s["d_normed"] = torch.randn(T, H, generator=g, device=DEV, dtype=bf16) if case["next"] else None
            s["d_res"] = torch.empty(T, H, dtype=bf16, device=DEV) if case["residual"] else None
            s["d_y"] = torch.empty(T * k, H, dtype=bf16, device=DEV) if k else None
            s["d_topk_w"] = torch.empty(T, k, device=DEV) if k else None
            s["d_shared"] = torch.empty(T, H, dtype=bf16, device=DEV) if case["shared"] else None
            s["d_gate"] = torch.empty(T, device=DEV) if case["gate"] else None
            s["d_post_w"] = torch.empty(H, device=DEV) if case["post"] else None
            s["d_next_w"] = torch.empty(H, device=DEV) if case["next"] else None
    return s


# ------------------------------------------------------------------ plain forms


def _scores(s):
    """Scores in 64 bits: which of two experts is chosen hangs on the last of their 32."""
    z = s["logits"].double()
    if s["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-z))
    p = torch.exp(z - z.amax(dim=1, keepdim=True))
    return p / p.sum(dim=1, keepdim=True)


def _route_plain(s):
    T, E, k, G = s["T"], s["E"], s["k"], s["G"]
    p = _scores(s)
    choice = p.float() if s["bias_e"] is None else p.float() + s["bias_e"]
    choice = choice.masked_fill(s["logits"] == -math.inf, -math.inf)
    if s["KG"] < G:
        best = torch.sort(choice.view(T, G, E // G), dim=2, descending=True).values
        group = best[:, :, 0] if s["top"] == 1 else best[:, :, 0] + best[:, :, 1]
        kept = torch.sort(group, dim=1, descending=True, stable=True).indices[:, :s["KG"]]
        out = torch.ones(T, G, dtype=torch.bool, device=DEV).scatter_(1, kept, False)
        # behind every expert of a kept group, those that are switched off among them
        order = torch.sort(out.repeat_interleave(E // G, dim=1).to(torch.int8), dim=1, stable=True).indices
        order = order[:, :s["KG"] * (E // G)]
        at = torch.sort(choice.gather(1, order), dim=1, descending=True, stable=True).indices[:, :k]
        ids = order.gather(1, at)
    else:
        ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    if s["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return {"topk_ids": ids.to(torch.int32), "topk_w": (s["scale"] * w).float()}


def _route_grad_plain(s):
    ids, p = s["topk_ids"].long(), _scores(s)
    dw, w = s["scale"] * s["d_topk_w"].double(), p.gather(1, ids)
    if s["renorm"]:
        tot = w.sum(dim=1, keepdim=True)
        dw = (dw - (dw * w).sum(dim=1, keepdim=True) / tot) / tot
    if s["score"] == "sigmoid":
        d = torch.zeros_like(p).scatter_(1, ids, dw * w * (1.0 - w))
    else:
        d = torch.zeros_like(p).scatter_(1, ids, dw * w) - p * (dw * w).sum(dim=1, keepdim=True)
    if s["mask"] is not None:
        d = torch.where(s["mask"][:, None] != 0, d, torch.zeros_like(d))
    return {"d_logits": d.float()}


def _codes(x):
    """Codes of the rows of x (fp32), as fp32, and their scales."""
    amax = x.abs().amax(dim=1, keepdim=True).clamp_min(TINY)
    top = torch.full_like(amax, I8_MAX)  # tensor by tensor: a correctly rounded quotient
    return torch.round(x * (top / amax)), amax / top


def _linear_plain(s):
    c, sx = _codes(s["x"].float())
    y = (c @ s["codes"].float().t()) * sx * s["scales"][None, :]
    return {"out": y.to(torch.bfloat16)}


def _experts_plain(s):
    E, I, k, P = s["E"], s["I"], s["k"], s["T"] * s["k"]
    rows = torch.arange(P, device=DEV)
    off = s["offsets"].long()
    e = torch.bucketize(rows, off[1:], right=True)
    at = rows - off[e]
    pair = s["sorted_pairs"].long()
    c, sx = _codes(s["x"].float())
    bucket = torch.zeros(E, s["max_rows"], s["H"], device=DEV)
    bucket[e, at] = c[pair // k]
    gu = torch.bmm(bucket, s["w13"].float().transpose(1, 2))[e, at] * sx[pair // k] * s["s13"][e]
    gate, up = gu[:, :I], gu[:, I:]
    c, sh = _codes((gate / (1.0 + torch.exp(-gate)) * up).to(torch.bfloat16).float())
    bucket = torch.zeros(E, s["max_rows"], I, device=DEV)
    bucket[e, at] = c
    y = torch.bmm(bucket, s["w2"].float().transpose(1, 2))[e, at] * sh * s["s2"][e]
    out = torch.empty(P, s["H"], dtype=torch.bfloat16, device=DEV)
    out[pair] = y.to(torch.bfloat16)
    return {"y": out}


def _sum_of(s):
    """The weighted sum of a token's rows, [T, H] in fp32."""
    m = torch.zeros(s["T"], s["H"], device=DEV)
    if s["k"]:
        m = m + (s["topk_w"][:, :, None] * s["y"].float().view(s["T"], s["k"], s["H"])).sum(dim=1)
    if s["shared"]:
        m = m + (s["shared_x"].float() if s["gate_t"] is None else s["gate_t"][:, None] * s["shared_x"].float())
    return m


def _rms(v, eps):
    return 1.0 / torch.sqrt((v * v).mean(dim=1, keepdim=True) + eps)


def _norm_plain(s):
    m = _sum_of(s)
    if s["post"]:
        m = m * _rms(m, s["eps"]) * s["post_w"].float()
    r = s["scale"] * m
    if s["residual"]:
        r = s["res"].float() + r
    o = {"out": r.to(torch.bfloat16)}
    if s["next"]:
        o["normed"] = (r * _rms(r, s["eps"]) * s["next_w"].float()).to(torch.bfloat16)
    return o


def _norm_grad_plain(s):
    T, H, k, bf16 = s["T"], s["H"], s["k"], torch.bfloat16
    o, d = {}, s["d_out"].float()
    if s["next"]:
        r = s["out"].float()
        q, dn = _rms(r, s["eps"]), s["d_normed"].float()
        r = r * q
        o["d_next_w"] = (dn * r).sum(dim=0)
        a = dn * s["next_w"].float()
        d = d + q * (a - r * (a * r).mean(dim=1, keepdim=True))
    if s["residual"]:
        o["d_res"] = d.to(bf16)
    d = s["scale"] * d
    if s["post"]:
        m = _sum_of(s)
        q = _rms(m, s["eps"])
        m = m * q
        o["d_post_w"] = (d * m).sum(dim=0)
        a = d * s["post_w"].float()
        d = q * (a - m * (a * m).mean(dim=1, keepdim=True))
    if k:
        o["d_topk_w"] = (s["y"].float().view(T, k, H) * d[:, None, :]).sum(dim=2)
        o["d_y"] = (s["topk_w"][:, :, None] * d[:, None, :]).to(bf16).view(T * k, H)
    if s["shared"]:
        if s["gate"]:
            o["d_gate"] = (s["shared_x"].float() * d).sum(dim=1)
            d = s["gate_t"][:, None] * d
        o["d_shared"] = d.to(bf16)
    return o


PLAIN = {"route": _route_plain, "route_grad": _route_grad_plain, "linear": _linear_plain, "experts": _experts_plain,
         "norm": _norm_plain, "norm_grad": _norm_grad_plain}


# ------------------------------------------------------------------ the library's calls


def _workspace(s, lib, nbytes):
    if "ws" not in s:  # sized once, kept like a user's program keeps it
        s["ws"] = torch.empty(max(nbytes(), 1), dtype=torch.uint8, device=DEV)
    return s["ws"]


def _router(s, lib):
    if "router" not in s:
        s["router"] = lib.make_router(s["E"], s["k"], s["score"], num_groups=s.get("G", 1), topk_groups=s.get("KG", 1),
                                      group_top=s.get("top", 1) if s.get("G", 1) > 1 else 1,
                                      renormalise=s["renorm"], scale=s["scale"])
    return s["router"]


def _route_own(s, lib):
    lib.moe_route_scores(_router(s, lib), s["T"], s["logits"], s["topk_ids"], s["topk_w"], bias=s["bias_e"])
    return {"topk_ids": s["topk_ids"], "topk_w": s["topk_w"]}


def _route_grad_own(s, lib):
    lib.moe_route_scores_backward(_router(s, lib), s["T"], s["logits"], s["topk_ids"], s["d_topk_w"], s["d_logits"],
                                  token_mask=s["mask"])
    return {"d_logits": s["d_logits"]}


def _linear_own(s, lib):
    M, N, K = s["M"], s["N"], s["K"]
    ws = _workspace(s, lib, lambda: lib.moe_int8_linear_workspace_bytes(M, N, K))
    lib.moe_int8_linear(M, N, K, s["codes"], s["scales"], s["x"], s["out"], ws)
    return {"out": s["out"]}


def _experts_own(s, lib):
    if "shape" not in s:
        s["shape"] = lib.make_shape(s["H"], s["I"], s["E"], s["k"], s["T"], "bf16")
    ws = _workspace(s, lib, lambda: lib.moe_int8_experts_workspace_bytes(s["shape"]))
    lib.moe_int8_experts(s["shape"], s["T"], s["w13"], s["s13"], s["w2"], s["s2"], s["offsets"], s["sorted_pairs"],
                         s["x"], s["out"], ws)
    return {"y": s["out"]}


def _norm_own(s, lib):
    lib.moe_combine_norm(s["T"], s["H"], s["k"], s["out"], s["normed"], y=s["y"], topk_w=s["topk_w"],
                         shared=s["shared_x"], shared_gate=s["gate_t"], residual=s["res"], post_weight=s["post_w"],
                         next_weight=s["next_w"], scale=s["scale"], eps=s["eps"])
    o = {"out": s["out"]}
    if s["next"]:
        o["normed"] = s["normed"]
    return o


def _norm_grad_own(s, lib):
    T, H = s["T"], s["H"]
    ws = _workspace(s, lib, lambda: lib.moe_combine_norm_backward_workspace_bytes(T, H))
    lib.moe_combine_norm_backward(
        T, H, s["k"], s["d_out"], s["d_normed"], s["out"], ws, y=s["y"], topk_w=s["topk_w"], shared=s["shared_x"],
        shared_gate=s["gate_t"], post_weight=s["post_w"], next_weight=s["next_w"], scale=s["scale"], eps=s["eps"],
        d_residual=s["d_res"], d_y=s["d_y"], d_topk_w=s["d_topk_w"], d_shared=s["d_shared"], d_gate=s["d_gate"],
        d_post_weight=s["d_post_w"], d_next_weight=s["d_next_w"])
    return {n: s[n] for n in ("d_next_w", "d_res", "d_post_w", "d_topk_w", "d_y", "d_gate", "d_shared")
            if s[n] is not None}


OWN = {"route": _route_own, "route_grad": _route_grad_own, "linear": _linear_own, "experts": _experts_own,
       "norm": _norm_own, "norm_grad": _norm_grad_own}


def run(state):
    if own:
        import mixture_experts_layer_sort_amd as lib

        return OWN[state["op"]](state, lib)
    return PLAIN[state["op"]](state)


# ------------------------------------------------------------------ work


def work(case):
    op = case["op"]
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": N * K + 4 * N + 2 * M * K + 2 * M * N, "flops": 2 * M * N * K}
    if op == "experts":
        T, H, I, E, k = (case[n] for n in "THIEk")
        active = E * (1.0 - (1.0 - k / E) ** T)
        return {"bytes": int(active * 3 * H * I + 2 * T * H + 2 * T * k * H + 8 * T * k), "flops": 6 * T * k * H * I}
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": 4 * T * E + 8 * T * k, "flops": 20 * T * E}
    if op == "route_grad":
        T, E, k = case["T"], case["E"], case["k"]
        read = 4 * T * E if case["score"] == "softmax" and not case["renorm"] else 4 * T * k
        return {"bytes": 4 * T * E + read + 8 * T * k, "flops": 4 * T * E}
    T, H, k = case["T"], case["H"], case["k"]
    rows = k + case["shared"]
    if op == "norm":
        return {"bytes": 2 * T * H * (rows + case["residual"] + 1 + case["next"]) + 4 * T * k,
                "flops": T * H * (2 * rows + 10)}
    # y and shared are read for the weights' gradients, out and d_normed for the next norm's
    return {"bytes": 2 * T * H * (2 * rows + 1 + case["residual"] + 2 * case["next"]) + 8 * T * k,
            "flops": T * H * (6 * rows + 20)}


# ------------------------------------------------------------------ the definition in 64 bits


def _route64(s):
    """Picks one after the other: the largest choice among the experts left, the lowest of equal ones."""
    T, E, k, G = s["T"], s["E"], s["k"], s["G"]
    z = s["logits"].double()
    p = torch.sigmoid(z) if s["score"] == "sigmoid" else torch.softmax(z, dim=1)
    # by definition a choice is the 32-bit score plus the bias, rounded to 32 bits, and so is a group's sum
    c = p.to(torch.float32)
    if s["bias_e"] is not None:
        c = (c.double() + s["bias_e"].double()).to(torch.float32)
    c = torch.where(torch.isinf(s["logits"]), torch.full_like(c, -math.inf), c)
    rows, none = torch.arange(T, device=DEV), torch.iinfo(torch.int64).max

    def picks(v, free, count):
        got, num = [], torch.arange(v.shape[1], device=DEV)
        for _ in range(count):
            top = torch.where(free, v.double(), -math.inf).amax(dim=1, keepdim=True)
            at = torch.where(free & (v.double() == top), num, none).amin(dim=1)
            free[rows, at] = False
            got.append(at)
        return torch.stack(got, dim=1)

    free = torch.ones(T, E, dtype=torch.bool, device=DEV)
    if s["KG"] < G:
        two = torch.topk(c.view(T, G, -1).double(), s["top"], dim=2).values.sum(dim=2).to(torch.float32)
        kept = picks(two, torch.ones(T, G, dtype=torch.bool, device=DEV), s["KG"])
        group = torch.arange(E, device=DEV) // (E // G)
        free = (group[None, None, :] == kept[:, :, None]).any(dim=1)
    ids = picks(c, free, k)
    w = p[rows[:, None], ids]
    return {"topk_ids": ids.to(torch.int32), "topk_w": s["scale"] * (w / w.sum(1, keepdim=True) if s["renorm"] else w)}


def _route_grad64(s):
    """The Jacobian of the weights, expert by pick, times their gradient."""
    z, ids = s["logits"].double(), s["topk_ids"].long()
    w_of = torch.sigmoid if s["score"] == "sigmoid" else (lambda v: torch.softmax(v, dim=1))
    z.requires_grad_(True)
    w = torch.gather(w_of(z), 1, ids)
    w = s["scale"] * (w / w.sum(dim=1, keepdim=True) if s["renorm"] else w)
    d, = torch.autograd.grad(w, z, s["d_topk_w"].double())
    return {"d_logits": d if s["mask"] is None else d * s["mask"].double()[:, None]}


def _codes64(x):
    """Codes and scales of x's rows.  By definition the factor 127 / amax and its product with x are fp32 numbers."""
    v = x.double()
    amax = torch.maximum(v.abs().max(dim=1, keepdim=True).values, torch.tensor(TINY, dtype=torch.float64, device=DEV))
    factor = (I8_MAX / amax).float().double()
    return torch.round((v * factor).float().double()), amax / I8_MAX


def _product64(x, codes, scales):
    c, sx = _codes64(x)
    return torch.mm(c, codes.double().t()) * sx * scales.double()


def _norm64(s):
    """By autograd in 64 bits, with a leaf for every input."""
    leaf = {n: s[n].double().requires_grad_(True) for n in
            ("y", "topk_w", "shared_x", "gate_t", "post_w", "next_w", "res") if s[n] is not None}
    T, H = s["T"], s["H"]
    m = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    if s["k"]:
        m = m + torch.matmul(leaf["topk_w"][:, None, :], leaf["y"].view(T, s["k"], H))[:, 0]
    if s["shared"]:
        m = m + leaf["shared_x"] * (leaf["gate_t"][:, None] if s["gate"] else 1.0)
    if s["post"]:
        m = leaf["post_w"] * m * torch.rsqrt(m.square().mean(1, keepdim=True) + s["eps"])
    return leaf, m * s["scale"]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _route64(s)
    if op == "route_grad":
        return _route_grad64(s)
    if op == "linear":
        return {"out": _product64(s["x"], s["codes"], s["scales"])}
    if op == "experts":
        off, I = s["offsets"].tolist(), s["I"]
        y = torch.zeros(s["T"] * s["k"], s["H"], dtype=torch.float64, device=DEV)
        for e in range(s["E"]):
            if off[e + 1] > off[e]:
                pairs = s["sorted_pairs"][off[e]:off[e + 1]].long()
                gu = _product64(s["x"][pairs // s["k"]], s["w13"][e], s["s13"][e])
                h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
                y[pairs] = _product64(h.to(torch.bfloat16), s["w2"][e], s["s2"][e])
        return {"y": y}
    leaf, m = _norm64(s)
    if op == "norm":
        r = m + leaf["res"] if s["residual"] else m
        o = {"out": r.detach()}
        if s["next"]:
            o["normed"] = (r * torch.rsqrt(r.square().mean(1, keepdim=True) + s["eps"]) * leaf["next_w"]).detach()
        return o
    # the gradient at the rows that the forward pass wrote
    o, d = {}, s["d_out"].double()
    if s["next"]:
        r = s["out"].double().requires_grad_(True)
        n = r * torch.rsqrt(r.square().mean(1, keepdim=True) + s["eps"]) * leaf["next_w"]
        dr, o["d_next_w"] = torch.autograd.grad(n, (r, leaf["next_w"]), s["d_normed"].double())
        d = d + dr
    if s["residual"]:
        o["d_res"] = d
    names = [n for n in ("post_w", "topk_w", "y", "gate_t", "shared_x") if n in leaf]
    grads = dict(zip(names, torch.autograd.grad(m, [leaf[n] for n in names], d)))
    for n, at in (("post_w", "d_post_w"), ("topk_w", "d_topk_w"), ("y", "d_y"), ("gate_t", "d_gate"),
                  ("shared_x", "d_shared")):
        if n in grads:
            o[at] = grads[n]
    return o
