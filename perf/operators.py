"""Cases of the operators around the expert FFN, each with its plain form.

route   scores over the router's logits, the groups with the best experts, the top-K experts of those
        groups and their weights (moe_route_grouped): from tokens and a router matrix, or from logits
linear  f(x W^T + b), or f(x W^T + b) * (x V^T + c), plus a residual (moe_linear)
norm    s = x + r, RMS norm of s times a weight; s and the norm are both outputs (moe_add_rms_norm)

The listed cases:
  route_1          one generated token through the router of the 8-token decode layer, experts in groups
  route_53         a small ragged batch, softmax scores, hidden size and experts off the powers of two
  route_4096       a prompt of 4096 tokens
  route_given      logits from elsewhere (a router that ran in another place), a long prompt
  linear_1_gated   one token through the gate and up matrices of a bf16 shared expert
  linear_8_down    eight sequences through its down matrix, added to the routed experts' sum
  linear_77        a ragged batch through a plain layer with bias and GELU, f16, sizes off the tiles
  linear_4096      the gate and up matrices for a prompt
  linear_16384     the down matrix for a long prompt, with bias, added to the routed experts' sum
  norm_1           the residual add and the norm before the block, one token
  norm_301         no residual yet (the first layer), f16, a hidden size off the vector width
  norm_32768       the residual add and the norm, a long prompt

The router's tokens and weights lie on fixed-point grids (1/16 and 2^-12, a few standard deviations
either side), so every logit is the same 32-bit number in whatever order it is summed and the chosen
experts are well defined.
"""
import math

import torch

own = False

SOFTMAX, SIGMOID, SQRTSOFTPLUS, SOFTMAX_BIAS = 0, 1, 3, 4  # the framework's scoring numbers
FUNCS = ("none", "silu", "gelu", "gelu_tanh", "relu")      # its function numbers, in order
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        dict(name="route_1", op="route", T=1, E=256, H=7168, k=8, groups=16, keep=6, group_top=2,
             scoring=SIGMOID, renorm=True, scaling=2.5, given=False),
        dict(name="route_53", op="route", T=53, E=180, H=1184, k=6, groups=12, keep=5, group_top=1,
             scoring=SOFTMAX, renorm=False, scaling=16.0, given=False),
        dict(name="route_4096", op="route", T=4096, E=256, H=7168, k=8, groups=16, keep=6, group_top=2,
             scoring=SIGMOID, renorm=True, scaling=2.5, given=False),
        dict(name="route_given", op="route", T=32768, E=128, H=0, k=8, groups=8, keep=3, group_top=2,
             scoring=SOFTMAX_BIAS, renorm=True, scaling=1.0, given=True),
        dict(name="linear_1_gated", op="linear", T=1, N=2048, K=7168, func="silu", gated=True, bias=False,
             residual=False, dtype="bf16"),
        dict(name="linear_8_down", op="linear", T=8, N=7168, K=2048, func="none", gated=False, bias=False,
             residual=True, dtype="bf16"),
        dict(name="linear_77", op="linear", T=77, N=1000, K=1544, func="gelu", gated=False, bias=True,
             residual=False, dtype="f16"),
        dict(name="linear_4096", op="linear", T=4096, N=2048, K=7168, func="silu", gated=True, bias=False,
             residual=False, dtype="bf16"),
        dict(name="linear_16384", op="linear", T=16384, N=7168, K=2048, func="none", gated=False, bias=True,
             residual=True, dtype="bf16"),
        dict(name="norm_1", op="norm", T=1, H=7168, residual=True, dtype="bf16"),
        dict(name="norm_301", op="norm", T=301, H=2050, residual=False, dtype="f16"),
        dict(name="norm_32768", op="norm", T=32768, H=7168, residual=True, dtype="bf16"),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("route", "linear", "linear", "norm"))
    if op == "route":
        groups = rng.choice((1, 2, 3, 4, 8, 12, 16))
        size = rng.randint(max(2, -(-24 // groups)), 512 // groups)
        keep = rng.randint(1, groups)
        given = rng.random() < 0.3
        scoring = rng.choice((SOFTMAX, SIGMOID, SIGMOID, SQRTSOFTPLUS, SOFTMAX_BIAS))
        H = 0 if given else 32 * _spread(rng, 4, 256)
        return dict(op=op, T=_spread(rng, 1, 32768 if given else 8192), E=groups * size, H=H,
                    k=rng.randint(1, min(16, keep * size)), groups=groups, keep=keep,
                    group_top=rng.choice((1, 2)), scoring=scoring, renorm=rng.random() < 0.7,
                    scaling=rng.choice((1.0, 2.5, 16.0)), given=given)
    if op == "linear":
        N, K, gated = _spread(rng, 32, 8192), 8 * _spread(rng, 8, 1024), rng.random() < 0.4
        most = 16384 * 7168 * 2048 // (N * K * (2 if gated else 1))
        return dict(op=op, T=_spread(rng, 1, max(1, min(16384, most))), N=N, K=K, func=rng.choice(FUNCS),
                    gated=gated, bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                    dtype=rng.choice(("bf16", "bf16", "f16")))
    H = _spread(rng, 64, 8192)
    return dict(op=op, T=_spread(rng, 1, min(32768, 32768 * 7168 // H)), H=H, residual=rng.random() < 0.7,
                dtype=rng.choice(("bf16", "bf16", "f16")))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    s = dict(case)
    T = case["T"]
    if case["op"] == "route":
        E, H, k = case["E"], case["H"], case["k"]
        if case["given"]:
            s["logits_in"] = normal(T, E) * 1.5
            s["x"] = s["w_router"] = None
        else:
            s["x"] = ((normal(T, H) * 16).round_().clamp_(-127, 127) / 16).to(torch.bfloat16)
            s["w_router"] = ((normal(E, H) * (1.5 / math.sqrt(H)) * 4096).round_().clamp_(-255, 255) / 4096).to(torch.bfloat16)
            s["logits_in"] = None
        s["bias"] = None if case["scoring"] == SOFTMAX else (torch.rand(E, generator=g, device="cuda") * 0.2 - 0.1) * (0.05 if case["scoring"] == SOFTMAX_BIAS else 1.0)
        s["ids"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        s["w"] = torch.empty(T, k, device="cuda")
        s["logits"] = None if case["given"] else torch.empty(T, E, device="cuda")
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        return s
    t = DTYPES[case["dtype"]]
    if case["op"] == "linear":
        N, K = case["N"], case["K"]
        s["x"] = normal(T, K).to(t)
        s["weight"] = (normal(N, K) * (1.0 / math.sqrt(K))).to(t)
        s["weight_mul"] = (normal(N, K) * (1.0 / math.sqrt(K))).to(t) if case["gated"] else None
        s["b"] = normal(N) * 0.1 if case["bias"] else None
        s["b_mul"] = normal(N) * 0.1 if case["bias"] and case["gated"] else None
        s["r"] = normal(T, N).to(t) if case["residual"] else None
        s["out"] = torch.empty(T, N, dtype=t, device="cuda")
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        return s
    H = case["H"]
    s["x"] = normal(T, H).to(t)
    s["r"] = (normal(T, H) * 4).to(t) if case["residual"] else None
    s["weight"] = (1 + 0.1 * normal(H)).to(t)
    s["out"] = torch.empty(T, H, dtype=t, device="cuda")
    s["sum"] = torch.empty(T, H, dtype=t, device="cuda") if case["residual"] else None
    return s


# ---- the plain forms ---------------------------------------------------------------------------
def _scores(scoring, logits):
    if scoring in (SOFTMAX, SOFTMAX_BIAS):
        e = torch.exp(logits - logits.amax(1, keepdim=True))
        return e / e.sum(1, keepdim=True)
    if scoring == SIGMOID:
        return 1 / (1 + torch.exp(-logits))
    return torch.sqrt(torch.log1p(torch.exp(logits)))


def _plain_route(s):
    logits = s["logits_in"] if s["given"] else s["x"].float() @ s["w_router"].float().t()
    T, E = logits.shape
    score = _scores(s["scoring"], logits.double())  # 64 bits: values next to a border decide the experts
    v = score if s["bias"] is None else score + s["bias"].double()
    grouped = v.view(T, s["groups"], E // s["groups"])
    of_group = grouped.sort(dim=2, descending=True).values[:, :, :s["group_top"]].sum(2)
    kept = of_group.sort(dim=1, descending=True, stable=True).indices[:, :s["keep"]]
    inside = torch.zeros_like(of_group, dtype=torch.bool).scatter_(1, kept, True)
    v = torch.where(inside[:, :, None], grouped, -math.inf).view(T, E)
    ids = v.sort(dim=1, descending=True, stable=True).indices[:, :s["k"]]
    w = score.gather(1, ids)
    w = w / w.sum(1, keepdim=True) * s["scaling"] if s["renorm"] else w * s["scaling"]
    out = {"ids": ids.to(torch.int32), "w": w.float()}
    return out if s["given"] else {**out, "logits": logits}


def _apply(func, z):
    if func == "silu":
        return z / (1 + torch.exp(-z))
    if func == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if func == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z.clamp(min=0) if func == "relu" else z


def _plain_linear(s):
    x = s["x"].float()
    z = x @ s["weight"].float().t()
    z = _apply(s["func"], z if s["b"] is None else z + s["b"])
    if s["gated"]:
        u = x @ s["weight_mul"].float().t()
        z = z * (u if s["b_mul"] is None else u + s["b_mul"])
    z = z if s["r"] is None else z + s["r"].float()
    return z.to(s["out"].dtype)


def _plain_norm(s):
    t = s["x"].float() if s["r"] is None else s["x"].float() + s["r"].float()
    y = t * torch.rsqrt(t.square().mean(1, keepdim=True) + 1e-6) * s["weight"].float()
    y = y.to(s["out"].dtype)
    return y if s["r"] is None else {"out": y, "sum": t.to(s["out"].dtype)}


# ---- the framework's calls -----------------------------------------------------------------------
def _own(s):
    from block_quantized_moe_router_gb300 import capi
    if s["op"] == "route":
        capi.moe_route_grouped(T=s["T"], E=s["E"], H=s["H"], top_k=s["k"], scoring=s["scoring"],
                               renormalize=s["renorm"], routed_scaling=s["scaling"], n_group=s["groups"],
                               topk_group=s["keep"], group_top=s["group_top"], x=s["x"],
                               w_router=s["w_router"], logits_in=s["logits_in"], logits_out=s["logits"],
                               correction_bias=s["bias"], topk_ids=s["ids"], topk_w=s["w"],
                               dev_status=s["status"])
        out = {"ids": s["ids"], "w": s["w"]}
        return out if s["given"] else {**out, "logits": s["logits"]}
    if s["op"] == "linear":
        capi.moe_linear(s["x"], s["weight"], s["out"], w_mul=s["weight_mul"], bias=s["b"],
                        bias_mul=s["b_mul"], residual=s["r"], func=FUNCS.index(s["func"]),
                        dev_status=s["status"])
        return s["out"]
    capi.moe_add_rms_norm(s["x"], s["weight"], s["out"], residual=s["r"], sum_out=s["sum"], eps=1e-6)
    return s["out"] if s["r"] is None else {"out": s["out"], "sum": s["sum"]}


def run(state):
    if own:
        return _own(state)
    return {"route": _plain_route, "linear": _plain_linear, "norm": _plain_norm}[state["op"]](state)


def work(case):
    T = case["T"]
    if case["op"] == "route":
        E, H, k = case["E"], case["H"], case["k"]
        out = T * k * 8 + (0 if case["scoring"] == SOFTMAX else 4 * E) + T * E * 4
        if case["given"]:
            return {"bytes": out, "flops": 0}
        return {"bytes": out + 2 * (T * H + E * H), "flops": 2 * T * E * H}
    if case["op"] == "linear":
        N, K, n = case["N"], case["K"], 2 if case["gated"] else 1
        return {"bytes": 2 * (T * K + n * N * K + T * N * (2 if case["residual"] else 1)) + (4 * n * N if case["bias"] else 0),
                "flops": 2 * T * N * K * n}
    H = case["H"]
    return {"bytes": 2 * H + 2 * T * H * (4 if case["residual"] else 2), "flops": 0}


# ---- the definitions in 64 bits ------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    up = torch.float64
    if case["op"] == "route":
        l = s["logits_in"].to(up) if case["given"] else torch.mm(s["x"].to(up), s["w_router"].to(up).t())
        if case["scoring"] in (SOFTMAX, SOFTMAX_BIAS):
            p = torch.softmax(l, 1)
        elif case["scoring"] == SIGMOID:
            p = torch.sigmoid(l)
        else:
            p = torch.logaddexp(l, torch.zeros_like(l)).sqrt()
        rank = p if s["bias"] is None else p + s["bias"].to(up)
        T, E = rank.shape
        size, left = E // case["groups"], rank.clone()
        best = rank.reshape(T, case["groups"], size).topk(case["group_top"], 2).values.sum(2)
        rows = torch.arange(T, device=l.device)
        for _ in range(case["groups"] - case["keep"]):  # the worst group goes, the last one of equals
            worst = case["groups"] - 1 - best.flip(1).argmin(1)
            best[rows, worst] = math.inf
            left.view(T, case["groups"], size)[rows, worst] = -math.inf
        ids = []
        for _ in range(case["k"]):
            ids.append(left.argmax(1))
            left[rows, ids[-1]] = -math.inf
        ids = torch.stack(ids, 1)
        w = torch.take_along_dim(p, ids, 1) * case["scaling"]
        if case["renorm"]:
            w = w * case["scaling"] / w.sum(1, keepdim=True)
        out = {"ids": ids, "w": w}
        return out if case["given"] else {**out, "logits": l}
    if case["op"] == "linear":
        z = torch.mm(s["x"].to(up), s["weight"].to(up).t())
        if s["b"] is not None:
            z += s["b"].to(up)
        f = case["func"]
        if f == "silu":
            z = z * torch.sigmoid(z)
        elif f == "gelu":
            z = z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
        elif f == "gelu_tanh":
            z = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        elif f == "relu":
            z = torch.maximum(z, torch.zeros_like(z))
        if case["gated"]:
            u = torch.mm(s["x"].to(up), s["weight_mul"].to(up).t())
            z = z * (u if s["b_mul"] is None else u + s["b_mul"].to(up))
        return z if s["r"] is None else z + s["r"].to(up)
    t = s["x"].to(up) + (0 if s["r"] is None else s["r"].to(up))
    y = s["weight"].to(up) * t / torch.sqrt((t * t).mean(1, keepdim=True) + 1e-6)
    return y if s["r"] is None else {"out": y, "sum": t}
