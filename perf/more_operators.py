"""Cases of the operators of a layer that serves many requests at once, each with its plain form.

adapters  a dense layer with low-rank adapters, each row with that of its request (moe_linear_adapters):
          f(x W^T + b + s (x A^T) B^T), or that times a second such factor, plus a residual
sandwich  the norm behind a block, its gate and residual scale, the residual add and the norm before the
          next block (moe_sandwich_norm): s = a r + g norm(y), n = norm(s); both are outputs

The listed cases:
  adapters_1          one generated token through the gate and up matrices of a bf16 shared expert
  adapters_8_down     eight sequences, an adapter each, through its down matrix, added to the routed experts' sum
  adapters_64         64 sequences, an adapter each of a larger rank, gate and up matrices of a smaller model
  adapters_77         a ragged batch through a plain layer with bias and GELU, f16, sizes off the tiles, some rows
                      without an adapter
  adapters_512        512 sequences that share 32 adapters, a row's neighbours with others, the down matrix
  adapters_4096       prompts of four requests, 4096 tokens in all, gate and up matrices
  adapters_16384      long prompts of twelve requests, adapters of rank 64, the down matrix with bias and residual
  sandwich_1          one token behind the expert block, norms on both sides, a gate per channel
  sandwich_301        a ragged batch, f16, a hidden size off the vector width, a sigmoid gate per row
  sandwich_4096       a prompt with the residual stream in 32 bits, weights that hold the distance from one
  sandwich_32768      a long prompt, norms on both sides, a gate per channel

Adapters come as a server has them: stacked for all the requests that it may serve, of which a batch meets a
few.  Prompts are runs of rows with one adapter, generated tokens of many requests stand in any order.
"""
import math

import torch

own = False

FUNCS = ("none", "silu", "gelu", "gelu_tanh", "relu")  # the framework's function numbers, in order
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


def listed():
    return [
        dict(name="adapters_1", op="adapters", T=1, N=2048, K=7168, R=16, L=64, used=1, bare=0, mixed=True,
             func="silu", gated=True, bias=False, residual=False, dtype="bf16"),
        dict(name="adapters_8_down", op="adapters", T=8, N=7168, K=2048, R=16, L=64, used=8, bare=0, mixed=True,
             func="none", gated=False, bias=False, residual=True, dtype="bf16"),
        dict(name="adapters_64", op="adapters", T=64, N=2048, K=4096, R=32, L=96, used=64, bare=0, mixed=True,
             func="silu", gated=True, bias=False, residual=False, dtype="bf16"),
        dict(name="adapters_77", op="adapters", T=77, N=1000, K=1544, R=24, L=20, used=9, bare=11, mixed=True,
             func="gelu", gated=False, bias=True, residual=False, dtype="f16"),
        dict(name="adapters_512", op="adapters", T=512, N=7168, K=2048, R=16, L=64, used=32, bare=0, mixed=True,
             func="none", gated=False, bias=False, residual=True, dtype="bf16"),
        dict(name="adapters_4096", op="adapters", T=4096, N=2048, K=7168, R=16, L=64, used=4, bare=0, mixed=False,
             func="silu", gated=True, bias=False, residual=False, dtype="bf16"),
        dict(name="adapters_16384", op="adapters", T=16384, N=7168, K=2048, R=64, L=16, used=12, bare=0, mixed=False,
             func="none", gated=False, bias=True, residual=True, dtype="bf16"),
        dict(name="sandwich_1", op="sandwich", T=1, H=7168, post=True, gate="channel", wide=False, offset=0.0,
             scale=1.0, next=True, dtype="bf16"),
        dict(name="sandwich_301", op="sandwich", T=301, H=2050, post=False, gate="row", wide=False, offset=0.0,
             scale=0.5, next=True, dtype="f16"),
        dict(name="sandwich_4096", op="sandwich", T=4096, H=4096, post=True, gate="none", wide=True, offset=1.0,
             scale=1.0, next=True, dtype="bf16"),
        dict(name="sandwich_32768", op="sandwich", T=32768, H=7168, post=True, gate="channel", wide=False, offset=0.0,
             scale=1.0, next=True, dtype="bf16"),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    if rng.random() < 0.6:
        N, K, gated = _spread(rng, 32, 8192), 8 * _spread(rng, 8, 1024), rng.random() < 0.4
        R = rng.choice((8, 16, 16, 24, 32, 64, 128))
        most = 16384 * 7168 * 2048 // ((N * K + 2 * R * (N + K)) * (2 if gated else 1))
        T = _spread(rng, 1, max(1, min(16384, most)))
        mixed = T <= 1024 and rng.random() < 0.7
        L = _spread(rng, 1, 96)
        bare = rng.randint(0, T // 2) if rng.random() < 0.4 else 0
        return dict(op="adapters", T=T, N=N, K=K, R=R, L=L, used=rng.randint(1, min(L, T - bare, 96 if mixed else 16)),
                    bare=bare, mixed=mixed, func=rng.choice(FUNCS), gated=gated, bias=rng.random() < 0.5,
                    residual=rng.random() < 0.5, dtype=rng.choice(("bf16", "bf16", "f16")))
    H = _spread(rng, 64, 8192)
    wide = rng.random() < 0.3
    return dict(op="sandwich", T=_spread(rng, 1, min(32768, (16384 if wide else 32768) * 7168 // H)), H=H,
                post=rng.random() < 0.7, gate=rng.choice(("none", "channel", "row")), wide=wide,
                offset=rng.choice((0.0, 1.0)), scale=rng.choice((1.0, 1.0, 0.5, 0.25)), next=rng.random() < 0.8,
                dtype=rng.choice(("bf16", "bf16", "f16")))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    s = dict(case)
    t = DTYPES[case["dtype"]]
    T = case["T"]
    if case["op"] == "adapters":
        N, K, R, L, used, bare = (case[k] for k in ("N", "K", "R", "L", "used", "bare"))
        n = 2 if case["gated"] else 1
        s["x"] = normal(T, K).to(t)
        s["weight"], s["weight_mul"] = [(normal(N, K) * (1.0 / math.sqrt(K))).to(t) for _ in range(n)] + [None] * (2 - n)
        s["a"], s["a_mul"] = [(normal(L, R, K) * (1.0 / math.sqrt(K))).to(t) for _ in range(n)] + [None] * (2 - n)
        s["b"], s["b_mul"] = [(normal(L, N, R) * (0.5 / math.sqrt(R))).to(t) for _ in range(n)] + [None] * (2 - n)
        s["scale"] = 0.5 + 1.5 * torch.rand(L, generator=g, device="cuda")
        s["bias"] = normal(N) * 0.1 if case["bias"] else None
        s["bias_mul"] = normal(N) * 0.1 if case["bias"] and case["gated"] else None
        s["r"] = normal(T, N).to(t) if case["residual"] else None
        # `used` of the adapters, each for one row at least; `bare` rows without
        which = torch.randperm(L, generator=g, device="cuda")[:used]
        rest = torch.randint(used, (T - bare - used,), generator=g, device="cuda")
        rows = torch.cat([which, which[rest], torch.full((bare,), -1, device="cuda")])
        if case["mixed"]:
            rows = rows[torch.randperm(T, generator=g, device="cuda")]
        else:  # runs of rows, the requests in any order
            place = torch.cat([torch.arange(used, device="cuda"), rest, torch.full((bare,), used, device="cuda")])
            rows = rows[torch.sort(place, stable=True).indices]
        s["ids"] = rows.to(torch.int32).contiguous()
        s["out"] = torch.empty(T, N, dtype=t, device="cuda")
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if own:
            from block_quantized_moe_router_gb300 import capi
            s["workspace"] = torch.empty(capi.moe_adapter_workspace_size(T, R, n), dtype=torch.uint8, device="cuda")
        return s
    H = case["H"]
    stream = torch.float32 if case["wide"] else t
    s["y"] = normal(T, H).to(t)
    s["r"] = (normal(T, H) * 4).to(stream)
    s["post_weight"] = (1 - case["offset"] + 0.1 * normal(H)).to(t) if case["post"] else None
    s["channel"] = (0.5 + 0.1 * normal(H)).to(t) if case["gate"] == "channel" else None
    s["row"] = normal(T) if case["gate"] == "row" else None
    s["weight"] = (1 - case["offset"] + 0.1 * normal(H)).to(t) if case["next"] else None
    s["sum"] = torch.empty(T, H, dtype=stream, device="cuda")
    s["out"] = torch.empty(T, H, dtype=t, device="cuda") if case["next"] else None
    return s


# ---- the plain forms ---------------------------------------------------------------------------
def _apply(func, z):
    if func == "silu":
        return z / (1 + torch.exp(-z))
    if func == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if func == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z.clamp(min=0) if func == "relu" else z


def _plain_product(s, x, weight, a, b, bias):
    """One matrix with its adapters: the rows' products with all of them, those of other requests set to zero."""
    T, (L, R, K) = x.shape[0], a.shape
    mine = s["ids"][:, None] == torch.arange(L, device=x.device, dtype=torch.int32)
    v = (x @ a.float().reshape(L * R, K).t()).view(T, L, R) * s["scale"][:, None]
    v = torch.where(mine[:, :, None], v, 0.0).view(T, L * R)
    z = x @ weight.float().t() + v @ b.float().transpose(1, 2).reshape(L * R, -1)
    return z if bias is None else z + bias


def _plain_adapters(s):
    x = s["x"].float()
    z = _apply(s["func"], _plain_product(s, x, s["weight"], s["a"], s["b"], s["bias"]))
    if s["gated"]:
        z = z * _plain_product(s, x, s["weight_mul"], s["a_mul"], s["b_mul"], s["bias_mul"])
    z = z if s["r"] is None else z + s["r"].float()
    return z.to(s["out"].dtype)


def _plain_norm(v, weight, offset):
    return v * torch.rsqrt(v.square().mean(1, keepdim=True) + EPS) * (weight.float() + offset)


def _plain_sandwich(s):
    p = s["y"].float()
    if s["post_weight"] is not None:
        p = _plain_norm(p, s["post_weight"], s["offset"])
    if s["channel"] is not None:
        p = p * s["channel"].float()
    if s["row"] is not None:
        p = p / (1 + torch.exp(-s["row"][:, None]))
    t = s["r"].float() * s["scale"] + p
    if s["weight"] is None:
        return t.to(s["sum"].dtype)
    return {"sum": t.to(s["sum"].dtype), "out": _plain_norm(t, s["weight"], s["offset"]).to(s["out"].dtype)}


# ---- the framework's calls -----------------------------------------------------------------------
def _own(s):
    from block_quantized_moe_router_gb300 import capi
    if s["op"] == "adapters":
        capi.moe_linear_adapters(s["x"], s["weight"], s["out"], s["ids"], a=s["a"], b=s["b"], a_mul=s["a_mul"],
                                 b_mul=s["b_mul"], scale=s["scale"], w_mul=s["weight_mul"], bias=s["bias"],
                                 bias_mul=s["bias_mul"], residual=s["r"], func=FUNCS.index(s["func"]),
                                 workspace=s["workspace"], dev_status=s["status"])
        return s["out"]
    capi.moe_sandwich_norm(s["y"], s["sum"], residual=s["r"], post_weight=s["post_weight"], gate=s["channel"],
                           row_gate=s["row"], row_sigmoid=s["row"] is not None, weight=s["weight"], out=s["out"],
                           residual_scale=s["scale"], weight_offset=s["offset"], eps=EPS)
    return s["sum"] if s["weight"] is None else {"sum": s["sum"], "out": s["out"]}


def run(state):
    if own:
        return _own(state)
    return _plain_adapters(state) if state["op"] == "adapters" else _plain_sandwich(state)


def work(case):
    T = case["T"]
    if case["op"] == "adapters":
        N, K, R, n = case["N"], case["K"], case["R"], 2 if case["gated"] else 1
        return {"bytes": 2 * (T * K + n * N * K + T * N * (2 if case["residual"] else 1) + n * case["used"] * R * (N + K)) +
                4 * (T + case["used"]) + (4 * n * N if case["bias"] else 0),
                "flops": 2 * n * (T * N * K + (T - case["bare"]) * R * (N + K))}
    H, wide = case["H"], 4 if case["wide"] else 2
    vectors = sum((case["post"], case["gate"] == "channel", case["next"]))
    return {"bytes": T * H * (2 + 2 * wide + (2 if case["next"] else 0)) + 2 * H * vectors +
            (4 * T if case["gate"] == "row" else 0), "flops": 0}


# ---- the definitions in 64 bits ------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    up = torch.float64
    if case["op"] == "adapters":
        x = s["x"].to(up)

        def product(weight, a, b, bias):
            z = torch.mm(x, weight.to(up).t())
            for j in sorted(set(s["ids"].tolist()) - {-1}):  # adapter by adapter, over the rows that have it
                rows = (s["ids"] == j).nonzero()[:, 0]
                low = torch.mm(x[rows], a[j].to(up).t()) * float(s["scale"][j])
                z.index_add_(0, rows, torch.mm(low, b[j].to(up).t()))
            return z if bias is None else z + bias.to(up)

        z = product(s["weight"], s["a"], s["b"], s["bias"])
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
            z = z * product(s["weight_mul"], s["a_mul"], s["b_mul"], s["bias_mul"])
        return z if s["r"] is None else z + s["r"].to(up)

    def norm(v, weight):
        return (weight.to(up) + case["offset"]) * v / torch.sqrt((v * v).sum(1, keepdim=True) / case["H"] + EPS)

    p = s["y"].to(up) if s["post_weight"] is None else norm(s["y"].to(up), s["post_weight"])
    if s["channel"] is not None:
        p = p * s["channel"].to(up)
    if s["row"] is not None:
        p = p * torch.sigmoid(s["row"].to(up))[:, None]
    t = p + case["scale"] * s["r"].to(up)
    return t if s["weight"] is None else {"sum": t, "out": norm(t, s["weight"])}
