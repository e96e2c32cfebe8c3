"""What is measured of a dense layer's operators: products with an epilogue, and heads' norms with rotation.

Operators (a case's "op"):

  linear       a product with bias, activation and residual in its epilogue; with "swiglu" or "geglu" both
               projections of a gated feed-forward block, the activation and the product of the two
  linear_grad  its backward pass: into the rows, the weight and the bias
  heads        norms of queries and keys for each head, with the position rotation in the same pass,
               positions of one or of several axes
  heads_grad   its backward pass: into queries and keys and the norms' weights

`run` computes them in elementary torch operations in 32 bits, or, where `own` is
true, by the calls a user makes of the framework.
"""
import math

import torch

own = False
sk = None      # the framework's package, once `own` calls for it

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp32": 4}
GATED = ("swiglu", "geglu")
EPS = 1e-6


def _package():
    global sk
    if sk is None:
        import latency_skinny_bf16_gb300
        sk = latency_skinny_bf16_gb300
        # a decode loop runs with programmatic dependent launch on
        sk.skinny_set_option(sk.SKINNY_OPT_PDL, 1)
    return sk


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a decode step, the first projection with its bias: latency
        {"name": "linear one token", "op": "linear", "M": 1, "N": 2112, "K": 7168, "act": "none", "bias": True,
         "residual": False, "save": False, "out": "bf16"},
        # a decode batch: the shared expert's down product, added to the residual stream
        {"name": "linear decode", "op": "linear", "M": 16, "N": 7168, "K": 2048, "act": "none", "bias": False,
         "residual": True, "save": False, "out": "bf16"},
        # a prompt of an odd length through the same product
        {"name": "linear prompt", "op": "linear", "M": 2047, "N": 7168, "K": 2048, "act": "none", "bias": True,
         "residual": True, "save": False, "out": "bf16"},
        # the shared expert's gate and up products: one token, a decode batch with an odd number of tokens
        {"name": "gated one token", "op": "linear", "M": 1, "N": 2048, "K": 7168, "act": "swiglu", "bias": False,
         "residual": False, "save": False, "out": "bf16"},
        {"name": "gated decode", "op": "linear", "M": 61, "N": 2048, "K": 7168, "act": "swiglu", "bias": False,
         "residual": False, "save": False, "out": "bf16"},
        # a training micro-batch, what the backward pass needs kept
        {"name": "gated train", "op": "linear", "M": 8192, "N": 2048, "K": 7168, "act": "swiglu", "bias": False,
         "residual": False, "save": True, "out": "bf16"},
        # its backward pass
        {"name": "gated grad train", "op": "linear_grad", "M": 8192, "N": 2048, "K": 7168, "act": "swiglu",
         "bias": False},
        # a small layer with sizes that are no multiple of anything
        {"name": "linear grad odd", "op": "linear_grad", "M": 1001, "N": 1437, "K": 2877, "act": "gelu",
         "bias": True},
        # a decode batch of 64 requests, far positions
        {"name": "heads decode", "op": "heads", "T": 64, "Hq": 32, "Hk": 8, "D": 128, "R": 128, "axes": 1,
         "interleaved": False, "norm": True, "dtype": "bf16"},
        # a prompt with images: positions of time, height and width
        {"name": "heads prompt axes", "op": "heads", "T": 16384, "Hq": 64, "Hk": 8, "D": 128, "R": 128, "axes": 3,
         "interleaved": False, "norm": True, "dtype": "bf16"},
        # the backward pass of a training micro-batch
        {"name": "heads grad train", "op": "heads_grad", "T": 8192, "Hq": 64, "Hk": 8, "D": 128, "R": 128, "axes": 1,
         "interleaved": False, "norm": True, "dtype": "bf16"},
        # a small vision tower: rows and columns as axes, an unusual head, fp32
        {"name": "heads grad odd", "op": "heads_grad", "T": 3001, "Hq": 12, "Hk": 12, "D": 72, "R": 36, "axes": 2,
         "interleaved": True, "norm": True, "dtype": "fp32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: a multiple of 64 mostly, of 8 sometimes, any at times."""
    v = _log(rng, lo, hi)
    m = rng.choice([64, 64, 64, 8, 1])
    return max(m, v // m * m)


LARGEST = 8192 * 4096 * 7168      # multiply-adds of one product of the largest listed case


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "heads", "heads_grad"])
    if op in ("linear", "linear_grad"):
        M, N, K = _log(rng, 1, 8192), _width(rng, 64, 8192), _width(rng, 64, 8192)
        act = rng.choice(["none", "silu", "gelu", "swiglu", "geglu"])
        rows = 2 * N if act in GATED else N
        M = max(1, min(M, LARGEST // (rows * K)))
        c = {"op": op, "M": M, "N": N, "K": K, "act": act, "bias": rng.random() < 0.5}
        if op == "linear":
            c["residual"] = rng.random() < 0.5
            c["save"] = act != "none" and rng.random() < 0.3
            c["out"] = rng.choice(["bf16", "bf16", "fp32"])
        return c
    D = rng.choice([64, 72, 80, 96, 128, 128, 192, 256, 61])
    R = rng.choice([D, D, D // 2]) // 2 * 2
    axes = rng.choice([1, 1, 2, 3])
    Hq = rng.choice([1, 7, 8, 12, 16, 32, 64, 128])
    Hk = rng.choice([h for h in (1, 2, 4, 7, 8, 12) if h <= Hq])
    T = max(1, min(_log(rng, 1, 32768), 8192 * 72 * 128 // ((Hq + Hk) * D)))
    return {"op": op, "T": T, "Hq": Hq, "Hk": Hk, "D": D, "R": R, "axes": axes,
            "interleaved": rng.random() < 0.3, "norm": rng.random() < 0.8, "dtype": rng.choice(["bf16", "bf16", "fp32"])}


# ------------------------------------------------------------------ inputs

def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _uniform(g, shape, K):
    """Weights U(-1/sqrt(K), 1/sqrt(K)) in bf16."""
    b = 1.0 / math.sqrt(K)
    return torch.empty(shape, device="cuda", dtype=torch.bfloat16).uniform_(-b, b, generator=g)


def _positions(g, c):
    """int32 [axes, T]: prompts one behind the other with one axis (a decode batch: anywhere), images of
    rows and columns behind one another with several."""
    T, A = c["T"], c["axes"]
    if A == 1:
        if T <= 256:
            return torch.randint(0, POSITIONS, (1, T), generator=g, device="cuda", dtype=torch.int32)
        start = torch.randint(0, POSITIONS - T, (1, 1), generator=g, device="cuda", dtype=torch.int32)
        return start + torch.arange(T, device="cuda", dtype=torch.int32)[None]
    at = torch.arange(T, device="cuda", dtype=torch.int32)
    image, inside = at // 1024, at % 1024
    rows, cols = image * 32 + inside // 32, image * 32 + inside % 32
    return torch.stack([image, rows, cols][-A:]).contiguous()


POSITIONS = 65536


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(1_000_003 * (seed + 1))
    s = {"case": c}
    op = c["op"]
    if own:
        _package()
    bf16 = torch.bfloat16
    if op in ("linear", "linear_grad"):
        M, N, K = c["M"], c["N"], c["K"]
        rows = 2 * N if c["act"] in GATED else N
        s["x"] = _normal(g, (M, K), bf16)
        s["w"] = _uniform(g, (rows, K), K)
        act = None if c["act"] == "none" else c["act"]
        s["act"] = act
        if op == "linear":
            dt = DTYPES[c["out"]]
            s["bias"] = 0.1 * _normal(g, (rows,), bf16) if c["bias"] else None
            s["residual"] = _normal(g, (M, N), dt) if c["residual"] else None
            if own:
                s["out"] = torch.empty((M, N), dtype=dt, device="cuda")
                s["pre"] = torch.empty((M, rows), dtype=bf16, device="cuda") if c["save"] else None
                s["workspace"] = torch.empty(sk.linear_workspace(s["x"], s["w"], act), dtype=torch.uint8, device="cuda")
            return s
        s["dy"] = _normal(g, (M, N), bf16)
        s["pre"] = 0.6 * _normal(g, (M, rows), bf16) if act else None
        if own:
            s["dx"], s["dw"] = torch.empty_like(s["x"]), torch.empty_like(s["w"])
            s["dbias"] = torch.empty(rows, dtype=torch.float32, device="cuda") if c["bias"] else None
            s["workspace"] = torch.empty(sk.linear_grad_workspace(s["dy"], s["x"], s["w"], act), dtype=torch.uint8,
                                         device="cuda")
        return s
    T, Hq, Hk, D, R = c["T"], c["Hq"], c["Hk"], c["D"], c["R"]
    dt = DTYPES[c["dtype"]]
    # queries and keys where the projection leaves them: beside the values in its rows
    qkv = _normal(g, (T, Hq + 2 * Hk, D), dt)
    s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    s["q_weight"], s["k_weight"] = (1 + 0.1 * _normal(g, (D,), torch.float32)).to(dt), (1 + 0.1 * _normal(g, (D,), torch.float32)).to(dt)
    if not c["norm"]:
        s["q_weight"] = s["k_weight"] = None
    s["eps"] = EPS if c["norm"] else None
    s["positions"] = _positions(g, c)
    angle = torch.arange(POSITIONS, device="cuda", dtype=torch.float64)[:, None] * \
        1e6 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
    s["table"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
    # which axis turns a pair: the pairs in as many sections as there are axes
    s["pair_axis"] = None
    if c["axes"] > 1:
        s["pair_axis"] = (torch.arange(R // 2, device="cuda") * c["axes"] // (R // 2)).to(torch.int32)
    if op == "heads_grad":
        s["dq"], s["dk"] = _normal(g, (T, Hq, D), dt), _normal(g, (T, Hk, D), dt)
    if own:
        s["q_out"], s["k_out"] = torch.empty((T, Hq, D), dtype=dt, device="cuda"), torch.empty((T, Hk, D), dtype=dt, device="cuda")
        if op == "heads_grad":
            s["workspace"] = torch.empty(sk.qk_norm_rope_grad_workspace(T, Hq, Hk, D), dtype=torch.uint8, device="cuda")
            s["dqw"] = s["dkw"] = None
            if c["norm"]:
                s["dqw"], s["dkw"] = torch.empty(D, dtype=torch.float32, device="cuda"), torch.empty(D, dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    c = s["case"]
    op = c["op"]
    if op == "linear":
        y = sk.linear(s["x"], s["w"], bias=s["bias"], activation=s["act"], residual=s["residual"], out=s["out"],
                      pre=s["pre"], workspace=s["workspace"])
        return {"y": y, "pre": s["pre"]} if c["save"] else {"y": y}
    if op == "linear_grad":
        dx, dw, dbias = sk.linear_grad(s["dy"], s["x"], s["w"], pre=s["pre"], activation=s["act"], dx=s["dx"], dw=s["dw"],
                                       dbias=s["dbias"], bias_grad=c["bias"], workspace=s["workspace"])
        return {"dx": dx, "dw": dw, "dbias": dbias} if c["bias"] else {"dx": dx, "dw": dw}
    if op == "heads":
        q, k = sk.qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["table"], s["positions"], eps=s["eps"],
                               pair_axis=s["pair_axis"], interleaved=c["interleaved"], q_out=s["q_out"], k_out=s["k_out"])
        return {"q": q, "k": k}
    q, k, qw, kw = sk.qk_norm_rope_grad(s["dq"], s["dk"], s["q"], s["k"], s["q_weight"], s["k_weight"], s["table"],
                                        s["positions"], eps=s["eps"], pair_axis=s["pair_axis"],
                                        interleaved=c["interleaved"], dq_in=s["q_out"], dk_in=s["k_out"],
                                        dq_weight=s["dqw"], dk_weight=s["dkw"], workspace=s["workspace"])
    return {"q": q, "k": k, "qw": qw, "kw": kw} if c["norm"] else {"q": q, "k": k}


GELU = math.sqrt(2 / math.pi)


def _activation(g, act):
    """(act(g), act'(g)): g * sigmoid(u) with u = g, or the tanh form of the Gaussian one."""
    if act in ("silu", "swiglu"):
        u, du = g, 1.0
    else:
        u, du = 2 * GELU * (g + 0.044715 * g * g * g), 2 * GELU * (1 + 3 * 0.044715 * g * g)
    sig = 1 / (1 + torch.exp(-u))
    return g * sig, sig + g * sig * (1 - sig) * du


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "linear":
        N = c["N"]
        z = s["x"].float() @ s["w"].float().t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = z
        if c["act"] in GATED:
            y = _activation(z[:, :N], c["act"])[0] * z[:, N:]
        elif s["act"]:
            y = _activation(z, c["act"])[0]
        if s["residual"] is not None:
            y = y + s["residual"].float()
        y = y.to(DTYPES[c["out"]])
        return {"y": y, "pre": z.to(torch.bfloat16)} if c["save"] else {"y": y}
    if op == "linear_grad":
        N = c["N"]
        dz = s["dy"].float()
        if s["act"]:
            z = s["pre"].float()
            a, da = _activation(z[:, :N], c["act"])
            dz = torch.cat([dz * z[:, N:] * da, dz * a], dim=1) if c["act"] in GATED else dz * da
        out = {"dx": (dz @ s["w"].float()).to(torch.bfloat16), "dw": (dz.t() @ s["x"].float()).to(torch.bfloat16)}
        if c["bias"]:
            out["dbias"] = dz.sum(0)
        return out
    out = {}
    R = c["R"]
    cos, sin = _angles(s)
    for name in ("q", "k"):
        x = s[name].float()
        w = s[name + "_weight"]
        if op == "heads":
            if c["norm"]:
                x = x / torch.sqrt((x * x).mean(2, keepdim=True) + EPS) * w.float()
            out[name] = _rotated(x, cos, sin, R, c["interleaved"]).to(s[name].dtype)
            continue
        d = _rotated(s["d" + name].float(), cos, -sin, R, c["interleaved"])
        if c["norm"]:
            r = 1 / torch.sqrt((x * x).mean(2, keepdim=True) + EPS)
            out[name + "w"] = (d * x * r).sum((0, 1))
            h = d * w.float()
            d = r * h - x * r ** 3 * (h * x).mean(2, keepdim=True)
        out[name] = d.to(s[name].dtype)
    return out


def _angles(s):
    """(cos, sin) [T, 1, R/2] of every token's pairs."""
    half = s["case"]["R"] // 2
    if s["pair_axis"] is None:
        row = s["table"][s["positions"][0].long()]
        return row[:, None, :half], row[:, None, half:]
    at = s["positions"].long()[s["pair_axis"].long()].t()
    pair = torch.arange(half, device=at.device)[None]
    return s["table"][at, pair][:, None], s["table"][at, half + pair][:, None]


def _rotated(x, cos, sin, R, interleaved):
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y[..., 0:R:2], y[..., 1:R:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y[..., :R // 2], y[..., R // 2:R] = a * cos - b * sin, b * cos + a * sin
    return y


# ------------------------------------------------------------------ the work of one pass

def work(case):
    c = case
    op = c["op"]
    if op in ("linear", "linear_grad"):
        M, N, K = c["M"], c["N"], c["K"]
        rows = 2 * N if c["act"] in GATED else N
        if op == "linear":
            o = SIZES[c["out"]]
            return {"bytes": 2 * rows * K + 2 * M * K + (1 + c["residual"]) * o * M * N + 2 * M * rows * c["save"] + 2 * rows * c["bias"],
                    "flops": 2 * M * rows * K}
        return {"bytes": 4 * rows * K + 4 * M * K + 2 * M * N + (2 * M * rows if c["act"] != "none" else 0) + 4 * rows * c["bias"],
                "flops": 4 * M * rows * K}
    T, H, D, R = c["T"], c["Hq"] + c["Hk"], c["D"], c["R"]
    b = SIZES[c["dtype"]]
    table = 4 * R * min(T, POSITIONS) + 4 * c["axes"] * T
    if op == "heads":
        return {"bytes": 2 * T * H * D * b + table + 2 * D * b * c["norm"], "flops": T * H * (4 * D * c["norm"] + 3 * R)}
    # without the norm the rows themselves are not needed
    return {"bytes": (3 if c["norm"] else 2) * T * H * D * b + table + 2 * D * (4 + b) * c["norm"],
            "flops": T * H * (12 * D * c["norm"] + 3 * R)}


# ------------------------------------------------------------------ from the definition, in 64 bits

def exact(case, seed):
    c = case
    s = prepare(case, seed)
    op = c["op"]
    f64 = torch.float64
    functional = torch.nn.functional

    def act(z):
        if c["act"] == "none":
            return z
        if c["act"] in GATED:
            gate, up = z.chunk(2, dim=1)
            return (functional.silu(gate) if c["act"] == "swiglu" else functional.gelu(gate, approximate="tanh")) * up
        return functional.silu(z) if c["act"] == "silu" else functional.gelu(z, approximate="tanh")

    if op == "linear":
        bias = None if s["bias"] is None else s["bias"].to(f64)
        z = functional.linear(s["x"].to(f64), s["w"].to(f64), bias)
        y = act(z)
        if s["residual"] is not None:
            y = y + s["residual"].to(f64)
        return {"y": y, "pre": z} if c["save"] else {"y": y}
    if op == "linear_grad":
        dz = s["dy"].to(f64)
        if c["act"] != "none":
            z = s["pre"].to(f64).requires_grad_(True)
            dz = torch.autograd.grad(act(z), z, dz)[0]
        out = {"dx": torch.matmul(dz, s["w"].to(f64)), "dw": torch.matmul(s["x"].to(f64).T, dz).T}
        if c["bias"]:
            out["dbias"] = dz.sum(dim=0)
        return out
    # heads turned as complex numbers
    half = c["R"] // 2
    which = torch.zeros(half, dtype=torch.int64, device="cuda") if s["pair_axis"] is None else s["pair_axis"].long()
    position = s["positions"].long().index_select(0, which)               # [pairs, T]
    pair = torch.arange(half, device="cuda")[:, None].expand_as(position)
    turn = torch.complex(s["table"][position, pair].to(f64), s["table"][position, half + pair].to(f64)).T[:, None]

    def heads(x, w):
        if c["norm"]:
            x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS) * w
        head, rest = x[..., :2 * half], x[..., 2 * half:]
        if c["interleaved"]:
            z = torch.view_as_complex(head.reshape(*head.shape[:-1], half, 2).contiguous()) * turn
            head = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(head[..., :half].contiguous(), head[..., half:].contiguous()) * turn
            head = torch.cat([z.real, z.imag], dim=-1)
        return torch.cat([head, rest], dim=-1)

    out = {}
    for name in ("q", "k"):
        x = s[name].to(f64).requires_grad_(op == "heads_grad")
        w = None if s[name + "_weight"] is None else s[name + "_weight"].to(f64).requires_grad_(op == "heads_grad")
        y = heads(x, w)
        if op == "heads":
            out[name] = y
            continue
        grads = torch.autograd.grad(y, [x, w] if c["norm"] else [x], s["d" + name].to(f64))
        out[name] = grads[0]
        if c["norm"]:
            out[name + "w"] = grads[1]
    return out
