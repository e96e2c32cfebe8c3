"""What is measured of the operators around the mixture of experts and the adapters.

Operators (a case's "op"):

  dispatch       tokens sorted by expert: counts, positions, and the rows copied into expert order
  combine        the experts' rows back to their tokens, weighted and summed
  combine_grad   its gradient: into the experts' rows and into the weights
  dispatch_grad  the gradient of the copies: each token's rows summed
  experts        the experts' products on rows in expert order, plain or with SwiGLU
  lora           a shared projection with a low-rank adapter per token beside it

`run` computes them in elementary torch operations in 32 bits, or, where `own` is
true, by the calls a user makes of the framework.
"""
import math

import torch

own = False
sk = None      # the framework's package, once `own` calls for it

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp32": 4}


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
        # one token of a decode step, the router's 256 experts: latency
        {"name": "dispatch one token", "op": "dispatch", "T": 1, "k": 8, "E": 256, "H": 7168, "dtype": "bf16",
         "drop": 0.0, "skew": 0.5},
        # a full decode batch, some entries dropped, an odd number of tokens
        {"name": "dispatch decode", "op": "dispatch", "T": 61, "k": 8, "E": 384, "H": 7168, "dtype": "bf16",
         "drop": 0.1, "skew": 0.5},
        # a training or prefill micro-batch
        {"name": "dispatch train", "op": "dispatch", "T": 8192, "k": 8, "E": 256, "H": 7168, "dtype": "bf16",
         "drop": 0.0, "skew": 1.0},
        # a decode batch: the down product's fp32 rows back to bf16 tokens
        {"name": "combine decode", "op": "combine", "T": 64, "k": 8, "E": 256, "H": 7168, "dtype": "fp32",
         "out": "bf16", "drop": 0.0, "skew": 0.5},
        # training, some entries dropped
        {"name": "combine train", "op": "combine", "T": 8192, "k": 8, "E": 256, "H": 7168, "dtype": "bf16",
         "out": "bf16", "drop": 0.05, "skew": 1.0},
        # the two backward passes of a training step; the second with a width that is no multiple of anything
        {"name": "combine grad train", "op": "combine_grad", "T": 8192, "k": 8, "E": 256, "H": 7168, "dtype": "bf16",
         "drop": 0.0, "skew": 1.0},
        {"name": "dispatch grad odd", "op": "dispatch_grad", "T": 3001, "k": 6, "E": 64, "H": 2881, "dtype": "fp32",
         "drop": 0.05, "skew": 1.0},
        # one token: the first product of the smaller model's layer
        {"name": "experts one token", "op": "experts", "T": 1, "k": 4, "E": 32, "N": 2880, "K": 2880,
         "act": "none", "out": "bf16", "drop": 0.0, "skew": 0.5},
        # a decode batch: gate and up products with SwiGLU, about half of the experts touched
        {"name": "experts swiglu", "op": "experts", "T": 16, "k": 8, "E": 256, "N": 2048, "K": 7168,
         "act": "swiglu", "out": "bf16", "drop": 0.0, "skew": 0.5},
        # a large decode batch: the down product, nearly all experts touched, some with many rows
        {"name": "experts down", "op": "experts", "T": 64, "k": 8, "E": 256, "N": 7168, "K": 2048,
         "act": "none", "out": "fp32", "drop": 0.0, "skew": 1.0},
        # one request with a small adapter on the first projection: latency
        {"name": "lora one token", "op": "lora", "M": 1, "slots": 8, "distinct": 1, "R": 16, "N": 2112, "K": 7168,
         "ranks": "same", "none": 0.0, "out": "fp32"},
        # a full batch on the wide projection, nearly every token with an adapter of its own, ranks mixed
        {"name": "lora many", "op": "lora", "M": 64, "slots": 96, "distinct": 48, "R": 64, "N": 24576, "K": 1536,
         "ranks": "mixed", "none": 0.1, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: a multiple of 64 mostly, of 8 sometimes, any at times."""
    v = _log(rng, lo, hi)
    m = rng.choice([64, 64, 64, 8, 1])
    return max(m, v // m * m)


def draw(rng):
    op = rng.choice(["dispatch", "combine", "combine_grad", "dispatch_grad", "experts", "lora", "experts", "lora"])
    if op in ("dispatch", "combine", "combine_grad", "dispatch_grad"):
        k = rng.choice([1, 2, 4, 6, 8, 10])
        E = _log(rng, max(8, k), 512)
        H = _width(rng, 64, 8192)
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        T = _log(rng, 1, 16384)
        T = max(1, min(T, 8192 * 8 * 7168 * 2 // (k * H * SIZES[dtype])))
        c = {"op": op, "T": T, "k": k, "E": E, "H": H, "dtype": dtype, "drop": rng.choice([0.0, 0.0, 0.1, 0.5]),
             "skew": rng.choice([0.0, 0.5, 1.0, 3.0])}
        if op == "combine":
            c["out"] = "bf16" if dtype == "bf16" else rng.choice(["bf16", "fp32"])
        return c
    if op == "experts":
        E = _log(rng, 4, 256)
        N = _width(rng, 64, 8192)
        K = _width(rng, 64, 8192)
        act = rng.choice(["none", "swiglu"])
        E = max(4, min(E, (1 << 31) // (N * K * (2 if act == "swiglu" else 1))))
        return {"op": op, "T": _log(rng, 1, 64), "k": min(E, rng.choice([1, 2, 4, 8])), "E": E, "N": N, "K": K,
                "act": act, "out": rng.choice(["bf16", "fp32"]), "drop": rng.choice([0.0, 0.0, 0.2]),
                "skew": rng.choice([0.0, 0.5, 1.0, 3.0])}
    M = _log(rng, 1, 64)
    slots = _log(rng, 1, 128)
    # an odd K or N is served up to 16 tokens
    N, K = _width(rng, 64, 16384), _width(rng, 64, 8192)
    if M > 16:
        K = max(64, K // 8 * 8)
    R = rng.choice([4, 8, 16, 16, 32, 64, 128, 24])
    return {"op": op, "M": M, "slots": slots, "distinct": min(slots, _log(rng, 1, M)), "R": R, "N": N, "K": K,
            "ranks": rng.choice(["same", "mixed"]), "none": rng.choice([0.0, 0.1, 0.5]),
            "out": rng.choice(["bf16", "fp32"])}


# ------------------------------------------------------------------ inputs

def _route(g, c):
    """The router's choices: k different experts a token, some experts liked more; dropped entries are -1."""
    T, k, E = c["T"], c["k"], c["E"]
    logits = torch.randn(T, E, generator=g, device="cuda")
    logits += c["skew"] * torch.randn(E, generator=g, device="cuda")
    top = logits.topk(k, dim=1)
    ids = top.indices.to(torch.int32)
    weights = torch.softmax(top.values, dim=1)
    if c["drop"] > 0:
        ids[torch.rand(T, k, generator=g, device="cuda") < c["drop"]] = -1
        if T > 1:
            ids[T // 2] = -1      # a token of which nothing is left
    return ids.contiguous(), weights.contiguous()


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _uniform(g, shape, K):
    """Weights U(-1/sqrt(K), 1/sqrt(K)) in bf16."""
    b = 1.0 / math.sqrt(K)
    return torch.empty(shape, device="cuda", dtype=torch.bfloat16).uniform_(-b, b, generator=g)


def _positions(ids, E):
    """(pos, order, offsets) of the stable sort by expert: what a dispatch before this call has left."""
    T, k = ids.shape
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    order = torch.sort(key, stable=True).indices
    counts = torch.zeros(E + 1, dtype=torch.int64, device=ids.device).index_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = counts[:E].cumsum(0)
    at = torch.arange(T * k, device=ids.device)
    live = at < offsets[E]
    pos = torch.empty_like(order)
    pos[order] = torch.where(live, at, torch.full_like(at, -1))
    order = torch.where(live, order, torch.full_like(order, -1))
    return pos.reshape(T, k).int(), order.int(), offsets.int()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(1_000_003 * (seed + 1))
    s = {"case": c}
    op = c["op"]
    if own:
        _package()
    if op == "lora":
        M, N, K, R, L = c["M"], c["N"], c["K"], c["R"], c["slots"]
        s["x"] = _normal(g, (M, K), torch.bfloat16)
        s["w"] = _uniform(g, (N, K), K)
        s["a"] = _uniform(g, (L, R, K), K)
        s["b"] = _uniform(g, (L, N, R), R)
        used = torch.randperm(L, generator=g, device="cuda")[:c["distinct"]]
        ids = used[torch.randint(0, c["distinct"], (M,), generator=g, device="cuda")]
        n = min(M, c["distinct"])
        ids[:n] = used[:n]
        ids = ids[torch.randperm(M, generator=g, device="cuda")]
        if c["none"] > 0:
            ids[torch.rand(M, generator=g, device="cuda") < c["none"]] = -1
        s["ids"] = ids.to(torch.int32)
        share = torch.randint(0, 3, (L,), generator=g, device="cuda") if c["ranks"] == "mixed" else torch.zeros(L, device="cuda", dtype=torch.int64)
        s["ranks"] = (torch.tensor(R, device="cuda") // (2 ** share)).clamp(min=1).to(torch.int32)
        s["scales"] = 0.5 + 1.5 * torch.rand(L, generator=g, device="cuda")
        s["out"] = torch.empty((M, N), dtype=DTYPES[c["out"]], device="cuda")
        if own:
            s["workspace"] = torch.empty(sk.lora_workspace(M, N, R, s["out"].dtype), dtype=torch.uint8, device="cuda")
        return s
    T, k, E = c["T"], c["k"], c["E"]
    ids, weights = _route(g, c)
    rows = T * k
    if op == "dispatch":
        dt = DTYPES[c["dtype"]]
        s["ids"] = ids
        s["x"] = _normal(g, (T, c["H"]), dt)
        if own:
            s["xs"] = torch.zeros((rows, c["H"]), dtype=dt, device="cuda")
            s["pos"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
            s["order"] = torch.empty(rows, dtype=torch.int32, device="cuda")
            s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        return s
    s["pos"], s["order"], s["offsets"] = _positions(ids, E)
    if op == "experts":
        N, K = c["N"], c["K"]
        s["w"] = _uniform(g, (E, 2 * N if c["act"] == "swiglu" else N, K), K)
        x = _normal(g, (T, K), torch.bfloat16)
        s["xs"] = x[(s["order"].long().clamp(min=0)) // k].contiguous()
        s["out"] = torch.zeros((rows, N), dtype=DTYPES[c["out"]], device="cuda")
        return s
    dt = DTYPES[c["dtype"]]
    H = c["H"]
    s["weights"] = weights
    if op == "combine_grad":
        s["dy"] = _normal(g, (T, H), dt)
        s["ys"] = _normal(g, (rows, H), dt)
        if own:
            s["dys"] = torch.zeros((rows, H), dtype=dt, device="cuda")
            s["dweights"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
        return s
    s["ys"] = _normal(g, (rows, H), dt)
    if own:
        s["out"] = torch.empty((T, H), dtype=DTYPES[c["out"]] if op == "combine" else dt, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    op = s["case"]["op"]
    if op == "dispatch":
        xs, pos, order, offsets = sk.expert_dispatch(s["ids"], s["case"]["E"], x=s["x"], xs=s["xs"], pos=s["pos"],
                                                     order=s["order"], offsets=s["offsets"])
        return {"xs": xs, "pos": pos, "order": order, "offsets": offsets}
    if op == "combine":
        return sk.expert_combine(s["ys"], s["pos"], s["weights"], out=s["out"])
    if op == "dispatch_grad":
        return sk.expert_combine(s["ys"], s["pos"], None, out=s["out"])
    if op == "combine_grad":
        dys, dw = sk.expert_combine_grad(s["dy"], s["ys"], s["pos"], s["weights"], dys=s["dys"], dweights=s["dweights"])
        return {"dys": dys, "dweights": dw}
    if op == "experts":
        return sk.experts_gemm(s["xs"], s["offsets"], s["w"], out=s["out"], activation=s["case"]["act"])
    return sk.lora_gemm(s["x"], s["w"], s["a"], s["b"], s["ids"], ranks=s["ranks"], scales=s["scales"], out=s["out"],
                        workspace=s["workspace"])


def _gathered(rows, pos_j):
    """rows[pos_j] in 32 bits, zeros where pos_j < 0."""
    live = (pos_j >= 0)[:, None]
    return torch.where(live, rows[pos_j.long().clamp(min=0)].float(), torch.zeros((), device=rows.device))


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "dispatch":
        pos, order, offsets = _positions(s["ids"], c["E"])
        n = pos.numel()
        xs = torch.zeros((n + 1, c["H"]), dtype=s["x"].dtype, device="cuda")
        to = torch.where(pos >= 0, pos, torch.full_like(pos, n)).long()
        for j in range(c["k"]):
            xs[to[:, j]] = s["x"]
        return {"xs": xs[:n], "pos": pos, "order": order, "offsets": offsets}
    if op in ("combine", "dispatch_grad"):
        y = torch.zeros((c["T"], c["H"]), dtype=torch.float32, device="cuda")
        for j in range(c["k"]):
            r = _gathered(s["ys"], s["pos"][:, j])
            y += r * s["weights"][:, j, None] if op == "combine" else r
        return y.to(DTYPES[c["out"]] if op == "combine" else s["ys"].dtype)
    if op == "combine_grad":
        n = s["pos"].numel()
        dys = torch.zeros((n + 1, c["H"]), dtype=s["ys"].dtype, device="cuda")
        dw = torch.zeros_like(s["weights"])
        dy = s["dy"].float()
        for j in range(c["k"]):
            p = s["pos"][:, j]
            dys[torch.where(p >= 0, p, torch.full_like(p, n)).long()] = (dy * s["weights"][:, j, None]).to(dys.dtype)
            dw[:, j] = (dy * _gathered(s["ys"], p)).sum(1)
        return {"dys": dys[:n], "dweights": dw}
    if op == "experts":
        out = torch.zeros_like(s["out"])
        off = s["offsets"].tolist()
        for e in range(c["E"]):
            a, b = off[e], off[e + 1]
            if a == b:
                continue
            y = s["xs"][a:b].float() @ s["w"][e].float().t()
            if c["act"] == "swiglu":
                gate, up = y[:, :c["N"]], y[:, c["N"]:]
                y = gate / (1 + torch.exp(-gate)) * up
            out[a:b] = y.to(out.dtype)
        return out
    y = s["x"].float() @ s["w"].float().t()
    ids = s["ids"].long()
    slot = ids.clamp(min=0)
    v = (s["a"][slot].float() * s["x"].float()[:, None, :]).sum(2)
    live = (ids >= 0)[:, None] & (torch.arange(c["R"], device="cuda")[None] < s["ranks"][slot][:, None])
    v = torch.where(live, v, torch.zeros((), device="cuda")) * s["scales"][slot][:, None]
    y += (s["b"][slot].float() @ v[:, :, None])[:, :, 0]
    return y.to(s["out"].dtype)


# ------------------------------------------------------------------ the work of one pass

def work(case):
    c = case
    op = c["op"]
    if op == "lora":
        o = SIZES[c["out"]]
        M, N, K = c["M"], c["N"], c["K"]
        rank = c["R"] * (1.0 if c["ranks"] == "same" else (1 + 0.5 + 0.25) / 3)
        live = M * (1 - c["none"])
        n = c["distinct"] * (1 - c["none"] ** max(1.0, M / c["distinct"]))
        return {"bytes": 2 * N * K + n * rank * 2 * (N + K) + 2 * M * K + o * M * N,
                "flops": 2 * M * N * K + 2 * live * rank * (N + K)}
    T, k, E = c["T"], c["k"], c["E"]
    n = T * k * (1 - c["drop"])
    if op == "experts":
        o = SIZES[c["out"]]
        N, K = c["N"], c["K"]
        rows = 2 * N if c["act"] == "swiglu" else N
        # the experts that a typical draw of this routing touches
        r = torch.Generator().manual_seed(7)
        touched = 0.0
        for _ in range(3):
            logits = torch.randn(T, E, generator=r) + c["skew"] * torch.randn(E, generator=r)
            ids = logits.topk(k, dim=1).indices
            ids = ids[torch.rand(T, k, generator=r) >= c["drop"]]
            touched += ids.unique().numel() / 3
        return {"bytes": max(1.0, touched) * rows * K * 2 + n * K * 2 + n * N * o + 4 * E, "flops": 2 * n * rows * K}
    b = SIZES[c["dtype"]]
    H = c["H"]
    if op == "dispatch":
        return {"bytes": T * H * b + n * H * b + 12 * T * k + 4 * E, "flops": 0}
    if op in ("combine", "dispatch_grad"):
        o = SIZES[c["out"]] if op == "combine" else b
        return {"bytes": n * H * b + T * H * o + T * k * (8 if op == "combine" else 4), "flops": 2 * n * H}
    return {"bytes": T * H * b + 2 * n * H * b + 12 * T * k, "flops": 3 * n * H}


# ------------------------------------------------------------------ from the definition, in 64 bits

def exact(case, seed):
    c = case
    s = prepare(case, seed)
    op = c["op"]
    f64 = torch.float64
    if op == "lora":
        x = s["x"].to(f64)
        y = torch.matmul(x, s["w"].to(f64).T)
        for m, a in enumerate(s["ids"].tolist()):
            if a < 0:
                continue
            r = int(s["ranks"][a])
            low = torch.mv(s["a"][a, :r].to(f64), x[m])
            y[m] += float(s["scales"][a].to(f64)) * torch.mv(s["b"][a, :, :r].to(f64), low)
        return y
    T, k, E = c["T"], c["k"], c["E"]
    if op == "dispatch":
        H = c["H"]
        lists = [[] for _ in range(E)]
        for f, e in enumerate(s["ids"].reshape(-1).tolist()):
            if 0 <= e < E:
                lists[e].append(f)
        order = [f for l in lists for f in l]
        pos, offsets = [-1] * (T * k), [0]
        for l in lists:
            offsets.append(offsets[-1] + len(l))
        for p, f in enumerate(order):
            pos[f] = p
        xs = torch.zeros((T * k, H), dtype=f64, device="cuda")
        token = torch.tensor(order, dtype=torch.int64, device="cuda") // k
        xs[:len(order)] = s["x"].to(f64).index_select(0, token)
        order += [-1] * (T * k - len(order))
        t32 = torch.int32
        return {"xs": xs, "pos": torch.tensor(pos, dtype=t32).reshape(T, k), "order": torch.tensor(order, dtype=t32),
                "offsets": torch.tensor(offsets, dtype=t32)}
    if op == "experts":
        N = c["N"]
        out = torch.zeros((T * k, N), dtype=f64, device="cuda")
        off = s["offsets"].cpu().numpy()
        for e in range(E):
            rows = slice(int(off[e]), int(off[e + 1]))
            if rows.start == rows.stop:
                continue
            h = torch.matmul(s["w"][e].to(f64), s["xs"][rows].to(f64).T).T
            out[rows] = torch.nn.functional.silu(h[:, :N]) * h[:, N:] if c["act"] == "swiglu" else h
        return out
    flat = s["pos"].reshape(-1).long()
    entry = torch.nonzero(flat >= 0).reshape(-1)
    H = c["H"]
    w = s["weights"].reshape(-1).to(f64)
    pieces = 16       # of the width, to bound the memory
    if op == "combine_grad":
        dys = torch.zeros((T * k, H), dtype=f64, device="cuda")
        dw = torch.zeros(T * k, dtype=f64, device="cuda")
        for cols in torch.arange(H, device="cuda").chunk(pieces):
            lo, hi = int(cols[0]), int(cols[-1]) + 1
            dy = s["dy"][:, lo:hi].to(f64)[entry // k]
            dys[flat[entry], lo:hi] = w[entry, None] * dy
            dw[entry] += (dy * s["ys"][flat[entry], lo:hi].to(f64)).sum(1)
        return {"dys": dys, "dweights": dw.reshape(T, k)}
    y = torch.zeros((T, H), dtype=f64, device="cuda")
    for cols in torch.arange(H, device="cuda").chunk(pieces):
        lo, hi = int(cols[0]), int(cols[-1]) + 1
        r = s["ys"][flat[entry], lo:hi].to(f64)
        if op == "combine":
            r = r * w[entry, None]
        y[:, lo:hi] = torch.zeros((T, hi - lo), dtype=f64, device="cuda").index_add_(0, entry // k, r)
    return y
