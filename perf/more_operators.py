"""The measured cases of the operators around the routed experts of a block: the
16-bit product with bias, activation and residual (a shared expert, a dense
layer) and its gradients; the norms after and before a block with its gate and
residual scale, and their gradients; the router's balance loss with the counts
of every expert, and the gradient of the logits.

`run` computes a case either in its plain form (elementary torch operations) or,
with `own` set, through the library's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6
COEF, Z_COEF = 0.01, 0.001


def listed():
    return [
        # one token through a shared expert's down product, added to the hidden state: a weight stream
        dict(name="product one token", op="matmul", M=1, N=7168, K=2048, dtype="bf16", out="bf16", act="none",
             bias=False, residual=True, pre=False),
        # a decode batch through the gate and up weights of a shared expert
        dict(name="product gated decode", op="matmul", M=24, N=2048, K=7168, dtype="bf16", out="bf16", act="swiglu",
             bias=False, residual=False, pre=False),
        # a training step's forward through a wide dense layer, its input of the activation kept
        dict(name="product training", op="matmul", M=8192, N=7168, K=7168, dtype="bf16", out="bf16", act="gelu",
             bias=True, residual=False, pre=True),
        # the backward of a shared expert's gate and up product
        dict(name="product gradient gated", op="matmul_grad", M=4096, N=2048, K=7168, dtype="bf16", grad="bf16",
             act="swiglu", bias=False),
        # ragged sizes, fp16, gradients in the weights' own type
        dict(name="product gradient odd", op="matmul_grad", M=1001, N=1030, K=777, dtype="f16", grad="f16",
             act="gelu", bias=True),
        # one token of a decode step between two blocks: latency
        dict(name="norm one token", op="norm", T=1, H=7168, dtype="bf16", weight="bf16", post=True, gate="none",
             scale=1.0),
        # a prefill between two blocks
        dict(name="norm prefill", op="norm", T=8192, H=7168, dtype="bf16", weight="bf16", post=True, gate="channel",
             scale=1.0),
        # the same place in a training step's backward
        dict(name="norm gradient", op="norm_grad", T=8192, H=7168, dtype="bf16", weight="f32", post=True,
             gate="channel", scale=1.0),
        # a block's output gated by token, in 32 bits, a width that no vector load divides
        dict(name="norm gradient odd", op="norm_grad", T=1023, H=2049, dtype="f32", weight="f32", post=False,
             gate="token", scale=0.5),
        # a small batch's load of the experts: latency
        dict(name="balance small", op="balance", T=64, E=896, k=16, dtype="f32", score="softmax", S=1, mask=0.0,
             grad=False),
        # a training step's router: the loss, then the logits' gradient with that of the routing weights
        dict(name="balance training", op="balance", T=16384, E=896, k=16, dtype="f32", score="softmax", S=1, mask=0.0,
             grad=True),
        # a loss for each sequence of a padded batch, 16-bit logits
        dict(name="balance sequences", op="balance", T=10007, E=61, k=6, dtype="bf16", score="sigmoid", S=37, mask=0.1,
             grad=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["matmul", "matmul", "matmul_grad", "norm", "norm_grad", "balance"])
    if op in ("matmul", "matmul_grad"):
        N, K = _log(rng, 64, 8192), _log(rng, 64, 8192)
        if rng.random() < 0.5:
            N, K = max(64, N // 64 * 64), max(64, K // 64 * 64)
        act = rng.choice(["none", "relu", "silu", "gelu", "swiglu"])
        # products of N x K: two rows of weights a column when gated, two products in a backward
        each = N * K * (2 if act == "swiglu" else 1) * (2 if op == "matmul_grad" else 1)
        M = max(1, min(_log(rng, 1, 8192), 400_000_000_000 // each))
        c = dict(op=op, M=M, N=N, K=K, dtype=rng.choice(["bf16", "f16"]), act=act, bias=rng.random() < 0.5)
        if op == "matmul":
            c.update(out=rng.choice([c["dtype"], "f32"]), residual=rng.random() < 0.5, pre=rng.random() < 0.4)
        else:
            # behind an activation the products take their gradient in 16 bits, and give theirs in the same
            c.update(grad=rng.choice([c["dtype"], "f32"]) if act == "none" else c["dtype"])
        return c
    if op in ("norm", "norm_grad"):
        H = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            H = max(64, H // 64 * 64)
        dtype = rng.choice(["bf16", "f16", "f32"])
        T = max(1, min(_log(rng, 1, 16384), 100_000_000 // (H * BYTES[dtype])))
        return dict(op=op, T=T, H=H, dtype=dtype, weight=rng.choice([dtype, "f32"]), post=rng.random() < 0.6,
                    gate=rng.choice(["none", "channel", "token", "full"]), scale=rng.choice([1.0, 1.0, 0.5]))
    E = _log(rng, 8, 1024)
    T = max(1, min(_log(rng, 1, 65536), 14_000_000 // E))
    return dict(op=op, T=T, E=E, k=rng.randint(1, min(E, 16)), dtype=rng.choice(["f32", "f32", "bf16", "f16"]),
                score=rng.choice(["softmax", "sigmoid"]), S=rng.choice([1, 1, min(T, rng.randint(2, 64))]),
                mask=rng.choice([0.0, 0.0, 0.2]), grad=rng.random() < 0.7)


# ---- inputs -----------------------------------------------------------------
def _padded(rows, cols, sigma, dt, g):
    """Normal values; rows of a multiple of 16 bytes, as the product takes its operands."""
    v = torch.randn(rows, -(-cols // 8) * 8, generator=g, device="cuda", dtype=torch.float32)
    return v.mul_(sigma).to(dt)


def _vector(n, mean, sigma, dt, g):
    return (mean + sigma * torch.randn(n, generator=g, device="cuda")).to(dt)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, dev, op = dict(case), "cuda", case["op"]
    dt = DTYPES[c["dtype"]]
    s = {"case": c}
    if op in ("matmul", "matmul_grad"):
        M, N, K = c["M"], c["N"], c["K"]
        wide = 2 * N if c["act"] == "swiglu" else N  # rows of w: the gate's, then the up product's
        s["x"] = _padded(M, K, 1.0, dt, g)
        s["w"] = _padded(wide, K, 1.5 * K ** -0.5, dt, g)
        s["bias"] = _vector(wide, 0.0, 0.3, dt, g) if c["bias"] else None
        if op == "matmul":
            out = DTYPES[c["out"]]
            s["residual"] = torch.randn(M, N, generator=g, device=dev).to(out) if c["residual"] else None
            s["y"] = torch.zeros(M, N, dtype=out, device=dev)
            s["pre"] = torch.zeros(M, wide, dtype=dt, device=dev) if c["pre"] else None
            return s
        grad = DTYPES[c["grad"]]
        s["dy"] = _padded(M, N, 0.1, dt, g)
        s["pre"] = _padded(M, wide, 1.5, dt, g) if c["act"] != "none" else None
        s["dz"] = torch.zeros(M, -(-wide // 8) * 8, dtype=dt, device=dev) if c["act"] != "none" else None
        s["dx"] = torch.zeros(M, K, dtype=dt, device=dev)
        s["dw"] = torch.zeros(wide, K, dtype=grad, device=dev)
        s["dbias"] = torch.zeros(wide, dtype=grad, device=dev) if c["bias"] else None
        return s
    if op in ("norm", "norm_grad"):
        T, H, wt = c["T"], c["H"], DTYPES[c["weight"]]
        spread = torch.exp(0.5 * torch.randn(T, 1, generator=g, device=dev))
        s["u"] = (torch.randn(T, H, generator=g, device=dev) * spread).to(dt)
        s["post_weight"] = _vector(H, 1.0, 0.2, wt, g) if c["post"] else None
        s["pre_weight"] = _vector(H, 1.0, 0.2, wt, g)
        if c["gate"] == "channel":
            s["gate"] = _vector(H, 0.5, 0.2, wt, g)
        elif c["gate"] == "token":  # the sigmoid of a product, in 32 bits
            s["gate"] = torch.sigmoid(torch.randn(T, generator=g, device=dev))
        elif c["gate"] == "full":
            s["gate"] = torch.sigmoid(torch.randn(T, H, generator=g, device=dev)).to(dt)
        else:
            s["gate"] = None
        hidden = (3.0 * torch.randn(T, H, generator=g, device=dev) * spread).to(dt)
        if op == "norm":
            s["residual"] = hidden
            s["h"], s["n"] = torch.zeros(T, H, dtype=dt, device=dev), torch.zeros(T, H, dtype=dt, device=dev)
            return s
        s["h"] = hidden
        s["dh"] = torch.randn(T, H, generator=g, device=dev).mul_(0.1).to(dt)
        s["dn"] = torch.randn(T, H, generator=g, device=dev).mul_(0.1).to(dt)
        s["du"], s["dresidual"] = torch.zeros(T, H, dtype=dt, device=dev), torch.zeros(T, H, dtype=dt, device=dev)
        s["dpost_weight"] = torch.zeros(H, device=dev) if c["post"] else None
        s["dpre_weight"] = torch.zeros(H, device=dev)
        s["dgate"] = {"none": None, "channel": torch.zeros(H, device=dev), "token": torch.zeros(T, device=dev),
                      "full": torch.zeros(T, H, dtype=dt, device=dev)}[c["gate"]]
        s["workspace"] = _workspace(lambda dfm: dfm.block_norm_grad_workspace(T, H))
        return s
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    logits = torch.randn(T, E, generator=g, device=dev) + 0.7 * torch.randn(E, generator=g, device=dev)
    top = logits.topk(k, dim=1)
    s["ids"] = top.indices.to(torch.int32).contiguous()
    scores = torch.sigmoid(top.values) if c["score"] == "sigmoid" else torch.softmax(top.values, dim=1)
    s["weights"] = (scores / scores.sum(1, keepdim=True)).contiguous()
    s["logits"] = logits.to(dt)
    s["mask"] = (torch.rand(T, generator=g, device=dev) >= c["mask"]).to(torch.uint8) if c["mask"] else None
    s["offs"] = None
    if S > 1:  # sequences of any lengths, all rows in one
        cut = torch.randint(0, T + 1, (S - 1,), generator=g, device=dev).sort().values
        s["offs"] = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), T)]).to(torch.int32)
    s["loss"], s["probs"] = torch.zeros(S, device=dev), torch.zeros(S, E, device=dev)
    s["counts"] = torch.zeros(S, E, dtype=torch.int32, device=dev)
    s["tokens"] = torch.zeros(S, dtype=torch.int32, device=dev)
    s["workspace"] = _workspace(lambda dfm: dfm.balance_loss_workspace(T, E, S))
    if c["grad"]:
        s["dloss"] = 0.5 + torch.rand(S, generator=g, device=dev)
        s["dweights"] = torch.randn(T, k, generator=g, device=dev).mul_(0.01 / T)
        s["dlogits"] = torch.zeros(T, E, dtype=dt, device=dev)
    return s


def _workspace(size):
    """The library's scratch, which a program allocates once."""
    if not own:
        return None
    import mxfp4_routed_expert_top_gb300 as dfm
    return torch.empty(size(dfm), dtype=torch.uint8, device="cuda")


# ---- the plain forms --------------------------------------------------------
def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    gate, up = z.chunk(2, dim=1)
    return gate / (1 + torch.exp(-gate)) * up


def _matmul(s):
    c = s["case"]
    z = s["x"][:, :c["K"]].float() @ s["w"][:, :c["K"]].float().t()
    if c["bias"]:
        z = z + s["bias"].float()
    y = _act(z, c["act"])
    if c["residual"]:
        y = y + s["residual"].float()
    out = {"y": y.to(DTYPES[c["out"]])}
    if c["pre"]:
        out["pre"] = z.to(DTYPES[c["dtype"]])
    return out


def _dact(dy, z, act):
    if act == "none":
        return dy
    if act == "relu":
        return dy * (z > 0)
    if act == "gelu":
        return dy * (0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi)))
    gate, up = (z, None) if act == "silu" else z.chunk(2, dim=1)
    sig = 1 / (1 + torch.exp(-gate))
    slope = sig * (1 + gate * (1 - sig))
    if act == "silu":
        return dy * slope
    return torch.cat([dy * up * slope, dy * gate * sig], dim=1)


def _matmul_grad(s):
    c = s["case"]
    wide = 2 * c["N"] if c["act"] == "swiglu" else c["N"]
    dt, grad = DTYPES[c["dtype"]], DTYPES[c["grad"]]
    z = s["pre"][:, :wide].float() if c["act"] != "none" else None
    dz = _dact(s["dy"][:, :c["N"]].float(), z, c["act"])
    out = {"dx": (dz @ s["w"][:, :c["K"]].float()).to(dt), "dw": (dz.t() @ s["x"][:, :c["K"]].float()).to(grad)}
    if c["bias"]:
        out["dbias"] = dz.sum(0).to(grad)
    return out


def _rstd(v):
    return 1 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)


def _gate(s):
    """The gate as it multiplies rows [T, H], or 1."""
    gate = s["gate"]
    if gate is None:
        return 1.0
    return gate.float()[:, None] if s["case"]["gate"] == "token" else gate.float()


def _norm(s):
    c, dt = s["case"], DTYPES[s["case"]["dtype"]]
    a = s["u"].float()
    if c["post"]:
        a = a * _rstd(a) * s["post_weight"].float()
    h = c["scale"] * s["residual"].float() + _gate(s) * a
    n = h * _rstd(h) * s["pre_weight"].float()
    return {"h": h.to(dt), "n": n.to(dt)}


def _norm_grad(s):
    c, dt = s["case"], DTYPES[s["case"]["dtype"]]
    h, dn, u = s["h"].float(), s["dn"].float(), s["u"].float()
    rstd, weighted = _rstd(h), dn * s["pre_weight"].float()
    hat = h * rstd
    dh = s["dh"].float() + rstd * (weighted - hat * (weighted * hat).mean(1, keepdim=True))
    out = {"dresidual": (c["scale"] * dh).to(dt), "dpre_weight": (dn * hat).sum(0)}
    du = _gate(s) * dh
    a = u
    if c["post"]:
        rstd = _rstd(u)
        hat = u * rstd
        a = hat * s["post_weight"].float()
        out["dpost_weight"] = (du * hat).sum(0)
        weighted = du * s["post_weight"].float()
        du = rstd * (weighted - hat * (weighted * hat).mean(1, keepdim=True))
    out["du"] = du.to(dt)
    if c["gate"] != "none":
        each = dh * a
        out["dgate"] = {"channel": lambda: each.sum(0), "token": lambda: each.sum(1), "full": lambda: each.to(dt)}[c["gate"]]()
    return out


def _sequence(s):
    """The sequence of every row."""
    T, offs = s["case"]["T"], s["offs"]
    rows = torch.arange(T, device=s["logits"].device)
    return torch.zeros_like(rows) if offs is None else torch.searchsorted(offs[1:].long(), rows, right=True)


def _balance(s):
    c = s["case"]
    E, k, S = c["E"], c["k"], c["S"]
    seq, z = _sequence(s), s["logits"].float()
    there = s["mask"].float() if s["mask"] is not None else torch.ones(c["T"], device=z.device)
    most = z.max(1, keepdim=True).values
    lse = most[:, 0] + torch.log(torch.exp(z - most).sum(1))
    if c["score"] == "sigmoid":
        sig = 1 / (1 + torch.exp(-z))
        p = sig / sig.sum(1, keepdim=True)
    else:
        sig = 0.0
        p = torch.exp(z - lse[:, None])
    tokens = torch.zeros(S, device=z.device).index_add_(0, seq, there)
    each = 1 / tokens.clamp(min=1)
    probs = torch.zeros(S, E, device=z.device).index_add_(0, seq, p * there[:, None]) * each[:, None]
    key = torch.where(there[:, None] > 0, seq[:, None] * E + s["ids"].long(), S * E)
    counts = torch.bincount(key.reshape(-1), minlength=S * E + 1)[:-1].view(S, E)
    f = counts.float() * (E / k) * each[:, None]
    zsum = torch.zeros(S, device=z.device).index_add_(0, seq, lse * lse * there)
    out = {"loss": COEF * (f * probs).sum(1) + Z_COEF * zsum * each, "counts": counts.to(torch.int32),
           "tokens": tokens.to(torch.int32), "probs": probs}
    if c["grad"]:
        ft = f[seq]
        d = COEF * p * (1 - sig) * (ft - (ft * p).sum(1, keepdim=True))
        d = d + 2 * Z_COEF * lse[:, None] * torch.exp(z - lse[:, None])
        d = d * (s["dloss"] * each)[seq][:, None]
        w, dw = s["weights"], s["dweights"]
        kept = w * (dw - (w * dw).sum(1, keepdim=True))
        if c["score"] == "sigmoid":
            kept = kept * (1 - sig.gather(1, s["ids"].long()))
        d = d.scatter_add(1, s["ids"].long(), kept)
        out["dlogits"] = (d * there[:, None]).to(s["logits"].dtype)
    return out


# ---- one pass ---------------------------------------------------------------
def _run_own(s):
    import mxfp4_routed_expert_top_gb300 as dfm
    c = s["case"]
    op = c["op"]
    if op == "matmul":
        dfm.matmul(s["x"], s["w"], c["dtype"], c["M"], c["N"], c["K"], s["y"], c["out"], bias=s["bias"], act=c["act"],
                   residual=s["residual"], pre=s["pre"], ldx=s["x"].shape[1], ldw=s["w"].shape[1])
        return {"y": s["y"], "pre": s["pre"]} if c["pre"] else {"y": s["y"]}
    if op == "matmul_grad":
        kw = {} if c["act"] == "none" else dict(pre=s["pre"], ldp=s["pre"].shape[1], dz=s["dz"], lddz=s["dz"].shape[1])
        dfm.matmul_grad(s["dy"], s["x"], s["w"], c["dtype"], c["M"], c["N"], c["K"], dx=s["dx"], dw=s["dw"],
                        dbias=s["dbias"], grad_dtype=c["grad"], act=c["act"], lddy=s["dy"].shape[1],
                        ldx=s["x"].shape[1], ldw=s["w"].shape[1], **kw)
        return {key: s[key] for key in ("dx", "dw", "dbias") if s[key] is not None}
    if op == "norm":
        dfm.block_norm(s["u"], s["residual"], c["dtype"], c["T"], c["H"], s["h"], s["n"], post=c["post"],
                       post_weight=s["post_weight"], gate=s["gate"], gate_kind=c["gate"], residual_scale=c["scale"],
                       pre_weight=s["pre_weight"], weight_dtype=c["weight"], eps=EPS)
        return {"h": s["h"], "n": s["n"]}
    if op == "norm_grad":
        dfm.block_norm_grad(s["dh"], s["dn"], s["u"], s["h"], c["dtype"], c["T"], c["H"], s["du"], s["dresidual"],
                            post=c["post"], post_weight=s["post_weight"], dpost_weight=s["dpost_weight"],
                            gate=s["gate"], gate_kind=c["gate"], dgate=s["dgate"], residual_scale=c["scale"],
                            pre_weight=s["pre_weight"], dpre_weight=s["dpre_weight"], weight_dtype=c["weight"], eps=EPS,
                            workspace=s["workspace"], workspace_bytes=s["workspace"].numel())
        return {key: s[key] for key in ("dresidual", "dpre_weight", "dpost_weight", "du", "dgate") if s[key] is not None}
    dfm.balance_loss(s["logits"], c["dtype"], c["T"], c["E"], s["ids"], c["k"], s["loss"], s["counts"], s["tokens"],
                     s["workspace"], s["workspace"].numel(), probs=s["probs"], offs=s["offs"], S=c["S"], mask=s["mask"],
                     score=c["score"], coef=COEF, z_coef=Z_COEF)
    out = {key: s[key] for key in ("loss", "counts", "tokens", "probs")}
    if c["grad"]:
        dfm.balance_loss_grad(s["dloss"], s["logits"], c["dtype"], c["T"], c["E"], s["ids"], c["k"], s["counts"],
                              s["tokens"], s["dlogits"], offs=s["offs"], S=c["S"], mask=s["mask"], score=c["score"],
                              coef=COEF, z_coef=Z_COEF, weights=s["weights"], dweights=s["dweights"])
        out["dlogits"] = s["dlogits"]
    return out


def run(state):
    if own:
        return _run_own(state)
    return {"matmul": _matmul, "matmul_grad": _matmul_grad, "norm": _norm, "norm_grad": _norm_grad,
            "balance": _balance}[state["case"]["op"]](state)


def work(case):
    c, op, size = case, case["op"], BYTES[case["dtype"]]
    if op in ("matmul", "matmul_grad"):
        M, N, K = c["M"], c["N"], c["K"]
        wide = 2 * N if c["act"] == "swiglu" else N
        bias = wide if c["bias"] else 0
        if op == "matmul":
            out = M * N * BYTES[c["out"]] * (2 if c["residual"] else 1) + (M * wide * size if c["pre"] else 0)
            return {"bytes": size * (M * K + wide * K + bias) + out, "flops": 2 * M * wide * K}
        pre = M * wide * size if c["act"] != "none" else 0
        return {"bytes": size * (M * N + 2 * M * K + wide * K) + pre + BYTES[c["grad"]] * (wide * K + bias),
                "flops": 4 * M * wide * K}
    if op in ("norm", "norm_grad"):
        T, H, wb = c["T"], c["H"], BYTES[c["weight"]]
        gate = {"none": 0, "channel": H * wb, "token": 4 * T, "full": T * H * size}[c["gate"]]
        weights = H * wb * (2 if c["post"] else 1)
        if op == "norm":
            return {"bytes": 4 * T * H * size + gate + weights, "flops": T * H * (10 if c["post"] else 6)}
        dgate = {"none": 0, "channel": 4 * H, "token": 4 * T, "full": T * H * size}[c["gate"]]
        return {"bytes": 6 * T * H * size + gate + weights + dgate + 4 * H * (2 if c["post"] else 1),
                "flops": T * H * (28 if c["post"] else 16)}
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    once = T * E * size + 4 * T * k + (T if c["mask"] else 0)
    forward = once + 8 * S * E + 8 * S
    if not c["grad"]:
        return {"bytes": forward, "flops": 6 * T * E}
    return {"bytes": forward + T * E * size + 8 * T * k + 4 * S, "flops": 14 * T * E}


# ---- the definitions in 64 bits ---------------------------------------------
def _phi(z):
    """The normal distribution function."""
    return torch.special.ndtr(z)


def _exact_matmul(s, c):
    N, K = c["N"], c["K"]
    x, w = s["x"][:, :K].double(), s["w"][:, :K].double()
    b = s["bias"].double() if c["bias"] else torch.zeros(w.shape[0], dtype=torch.float64, device=x.device)
    z = torch.addmm(b, x, w.t())
    act = {"none": lambda: z, "relu": lambda: torch.maximum(z, torch.zeros_like(z)), "silu": lambda: z * torch.sigmoid(z),
           "gelu": lambda: z * _phi(z), "swiglu": lambda: z[:, :N] * torch.sigmoid(z[:, :N]) * z[:, N:]}[c["act"]]()
    out = {"y": act + s["residual"].double() if c["residual"] else act}
    if c["pre"]:
        out["pre"] = z
    return out


def _exact_matmul_grad(s, c):
    N, K = c["N"], c["K"]
    dy = s["dy"][:, :N].double()
    if c["act"] == "none":
        dz = dy
    else:
        z = s["pre"][:, :2 * N if c["act"] == "swiglu" else N].double()
        g = z[:, :N]
        sig = torch.sigmoid(g)
        slope = {"relu": lambda: (g > 0).double(), "gelu": lambda: _phi(g) + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi),
                 "silu": lambda: sig + g * sig * (1 - sig), "swiglu": lambda: sig + g * sig * (1 - sig)}[c["act"]]()
        if c["act"] == "swiglu":
            dz = torch.empty_like(z)
            dz[:, :N], dz[:, N:] = dy * z[:, N:] * slope, dy * g * sig
        else:
            dz = dy * slope
    out = {"dx": torch.mm(dz, s["w"][:, :K].double()), "dw": torch.mm(dz.t(), s["x"][:, :K].double())}
    if c["bias"]:
        out["dbias"] = torch.ones(1, c["M"], dtype=torch.float64, device=dz.device).mm(dz)[0]
    return out


def _exact_norm(s, c, grad):
    H = c["H"]
    one = torch.ones(H, dtype=torch.float64, device=s["u"].device)
    u, v = s["u"].double(), s["pre_weight"].double()
    q = s["post_weight"].double() if c["post"] else one
    gate = one if s["gate"] is None else s["gate"].double()
    if c["gate"] == "token":
        gate = gate.unsqueeze(1)
    ru = torch.rsqrt(torch.einsum("th,th->t", u, u) / H + EPS) if c["post"] else torch.ones_like(u[:, 0])
    a = u * q * ru[:, None]
    if not grad:
        h = torch.addcmul(c["scale"] * s["residual"].double(), gate.expand_as(a), a)
        rh = torch.rsqrt(torch.einsum("th,th->t", h, h) / H + EPS)
        return {"h": h, "n": h * v * rh[:, None]}
    h, dn = s["h"].double(), s["dn"].double()
    rh = torch.rsqrt(torch.einsum("th,th->t", h, h) / H + EPS)
    # d(h rh)/dh: rh (1 - h h' rh^2 / H)
    along = torch.einsum("th,th,h->t", h, dn, v) * rh ** 3 / H
    dh = s["dh"].double() + dn * v * rh[:, None] - h * along[:, None]
    out = {"dresidual": dh * c["scale"], "dpre_weight": torch.einsum("th,th,t->h", dn, h, rh)}
    da = dh * gate
    if c["post"]:
        along = torch.einsum("th,th,h->t", u, da, q) * ru ** 3 / H
        out["dpost_weight"] = torch.einsum("th,th,t->h", da, u, ru)
        out["du"] = da * q * ru[:, None] - u * along[:, None]
    else:
        out["du"] = da
    if c["gate"] == "channel":
        out["dgate"] = torch.einsum("th,th->h", dh, a)
    elif c["gate"] == "token":
        out["dgate"] = torch.einsum("th,th->t", dh, a)
    elif c["gate"] == "full":
        out["dgate"] = dh * a
    return out


def _exact_balance(s, c):
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    at = s["offs"].tolist() if s["offs"] is not None else [0, T]
    loss, probs = [], []
    dlogits = torch.zeros(T, E, dtype=torch.float64, device=s["logits"].device)
    for i in range(S):
        rows = torch.arange(at[i], at[i + 1], device=dlogits.device)
        if s["mask"] is not None:
            rows = rows[s["mask"][rows] != 0]
        n = rows.numel()
        if n == 0:
            loss.append(dlogits.new_zeros(()))
            probs.append(dlogits.new_zeros(E))
            continue
        z, ids = s["logits"][rows].double(), s["ids"][rows].long()
        score = torch.nn.functional.logsigmoid(z) if c["score"] == "sigmoid" else z
        p = torch.softmax(score, dim=1)
        lse = torch.logsumexp(z, dim=1)
        # how a score moves with its logit
        slope = torch.sigmoid(-z) if c["score"] == "sigmoid" else torch.ones_like(z)
        chosen = torch.zeros_like(z).scatter_add_(1, ids, torch.ones_like(ids, dtype=torch.float64))
        f = chosen.sum(0) * E / (k * n)
        probs.append(p.mean(0))
        loss.append(COEF * torch.dot(f, probs[-1]) + Z_COEF * lse.square().mean())
        if c["grad"]:
            d = COEF / n * slope * (p * f - p * (p @ f)[:, None]) + 2 * Z_COEF / n * lse[:, None] * torch.softmax(z, dim=1)
            w, dw = s["weights"][rows].double(), s["dweights"][rows].double()
            kept = w * dw - w * (w * dw).sum(1, keepdim=True)
            d = float(s["dloss"][i]) * d + slope * torch.zeros_like(z).scatter_add_(1, ids, kept)
            dlogits[rows] = d
    out = {"loss": torch.stack(loss), "counts": None, "tokens": None, "probs": torch.stack(probs)}
    if c["grad"]:
        out["dlogits"] = dlogits
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "matmul":
        return _exact_matmul(s, case)
    if op == "matmul_grad":
        return _exact_matmul_grad(s, case)
    if op == "balance":
        return _exact_balance(s, case)
    return _exact_norm(s, case, op == "norm_grad")
