"""The measured cases of the expert-path operators: tokens sorted by expert and
back (with their gradients), rows rounded to 8 bits with a scale per 128, and the
8-bit product of the sorted rows with the experts' weights.

`run` computes a case either in its plain form (elementary torch operations) or,
with `own` set, through the library's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
          "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
BLOCK = 128


def listed():
    return [
        # one token of a decode step on its way to its experts: latency
        dict(name="permute one token", op="permute", T=1, k=16, E=896, H=7168, dtype="bf16", drop=0.0),
        # a prefill of the layer's own width
        dict(name="permute prefill", op="permute", T=4096, k=16, E=896, H=7168, dtype="bf16", drop=0.0),
        # rows already in 8 bits, with their scales; some assignments dropped by a capacity limit
        dict(name="permute 8 bits", op="permute", T=777, k=8, E=61, H=7168, dtype="e4m3", drop=0.1),
        # backward of a training step
        dict(name="permute gradient", op="permute_grad", T=2048, k=8, E=128, H=7168, dtype="bf16", drop=0.02),
        # one token's expert outputs back
        dict(name="unpermute one token", op="unpermute", T=1, k=16, E=896, H=7168, dtype="bf16", drop=0.0),
        # a prefill's expert outputs back
        dict(name="unpermute prefill", op="unpermute", T=4096, k=16, E=896, H=7168, dtype="bf16", drop=0.0),
        # backward in 32 bits, a width that no vector load divides
        dict(name="unpermute gradient odd", op="unpermute_grad", T=1023, k=6, E=64, H=2049, dtype="f32", drop=0.05),
        # a decode step's hidden state
        dict(name="quantize one token", op="quantize", M=1, K=7168, dtype="bf16"),
        # a prefill's sorted intermediate rows
        dict(name="quantize prefill", op="quantize", M=65536, K=1536, dtype="bf16"),
        # one token through the gate weights of its 16 experts: a weight stream
        dict(name="product one token", op="product", T=1, k=16, G=128, N=1536, K=7168, out="bf16", trans=False),
        # a prefill through the gate weights
        dict(name="product prefill", op="product", T=2048, k=16, G=32, N=1536, K=7168, out="bf16", trans=False),
        # backward: the gradient of the rows, ragged sizes
        dict(name="product gradient odd", op="product", T=501, k=6, G=21, N=2050, K=1111, out="f32", trans=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["permute", "permute_grad", "unpermute", "unpermute_grad", "quantize", "product", "product"])
    if op == "quantize":
        K = _log(rng, 100, 8192)
        M = min(_log(rng, 1, 65536), 100_000_000 // K)
        return dict(op=op, M=M, K=K, dtype=rng.choice(["bf16", "f16", "f32"]))
    if op == "product":
        k = rng.randint(1, 16)
        G = rng.randint(k, 64)
        N, K = _log(rng, 64, 7168), _log(rng, 64, 7168)
        if rng.random() < 0.5:
            N, K = max(128, N // 128 * 128), max(128, K // 128 * 128)
        G = max(k, min(G, 700_000_000 // (N * K)))
        T = min(_log(rng, 1, 2048), max(1, 360_000_000_000 // (k * N * K)))
        return dict(op=op, T=T, k=k, G=G, N=N, K=K, out=rng.choice(["bf16", "f16", "f32"]), trans=rng.random() < 0.4)
    E = _log(rng, 8, 1024)
    k = rng.randint(1, min(E, 16))
    H = _log(rng, 64, 8192)
    if rng.random() < 0.6:
        H = max(64, H // 64 * 64)
    T = max(1, min(_log(rng, 1, 8192), 200_000_000 // (k * H)))
    kinds = ["bf16", "f16", "f32"] + (["e4m3"] if op == "permute" else [])
    return dict(op=op, T=T, k=k, E=E, H=H, dtype=rng.choice(kinds), drop=rng.choice([0.0, 0.0, 0.1, 0.5]))


# ---- inputs -----------------------------------------------------------------
def _route(T, k, E, drop, g):
    """Distinct experts a token, some more popular than others; dropped ones -1."""
    dev = "cuda"
    logits = torch.randn(T, E, generator=g, device=dev) + 0.5 * torch.randn(E, generator=g, device=dev)
    top = logits.topk(k, dim=1)
    ids = top.indices.to(torch.int32)
    weights = torch.softmax(top.values, dim=1)
    if drop:
        gone = torch.rand(T, k, generator=g, device=dev) < drop
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    return ids.contiguous(), weights.contiguous()


def _sorted(ids, E):
    """offs [E+1], pos [T*k] and src [T*k] of the stable sort by expert."""
    a = ids.reshape(-1).long()
    key = torch.where((a >= 0) & (a < E), a, torch.full_like(a, E))
    order = torch.argsort(key, stable=True)
    skey = key[order]
    offs = torch.searchsorted(skey, torch.arange(E + 1, device=a.device)).to(torch.int32)
    index = torch.arange(a.numel(), device=a.device)
    pos = torch.empty_like(a)
    pos[order] = torch.where(skey < E, index, torch.full_like(index, -1))
    src = torch.where(skey < E, order, torch.full_like(order, -1))
    return offs, pos.to(torch.int32), src.to(torch.int32)


def _codes(shape, sigma, g):
    """e4m3 codes of normal values whose blocks have been scaled to the format's range."""
    v = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    return v.mul_(sigma).clamp_(-448, 448).to(torch.float8_e4m3fn)


def _up(n, m):
    return -(-n // m) * m


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, dev, op = dict(case), "cuda", case["op"]
    s = {"case": c}
    if op == "quantize":
        dt = DTYPES[c["dtype"]]
        M, K = c["M"], c["K"]
        spread = torch.exp(torch.randn(M, 1, generator=g, device=dev))
        s["x"] = (torch.randn(M, K, generator=g, device=dev) * spread).to(dt)
        s["codes"] = torch.zeros(M, K, dtype=torch.float8_e4m3fn, device=dev)
        s["scales"] = torch.zeros(M, -(-K // BLOCK), device=dev)
        return s
    if op == "product":
        T, k, G, N, K = c["T"], c["k"], c["G"], c["N"], c["K"]
        ids, _ = _route(T, k, G, 0.0, g)
        offs, _, _ = _sorted(ids, G)
        M, nb, kb = T * k, -(-N // BLOCK), -(-K // BLOCK)
        # rows of a multiple of 16 bytes, as the product takes its 8-bit operands
        s["x"] = _codes((M, _up(K, 16)), 150.0, g)
        s["xs"] = torch.exp(0.3 * torch.randn(M, kb, generator=g, device=dev)) / 150.0
        shape, blocks = ((G, K, _up(N, 16)), (G, kb, nb)) if c["trans"] else ((G, N, _up(K, 16)), (G, nb, kb))
        s["w"] = _codes(shape, 110.0, g)
        s["ws"] = torch.exp(0.1 * torch.randn(blocks, generator=g, device=dev)) * (0.02 / 110.0)
        s["offs"] = offs
        # the plan that the plain form pads its groups by
        count = (offs[1:] - offs[:-1]).long()
        active = torch.nonzero(count).reshape(-1)
        s["active"] = active
        s["cap"] = int(count.max())
        s["group"] = torch.repeat_interleave(torch.arange(active.numel(), device=dev), count[active])
        s["within"] = torch.arange(M, device=dev) - offs[active].long()[s["group"]]
        s["y"] = torch.zeros(M, N, dtype=DTYPES[c["out"]], device=dev)
        return s
    T, k, E, H, dt = c["T"], c["k"], c["E"], c["H"], DTYPES[c["dtype"]]
    A = T * k
    s["ids"], s["weights"] = _route(T, k, E, c["drop"], g)
    if op == "permute":
        if c["dtype"] == "e4m3":
            s["x"] = _codes((T, H), 150.0, g)
            s["xs"] = torch.exp(0.3 * torch.randn(T, -(-H // BLOCK), generator=g, device=dev)) / 150.0
            s["rows_scales"] = torch.zeros(A, s["xs"].shape[1], device=dev)
        else:
            s["x"] = torch.randn(T, H, generator=g, device=dev).to(dt)
        s["rows"] = torch.zeros(A, H, dtype=dt, device=dev)
        s["offs"] = torch.zeros(E + 1, dtype=torch.int32, device=dev)
        s["pos"] = torch.zeros(A, dtype=torch.int32, device=dev)
        s["src"] = torch.full((A,), -1, dtype=torch.int32, device=dev)
        # the library's scratch, of the size that serves any call
        s["workspace"] = torch.empty(4 << 20, dtype=torch.uint8, device=dev)
        return s
    _, s["pos"], _ = _sorted(s["ids"], E)
    if op in ("permute_grad", "unpermute"):
        s["rows"] = torch.randn(A, H, generator=g, device=dev).to(dt)
        s["y"] = torch.zeros(T, H, dtype=dt, device=dev)
    else:
        s["rows"] = torch.randn(A, H, generator=g, device=dev).to(dt)
        s["dy"] = torch.randn(T, H, generator=g, device=dev).to(dt)
        s["drows"] = torch.zeros(A, H, dtype=dt, device=dev)
        s["dweights"] = torch.zeros(T, k, device=dev)
    return s


# ---- the plain forms --------------------------------------------------------
def _permute(s):
    c = s["case"]
    offs, pos, src = _sorted(s["ids"], c["E"])
    token = torch.div(src.clamp(min=0), c["k"], rounding_mode="floor").long()
    gone = (src < 0)[:, None]
    if c["dtype"] == "e4m3":
        rows = s["x"].view(torch.uint8)[token].masked_fill_(gone, 0).view(torch.float8_e4m3fn)
        return {"rows": rows, "rows_scales": s["xs"][token].masked_fill_(gone, 0), "offs": offs, "pos": pos, "src": src}
    return {"rows": s["x"][token].masked_fill_(gone, 0), "offs": offs, "pos": pos, "src": src}


def _gathered(s):
    """The rows of every assignment in 32 bits [T, k, H], zeros where dropped."""
    c = s["case"]
    pos = s["pos"].long()
    rows = s["rows"][pos.clamp(min=0)].float().masked_fill_((pos < 0)[:, None], 0)
    return rows.view(c["T"], c["k"], c["H"])


def _unpermute_grad(s):
    c = s["case"]
    rows, dy, pos = _gathered(s), s["dy"].float(), s["pos"].long()
    dweights = (rows.double() * dy.double()[:, None, :]).sum(-1).float()
    each = (s["weights"][:, :, None] * dy[:, None, :]).to(s["dy"].dtype).view(-1, c["H"])
    drows = torch.zeros(pos.numel() + 1, c["H"], dtype=each.dtype, device=each.device)
    drows[torch.where(pos < 0, torch.full_like(pos, pos.numel()), pos)] = each
    return {"drows": drows[:-1], "dweights": dweights}


def _quantize(s):
    x = s["x"].float()
    M, K = x.shape
    nb = -(-K // BLOCK)
    x = torch.nn.functional.pad(x, (0, nb * BLOCK - K)).view(M, nb, BLOCK)
    most = x.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -100)
    # 448 x / most: 448 = 0.875 * 512, so that neither factor overflows
    codes = (x * 0.875 / (most * 2.0 ** -9)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return {"codes": codes.view(M, nb * BLOCK)[:, :K].contiguous(), "scales": (most / 448.0).view(M, nb)}


def _product(s):
    c = s["case"]
    N, K = c["N"], c["K"]
    x = s["x"][:, :K].float() * s["xs"].repeat_interleave(BLOCK, 1)[:, :K]
    w = s["w"].view(torch.uint8)[s["active"]].view(torch.float8_e4m3fn).float()
    ws = s["ws"][s["active"]].repeat_interleave(BLOCK, 1).repeat_interleave(BLOCK, 2)
    w = w[:, :K, :N] * ws[:, :K, :N] if c["trans"] else (w[:, :N, :K] * ws[:, :N, :K]).transpose(1, 2)
    padded = torch.zeros(w.shape[0], s["cap"], K, device=x.device)
    padded[s["group"], s["within"]] = x
    return {"y": torch.bmm(padded, w)[s["group"], s["within"]].to(DTYPES[c["out"]])}


# ---- one pass ---------------------------------------------------------------
def _run_own(s):
    import mxfp4_routed_expert_top_gb300 as dfm
    c = s["case"]
    op = c["op"]
    if op == "permute":
        if c["dtype"] == "e4m3":
            dfm.permute(s["ids"], c["T"], c["k"], c["E"], s["x"], "e4m3", c["H"], s["rows"], s["offs"], s["pos"],
                        s["src"], s["workspace"], 4 << 20, scales=s["xs"], n_scales=s["xs"].shape[1],
                        rows_scales=s["rows_scales"])
            return {key: s[key] for key in ("rows", "rows_scales", "offs", "pos", "src")}
        dfm.permute(s["ids"], c["T"], c["k"], c["E"], s["x"], c["dtype"], c["H"], s["rows"], s["offs"], s["pos"],
                    s["src"], s["workspace"], 4 << 20)
        return {key: s[key] for key in ("rows", "offs", "pos", "src")}
    if op == "permute_grad":
        dfm.permute_grad(s["rows"], c["dtype"], c["T"] * c["k"], s["pos"], c["T"], c["k"], c["H"], s["y"])
        return {"dx": s["y"]}
    if op == "unpermute":
        dfm.unpermute(s["rows"], c["dtype"], c["T"] * c["k"], s["pos"], s["weights"], c["T"], c["k"], c["H"], s["y"])
        return {"y": s["y"]}
    if op == "unpermute_grad":
        dfm.unpermute_grad(s["dy"], s["rows"], c["dtype"], c["T"] * c["k"], s["pos"], s["weights"], c["T"], c["k"],
                           c["H"], s["drows"], s["dweights"])
        return {"drows": s["drows"], "dweights": s["dweights"]}
    if op == "quantize":
        dfm.fp8_quantize(s["x"], c["dtype"], c["M"], c["K"], s["codes"], s["scales"])
        return {"codes": s["codes"], "scales": s["scales"]}
    dfm.fp8_matmul(s["x"], s["xs"], s["w"], s["ws"], s["offs"], c["G"], c["T"] * c["k"], c["N"], c["K"], s["y"],
                   c["out"], transposed=c["trans"], ldx=s["x"].shape[1], ldw=s["w"].shape[2])
    return {"y": s["y"]}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "permute":
        return _permute(state)
    if op == "permute_grad":
        return {"dx": _gathered(state).sum(1).to(state["y"].dtype)}
    if op == "unpermute":
        return {"y": (_gathered(state) * state["weights"][:, :, None]).sum(1).to(state["y"].dtype)}
    if op == "unpermute_grad":
        return _unpermute_grad(state)
    return _quantize(state) if op == "quantize" else _product(state)


def work(case):
    c, op = case, case["op"]
    if op == "quantize":
        return {"bytes": c["M"] * c["K"] * (BYTES[c["dtype"]] + 1) + 4 * c["M"] * -(-c["K"] // BLOCK),
                "flops": 2 * c["M"] * c["K"]}
    if op == "product":
        M, N, K, G = c["T"] * c["k"], c["N"], c["K"], c["G"]
        active = G * (1 - (1 - c["k"] / G) ** c["T"])  # groups that have a row, about
        kb, nb = -(-K // BLOCK), -(-N // BLOCK)
        return {"bytes": M * (K + 4 * kb) + active * (N * K + 4 * nb * kb) + M * N * BYTES[c["out"]],
                "flops": 2 * M * N * K}
    T, k, H, A, size = c["T"], c["k"], c["H"], c["T"] * c["k"], BYTES[c["dtype"]]
    n = A * (1 - c["drop"])  # rows that are there, about
    if op == "permute":
        row = H * size + (4 * -(-H // BLOCK) if c["dtype"] == "e4m3" else 0)
        return {"bytes": (T + n) * row + 12 * A + 4 * (c["E"] + 1), "flops": 0}
    if op == "permute_grad":
        return {"bytes": (T + n) * H * size + 4 * A, "flops": n * H}
    if op == "unpermute":
        return {"bytes": (T + n) * H * size + 8 * A, "flops": 2 * n * H}
    return {"bytes": (T + 2 * n) * H * size + 12 * A, "flops": 3 * n * H}


# ---- the definitions in 64 bits ---------------------------------------------
def _e4m3(v):
    """Nearest e4m3 value, ties to even, saturating at 448."""
    mag = v.abs()
    e = torch.floor(torch.log2(mag.clamp(min=2.0 ** -20))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return torch.sign(v) * (torch.round(mag / step) * step).clamp(max=448.0)


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "quantize":
        x = s["x"].double()
        codes, scales = torch.empty_like(x), torch.empty(x.shape[0], -(-c["K"] // BLOCK), dtype=x.dtype, device=x.device)
        for b in range(scales.shape[1]):
            part = x[:, b * BLOCK:(b + 1) * BLOCK]
            most = part.abs().max(1).values.clamp(min=2.0 ** -100)
            scales[:, b] = most / 448
            codes[:, b * BLOCK:(b + 1) * BLOCK] = _e4m3(part * 448 / most[:, None])
        return {"codes": codes, "scales": scales}
    if op == "product":
        y = torch.zeros(c["T"] * c["k"], c["N"], dtype=torch.float64, device="cuda")
        at = s["offs"].tolist()
        k_of = torch.arange(c["K"], device="cuda") // BLOCK
        n_of = torch.arange(c["N"], device="cuda") // BLOCK
        for e in range(c["G"]):
            if at[e] < at[e + 1]:
                r = slice(at[e], at[e + 1])
                w = s["w"][e].double().t() if c["trans"] else s["w"][e].double()
                ws = s["ws"][e].double().t() if c["trans"] else s["ws"][e].double()
                w = w[:c["N"], :c["K"]] * ws[n_of][:, k_of]
                y[r] = (s["x"][r, :c["K"]].double() * s["xs"][r].double()[:, k_of]) @ w.t()
        return {"y": y}
    T, k, H = c["T"], c["k"], c["H"]
    A = T * k
    if op == "permute":
        rows = torch.zeros(A, H, dtype=torch.float64, device="cuda")
        a = s["ids"].reshape(-1).tolist()
        order = sorted((i for i in range(A) if 0 <= a[i] < c["E"]), key=lambda i: (a[i], i))
        token = torch.tensor([i // k for i in order], dtype=torch.long, device="cuda")
        rows[:len(order)] = s["x"].double()[token]
        if c["dtype"] == "e4m3":
            scales = torch.zeros(A, s["xs"].shape[1], dtype=torch.float64, device="cuda")
            scales[:len(order)] = s["xs"].double()[token]
            return {"rows": rows, "rows_scales": scales, "offs": None, "pos": None, "src": None}
        return {"rows": rows, "offs": None, "pos": None, "src": None}
    pos = s["pos"].view(T, k).long()
    there = (pos >= 0).double()
    if op == "unpermute_grad":
        drows = torch.zeros(A, H, dtype=torch.float64, device="cuda")
        dweights = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        dy = s["dy"].double()
        for j in range(k):
            p = pos[:, j]
            dweights[:, j] = there[:, j] * (s["rows"][p.clamp(min=0)].double() * dy).sum(1)
            drows[p[p >= 0]] = (s["weights"][:, j, None].double() * dy)[p >= 0]
        return {"drows": drows, "dweights": dweights}
    y = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for j in range(k):
        scale = there[:, j] * (s["weights"][:, j].double() if op == "unpermute" else 1.0)
        y += scale[:, None] * s["rows"][pos[:, j].clamp(min=0)].double()
    return {"dx" if op == "permute_grad" else "y": y}
