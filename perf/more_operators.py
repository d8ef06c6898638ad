"""Cases of the operators of a training step around the projections, and how each is computed.

Three operators of the package, each in a plain form (elementary torch
operations in 32 bits) and as a user's program calls the package:

- ``grouped_linear``: rows sorted by expert times their expert's weight,
  Y[i] = X[i]·W[e]ᵀ for the rows ends[e-1] <= i < ends[e], alone ("infer") or
  with the gradients of X and W ("train"); rows behind the last expert's are zero;
- ``embedding``: Y[i] = scale·W[tokens[i]], alone ("lookup") or with the gradient
  of W, dW[v] = scale·Σ dY[i] over the i with tokens[i] = v ("train");
- ``adamw`` / ``adamw_8bit``: a decoupled-weight-decay Adam step over a list of
  tensors, with moments in 32 bits, or in 8 (E4M3 values of the first moment and
  of the second moment's root, in units of one scale for each 256 elements).

``listed`` holds the fixed cases, ``draw`` makes more of the same ranges,
``prepare`` makes a case's inputs from a seed, ``run`` is one pass, ``exact``
the same outputs from the definitions in 64 bits, ``work`` what a pass cannot
do without.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = 256          # elements of a tensor that share one scale
E4M3 = torch.float8_e4m3fn
TOP = 448.0          # E4M3's largest value
LEAST = 2.0 ** -9    # and its smallest above zero
FLUSH = 2.0 ** -110  # a block whose largest magnitude is below is held as zeros
LR, BETAS, EPS, DECAY = 1e-3, (0.9, 0.95), 1e-8, 0.1


def _grouped(name, rows, experts, n, k, dtype, mode, skew=0.5, behind=0):
    return {"name": name, "op": "grouped", "rows": rows, "experts": experts, "n": n, "k": k, "dtype": dtype,
            "mode": mode, "skew": skew, "behind": behind}


def _embedding(name, tokens, vocab, hidden, dtype, mode, scale=1.0, pad=False):
    return {"name": name, "op": "embedding", "tokens": tokens, "vocab": vocab, "hidden": hidden, "dtype": dtype,
            "mode": mode, "scale": scale, "pad": pad}


def _adamw(name, shapes, dtype, grad, bits, copies=False):
    return {"name": name, "op": "adamw", "shapes": shapes, "dtype": dtype, "grad": grad, "bits": bits,
            "copies": copies}


def listed():
    layer = "4096x1024,1024x1024,1024x1024,1024x1024,1024x4096,4096x1024,1024,1024,64"
    return [
        # one token after a decode step, sent to 8 of 64 experts: latency, a few weights stream once
        _grouped("infer_8x64e_1024x2048_bf16", 8, 64, 1024, 2048, "bf16", "infer", skew=0.0),
        # 64 requests decoding, two of 8 experts each: every weight streams once
        _grouped("infer_128x8e_14336x4096_f16", 128, 8, 14336, 4096, "f16", "infer"),
        # a prompt over many small experts, in a buffer with room behind the rows
        _grouped("infer_4096x64e_1024x2048_bf16", 4096, 64, 1024, 2048, "bf16", "infer", behind=100),
        # fine-tuning on the benchmark's ragged sizes
        _grouped("train_1000x7e_1000x1000_f16", 1000, 7, 1000, 1000, "f16", "train", behind=13),
        # the largest: a long batch through experts of the benchmark's linear layer
        _grouped("train_16384x8e_14336x4096_bf16", 16384, 8, 14336, 4096, "bf16", "train"),
        # one decode step of 64 requests: latency
        _embedding("lookup_64x32000x4096_bf16", 64, 32000, 4096, "bf16", "lookup"),
        # an odd vocabulary and an odd number of tokens, scaled by the root of the width
        _embedding("train_333x50001x1000_f32", 333, 50001, 1000, "f32", "train", scale=31.625, pad=True),
        # an ordinary pre-training micro-batch on a large vocabulary: most rows get no token
        _embedding("train_8192x131072x4096_bf16", 8192, 131072, 4096, "bf16", "train"),
        # a long batch on a smaller vocabulary: tokens that come up thousands of times, and padding
        _embedding("train_65536x32000x2048_f16", 65536, 32000, 2048, "f16", "train", scale=45.25, pad=True),
        # a bias, a norm and one small weight: latency
        _adamw("adamw_3_small_f32", "128x128,128,1000", "f32", "f32", 32),
        # a small model: many tensors, 32-bit weights with gradients and copies of 16 bits
        _adamw("adamw_109_tensors_f32_bf16", ",".join([layer] * 12 + ["50001x1000"]), "f32", "bf16", 32, copies=True),
        # the largest: projections of the benchmark's linear layer, moments in 8 bits
        _adamw("adamw8_4x14336x4096_bf16", "14336x4096,14336x4096,4096x14336,32000x4096,4096", "bf16", "bf16", 8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("grouped", "grouped", "embedding", "adamw"))
    if op == "grouped":
        while True:
            rows, experts, n, k = _log(rng, 1, 16384), _log(rng, 1, 128), _log(rng, 64, 14336), _log(rng, 64, 14336)
            if 2 ** 20 <= rows * n * k <= 2 ** 39 and experts * n * k <= 2 ** 28:
                break
        if rng.random() < 0.8:
            n, k = (n + 7) // 8 * 8, (k + 7) // 8 * 8
        return {"op": op, "rows": rows, "experts": experts, "n": n, "k": k, "dtype": rng.choice(("bf16", "f16")),
                "mode": rng.choice(("infer", "train")), "skew": rng.choice((0.0, 0.5, 1.0)),
                "behind": rng.choice((0, 0, rng.randrange(1, 300)))}
    if op == "embedding":
        while True:
            tokens, vocab, hidden = _log(rng, 1, 65536), _log(rng, 64, 131072), _log(rng, 64, 8192)
            if tokens * hidden <= 2 ** 27 and vocab * hidden <= 2 ** 29:
                break
        return {"op": op, "tokens": tokens, "vocab": vocab, "hidden": hidden,
                "dtype": rng.choice(("bf16", "f16", "f32")), "mode": rng.choice(("lookup", "train", "train")),
                "scale": rng.choice((1.0, 1.0, round(math.sqrt(hidden), 3))), "pad": rng.random() < 0.4}
    shapes, left = [], _log(rng, 2 ** 14, 2 ** 28)
    for _ in range(_log(rng, 1, 100)):
        n = _log(rng, 1, max(2, left))
        cols = min(n, _log(rng, 1, 8192))
        shapes.append(f"{n // cols}x{cols}")
        left -= n // cols * cols
        if left < 2:
            break
    dtype = rng.choice(("f32", "f32", "bf16", "f16"))
    grad = rng.choice(("f32", "bf16", "f16")) if dtype == "f32" else dtype
    return {"op": op, "shapes": ",".join(shapes), "dtype": dtype, "grad": grad, "bits": rng.choice((8, 32)),
            "copies": dtype == "f32" and rng.random() < 0.5}


def _shapes(case):
    return [tuple(int(x) for x in s.split("x")) for s in case["shapes"].split(",")]


def _popularity(case):
    return [(e + 1.0) ** -case["skew"] for e in range(case["experts"])]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    dt = DTYPES[case["dtype"]]
    if case["op"] == "grouped":
        M, E, N, K = case["rows"], case["experts"], case["n"], case["k"]
        host = torch.Generator().manual_seed(seed)
        p = torch.tensor(_popularity(case), dtype=torch.float64)[torch.randperm(E, generator=host)]
        expert = torch.multinomial(p, M, replacement=True, generator=host)
        ends = torch.bincount(expert, minlength=E).cumsum(0)
        total = M + case["behind"]
        state = {"case": case, "ends": ends.cuda(), "X": normal(total, K).to(dt),
                 "W": torch.stack([(normal(N, K) / math.sqrt(K)).to(dt) for _ in range(E)]),
                 "spans": list(zip([0] + ends.tolist()[:-1], ends.tolist()))}  # a loop over experts needs them on the host
        if case["mode"] == "train":
            state["dY"] = normal(total, N).to(dt)
        return state
    if case["op"] == "embedding":
        M, V, K = case["tokens"], case["vocab"], case["hidden"]
        # token frequencies fall off like 1/rank; with padding, of every sequence's last tenth
        u = torch.rand(M, generator=gen, device="cuda", dtype=torch.float64)
        tokens = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1)
        if case["pad"]:
            tokens = torch.where(torch.rand(M, generator=gen, device="cuda") < 0.1, torch.full_like(tokens, V - 1),
                                 tokens)
        state = {"case": case, "tokens": tokens, "W": (0.02 * normal(V, K)).to(dt),
                 "pad": V - 1 if case["pad"] else None}
        if case["mode"] == "train":
            state["dY"] = normal(M, K).to(dt)
        return state
    # the tensors lie one after another in one buffer for each role, from multiples of BLOCK on
    shapes = _shapes(case)
    starts, at = [], 0
    for s in shapes:
        starts.append(at)
        at += (math.prod(s) + BLOCK - 1) // BLOCK * BLOCK
    live = torch.zeros(at, dtype=torch.bool, device="cuda")
    for s, a in zip(shapes, starts):
        live[a:a + math.prod(s)] = True
    size = 1e-3 * torch.exp(2.0 * normal(at // BLOCK)).repeat_interleave(BLOCK)  # gradients' magnitudes differ
    # moments after some steps: the second one larger than the square of the first
    flat = {"p": torch.where(live, 0.02 * normal(at), 0.0).to(dt),
            "g": torch.where(live, size * normal(at), 0.0).to(DTYPES[case["grad"]]),
            "m": torch.where(live, 0.3 * size * normal(at), 0.0),
            "v": torch.where(live, (size * (0.5 + torch.rand(at, generator=gen, device="cuda"))) ** 2, 0.0)}
    if case["bits"] == 8:
        flat["m"], flat["ms"] = _encode(flat["m"], False)
        flat["v"], flat["vs"] = _encode(torch.sqrt(flat["v"]), True)
    if case["copies"]:
        flat["copy"] = flat["p"].to(DTYPES[case["grad"]] if case["grad"] != "f32" else torch.bfloat16)
    views = {}
    for role, t in flat.items():
        if role in ("ms", "vs"):
            views[role] = [t[a // BLOCK:(a + math.prod(s) + BLOCK - 1) // BLOCK] for s, a in zip(shapes, starts)]
        else:
            views[role] = [t[a:a + math.prod(s)].view(s) for s, a in zip(shapes, starts)]
    return {"case": case, "flat": flat, "views": views, "step": 10}


def _encode(x, root):
    """E4M3 values in units of a scale for each block, and the scales; a root
    above zero is held above zero."""
    b = x.view(-1, BLOCK)
    top = b.abs().amax(dim=1, keepdim=True)
    held = top >= FLUSH
    q = b * torch.where(held, TOP / top, torch.zeros_like(top))
    if root:
        q = torch.where((q > 0.0) & (q < LEAST), torch.full_like(q, LEAST), q)
    q = torch.clamp(q, -TOP, TOP).to(E4M3)
    return q.view(-1), torch.where(held, top / TOP, torch.zeros_like(top)).view(-1)


def _decode(codes, scales):
    return (codes.float().view(-1, BLOCK) * scales[:, None]).view(-1)


def _run_own(state):
    import dense_fp16_gemm_02_amd as tg

    case = state["case"]
    if case["op"] == "grouped":
        if case["mode"] == "infer":
            return tg.grouped_linear(state["X"], state["W"], state["ends"])
        X = state["X"].detach().requires_grad_()
        W = state["W"].detach().requires_grad_()
        Y = tg.grouped_linear(X, W, state["ends"])
        dX, dW = torch.autograd.grad(Y, (X, W), state["dY"])
        return {"Y": Y.detach(), "dX": dX, "dW": dW}
    if case["op"] == "embedding":
        if case["mode"] == "lookup":
            return tg.embedding(state["tokens"], state["W"], scale=case["scale"], padding_idx=state["pad"])
        W = state["W"].detach().requires_grad_()
        Y = tg.embedding(state["tokens"], W, scale=case["scale"], padding_idx=state["pad"])
        return {"Y": Y.detach(), "dW": torch.autograd.grad(Y, W, state["dY"])[0]}
    v = state["views"]
    how = dict(lr=LR, betas=BETAS, eps=EPS, weight_decay=DECAY, copies=v.get("copy"))
    if case["bits"] == 8:
        tg.adamw_8bit(v["p"], v["g"], v["m"], v["ms"], v["v"], v["vs"], state["step"], **how)
    else:
        tg.adamw(v["p"], v["g"], v["m"], v["v"], state["step"], **how)
    return {k: t for k, t in state["flat"].items() if k != "g"}


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    if case["op"] == "grouped":
        X, W, dt = state["X"].float(), state["W"].float(), state["X"].dtype
        Y = torch.zeros(X.shape[0], W.shape[1], device=X.device)
        train = case["mode"] == "train"
        if train:
            dY, dX, dW = state["dY"].float(), torch.zeros_like(X), torch.zeros_like(W)
        for e, (a, b) in enumerate(state["spans"]):
            if a == b:
                continue
            Y[a:b] = torch.matmul(X[a:b], W[e].t())
            if train:
                dX[a:b] = torch.matmul(dY[a:b], W[e])
                dW[e] = torch.matmul(dY[a:b].t(), X[a:b])
        if train:
            return {"Y": Y.to(dt), "dX": dX.to(dt), "dW": dW.to(dt)}
        return Y.to(dt)
    if case["op"] == "embedding":
        tokens, W = state["tokens"], state["W"]
        Y = (W[tokens].float() * case["scale"]).to(W.dtype)
        if case["mode"] == "lookup":
            return Y
        dW = torch.zeros(W.shape, device=W.device).index_add(0, tokens, state["dY"].float())
        if state["pad"] is not None:
            dW[state["pad"]] = 0.0
        return {"Y": Y, "dW": (dW * case["scale"]).to(W.dtype)}
    f, step, (b1, b2) = state["flat"], state["step"], BETAS
    p, g = f["p"].float(), f["g"].float()
    if case["bits"] == 8:
        m, r = _decode(f["m"], f["ms"]), _decode(f["v"], f["vs"])
        v = r * r
    else:
        m, v = f["m"], f["v"]
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + (g * g) * (1.0 - b2)
    root = torch.sqrt(v)
    p = p * (1.0 - LR * DECAY) - (m / (root * (1.0 / math.sqrt(1.0 - b2 ** step)) + EPS)) * (LR / (1.0 - b1 ** step))
    f["p"].copy_(p)
    if case["bits"] == 8:
        for role, scale, t in (("m", "ms", m), ("v", "vs", root)):
            codes, scales = _encode(t, role == "v")
            f[role].copy_(codes)
            f[scale].copy_(scales)
    else:
        f["m"].copy_(m)
        f["v"].copy_(v)
    if case["copies"]:
        f["copy"].copy_(p)
    return {k: t for k, t in f.items() if k != "g"}


def work(case):
    size = SIZES[case["dtype"]]
    if case["op"] == "grouped":
        M, E, N, K = case["rows"], case["experts"], case["n"], case["k"]
        weight = _popularity(case)
        hit = sum(1.0 - (1.0 - w / sum(weight)) ** M for w in weight)  # experts that get a row
        total = M + case["behind"]
        if case["mode"] == "infer":
            return {"bytes": size * (M * K + hit * N * K + total * N) + 8.0 * E, "flops": 2.0 * M * N * K}
        return {"bytes": size * (M * K + M * N + hit * N * K + total * (N + K) + E * N * K) + 8.0 * E,
                "flops": 6.0 * M * N * K}
    if case["op"] == "embedding":
        M, V, K = case["tokens"], case["vocab"], case["hidden"]
        # different tokens among M whose rank is log-uniform
        hit = sum(1.0 - (1.0 - math.log1p(1.0 / (i + 1.0)) / math.log(V + 1.0)) ** M for i in range(V))
        nbytes = 8.0 * M + size * (hit * K + M * K)
        if case["mode"] == "lookup":
            return {"bytes": nbytes, "flops": 1.0 * M * K}
        return {"bytes": nbytes + size * (M * K + V * K), "flops": 2.0 * M * K + V * K}
    n = sum(math.prod(s) for s in _shapes(case))
    state = 16.0 if case["bits"] == 32 else 4.0 + 16.0 / BLOCK
    return {"bytes": n * (2.0 * size + SIZES[case["grad"]] + state + (2.0 if case["copies"] else 0.0)), "flops": 16.0 * n}


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "grouped":
        X, W = state["X"].double(), state["W"]
        train = case["mode"] == "train"
        dY = state["dY"].double() if train else None
        Y, dX, dW = [], [], []
        for e, (a, b) in enumerate(state["spans"]):
            We = W[e].double()
            Y.append(X[a:b] @ We.t())
            if train:
                dX.append(dY[a:b] @ We)
                dW.append(dY[a:b].t() @ X[a:b])
        behind = X.shape[0] - state["spans"][-1][1]
        Y = torch.cat(Y + [X.new_zeros(behind, W.shape[1])])
        if not train:
            return Y
        return {"Y": Y, "dX": torch.cat(dX + [X.new_zeros(behind, W.shape[2])]), "dW": torch.stack(dW)}
    if case["op"] == "embedding":
        tokens, W = state["tokens"], state["W"]
        Y = case["scale"] * torch.index_select(W, 0, tokens).double()
        if case["mode"] == "lookup":
            return Y
        # by sorted tokens: runs of the same token are differences of a running sum
        order = torch.argsort(tokens, stable=True)
        ids, counts = torch.unique_consecutive(tokens[order], return_counts=True)
        dW = torch.zeros(W.shape, dtype=torch.float64, device=W.device)
        for lo in range(0, W.shape[1], 256):
            sums = torch.cumsum(state["dY"][order, lo:lo + 256].double(), 0)[counts.cumsum(0) - 1]
            dW[ids, lo:lo + 256] = case["scale"] * torch.diff(sums, dim=0, prepend=torch.zeros_like(sums[:1]))
        if state["pad"] is not None:
            dW[state["pad"]] = 0.0
        return {"Y": Y, "dW": dW}
    f, step, (b1, b2) = state["flat"], state["step"], BETAS
    g, m, v = f["g"].double(), f["m"].double(), f["v"].double()
    if case["bits"] == 8:
        m, v = m.view(-1, BLOCK) * f["ms"].double()[:, None], (v.view(-1, BLOCK) * f["vs"].double()[:, None]) ** 2
        m, v = m.flatten(), v.flatten()
    m.mul_(b1).add_(g, alpha=1.0 - b1)
    v.mul_(b2).addcmul_(g, g, value=1.0 - b2)
    mean, var = m / (1.0 - b1 ** step), v / (1.0 - b2 ** step)
    p = f["p"].double()
    out = {"p": p - LR * (DECAY * p + mean / (var.sqrt() + EPS))}
    if case["copies"]:
        out["copy"] = out["p"]
    if case["bits"] == 32:
        return {**out, "m": m, "v": v}
    for role, t in (("m", m), ("v", v.sqrt())):  # in units of the block's scale, unrounded
        t = t.view(-1, BLOCK)
        scale = t.abs().amax(1) / TOP
        out[role + "s"] = scale
        out[role] = (t / torch.where(scale > 0.0, scale, torch.ones_like(scale))[:, None]).flatten()
    return out
