"""Plain 64-bit forms of the training operators and the error bounds that the tests
hold the kernels to (torch, on whatever device the inputs are).

u is the rounding of a type, half a step relative to the value (binary16 2^-11,
bfloat16 2^-8, fp32 2^-24); binary16 has an absolute floor of half its subnormal
spacing, 2^-25.  f32 sums of n terms err by at most n·2^-24 of the sum of
magnitudes (Higham, Accuracy and Stability of Numerical Algorithms, §3)."""
import math

import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
FLOOR = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0, torch.float32: 0.0}
E32 = 2.0 ** -24
BLOCK = 256


def clean(ends, rows):
    """What `ends` counts as: 0 to rows, none below the one before."""
    out, last = [], 0
    for x in ends.tolist():
        last = max(last, min(max(x, 0), rows))
        out.append(last)
    return out


def _product(a, b, dt):
    """a @ b in 64 bits and the bound of an fp32 sum of exact products, rounded once."""
    a, b = a.double(), b.double()
    y = a @ b
    s = a.shape[1] * E32 * (a.abs() @ b.abs())
    return y, s + U[dt] * (y.abs() + s) + FLOOR[dt]


def grouped(X, W, ends, dY=None):
    """dict of Y and, with dY, dX and dW, and for each the bound ``tol_*``."""
    dt, dev = X.dtype, X.device
    M, (E, N, K) = X.shape[0], W.shape
    out = {}

    def zeros(name, *shape):
        out[name] = torch.zeros(*shape, dtype=torch.float64, device=dev)
        out["tol_" + name] = torch.zeros(*shape, dtype=torch.float64, device=dev)

    zeros("Y", M, N)
    if dY is not None:
        zeros("dX", M, K)
        zeros("dW", E, N, K)
    a = 0
    for e, b in enumerate(clean(ends, M)):
        if b > a:
            out["Y"][a:b], out["tol_Y"][a:b] = _product(X[a:b], W[e].t(), dt)
            if dY is not None:
                out["dX"][a:b], out["tol_dX"][a:b] = _product(dY[a:b], W[e], dt)
                out["dW"][e], out["tol_dW"][e] = _product(dY[a:b].t(), X[a:b], dt)
        a = max(a, b)
    return out


def lookup(tokens, W, scale=1.0):
    """Y and its bound; NaN rows for tokens outside."""
    V, dt = W.shape[0], W.dtype
    inside = (tokens >= 0) & (tokens < V)
    scale = float(torch.tensor(scale, dtype=torch.float32))
    if V:
        y = scale * W[torch.where(inside, tokens, torch.zeros_like(tokens))].double()
        y[~inside] = math.nan
    else:
        y = torch.full((*tokens.shape, W.shape[1]), math.nan, dtype=torch.float64, device=W.device)
    # the product in fp32, then one rounding
    return y, (U[dt] + 2 * E32) * y.abs() + FLOOR[dt]


def lookup_gradient(tokens, dY, V, scale=1.0, padding=None):
    """dW and its bound."""
    dt, K = dY.dtype, dY.shape[-1]
    tokens, dY = tokens.flatten(), dY.reshape(-1, K).double()
    keep = (tokens >= 0) & (tokens < V)
    if padding is not None:
        keep &= tokens != padding
    t, g = tokens[keep], dY[keep]
    zeros = torch.zeros(V, K, dtype=torch.float64, device=dY.device)
    scale = float(torch.tensor(scale, dtype=torch.float32))
    s = zeros.index_add(0, t, g)
    size = zeros.index_add(0, t, g.abs())
    n = torch.bincount(t, minlength=V)[:, None].double()
    tol = abs(scale) * n * E32 * size
    return scale * s, tol + (U[dt] + 2 * E32) * ((scale * s).abs() + tol) + FLOOR[dt] * (n > 0)


def adamw(p, g, m, v, step, lr, betas, eps, weight_decay, g_scale=1.0):
    """(p, m, v) in 64 bits and a bound for each, without the rounding of a 16-bit p.

    Each fp32 operation and each factor errs by 2^-24 of itself: m is a sum of two
    products of a rounded factor, v of two with the square, so 3 and 5 roundings at
    most on the way to a term (one more for a scaled gradient) and one of the sum.
    The quotient has the error of m, half of v's, and the roundings of the root, its
    factor, product, sum and rate, and is itself a product with a reciprocal that is
    off by at most one unit in the last place: 2 + 1 half units."""
    b1, b2 = betas
    p, g, m, v = (t.double() for t in (p, g, m, v))
    g = g * g_scale
    m1 = b1 * m + (1 - b1) * g
    v1 = b2 * v + (1 - b2) * g * g
    # 1 − β is rounded from 64 bits: as near to its value as β is to its own
    tm = 4 * E32 * (b1 * m.abs() + (1 - b1) * g.abs()) + 2.0 ** -149
    tv = 7 * E32 * v1 + 2.0 ** -148
    denom = torch.sqrt(v1) / math.sqrt(1 - b2 ** step) + eps
    rate = lr / (1 - b1 ** step)
    q = m1 / denom
    # √(v + t) − √v <= √t, and t/√v where v is larger
    troot = torch.minimum(torch.sqrt(tv), tv / torch.sqrt(v1).clamp_min(1e-300)) + 3 * E32 * torch.sqrt(v1)
    tdenom = 1.01 * troot / math.sqrt(1 - b2 ** step) + 2 * E32 * denom
    tq = 1.01 * tm / denom + q.abs() * (1.01 * torch.minimum(tdenom / denom, torch.ones_like(denom)) + 3 * E32)
    p1 = (1 - lr * weight_decay) * p - rate * q
    tp = 3 * E32 * p.abs() + rate * (1.01 * tq + 3 * E32 * q.abs()) + E32 * p1.abs() + 2.0 ** -148
    return (p1, m1, v1), (tp, tm, tv)


def encode(x, root):
    """What adamw_8bit holds of fp32 values (m, or √v with ``root``), operation for operation: E4M3 values
    and scales of the blocks of 256, in torch on the CPU."""
    flat = x.detach().cpu().flatten().float()
    n = flat.numel()
    blocks = (n + BLOCK - 1) // BLOCK
    b = torch.zeros(blocks * BLOCK)
    b[:n] = flat
    b = b.view(blocks, BLOCK)
    top = b.abs().amax(1)
    held = ~(top < 2.0 ** -110)
    top_or_one = torch.where(held, top, torch.ones_like(top))
    q = b * torch.where(held, torch.ones_like(top) / top_or_one * 448.0, torch.zeros_like(top))[:, None]
    if root:
        q = torch.where(q > 0, torch.clamp(q, min=2.0 ** -9), q)
    codes = torch.clamp(q, -448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.view(-1)[:n].view(x.shape), torch.where(held, top * float(torch.tensor(1.0) / torch.tensor(448.0)), torch.zeros_like(top))


def decode(codes, scales):
    """fp32 values of E4M3 values and their blocks' scales, on the CPU."""
    n = codes.numel()
    flat = codes.detach().cpu().flatten().float()
    return (flat * scales.detach().cpu().repeat_interleave(BLOCK)[:n]).view(codes.shape)


def adamw_in_f32(p, g, m, v, step, lr, betas, eps, weight_decay, g_scale=None):
    """The step operation for operation in fp32 on the CPU: p (unrounded), m, v, √v, and how
    far p may be off where its quotient is within three half units instead of one half."""
    b1, b2 = betas
    f = lambda x: float(torch.tensor(x, dtype=torch.float64).float())  # noqa: E731  rounded once
    p, g, m, v = (t.detach().cpu().float() for t in (p, g, m, v))
    if g_scale is not None:
        g = g * g_scale
    m = m * f(b1) + g * f(1.0 - b1)
    v = v * f(b2) + (g * g) * f(1.0 - b2)
    r = v.double().sqrt().float()  # rounded to nearest, which torch's fp32 root is not always
    update = (m / (r * f(1.0 / math.sqrt(1.0 - b2 ** step)) + f(eps))) * f(lr / (1.0 - b1 ** step))
    p = p * f(1.0 - lr * weight_decay) - update
    # the quotients' 4 half units apart, one rounding of the product with the rate and one
    # of p in either computation
    return p, m, v, r, (6 * E32 * update.abs().double() + 2 * E32 * p.abs().double()) * (1 + 2.0 ** -20) + 2.0 ** -147
