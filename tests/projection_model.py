"""The Newton–Schulz update with the roundings its kernels make (csrc/tg_ortho.hip):
X in fp32, the products' operands in one or two binary16 parts under their scales, the
diagonals of A and B in fp32, one rounding to bfloat16 at the end.  Sums are taken in
64 bits and rounded to fp32 once, where the kernels sum in fp32."""
import torch

X_SCALE, S_SCALE = 16384.0, 4096.0


def f32(x):
    return x.float().double()


def parts(v, two):
    high = v.half().double()
    return [high, f32(v - high).half().double()] if two else [high]


def product(a, b):
    """a·bᵀ; of two parts each, without the two low ones."""
    t = [x.transpose(-1, -2).contiguous() for x in b]
    out = a[0] @ t[0]
    return f32(out + a[0] @ t[1] + a[1] @ t[0] if len(a) == 2 else out)


def newton_schulz(G, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, two=None):
    """batch × rows × cols in 64 bits, the result's values as the bfloat16 holds them.
    `two`: operands in two parts (as the kernels for a short side of up to 64)."""
    a, b, c = (float(torch.tensor(k, dtype=torch.float32)) for k in coefficients)
    X = G.double()
    X = X / (X.flatten(1).norm(dim=1)[:, None, None] + eps)
    flip = X.shape[1] > X.shape[2]
    if flip:
        X = X.transpose(1, 2).contiguous()
    two = X.shape[1] <= 64 if two is None else two
    x = f32(X)
    off = 1.0 - torch.eye(X.shape[1], dtype=torch.float64, device=X.device)
    for _ in range(steps):
        xp = parts(x * X_SCALE, two)
        A = product(xp, xp) / X_SCALE ** 2
        d = f32(A.diagonal(dim1=1, dim2=2))
        op = parts(f32(A * S_SCALE) * off, two)  # of A·2^12, symmetric
        o, oo = sum(op), product(op, op) / S_SCALE
        h = f32(b * o + c * ((d[:, :, None] + d[:, None, :]) * o + oo)) * off
        e = f32(b * d + c * (d * d + oo.diagonal(dim1=1, dim2=2) / S_SCALE))
        xt = [p.transpose(1, 2).contiguous() for p in xp]
        x = f32(f32(a + e)[:, :, None] * x + product(parts(h, two), xt) / (S_SCALE * X_SCALE))
    out = x.bfloat16().double()
    return out.transpose(1, 2).contiguous() if flip else out
