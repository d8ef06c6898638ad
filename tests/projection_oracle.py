"""Plain 64-bit forms of the projection operators and the error bounds that the
tests hold the kernels to (torch, on whatever device the inputs are).

u is the rounding of the operands' type, half a step relative to the value
(binary16 2^-11, bfloat16 2^-8); f32 sums of n terms err by at most n·2^-24 of the
sum of magnitudes (Higham, Accuracy and Stability of Numerical Algorithms, §3)."""
import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
E32 = 2.0 ** -24


def live_rows(target, ignore):
    return torch.nonzero(target != ignore)[:, 0]


def xent(H, W, target, ignore=-100, reduction="mean", dloss=None, dlse=None):
    """dict of loss, lse and, with dloss (a scalar, or one per row for "none"),
    dH, dW, and for each the bound ``tol_*`` on the kernels' error."""
    M, V = H.shape[0], W.shape[0]
    K = H.shape[1]
    dt, dev = H.dtype, H.device
    rows = live_rows(target, ignore)
    n = max(1, rows.numel())
    h, w = H[rows].double(), W.double()
    t = target[rows]
    z = h @ w.t()
    lse = torch.logsumexp(z, 1)
    nll = lse - z[torch.arange(rows.numel(), device=dev), t]
    # a logit is an f32 sum of K exact products
    dz = (K * E32) * (h.abs() @ w.abs().t()).amax(1) if rows.numel() else torch.zeros(0, dtype=torch.float64, device=dev)
    # exponentials: the argument's rounding (for the terms that count |x| < 20, so
    # 30·2^-24) and the instruction's ulp, sums of at most 64 partial values in
    # sequence: below 2^-17 together; lse is rounded in base 2 and to f32
    per = dz + 2.0 ** -17 + 2.0 ** -21 * lse.abs()
    full = lambda x: torch.zeros(M, dtype=torch.float64, device=dev).index_copy(0, rows, x)  # noqa: E731
    out = {"lse": full(lse), "tol_lse": full(per), "loss": full(nll), "tol_loss": full(2 * per)}
    if reduction != "none":
        d = n if reduction == "mean" else 1
        out["loss"] = nll.sum() / d
        # and the f32 sum over the rows
        out["tol_loss"] = (2 * per).sum() / d + (rows.numel() + 64) * E32 * nll.abs().sum() / d
    if dloss is None:
        return out
    g = dloss.double() * torch.ones(M, dtype=torch.float64, device=dev) / (n if reduction == "mean" else 1)
    l = torch.zeros_like(g) if dlse is None else dlse.double()
    g, l = g[rows][:, None], l[rows][:, None]
    p = torch.softmax(z, 1)
    one = torch.zeros_like(z)
    one[torch.arange(rows.numel(), device=dev), t] = 1.0
    G = (g + l) * p - g * one
    u = U[dt]
    # each element of G: the exponential's relative error and one rounding of the
    # scaled sum; the scaled value's own floor is far below (2^-38 of the largest)
    top = float(torch.maximum(g.abs(), (g + l).abs()).amax()) if rows.numel() else 0.0
    eG = u * G.abs() + ((g + l) * p).abs() * (2 * dz[:, None] + 2.0 ** -15) + g.abs() * one * 2.0 ** -22 + top * 2.0 ** -38
    dH, dW = G @ w, G.t() @ h
    floor = 2.0 ** -25 if dt == torch.float16 else 0.0  # binary16's subnormal spacing, halved
    tH = eG @ w.abs() + (V + 64) * E32 * (G.abs() @ w.abs())
    tW = eG.t() @ h.abs() + (n + 64) * E32 * (G.abs().t() @ h.abs())
    out["dH"] = torch.zeros(M, K, dtype=torch.float64, device=dev).index_copy(0, rows, dH)
    out["tol_dH"] = torch.zeros(M, K, dtype=torch.float64, device=dev).index_copy(
        0, rows, tH + (u + 2.0 ** -22) * (dH.abs() + tH) + floor)
    out["dW"] = dW
    out["tol_dW"] = tW + (u + 2.0 ** -22) * (dW.abs() + tW) + floor
    return out


def newton_schulz(G, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7):
    """The iteration in 64 bits, batch × rows × cols."""
    X = G.double()
    X = X / (X.flatten(1).norm(dim=1)[:, None, None] + eps)
    flip = X.shape[1] > X.shape[2]
    if flip:
        X = X.transpose(1, 2).contiguous()
    for t in range(steps):
        a, b, c = coefficients[t] if hasattr(coefficients[0], "__len__") else coefficients
        A = X @ X.transpose(1, 2).contiguous()
        X = a * X + (b * A + c * (A @ A)) @ X
    return X.transpose(1, 2).contiguous() if flip else X


def newton_schulz_one_step_bound(G, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7):
    """Elementwise bound on the error of one step's bfloat16 result.

    With v = 2^-11 the rounding of a binary16 operand and q = (n + 8)·2^-24 that
    of an f32 sum of n terms: X's image errs by v|X|, A by (2v + v² + q)|X||X|ᵀ and
    its stored part by v more, B by the propagated error, its own sum and one
    rounding, the update by B's error, X's and its sum's.  The diagonals are exact
    to f32 and are covered by the same bound."""
    a, b, c = coefficients
    v = 2.0 ** -11
    X = G.double()
    X = X / (X.flatten(1).norm(dim=1)[:, None, None] + eps)
    flip = X.shape[1] > X.shape[2]
    if flip:
        X = X.transpose(1, 2).contiguous()
    s, l = X.shape[1], X.shape[2]
    Xa = X.abs()
    ql, qs = (l + 8) * E32, (s + 8) * E32
    A = X @ X.transpose(1, 2).contiguous()
    AA = Xa @ Xa.transpose(1, 2).contiguous()
    eA = (2 * v + v * v + ql) * AA + v * (A.abs() + (2 * v + ql) * AA) + 2.0 ** -37
    Ab = A.abs() + eA
    B = b * A + c * (A @ A)
    eB = abs(b) * eA + abs(c) * (Ab @ Ab - A.abs() @ A.abs() + qs * (Ab @ Ab)) + 8 * E32 * (abs(b) * Ab + abs(c) * (Ab @ Ab))
    eB = eB + v * (B.abs() + eB) + 2.0 ** -37
    Xn = a * X + B @ X
    e = eB @ Xa + (v + qs) * ((B.abs() + eB) @ Xa) + 8 * E32 * (abs(a) * Xa + (B.abs() + eB) @ Xa)
    e = e + 2.0 ** -8 * (Xn.abs() + e)
    if flip:
        Xn, e = Xn.transpose(1, 2).contiguous(), e.transpose(1, 2).contiguous()
    return Xn, e
