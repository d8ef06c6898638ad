"""The projection operators on tensors of more than 2^31 elements, each kind of operand
in turn, against 64-bit forms taken a slice at a time."""
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
tg = pytest.importorskip("dense_fp16_gemm_02_amd")

import projection_oracle as po  # noqa: E402

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
LIMIT = 2 ** 31


@pytest.fixture(autouse=True)
def room():
    yield
    torch.cuda.empty_cache()


def say(*a):
    print("[gpu-case]", *a, file=sys.stderr, flush=True)


def noise(shape, dt, seed, scale=1.0):
    """Standard normal values, made a slice at a time."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty(shape, dtype=dt, device="cuda")
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 28):
        part = flat[at:at + (1 << 28)]
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda") * scale)
    return out


def gradients(H, W, t):
    h, w = H.requires_grad_(), W.requires_grad_()
    loss, lse = tg.linear_cross_entropy(h, w, t, reduction="sum", return_lse=True)
    dH, dW = torch.autograd.grad(loss, (h, w), torch.full((), 0.75, device="cuda"))
    return loss.detach(), lse.detach(), dH, dW


def test_a_vocabulary_of_more_than_2_to_the_31_weights():
    M, V, K = 8, 600011, 4096
    W = noise((V, K), BF16, 1, K ** -0.5)
    assert W.numel() > LIMIT
    t = torch.tensor([0, 1, V - 1, V - 2, V // 2, -100, 524288, 524287], device="cuda")  # 2^31 / K and before
    live = t >= 0
    H = (noise((M, K), BF16, 2).float() + 5.0 * W[t.clamp(min=0)].float()).to(BF16)
    say(M, V, K, tg.tg_xent_plan(H, W, M, V, K, K, K, 1))
    loss, lse, dH, dW = gradients(H, W.detach(), t)
    h = H.detach().double()
    step = 1 << 16
    z = torch.cat([h @ W.detach()[v:v + step].double().t().contiguous() for v in range(0, V, step)], 1)
    want = torch.logsumexp(z, 1)
    # a logit's fp32 sum of K products, exponentials and sums as in projection_oracle
    dz = K * po.E32 * max(float((h.abs() @ W.detach()[v:v + step].double().abs().t().contiguous()).max()) for v in range(0, V, step))
    assert float((lse.double() - want)[live].abs().max()) <= dz + 2.0 ** -17 + 2.0 ** -21 * float(want.abs().max())
    assert float(lse[5]) == 0.0
    G = torch.softmax(z, 1)
    G[torch.arange(M, device="cuda"), t.clamp(min=0)] -= 1.0
    G *= 0.75 * live[:, None]
    u = po.U[BF16]
    # G half a step of its type and the exponential's error, the product's fp32 sum, one rounding
    eG = u * G.abs() + 0.75 * torch.softmax(z, 1) * (2 * dz + 2.0 ** -15) + 0.75 * 2.0 ** -38
    eG[torch.arange(M, device="cuda"), t.clamp(min=0)] += 0.75 * 2.0 ** -22
    exact, tol = torch.zeros(M, K, dtype=torch.float64, device="cuda"), torch.zeros(M, K, dtype=torch.float64, device="cuda")
    for v in range(0, V, step):
        w = W.detach()[v:v + step].double()
        g, e = G[:, v:v + step].contiguous(), eG[:, v:v + step].contiguous()
        exact += g @ w
        tol += (e + (V + 64) * po.E32 * g.abs()) @ w.abs()
        dw, tw = g.t().contiguous() @ h, (e + (M + 64) * po.E32 * g.abs()).t().contiguous() @ h.abs()
        bad = ~((dW[v:v + step].double() - dw).abs() <= tw + (u + 2.0 ** -22) * (dw.abs() + tw))
        assert not bool(bad.any()), (v, int(bad.sum()))
    assert bool(((dH.double() - exact).abs()[live] <= (tol + (u + 2.0 ** -22) * (exact.abs() + tol))[live]).all())
    assert not dH[5].any()


def test_tokens_of_more_than_2_to_the_31_elements():
    M, V, K = 600011, 100, 4096
    H = noise((M, K), F16, 3)
    assert H.numel() > LIMIT
    W = noise((V, K), F16, 4, K ** -0.5)
    t = torch.randint(0, V, (M,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    t[::7] = -100
    say(M, V, K, tg.tg_xent_plan(H, W, M, V, K, K, K, 1))
    loss, lse, dH, dW = gradients(H, W, t)
    H, W = H.detach(), W.detach()
    total, tol_loss, nll, dw = 0.0, 0.0, 0.0, torch.zeros(V, K, dtype=torch.float64, device="cuda")
    step = 1 << 16
    for m in range(0, M, step):
        ref = po.xent(H[m:m + step], W, t[m:m + step], reduction="sum", dloss=torch.full((), 0.75, device="cuda"))
        assert bool(((lse[m:m + step].double() - ref["lse"]).abs() <= ref["tol_lse"]).all()), m
        assert bool(((dH[m:m + step].double() - ref["dH"]).abs() <= ref["tol_dH"]).all()), m
        total, tol_loss, nll = total + float(ref["loss"]), tol_loss + float(ref["tol_loss"]), nll + float(ref["loss"].abs())
        dw += ref["dW"]
    assert abs(float(loss) - total) <= tol_loss + (M + 64) * po.E32 * nll
    # (the worst case of so long a sum in fp32 is beyond its value.)  The roundings of G
    # and of the result are at most 2^-11 each and independent of one another, those of
    # the sum some (M/32)^1/2·2^-24 of it
    assert float((dW.double() - dw).norm()) <= 2.0 ** -10 * float(dw.norm())


def gram_form(G, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, step=1 << 16):
    """X after the steps as factor·X0 with the long side a slice at a time: the iteration
    acts on the Gram matrix of the shorter side.  Yields (slice, its exact columns)."""
    wide = G.shape[0] <= G.shape[1]
    s, l = (G.shape if wide else G.shape[::-1])
    part = lambda c: (G[:, c:c + step] if wide else G[c:c + step].t()).double().contiguous()  # noqa: E731
    A = torch.zeros(s, s, dtype=torch.float64, device=G.device)
    for c in range(0, l, step):
        X = part(c)
        A += X @ X.t().contiguous()
    scale = 1.0 / (float(A.diagonal().sum().sqrt()) + eps)
    A *= scale ** 2
    eye = torch.eye(s, dtype=torch.float64, device=G.device)
    factor, (a, b, k) = eye * scale, coefficients
    for _ in range(steps):
        P = a * eye + b * A + k * (A @ A)
        factor, A = P @ factor, P @ A @ P
    for c in range(0, l, step):
        yield slice(c, c + step), factor @ part(c)


@pytest.mark.parametrize("m,n", [(1100, 2000003), (2000003, 1100)])
def test_a_matrix_of_more_than_2_to_the_31_elements(m, n):
    G = noise((m, n), BF16, 6)
    assert G.numel() > LIMIT
    say(m, n, tg.tg_newton_schulz_plan(1, m, n))
    O = tg.newton_schulz(G)
    off = of = 0.0
    for at, want in gram_form(G):
        got = (O[:, at] if m <= n else O[at].t()).double()
        e, w = float((got - want).norm()), float(want.norm())
        assert e <= 2.0 ** -8 * w, (at, e / w)  # every slice alone
        off, of = off + e * e, of + w * w
    say("off", (off / of) ** 0.5)


@pytest.mark.parametrize("b,m,n", [(33, 8192, 8192), (520, 64, 65601)])
def test_a_batch_of_more_than_2_to_the_31_elements(b, m, n):
    G = noise((b, m, n), BF16, 7)
    assert G.numel() > LIMIT
    say(b, m, n, tg.tg_newton_schulz_plan(b, m, n))
    O = tg.newton_schulz(G)
    for i in (0, LIMIT // (m * n), b - 1):  # that around element 2^31 among them
        for at, want in gram_form(G[i]):
            e, w = float((O[i][:, at].double() - want).norm()), float(want.norm())
            assert e <= 2.0 ** -8 * w, (i, at, e / w)
