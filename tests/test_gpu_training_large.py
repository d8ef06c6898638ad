"""The training operators on tensors of more than 2^31 elements: offsets past 32
bits, at the ends and around the border."""
import gc
import math

import pytest

torch = pytest.importorskip("torch")
tg = pytest.importorskip("dense_fp16_gemm_02_amd")

import training_oracle as oracle  # noqa: E402

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def free():
    yield
    gc.collect()
    torch.cuda.empty_cache()


def noise(*shape, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda", dtype=BF16)


def close(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()))


def test_embedding_of_a_large_table():
    V, K, M = 600011, 4096, 3000
    W = noise(V, K)
    gen = torch.Generator().manual_seed(1)
    border = (1 << 31) // K
    tokens = torch.cat([torch.randint(0, V, (M - 300,), generator=gen), torch.arange(V - 100, V),
                        torch.arange(border - 50, border + 50), torch.full((100,), V - 1)]).cuda()
    Y = tg.embedding(tokens, W)
    assert torch.equal(Y, W[tokens])
    dY = noise(M, K, seed=2)
    w = W.requires_grad_()
    dW, = torch.autograd.grad(tg.embedding(tokens, w), w, dY)
    rows = tokens.unique()
    order = torch.searchsorted(rows, tokens)
    want, tol = oracle.lookup_gradient(order, dY, rows.numel())
    close(dW[rows], want, tol, "dW")
    dW[rows] = 0
    assert not dW.any()


def test_embedding_of_many_tokens():
    V, K, M = 1000, 1024, 2200007
    gen = torch.Generator().manual_seed(3)
    tokens = torch.randint(0, V, (M,), generator=gen).cuda()
    W, dY = noise(V, K), noise(M, K, seed=4)
    w = W.requires_grad_()
    Y = tg.embedding(tokens, w)
    for a in (0, (1 << 31) // K - 500, M - 1000):
        assert torch.equal(Y[a:a + 1000], W[tokens[a:a + 1000]])
    dW, = torch.autograd.grad(Y, w, dY)
    for v in (0, 517, V - 1):
        i = torch.nonzero(tokens == v)[:, 0]
        want, tol = oracle.lookup_gradient(torch.zeros_like(i), dY[i], 1)
        close(dW[v:v + 1], want, tol, v)


def test_grouped_products_of_many_rows():
    M, E, N, K = 530000, 3, 136, 4096
    ends = torch.tensor([100, 529000, 529990]).cuda()
    X, W, dY = noise(M, K), noise(E, N, K, seed=1) / math.sqrt(K), noise(M, N, seed=2)
    x, w = X.requires_grad_(), W.requires_grad_()
    Y = tg.grouped_linear(x, w, ends)
    dX, dW = torch.autograd.grad(Y, (x, w), dY)
    assert not Y[529990:].any() and not dX[529990:].any()
    border = (1 << 31) // K
    for a, b, e in ((0, 100, 0), (100, 400, 1), (border - 200, border + 200, 1), (528800, 529000, 1), (529000, 529990, 2)):
        close(Y[a:b], *oracle._product(X[a:b], W[e].t(), BF16), "Y")
        close(dX[a:b], *oracle._product(dY[a:b], W[e], BF16), "dX")
    close(dW[0], *oracle._product(dY[:100].t(), X[:100], BF16), "dW")
    close(dW[2], *oracle._product(dY[529000:529990].t(), X[529000:529990], BF16), "dW")
    # over the long group in pieces
    want = torch.zeros(N, K, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    for a in range(100, 529000, 20000):
        b = min(a + 20000, 529000)
        p, q = dY[a:b].double().t(), X[a:b].double()
        want += p @ q
        size += p.abs() @ q.abs()
    # fp32 sums of 8192 rows or more of one part after the other: their number bounds them all
    tol = 529000 * oracle.E32 * size
    close(dW[1], want, tol + oracle.U[BF16] * (want.abs() + tol), "dW")


@pytest.mark.parametrize("M", [40, 2000])
def test_grouped_products_of_large_weights(M):
    E, N, K = 140, 4096, 4096
    W = noise(E, N, K)
    gen = torch.Generator().manual_seed(5)
    ends = torch.randint(0, E, (M,), generator=gen).bincount(minlength=E).cumsum(0)
    ends[:-1] -= ends[:-1] // 3  # so that the last expert has many
    X, dY = noise(M, K, seed=1), noise(M, N, seed=2)
    x, w = X.requires_grad_(), W.requires_grad_()
    ends = ends.cuda()
    Y = tg.grouped_linear(x, w, ends)
    dX, dW = torch.autograd.grad(Y, (x, w), dY)
    a = 0
    for e, b in enumerate(ends.tolist()):
        if b > a and (e < 3 or e > 125):
            close(Y[a:b], *oracle._product(X[a:b], W[e].t(), BF16), "Y")
            close(dX[a:b], *oracle._product(dY[a:b], W[e], BF16), "dX")
            close(dW[e], *oracle._product(dY[a:b].t(), X[a:b], BF16), "dW")
        elif b == a:
            assert not dW[e].any()
        a = b


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_of_a_large_tensor(bits):
    """What a call on the whole tensor gives for its ends and its middle is what calls on those give."""
    n = (1 << 31) + 4096 * 3 + 77
    how = dict(lr=1e-2, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)
    p, g = noise(n), noise(n, seed=1)
    if bits == 32:
        state = [torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")]
        call = tg.adamw
    else:
        state = list(tg.adamw_8bit_state(p))
        call = tg.adamw_8bit
    windows = [slice(0, 4096), slice((1 << 31) - 2048, (1 << 31) + 2048), slice((1 << 31) + 4096 * 3 - 1024, n)]
    scale = lambda s: slice(s.start // 256, -(-s.stop // 256))  # noqa: E731
    parts = [[[p[s].clone()], [g[s].clone()]] + [[t[scale(s) if t.numel() < n else s].clone()] for t in state] for s in windows]
    for step in (1, 2):
        call([p], [g], *[[t] for t in state], step, **how)
        for part in parts:
            call(*part, step, **how)
    for s, part in zip(windows, parts):
        assert torch.equal(p[s], part[0][0])
        for t, q in zip(state, part[2:]):
            assert torch.equal(t[scale(s) if t.numel() < n else s].view(torch.uint8), q[0].view(torch.uint8))
    assert torch.isfinite(p).all()
