"""The training operators called as programs call them: from two threads, with a graph
kept for a second backward pass, in inference mode, recomputed under a checkpoint, and with
the same operand in two places.  Every result is compared with that of one plain call, bit
for bit, as the operators give the same bits at every call."""
import threading

import pytest

torch = pytest.importorskip("torch")
tg = pytest.importorskip("dense_fp16_gemm_02_amd")

from torch.utils.checkpoint import checkpoint  # noqa: E402

pytestmark = pytest.mark.gpu


def problem(seed, M=700, E=5, N=96, K=160, V=300):
    gen = torch.Generator().manual_seed(seed)
    T = torch.randn(V, K, generator=gen).bfloat16().cuda().requires_grad_()
    W = (torch.randn(E, N, K, generator=gen) / 8).bfloat16().cuda().requires_grad_()
    tokens = torch.randint(0, V, (M,), generator=gen).cuda()
    ends = torch.randint(0, M, (E,), generator=gen).sort().values.cuda()
    dY = torch.randn(M, N, generator=gen).bfloat16().cuda()
    return T, W, tokens, ends, dY


def layer(T, W, tokens, ends):
    return tg.grouped_linear(tg.embedding(tokens, T, 0.5), W, ends)


def step(T, W, tokens, ends, dY):
    Y = layer(T, W, tokens, ends)
    return (Y.detach(), *torch.autograd.grad(Y, (T, W), dY))


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b, strict=True))


def test_two_threads():
    """Each with a stream of its own; the updates of AdamW come in between."""
    problems = [problem(1), problem(2, M=9000, V=70000)]
    states = [[torch.zeros(5000, device="cuda") for _ in range(3)] for _ in problems]
    torch.cuda.synchronize()
    want = [step(*p) for p in problems]
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def work(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                p, m, v = states[k]
                g = torch.full_like(p, k + 1.0)
                for i in range(20):
                    got[k].append(step(*problems[k]))
                    tg.adamw([p], [g], [m], [v], i + 1, weight_decay=0.0)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # shown by the assertion below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for k in (0, 1):
        assert all(same(x, want[k]) for x in got[k])
    p, m, v = (torch.zeros(5000, device="cuda") for _ in range(3))
    for i in range(20):
        tg.adamw([p], [torch.ones_like(p)], [m], [v], i + 1, weight_decay=0.0)
    assert torch.equal(states[0][0], p)


def test_a_graph_that_is_kept():
    T, W, tokens, ends, dY = problem(3)
    Y = layer(T, W, tokens, ends)
    a = torch.autograd.grad(Y, (T, W), dY, retain_graph=True)
    b = torch.autograd.grad(Y, (T, W), dY)
    assert same(a, b)


def test_recomputed_under_a_checkpoint():
    T, W, tokens, ends, dY = problem(4)
    Y = checkpoint(layer, T, W, tokens, ends, use_reentrant=False)
    assert same((Y.detach(), *torch.autograd.grad(Y, (T, W), dY)), step(T, W, tokens, ends, dY))


def test_inference_mode():
    T, W, tokens, ends, dY = problem(5)
    want = layer(T, W, tokens, ends).detach()
    with torch.inference_mode():
        Y = layer(T, W, tokens.clone(), ends.clone())
        Z = tg.grouped_linear(tg.embedding(tokens, T.detach().clone(), 0.5), W.detach().clone(), ends)
    assert torch.equal(Y, want) and torch.equal(Z, want) and not Y.requires_grad


def test_one_weight_in_two_places():
    """Autograd adds up what each use of a weight gives, rounded to its type."""
    T, W, tokens, ends, dY = problem(6)
    X = tg.embedding(tokens, T)
    first, second = tg.grouped_linear(X, W, ends), tg.grouped_linear(X, W, ends // 2)
    both = torch.autograd.grad((first, second), W, (dY, dY), retain_graph=True)[0]
    one = torch.autograd.grad(first, W, dY, retain_graph=True)[0]
    two = torch.autograd.grad(second, W, dY)[0]
    assert torch.equal(both, one + two)


def test_a_table_that_is_the_projection_too():
    """Tied weights: the lookup's gradient and the vocabulary projection's are added."""
    T, W, tokens, ends, dY = problem(7)
    target = tokens.roll(-1)
    loss = tg.linear_cross_entropy(tg.embedding(tokens, T), T, target)
    both = torch.autograd.grad(loss, T)[0]
    looked, projected = T.detach().clone().requires_grad_(), T.detach().clone().requires_grad_()
    loss = tg.linear_cross_entropy(tg.embedding(tokens, looked), projected, target)
    a, b = torch.autograd.grad(loss, (looked, projected))
    assert torch.equal(both, a + b)


@pytest.mark.parametrize("pin", [False, True])
@pytest.mark.parametrize("layout", ["contiguous", "window of X", "window of W", "experts inside", "shared weight"])
def test_saved_tensors_that_were_offloaded(layout, pin):
    """torch.autograd.graph.save_on_cpu brings operands back in rows without what lay between them."""
    T, W, tokens, ends, dY = problem(8)
    E, N, K = W.shape
    X = tg.embedding(tokens, T).detach()
    W = W.detach()
    if layout == "window of X":
        wide = torch.full((X.shape[0], 3 * K), float("nan"), dtype=X.dtype, device="cuda")
        wide[:, K:2 * K] = X
        X = wide[:, K:2 * K]
    elif layout == "window of W":
        deep = torch.full((E, N + 5, K + 8), float("nan"), dtype=W.dtype, device="cuda")
        deep[:, 2:2 + N, :K] = W
        W = deep[:, 2:2 + N, :K]
    elif layout == "experts inside":
        W = W.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    elif layout == "shared weight":
        W = W[:1].expand(E, N, K)
    X.requires_grad_(), W.requires_grad_()
    Y = tg.grouped_linear(X, W, ends)
    want = (Y.detach(), *torch.autograd.grad(Y, (X, W), dY))
    with torch.autograd.graph.save_on_cpu(pin_memory=pin):
        Z = tg.grouped_linear(X, W, ends)
        rows = tg.embedding(tokens.view(7, 100), T)
    assert same((Z.detach(), *torch.autograd.grad(Z, (X, W), dY)), want)
    up = torch.ones_like(rows)
    assert torch.equal(torch.autograd.grad(rows, T, up)[0], torch.autograd.grad(tg.embedding(tokens.view(7, 100), T), T, up)[0])
