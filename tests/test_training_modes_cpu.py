"""Modes of autograd and tracing that the training operators do not follow: each is
refused, or raises where it would be used, instead of giving a number without its
derivative.  On the CPU: the wrappers run as they are, with the library's passes replaced
by the same formulas in torch and tensors that say they are on a GPU."""
import pytest

torch = pytest.importorskip("torch")
tg = pytest.importorskip("dense_fp16_gemm_02_amd")

import torch.autograd.forward_ad as fwad  # noqa: E402

from dense_fp16_gemm_02_amd import training as tr  # noqa: E402


class OnCard(torch.Tensor):
    is_cuda = True

    def get_device(self):
        return -1


def spans(ends):
    return zip([0] + ends.tolist()[:-1], ends.tolist())


def grouped_forward(X, W, ends, strides):
    with torch.no_grad():
        Y = torch.zeros(X.shape[0], W.shape[1])
        for e, (a, b) in enumerate(spans(ends)):
            Y[a:b] = X[a:b].float() @ W[e].float().t()
    return Y.to(X.dtype).as_subclass(OnCard)


def grouped_backward(X, W, ends, dY, strides, need_x, need_w):
    with torch.no_grad():
        dX, dW = torch.zeros(X.shape), torch.zeros(W.shape)
        for e, (a, b) in enumerate(spans(ends)):
            dX[a:b] = dY[a:b].float() @ W[e].float()
            dW[e] = dY[a:b].float().t() @ X[a:b].float()
    return dX.to(X.dtype) if need_x else None, dW.to(W.dtype) if need_w else None


def embedding_forward(tokens, W, ldw, scale):
    with torch.no_grad():
        return (W[tokens].float() * scale).to(W.dtype).as_subclass(OnCard)


def embedding_backward(tokens, dY, V, scale, padding):
    with torch.no_grad():
        dW = torch.zeros(V, dY.shape[-1]).index_add(0, tokens.flatten(), dY.reshape(-1, dY.shape[-1]).float()) * scale
        if padding >= 0:
            dW[padding] = 0
    return dW.to(dY.dtype)


@pytest.fixture
def card(monkeypatch):
    monkeypatch.setattr(tr, "_grouped_forward", grouped_forward)
    monkeypatch.setattr(tr, "_grouped_backward", grouped_backward)
    monkeypatch.setattr(tr, "_embedding_forward", embedding_forward)
    monkeypatch.setattr(tr, "_embedding_backward", embedding_backward)
    gen = torch.Generator().manual_seed(0)
    X = torch.randn(6, 8, generator=gen).half().as_subclass(OnCard)
    W = torch.randn(3, 4, 8, generator=gen).half().as_subclass(OnCard)
    ends = torch.tensor([2, 2, 6]).as_subclass(OnCard)
    T = torch.randn(5, 8, generator=gen).half().as_subclass(OnCard)
    tokens = torch.tensor([0, 3, 3, 1]).as_subclass(OnCard)
    return X, W, ends, T, tokens


def calls(card):
    """Each operator as a function of its differentiable arguments."""
    X, W, ends, T, tokens = card
    return [(lambda x, w: tg.grouped_linear(x, w, ends), (X, W)), (lambda t: tg.embedding(tokens, t, 2.0), (T,))]


def test_the_stubs_stand_for_the_library(card):
    """Otherwise the other tests would say nothing."""
    X, W, ends, T, tokens = card
    x, w = X.clone().requires_grad_(), W.clone().requires_grad_()
    dX, dW = torch.autograd.grad(tg.grouped_linear(x, w, ends).float().square().sum(), (x, w))
    x32, w32 = X.detach().float().requires_grad_(), W.detach().float().requires_grad_()
    y = torch.cat([x32[a:b] @ w32[e].t() for e, (a, b) in enumerate(spans(ends))])
    eX, eW = torch.autograd.grad(y.square().sum(), (x32, w32))
    assert torch.allclose(dX.float(), eX, rtol=1e-2, atol=1e-2) and torch.allclose(dW.float(), eW, rtol=1e-2, atol=1e-2)
    t = T.clone().requires_grad_()
    dT, = torch.autograd.grad(tg.embedding(tokens, t, 2.0, padding_idx=1).float().sum(), t)
    assert dT[:, 0].tolist() == [2.0, 0.0, 0.0, 4.0, 0.0]


@pytest.mark.parametrize("op", [0, 1])
@pytest.mark.parametrize("requires_grad", [False, True])
def test_forward_mode_is_refused(card, op, requires_grad):
    call, args = calls(card)[op]
    for k in range(len(args)):
        with fwad.dual_level():
            dual = [fwad.make_dual(a, torch.ones_like(a)) if i == k else a.clone().requires_grad_(requires_grad)
                    for i, a in enumerate(args)]
            with pytest.raises(NotImplementedError, match="forward-mode"):
                call(*dual)
            call(*args)  # a dual level without dual tensors is nothing to object to


@pytest.mark.parametrize("op", [0, 1])
def test_forward_mode_through_the_upstream_gradient_is_refused(card, op):
    call, args = calls(card)[op]
    leaves = [a.clone().requires_grad_() for a in args]
    y = call(*leaves)
    with fwad.dual_level():
        up = fwad.make_dual(torch.ones_like(y), torch.ones_like(y))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            torch.autograd.grad(y, leaves, up)


@pytest.mark.parametrize("op", [0, 1])
def test_second_derivatives_raise_where_they_are_taken(card, op):
    call, args = calls(card)[op]
    leaves = [a.clone().requires_grad_() for a in args]
    y = call(*leaves)
    loss = y.float().square().sum()  # so that the upstream gradient depends on the leaves
    plain = torch.autograd.grad(loss, leaves, retain_graph=True)
    grads = torch.autograd.grad(loss, leaves, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(plain, grads))
    with pytest.raises(RuntimeError, match="differentiated once"):
        sum(g.float().square().sum() for g in grads).backward()


def test_the_gradient_of_a_lookup_does_not_depend_on_the_table(card):
    X, W, ends, T, tokens = card
    t = T.clone().requires_grad_()
    y = tg.embedding(tokens, t)
    dT, = torch.autograd.grad(y, t, torch.ones_like(y), create_graph=True)
    assert not dT.requires_grad


@pytest.mark.parametrize("op", [0, 1])
def test_tracing_is_refused(card, op):
    from torch.fx.experimental.proxy_tensor import make_fx

    call, args = calls(card)[op]
    with pytest.raises(Exception, match="cannot be traced"):
        torch.jit.trace(call, tuple(args), check_trace=False)
    with pytest.raises(NotImplementedError, match="cannot be traced"):
        make_fx(call)(*args)


def test_an_update_of_a_saved_operand_is_noticed(card):
    X, W, ends, T, tokens = card
    w = W.clone().requires_grad_()
    y = tg.grouped_linear(X, w, ends)
    with torch.no_grad():
        ends.add_(0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.float().sum().backward()
    t = T.clone().requires_grad_()
    y = tg.embedding(tokens, t)
    with torch.no_grad():
        t.add_(1.0)  # the table itself is not needed for its gradient
    y.float().sum().backward()
    y = tg.embedding(tokens, t)
    tokens.add_(0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.float().sum().backward()


def test_refusals_of_the_wrappers(card):
    X, W, ends, T, tokens = card
    for bad in (lambda: tg.grouped_linear(X[0], W, ends), lambda: tg.grouped_linear(X, W[0], ends),
                lambda: tg.grouped_linear(X, W, ends[None]), lambda: tg.grouped_linear(X[:, :4], W, ends),
                lambda: tg.grouped_linear(X, W, ends[:2]), lambda: tg.grouped_linear(X[:1].expand(6, 8), W, ends),
                lambda: tg.grouped_linear(X.t().contiguous().t(), W, ends),
                lambda: tg.grouped_linear(X, W.transpose(1, 2).contiguous().transpose(1, 2), ends),
                lambda: tg.grouped_linear(X, W[:, :1].expand(3, 4, 8), ends),
                lambda: tg.embedding(tokens, T[0]), lambda: tg.embedding(tokens, T[:1].expand(5, 8)),
                lambda: tg.embedding(tokens, T.t()), lambda: tg.embedding(tokens, T, padding_idx=5),
                lambda: tg.embedding(tokens, T, padding_idx=-1), lambda: tg.embedding(tokens, T, scale=float("nan")),
                lambda: tg.embedding(tokens, T, scale=1e39)):
        with pytest.raises(ValueError):
            bad()


def test_refusals_of_adamw():
    def on_card(*shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype).as_subclass(OnCard)

    p, g, m, v = ([on_card(4, 4)] for _ in range(4))
    half, short = [on_card(4, 4, dtype=torch.float16)], [on_card(3, 4)]
    for kind, bad in (
            (TypeError, lambda: tg.adamw(half, [on_card(4, 4, dtype=torch.bfloat16)], m, v, 1)),
            (TypeError, lambda: tg.adamw(half, g, m, v, 1)), (TypeError, lambda: tg.adamw(p, g, half, v, 1)),
            (TypeError, lambda: tg.adamw([on_card(4, 4, dtype=torch.float64)], g, m, v, 1)),
            (TypeError, lambda: tg.adamw(p + half, g + half, m + m, v + v, 1)),
            (ValueError, lambda: tg.adamw(p, short, m, v, 1)), (ValueError, lambda: tg.adamw(p, g, short, v, 1)),
            (ValueError, lambda: tg.adamw(p, [on_card(16)], m, v, 1)), (ValueError, lambda: tg.adamw(p, g, m, [], 1)),
            (ValueError, lambda: tg.adamw(p, [on_card(8, 4)[::2]], m, v, 1)),
            (ValueError, lambda: tg.adamw(half, half, m, v, 1, copies=half)),
            (ValueError, lambda: tg.adamw(p, g, m, v, 1, copies=half + half)),
            (TypeError, lambda: tg.adamw(p, g, m, v, 1, copies=g)),
            (TypeError, lambda: tg.adamw_8bit(p, g, m, [on_card(1)], v, [on_card(1)], 1)),
            (ValueError, lambda: tg.adamw(p, g, m, v, torch.ones(2, dtype=torch.int64))),
            (ValueError, lambda: tg.adamw(p, g, m, v, torch.ones(1))),
            (ValueError, lambda: tg.adamw(p, g, m, v, 1, lr=torch.ones(1, dtype=torch.float64)))):
        with pytest.raises(kind):
            bad()
    with fwad.dual_level():
        with pytest.raises(NotImplementedError, match="forward-mode"):
            tg.adamw(p, [fwad.make_dual(g[0], g[0].clone())], m, v, 1)


def test_a_parameter_without_a_gradient_is_refused():
    def on_card():
        return torch.zeros(4).as_subclass(OnCard)

    with pytest.raises(TypeError, match="grads"):
        tg.adamw([on_card(), on_card()], [on_card(), None], [on_card(), on_card()], [on_card(), on_card()], 1)
