"""Modes of autograd and tracing that the projection operators do not follow: each
is refused, or raises where it would be used, instead of giving a number without its
derivative.  On the CPU: the wrappers run as they are, with the library's two passes
replaced by the same formulas in torch and tensors that say they are on a GPU."""
import pytest

torch = pytest.importorskip("torch")
tg = pytest.importorskip("dense_fp16_gemm_02_amd")

import torch.autograd.forward_ad as fwad  # noqa: E402

from dense_fp16_gemm_02_amd import projection as pr  # noqa: E402


class OnCard(torch.Tensor):
    is_cuda = True


def forward(H, W, target, ignore_index, reduction, want_lse):
    with torch.no_grad():
        z = H.float() @ W.float().t()
        lse = torch.logsumexp(z, 1)
        loss = (lse - z.gather(1, target[:, None])[:, 0]).mean()
    return loss, lse if want_lse else None


def backward(H, W, target, lse, dloss, dlse, need_h, need_w, ignore_index, reduction):
    with torch.no_grad():
        G = torch.exp(H.float() @ W.float().t() - lse[:, None])
        G = (G - torch.nn.functional.one_hot(target, W.shape[0])) * dloss / H.shape[0]
        if dlse is not None:
            G = G + dlse[:, None] * torch.exp(H.float() @ W.float().t() - lse[:, None])
        return (G @ W.float()).to(H.dtype) if need_h else None, (G.t() @ H.float()).to(W.dtype) if need_w else None


@pytest.fixture
def card(monkeypatch):
    monkeypatch.setattr(pr, "_forward", forward)
    monkeypatch.setattr(pr, "_backward", backward)
    gen = torch.Generator().manual_seed(0)
    H = torch.randn(6, 16, generator=gen).half().as_subclass(OnCard)
    W = torch.randn(9, 16, generator=gen).half().as_subclass(OnCard)
    return H, W, torch.arange(6).as_subclass(OnCard)


def test_the_stubs_stand_for_the_library(card):
    """Otherwise the other tests would say nothing."""
    H, W, t = card
    h, w = H.clone().requires_grad_(), W.clone().requires_grad_()
    loss = tg.linear_cross_entropy(h, w, t)
    dH, dW = torch.autograd.grad(loss, (h, w))
    h32, w32 = H.detach().float().requires_grad_(), W.detach().float().requires_grad_()
    want = torch.nn.functional.cross_entropy(h32 @ w32.t(), t)
    eH, eW = torch.autograd.grad(want, (h32, w32))
    assert torch.allclose(loss, want, rtol=1e-6)
    assert torch.allclose(dH.float(), eH, rtol=2e-3, atol=1e-6) and torch.allclose(dW.float(), eW, rtol=2e-3, atol=1e-6)


@pytest.mark.parametrize("which", ["H", "W"])
@pytest.mark.parametrize("requires_grad", [False, True])
def test_forward_mode_is_refused(card, which, requires_grad):
    H, W, t = card
    with fwad.dual_level():
        h = fwad.make_dual(H, torch.ones_like(H)) if which == "H" else H
        w = fwad.make_dual(W, torch.ones_like(W)) if which == "W" else W
        if requires_grad:
            h = h.requires_grad_() if which == "W" else h
            w = w.requires_grad_() if which == "H" else w
        with pytest.raises(NotImplementedError, match="forward-mode"):
            tg.linear_cross_entropy(h, w, t)
        tg.linear_cross_entropy(H, W, t)  # a dual level without dual tensors is nothing to object to


def test_forward_mode_through_the_upstream_gradient_is_refused(card):
    H, W, t = card
    h = H.clone().requires_grad_()
    loss = tg.linear_cross_entropy(h, W, t)
    with fwad.dual_level():
        up = fwad.make_dual(torch.ones(()), torch.ones(()))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            torch.autograd.grad(loss, h, up)


def test_forward_mode_of_the_update_is_refused():
    G = torch.ones(3, 4).as_subclass(OnCard)
    with fwad.dual_level():
        with pytest.raises(NotImplementedError, match="forward-mode"):
            tg.newton_schulz(fwad.make_dual(G, G))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            tg.newton_schulz(G, out=fwad.make_dual(G.bfloat16(), G.bfloat16()))


def test_a_second_derivative_raises_where_it_is_taken(card):
    H, W, t = card
    h, w = H.clone().requires_grad_(), W.clone().requires_grad_()
    plain = torch.autograd.grad(tg.linear_cross_entropy(h, w, t), (h, w))
    loss = tg.linear_cross_entropy(h, w, t)
    dH, dW = torch.autograd.grad(loss, (h, w), create_graph=True)
    # the first derivatives are there and are the same
    assert torch.equal(dH, plain[0]) and torch.equal(dW, plain[1])
    for term in (dH, dW):
        with pytest.raises(RuntimeError, match="once"):
            (loss + term.float().square().sum()).backward(retain_graph=True)
        assert h.grad is None and w.grad is None
    # what does not go through them is not held up
    (loss + dH.detach().float().square().sum()).backward()
    assert torch.equal(h.grad, plain[0]) and torch.equal(w.grad, plain[1])


def test_a_second_derivative_of_one_operand_raises(card):
    H, W, t = card
    h = H.clone().requires_grad_()
    dH, = torch.autograd.grad(tg.linear_cross_entropy(h, W, t), h, create_graph=True)
    with pytest.raises(RuntimeError, match="once"):
        dH.float().sum().backward()
    w = W.clone().requires_grad_()
    loss, lse = tg.linear_cross_entropy(H, w, t, return_lse=True)
    dW, = torch.autograd.grad(loss + lse.square().sum(), w, create_graph=True)
    with pytest.raises(RuntimeError, match="once"):
        dW.float().sum().backward()


def test_a_derivative_along_the_upstream_gradient_raises(card):
    H, W, t = card
    h = H.clone().requires_grad_()
    up = torch.ones((), requires_grad=True)
    dH, = torch.autograd.grad(tg.linear_cross_entropy(h, W, t) * up, h, create_graph=True)
    with pytest.raises(RuntimeError, match="once"):
        torch.autograd.grad(dH.float().sum(), up)


def test_hessian_products_raise(card):
    H, W, t = card
    with pytest.raises(RuntimeError, match="once"):
        torch.autograd.functional.hvp(lambda h: tg.linear_cross_entropy(h, W, t), H, torch.ones_like(H))


def traced(fn, *args):
    from torch.fx.experimental.proxy_tensor import make_fx

    yield "make_fx", lambda: make_fx(fn)(*args)
    yield "jit.trace", lambda: torch.jit.trace(fn, args, check_trace=False)
    yield "symbolic_trace", lambda: torch.fx.symbolic_trace(fn)


def test_tracing_is_refused(card):
    """A trace would hold the torch.empty of the result and not the call that fills it."""
    H, W, t = (x.as_subclass(torch.Tensor) for x in card)
    as_is = lambda x: x if isinstance(x, torch.fx.Proxy) else x.as_subclass(OnCard)  # noqa: E731
    cases = {
        "cross entropy": (lambda h, w: tg.linear_cross_entropy(as_is(h), as_is(w), as_is(t)), (H, W)),
        "update": (lambda g: tg.newton_schulz(as_is(g)), (H,)),
    }
    for what, (fn, args) in cases.items():
        for how, call in traced(fn, *args):
            with pytest.raises((NotImplementedError, TypeError, torch.fx.proxy.TraceError)) as e:
                call()
            if how != "symbolic_trace":  # its proxies stop at the first check of a type
                assert e.type is NotImplementedError and "traced" in str(e.value), (what, how, e.value)


def test_tracing_a_backward_pass_is_refused(card):
    from torch.fx.experimental.proxy_tensor import make_fx

    H, W, t = card
    h = H.clone().requires_grad_()
    loss = tg.linear_cross_entropy(h, W, t)
    with pytest.raises(NotImplementedError, match="traced"):
        make_fx(lambda up: torch.autograd.grad(loss, h, up)[0])(torch.ones(()))


@pytest.fixture
def update(monkeypatch):
    """newton_schulz as far as the library's entry point, which accepts the call."""
    from types import SimpleNamespace

    entry = SimpleNamespace(tg_newton_schulz_workspace_bytes=lambda *a: 0, tg_newton_schulz_bf16=lambda *a: 0,
                            tg_newton_schulz_f16=lambda *a: 0, tg_newton_schulz_f32=lambda *a: 0)
    monkeypatch.setattr(pr, "_lib", lambda: entry)
    monkeypatch.setattr(pr, "_ns_size", lambda *a: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    return lambda *shape: torch.ones(*shape, dtype=torch.bfloat16).as_subclass(OnCard)


def test_out_is_written_as_torch_sees_it(update):
    """A tensor saved for a backward pass must not be overwritten unnoticed."""
    out = update(3, 4)
    w = torch.ones(3, 4, dtype=torch.bfloat16, requires_grad=True)
    loss = (w * out).sum()
    before = out._version
    assert tg.newton_schulz(update(3, 4), out=out) is out and out._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    base = update(2, 3, 4)
    before = base._version
    tg.newton_schulz(update(3, 4), out=base[1])
    assert base._version > before  # through a view too
    same = update(3, 4)
    before = same._version
    tg.newton_schulz(same, out=same)
    assert same._version > before
    before = same._version
    tg.newton_schulz(same)
    assert same._version == before
    with torch.inference_mode():
        tg.newton_schulz(update(3, 4), out=update(3, 4))


def test_out_that_requires_grad_is_refused(update):
    leaf = update(3, 4).requires_grad_()
    for out in (leaf, leaf.view(3, 4), (leaf * 1.0)):
        with pytest.raises(ValueError, match="requires grad"):
            tg.newton_schulz(update(3, 4), out=out)
    with torch.no_grad():  # as an optimizer writes its parameters
        before = leaf._version
        assert tg.newton_schulz(update(3, 4), out=leaf) is leaf and leaf._version > before


def elements(t):
    """Byte addresses of every element of a 3-D tensor."""
    b, m, n = t.shape
    return {t.data_ptr() + t.element_size() * (i * t.stride(0) + j * t.stride(1) + k * t.stride(2)) + byte
            for i in range(b) for j in range(m) for k in range(n) for byte in range(t.element_size())}


def test_out_beside_g_in_one_buffer_is_taken(update):
    """Windows that share no element, whatever lies between their first and last."""
    room = update(6, 40)
    tg.newton_schulz(room[:, :12], out=room[:, 12:24])
    tg.newton_schulz(room[0::2, :12], out=room[1::2, :12])
    batch = update(3, 6, 40)
    tg.newton_schulz(batch[:, :, :7], out=batch[:, :, 7:14])
    tg.newton_schulz(batch[:, :3], out=batch[:, 3:])
    wide = torch.ones(4, 20).as_subclass(OnCard)  # fp32 on the left, the result on the right half of each row
    tg.newton_schulz(wide[:, :10], out=wide.view(torch.bfloat16)[:, 20:30])
    with pytest.raises(ValueError, match="overlaps G"):
        tg.newton_schulz(wide[:, :10], out=wide.view(torch.bfloat16)[:, 19:29])
    with pytest.raises(ValueError, match="overlaps G"):
        tg.newton_schulz(room[:, :12], out=room[:, 11:23])
    with pytest.raises(ValueError, match="overlaps G"):
        tg.newton_schulz(batch[:, :4], out=batch[:, 2:])


def test_overlap_is_found_as_by_listing_every_byte():
    import random

    rng = random.Random(0)
    room = torch.zeros(4096, dtype=torch.uint8)
    seen = {True: 0, False: 0}
    for _ in range(3000):
        b, m, n = rng.randint(1, 3), rng.randint(1, 4), rng.randint(1, 6)
        pair = []
        for dt in (rng.choice((torch.float32, torch.bfloat16)), torch.bfloat16):
            row = rng.randint(n, 14)
            stride = rng.choice((0, rng.randint(1, 3), rng.randint(n, 60)))
            pair.append(torch.as_strided(room.view(dt), (b, m, n), (stride, row, 1), rng.randint(0, 40)))
        want = bool(elements(pair[0]) & elements(pair[1]))
        assert pr._meet(*pair) == want, [(t.shape, t.stride(), t.dtype, t.storage_offset()) for t in pair]
        seen[want] += 1
    assert min(seen.values()) > 300


def test_in_place_is_not_compared_row_by_row(update, monkeypatch):
    monkeypatch.setattr(pr, "_meet", lambda *a: pytest.fail("compared"))
    G = update(2, 3, 4)
    tg.newton_schulz(G, out=G)
    tg.newton_schulz(G[1], out=G[1])
    tg.newton_schulz(G.half(), out=None)
    half = G.half()
    tg.newton_schulz(half, out=half.view(torch.bfloat16))
