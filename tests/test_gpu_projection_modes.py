"""The projection operators under torch.compile (the call runs as it is, between the
compiled parts, and gives what it gives without) and create_graph.  (What is refused is in
test_projection_modes_cpu.py.)"""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
tg = pytest.importorskip("dense_fp16_gemm_02_amd")


def operands():
    gen = torch.Generator(device="cuda").manual_seed(0)
    H = torch.randn(60, 136, generator=gen, device="cuda").half()
    W = torch.randn(300, 136, generator=gen, device="cuda").half()
    return H, W, torch.randint(0, 300, (60,), generator=gen, device="cuda")


@pytest.mark.parametrize("backend", ["eager", "aot_eager"])
@pytest.mark.parametrize("grad", [False, True])
def test_compiled_cross_entropy(backend, grad):
    torch._dynamo.reset()
    H, W, t = operands()

    def f(h, w):
        loss, lse = tg.linear_cross_entropy(h * 0.5, w, t, return_lse=True)
        return 2.0 * loss + 1e-4 * lse.square().sum()

    compiled = torch.compile(f, backend=backend)
    for scale in (1.0, 2.0):
        h, w = (H * scale).requires_grad_(grad), W.clone().requires_grad_(grad)
        want, got = f(h, w), compiled(h, w)
        assert torch.equal(got, want)
        if grad:
            for a, b in zip(torch.autograd.grad(got, (h, w)), torch.autograd.grad(want, (h, w))):
                assert torch.equal(a, b)


@pytest.mark.parametrize("backend", ["eager", "aot_eager"])
def test_compiled_update(backend):
    torch._dynamo.reset()
    H, W, _ = operands()

    def f(g, out):
        tg.newton_schulz(g * 2.0, steps=3, out=out)
        return out.float() + tg.newton_schulz(g, coefficients=(1.5, -0.5, 0.0)).float()

    compiled = torch.compile(f, backend=backend)
    for scale in (1.0, 3.0):
        g = W * scale
        a, b = (torch.empty_like(g, dtype=torch.bfloat16) for _ in range(2))
        assert torch.equal(compiled(g, a), f(g, b)) and torch.equal(a, b)


def test_first_derivatives_under_create_graph_and_no_second_ones():
    H, W, t = operands()
    h, w = H.requires_grad_(), W.requires_grad_()
    plain = torch.autograd.grad(tg.linear_cross_entropy(h, w, t), (h, w))
    loss, lse = tg.linear_cross_entropy(h, w, t, return_lse=True)
    dH, dW = torch.autograd.grad(loss, (h, w), create_graph=True)
    assert torch.equal(dH, plain[0]) and torch.equal(dW, plain[1])
    for term in (dH, dW):
        with pytest.raises(RuntimeError, match="once"):
            torch.autograd.grad(term.float().square().sum(), (h, w), retain_graph=True)
    # the update written over a tensor that a graph holds
    out = torch.zeros_like(W, dtype=torch.bfloat16)
    held = (torch.ones_like(out, requires_grad=True) * out).sum()
    assert torch.equal(tg.newton_schulz(W.detach(), out=out), tg.newton_schulz(W.detach()))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        held.backward()


@pytest.mark.parametrize("pin", [False, True])
def test_saved_tensors_that_were_offloaded(pin):
    """torch.autograd.graph.save_on_cpu brings a window back without what lay between its rows."""
    H, W, t = operands()
    wide = torch.full((60, 400), float("nan"), dtype=H.dtype, device="cuda")
    wide[:, 136:272] = H
    h, w, spread = wide[:, 136:272].requires_grad_(), W.requires_grad_(), torch.zeros(60, 2, dtype=t.dtype, device="cuda")
    spread[:, 1] = t
    want = torch.autograd.grad(tg.linear_cross_entropy(h, w, t), (h, w))
    with torch.autograd.graph.save_on_cpu(pin_memory=pin):
        loss = tg.linear_cross_entropy(h, w, spread[:, 1])
    assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(loss, (h, w)), want))
