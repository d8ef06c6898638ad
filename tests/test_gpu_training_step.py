"""The training operators as they are used together: a table looked up and tied to the
vocabulary projection, rows gathered by expert, the experts' products, the loss with
its gradients, the experts' Newton–Schulz update and AdamW for the table."""
import math

import pytest

torch = pytest.importorskip("torch")
tg = pytest.importorskip("dense_fp16_gemm_02_amd")

import training_oracle as oracle  # noqa: E402

pytestmark = pytest.mark.gpu
M, V, K, E, TOP = 192, 500, 128, 6, 2
HOW = dict(lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)


class Model:
    """Parameters in fp32 with bf16 copies that the model computes with."""

    def __init__(self, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.table32 = (0.1 * torch.randn(V, K, generator=gen)).cuda()
        self.gain32 = torch.ones(K).cuda()
        self.table = self.table32.bfloat16().requires_grad_()
        self.gain = self.gain32.bfloat16().requires_grad_()
        self.W = (torch.randn(E, K, K, generator=gen) / math.sqrt(K)).bfloat16().cuda().requires_grad_()
        self.moments = [[torch.zeros_like(t) for t in (self.table32, self.gain32)] for _ in range(2)]
        self.momentum = torch.zeros_like(self.W, requires_grad=False)
        self.step = torch.zeros((), dtype=torch.int64, device="cuda")


def batch(seed):
    gen = torch.Generator().manual_seed(100 + seed)
    tokens, target = torch.randint(0, V, (M,), generator=gen), torch.randint(0, V, (M,), generator=gen)
    target[::7] = -100
    expert = torch.stack([torch.randperm(E, generator=gen)[:TOP] for _ in range(M)])
    gate = torch.rand(M, TOP, generator=gen)
    return [t.cuda() for t in (tokens, target, expert, gate)]


def forward(table, gain, W, tokens, target, expert, gate, lookup, grouped, loss):
    order = torch.argsort(expert.flatten(), stable=True)
    ends = (expert.flatten()[:, None] == torch.arange(E, device=expert.device)).sum(0).cumsum(0)
    h = lookup(tokens, table)
    x = lookup(order // TOP, h)                      # a token's row once for each of its experts
    y = lookup(torch.argsort(order), grouped(x, W, ends)).view(M, TOP, K)
    z = (h + (gate[..., None] * y).sum(1).to(h.dtype)) * gain
    return loss(z, table, target)


def loss_of(model, data):
    return forward(model.table, model.gain, model.W, *data, tg.embedding, tg.grouped_linear, tg.linear_cross_entropy)


def plain(model, data):
    """The same in 64 bits."""
    def grouped(x, W, ends):
        e = torch.bucketize(torch.arange(x.shape[0], device=x.device), ends, right=True)
        return torch.stack([W[k] @ r for k, r in zip(e.tolist(), x)])

    leaves = [t.detach().double().requires_grad_() for t in (model.table, model.gain, model.W)]
    loss = forward(*leaves, *data[:3], data[3].double(), lambda t, w: w[t], grouped,
                   lambda z, w, t: torch.nn.functional.cross_entropy(z @ w.t(), t))
    return loss, torch.autograd.grad(loss, leaves)


def update(model, grads):
    dT, dg, dW = grads
    model.step += 1
    tg.adamw([model.table32, model.gain32], [dT, dg], *model.moments, model.step, copies=[model.table, model.gain], **HOW)
    with torch.no_grad():
        model.momentum.mul_(0.9).add_(dW)
        model.W.sub_(0.02 * tg.newton_schulz(model.momentum))


def test_gradients_of_a_step():
    model, data = Model(), batch(0)
    loss = loss_of(model, data)
    grads = torch.autograd.grad(loss, (model.table, model.gain, model.W))
    want_loss, want = plain(model, data)
    # each of some eight roundings on the way (Y, the sum, z, G; dz, dY, dX, dh) is at most 2^-8 of what it rounds
    assert abs(float(loss.detach()) - float(want_loss)) <= 8 * 2.0 ** -8 * abs(float(want_loss))
    for got, ref in zip(grads, want):
        assert float((got.double() - ref).norm()) <= 8 * 2.0 ** -8 * float(ref.norm())


def test_steps_update_every_parameter():
    model = Model()
    for k in range(3):
        before = [t.detach().clone() for t in (model.table32, model.gain32, model.W)]
        old = [[t.clone() for t in x] for x in model.moments]
        grads = torch.autograd.grad(loss_of(model, batch(k)), (model.table, model.gain, model.W))
        update(model, grads)
        for i, (p32, copy) in enumerate(((model.table32, model.table), (model.gain32, model.gain))):
            (p, m, v), (tp, tm, tv) = oracle.adamw(before[i], grads[i], old[0][i], old[1][i], k + 1, **HOW)
            assert ((p32.double() - p).abs() <= tp).all() and ((model.moments[0][i].double() - m).abs() <= tm).all()
            assert ((model.moments[1][i].double() - v).abs() <= tv).all() and torch.equal(copy, p32.bfloat16())
        assert not torch.equal(model.W, before[2]) and torch.isfinite(model.W).all()


def test_a_captured_step_does_what_an_eager_one_does():
    data = batch(0)
    eager, model = Model(), Model()

    def step(m, d):
        grads = torch.autograd.grad(loss_of(m, d), (m.table, m.gain, m.W))
        update(m, grads)
        return grads

    warm = Model()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(warm, data)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = step(model, data)
    for k in range(4):
        for slot, new in zip(data, batch(k)):
            slot.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        want = step(eager, batch(k))
        assert all(torch.equal(a, b) for a, b in zip(grads, want)), k
        assert all(torch.equal(a, b) for a, b in zip(model.moments[0] + model.moments[1], eager.moments[0] + eager.moments[1]))
        # the factors of the step are found on the device in either case
        assert torch.equal(model.table32, eager.table32) and torch.equal(model.W, eager.W), k


def test_moments_in_8_bits_train_the_same_table():
    model, data = Model(), batch(1)
    state = [[t] for t in tg.adamw_8bit_state(model.table32)]
    p8, p32 = [model.table32.clone()], [model.table32.clone()]
    moments = [[torch.zeros_like(p32[0])] for _ in range(2)]
    for k in range(1, 6):
        dT, = torch.autograd.grad(loss_of(model, batch(k)), (model.table,))
        tg.adamw_8bit(p8, [dT], *state, k, **HOW)
        tg.adamw(p32, [dT], *moments, k, **HOW)
    moved = (p32[0] - model.table32).norm()
    # the held moments are off by 2^-4 and carry a part of the errors before: 2·2^-4·(1 + β1 + …) of an update at most
    assert float((p8[0] - p32[0]).norm()) <= 2 * 2.0 ** -4 * 5 * float(moved)


def test_under_compile_the_calls_stay_between_the_compiled_parts():
    model, data = Model(), batch(2)

    @torch.compile(backend="eager")
    def compiled(table, gain, W):
        return forward(table * 1.0, gain, W, *data, tg.embedding, tg.grouped_linear, tg.linear_cross_entropy) * 2.0

    leaves = (model.table, model.gain, model.W)
    got = torch.autograd.grad(compiled(*leaves), leaves)
    want = torch.autograd.grad(2.0 * loss_of(model, data), leaves)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    p, g = [model.gain32.clone()], [model.gain.detach().float()]
    m, v = [torch.zeros_like(p[0])], [torch.zeros_like(p[0])]
    q, n, w = p[0].clone(), m[0].clone(), v[0].clone()
    torch.compile(lambda: tg.adamw(p, g, m, v, 1, **HOW), backend="eager")()
    tg.adamw([q], g, [n], [w], 1, **HOW)
    assert torch.equal(p[0], q) and torch.equal(m[0], n) and torch.equal(v[0], w)
