"""What the backward pass of linear_cross_entropy makes of saved tensors that come back from
hooks (offloading, packing): the same values, in memory of other strides.  On the CPU: the
library's call is replaced by torch on ``as_strided`` views with the strides that the call was
given, which raises where those leave the operand's memory."""
import pytest

torch = pytest.importorskip("torch")
tg = pytest.importorskip("dense_fp16_gemm_02_amd")

from dense_fp16_gemm_02_amd import projection as pr  # noqa: E402

M, V, K = 6, 9, 16


class OnCard(torch.Tensor):
    is_cuda = True


def plain(t):
    return t.detach().as_subclass(torch.Tensor)


class Held:
    """Tensors by address, alive, so that an address is one tensor's."""

    def __init__(self):
        self.kept = []

    def keep(self, t):
        self.kept.append(t)
        return t

    def window(self, at, shape, strides):
        t = next(plain(t) for t in self.kept if t.data_ptr() == at)
        return torch.as_strided(t, shape, strides, t.storage_offset()).double()


def columns(t):
    return t.clone() if t.dim() < 2 else t.t().contiguous().t()


def spread(t):
    out = torch.zeros(*t.shape, 2, dtype=t.dtype)
    out[..., 0] = t
    return out[..., 0]


def padded(t):
    if t.dim() < 2:
        return spread(t)
    out = torch.full((t.shape[0], t.shape[1] + 16), 9, dtype=t.dtype)
    out[:, 3:3 + t.shape[1]] = t
    return out[:, 3:3 + t.shape[1]]


def gradients(monkeypatch, back, wide=False):
    """dH and dW through hooks that bring saved tensors back by ``back``, and what they should be."""
    gen = torch.Generator().manual_seed(0)
    h, w, target = torch.randn(M, K, generator=gen).half(), torch.randn(V, K, generator=gen).half(), torch.arange(M)
    held, contiguous = Held(), torch.Tensor.contiguous

    def forward(H, W, target, ignore_index, reduction, want_lse):
        z = plain(H).double() @ plain(W).double().t()
        lse = torch.logsumexp(z, 1)
        return (lse - z.gather(1, plain(target)[:, None])[:, 0]).mean().float(), lse.float()

    def call(backward, H, W, lead, tail, args):
        at, lse_at, dloss, dlse, dH, dW = lead
        strides = pr._row_stride(H, "H", K), pr._row_stride(W, "W", K)
        x, y = held.window(H.data_ptr(), (M, K), (strides[0], 1)), held.window(W.data_ptr(), (V, K), (strides[1], 1))
        t, lse = held.window(at, (M,), (1,)).long(), held.window(lse_at, (M,), (1,))
        assert H.dtype == W.dtype == torch.half
        results.append((x, y, t, lse))

    results = []
    monkeypatch.setattr(pr, "_forward", forward)
    monkeypatch.setattr(pr, "_xent_call", call)
    if wide:
        h = padded(h)
    H, W = (t.as_subclass(OnCard).requires_grad_() for t in (h, w))
    with torch.autograd.graph.saved_tensors_hooks(plain, lambda t: held.keep(back(t).as_subclass(OnCard))):
        loss = tg.linear_cross_entropy(H, W, target.as_subclass(OnCard))
    monkeypatch.setattr(torch.Tensor, "contiguous", lambda self, *how: held.keep(contiguous(self, *how)))
    torch.autograd.grad(loss, (H, W))
    (x, y, t, lse), = results
    return all(torch.equal(a, b) for a, b in ((x, h.double()), (y, w.double()), (t, target))) and torch.allclose(
        lse, torch.logsumexp(h.double() @ w.double().t(), 1), rtol=2.0 ** -23)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("back", [lambda t: t, lambda t: t.clone(memory_format=torch.contiguous_format), columns, spread, padded],
                         ids=["as saved", "contiguous", "columns", "spread", "padded"])
def test_operands_by_saved_layout(monkeypatch, back, wide):
    assert gradients(monkeypatch, back, wide)


@pytest.mark.parametrize("back", [
    lambda t: t.double() if t.dtype == torch.half and t.shape[0] == V else t, lambda t: t.int() if t.dtype == torch.int64 else t,
    lambda t: t[:-1] if t.shape == (M,) else t, lambda t: t[:, :-1] if t.dim() == 2 else t,
    lambda t: t.double() if t.dtype == torch.float32 else t], ids=["W's type", "target's type", "number", "width", "lse's type"])
def test_operands_that_are_others_are_refused(monkeypatch, back):
    with pytest.raises((TypeError, ValueError)):
        gradients(monkeypatch, back)
