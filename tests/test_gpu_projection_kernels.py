"""Every kernel the projection operators' plans choose, at ragged sizes, against the
64-bit forms (projection_oracle) within the bounds of the roundings made."""
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
tg = pytest.importorskip("dense_fp16_gemm_02_amd")

import projection_oracle as po  # noqa: E402
from projection_cases import NEWTON_SCHULZ, XENT  # noqa: E402
from test_gpu_newton_schulz import BF16, F32, matrix, norm_check  # noqa: E402
from test_gpu_xent import IGNORE, check, inputs  # noqa: E402


def say(*a):
    print("[gpu-case]", *a, file=sys.stderr, flush=True)


@pytest.mark.parametrize("b,m,n,plan", NEWTON_SCHULZ)
def test_newton_schulz(b, m, n, plan):
    say(b, m, n, plan)
    assert tg.tg_newton_schulz_plan(b, m, n) == (tg.TG_OK, plan)
    G = matrix(b, m, n, F32, seed=40)
    want = tg.newton_schulz(G)
    norm_check(want, G)
    # the last step's stores beside and between rows that are not aligned
    room = torch.full((b, m + 1, n + 5), 9.0, dtype=BF16, device="cuda")
    out = room[:, 1:, 3:3 + n]
    tg.newton_schulz(G, out=out)
    assert torch.equal(out, want)
    out.fill_(9.0)
    assert bool((room == 9.0).all())
    # one step, each element within the bound of its roundings
    G = matrix(b, m, n, BF16, seed=41, kind="spikes")
    O = tg.newton_schulz(G, steps=1)
    exact, tol = po.newton_schulz_one_step_bound(G)
    bad = ~((O.double() - exact).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), float(((O.double() - exact).abs() / tol).max()))


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("M,V,K,fwd,fwd_pieces,bwd,bwd_pieces", XENT)
def test_cross_entropy(M, V, K, fwd, fwd_pieces, bwd, bwd_pieces, dt):
    say(M, V, K, dt, fwd, fwd_pieces, bwd, bwd_pieces)
    H, W, t = inputs(M, V, K, dt, seed=42, ignored=0.1)
    for backward, plan in enumerate(((fwd, fwd_pieces), (bwd, bwd_pieces))):
        assert tg.tg_xent_plan(H, W, M, V, K, K, K, backward) == (tg.TG_OK, *plan)
    # targets in every piece, its first and last entry among them
    at = torch.linspace(0, V - 1, M, dtype=torch.float64, device="cuda").long()
    t[::3] = at[::3]
    t[0], t[M - 1], t[M // 2] = 0, V - 1, IGNORE
    check(H, W, t)
    torch.cuda.empty_cache()
