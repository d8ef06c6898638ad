"""Every kernel the projection operators' plans choose, at ragged sizes, against the
64-bit forms (projection_oracle) within the bounds of the roundings made."""
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
tg = pytest.importorskip("dense_fp16_gemm_02_amd")

import projection_oracle as po  # noqa: E402
from projection_cases import NEWTON_SCHULZ  # noqa: E402
from test_gpu_newton_schulz import BF16, F32, matrix, norm_check  # noqa: E402


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
