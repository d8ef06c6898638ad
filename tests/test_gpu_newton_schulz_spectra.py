"""Newton–Schulz update of matrices whose singular values are far apart.

A direction with a small part of the norm is amplified by up to 485 in five steps,
and what an operand's rounding puts there with it."""
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
tg = pytest.importorskip("dense_fp16_gemm_02_amd")

import projection_oracle as po  # noqa: E402

F32 = torch.float32


def spectrum(m, n, values, gen):
    """A matrix with these singular values and random singular vectors."""
    s = min(m, n)
    U, _ = torch.linalg.qr(torch.randn(m, s, generator=gen, dtype=torch.float64))
    V, _ = torch.linalg.qr(torch.randn(n, s, generator=gen, dtype=torch.float64))
    return (U * values) @ V.t().contiguous()


def matrix(kind, m, n, seed=0):
    gen = torch.Generator().manual_seed(1009 * m + n + seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    s = min(m, n)
    wide = (s, max(m, n))
    if kind == "half at 1e-2":
        sv = torch.full((s,), 1e-2, dtype=torch.float64)
        sv[: (s + 1) // 2] = 1.0
        return spectrum(m, n, sv, gen)
    if kind == "an eighth above 1e-3":
        sv = torch.full((s,), 1e-3, dtype=torch.float64)
        sv[: (s + 7) // 8] = 1.0
        return spectrum(m, n, sv, gen)
    if kind == "1 to 1e-2":
        return spectrum(m, n, torch.logspace(0, -2, s, dtype=torch.float64), gen)
    if kind == "rank one":
        return rnd(m, 1) * rnd(1, n)
    if kind == "rank four":
        return rnd(m, 4) @ rnd(4, n)
    if kind == "parallel to 1e-2":
        G = rnd(1, wide[1]) + 1e-2 * rnd(*wide)
    elif kind == "parallel to 1e-3":
        G = rnd(1, wide[1]) + 1e-3 * rnd(*wide)
    elif kind == "equal rows":
        G = rnd(1, wide[1]).expand(*wide)
    elif kind == "two parallel rows":
        G = torch.zeros(*wide, dtype=torch.float64)
        G[:2] = rnd(1, wide[1]) + 1e-2 * rnd(2, wide[1])[:s]
    else:
        raise ValueError(kind)
    return G if m <= n else G.t()


KINDS = ["half at 1e-2", "an eighth above 1e-3", "1 to 1e-2", "rank one", "rank four", "parallel to 1e-2",
         "parallel to 1e-3", "equal rows", "two parallel rows"]


def off(O, G):
    want = po.newton_schulz(G)
    return (O.double() - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)


# a short side of up to 64: in the one-workgroup forms with the long side in and
# beyond 64 columns, and in strips
@pytest.mark.parametrize("m,n", [(2, 40), (2, 100), (100, 2), (4, 128), (16, 100), (64, 128), (128, 64), (33, 65), (65, 3),
                                 (1, 65), (128, 17), (64, 64), (2, 129), (129, 4), (64, 700)])
def test_short_sides_of_up_to_64_hold_any_spectrum(m, n):
    """Within 2^-8 in the 2-norm, the half step of the result's type.  The result's
    own rounding is 2^-9.2 of it root mean square (at most 2^-8); operands in two parts
    err by 2^-22 each, which amplified 485 times, in each of five steps' products, stay
    below 2^-10 in all."""
    for kind in KINDS:
        print("[gpu-case]", m, n, kind, tg.tg_newton_schulz_plan(2, m, n), file=sys.stderr, flush=True)
        G = torch.stack([matrix(kind, m, n, seed) for seed in (0, 1)]).to(F32).cuda()
        e = off(tg.newton_schulz(G), G)
        assert bool((e <= 2.0 ** -8).all()), (kind, e)
