"""Newton–Schulz update of matrices whose singular values are far apart.

A direction with a small part of the norm is amplified by up to 485 in five steps,
and what an operand's rounding puts there with it."""
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
tg = pytest.importorskip("dense_fp16_gemm_02_amd")

import projection_model as pm  # noqa: E402
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


def model_off(G):
    want = po.newton_schulz(G)
    return (pm.newton_schulz(G) - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)


# the largest error that include/tg_ortho.h gives for a short side above 64
MEASURED = {"half at 1e-2": 4e-3, "an eighth above 1e-3": 4e-3, "1 to 1e-2": 2e-3, "rank one": 1.2e-2, "rank four": 5e-3,
            "parallel to 1e-2": 2e-3, "parallel to 1e-3": 3e-3, "equal rows": 5e-3, "two parallel rows": 2e-2}


@pytest.mark.parametrize("m,n", [(65, 70), (65, 130), (130, 65), (100, 100), (128, 700), (700, 128), (100, 2500), (2500, 100),
                                 (200, 300), (515, 513), (300, 5000), (5000, 300), (512, 2048), (1025, 1500)])
def test_longer_short_sides_err_by_their_operands_roundings(m, n):
    """One part above 64 rows: the error is that of the same roundings in 64 bits.  The
    kernels' fp32 sums of l terms err by some l^1/2·2^-24, which moves less than one
    operand in 2^6 across a rounding (a step of 2^-11), by a step, 3.5 times the root
    mean square of a rounding: a change of the error by less than 3.5·2^-3, a half."""
    for kind in KINDS:
        print("[gpu-case]", m, n, kind, tg.tg_newton_schulz_plan(2, m, n), file=sys.stderr, flush=True)
        G = torch.stack([matrix(kind, m, n, seed) for seed in (0, 1)]).to(F32).cuda()
        e, model = off(tg.newton_schulz(G), G), model_off(G)
        print("[off]", e.tolist(), model.tolist(), file=sys.stderr, flush=True)
        assert bool((e <= 1.5 * model).all()), (kind, e, model)
        assert bool((e <= MEASURED[kind]).all()), (kind, e)


@pytest.mark.parametrize("rows,most", [(1, 2e-3), (2, 6e-2), (4, 6e-2), (16, 4e-2), (64, 1.2e-2)])
def test_all_of_a_matrix_in_a_few_rows(rows, most):
    """The same where the other rows are zero: what the header gives for them."""
    for m, n in ((65, 130), (300, 1000), (1000, 300)):
        for kind in ("rank one", "parallel to 1e-2", "parallel to 1e-3"):
            print("[gpu-case]", m, n, rows, kind, file=sys.stderr, flush=True)
            s, long = min(m, n), max(m, n)
            G = torch.zeros(2, s, long, dtype=torch.float64)
            for i in range(2):
                G[i, :rows] = matrix(kind, rows, long, i)
            G = (G if m <= n else G.transpose(1, 2)).to(F32).contiguous().cuda()
            e, model = off(tg.newton_schulz(G), G), model_off(G)
            print("[off]", e.tolist(), model.tolist(), file=sys.stderr, flush=True)
            assert bool((e <= 1.5 * model).all()), (kind, e, model)
            assert bool((e <= most).all()), (kind, e)
