"""Newton–Schulz update of matrices with one element in each row of the short side.

All singular values are equal, X = x·P with one number x: the Gram matrix and its
square are diagonal, so the products' operands hold nothing but x itself (rounded to
binary16, in two parts for up to 64 rows) and all else is fp32.  x is followed in 64
bits with that rounding; the result has to be x rounded once, to bfloat16."""
import math
import sys

import pytest

torch = pytest.importorskip("torch")
tg = pytest.importorskip("dense_fp16_gemm_02_amd")

C = (3.4445, -4.7750, 2.0315)
E32 = 2.0 ** -24  # half a step of fp32
SIZES = [(8, 8), (64, 64), (2, 100), (64, 128), (60, 5000), (5000, 60),                       # two parts
         (100, 100), (128, 128), (100, 2100), (2100, 100), (192, 192), (300, 700), (700, 300), (1000, 1000)]


def chain(rows, steps=5):
    """x after the steps, a bound on the relative error of the kernels' x, and whether
    no rounding of it to binary16 could fall otherwise within that bound."""
    a, b, c = (float(torch.tensor(v, dtype=torch.float32)) for v in C)
    half = lambda v: float(torch.tensor(v, dtype=torch.float64).half())  # noqa: E731
    x, r, clear = 1.0 / math.sqrt(rows), 2 * E32, True
    for _ in range(steps):
        if rows > 64:
            h = half(x * 2.0 ** 14) / 2.0 ** 14  # what the Gram product sees
            clear = clear and half(x * (1 - r) * 2.0 ** 14) == half(x * (1 + r) * 2.0 ** 14)
            d, rd = h * h, 2 * E32
        else:
            d, rd = x * x, 3 * 2.0 ** -22  # the two parts' 2^-22, twice, and their low parts' product
            r *= abs((a + 3 * b * d + 5 * c * d * d) / (a + b * d + c * d * d))  # x's own error, through both factors
        e = b * d + c * d * d
        # the roundings of d, of e's four operations and of (a + e)·x with e's own error
        re = rd * (abs(b) * d + 2 * c * d * d) + 4 * E32 * (abs(b) * d + c * d * d)
        r = r + (re + 2 * E32 * (a + abs(b) * d + c * d * d)) / abs(a + e)
        x = (a + e) * x
    return x, r, clear


@pytest.mark.parametrize("m,n", SIZES)
def test_the_sizes_leave_no_doubt(m, n):
    """(On the CPU.)  No rounding of these sizes' chains is close: neither an operand's
    nor the result's."""
    x, r, clear = chain(min(m, n))
    bf16 = lambda v: float(torch.tensor(v, dtype=torch.float64).bfloat16())  # noqa: E731
    assert clear and r < 2.0 ** -14 and bf16(x * (1 - r)) == bf16(x * (1 + r)), (m, n, x, r)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", SIZES)
def test_the_result_is_rounded_once(m, n):
    print("[gpu-case]", m, n, tg.tg_newton_schulz_plan(1, m, n), file=sys.stderr, flush=True)
    s = min(m, n)
    gen = torch.Generator().manual_seed(m + n)
    at = torch.arange(s), torch.randperm(max(m, n), generator=gen)[:s]
    if m > n:
        at = at[1], at[0]
    G = torch.zeros(m, n)
    G[at] = torch.where(torch.rand(s, generator=gen) < 0.5, -3.0, 3.0)
    x, _, _ = chain(s)
    want = (G.sign().double() * x).bfloat16()
    for dt in (torch.float32, torch.float16, torch.bfloat16):
        O = tg.newton_schulz(G.to(dt).cuda(), eps=0.0)
        assert torch.equal(O.cpu(), want), (dt, x, O.abs().max())
