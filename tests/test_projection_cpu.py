"""Host-side checks of the projection operators that need no GPU: refusals,
workspace sizes, plans, and a C99 caller of the headers."""
import itertools
import os
import shutil
import subprocess

import pytest

tg = pytest.importorskip("dense_fp16_gemm_02_amd")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20          # 16-byte aligned, never dereferenced
BIG = 1 << 62
LIM = 1 << 31


def fwd(H=A, W=A, t=A, loss=A, lse=A, M=4, V=8, K=16, ldh=16, ldw=16, ignore=-100, red=2, ws=A, size=BIG,
        fn=None):
    return (fn or tg.tg_xent_f16)(H, W, t, loss, lse, M, V, K, ldh, ldw, ignore, red, ws, size, None)


def bwd(H=A, W=A, t=A, lse=A, dloss=A, dlse=None, dH=A, dW=A, M=4, V=8, K=16, ldh=16, ldw=16, lddh=16, lddw=16,
        ignore=-100, red=2, ws=A, size=BIG, fn=None):
    return (fn or tg.tg_xent_bwd_bf16)(H, W, t, lse, dloss, dlse, dH, dW, M, V, K, ldh, ldw, lddh, lddw, ignore, red,
                                       ws, size, None)


def ns(G=A, O=A, batch=1, rows=300, cols=200, ldg=200, gs=60000, ldo=200, os_=60000, steps=5, co=None, eps=1e-7, ws=A,
       size=BIG, fn=None):
    return (fn or tg.tg_newton_schulz_f32)(G, O, batch, rows, cols, ldg, gs, ldo, os_, steps, co, eps, ws, size, None)


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(V=-1), dict(K=-1), dict(ldh=15), dict(ldw=15), dict(H=None), dict(W=None), dict(t=None),
    dict(loss=None), dict(V=0), dict(K=0, ldh=0, ldw=0), dict(red=3), dict(red=-1), dict(ws=None), dict(ws=A + 8),
    dict(size=0), dict(M=0, loss=None),
])
def test_forward_refuses(kw):
    for fn in (tg.tg_xent_f16, tg.tg_xent_bf16):
        assert fwd(fn=fn, **kw) == tg.TG_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(ldh=15), dict(ldw=15), dict(lddh=15), dict(lddw=15), dict(lse=None), dict(dloss=None),
    dict(t=None), dict(V=0), dict(red=7), dict(ws=None), dict(ws=A + 16), dict(size=100),
])
def test_backward_refuses(kw):
    for fn in (tg.tg_xent_bwd_f16, tg.tg_xent_bwd_bf16):
        assert bwd(fn=fn, **kw) == tg.TG_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(M=LIM), dict(V=LIM), dict(K=LIM, ldh=LIM, ldw=LIM), dict(ldh=LIM), dict(ldw=LIM),
                                dict(M=LIM - 5000, V=LIM - 5000)])
def test_too_large_refused(kw):
    assert fwd(**kw) == tg.TG_ERR_TOO_LARGE
    if kw.get("K", 0) != LIM:
        assert bwd(**kw) == tg.TG_ERR_TOO_LARGE
    assert bwd(lddh=LIM) == tg.TG_ERR_TOO_LARGE


@pytest.mark.parametrize("kw", [
    dict(M=1 << 25), dict(V=1 << 30), dict(K=(1 << 21) + 1, ldh=1 << 22, ldw=1 << 22),
    dict(M=(1 << 25) - 1, V=1 << 29),  # launches of 2^32 threads and more
])
def test_sizes_beyond_the_kernels_offsets_are_refused(kw):
    assert fwd(**kw) == tg.TG_ERR_TOO_LARGE
    sizes = {**dict(M=5, V=100, K=16, ldh=4096, ldw=4096), **kw}
    args = (A, A, sizes["M"], sizes["V"], sizes["K"], sizes["ldh"], sizes["ldw"])
    assert tg.tg_xent_workspace_bytes(*args) == -1
    if kw.get("M") != (1 << 25) - 1:  # the backward pass takes the vocabulary in pieces
        assert bwd(**kw) == tg.TG_ERR_TOO_LARGE and tg.tg_xent_bwd_workspace_bytes(*args) == -1


def test_largest_sizes_are_planned():
    for args in ((A, A, 1, (1 << 30) - 128, 64, 64, 64), (A, A, 4, 1000, 1 << 21, 1 << 21, 1 << 21),
                 (A + 2, A + 2, 1 << 20, 131072, 4096, 4097, 4097)):
        for fn in (tg.tg_xent_workspace_bytes, tg.tg_xent_bwd_workspace_bytes):
            assert fn(*args) > 0
    # a piece's columns stay few enough for 32-bit offsets inside a tile, however few the tokens
    status, name, pieces = tg.tg_xent_plan(A, A, 1, (1 << 30) - 128, 64, 64, 64, 1)
    assert status == tg.TG_OK and pieces >= ((1 << 30) - 128) / 2 ** 20
    assert tg.tg_newton_schulz_workspace_bytes(1, 64, (1 << 21) - 65) > 0
    assert tg.tg_newton_schulz_workspace_bytes((1 << 23) - 1, 8, 8) == 0  # one workgroup each
    assert tg.tg_newton_schulz_workspace_bytes(1 << 23, 8, 8) == -1


def test_workspace_one_byte_short_is_refused():
    n = tg.tg_xent_workspace_bytes(A, A, 100, 1000, 64, 64, 64)
    b = tg.tg_xent_bwd_workspace_bytes(A, A, 100, 1000, 64, 64, 64)
    assert n > 0 and b > n and n % 256 == 0 and b % 256 == 0
    assert fwd(M=100, V=1000, K=64, ldh=64, ldw=64, size=n - 1) == tg.TG_ERR_INVALID_ARG
    assert bwd(M=100, V=1000, K=64, ldh=64, ldw=64, lddh=64, lddw=64, size=b - 1) == tg.TG_ERR_INVALID_ARG
    w = tg.tg_newton_schulz_workspace_bytes(2, 300, 200)
    assert w > 0 and ns(batch=2, size=w - 1) == tg.TG_ERR_INVALID_ARG


def test_no_tokens_needs_no_workspace():
    assert tg.tg_xent_workspace_bytes(A, A, 0, 8, 16, 16, 16) == 0
    assert fwd(M=0, red=0, ws=None, size=0) == tg.TG_OK
    assert bwd(M=0, dW=None, ws=None, size=0) == tg.TG_OK
    assert bwd(dH=None, dW=None) == tg.TG_OK  # nothing asked for
    assert tg.tg_xent_workspace_bytes(A, A, -1, 8, 16, 16, 16) == -1


def test_logits_are_not_kept():
    """Workspaces stay far below the logits: 4 bytes each for the forward pass's
    pairs per 256 columns, and a bounded piece of G for the backward pass."""
    M, V, K = 8192, 131072, 4096
    logits = 4 * M * V
    assert tg.tg_xent_workspace_bytes(A, A, M, V, K, K, K) < logits / 20
    assert tg.tg_xent_bwd_workspace_bytes(A, A, M, V, K, K, K) < logits / 3
    st, name, pieces = tg.tg_xent_plan(A, A, M, V, K, K, K, True)
    assert st == tg.TG_OK and pieces > 1 and "grad_256x256" in name


@pytest.mark.parametrize("args,backward,part", [
    ((A, A, 8192, 131072, 4096, 4096, 4096), False, "gather stats_256x256"),
    ((A, A, 64, 28672, 8192, 8192, 8192), False, "stats_64x128"),
    ((A, A, 1, 28672, 8192, 8192, 8192), False, "stats_64x128"),
    ((A, A, 1000, 1000, 1000, 1000, 1000), False, "stats_64x64"),
    ((A, A, 333, 50001, 1000, 1000, 1000), True, "grad_128x128"),
    ((A, A, 100, 50001, 4096, 4096, 4096), True, "grad_128x128_stream"),
    ((A, A, 250, 131072, 2048, 2048, 2048), False, "stats_256x256_stream"),
    ((A, A, 100, 50001, 1024, 1024, 1024), True, "grad_128x128 "),
    ((A + 2, A, 16, 100, 64, 64, 64), False, "gather"),      # H not aligned
    ((A, A + 2, 16, 100, 64, 64, 64), False, "pack"),        # W not aligned
    ((A, A, 16, 100, 63, 64, 64), True, "pack"),             # K not a multiple of 8
    ((A, A, 16, 100, 64, 64, 65), True, "pack"),             # ldw not a multiple of 8
])
def test_plan_names(args, backward, part):
    st, name, _ = tg.tg_xent_plan(*args, backward)
    assert st == tg.TG_OK and part in name, name


def test_every_tile_class_is_reached():
    seen = set()
    for M, V, K in itertools.product((1, 64, 65, 200, 333, 576, 1000, 1500, 3000, 8192),
                                     (1000, 2000, 5000, 16000, 50001, 131072), (64, 192, 512, 1000, 4096)):
        seen.update(tg.tg_xent_plan(A, A, M, V, K, K + 8, K + 8, True)[1].split())
    for what, classes in (("grad", ("256x256", "192x192", "128x128", "64x64", "64x128")),
                          ("dh", ("256x256", "128x128", "64x64", "64x128")),
                          ("dw", ("256x256", "192x192", "128x128", "64x64"))):
        for c in classes:
            assert f"{what}_{c}" in seen, (what, c)
    seen = set()
    for b, m, n in itertools.product((1, 2, 8, 64), (64, 128, 129, 700, 1000, 2048, 4096, 9000), (64, 200, 1000, 4096, 9000)):
        st, name = tg.tg_newton_schulz_plan(b, m, n)
        assert st == tg.TG_OK
        seen.update(name.split())
    for what in ("gram", "square", "update"):
        for c in ("256x256", "192x192", "128x128", "64x64"):
            assert f"{what}_{c}" in seen, (what, c)
    assert {"gram_64x64_split", "gram_128x128_split"} <= seen
    assert {"small_64", "tall", "wide"} <= seen and tg.tg_newton_schulz_plan(1, 65, 3)[1] == "small_128"
    assert {"thin_64", "thin_128"} <= seen


@pytest.mark.parametrize("kw", [
    dict(batch=-1), dict(rows=-1), dict(cols=-1), dict(ldg=199), dict(ldo=199), dict(steps=-1), dict(steps=33),
    dict(eps=-1e-3), dict(eps=float("nan")), dict(G=None), dict(O=None), dict(ws=None), dict(ws=A + 128),
    dict(batch=2, os_=59999), dict(gs=-1),
])
def test_newton_schulz_refuses(kw):
    for fn in (tg.tg_newton_schulz_f32, tg.tg_newton_schulz_f16, tg.tg_newton_schulz_bf16):
        assert ns(fn=fn, **kw) == tg.TG_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(rows=1 << 21, gs=0), dict(cols=1 << 21, ldg=1 << 21, ldo=1 << 21),
                                dict(batch=LIM), dict(batch=1 << 30, rows=4096)])
def test_newton_schulz_too_large(kw):
    assert ns(**kw) == tg.TG_ERR_TOO_LARGE


def test_newton_schulz_empty_is_a_no_op():
    for kw in (dict(batch=0), dict(rows=0), dict(cols=0)):
        assert ns(G=None, O=None, ws=None, size=0, **kw) == tg.TG_OK
    assert tg.tg_newton_schulz_workspace_bytes(3, 128, 128) == 0


def test_wrappers_refuse_tensors_they_cannot_take():
    torch = pytest.importorskip("torch")
    H, W, t = torch.zeros(4, 16).half(), torch.zeros(8, 16).half(), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):
        tg.linear_cross_entropy(H, W, t)
    with pytest.raises(TypeError):
        tg.linear_cross_entropy(H.float(), W.float(), t)
    with pytest.raises(TypeError):
        tg.linear_cross_entropy(H, W.bfloat16(), t)
    with pytest.raises(TypeError):
        tg.linear_cross_entropy(H, W, t.int())
    with pytest.raises(ValueError, match="GPU"):
        tg.newton_schulz(torch.zeros(4, 4))
    with pytest.raises(TypeError):
        tg.newton_schulz(torch.zeros(4, 4, dtype=torch.float64))


PROGRAM = r"""
#include <stdint.h>
#include <stdio.h>
#include <string.h>
#include "tg_gemm.h"
#include "tg_xent.h"
#include "tg_ortho.h"

int main(void)
{
    const void *H = (const void *)(uintptr_t)0x100000, *W = (const void *)(uintptr_t)0x200000;
    char name[128];
    int64_t pieces = 0;
    int fails = 0;
    if (tg_xent_plan(H, W, 64, 28672, 8192, 8192, 8192, 0, name, sizeof name, &pieces) != TG_OK) ++fails;
    if (strcmp(name, "stats_64x128") != 0 || pieces != 1) ++fails;
    if (tg_xent_bf16(H, W, 0, 0, 0, 4, 8, 16, 16, 16, -100, TG_XENT_MEAN, 0, 0, 0) != TG_ERR_INVALID_ARG) ++fails;
    if (tg_newton_schulz_plan(1, 64, 64, name, 4) != TG_OK || strcmp(name, "sma") != 0) ++fails;
    if (tg_newton_schulz_bf16(H, 0, 1, 8, 8, 8, 64, 8, 64, TG_NS_MAX_STEPS + 1, 0, 0.0f, 0, 0, 0) != TG_ERR_INVALID_ARG)
        ++fails;
    printf("fails %d\n", fails);
    return fails;
}
"""


def test_c99_caller(tmp_path):
    cc = shutil.which("gcc")
    if not cc:
        pytest.skip("gcc not available")
    src, exe = tmp_path / "p.c", tmp_path / "p"
    src.write_text(PROGRAM)
    lib = os.path.dirname(tg.lib_path())
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", f"-I{os.path.join(ROOT, 'include')}",
                    str(src), "-o", str(exe), tg.lib_path(), f"-Wl,-rpath,{lib}"], check=True)
    p = subprocess.run([str(exe)], capture_output=True, text=True)
    assert p.returncode == 0, p.stdout
