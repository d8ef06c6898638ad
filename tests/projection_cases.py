"""Sizes at which the projection operators take each of their kernels, with the plan
each is there for: ragged in every dimension, as small as the kernel's choice
allows.  What the other GPU tests' sizes reach is not repeated here; together they
reach every kernel (test_projection_plan_cpu.py)."""
import dense_fp16_gemm_02_amd as tg

ALIGNED = 1 << 20  # an address that is a multiple of 16, never dereferenced

# batch, rows, cols, plan
NEWTON_SCHULZ = [
    (26, 4659, 209, "tall gram_128x128_split square_64x64 update_128x128"),
    (37, 551, 539, "tall gram_192x192 square_192x192 update_128x128"),
    (52, 1333, 387, "tall gram_256x256 square_128x128 update_128x128"),
    (18, 1801, 131, "tall gram_64x64 square_64x64 update_192x192"),
    (21, 949, 597, "tall gram_128x128 square_128x128 update_256x256"),
    (53, 391, 1361, "wide gram_256x256 square_128x128 update_128x128"),
    (5, 131, 6599, "wide gram_64x64_split square_64x64 update_192x192"),
    (37, 701, 651, "tall gram_256x256 square_256x256 update_128x128"),
    (9, 2385, 3733, "wide gram_256x256 square_256x256 update_256x256"),
]

# tokens, vocabulary, hidden, forward plan and pieces, backward plan and pieces
XENT = [
    (3, 8377, 9, "gather pack stats_64x128", 1, "gather pack grad_64x128 dh_64x128 dw_64x64", 1),
    (345, 50271, 152, "stats_128x128", 1, "gather grad_128x128 dh_128x128 dw_256x256", 1),
    (16667, 65, 10, "gather pack stats_128x128", 1, "gather pack grad_128x128 dh_64x64 dw_64x64", 1),
    (135, 35441, 9, "gather pack stats_192x192", 1, "gather pack grad_192x192 dh_128x128 dw_128x128", 1),
    (171, 61177, 331, "gather pack stats_256x256", 1, "gather pack grad_256x256 dh_128x128 dw_128x128", 1),
    (69, 52373, 2585, "gather pack stats_128x128_stream", 1,
     "gather pack grad_128x128_stream dh_128x128 dw_128x128", 1),
    (151, 100003, 1432, "stats_256x256_stream", 1, "gather grad_256x256_stream dh_128x128 dw_128x128", 1),
    (141, 108911, 1411, "gather pack stats_256x256_stream", 1,
     "gather pack grad_256x256_stream dh_128x128 dw_128x128", 1),
    # a W that is packed a piece at a time, in both passes
    (5, 64061, 4211, "gather pack stats_64x128", 2, "gather pack grad_64x128 dh_64x128 dw_128x128", 2),
    (66, 147233, 1915, "gather pack stats_128x128_stream", 2,
     "gather pack grad_128x128_stream dh_128x128 dw_128x128", 2),
    (133, 43451, 6525, "gather pack stats_192x192", 2, "gather pack grad_192x192 dh_128x128 dw_128x128", 2),
    (293, 63421, 4402, "gather pack stats_256x256", 2, "gather pack grad_256x256 dh_256x256 dw_128x128", 2),
    (153, 256811, 1050, "gather pack stats_256x256_stream", 2,
     "gather pack grad_256x256_stream dh_128x128 dw_128x128", 2),
    (2245, 121341, 133, "gather pack stats_128x128", 1, "gather pack grad_128x128 dh_128x128 dw_256x256", 2),
    # an aligned W, in pieces for the backward pass
    (945, 299093, 8, "stats_128x128", 1, "gather grad_128x128 dh_128x128 dw_128x128", 2),
    (6161, 44309, 136, "stats_128x128", 1, "gather grad_128x128 dh_128x128 dw_192x192", 2),
    (19459, 15519, 56, "stats_128x128", 1, "gather grad_128x128 dh_256x256 dw_64x64", 2),
]


def newton_schulz_kernels(batch, rows, cols):
    """The kernels a call takes: the Gram and update products by their side, the
    square, which has none; or the one-workgroup or strip form."""
    status, name = tg.tg_newton_schulz_plan(batch, rows, cols)
    assert status == tg.TG_OK, (batch, rows, cols)
    if " " not in name:
        # the columns of the image are in the name, its rows follow from the short side
        return {(name, 64 if min(rows, cols) <= 64 else 128)}
    side, gram, square, update = name.split()
    return {(side, gram), square, (side, update)}


def xent_kernels(M, V, K):
    """The kernels the two passes take for aligned operands, with whether the rows are
    gathered (forward) or the vocabulary is taken in pieces."""
    out = set()
    for backward in (0, 1):
        status, name, pieces = tg.tg_xent_plan(ALIGNED, ALIGNED, M, V, K, K, K, backward)
        assert status == tg.TG_OK, (M, V, K)
        words, many = name.split(), pieces > 1
        kernels = [w for w in words if "_" in w]
        out.update((w, "gathered" if "gather" in words else "as it is") if not backward else (w, many) for w in kernels)
        out.add(("forward" if not backward else "backward", "packed" if "pack" in words else "aligned", many))
    return out
