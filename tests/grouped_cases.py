"""Sizes at which the grouped products take each of their kernels, ragged in every
dimension, with the plans that they are there for (contiguous, aligned operands of
odd widths, which are packed first).  The GPU tests run them, and the CPU tests hold
them to the plans and the plans to every kernel there is."""
import dense_fp16_gemm_02_amd as tg

ALIGNED = 1 << 20  # an address that is a multiple of 16, never dereferenced

# rows, experts, N, K: plans of Y, dX and dW
GROUPED = [
    (1, 1, 10, 9, "pack_a pack_b y_64x64", "pack_a pack_b dx_64x64", "pack_a pack_b dw_64x64"),
    (22, 20, 1544, 8, "y_64x128", "dx_64x64", "dw_64x64"),
    (1, 5, 2633, 132, "pack_a pack_b y_16x32", "pack_a pack_b dx_64x64_split", "pack_a pack_b dw_128x128x4"),
    (12190, 5, 8, 79, "pack_a pack_b y_64x64", "pack_b dx_64x128", "pack_b dw_64x64_split"),
    (405, 5, 8, 10340, "pack_a pack_b y_64x64_split", "pack_b dx_128x128x4", "pack_b dw_128x128"),
    (25, 20, 11335, 73, "pack_a pack_b y_128x128x4", "pack_a pack_b dx_64x128_split", "pack_a pack_b dw_128x128x4"),
    (1, 1, 7761, 7684, "pack_a pack_b y_16x32", "pack_a pack_b dx_64x64_split", "pack_a pack_b dw_128x128x4"),
    (2, 1, 11280, 6398, "pack_a pack_b y_64x128_split", "pack_b dx_64x64_split", "pack_b dw_128x128x4"),
    (13244, 5, 130, 147, "pack_a pack_b y_128x128", "pack_a pack_b dx_128x128", "pack_a pack_b dw_64x64_split"),
    (7789, 5, 6834, 8, "y_128x128x4", "pack_a dx_128x128x4_split", "pack_a dw_128x128"),
    (9722, 70, 419, 488, "y_192x192", "pack_a dx_128x128x4", "pack_a dw_128x128x4"),
    (3886, 3, 73, 7473, "pack_a pack_b y_128x128_split", "pack_a pack_b dx_128x128x4", "pack_a pack_b dw_128x128"),
    (2389, 5, 161, 8155, "pack_a pack_b y_192x192_split", "pack_a pack_b dx_128x128x4", "pack_a pack_b dw_192x192"),
    (6094, 1, 70, 10950, "pack_a pack_b y_128x128x4_split", "pack_a pack_b dx_128x128x4", "pack_a pack_b dw_128x128_split"),
    (8120, 70, 756, 823, "pack_a pack_b y_256x256", "pack_a pack_b dx_128x128x4", "pack_a pack_b dw_128x128x4"),
    (11614, 2, 4052, 165, "pack_a pack_b y_128x128x4", "pack_a pack_b dx_256x256_split", "pack_a pack_b dw_192x192_split"),
    (1609, 9, 1230, 4700, "pack_a pack_b y_256x256_split", "pack_a pack_b dx_128x128x4", "pack_a pack_b dw_128x128x4"),
    (1, 1, 9216, 9889, "pack_a pack_b y_16x32", "pack_b dx_128x128_split", "pack_b dw_128x128x4"),
    (2296, 5, 1163, 3962, "pack_a pack_b y_256x256_split", "pack_a pack_b dx_256x256", "pack_a pack_b dw_128x128x4"),
    (16381, 9, 168, 6432, "y_256x256_split", "dx_128x128x4", "dw_256x256"),
]
# the kernels of dW for so many rows that only dW is compared
LONG = [
    (184321, 3, 392, 392, "dw_256x256_split"),
    (623363, 5, 400, 264, "dw_128x128x4_split"),
]
TILES = {"y": ("256x256", "192x192", "128x128", "64x64", "64x128", "128x128x4"),
         "dx": ("256x256", "128x128", "64x64", "64x128", "128x128x4"),
         "dw": ("256x256", "192x192", "128x128", "64x64", "128x128x4")}
KERNELS = {f"{what}_{tile}{split}" for what, tiles in TILES.items() for tile in tiles for split in ("", "_split")} | {"y_16x32"}


def plans(M, E, N, K):
    """The plans of Y, dX and dW for contiguous operands."""
    out = []
    for product, lda in ((tg.TG_GROUPED_Y, K), (tg.TG_GROUPED_DX, N), (tg.TG_GROUPED_DW, N)):
        status, name = tg.tg_grouped_plan(product, ALIGNED, ALIGNED, M, E, N, K, lda, K, N * K)
        assert status == tg.TG_OK, (M, E, N, K)
        out.append(name)
    return tuple(out)
