"""Sizes at which the grouped products take each of their kernels, ragged where the
kernel's choice allows, with the plans that they are there for: together they reach
every kernel (test_training_plan_cpu.py), and the GPU tests run them."""
import dense_fp16_gemm_02_amd as tg

ALIGNED = 1 << 20  # an address that is a multiple of 16, never dereferenced

# rows, experts, N, K: plans of Y, dX and dW
GROUPED = [
    (1, 1, 9, 9, "pack_a pack_b y_16x32", "pack_a pack_b dx_64x64", "pack_a pack_b dw_64x64"),
    (27, 5, 520, 5000, "y_16x32", "dx_64x128", "dw_128x128"),
    (66, 70, 226, 72, "y_64x64", "pack_a dx_64x64", "pack_a dw_128x128"),
    (75, 70, 432, 8, "y_64x128", "dx_64x64", "dw_192x192"),
    (66, 70, 240, 7992, "y_64x64_split", "dx_64x128", "dw_256x256"),
    (20, 20, 1375, 4930, "pack_a pack_b y_64x128_split", "pack_a pack_b dx_64x128", "pack_a pack_b dw_256x256"),
    (30, 20, 10952, 88, "y_64x128", "dx_64x128_split", "dw_128x128"),
    (5, 2, 5909, 24, "y_16x32", "pack_a dx_64x64_split", "pack_a dw_64x64"),
    (2906, 9, 7134, 65, "pack_a pack_b y_128x128", "pack_a pack_b dx_128x128_split", "pack_a pack_b dw_192x192"),
    (3682, 5, 72, 6008, "y_128x128_split", "dx_128x128", "dw_64x64_split"),
    (2243, 20, 144, 7144, "y_192x192_split", "dx_128x128", "dw_256x256"),
    (5713, 5, 7016, 196, "y_192x192", "pack_b dx_256x256_split", "pack_b dw_128x128"),
    (6015, 1, 201, 6312, "y_256x256_split", "pack_a dx_128x128", "pack_a dw_128x128"),
    (3893, 3, 3515, 9, "pack_a pack_b y_256x256", "pack_a pack_b dx_128x128", "pack_a pack_b dw_64x64"),
    (5450, 3, 8, 2536, "y_64x64", "dx_256x256", "dw_64x64"),
    (9677, 2, 4169, 65, "pack_a pack_b y_256x256", "pack_a pack_b dx_128x128_split", "pack_a pack_b dw_128x128_split"),
    (13060, 2, 144, 2792, "y_128x128", "dx_256x256", "dw_192x192_split"),
    (11782, 2, 8618, 197, "pack_a pack_b y_256x256", "pack_a pack_b dx_256x256_split", "pack_a pack_b dw_256x256_split"),
    (8192, 20, 200, 264, "y_192x192", "dx_128x128", "dw_64x64_split"),
]


def plans(M, E, N, K):
    """The plans of Y, dX and dW for contiguous operands."""
    out = []
    for product, lda in ((tg.TG_GROUPED_Y, K), (tg.TG_GROUPED_DX, N), (tg.TG_GROUPED_DW, N)):
        status, name = tg.tg_grouped_plan(product, ALIGNED, ALIGNED, M, E, N, K, lda, K, N * K)
        assert status == tg.TG_OK, (M, E, N, K)
        out.append(name)
    return tuple(out)
