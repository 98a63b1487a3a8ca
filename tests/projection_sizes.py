"""Sizes of the 8-bit products that reach each of their kernels: test_projection_routes_host.py checks that they do,
test_gpu_projection_edges.py runs them."""

TURNS, DMA, TILE, FEW_DMA, FEW = ("linear_turns_kernel", "linear_dma_kernel", "linear_tile_kernel", "linear_few_dma_kernel",
                                  "linear_few_kernel")

# T, N, the Ks and, for a plain product, the kernels (with their tile where there are several) that bf16 and fp32 take
PLAIN = [
    (1, 9000, (1040, 16), (FEW_DMA, 4, 1, 2)),
    (5, 400, (1040, 128), (FEW_DMA, 8, 1, 1)),
    (20, 9000, (272,), (FEW_DMA, 4, 2, 2)),
    (20, 400, (1040,), (FEW_DMA, 4, 2, 1)),
    (50, 9000, (272,), (FEW_DMA, 4, 4, 2)),
    (130, 400, (1040, 2064), (FEW_DMA, 4, 4, 1)),
    (700, 1500, (1040, 128), (DMA, 2, 2, 2, 2, 4)),
    (1100, 1500, (1040, 128), (DMA, 2, 2, 4, 4, 2)),
    (2100, 2100, (128, 272, 1040), (DMA, 2, 2, 4, 4, 1)),
    # the largest tiles: one run, two, more, with a shorter last one and without, many
    (2100, 4000, (128, 256, 272, 384, 400, 1024, 1040, 2064), {"bf16": (TURNS,), "fp32": (DMA, 4, 2, 4, 8, 1)}),
    (5, 400, (1041, 1), (FEW,)),
    (40, 1000, (301,), (FEW,)),
    (300, 1000, (1041,), (TILE, 2, 2, 2, 2, 2)),
    (2100, 2100, (129, 1041), (TILE, 2, 2, 4, 4, 1)),
]
GATED = [
    (5, 9000, (272,), (FEW_DMA, 4, 1, 1)),
    (5, 400, (1040, 128), (FEW_DMA, 8, 1, 1)),
    (20, 400, (1040,), (FEW_DMA, 4, 2, 1)),
    (130, 400, (1040,), (FEW_DMA, 4, 4, 1)),
    (700, 800, (1040, 128), (DMA, 2, 2, 2, 4, 2)),
    (1100, 800, (1040, 128), (DMA, 2, 2, 4, 4, 2)),
    (2100, 1100, (128, 272, 1040), (DMA, 2, 2, 4, 4, 1)),
    (2100, 2000, (128, 256, 272, 384, 400, 1024, 1040), {"bf16": (TURNS,), "fp32": (DMA, 4, 2, 4, 8, 1)}),
    (5, 400, (1041,), (FEW,)),
    (300, 600, (1041,), (TILE, 2, 2, 2, 4, 2)),
    (2100, 1100, (129, 1041), (TILE, 2, 2, 4, 4, 1)),
]
# e4m3 outputs of a single launch
CODES = [
    (2100, 4400, (128, 256, 272, 400, 1024, 1040), (DMA, 4, 2, 4, 8, 1)),
    (2100, 4400, (129, 1041), (TILE, 4, 2, 2, 8, 1)),
]


def cases(table):
    return [(T, K, N) for T, N, ks, _ in table for K in ks]
