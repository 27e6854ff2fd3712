"""Cases of the bf16 expert products by the kernel that each has to take: groups' sizes, rows behind the last
group, N (gated: 2I), epilogue and layout of the weights.  K is 328 or 360 (split: 1800), so every kernel goes round its
ring of stages more than once and ends in a part of one, after an odd and an even number of stages."""
import block_scaled_fp4_02_amd as moe

PLAIN, GATED, BACK = moe.MOE_EPI_NONE, moe.MOE_EPI_SWIGLU, moe.MOE_EPI_SWIGLU_BACKWARD
ROWMAJOR, TRANSPOSED = moe.MOE_LAYOUT_ROWMAJOR, moe.MOE_LAYOUT_TRANSPOSED
TILES = ["256x256", "128x128", "64 rows", "32 rows", "split 16", "split 32"]   # in the order of GemmTile

PAD = 5
SIZES = {  # sizes and N
    "256x256": ([300, 0, 517, 45], 12808), "128x128": ([130, 200, 0, 95], 12808), "64 rows": ([50] * 9 + [0, 70], 4104),
    "32 rows": ([64, 128, 0, 1], 2600), "split 16": ([1, 0, 3], 24), "split 32": ([5], 4808),
}
WAYS = {"plain, row-major": (PLAIN, ROWMAJOR), "plain, transposed": (PLAIN, TRANSPOSED), "gated": (GATED, ROWMAJOR), "backward": (BACK, TRANSPOSED)}


def taken(way):
    """The kernels that an epilogue and a layout have."""
    epilogue, layout = WAYS[way]
    return [t for t in TILES if not (layout == TRANSPOSED and t.startswith("split")) and not (epilogue == GATED and t in ("128x128", "32 rows"))]


CASES = [(way, tile, K) for way in WAYS for tile in taken(way) for K in ((1800,) if tile.startswith("split") else (328, 360))]


def sizes_of(way, tile):
    sizes, N = SIZES[tile]
    # (a gated product's N is twice its columns, a multiple of 16)
    return sizes, N if WAYS[way][0] != GATED else (N + 15) // 16 * 16
