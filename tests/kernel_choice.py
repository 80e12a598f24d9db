"""Which kernel a product takes at which sizes: the library's rules written again, so
that a test can assert that its shapes reach the kernel that it is about.
test_kernel_choice_cpu holds them against the source."""
from __future__ import annotations


def _up(a: int, b: int) -> int:
    return -(-a // b)


def fp8_gemm(T: int, N: int, K: int) -> str:
    """Columns a workgroup, or the block (tokens x columns) and its groups of waves."""
    def tiles(rows, cols):
        return _up(T, rows) * _up(N, cols)

    if T <= 16 and N <= 8192:
        return "16 tokens"
    if T <= 32 and N <= 4096:
        return "32 tokens"
    if tiles(64, 64) <= 256:
        return "64 x 64, two groups" if K > 2048 else "64 x 64"
    if tiles(64, 128) <= 256:
        return "64 x 128, two groups"
    if tiles(64, 128) <= 512:
        return "64 x 128"
    if tiles(128, 128) <= 512:
        return "128 x 128"
    return "256 x 256"


def _filled(blocks: int) -> bool:
    return blocks >= 1024 or 10 * blocks >= 8 * (_up(blocks, 256) * 256)


def grouped_side(rows_max: int, E: int, cols: int) -> int:
    """The block's rows of the forward product and the input's gradient."""
    least = min(rows_max, E)

    def blocks(side):
        return max(rows_max // side + least // 2, least) * _up(cols, side)

    wide = blocks(256)
    if rows_max >= 32 * E and wide >= 200 and (wide >= 448 or (rows_max >= 96 * E and _filled(wide))):
        return 256
    return 128 if rows_max >= 32 * E and blocks(128) >= 150 else 32


def _row_blocks(rows: int, end: int, side: int) -> tuple[int, int]:
    """Blocks of an expert's rows that hold some, and all with its padding's."""
    held, padded = _up(rows, side), (end + side - 1 - side // 2) // side
    return held, 0 if end == 0 else max(held, padded, 1)


def grouped_tall(rows: int, end: int, cols: int) -> bool:
    """Whether an expert of `rows` rows, `end` with its padding, takes blocks of 320 x
    192 where blocks of 256 x 256 are the others'."""
    held, tiles = _row_blocks(rows, end, 256)
    held_tall, tiles_tall = _row_blocks(rows, end, 320)
    return held_tall < held and 15 * tiles_tall * _up(cols, 192) < 16 * tiles * _up(cols, 256)


def weight_side(rows_max: int, E: int, N: int, D: int) -> int:
    wide = E * _up(N, 256) * _up(D, 256)
    return 256 if rows_max >= (96 if wide >= 4096 else 192) * E and wide >= 200 and _filled(wide) else 128
