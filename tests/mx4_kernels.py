"""Sizes of the 4-bit linear layer for each of its kernels: a CPU test holds them to
fl_mx4_linear_plan, so that a change of its estimates shows, the GPU tests run them.

A kernel: (1 streaming or 2 tiles, rows and columns of a workgroup, its waves, whether K is in
parts, the waves of the second launch or 0).  Depths are counts of blocks of 32; K is less by
up to two (depth()).
"""
from typing import NamedTuple


class Kernel(NamedTuple):
    plan: tuple
    M: int
    N: int
    sweep: tuple  # depths, every place in a stage of 8 blocks and in the scales of four stages where it can
    deep: int     # one of them, for the epilogue's tests
    inside: bool = False  # values of A are quantised by the kernel itself


KERNELS = {
    "stream_16x16_16": Kernel((1, 16, 16, 16, False, 0), 30, 101, (*range(1, 42), 300), 37),
    "stream_16x16_16_values": Kernel((1, 16, 16, 16, False, 0), 16, 101, (*range(1, 42), 90), 37, True),
    "stream_16x16_8": Kernel((1, 16, 16, 8, False, 0), 130, 1807, (*range(1, 42),), 37),
    "stream_16x16_8_values": Kernel((1, 16, 16, 8, False, 0), 1, 4497, (*range(1, 42), 300), 37, True),
    "stream_16x32_8": Kernel((1, 16, 32, 8, False, 0), 34, 1395, (*range(1, 42), 63), 37),
    "stream_16x32_8_values": Kernel((1, 16, 32, 8, False, 0), 7, 4497, (*range(1, 42), 199), 37, True),
    "stream_32x16_8": Kernel((1, 32, 16, 8, False, 0), 17, 2073, (*range(1, 42), 300), 37),
    "stream_32x32_8": Kernel((1, 32, 32, 8, False, 0), 18, 7191, (*range(1, 42), 300, 519), 37),
    "stream_32x64_8": Kernel((1, 32, 64, 8, False, 0), 18, 15043, (*range(1, 42), 255, 300), 37),
    "stream_64x32_8": Kernel((1, 64, 32, 8, False, 0), 49, 7685, (*range(1, 42), 257, 280), 37),
    "stream_64x64_8": Kernel((1, 64, 64, 8, False, 0), 33, 13961, (*range(129, 170),), 165),
    "tile_128x128_alone": Kernel((2, 128, 128, 8, False, 0), 1025, 511, (*range(1, 42), 74, 131), 74),
    "tile_128x128": Kernel((2, 128, 128, 4, False, 0), 2490, 2437, (*range(1, 42), 74, 131), 74),
    "tile_256x256": Kernel((2, 256, 256, 8, False, 0), 4090, 4095, (*range(1, 42), 74, 131), 74),
    "tile_256x256_then_128x128_alone": Kernel((2, 256, 256, 8, False, 8), 4643, 3515, (*range(1, 42), 74), 74),
    "tile_256x256_then_128x128": Kernel((2, 256, 256, 8, False, 4), 4613, 4811, (*range(1, 42), 74), 74),
    "parts_of_128x128_alone": Kernel((2, 128, 128, 8, True, 0), 701, 131, (*range(97, 138), 300), 130),
    "parts_of_128x128": Kernel((2, 128, 128, 4, True, 0), 14, 16621, (*range(569, 574), *range(753, 769)), 765),
    "parts_of_256x256": Kernel((2, 256, 256, 8, True, 0), 271, 11595, (*range(329, 370, 4), 400, 519), 333),
}


def depth(blocks):
    return 32 * blocks - blocks % 3


def plan_of(p):
    """The kernel of an Mx4Plan."""
    return (p.kernel, p.rows, p.columns, p.waves, p.parts > 1, p.second_waves)
