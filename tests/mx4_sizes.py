"""Sizes of the products with 4-bit weights by the tile that they take (held to
it by test_mx4_index.py, run by test_gpu_mx4.py)."""

# contractions: one block, parts of a step, whole steps, whole units of 16 blocks
# and parts of one, rows of scales that start inside a word and that do not
SHORT = (32, 96, 128, 256, 288, 384, 512, 544, 800, 1024, 1056, 1568)
# past what the waves of the kernels for few rows take at once
LONG = SHORT + (2048, 2080, 4256)

# batch, rows, columns
DENSE = {
    "few16x16": (1, 17, 80, LONG), "few16x32": (1, 16, 4112, LONG), "few32x32": (1, 257, 528, SHORT + (2048,)),
    "t32x64g2": (1, 400, 1200, SHORT), "t32x64": (9, 20, 1904, SHORT), "t64x64g2": (1, 700, 1296, SHORT),
    "t64x128g2": (1, 1000, 1504, SHORT), "t64x128": (3, 500, 1712, SHORT), "t128x128": (1, 1700, 2000, SHORT),
    "t256x256": (1, 4100, 3600, SHORT), "t256x256 batch": (3, 1300, 3408, (96, 544, 1056))}

# rows of each expert (with holes and a tail, see test_gpu_mx4.ragged), align, columns
RAGGED = {
    "few16x16": ([1, 0, 2, 1], 1, 80, (32, 160, 1056)), "few16x32": ([3, 16, 17, 0, 1, 40], 4, 640, (96, 288, 2080)),
    "few32x32": ([30, 9, 0, 1, 44, 3, 17, 33], 1, 1008, (32, 544, 1056)),
    "t32x64g2": ([30, 9, 0, 1, 44, 3, 17, 33], 2, 1200, (128, 288, 1056)),
    "t32x64": ([30, 9, 0, 1, 44, 3, 17, 33], 1, 2576, (128, 288, 1056)),
    "t64x64g2": ([130, 9, 0, 1, 144, 63, 65, 64], 1, 1392, (128, 288, 1056)),
    "t64x128g2": ([130, 9, 0, 1, 144, 63, 65, 64], 4, 2000, (128, 288, 1056)),
    "t64x128": ([130, 9, 0, 1, 144, 63, 65, 64], 1, 4000, (128, 288, 1056)),
    "t128x128": ([300, 0, 433, 157, 250, 1, 240], 8, 2576, (128, 288, 1056)),
    "t256x256": ([1600, 0, 2033, 1257, 1900, 1, 1640], 1, 1776, (128, 288, 1056))}


def cap_of(counts, align):
    return sum(n + -n % align for n in counts) + 5
