"""Products for every way the 4-bit product is computed, with the way each is
meant to take: tests/test_mx4_plan.py checks on the CPU that it does, and
tests/test_gpu_mx4_ways.py runs it.

A row: output rows, output columns, contraction length, workspace bytes, and the
way: T/P (T x T tiles, the contraction in P parts; 64xW/P: W waves a tile), "few F" (16 F columns a
workgroup), or a cut into two outputs (columns, rows) and their ways.
"""

MIB = 1 << 20

ROUTES = [
    (1, 16 * 256, 700, 0, "few 1"),
    (16, 2 * 16 * 256 - 5, 700, 0, "few 2"),
    (9, 3 * 16 * 256 - 5, 1100, 0, "few 3"),
    (16, 4 * 16 * 256 - 5, 300, 0, "few 4"),
    (1, 20000, 700, 0, "64x2/1"),
    (16, 16 * 1024 + 1, 300, 0, "64x2/1"),
    (17, 300, 900, 64 * MIB, "64x4/1"),
    (1000, 1000, 2050, 64 * MIB, "64x4/1"),
    (64, 64, 16385, 64 * MIB, "64x4/7"),
    (70, 130, 40001, 64 * MIB, "64x4/16"),
    (300, 200, 20000, 1 * MIB, "64x4/4"),
    (2048, 2060, 1300, 64 * MIB, "128/1"),
    (1024, 1365, 2047, 64 * MIB, "64x2/1"),
    (500, 4096, 513, 64 * MIB, "64x2/1"),
    (1024, 2049, 2047, 64 * MIB, "128/1"),
    (4000, 4080, 3000, 64 * MIB, "256/1"),
    (4096, 4100, 4096, 64 * MIB, "columns 256/1 64x4/1"),
    (4100, 4096, 4096, 64 * MIB, "rows 256/1 few 1"),
    (4196, 4096, 4096, 64 * MIB, "rows 256/1 64x4/1"),
]
