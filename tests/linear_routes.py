"""Products for every way the linear layer computes one, with the way each is
meant to take: tests/test_linear_plan.py checks on the CPU that it does (so that
other constants in the choice cannot quietly leave a way untested), and
tests/test_gpu_linear.py runs it.

A row: call, weight type, output rows, output columns, contraction length,
workspace bytes, elements that every matrix starts off its buffer and that its
rows are apart beyond their length, and the way:

  direct T/P        T x T tiles, the contraction in P parts
  direct rows A B   cut into two outputs (columns: side by side)
  pieces RxC A      operands laid out anew, the output in R x C pieces, the first A
  staged T/P        operands staged through registers
  few TxF           up to 16 T tokens, 16 F features a workgroup
"""

MIB = 1 << 20
KINDS = [("forward", "bf16"), ("forward", "e4m3"), ("grad_input", "bf16"), ("grad_input", "e4m3"),
         ("grad_weight", "bf16")]


def each(m, n, k, workspace, off, pad, way, kinds=KINDS):
    return [(call, wt, m, n, k, workspace, off, pad, way) for call, wt in kinds]


ROUTES = (
    each(4000, 4080, 1008, 64 * MIB, 0, 0, "direct 256/1")
    + each(2048, 2064, 336, 64 * MIB, 0, 0, "direct 128/1")
    + each(1472, 208, 8304, 64 * MIB, 0, 0, "direct 128/10")
    + each(1456, 208, 8304, 5 * MIB, 0, 16, "direct 64/2")
    + each(16, 32, 1888, 64 * MIB, 0, 0, "direct 128/15", KINDS[2:])
    + each(528, 1040, 1008, 64 * MIB, 0, 0, "direct 64/1")
    + each(304, 128, 8208, 64 * MIB, 0, 0, "direct 64/15")
    + each(48, 64, 11008, 64 * MIB, 0, 0, "direct 64/20")
    + each(4096, 4112, 1024, 64 * MIB, 0, 0, "direct columns 256/1 64/1")
    + each(4112, 4096, 1024, 64 * MIB, 0, 0, "direct rows 256/1 64/1")
    + each(130, 130, 8197, 1 * MIB, 0, 0, "staged 128/13")
    + each(257, 300, 4099, 2 * MIB, 1, 2, "staged 128/6")
    + each(40, 70, 20001, 256 << 10, 3, 1, "staged 128/21")
    + each(601, 523, 2051, 0, 0, 0, "staged 128/1")
    + each(601, 523, 2051, 2 * MIB, 0, 0, "pieces 3x3 64/1", KINDS[3:4])
    + each(300, 1000, 1365, 64 * MIB, 0, 0, "pieces 1x1 64/1")
    + each(130, 77, 8197, 64 * MIB, 1, 1, "pieces 1x1 64/15")
    + [("forward", wt, m, n, 333 if off else 336, 0, off, off, f"few {1 + (m > 16)}x{f}")
       for wt in ("bf16", "e4m3") for off in (0, 1) for m in (1, 16, 17, 32) if m <= 16 or off
       for n, f in ((16 * 256, 1), (2 * 16 * 256 - 5, 2), (3 * 16 * 256 - 5, 3), (4 * 16 * 256 - 5, 4))]
)


def aligned(rows, cols, off, pad, per, size):
    """Whether a matrix takes the direct loads: `per` elements of `size` bytes in 16."""
    return off * size % 16 == 0 and cols % per == 0 and (rows <= 1 or (cols + pad) % per == 0)


def program_case(call, wt, m, n, k, workspace, off, pad):
    """The line that tests/c/linear_plan.cpp takes for a row."""
    fp8 = wt == "e4m3"
    a = (k, m) if call == "grad_weight" else (m, k)
    b = (n, k) if call == "forward" else (k, n)
    a_ok = aligned(*a, off, pad, 8, 2)
    b_ok = aligned(*b, off, pad, 16 if fp8 else 8, 1 if fp8 else 2)
    return f"{call} {int(fp8)} {m} {n} {k} {int(a_ok)} {int(b_ok)} {workspace}\n"
