"""The norm's column sums where many rows pass through one place.

A thread adds its rows in chains of at most 64, which it joins in 64 bits; then
come the 8 waves of a workgroup at most, rounded to fp32 first, and the rows of
sums, of which there are at most 2048: 64 for each of 32 places, joined by halves.
So a term passes through at most 64 + 8 + 64 + 5 additions in fp32, however many
rows there are: with 2 for its own product and the rounding, 143 u of the terms'
magnitudes, u = 2^-24.
"""

import pytest
import torch

from rank_step_amd import binding as B
from tests.test_gpu_linear import U, gen

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def workspace(parts, n, gpu):
    """Room for so many rows of sums; None: all that a call uses."""
    size = B.NORM_WORKSPACE_BYTES if parts is None else parts * 8 * n
    return torch.empty(size, dtype=torch.uint8, device=gpu) if size else None


# without room for parts and with room for three, for 64 (the fewest that are
# summed beside dx), by each division of a row, with elements behind its last
# chunk and without; and rows enough for long chains in the whole workspace
LONG = [(1 << 17, 5, "f32", 0), (1 << 17, 40, "bf16", 0), (1 << 18, 24, "f32", 3), (1 << 17, 11008, "bf16", 8),
        (1 << 20, 24, "f32", 64), (1 << 20, 25, "bf16", 64), (1 << 19, 501, "f32", 64), (1 << 19, 1000, "bf16", 64),
        (1 << 17, 1023, "f32", 64), (1 << 17, 2048, "bf16", 64), (1 << 17, 2048, "f32", 64), (1 << 17, 4095, "bf16", 64),
        (1 << 17, 4095, "f32", 64), (1 << 17, 8192, "bf16", 64), (1 << 23, 8, "f32", None)]


@pytest.mark.parametrize("m,n,dtype,parts", LONG)
def test_long_chains(gpu, m, n, dtype, parts):
    """Every row the same: the roundings of one long chain all go one way."""
    g, t = gen(m + n), DTYPES[dtype]
    dy, x = ((1 + torch.rand(n, generator=g, device=gpu)).to(t) for _ in range(2))
    mean, rstd = torch.full((m,), -0.375, device=gpu), torch.full((m,), 1.2345678, device=gpu)
    rows_dy, rows_x = dy.expand(m, n).contiguous(), x.expand(m, n).contiguous()
    dx = torch.empty_like(rows_x)
    dw, db = torch.empty(n, device=gpu), torch.empty(n, device=gpu)
    B.fsdp_norm_backward(dx, rows_dy, rows_x, m, n, dtype=dtype, mean=mean, rstd=rstd, dw=dw, db=db,
                         workspace=workspace(parts, n, gpu))
    want_db = m * dy.double()
    want_dw = want_db * (x.double() + 0.375) * rstd[0].double()
    for name, got, want in (("db", db, want_db), ("dw", dw, want_dw)):
        off = ((got.double() - want).abs() / (143 * U * want)).max().item()
        assert off <= 1, (name, off)


EXACT = [(n, t) for n in (24, 251, 1000, 1365, 2048, 4095, 4096, 8191, 11008) for t in ("bf16", "f32")]


@pytest.mark.parametrize("m", [1500, 8195, 70001])
@pytest.mark.parametrize("n,dtype", EXACT)
def test_sums_of_whole_numbers(gpu, m, n, dtype):
    """Terms of whole numbers, sums under 2^24: every order gives the same, and one
    row that is left out, or taken twice, shows."""
    g, t = gen(m + n), DTYPES[dtype]
    dy, x = (torch.randint(-7, 8, (m, n), generator=g, device=gpu, dtype=torch.int8).to(t) for _ in range(2))
    rstd = torch.ones(m, device=gpu)
    dx = torch.empty_like(x)
    want_db, want_dw = torch.zeros(n, dtype=torch.float64, device=gpu), torch.zeros(n, dtype=torch.float64, device=gpu)
    for a, b in zip(dy.split(8192), x.split(8192)):
        want_db += a.double().sum(0)
        want_dw += (a.double() * b.double()).sum(0)
    assert m * 49 < 2 ** 24
    for parts in (None, 64, 3, 0) if m < 70001 else (None, 64):
        dw, db = torch.empty(n, device=gpu), torch.empty(n, device=gpu)
        B.fsdp_norm_backward(dx, dy, x, m, n, dtype=dtype, kind="rms", rstd=rstd, dw=dw, db=db,
                             workspace=workspace(parts, n, gpu))
        assert torch.equal(dw.double(), want_dw) and torch.equal(db.double(), want_db), parts
