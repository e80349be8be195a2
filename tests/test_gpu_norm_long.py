"""The norm of rows that registers do not hold, long enough that a thread's sums
in fp32 would show: values of one sign and size, whose partial sums' roundings
all go one way.

Tolerances, with u = 2^-24: a chunk's sum takes at most 8 fp32 additions, a
thread's is rounded to fp32 once (its 64-bit error is nothing beside that), 6
additions join a wave's and 16 the waves', so 32u with the quotient.  Of the mean:
32u of the mean magnitude and u of itself, which enters the variance squared; half
of the variance's 34u in rstd, and 4u for eps, root and quotient; the rest as in
tests/test_gpu_norm.py."""

import numpy as np
import pytest
import torch

from oracle import norm as ON
from rank_step_amd import binding as B
from tests.test_gpu_linear import U, gen, randn
from tests.test_gpu_norm import close

pytestmark = pytest.mark.gpu

L = 32


@pytest.mark.parametrize("n", [1 << 22, (1 << 22) + 12345])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_long_rows(gpu, n, dtype, kind):
    m, g = 2, gen(n)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = (1.0 + 0.4 * torch.rand(m, n, generator=g, device=gpu)).to(t)
    y, rstd = torch.empty_like(x), torch.empty(m, device=gpu)
    mean = torch.empty(m, device=gpu) if kind == "layer" else None
    B.fsdp_norm_forward(y, x, m, n, dtype=dtype, kind=kind, mean=mean, rstd=rstd)
    xv = x.double().cpu().numpy()
    yv, mv, rv = ON.forward(xv, None, None, 1e-5, kind)
    # mean^2 is over 16 variances: corrected by the mean distance, L u of the spread
    spread = xv.std(axis=1) if kind == "layer" else 0
    em = (2 * U * np.abs(mv) + (L + 3) * U * (spread + L * U * np.abs(mv))) if kind == "layer" else 0 * rv
    er = rv * ((0.5 * (L + 2) + 4) * U + (em * rv) ** 2)
    close(rstd.double().cpu().numpy(), rv, er, "f32", "rstd")
    if kind == "layer":
        close(mean.double().cpu().numpy(), mv, em, "f32", "mean")
    d = np.abs(xv - (mv[:, None] if kind == "layer" else 0))
    ey = em[:, None] * rv[:, None] + d * er[:, None] + 3 * U * d * rv[:, None] + U * np.abs(yv)
    close(y.double().cpu().numpy(), yv, ey, dtype, "y")

    dy = (1e-3 * (1 + torch.rand(m, n, generator=g, device=gpu))).to(t)
    dx = torch.empty_like(x)
    B.fsdp_norm_backward(dx, dy, x, m, n, dtype=dtype, kind=kind, mean=mean, rstd=rstd)
    mv = mean.double().cpu().numpy() if kind == "layer" else np.zeros(m)
    rv = rstd.double().cpu().numpy()
    gv = dy.double().cpu().numpy()
    dxv = ON.backward(gv, xv, mv, rv, None, kind)[0]
    xhat = np.abs(xv - mv[:, None]) * rv[:, None]
    m1 = gv.mean(axis=1, keepdims=True) if kind == "layer" else 0.0
    m2 = (gv * xhat).mean(axis=1, keepdims=True)
    e = rv[:, None] * ((L + 2) * U * (m1 + xhat * m2) + 6 * U * (gv + m1 + xhat * m2)) + 2 * U * np.abs(dxv)
    close(dx.double().cpu().numpy(), dxv, e, dtype, "dx")


def test_long_rows_in_place(gpu):
    n = (1 << 20) + 3
    x = randn(gen(3), 3, n)
    want = torch.empty_like(x)
    B.fsdp_norm_forward(want, x, 3, n, dtype="f32")
    B.fsdp_norm_forward(x, x, 3, n, dtype="f32")
    assert torch.equal(x, want)
    assert bool(x.isfinite().all())
