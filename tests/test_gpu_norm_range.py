"""The norm over the whole range of finite values: rows whose squares, or whose
sum, lie past fp32's range, and rows whose squares lie below it.  Tolerances are
tests/test_gpu_norm.py's."""

import numpy as np
import pytest
import torch

from oracle import norm as ON
from rank_step_amd import binding as B
from tests.test_gpu_linear import U, gen, randn
from tests.test_gpu_norm import EPS, check_forward, close

pytestmark = pytest.mark.gpu

# rows by one wave, by several, and past the registers; with elements behind the last chunk and without
WIDTHS = [1, 5, 64, 501, 1365, 4096, 9000, 40000]
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def limited(x):
    """Within both types' range."""
    return x.double().clamp(-3.3e38, 3.3e38).float()


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_large_values(gpu, n, dtype, kind):
    g = gen(1)
    r = randn(g, 9, n)
    signs = torch.where(r < 0, -3.2e38, 3.2e38)  # their sums pass the range in both directions
    for x in (r * 2.0 ** 63, r * 1e25, limited(1e38 * r.double()), limited(2e38 + 4e37 * r.double()), signs):
        check_forward(9, n, dtype, kind, values=x)
    check_forward(9, n, dtype, kind, values=1e25 * r, same=True, off=1, pad=3)


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_constant_rows_of_large_values(gpu, n, dtype):
    """A layer norm of a constant row is its bias, and rstd 1 / sqrt(eps), where
    the mean is a number of the type: where the sum overflows as elsewhere."""
    x = torch.full((3, n), 3.25 * 2.0 ** 125, device=gpu).to(DTYPES[dtype])
    y, mean, rstd = torch.empty_like(x), torch.empty(3, device=gpu), torch.empty(3, device=gpu)
    b = randn(gen(2), 1, n).to(DTYPES[dtype])
    B.fsdp_norm_forward(y, x, 3, n, dtype=dtype, bias=b, w_dtype=dtype, mean=mean, rstd=rstd)
    assert torch.equal(y, b.expand(3, n)) and bool((mean == x[:, 0].float()).all())
    assert bool(((rstd.double() - EPS ** -0.5).abs() <= 4 * U * EPS ** -0.5).all())
    check_forward(3, n, dtype, "rms", values=x.float())


@pytest.mark.parametrize("n", WIDTHS[1:])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_small_values_without_eps(gpu, n, kind):
    r = randn(gen(3), 9, n)
    for scale in (1e-15, 1e-18, 1e-21, 1e-25, 1e-33):
        check_forward(9, n, "f32", kind, values=scale * r, eps=0.0)
    check_forward(9, n, "bf16", kind, values=1e-25 * r, eps=0.0)
    check_forward(9, n, "f32", kind, values=1e-21 * r, eps=1e-42)


@pytest.mark.parametrize("m,n", [(70, 40), (70, 4096), (600, 33000)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_other_rows_keep_their_bits(gpu, m, n, kind):
    """Rows in and out of the range side by side; those within it as in a call of their own."""
    r = randn(gen(4), m, n)
    scale = torch.tensor([1.0, 1e25, 1.0, 1e37, 1e19], device=gpu).repeat(m)[:m, None]
    x = r * scale
    check_forward(m, n, "f32", kind, values=x)
    out = {}
    for name, v in (("mixed", x), ("alone", r)):
        y, rstd = torch.empty_like(v), torch.empty(m, device=gpu)
        B.fsdp_norm_forward(y, v, m, n, dtype="f32", kind=kind, rstd=rstd)
        out[name] = y[scale[:, 0] == 1], rstd[scale[:, 0] == 1]
    assert all(torch.equal(a, b) for a, b in zip(out["mixed"], out["alone"]))


@pytest.mark.parametrize("m,n", [(9, 64), (9, 1365), (9, 40000), (1500, 64)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_gradients_of_large_values(gpu, m, n, kind):
    g = gen(5)
    x, dy = 1e25 * (randn(g, m, n) + 0.5), randn(g, m, n)
    y, dx, dw, db = torch.empty_like(x), torch.empty_like(x), torch.empty(n, device=gpu), torch.empty(n, device=gpu)
    mean, rstd = torch.empty(m, device=gpu) if kind == "layer" else None, torch.empty(m, device=gpu)
    B.fsdp_norm_forward(y, x, m, n, dtype="f32", kind=kind, mean=mean, rstd=rstd)
    B.fsdp_norm_backward(dx, dy, x, m, n, dtype="f32", kind=kind, mean=mean, rstd=rstd, dw=dw, db=db,
                         workspace=torch.empty(B.NORM_WORKSPACE_BYTES, dtype=torch.uint8, device=gpu))
    xv, dyv, rv = (t.double().cpu().numpy() for t in (x, dy, rstd))
    mv = mean.double().cpu().numpy() if mean is not None else 0 * rv
    _, m64, r64 = ON.forward(xv, kind=kind)
    assert np.all(np.abs(rv - r64) <= 1e-5 * r64) and np.all(np.abs(mv - m64) <= 1e-5 * np.abs(m64))
    dxv, dwv, dbv = ON.backward(dyv, xv, mv, rv, None, kind)
    xhat = np.abs(xv - mv[:, None]) * rv[:, None]
    ag, long = np.abs(dyv), 64 + n / 1024
    m1 = ag.mean(axis=1, keepdims=True) if kind == "layer" else 0.0
    m2 = (ag * xhat).mean(axis=1, keepdims=True)
    e = rv[:, None] * ((long + 8) * U * (m1 + xhat * m2) + 6 * U * (ag + m1 + xhat * m2))
    # dx is about 1e-25, far from the smallest fp32: scaled so that `close` counts rounding alone
    close(2.0 ** 80 * dx.double().cpu().numpy(), 2.0 ** 80 * dxv, 2.0 ** 80 * (e + 2 * U * np.abs(dxv)), "f32", "dx")
    close(dw.double().cpu().numpy(), dwv, 143 * U * (ag * xhat).sum(axis=0), "f32", "dw")
    close(db.double().cpu().numpy(), dbv, 143 * U * ag.sum(axis=0), "f32", "db")
