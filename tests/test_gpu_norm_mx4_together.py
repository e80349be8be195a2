"""The norm and the 4-bit calls in the layouts and captures that a program would
put them in: parts of one buffer, masks that move on between replays."""

import numpy as np
import pytest
import torch

from oracle import mx4 as Q
from rank_step_amd import binding as B
from tests.test_gpu_linear import gen, randn
from tests.test_gpu_mx4 import packed

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols", [(40, 70), (300, 1100)])
def test_codes_and_scales_in_one_row(gpu, rows, cols):
    """A gathered row that holds its codes and then its scales: one buffer, one stride."""
    x = randn(gen(1), rows, cols).to(torch.bfloat16)
    cb, sb = B.mx4_code_bytes(cols), B.mx4_scale_bytes(cols)
    both = torch.full((rows, cb + sb + 16), 0x5A, dtype=torch.uint8, device=gpu)
    at, ld = both.data_ptr(), both.stride(0)
    B.fsdp_mx4_quantize(x, rows, cols, codes=both, scales=at + cb, ldc=ld, lds=ld)
    codes, scales = Q.quantize(x.double().cpu().numpy())
    got = both.cpu().numpy()
    assert np.array_equal(got[:, :cb], codes) and np.array_equal(got[:, cb:cb + sb], scales)
    assert (got[:, cb + sb:] == 0x5A).all()
    c, s = (torch.from_numpy(t).to(gpu) for t in (codes, scales))
    v = [torch.empty(rows, cols, dtype=torch.bfloat16, device=gpu) for _ in range(2)]
    B.fsdp_mx4_dequantize(v[0], at, at + cb, rows, cols, ldc=ld, lds=ld)
    B.fsdp_mx4_dequantize(v[1], c, s, rows, cols)
    assert torch.equal(v[0], v[1])
    y = [torch.empty(rows, rows, device=gpu) for _ in range(2)]
    B.fsdp_mx4_product(y[0], at, at + cb, at, at + cb, rows, rows, cols, y_dtype="f32", lda=ld, ldas=ld, ldb=ld, ldbs=ld)
    B.fsdp_mx4_product(y[1], c, s, c, s, rows, rows, cols, y_dtype="f32")
    assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[0].t())


@pytest.mark.parametrize("m", [3, 200])
def test_masks_move_on_between_replays(gpu, m):
    n, k = 136, 300
    g = gen(2)
    a, asc, *_ = packed(g, m, k)
    b, bsc, *_ = packed(g, n, k)
    count = torch.zeros(1, dtype=torch.int64, device=gpu)
    y, eager = torch.empty(m, n, device=gpu), torch.empty(m, n, device=gpu)

    def call(out, **mask):
        B.fsdp_mx4_product(out, a.t, asc.t, b.t, bsc.t, m, n, k, y_dtype="f32", dropout=dict(p=0.5, seed=3, **mask))

    call(y, offset=10, offset_dev=count)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        count.add_(1)
        call(y, offset=10, offset_dev=count)
    seen = []
    for turn in (1, 2, 3):
        graph.replay()
        call(eager, offset=10 + turn)
        torch.cuda.synchronize()
        assert torch.equal(y, eager), turn
        seen.append(y == 0)
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m", [90, 2100])
def test_norms_of_the_parts_of_a_row(gpu, m, dtype):
    """Queries and keys side by side in a projection's rows, each normed in place
    and its gradient written in place over the residual's: the same as apart."""
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    parts, g = ((0, 128), (128, 37), (165, 259)), gen(3)
    x, dy, grad = (randn(g, m, 424).to(t) for _ in range(3))
    whole, dwhole = x.clone(), grad.clone()
    ws = torch.empty(4 << 20, dtype=torch.uint8, device=gpu)
    for first, n in parts:
        cut = slice(first, first + n)
        xs, ds, gs = (v[:, cut].contiguous() for v in (x, dy, grad))
        y, dx, rstd = torch.empty_like(xs), torch.empty_like(xs), torch.empty(m, device=gpu)
        w = randn(g, 1, n).to(t)
        dw = [torch.empty(n, device=gpu) for _ in range(2)]
        B.fsdp_norm_forward(y, xs, m, n, dtype, "rms", weight=w, w_dtype=dtype, rstd=rstd)
        B.fsdp_norm_backward(dx, ds, xs, m, n, dtype, "rms", weight=w, w_dtype=dtype, rstd=rstd, residual=gs, dw=dw[0],
                             workspace=ws)
        B.fsdp_norm_backward(dwhole[:, cut], dy[:, cut], x[:, cut], m, n, dtype, "rms", weight=w, w_dtype=dtype, rstd=rstd,
                             residual=dwhole[:, cut], dw=dw[1], workspace=ws, lddx=424, lddy=424, ldx=424, ldr=424)
        B.fsdp_norm_forward(whole[:, cut], whole[:, cut], m, n, dtype, "rms", weight=w, w_dtype=dtype, ldy=424, ldx=424)
        assert torch.equal(whole[:, cut], y) and torch.equal(dwhole[:, cut], dx) and torch.equal(dw[0], dw[1])
