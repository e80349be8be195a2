"""The 4-bit layer over ranks that each quantise their rows of the weight: the
gathered copy is the whole weight's, byte for byte; the transposes' pieces are
operands of their own, whose products add up to the input gradient.

Tolerance: each piece's product is off by tests/test_gpu_mx4.py's bound, with a
rounding to fp32 of what has been added so far."""

import numpy as np
import pytest
import torch

from oracle import mx4 as Q
from rank_step_amd import binding as B
from tests.test_gpu_linear import U, gen, randn
from tests.test_gpu_mx4 import product_err, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ranks,own,k,m", [(4, 43, 100, 17), (8, 1376, 512, 300), (2, 512, 1100, 5)])
def test_ranks_copies(gpu, ranks, own, k, m):
    g, n = gen(ranks), ranks * own
    bytes_ = lambda rows, cols: (torch.empty(rows, f(cols), dtype=torch.uint8, device=gpu)  # noqa: E731
                                 for f in (B.mx4_code_bytes, B.mx4_scale_bytes))
    weight, dz = randn(g, n, k, 0.05), randn(g, m, n, 0.1).to(torch.bfloat16)
    ws = torch.empty(B.MX4_WORKSPACE_BYTES, dtype=torch.uint8, device=gpu)
    codes, scales = bytes_(n, k)
    pieces = []
    for r in range(ranks):
        rows = slice(r * own, (r + 1) * own)
        pieces.append(tuple(bytes_(k, own)))
        B.fsdp_mx4_quantize(weight[rows], own, k, "f32", codes[rows], scales[rows], *pieces[-1])
    whole, whole_scales = bytes_(n, k)
    B.fsdp_mx4_quantize(weight, n, k, "f32", whole, whole_scales)
    assert torch.equal(codes, whole) and torch.equal(scales, whole_scales)

    # dx = sum over the ranks' rows of dz's columns times them
    dx = torch.zeros(m, k, device=gpu)
    dcodes, dscales = bytes_(m, own)
    want, err, dzv, wv = 0.0, 0.0, dz.double().cpu().numpy(), weight.double().cpu().numpy()
    for r, (ct, st) in enumerate(pieces):
        B.fsdp_mx4_quantize(dz[:, r * own:], m, own, "bf16", dcodes, dscales, ldx=n)
        B.fsdp_mx4_product(dx, dcodes, dscales, ct, st, m, k, own, y_dtype="f32", residual=dx, workspace=ws)
        cols = slice(r * own, (r + 1) * own)
        a, b = Q.quantize(np.ascontiguousarray(dzv[:, cols])), Q.quantize(np.ascontiguousarray(wv[cols].T))
        assert np.array_equal(ct.cpu().numpy(), b[0]) and np.array_equal(st.cpu().numpy(), b[1])
        part, s, room = reference(*a, *b, own)
        want = want + part
        err = err + product_err(own, s, room) + 2 * U * np.abs(want)
    assert np.all(np.abs(dx.double().cpu().numpy() - want) <= err)
