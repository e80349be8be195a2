"""The 4-bit product by every way that its plan takes (tests/mx4_routes.py, where
each size's way is checked on the CPU), with sums that are exact and with NaN
blocks: 256-tiles with ragged edges, 64-tiles by two waves and by four, parts of
the contraction, and outputs cut by columns and by rows."""

import numpy as np
import pytest
import torch

from oracle import mx4 as Q
from rank_step_amd import binding as B
from tests.mx4_routes import ROUTES
from tests.test_gpu_linear import gen
from tests.test_gpu_mx4 import Bytes, packed

pytestmark = pytest.mark.gpu


def whole_quarters(r, rows, k):
    """Codes of magnitudes 0 to 1.5 and scales of 1, 2 and 4: products are multiples of 1/4."""
    kb, ks = Q.code_bytes(k), Q.scale_bytes(k)
    flat = r.integers(0, 16, (rows, kb * 2), dtype=np.uint8)
    flat = np.where(flat & 7 > 3, flat & 8 | 1, flat)
    flat[:, k:] = 0
    scales = np.zeros((rows, ks), np.uint8)
    scales[:, :kb // 16] = r.integers(127, 130, (rows, kb // 16))
    return flat[:, 0::2] | flat[:, 1::2] << 4, scales


@pytest.mark.parametrize("m,n,k,workspace,way", ROUTES)
def test_exact_sums(gpu, m, n, k, workspace, way):
    """Every sum of magnitudes is under 2^22, so in any order exact in fp32; one
    wrong element or scale shows."""
    r = np.random.default_rng(m + n + k)
    (a, asc), (b, bsc) = whole_quarters(r, m, k), whole_quarters(r, n, k)
    x, w = (torch.from_numpy(Q.values(c, s, k)).cuda() for c, s in ((a, asc), (b, bsc)))
    assert (x.abs().sum(dim=1).max() * w.abs().max()).item() < 2 ** 22
    want = x @ w.T
    ws = torch.empty(workspace, dtype=torch.uint8, device=gpu) if workspace else None
    a, asc, b, bsc = (torch.from_numpy(v).cuda() for v in (a, asc, b, bsc))
    y = torch.full((m, n), float("nan"), device=gpu)
    B.fsdp_mx4_product(y, a, asc, b, bsc, m, n, k, y_dtype="f32", workspace=ws)
    assert torch.equal(y.double(), want)


@pytest.mark.parametrize("m,n,k,workspace,way", ROUTES)
def test_nan_blocks(gpu, m, n, k, workspace, way):
    """One in A's last row and last block, one in B's last row, others in B's first
    and in the middle of both."""
    g = gen(m)
    a, asc, *_ = packed(g, m, k)
    b, bsc, *_ = packed(g, n, k)
    last = Q.code_bytes(k) // 16 - 1
    want = torch.zeros(m, n, dtype=torch.bool, device=gpu)
    if m > 1:
        for row, block in ((m - 1, last), (m // 2, last // 2)):
            asc.t[row, block], want[row] = 255, True
    for row, block in ((n - 1, last), (n // 2, last // 2), (0, 0)):
        bsc.t[row, block], want[:, row] = 255, True
    ws = torch.empty(workspace, dtype=torch.uint8, device=gpu) if workspace else None
    y = torch.empty(m, n, device=gpu)
    B.fsdp_mx4_product(y, a.t, asc.t, b.t, bsc.t, m, n, k, y_dtype="f32", workspace=ws)
    assert torch.equal(y.isnan(), want)


@pytest.mark.parametrize("m,n", [(1, 1), (17, 40), (200, 130)])
def test_the_longest_contraction(gpu, m, n):
    """2^23 ones, by few rows and by 64-tiles in parts and not: exact in fp32."""
    k = 1 << 23
    a, b = (Bytes(rows, Q.code_bytes(k)) for rows in (m, n))
    asc, bsc = (Bytes(rows, Q.scale_bytes(k)) for rows in (m, n))
    for t, v in ((a, 0x22), (b, 0x22), (asc, 127), (bsc, 127)):
        t.t.fill_(v)
    for ws in (torch.empty(B.MX4_WORKSPACE_BYTES, dtype=torch.uint8, device=gpu), None):
        y = torch.empty(m, n, device=gpu)
        B.fsdp_mx4_product(y, a.ptr, asc.ptr, b.ptr, bsc.ptr, m, n, k, y_dtype="f32", workspace=ws)
        assert bool((y == k).all())
