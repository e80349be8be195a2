"""The 4-bit product by every way that its plan takes (tests/mx4_routes.py; that
each size takes the way that is named is checked on the CPU)."""

import pytest
import torch

from tests.mx4_routes import ROUTES
from tests.test_gpu_mx4 import check_product

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,k,workspace,way", ROUTES)
def test_way(gpu, m, n, k, workspace, way):
    ws = torch.empty(workspace, dtype=torch.uint8, device=gpu) if workspace else None
    check_product(m, n, k, ws, act="silu", bias=True, res=True, keep_z=True, p=0.1)
    check_product(m, n, k, ws, yt="f32", pad=1)
