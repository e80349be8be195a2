"""The linear layer's calls on the GPU against the float64 oracle.

Each input lies in a buffer whose other elements (before it, after it, and
between its rows) are NaN, so that reading one shows; each output in a buffer
of a fixed pattern that must be whole outside the output afterwards.

Tolerances, with u = 2^-24 (half an fp32 step):

* a product of length l: the matrix instructions add 32 terms at a time, and
  a product may be joined from up to 64 parts, so a term passes through at
  most l/32 + 32 + 64 + 8 additions, each off by a whole step (2u) of a
  partial sum that is at most S, the sum of the terms' magnitudes;
* the division by a scale as a product with a rounded reciprocal: 2u each;
* activations: relative errors (in units of u) of 16 + 2 z^2 for gelu (its
  fit's 4.4e-7 is 7.4u, the rounding of z^2 in the exponent, the hardware's
  exponential and reciprocal at 2u) and 16 + 2 |z| for silu, on the magnitudes
  that form the value, and a slope of at most 1.13 on z's own error;
* 2u for each of the mask's factor, the residual's sum and the store;
* half a step of the output's type: 2^-8 of the value for bf16;
* 129 * 2^-126 (1.5e-36) absolute: the hardware's exponential and reciprocal
  give 0 for results under 2^-126.  That happens to exp(-|z|) (or its inverse's
  reciprocal) for |z| > 87.3 and to exp(-z^2/2) for |z| > 13.2; the value it
  forms is off by at most (1 + |z|) 2^-126, and from |z| = 128 on the true
  value, at most (1 + |z|) exp(-|z|) < 2^-177, is below that anyway.
"""

import itertools

import numpy as np
import pytest
import torch

from oracle import fp8 as F8
from oracle import linear as OL
from rank_step_amd import binding as B
from tests.linear_routes import ROUTES

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
FLUSHED = 129 * 2.0 ** -126
HALF = {"bf16": 2.0 ** -8, "f32": U}
TT = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.uint8}
BITS = {"bf16": torch.int16, "f32": torch.int32, "e4m3": torch.uint8}
PATTERN = {"bf16": 0x1234, "f32": 0x12345678}


class Mat:
    """A matrix inside a larger buffer: `off` elements in, rows `ld` apart."""

    def __init__(self, rows, cols, dtype, values=None, off=0, pad=0, dev="cuda"):
        self.rows, self.cols, self.dtype, self.off, self.ld = rows, cols, dtype, off, cols + pad
        n = off + rows * self.ld + 24
        if values is None:
            self.buf = torch.full((n,), PATTERN[dtype], dtype=BITS[dtype], device=dev).view(TT[dtype])
        elif dtype == "e4m3":
            self.buf = torch.full((n,), 0x7F, dtype=torch.uint8, device=dev)  # NaN codes
        else:
            self.buf = torch.full((n,), float("nan"), dtype=TT[dtype], device=dev)
        self.t = self.buf[off:off + rows * self.ld].view(rows, self.ld)[:, :cols]
        if values is not None:
            self.t.copy_(values)

    @property
    def ptr(self):
        return self.buf.data_ptr() + self.off * self.buf.element_size()

    def np(self):
        if self.dtype == "e4m3":
            return F8.e4m3_value(self.t.cpu().numpy())
        return self.t.double().cpu().numpy()

    def check_surroundings(self):
        b = self.buf.view(BITS[self.dtype]).clone()
        b[self.off:self.off + self.rows * self.ld].view(self.rows, self.ld)[:, :self.cols] = PATTERN[self.dtype]
        assert bool((b == PATTERN[self.dtype]).all()), "written outside the output"


def close(got, ref, err, dtype, what):
    tol = err + HALF[dtype] * (np.abs(ref) + err) + FLUSHED
    off = np.abs(got - ref) / tol
    bad = ~(off <= 1)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, worst {np.nanmax(off):.3g} at "
                           f"{np.argwhere(bad)[0].tolist()}, {got[bad][0]} against {ref[bad][0]}")


def product(a, b):
    """The oracle's product; the same two sums by the GPU in float64 where the host would take seconds."""
    if a.shape[0] * b.shape[0] * a.shape[1] < 3e8:
        return OL.product(a, b)
    x, y = (torch.from_numpy(np.ascontiguousarray(v)).cuda() for v in (a, b.T))
    return (x @ y).cpu().numpy(), (x.abs() @ y.abs()).cpu().numpy()


def product_err(length, s):
    return (length / 32 + 104) * 2 * U * s


def act_err(z, ez, name):
    a = np.abs(OL.act(z, name))
    rel = {"none": 0.0, "relu": 0.0, "gelu": 16 + 2 * z * z, "silu": 16 + 2 * np.abs(z)}[name]
    return 1.13 * ez + a * rel * U


def grad_rel(z, name):
    return {"none": 0.0, "relu": 0.0, "gelu": 16 + 2 * z * z, "silu": 32 + 4 * np.abs(z)}[name] * U


@pytest.fixture(scope="module")
def space(gpu):
    return torch.empty(B.LINEAR_WORKSPACE_BYTES, dtype=torch.uint8, device=gpu)


def randn(g, rows, cols, std=1.0):
    return torch.randn(rows, cols, generator=g, device="cuda") * std


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def weight(g, n, k, dtype, off, pad):
    """(matrix, scale tensor or None, float64 values)"""
    v = randn(g, n, k, 0.1)
    if dtype == "bf16":
        w = Mat(n, k, dtype, v, off, pad)
        return w, None, w.np()
    scale = (448.0 / v.abs().max().clamp(min=1e-12)).reshape(1) if v.numel() else torch.ones(1, device="cuda")
    codes = (v * scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    w = Mat(n, k, dtype, codes, off, pad)
    return w, scale, w.np() / float(scale)


def check_forward(m, n, k, space, wt="bf16", yt="bf16", act="none", bias=False, res=False, keep_z=False, p=0.0,
                  off=0, pad=0, seed=1, same=False, offset_dev=None):
    g = gen(seed)
    x = Mat(m, k, "bf16", randn(g, m, k), off, pad)
    w, scale, wv = weight(g, n, k, wt, off, pad)
    b = Mat(1, n, "bf16", randn(g, 1, n), off) if bias else None
    r = Mat(m, n, yt, randn(g, m, n), off, pad) if res else None
    y = r if same else Mat(m, n, yt, None, off, pad)
    z = Mat(m, n, "bf16", None, off, pad) if keep_z else None
    d = dict(p=p, seed=0xFEDCBA9876543210 + seed, offset=(1 << 35) + seed) if p else None
    rv = r.np() if res else 0.0
    B.fsdp_linear_forward(y.ptr, x.ptr, w.ptr, m, n, k, w_dtype=wt, w_scale=scale, y_dtype=yt,
                          bias=b.ptr if bias else None, residual=r.ptr if res else None, act=act,
                          z=z.ptr if keep_z else None, dropout=d, workspace=space, ldy=y.ld, ldx=x.ld, ldw=w.ld,
                          ldr=r.ld if res else None, ldz=z.ld if keep_z else None)
    torch.cuda.synchronize()
    zv, s = product(x.np(), wv)
    if bias:
        zv = zv + b.np()
    ez = product_err(k, s) + 4 * U * (s + np.abs(zv))
    if keep_z:
        close(z.np(), zv, ez, "bf16", "z")
        z.check_surroundings()
    f = OL.keep_factor(m, n, p, d["seed"], d["offset"]) if p else 1.0
    yv = OL.act(zv, act) * f
    ey = act_err(zv, ez, act) * f + 2 * U * np.abs(yv)
    yv = yv + rv
    close(y.np(), yv, ey + 2 * U * np.abs(yv), yt, "y")
    if not same:
        y.check_surroundings()
    return y


# one and few tokens, sizes under, at and over the tiles, odd ones, a long product over few tiles, many tiles
SHAPES = [(1, 1, 1), (1, 64, 64), (1, 512, 1365), (1, 96, 4096), (3, 8, 8), (7, 33, 65), (16, 256, 512), (17, 130, 72), (31, 100, 999),
          (33, 64, 128), (64, 64, 4096), (65, 40, 2056), (100, 1024, 17), (128, 128, 128), (129, 257, 191),
          (300, 264, 520), (257, 1000, 1365), (512, 384, 64)]
BIG = [(4096, 2048, 192), (4001, 2056, 200)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("wt", ["bf16", "e4m3"])
def test_forward_shapes(gpu, space, m, n, k, wt):
    check_forward(m, n, k, space, wt)
    check_forward(m, n, k, space, wt, yt="f32", act="silu", bias=True, res=True, keep_z=True, p=0.25)
    check_forward(m, n, k, None, wt, act="gelu", bias=True, off=3, pad=5, keep_z=True)


@pytest.mark.parametrize("m", [1, 16, 30])
@pytest.mark.parametrize("wt", ["bf16", "e4m3"])
@pytest.mark.parametrize("k", [64 * 8 * 15 + 64 * 5 + 40, 64 * 8 * 7 + 8, 64 * 8 * 3, 64 * 9])
def test_few_tokens_by_batches_of_chunks(gpu, space, m, wt, k):
    """Contractions that leave each wave chunks for every size of batch, and a part of one."""
    check_forward(m, 40, k, space, wt, bias=True)
    check_forward(m, 70, k - 3, space, wt, off=1, pad=1, yt="f32")


@pytest.mark.parametrize("m,n,k", BIG)
def test_forward_many_tiles(gpu, space, m, n, k):
    check_forward(m, n, k, space, act="gelu", bias=True, res=True, keep_z=True, p=0.1)
    check_forward(m, n, k, space, "e4m3", yt="f32")


# Sizes for each way to compute a product: 256-tiles (ragged in every length),
# 128-tiles, 64-tiles, split ones, and ones that are cut after their whole
# rounds of 256-tiles, by columns and by rows.
WAYS = [(4000, 4080, 1008), (2048, 2064, 336), (520, 1040, 1008), (300, 128, 8208), (4096, 4112, 1024), (4104, 4096, 1024)]


@pytest.mark.parametrize("m,n,k", WAYS)
def test_ways(gpu, space, m, n, k):
    check_forward(m, n, k, space, act="silu", bias=True, res=True, keep_z=True, p=0.1)
    check_forward(m, n, k, space, "e4m3", yt="f32", res=True, same=True, p=0.5)
    check_grad_input(m, k, n, space)
    check_grad_input(m, k, n, space, "e4m3")
    check_grad_weight(k, m, n, space, "bf16", True)
    check_grad_weight(k, m, n, space, "f32", False)


@pytest.mark.parametrize("m,n,k", [(300, 1000, 1365), (600, 1543, 515), (64, 100, 333)])
@pytest.mark.parametrize("size", [0, 1 << 10, 600 << 10, 1 << 20, 2 << 20, 5 << 20])
def test_small_workspaces(gpu, m, n, k, size):
    """Operands that have to be laid out anew, with room for neither, for some
    of their columns at a time, for one, for both; what lies behind the
    workspace stays."""
    buf = torch.full((size + 64,), 0x5A, dtype=torch.uint8, device=gpu)
    ws = buf[:size] if size else None
    check_forward(m, n, k, ws, act="gelu", bias=True, res=True, keep_z=True, p=0.2)
    check_forward(m, n, k, ws, "e4m3", off=3, pad=2)
    check_grad_input(m, n, k, ws, "e4m3")
    check_grad_input(m, n, k, ws, off=1)
    check_grad_weight(m, n, k, ws, "f32", True)
    check_backward(m, n, ws, "silu", 0.1)
    assert bool((buf[size:] == 0x5A).all())


@pytest.mark.parametrize("mib", [24, 33, 48])
def test_unaligned_products_in_pieces(gpu, mib):
    """Large unaligned operands of which neither fits in the workspace: the output
    in pieces of rows and columns, each with its part of every epilogue operand."""
    size = mib << 20
    buf = torch.full((size + 64,), 0x5A, dtype=torch.uint8, device=gpu)
    ws = buf[:size]
    check_forward(2999, 2901, 8191, ws, act="silu", bias=True, res=True, keep_z=True, p=0.3)
    check_forward(2999, 2901, 8191, ws, "e4m3", yt="f32", bias=True, res=True, same=True, p=0.2, off=1)
    check_grad_input(2999, 8191, 2901, ws)
    check_grad_input(2999, 8191, 2901, ws, "e4m3", off=3, pad=1)
    check_grad_weight(8191, 2999, 2901, ws, "f32", True)
    assert bool((buf[size:] == 0x5A).all())


@pytest.mark.parametrize("act,bias,res,keep_z,p,yt", [
    c for i, c in enumerate(itertools.product(["none", "relu", "gelu", "silu"], [False, True], [False, True],
                                              [False, True], [0.0, 0.5], ["bf16", "f32"])) if i % 5 == 0])
def test_forward_epilogues(gpu, space, act, bias, res, keep_z, p, yt):
    check_forward(40, 72, 136, space, act=act, bias=bias, res=res, keep_z=keep_z, p=p, yt=yt)
    check_forward(2, 72, 136, space, act=act, bias=bias, res=res, keep_z=keep_z, p=p, yt=yt)
    check_forward(9, 65, 4096, space, act=act, bias=bias, res=res, keep_z=keep_z, p=p, yt=yt, off=1, pad=2)


@pytest.mark.parametrize("m,n,k", [(5, 64, 64), (40, 72, 136), (33, 64, 4096), (4096, 2048, 64)])
@pytest.mark.parametrize("yt", ["bf16", "f32"])
def test_forward_residual_in_place(gpu, space, m, n, k, yt):
    check_forward(m, n, k, space, yt=yt, act="relu", res=True, same=True, p=0.3)


@pytest.mark.parametrize("off,pad", [(0, 8), (8, 0), (1, 0), (0, 1), (4, 4), (7, 9), (8, 64)])
@pytest.mark.parametrize("wt", ["bf16", "e4m3"])
def test_views(gpu, space, off, pad, wt):
    for m, n, k in ((3, 128, 256), (70, 136, 264)):
        check_forward(m, n, k, space, wt, bias=True, res=True, keep_z=True, off=off, pad=pad)
        check_grad_input(m, n, k, space, wt, off, pad)
        check_grad_weight(m, n, k, space, "bf16", True, off, pad)


@pytest.mark.parametrize("m", [1, 20, 130])
def test_empty_product(gpu, space, m):
    """k = 0: the epilogue of zero.  The weight gradient of no tokens."""
    n = 70
    b = randn(gen(1), 1, n).to(torch.bfloat16)
    y = Mat(m, n, "f32")
    B.fsdp_linear_forward(y.ptr, None, None, m, n, 0, y_dtype="f32", bias=b, act="relu", workspace=space)
    torch.cuda.synchronize()
    assert np.array_equal(y.np(), np.broadcast_to(np.maximum(b.double().cpu().numpy(), 0), (m, n)))
    dx = Mat(m, n, "bf16")
    B.fsdp_linear_grad_input(dx.ptr, None, None, m, 0, n, workspace=space)
    for add in (False, True):
        dw = Mat(m, n, "f32", randn(gen(2), m, n))
        old = dw.np()
        B.fsdp_linear_grad_weight(dw.ptr, None, None, 0, m, n, dw_dtype="f32", accumulate=add, workspace=space)
        torch.cuda.synchronize()
        assert np.array_equal(dw.np(), old if add else np.zeros_like(old))
    assert not dx.np().any()
    db = torch.full((n,), 3.0, device=gpu)
    B.fsdp_linear_epilogue_backward(None, None, 0, n, db=db)
    torch.cuda.synchronize()
    assert not db.any()


@pytest.mark.parametrize("m,n,k", [(4, 64, 64), (40, 100, 200), (64, 40, 4096)])
def test_nonfinite_values_stay_in_their_rows(gpu, space, m, n, k):
    """NaN and Inf in one token or one weight row reach that row or column
    only, and dropped elements are +0 whatever they held."""
    g = gen(7)
    x, w = randn(g, m, k).to(torch.bfloat16), randn(g, n, k).to(torch.bfloat16)
    x[1, 3] = float("nan")
    x[2, k - 1] = float("inf")
    w[5, 0] = float("nan")
    y = torch.empty(m, n, dtype=torch.bfloat16, device=gpu)
    d = dict(p=0.5, seed=3, offset=4)
    B.fsdp_linear_forward(y, x, w, m, n, k, dropout=d, workspace=space)
    keep = OL.keep_factor(m, n, **d) > 0
    v = y.float().cpu().numpy()
    odd = np.zeros((m, n), bool)
    odd[1:3] = True
    odd[:, 5] = True
    assert np.isnan(v[1][keep[1]]).all() and not np.isfinite(v[2][keep[2]]).any()
    assert np.isnan(v[:, 5][keep[:, 5]]).all()
    assert np.isfinite(v[~odd]).all()
    assert not v[~keep].any() and not np.signbit(v[~keep]).any()


def test_every_e4m3_code(gpu, space):
    """Each of the 256 codes against a one-hot token: exact in fp32, by the
    one-token path and by tiles."""
    codes = torch.arange(256, dtype=torch.uint8, device=gpu).reshape(1, 256).repeat(8, 1).contiguous()
    scale = torch.full((1,), 4.0, device=gpu)
    want = F8.e4m3_value(np.arange(256)) / 4.0
    x = torch.eye(256, device=gpu).to(torch.bfloat16)
    for rows in (256, 1):
        for first in range(0, 256, rows):
            finite = ~np.isnan(want)
            # NaN times 0 is NaN: those codes are taken out of the others' sums
            c = codes.clone()
            c[:, ~torch.from_numpy(finite).to(gpu)] = 0
            y = torch.empty(rows, 8, device=gpu)
            B.fsdp_linear_forward(y, x[first:first + rows], c, rows, 8, 256, w_dtype="e4m3", w_scale=scale,
                                  y_dtype="f32", workspace=space)
            got = y.double().cpu().numpy()
            for i in range(rows):
                assert (got[i] == (want[first + i] if finite[first + i] else 0.0)).all()
    y = torch.empty(1, 8, device=gpu)
    B.fsdp_linear_forward(y, x[:1], codes, 1, 8, 256, w_dtype="e4m3", w_scale=scale, y_dtype="f32")
    assert bool(y.isnan().all())
    # as the right operand of the input gradient
    dz = torch.zeros(1, 8, dtype=torch.bfloat16, device=gpu)
    dz[0, 2] = 1.0
    codes[:, 0x7F] = 0
    codes[:, 0xFF] = 0
    dx = torch.empty(1, 256, dtype=torch.bfloat16, device=gpu)
    B.fsdp_linear_grad_input(dx, dz, codes, 1, 8, 256, w_dtype="e4m3", w_scale=scale)
    assert np.array_equal(dx.double().cpu().numpy()[0], np.where(np.isnan(want), 0, want))


@pytest.mark.parametrize("scale", [3.0, 448.0 / 1e-12, 448.0 / 3.38e38, 0.7])
def test_e4m3_scale_is_a_product_with_its_reciprocal(gpu, space, scale):
    """One code a sum, so the only roundings are the reciprocal's and the product's."""
    codes = torch.arange(0, 0x7F, dtype=torch.uint8, device=gpu).reshape(1, -1).repeat(16, 1).contiguous()
    k = codes.shape[1]
    s = torch.full((1,), scale, device=gpu)
    recip = np.float32(1) / np.float32(s.item())
    want = F8.e4m3_value(np.arange(k)).astype(np.float32) * recip
    for m in (16, k):  # few tokens, and tiles
        x = torch.eye(m, k, device=gpu).bfloat16()
        y = torch.empty(m, 16, device=gpu)
        B.fsdp_linear_forward(y, x, codes, m, 16, k, w_dtype="e4m3", w_scale=s, y_dtype="f32", workspace=space)
        assert np.array_equal(y.cpu().numpy(), np.repeat(want[:m, None], 16, 1))
    dx = torch.empty(16, k, dtype=torch.bfloat16, device=gpu)
    B.fsdp_linear_grad_input(dx, torch.eye(16, device=gpu).bfloat16(), codes, 16, 16, k, w_dtype="e4m3", w_scale=s,
                             workspace=space)
    assert torch.equal(dx, torch.from_numpy(want).to(gpu).bfloat16().expand(16, k))


def test_subnormal_values(gpu, space):
    """bf16 operands under 2^-126 count as what they are, and an fp32 output under it is kept."""
    x = torch.zeros(40, 64, dtype=torch.bfloat16, device=gpu)
    w = torch.zeros(64, 64, dtype=torch.bfloat16, device=gpu)
    for i in range(40):
        x[i, i] = 2.0 ** -(94 + i)  # 2^-133 is bf16's least
    w[torch.arange(64), torch.arange(64)] = 2.0 ** 100
    for m in (3, 40):
        y = torch.empty(m, 64, device=gpu)
        B.fsdp_linear_forward(y, x[40 - m:], w, m, 64, 64, y_dtype="f32", workspace=space)
        want = torch.zeros_like(y)
        for i in range(m):
            want[i, 40 - m + i] = 2.0 ** (6 - (40 - m + i))
        assert torch.equal(y, want), (m, (y != want).nonzero()[:4].tolist())


# ---------------------------------------------------------------- gradients

def check_grad_input(m, n, k, space, wt="bf16", off=0, pad=0, seed=2):
    g = gen(seed)
    dz = Mat(m, n, "bf16", randn(g, m, n), off, pad)
    w, scale, wv = weight(g, n, k, wt, off, pad)
    dx = Mat(m, k, "bf16", None, off, pad)
    B.fsdp_linear_grad_input(dx.ptr, dz.ptr, w.ptr, m, n, k, w_dtype=wt, w_scale=scale, workspace=space,
                             lddx=dx.ld, lddz=dz.ld, ldw=w.ld)
    torch.cuda.synchronize()
    v, s = product(dz.np(), wv.T)
    close(dx.np(), v, product_err(n, s) + 4 * U * s, "bf16", "dx")
    dx.check_surroundings()


def check_grad_weight(m, n, k, space, dt="bf16", add=False, off=0, pad=0, seed=3):
    g = gen(seed)
    dz = Mat(m, n, "bf16", randn(g, m, n), off, pad)
    x = Mat(m, k, "bf16", randn(g, m, k), off, pad)
    dw = Mat(n, k, dt, None, off, pad)
    old = 0.0
    if add:
        dw.t.copy_(randn(g, n, k))
        old = dw.np()
    B.fsdp_linear_grad_weight(dw.ptr, dz.ptr, x.ptr, m, n, k, dw_dtype=dt, accumulate=add, workspace=space,
                              lddw=dw.ld, lddz=dz.ld, ldx=x.ld)
    torch.cuda.synchronize()
    v, s = product(dz.np().T, x.np().T)
    close(dw.np(), v + old, product_err(m, s) + 2 * U * np.abs(v + old), dt, "dw")
    dw.check_surroundings()


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gradient_shapes(gpu, space, m, n, k):
    for wt in ("bf16", "e4m3"):
        check_grad_input(m, n, k, space, wt)
        check_grad_input(m, k, n, None, wt, off=5, pad=3)
    for dt, add in (("bf16", False), ("bf16", True), ("f32", False), ("f32", True)):
        check_grad_weight(m, n, k, space, dt, add)
    check_grad_weight(k, n, m, None, "f32", True, off=5, pad=3)


@pytest.mark.parametrize("m,n,k", BIG)
def test_gradients_many_tiles(gpu, space, m, n, k):
    check_grad_input(m, k, n, space)
    check_grad_input(m, k, n, space, "e4m3")
    check_grad_weight(k, m, n, space, "bf16", True)
    check_grad_weight(k, m, n, space, "f32", False)


def check_backward(m, n, space, act="none", p=0.0, db="f32", add=False, dz=True, off=0, pad=0, seed=4, same=None):
    g = gen(seed)
    dy = Mat(m, n, "bf16", randn(g, m, n), off, pad)
    z = Mat(m, n, "bf16", randn(g, m, n, 2.0), off, pad) if act != "none" else None
    if z is not None and m > 1:
        z.t[0, 0] = 0.0
    out = {None: lambda: Mat(m, n, "bf16", None, off, pad), "dy": lambda: dy, "z": lambda: z}[same]() if dz else None
    s = Mat(1, n, db, None, off) if db else None
    old = 0.0
    if add:
        s.t.copy_(randn(g, 1, n))
        old = s.np()
    d = dict(p=p, seed=77 + seed, offset=1 << 63) if p else None
    dyv, zv = dy.np(), z.np() if z is not None else np.zeros((m, n))
    B.fsdp_linear_epilogue_backward(out.ptr if dz else None, dy.ptr, m, n, z=z.ptr if z is not None else None,
                                    act=act, dropout=d, db=s.ptr if db else None, db_dtype=db or "f32",
                                    accumulate=add, workspace=space, lddz=out.ld if dz else None, lddy=dy.ld,
                                    ldz=z.ld if z is not None else None)
    torch.cuda.synchronize()
    f = OL.keep_factor(m, n, p, d["seed"], d["offset"]) if p else 1.0
    v = dyv * f * OL.act_grad(zv, act)
    e = np.abs(dyv) * f * OL.act_grad_slack(zv, act) * (grad_rel(zv, act) + 4 * U)
    if dz:
        close(out.np(), v, e, "bf16", "dz")
        if same is None:
            out.check_surroundings()
    if db:
        e = e.sum(0) + (m + 72) * U * np.abs(v).sum(0)
        close(s.np(), v.sum(0, keepdims=True) + old, e + 2 * U * np.abs(v.sum(0) + old), db, "db")
        s.check_surroundings()


@pytest.mark.parametrize("m,n", [(1, 1), (1, 1000), (2, 7), (5, 8), (37, 251), (64, 512), (333, 1024), (1000, 40),
                                 (2049, 9), (700, 4100), (100, 520)])
def test_epilogue_backward_shapes(gpu, space, m, n):
    check_backward(m, n, space, "gelu", 0.1)
    check_backward(m, n, space, "silu", 0.0, "bf16", True, off=3, pad=5)
    check_backward(m, n, None, "relu", 0.5, "f32", True)
    check_backward(m, n, space, "none", 0.5, None)
    check_backward(m, n, space, "none", 0.0, "f32", dz=False)


@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
@pytest.mark.parametrize("same", ["dy", "z"])
def test_epilogue_backward_in_place(gpu, space, act, same):
    check_backward(130, 523, space, act, 0.2, same=same)


def test_epilogue_backward_selects(gpu, space):
    """Dropped elements and relu's flat side give 0 whatever dy holds there."""
    m, n = 40, 100
    z = randn(gen(1), m, n).to(torch.bfloat16)
    d = dict(p=0.5, seed=5, offset=6)
    keep = torch.from_numpy(OL.keep_factor(m, n, **d) > 0).to(gpu) & (z > 0)
    dy = torch.where(keep, torch.ones_like(z), torch.full_like(z, float("nan")))
    dz, db = torch.empty_like(z), torch.empty(n, device=gpu)
    B.fsdp_linear_epilogue_backward(dz, dy, m, n, z=z, act="relu", dropout=d, db=db, workspace=space)
    assert torch.equal(dz, torch.where(keep, 2 * torch.ones_like(z), torch.zeros_like(z)))
    assert torch.equal(db, 2 * keep.sum(0).float())


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("rows", [40, 600])
def test_epilogue_backward_drops_whatever_z_holds(gpu, space, act, rows):
    """The forward call drops an element whose z is not finite to +0; so does its gradient."""
    n = 100
    d = dict(p=0.5, seed=8, offset=9)
    keep = torch.from_numpy(OL.keep_factor(rows, n, **d) > 0).to(gpu)
    for bad in ("nan", "inf", "-inf"):
        z = torch.where(keep, torch.zeros(rows, n, device=gpu), torch.full((rows, n), float(bad), device=gpu))
        z = z.to(torch.bfloat16)
        dy = torch.where(keep, torch.ones_like(z), torch.full_like(z, float("-inf")))
        dz, db = torch.empty_like(z), torch.empty(n, device=gpu)
        B.fsdp_linear_epilogue_backward(dz, dy, rows, n, z=z, act=act, dropout=d, db=db, workspace=space)
        slope = {"none": 1.0, "relu": 0.0}.get(act, 0.5)  # at 0; times the scale 2
        assert torch.equal(dz, torch.where(keep, torch.full_like(z, 2 * slope), torch.zeros_like(z)))
        # a slope is off by less than 2^-20 (far below dz's rounding), each of `rows` sums by 2^-24
        want = 2 * slope * keep.sum(0).double()
        assert bool(((db.double() - want).abs() <= want * (2.0 ** -20 + rows * 2.0 ** -24)).all())


@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
@pytest.mark.parametrize("rows", [40, 600])
def test_epilogue_backward_nan_of_z_stays(gpu, space, act, rows):
    """A kept element whose z is NaN has a NaN gradient, and its column a NaN sum; no other."""
    n = 100
    z = randn(gen(11), rows, n).to(torch.bfloat16)
    hit = torch.zeros(rows, n, dtype=torch.bool, device=gpu)
    hit[3, 5] = hit[rows - 1, 99] = hit[rows // 2, 64:70] = True
    z[hit] = float("nan")
    dy = torch.ones_like(z)
    for d in (None, dict(p=0.5, seed=12, offset=13)):
        keep = torch.ones_like(hit) if d is None else torch.from_numpy(OL.keep_factor(rows, n, **d) > 0).to(gpu)
        dz, db = torch.empty_like(z), torch.empty(n, device=gpu)
        B.fsdp_linear_epilogue_backward(dz, dy, rows, n, z=z, act=act, dropout=d, db=db, workspace=space)
        assert torch.equal(dz.isnan(), hit & keep)
        assert torch.equal(db.isnan(), (hit & keep).any(0))


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_activation_range(gpu, space, act):
    """The whole range of z: bf16 values from the smallest to the largest."""
    z = torch.arange(0, 0x7F80, device=gpu, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    z = torch.cat([z, -z]).reshape(2, -1).contiguous()
    m, n = z.shape
    zv = z.double().cpu().numpy()
    dz, dy = torch.empty_like(z), torch.ones_like(z)
    B.fsdp_linear_epilogue_backward(dz, dy, m, n, z=z, act=act)
    got, ref = dz.double().cpu().numpy(), OL.act_grad(zv, act)
    assert np.isfinite(got).all()
    close(got, ref, OL.act_grad_slack(zv, act) * np.minimum(grad_rel(zv, act) + 4 * U, 1.0), "bf16", "slope")
    # forward, through a product with 1
    y, one = torch.empty(m * n, 1, device=gpu), torch.ones(1, 1, dtype=torch.bfloat16, device=gpu)
    B.fsdp_linear_forward(y, z, one, m * n, 1, 1, y_dtype="f32", act=act)
    got, zv = y.double().cpu().numpy()[:, 0], zv.reshape(-1)
    err = np.minimum(act_err(zv, 0.0, act), np.abs(OL.act(zv, act)))
    assert np.isfinite(got).all()
    close(got, OL.act(zv, act), err, "f32", "activation")


# ---------------------------------------------------------------- dropout

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 9), (3, 8), (37, 251), (5, 4099), (260, 64), (1000, 24)])
def test_dropout(gpu, dtype, rows, cols):
    for p, res, off, pad in ((0.5, False, 0, 0), (0.1, True, 3, 7), (0.0, True, 0, 8), (1.0, False, 1, 0),
                             (2.0 ** -16, False, 0, 0)):
        g = gen(9)
        x = Mat(rows, cols, dtype, randn(g, rows, cols), off, pad)
        r = Mat(rows, cols, dtype, randn(g, rows, cols), off, pad) if res else None
        y = Mat(rows, cols, dtype, None, off, pad)
        d = dict(p=p, seed=(1 << 64) - 5, offset=12)
        B.fsdp_dropout(y.ptr, x.ptr, rows, cols, dtype, d, residual=r.ptr if res else None, ldy=y.ld, ldx=x.ld,
                       ldr=r.ld if res else None)
        torch.cuda.synchronize()
        f = OL.keep_factor(rows, cols, **d)
        v = x.np() * f
        e = 4 * U * np.abs(v)
        if res:
            v = v + r.np()
        close(y.np(), v, e, dtype, "y")
        if not res:
            assert np.array_equal(y.np() == 0, (f == 0) | (x.np() == 0))
        y.check_surroundings()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dropout_in_place_and_nonfinite(gpu, dtype):
    rows, cols = 60, 333
    x = randn(gen(4), rows, cols).to(TT[dtype])
    d = dict(p=0.4, seed=1, offset=2)
    out = torch.empty_like(x)
    B.fsdp_dropout(out, x, rows, cols, dtype, d)
    a = x.clone()
    B.fsdp_dropout(a, a, rows, cols, dtype, d)
    assert torch.equal(a, out)
    r = x.clone()
    B.fsdp_dropout(r, x, rows, cols, dtype, d, residual=r)
    B.fsdp_dropout(out, x, rows, cols, dtype, d, residual=x)
    assert torch.equal(r, out)
    x[:] = float("nan")
    B.fsdp_dropout(out, x, rows, cols, dtype, d)
    drop = torch.from_numpy(OL.keep_factor(rows, cols, **d) == 0).to(gpu)
    assert torch.equal(out.isnan(), ~drop)
    assert not out[drop].view(BITS[dtype]).any()


def test_one_mask_everywhere(gpu, space):
    """The forward's epilogue, its gradient and the call alone draw one mask
    from one record, whatever the path and the strides."""
    d = dict(p=0.3, seed=99, offset=(7 << 32) + 1)
    for m, n, k in ((1, 250, 64), (16, 264, 128), (300, 250, 64), (64, 72, 4096), (4096, 2048, 64)):
        one = torch.ones(m, n, dtype=torch.bfloat16, device=gpu)
        alone = torch.empty_like(one)
        B.fsdp_dropout(alone, one, m, n, "bf16", d)
        x = torch.zeros(m, k, dtype=torch.bfloat16, device=gpu)
        w = torch.zeros(n, k, dtype=torch.bfloat16, device=gpu)
        x[:, 0] = 1
        w[:, 0] = 1
        y, dz = torch.empty_like(one), torch.empty_like(one)
        B.fsdp_linear_forward(y, x, w, m, n, k, dropout=d, workspace=space)
        B.fsdp_linear_epilogue_backward(dz, one, m, n, dropout=d)
        assert torch.equal(y, alone) and torch.equal(dz, alone), (m, n, k)


@pytest.mark.parametrize("call,wt,m,n,k,size,off,pad,way", ROUTES)
def test_every_way(gpu, call, wt, m, n, k, size, off, pad, way):
    """Every way to compute a product, in every call and weight type; what lies
    behind the workspace stays."""
    buf = torch.full((size + 64,), 0x5A, dtype=torch.uint8, device=gpu)
    ws = buf[:size] if size else None
    if call == "forward":
        check_forward(m, n, k, ws, wt, act="silu", bias=True, res=True, keep_z=True, p=0.2, off=off, pad=pad)
        check_forward(m, n, k, ws, wt, yt="f32", off=off, pad=pad, seed=6)
    elif call == "grad_input":
        check_grad_input(m, k, n, ws, wt, off, pad)
    else:
        check_grad_weight(k, m, n, ws, "f32", True, off, pad)
        check_grad_weight(k, m, n, ws, "bf16", False, off, pad)
    assert bool((buf[size:] == 0x5A).all())


def test_tensors_as_they_come(gpu, space):
    """Parameters, E4M3 tensors, raw bits and views with their row stride give what packed tensors give."""
    m, n, k = 40, 48, 64
    g = gen(61)
    x, w = randn(g, m, k).bfloat16(), randn(g, n, k, 0.1).bfloat16()
    y, got = (torch.empty(m, n, dtype=torch.bfloat16, device=gpu) for _ in range(2))
    B.fsdp_linear_forward(y, x, w, m, n, k, workspace=space)
    wide = torch.full((n, 2 * k), float("nan"), dtype=torch.bfloat16, device=gpu)
    wide[:, k:] = w
    for wt, kw in ((torch.nn.Parameter(w), {}), (w.view(torch.int16), {}), (wide[:, k:], dict(ldw=2 * k))):
        B.fsdp_linear_forward(got.zero_(), x, wt, m, n, k, workspace=space, **kw)
        assert torch.equal(got, y)
    f8, one = w.to(torch.float8_e4m3fn), torch.ones(1, device=gpu)
    B.fsdp_linear_forward(y, x, f8.view(torch.uint8), m, n, k, w_dtype="e4m3", w_scale=one, workspace=space)
    B.fsdp_linear_forward(got, x, f8, m, n, k, w_dtype="e4m3", w_scale=one, workspace=space)
    assert torch.equal(got, y)
    for bad, kw in ((x.t(), {}), (x[:, :32], {}), (x[:20], {}), (x.float(), {}), (x.cpu(), {}), (x.t(), dict(ldx=k))):
        with pytest.raises(B.FsdpError):
            B.fsdp_linear_forward(got, bad, w, m, n, k, workspace=space, **kw)


# ---------------------------------------------------------------- streams, graphs, runs

def layer(gpu, m, n, k, seed):
    """The tensors of one layer's forward and backward calls, and the calls."""
    g = gen(seed)
    t = {"x": randn(g, m, k).bfloat16(), "w": randn(g, n, k, 0.1).bfloat16(), "b": randn(g, 1, n).bfloat16(),
         "dy": randn(g, m, n).bfloat16(), "y": torch.zeros(m, n, dtype=torch.bfloat16, device=gpu)}
    t["z"], t["dz"] = torch.zeros_like(t["y"]), torch.zeros_like(t["y"])
    t["dx"], t["dw"] = torch.zeros_like(t["x"]), torch.zeros(n, k, device=gpu)
    t["db"] = torch.zeros(n, device=gpu)
    t["ws"] = torch.empty(8 << 20, dtype=torch.uint8, device=gpu)
    t["out"] = ("y", "z", "dz", "dx", "dw", "db")
    t["mask"] = dict(p=0.2, seed=5, offset=seed)

    def calls(stream=None):
        B.fsdp_linear_forward(t["y"], t["x"], t["w"], m, n, k, bias=t["b"], act="gelu", z=t["z"],
                              dropout=t["mask"], workspace=t["ws"], stream=stream)
        B.fsdp_linear_epilogue_backward(t["dz"], t["dy"], m, n, z=t["z"], act="gelu", dropout=t["mask"],
                                        db=t["db"], workspace=t["ws"], stream=stream)
        B.fsdp_linear_grad_input(t["dx"], t["dz"], t["w"], m, n, k, workspace=t["ws"], stream=stream)
        B.fsdp_linear_grad_weight(t["dw"], t["dz"], t["x"], m, n, k, dw_dtype="f32", workspace=t["ws"],
                                  stream=stream)
    return t, calls


LAYERS = [(1, 264, 1032), (40, 130, 2048), (300, 520, 264), (65, 200, 999)]


def snapshot(t):
    return [t[o].clone() for o in t["out"]]


@pytest.mark.parametrize("m,n,k", LAYERS)
def test_two_streams_at_once(gpu, m, n, k):
    """Two layers' calls interleaved on two streams, a workspace each, give
    bit for bit what each gives alone; so does running again."""
    a, ca = layer(gpu, m, n, k, 1)
    b, cb = layer(gpu, m, n, k, 2)
    ca()
    cb()
    torch.cuda.synchronize()
    ra, rb = snapshot(a), snapshot(b)
    for t in (a, b):
        for o in t["out"]:
            t[o].zero_()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        ca(s1)
        cb(s2)
    torch.cuda.synchronize()
    for want, got in zip(ra + rb, snapshot(a) + snapshot(b)):
        assert torch.equal(want, got)


@pytest.mark.parametrize("m,n,k", LAYERS)
def test_graph_replays_with_a_device_offset(gpu, m, n, k):
    """A captured layer whose masks come from a device counter: each replay
    equals the eager calls at that count, with eager work between replays."""
    t, calls = layer(gpu, m, n, k, 3)
    count = torch.zeros(1, dtype=torch.int64, device=gpu)
    eager = t["mask"]
    t["mask"] = dict(eager, offset_dev=count)
    calls()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    seen = []
    for step in (0, 1, 5, 1, 1 << 40):
        count.fill_(step)
        g.replay()
        torch.cuda.synchronize()
        got = snapshot(t)
        t["mask"] = dict(eager, offset=eager["offset"] + step)
        calls()
        torch.cuda.synchronize()
        for a, b in zip(got, snapshot(t)):
            assert torch.equal(a, b)
        seen.append(got[0])
    assert torch.equal(seen[1], seen[3])
    assert not torch.equal(seen[0], seen[1])


WAYS_CAPTURED = [r for r in ROUTES if r[8] in ("direct 256/1", "direct 128/10", "direct 64/15", "staged 128/6",
                                               "pieces 3x3 64/1", "pieces 1x1 64/15", "few 2x2")
                 or r[8].startswith("direct columns")]


@pytest.mark.parametrize("call,wt,m,n,k,size,off,pad,way", WAYS_CAPTURED)
def test_every_way_captured(gpu, call, wt, m, n, k, size, off, pad, way):
    """The call in a graph, replayed over changed inputs with eager work between: each
    replay gives the eager call's bits."""
    g = gen(71)
    rows, cols = (k, m) if call == "grad_weight" else (m, k)
    a = Mat(rows, cols, "bf16", randn(g, rows, cols), off, pad)
    b = Mat(k, n, "bf16", randn(g, k, n), off, pad) if call == "grad_weight" else \
        weight(g, *((n, k) if call == "forward" else (k, n)), wt, off, pad)
    out = Mat(m, n, "bf16", None, off, pad)
    ws = torch.empty(size, dtype=torch.uint8, device=gpu) if size else None

    def run():
        if call == "forward":
            B.fsdp_linear_forward(out.ptr, a.ptr, b[0].ptr, m, n, k, w_dtype=wt, w_scale=b[1], act="gelu", workspace=ws,
                                  ldy=out.ld, ldx=a.ld, ldw=b[0].ld, dropout=dict(p=0.1, seed=1, offset=2))
        elif call == "grad_input":
            B.fsdp_linear_grad_input(out.ptr, a.ptr, b[0].ptr, m, k, n, w_dtype=wt, w_scale=b[1], workspace=ws,
                                     lddx=out.ld, lddz=a.ld, ldw=b[0].ld)
        else:
            B.fsdp_linear_grad_weight(out.ptr, a.ptr, b.ptr, k, m, n, workspace=ws, lddw=out.ld, lddz=a.ld, ldx=b.ld)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        a.t.copy_(randn(g, rows, cols))
        run()
        want = out.t.clone()
        out.t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.t, want)
    out.check_surroundings()


def test_parts_of_a_packed_projection(gpu, space):
    """Three products into the columns of one buffer, whose rows they share."""
    m, k, parts = 50, 256, (128, 64, 72)
    g = gen(8)
    x, buf = randn(g, m, k).bfloat16(), torch.zeros(m, sum(parts), dtype=torch.bfloat16, device=gpu)
    at = 0
    for i, n in enumerate(parts):
        w = randn(g, n, k, 0.1).bfloat16()
        alone = torch.empty(m, n, dtype=torch.bfloat16, device=gpu)
        B.fsdp_linear_forward(alone, x, w, m, n, k, workspace=space)
        # the residual is the next part's columns, still zero
        res = buf[:, (at + n) % sum(parts):] if i < 2 and parts[i + 1] >= n else None
        B.fsdp_linear_forward(buf[:, at:], x, w, m, n, k, workspace=space, ldy=buf.shape[1], residual=res,
                              ldr=buf.shape[1])
        assert torch.equal(buf[:, at:at + n], alone)
        at += n


def test_captured_training_step(gpu, space):
    """Forward, backward and the optimizer's step in one graph, with dropout's
    offset read from the count that the step advances: replays equal the eager
    calls at t = 1, 2, 3, with eager work between them."""
    from rank_step_amd.workloads import HPARAMS
    m, n, k = 48, 136, 264
    g = gen(51)
    x, dy = randn(g, m, k).bfloat16(), randn(g, m, n).bfloat16()
    p0 = randn(g, n, k, 0.05)

    class Run:
        def __init__(self):
            self.p, self.m, self.v = p0.clone(), torch.zeros_like(p0), torch.zeros_like(p0)
            self.w, self.dw = p0.bfloat16(), torch.zeros(n, k, dtype=torch.bfloat16, device=gpu)
            self.y, self.z, self.dz = (torch.zeros(m, n, dtype=torch.bfloat16, device=gpu) for _ in range(3))
            self.db = torch.zeros(n, device=gpu)
            self.plan = B.MtPlan([{"param_fp32": self.p, "exp_avg": self.m, "exp_avg_sq": self.v,
                                   "grad_slices": self.dw, "slice_stride": n * k, "unshard_bf16_out": self.w,
                                   "shard_numel": n * k, "valid": n * k}], 1, "bf16")

        def layer(self, mask):
            B.fsdp_linear_forward(self.y, x, self.w, m, n, k, act="silu", z=self.z, dropout=mask, workspace=space)
            B.fsdp_linear_epilogue_backward(self.dz, dy, m, n, z=self.z, act="silu", dropout=mask, db=self.db,
                                            workspace=space)
            B.fsdp_linear_grad_weight(self.dw, self.dz, x, m, n, k, workspace=space)

        def out(self):
            return [t.clone() for t in (self.p, self.m, self.v, self.w, self.dw, self.y, self.dz, self.db)]

    eager, graphed = Run(), Run()
    count = torch.zeros(1, dtype=torch.int64, device=gpu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.layer(dict(p=0.3, seed=8, offset=1 << 40, offset_dev=count))
        graphed.plan.step_capturable(HPARAMS, count)
    for t in (1, 2, 3):
        eager.layer(dict(p=0.3, seed=8, offset=(1 << 40) + t - 1))
        eager.plan.step(HPARAMS, t)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert int(count) == t
        for i, (a, b) in enumerate(zip(eager.out(), graphed.out())):
            assert torch.equal(a, b), (t, i)
    del graph
    eager.plan.close()
    graphed.plan.close()


@pytest.mark.parametrize("copy", ["bf16", "e4m3"])
def test_layer_between_two_steps(gpu, space, copy):
    """A two-layer MLP as a rank runs it: the step writes the weight copies,
    the forward reads them, the backward writes the gradient slices, the next
    step reduces those and updates; every result against the oracle from the
    bits that its call read."""
    from oracle import step as OS
    from rank_step_amd.workloads import HPARAMS

    N, m, h, f = 2, 96, 136, 264          # ranks, tokens, width, hidden
    g = gen(21)
    shapes = [(f, h), (h, f)]
    sizes = [a * b for a, b in shapes]
    p = [randn(g, 1, s, 0.05)[0].contiguous() for s in sizes]
    mom = [torch.zeros_like(q) for q in p]
    var = [torch.zeros_like(q) for q in p]
    slices = [torch.zeros(N, s, dtype=torch.bfloat16, device=gpu) for s in sizes]
    b16 = [torch.zeros(s, dtype=torch.bfloat16, device=gpu) for s in sizes]
    f8 = [torch.zeros(s, dtype=torch.uint8, device=gpu) for s in sizes]
    amax, scale = torch.zeros(2, device=gpu), torch.zeros(2, device=gpu)
    with B.MtPlan([{"param_fp32": p[i], "exp_avg": mom[i], "exp_avg_sq": var[i], "grad_slices": slices[i],
                    "slice_stride": sizes[i], "unshard_bf16_out": b16[i], "unshard_fp8_out": f8[i],
                    "shard_numel": sizes[i], "valid": sizes[i]} for i in range(2)], N, "bf16") as plan:
        for t in (1, 2):
            before = [(q.double().cpu().numpy(), a.double().cpu().numpy(), v.double().cpu().numpy(),
                       s.double().cpu().numpy()) for q, a, v, s in zip(p, mom, var, slices)]
            B.fsdp_mt_step_amax(plan.handle, HPARAMS, t, amax)
            B.fsdp_mt_cast_fp8(plan.handle, amax, 1, scale)
            torch.cuda.synchronize()
            for i in range(2):
                ref = OS.rank_step(before[i][0], before[i][1], before[i][2], before[i][3], sizes[i], t, HPARAMS)
                got = p[i].double().cpu().numpy()
                floor = np.abs(ref["p"]) + HPARAMS["lr"]
                assert (np.abs(got - ref["p"]) / floor).max() <= 2e-6, (t, i)
            if copy == "bf16":
                w, ws = b16, [None, None]
                wv = [b.double().cpu().numpy().reshape(s) for b, s in zip(b16, shapes)]
            else:
                w, ws = f8, [scale[0:1], scale[1:2]]
                wv = [F8.e4m3_value(c.cpu().numpy()).reshape(s) / float(q) for c, s, q in zip(f8, shapes, scale)]
            for rank in range(N):  # each rank's batch gives one slice
                x = randn(g, m, h).bfloat16()
                mask = dict(p=0.1, seed=rank, offset=t)
                a1, z1 = (torch.empty(m, f, dtype=torch.bfloat16, device=gpu) for _ in range(2))
                y = torch.empty(m, h, dtype=torch.bfloat16, device=gpu)
                kw = [dict(w_dtype=copy, w_scale=ws[i], workspace=space) for i in range(2)]
                B.fsdp_linear_forward(a1, x, w[0], m, f, h, act="silu", z=z1, **kw[0])
                B.fsdp_linear_forward(y, a1, w[1], m, h, f, residual=x, dropout=mask, **kw[1])
                dy = randn(g, m, h).bfloat16()
                dz2, da1, dz1 = torch.empty_like(y), torch.empty_like(a1), torch.empty_like(a1)
                dx = torch.empty_like(x)
                B.fsdp_linear_epilogue_backward(dz2, dy, m, h, dropout=mask, workspace=space)
                B.fsdp_linear_grad_input(da1, dz2, w[1], m, h, f, **kw[1])
                B.fsdp_linear_grad_weight(slices[1][rank], dz2, a1, m, h, f, workspace=space)
                B.fsdp_linear_epilogue_backward(dz1, da1, m, f, z=z1, act="silu", workspace=space)
                B.fsdp_linear_grad_input(dx, dz1, w[0], m, f, h, **kw[0])
                B.fsdp_linear_grad_weight(slices[0][rank], dz1, x, m, f, h, workspace=space)
                torch.cuda.synchronize()
                v = {k_: t_.double().cpu().numpy() for k_, t_ in
                     dict(x=x, a1=a1, z1=z1, dz2=dz2, da1=da1, dz1=dz1, dy=dy).items()}
                fac = OL.keep_factor(m, h, **mask)
                z1v, s = OL.product(v["x"], wv[0])
                close(v["z1"], z1v, product_err(h, s) + 4 * U * s, "bf16", "z1")
                y2, s = OL.product(v["a1"], wv[1])
                close(y.double().cpu().numpy(), y2 * fac + v["x"],
                      (product_err(f, s) + 6 * U * s) * fac + 2 * U * np.abs(v["x"]), "bf16", "y")
                close(v["dz2"], v["dy"] * fac, 4 * U * np.abs(v["dy"]) * fac, "bf16", "dz2")
                d, s = OL.product(v["dz2"], wv[1].T)
                close(v["da1"], d, product_err(h, s) + 4 * U * s, "bf16", "da1")
                d, s = OL.product(v["dz1"], wv[0].T)
                close(dx.double().cpu().numpy(), d, product_err(f, s) + 4 * U * s, "bf16", "dx")
                for i, (da, xa) in enumerate((("dz1", "x"), ("dz2", "a1"))):
                    d, s = OL.product(v[da].T, v[xa].T)
                    close(slices[i][rank].double().cpu().numpy().reshape(shapes[i]), d, product_err(m, s), "bf16",
                          f"slice {i}")


# ---------------------------------------------------------------- strides of one row, offsets past 32 bits

@pytest.mark.parametrize("ld", [0, 1, 5, 1 << 40])
def test_the_stride_of_a_single_row_says_nothing(gpu, space, ld):
    g = gen(31)
    n, k = 72, 136
    x, w = randn(g, 1, k).bfloat16(), randn(g, n, k).bfloat16()
    dz, one = randn(g, 1, n).bfloat16(), randn(g, 1, k).bfloat16()
    pairs = []
    for s in (None, ld):
        y, dx = torch.empty(1, n, device=gpu), torch.empty(1, k, dtype=torch.bfloat16, device=gpu)
        dw, out = torch.empty(n, k, device=gpu), torch.empty(300, 1, device=gpu)
        dxw = torch.empty(300, k, dtype=torch.bfloat16, device=gpu)
        B.fsdp_linear_forward(y, x, w, 1, n, k, y_dtype="f32", workspace=space, ldx=s, ldy=s)
        B.fsdp_linear_grad_input(dx, dz, w, 1, n, k, workspace=space, lddz=s, lddx=s)
        B.fsdp_linear_grad_weight(dw, dz, x, 1, n, k, dw_dtype="f32", workspace=space, lddz=s, ldx=s)
        many = torch.ones(300, k, dtype=torch.bfloat16, device=gpu)
        B.fsdp_linear_forward(out, many, one, 300, 1, k, y_dtype="f32", workspace=space, ldw=s)
        B.fsdp_linear_grad_input(dxw, torch.ones(300, 1, dtype=torch.bfloat16, device=gpu), one, 300, 1, k,
                                 workspace=space, ldw=s)
        pairs.append([y, dx, dw, out, dxw])
    for a, b in zip(*pairs):
        assert torch.equal(a, b)
    assert torch.equal(pairs[0][2], dz.float().t() * x.float())
    assert torch.equal(pairs[0][4], one.expand(300, k))


def test_offsets_past_32_bits(gpu, space):
    """2.2 G elements a matrix: products, gradients and dropout, on rows from all
    over it."""
    m, n, k = (1 << 21) + 5, 1032, 16
    g = gen(41)
    x, w = randn(g, m, k).bfloat16(), randn(g, n, k).bfloat16()
    d = dict(p=0.25, seed=6, offset=7)
    y = torch.empty(m, n, dtype=torch.bfloat16, device=gpu)
    rows = [0, 1, 65, m // 2, (1 << 32) // (2 * n), (1 << 31) // n, (1 << 32) // (2 * n) + 1, m - 70, m - 1]
    B.fsdp_linear_forward(y, x, w, m, n, k, dropout=d, workspace=space)
    keep = np.concatenate([OL.keep_factor(1, n, **d, first=r) for r in rows])
    xv, wv = x[rows].double().cpu().numpy(), w.double().cpu().numpy()
    v, s = OL.product(xv, wv)
    close(y[rows].double().cpu().numpy(), v * keep, product_err(k, s) * keep + 4 * U * np.abs(v * keep), "bf16", "y")
    # the gradients, with y as dz: every row counts in dW
    dx = torch.empty(m, k, dtype=torch.bfloat16, device=gpu)
    B.fsdp_linear_grad_input(dx, y, w, m, n, k, workspace=space)
    dv = y[rows].double().cpu().numpy()
    v, s = OL.product(dv, wv.T)
    close(dx[rows].double().cpu().numpy(), v, product_err(n, s), "bf16", "dx")
    dw = torch.empty(n, k, device=gpu)
    B.fsdp_linear_grad_weight(dw, y, x, m, n, k, dw_dtype="f32", workspace=space)
    ref, mag = (torch.zeros(n, k, dtype=torch.float64, device=gpu) for _ in range(2))
    for a in range(0, m, 1 << 18):
        t, u = y[a:a + (1 << 18)].double(), x[a:a + (1 << 18)].double()
        ref += t.t().contiguous() @ u
        mag += t.abs().t().contiguous() @ u.abs()
    close(dw.double().cpu().numpy(), ref.cpu().numpy(), product_err(m, mag.cpu().numpy()), "f32", "dw")
    # the elementwise passes, in place
    before = y[rows].double().cpu().numpy()
    B.fsdp_dropout(y, y, m, n, "bf16", d)
    once = y[rows].double().cpu().numpy()
    close(once, before * keep, 4 * U * np.abs(before * keep), "bf16", "dropout")
    db = torch.empty(n, device=gpu)
    B.fsdp_linear_epilogue_backward(y, y, m, n, dropout=d, db=db, workspace=space)
    again = y[rows].double().cpu().numpy()
    close(again, once * keep, 4 * U * np.abs(once) * keep, "bf16", "dz")


@pytest.mark.parametrize("n", [1032, 1033])
def test_every_row_counts_past_32_bits(gpu, space, n):
    """The weight gradient of 2.2 G elements of dz, exactly: dz is +-1 and x an
    integer of at most 2, so every partial sum is an integer of at most 2^22 and
    exact in fp32, and one row left out or taken twice would show."""
    m, k = (1 << 21) + 5, 16
    g = gen(43)
    dz = torch.empty(m, n, dtype=torch.bfloat16, device=gpu)
    x = (torch.randint(0, 2, (m, k), generator=g, device=gpu) * 3 - 1).bfloat16()  # -1 or 2: no row adds nothing
    old = torch.randint(-9, 10, (n, k), generator=g, device=gpu).float()
    ref = old.double()
    for a in range(0, m, 1 << 18):
        b = min(m, a + (1 << 18))
        dz[a:b] = (torch.randint(0, 2, (b - a, n), generator=g, device=gpu, dtype=torch.int8) * 2 - 1).bfloat16()
        ref += dz[a:b].double().t().contiguous() @ x[a:b].double()
    dw = old.clone()
    B.fsdp_linear_grad_weight(dw, dz, x, m, n, k, dw_dtype="f32", accumulate=True, workspace=space)
    assert torch.equal(dw.double(), ref)
    # column sums of the same rows: every one counts in db too
    db = torch.empty(n, device=gpu)
    B.fsdp_linear_epilogue_backward(None, dz, m, n, db=db, workspace=space)
    assert torch.equal(db.double(), sum(dz[a:a + (1 << 18)].double().sum(0) for a in range(0, m, 1 << 18)))


@pytest.mark.parametrize("wt", ["bf16", "e4m3"])
def test_weights_past_32_bits(gpu, space, wt):
    """A weight of 2.2 G elements, exactly: its elements are -1 or 2 and the other
    operand's +-1, so every sum is an integer under 2^24."""
    n, k = (1 << 22) + 24, 528
    g = gen(81)
    w = torch.empty(n, k, dtype=TT[wt], device=gpu)
    for a in range(0, n, 1 << 18):
        b = min(n, a + (1 << 18))
        two = torch.randint(0, 2, (b - a, k), generator=g, device=gpu, dtype=torch.uint8)
        w[a:b] = 0xB8 - two * 0x78 if wt == "e4m3" else (two.char() * 3 - 1).bfloat16()  # codes of -1 and 2
    one = torch.ones(1, device=gpu) if wt == "e4m3" else None

    def values(a, b):
        return w[a:b].view(torch.float8_e4m3fn).double() if wt == "e4m3" else w[a:b].double()

    def signs(*shape):
        return (torch.randint(0, 2, shape, generator=g, device=gpu, dtype=torch.int8) * 2 - 1).bfloat16()

    for m in (3, 40):
        x, dz = signs(m, k), signs(m, n)
        y = torch.empty(m, n, device=gpu)
        B.fsdp_linear_forward(y, x, w, m, n, k, w_dtype=wt, w_scale=one, y_dtype="f32", workspace=space)
        dx = torch.empty(m, k, dtype=torch.bfloat16, device=gpu)
        B.fsdp_linear_grad_input(dx, dz, w, m, n, k, w_dtype=wt, w_scale=one, workspace=space)
        ref = torch.zeros(m, k, dtype=torch.float64, device=gpu)
        for a in range(0, n, 1 << 18):
            b = min(n, a + (1 << 18))
            v = values(a, b)
            assert torch.equal(y[:, a:b].double(), x.double() @ v.t().contiguous()), (m, a)
            ref += dz[:, a:b].double().contiguous() @ v
        assert torch.equal(dx, ref.bfloat16()), m
