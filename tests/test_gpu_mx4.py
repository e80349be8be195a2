"""The 4-bit matrices' calls on the GPU against the float64 oracle.

Copies and values are compared bit for bit.  Inputs lie in buffers whose other
elements are NaN (codes: 0xFF, scales: 255, which is NaN), outputs in buffers of
a fixed pattern that must be whole around the output afterwards.

Tolerances of the product, with u = 2^-24 (half an fp32 step).  Products of two
elements are exact.  A matrix instruction adds 128 of them, off by at most a
whole step (2u) of the largest that one of them could be, each; that is 2u R
over all instructions, with R the sum over blocks of 32 * 6 * 6 times both scales.
Its accumulator, and the joining of up to 64 parts and 8 waves, is off by 2u of
the sum S of the terms' magnitudes at most k / 128 + 104 times.  The epilogue's
are the linear layer's.
"""

import itertools

import numpy as np
import pytest
import torch

from oracle import linear as OL
from oracle import mx4 as Q
from rank_step_amd import binding as B
from tests.test_gpu_linear import HALF, U, Mat, act_err, close, gen, randn

pytestmark = pytest.mark.gpu


class Bytes:
    """Rows of bytes `ld` apart inside a larger buffer, 16-byte aligned."""

    def __init__(self, rows, cols, values=None, off=0, pad=0, fill=None):
        self.rows, self.cols, self.off, self.ld = rows, cols, off * 16, cols + pad * 16
        self.fill = fill if fill is not None else 0x5A if values is None else 0xFF
        self.buf = torch.full((self.off + rows * self.ld + 64,), self.fill, dtype=torch.uint8, device="cuda")
        self.t = self.buf[self.off:self.off + rows * self.ld].view(rows, self.ld)[:, :cols]
        if values is not None:
            self.t.copy_(torch.from_numpy(values) if isinstance(values, np.ndarray) else values)

    @property
    def ptr(self):
        return self.buf.data_ptr() + self.off

    def np(self):
        return self.t.cpu().numpy()

    def check_surroundings(self):
        b = self.buf.clone()
        b[self.off:self.off + self.rows * self.ld].view(self.rows, self.ld)[:, :self.cols] = self.fill
        assert bool((b == self.fill).all()), "written outside the output"


def check_quantize(rows, cols, dtype, values, form="both", off=0, pad=0):
    x = Mat(rows, cols, dtype, values, off, pad)
    out = {}
    for t, r, c in (("", rows, cols), ("_t", cols, rows)):
        if form in ("both", "rows" if t == "" else "columns"):
            out["codes" + t] = Bytes(r, Q.code_bytes(c), None, off, pad)
            out["scales" + t] = Bytes(r, Q.scale_bytes(c), None, off, pad)
    ld = {"codes": "ldc", "scales": "lds", "codes_t": "ldct", "scales_t": "ldst"}
    B.fsdp_mx4_quantize(x.ptr, rows, cols, x_dtype=dtype, ldx=x.ld, **{k: v.ptr for k, v in out.items()},
                        **{ld[k]: v.ld for k, v in out.items()})
    torch.cuda.synchronize()
    xv = x.np()
    for t, v in (("", xv), ("_t", xv.T)):
        if "codes" + t not in out:
            continue
        codes, scales = Q.quantize(v)
        got = out["codes" + t].np(), out["scales" + t].np()
        assert np.array_equal(got[1], scales), ("scales" + t, np.argwhere(got[1] != scales)[:3].tolist())
        # a block of scale 255 has codes 0, one with a zero may have either sign of it
        finite = np.repeat(scales == 255, 16, axis=1)[:, :codes.shape[1]] == 0
        nan = np.where(finite, 0, got[0])
        assert not nan.any()
        assert np.array_equal(np.where(finite, got[0], 0), np.where(finite, codes, 0)), "codes" + t
    for v in out.values():
        v.check_surroundings()
    for t, r, c in (("", rows, cols), ("_t", cols, rows)):
        if "codes" + t not in out:
            continue
        for yt in ("bf16", "f32"):
            y = Mat(r, c, yt, None, off, pad)
            q, s = out["codes" + t], out["scales" + t]
            B.fsdp_mx4_dequantize(y.ptr, q.ptr, s.ptr, r, c, y_dtype=yt, ldy=y.ld, ldc=q.ld, lds=s.ld)
            torch.cuda.synchronize()
            want = Q.values(q.np(), s.np(), c)
            got = y.np()
            assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.nan_to_num(got), np.nan_to_num(want)), yt
            y.check_surroundings()


SIZES = [(1, 1), (1, 31), (1, 32), (1, 33), (2, 8), (3, 7), (31, 5), (32, 64), (33, 65), (37, 251), (1, 4096), (4096, 1),
         (64, 511), (65, 513), (128, 128), (129, 127), (200, 1365), (1000, 100), (7, 5000), (513, 33), (300, 1056)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_sizes(gpu, rows, cols, dtype):
    g = gen(1)
    for form, off, pad in (("both", 0, 0), ("rows", 1, 3), ("columns", 3, 1), ("both", 5, 2)):
        check_quantize(rows, cols, dtype, randn(g, rows, cols, 0.02), form, off, pad)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_many_rows(gpu, dtype):
    check_quantize(9000, 160, dtype, randn(gen(2), 9000, 160))
    check_quantize(40, 20000, dtype, randn(gen(2), 40, 20000))


def test_every_bf16_value(gpu):
    """All finite bf16 values with each block's largest one from 2^-130 to 2^127:
    the whole range of scales, subnormal inputs and saturated elements."""
    bits = np.arange(0x7F80, dtype=np.uint16)
    v = (bits.astype(np.uint32) << 16).view(np.float32)
    x = np.resize(v, (1021, 32)).astype(np.float32)  # blocks of 32 neighbours in size
    x[:, 1::2] *= -1
    check_quantize(1021, 32, "bf16", torch.from_numpy(x))
    check_quantize(1021, 32, "f32", torch.from_numpy(x))
    # one large element a block, the others spread below it
    r = np.random.default_rng(1)
    e = np.repeat(np.arange(-149, 128), 4)[:, None]
    y = np.ldexp(1 + r.random((e.size, 64)), e - np.minimum(r.integers(0, 6, (e.size, 64)), 149 + e)).astype(np.float32)
    check_quantize(e.size, 64, "f32", torch.from_numpy(y))


def test_rounding_of_fp32(gpu):
    """Values at the middle between two codes and one fp32 step to either side, under every scale."""
    middle = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=np.float32)
    around = np.concatenate([middle, np.nextafter(middle, np.float32(0)), np.nextafter(middle, np.float32(9)), [4.0]])
    x = np.zeros((250, 32), np.float32)
    x[:, :around.size] = around[None] * np.exp2(np.arange(-125, 125, dtype=np.float32))[:, None]
    x[1::2] *= -1
    check_quantize(250, 32, "f32", torch.from_numpy(x))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nonfinite_blocks(gpu, dtype):
    x = randn(gen(3), 70, 100)
    x[3, 5], x[40, 99], x[65, 64] = float("nan"), float("inf"), float("-inf")
    x[10] = 0.0
    x[:, 20] = -0.0
    check_quantize(70, 100, dtype, x)


def test_every_code_and_scale(gpu):
    """Values of all 16 codes under all 256 scales."""
    codes = np.tile(np.arange(16, dtype=np.uint8) | (np.arange(15, -1, -1, dtype=np.uint8) << 4), (256, 1))
    scales = np.zeros((256, 16), np.uint8)
    scales[:, 0] = np.arange(256)
    q, s = Bytes(256, 16, codes), Bytes(256, 16, scales)
    want = Q.values(codes, scales, 32)
    want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)
    for yt in ("bf16", "f32"):
        y = Mat(256, 32, yt)
        B.fsdp_mx4_dequantize(y.ptr, q.ptr, s.ptr, 256, 32, y_dtype=yt)
        torch.cuda.synchronize()
        assert np.array_equal(y.np(), want, equal_nan=True)


# ---------------------------------------------------------------- products

@pytest.fixture(scope="module")
def space(gpu):
    return torch.empty(B.MX4_WORKSPACE_BYTES, dtype=torch.uint8, device=gpu)


def packed(g, rows, k, off=0, pad=0, std=1.0, spread=True):
    """Codes and scales of a random matrix whose rows differ in size."""
    v = randn(g, rows, k, std)
    if spread:
        v = v * torch.exp2(torch.randint(-3, 4, (rows, 1), generator=g, device="cuda").float())
    codes, scales = Q.quantize(v.double().cpu().numpy())
    return Bytes(rows, codes.shape[1], codes, off, pad), Bytes(rows, scales.shape[1], scales, off, pad), codes, scales


def reference(a, asc, b, bsc, k):
    """The product, its terms' magnitudes, and what its blocks have room for; on the GPU in float64."""
    x, y = (torch.from_numpy(Q.values(c, s, k)).cuda() for c, s in ((a, asc), (b, bsc)))
    ra, rb = (torch.from_numpy(Q.room(s, k)).cuda() for s in (asc, bsc))
    return ((x @ y.T).cpu().numpy(), (x.abs() @ y.abs().T).cpu().numpy(), (ra @ rb.T).cpu().numpy() / 32)


def product_err(k, s, room):
    return 2 * U * ((k / 128 + 104) * s + room)


def check_product(m, n, k, space, yt="bf16", act="none", bias=False, res=False, keep_z=False, p=0.0, off=0, pad=0,
                  same=False, seed=1):
    g = gen(seed)
    a, asc, av, asv = packed(g, m, k, off, pad)
    b, bsc, bv, bsv = packed(g, n, k, off, pad, 0.1)
    c = Mat(1, n, "bf16", randn(g, 1, n), off) if bias else None
    r = Mat(m, n, yt, randn(g, m, n), off, pad) if res else None
    y = r if same else Mat(m, n, yt, None, off, pad)
    z = Mat(m, n, "bf16", None, off, pad) if keep_z else None
    d = dict(p=p, seed=0xFEDCBA9876543210 + seed, offset=(1 << 35) + seed) if p else None
    rv = r.np() if res else 0.0
    ptr = lambda t: None if t is None else t.ptr  # noqa: E731
    B.fsdp_mx4_product(y.ptr, a.ptr, asc.ptr, b.ptr, bsc.ptr, m, n, k, y_dtype=yt, bias=ptr(c), residual=ptr(r), act=act,
                       z=ptr(z), dropout=d, workspace=space, ldy=y.ld, lda=a.ld, ldas=asc.ld, ldb=b.ld, ldbs=bsc.ld,
                       ldr=r.ld if r else None, ldz=z.ld if z else None)
    torch.cuda.synchronize()
    zv, s, room = reference(av, asv, bv, bsv, k)
    ez = product_err(k, s, room)
    if bias:
        zv = zv + c.np()
        ez = ez + 2 * U * np.abs(zv)
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


SHAPES = [(1, 1, 1), (1, 64, 64), (1, 512, 1365), (1, 96, 4096), (3, 8, 8), (7, 33, 65), (15, 70, 32), (16, 256, 512),
          (17, 130, 72), (31, 100, 999), (32, 48, 700), (33, 64, 128), (64, 64, 4096), (65, 40, 2056), (100, 1024, 17), (128, 128, 128),
          (129, 257, 191), (300, 264, 520), (257, 1000, 1365), (512, 384, 64), (256, 256, 8200)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product_shapes(gpu, space, m, n, k):
    check_product(m, n, k, space)
    check_product(m, n, k, space, yt="f32", act="silu", bias=True, res=True, keep_z=True, p=0.25)
    check_product(m, n, k, None, act="gelu", bias=True, off=1, pad=3, keep_z=True)


# 256-tiles with ragged edges, 128-tiles, few tiles over long contractions, and outputs
# that are cut after their whole rounds of 256-tiles, by columns and by rows
WAYS = [(4000, 4080, 1000), (2048, 2064, 1300), (520, 1040, 4000), (300, 128, 33000), (4096, 4112, 2048), (4104, 4096, 2048)]


@pytest.mark.parametrize("m,n,k", WAYS)
def test_ways(gpu, space, m, n, k):
    check_product(m, n, k, space, act="silu", bias=True, res=True, keep_z=True, p=0.1)
    check_product(m, n, k, space, yt="f32", res=True, same=True)


@pytest.mark.parametrize("size", [0, 1 << 10, 64 << 10, 600 << 10, 5 << 20])
@pytest.mark.parametrize("m,n,k", [(64, 100, 8200), (300, 200, 20000)])
def test_product_workspaces(gpu, m, n, k, size):
    buf = torch.full((size + 64,), 0x5A, dtype=torch.uint8, device=gpu)
    ws = buf[:size] if size else None
    check_product(m, n, k, ws, act="gelu", bias=True, res=True, keep_z=True, p=0.2)
    assert bool((buf[size:] == 0x5A).all())


@pytest.mark.parametrize("k", list(range(1, 34)) + [255, 256, 257, 480, 481, 511, 512, 513, 767, 768, 769, 1023, 1024, 1025, 1536, 2049])
@pytest.mark.parametrize("m", [1, 20, 130])
def test_every_end_of_the_contraction(gpu, space, m, k):
    check_product(m, 70, k, space, yt="f32", pad=2)


@pytest.mark.parametrize("m", [1, 16, 30])
@pytest.mark.parametrize("k", [256 * 8 * 15 + 256 * 5 + 40, 256 * 8 * 7 + 8, 256 * 8 * 3, 256 * 9])
def test_few_tokens_by_batches(gpu, space, m, k):
    """Contractions that leave each wave chunks for every size of batch, and a part of one."""
    check_product(m, 40, k, space, bias=True)
    check_product(m, 70, k - 3, space, yt="f32", off=1, pad=1)


@pytest.mark.parametrize("act,bias,res,keep_z,p,yt", [
    c for i, c in enumerate(itertools.product(["none", "relu", "gelu", "silu"], [False, True], [False, True],
                                              [False, True], [0.0, 0.5], ["bf16", "f32"])) if i % 5 == 0])
def test_epilogues(gpu, space, act, bias, res, keep_z, p, yt):
    check_product(40, 72, 136, space, act=act, bias=bias, res=res, keep_z=keep_z, p=p, yt=yt)
    check_product(2, 72, 136, space, act=act, bias=bias, res=res, keep_z=keep_z, p=p, yt=yt)
    check_product(9, 65, 4096, space, act=act, bias=bias, res=res, keep_z=keep_z, p=p, yt=yt, off=1, pad=2)


@pytest.mark.parametrize("m,n,k", [(5, 64, 64), (40, 72, 136), (33, 64, 8192), (4096, 2048, 256)])
@pytest.mark.parametrize("yt", ["bf16", "f32"])
def test_residual_in_place(gpu, space, m, n, k, yt):
    check_product(m, n, k, space, yt=yt, act="relu", res=True, same=True, p=0.3)


EXACT = [(1, 40, 600), (16, 200, 2100), (30, 70, 4096), (64, 64, 9000), (130, 300, 1500), (700, 600, 512), (2048, 2064, 520), (4000, 4080, 300)]


@pytest.mark.parametrize("m,n,k", EXACT)
def test_exact_sums(gpu, space, m, n, k):
    """Scales of 1 to 8: every sum is a multiple of 1/4 under 2^22, exact in fp32, by
    whatever tile, split and order; one wrong element or scale shows."""
    r = np.random.default_rng(m + k)
    kb, ks = Q.code_bytes(k), Q.scale_bytes(k)
    sets = []
    for rows in (m, n):
        codes = r.integers(0, 256, (rows, kb), dtype=np.uint8)
        scales = np.zeros((rows, ks), np.uint8)
        scales[:, :kb // 16] = r.integers(127, 130, (rows, kb // 16))
        flat = np.empty((rows, kb * 2), np.uint8)
        flat[:, 0::2], flat[:, 1::2] = codes & 15, codes >> 4
        flat[:, k:] = 0
        # magnitudes of 0.5 to 1.5, so that the sums stay small
        flat = np.where(flat & 7 > 3, flat & 8 | 1, flat)
        sets.append((flat[:, 0::2] | flat[:, 1::2] << 4, scales))
    (a, asc), (b, bsc) = sets
    dev = [torch.from_numpy(v).cuda() for v in (a, asc, b, bsc)]
    y = torch.empty(m, n, device=gpu)
    B.fsdp_mx4_product(y, *dev, m, n, k, y_dtype="f32", workspace=space)
    want, s, _ = reference(a, asc, b, bsc, k)
    assert s.max() < 2 ** 22
    assert np.array_equal(y.double().cpu().numpy(), want)
    again = torch.empty(m, n, device=gpu)
    B.fsdp_mx4_product(again, *dev, m, n, k, y_dtype="f32")
    assert torch.equal(again, y)  # without a workspace


@pytest.mark.parametrize("m", [4, 20, 70, 300])
def test_nan_blocks_stay_in_their_rows(gpu, space, m):
    n, k = 300, 1300
    g = gen(8)
    a, asc, *_ = packed(g, m, k)
    b, bsc, *_ = packed(g, n, k)
    asc.t[1, 0], asc.t[3, Q.code_bytes(k) // 16 - 1], bsc.t[77, 20] = 255, 255, 255
    y = torch.empty(m, n, device=gpu)
    B.fsdp_mx4_product(y, a.t, asc.t, b.t, bsc.t, m, n, k, y_dtype="f32", workspace=space)
    want = torch.zeros(m, n, dtype=torch.bool, device=gpu)
    want[1], want[3], want[:, 77] = True, True, True
    assert torch.equal(y.isnan(), want)


def test_extreme_scales(gpu, space):
    """2^-127 times 2^127 is 1; products past fp32's range overflow and underflow as fp32 does."""
    k = 64
    for m in (1, 40):
        codes = np.full((m, 32), 0x22, np.uint8)  # ones
        for sa, sb, want in ((0, 254, 64.0), (254, 0, 64.0), (0, 127, 64 * 2.0 ** -127), (254, 254, np.inf), (3, 3, 0.0)):
            s1, s2 = (np.zeros((m, 16), np.uint8) for _ in range(2))
            s1[:, :2], s2[:, :2] = sa, sb
            dev = [torch.from_numpy(v).cuda() for v in (codes, s1, codes, s2)]
            y = torch.empty(m, m, device=gpu)
            B.fsdp_mx4_product(y, *dev, m, m, k, y_dtype="f32", workspace=space)
            assert bool((y == want).all()), (m, sa, sb, y[0, 0])


@pytest.mark.parametrize("m", [1, 20, 130])
def test_empty_contraction(gpu, space, m):
    n = 70
    b = randn(gen(1), 1, n).to(torch.bfloat16)
    y = Mat(m, n, "f32")
    B.fsdp_mx4_product(y.ptr, None, None, None, None, m, n, 0, y_dtype="f32", bias=b, act="relu", workspace=space)
    torch.cuda.synchronize()
    assert np.array_equal(y.np(), np.broadcast_to(np.maximum(b.double().cpu().numpy(), 0), (m, n)))
    y.check_surroundings()


# ---------------------------------------------------------------- a layer in 4 bits

def layer(gpu, m, n, k, seed=4):
    """norm, quantise, product forward; epilogue gradient, quantise both ways, two products, norm backward."""
    g = gen(seed)
    bf, f = torch.bfloat16, torch.float32
    e = lambda r, c, t=bf: torch.empty(r, c, dtype=t, device=gpu)  # noqa: E731
    s = dict(x=randn(g, m, k).to(bf), gamma=(1 + 0.1 * randn(g, 1, k)).to(bf), master=randn(g, n, k, 0.05),
             dy=randn(g, m, n, 0.1).to(bf), res=randn(g, m, n).to(bf))
    s |= dict(h=e(m, k), rstd=torch.empty(m, device=gpu), y=e(m, n), z=e(m, n), dz=e(m, n), dh=e(m, k), dx=e(m, k),
              dw=torch.zeros(n, k, device=gpu), dgamma=torch.empty(k, device=gpu),
              ws=torch.empty(B.MX4_WORKSPACE_BYTES, dtype=torch.uint8, device=gpu))
    for name, r, c in (("w", n, k), ("wt", k, n), ("h", m, k), ("ht", k, m), ("dz", m, n), ("dzt", n, m)):
        s["c_" + name], s["s_" + name] = e(r, Q.code_bytes(c), torch.uint8), e(r, Q.scale_bytes(c), torch.uint8)
    return s


def layer_pass(s, m, n, k, stream=None):
    kw = dict(stream=stream)
    drop = dict(p=0.1, seed=7, offset=1)
    B.fsdp_mx4_quantize(s["master"], n, k, "f32", s["c_w"], s["s_w"], s["c_wt"], s["s_wt"], **kw)
    B.fsdp_norm_forward(s["h"], s["x"], m, k, kind="rms", weight=s["gamma"], rstd=s["rstd"], **kw)
    B.fsdp_mx4_quantize(s["h"], m, k, "bf16", s["c_h"], s["s_h"], s["c_ht"], s["s_ht"], **kw)
    B.fsdp_mx4_product(s["y"], s["c_h"], s["s_h"], s["c_w"], s["s_w"], m, n, k, residual=s["res"], act="gelu", z=s["z"],
                       dropout=drop, workspace=s["ws"], **kw)
    B.fsdp_linear_epilogue_backward(s["dz"], s["dy"], m, n, z=s["z"], act="gelu", dropout=drop, workspace=s["ws"], **kw)
    B.fsdp_mx4_quantize(s["dz"], m, n, "bf16", s["c_dz"], s["s_dz"], s["c_dzt"], s["s_dzt"], **kw)
    B.fsdp_mx4_product(s["dh"], s["c_dz"], s["s_dz"], s["c_wt"], s["s_wt"], m, k, n, workspace=s["ws"], **kw)
    B.fsdp_mx4_product(s["dw"], s["c_dzt"], s["s_dzt"], s["c_ht"], s["s_ht"], n, k, m, y_dtype="f32", residual=s["dw"],
                       workspace=s["ws"], **kw)
    B.fsdp_norm_backward(s["dx"], s["dh"], s["x"], m, k, kind="rms", weight=s["gamma"], rstd=s["rstd"], dw=s["dgamma"],
                         workspace=s["ws"], **kw)


IN, OUT = ("x", "gamma", "master", "dy", "res"), ("y", "z", "dz", "dh", "dx", "dw", "dgamma", "c_w", "s_wt", "c_dzt", "s_ht")
LAYERS = [(37, 100, 70), (16, 512, 256), (300, 520, 1100), (1000, 1365, 1024)]


@pytest.mark.parametrize("m,n,k", LAYERS)
def test_layer(gpu, m, n, k):
    """Each call against the oracle on what the calls before it wrote."""
    from oracle import norm as ON
    s = layer(gpu, m, n, k)
    layer_pass(s, m, n, k)
    v = {name: t.double().cpu().numpy() for name, t in s.items() if t.dtype in (torch.bfloat16, torch.float32)}
    q = {}
    for name, t in (("w", v["master"]), ("wt", v["master"].T), ("h", v["h"]), ("ht", v["h"].T), ("dz", v["dz"]), ("dzt", v["dz"].T)):
        q[name] = Q.quantize(np.ascontiguousarray(t))
        assert np.array_equal(s["c_" + name].cpu().numpy(), q[name][0]) and np.array_equal(s["s_" + name].cpu().numpy(), q[name][1]), name
    h, _, rstd = ON.forward(v["x"], v["gamma"][0], None, 1e-5, "rms")
    assert np.all(np.abs(v["h"] - h) <= (HALF["bf16"] + 100 * U) * np.abs(h) + 1e-30)
    z, zs, room = reference(*q["h"], *q["w"], k)
    ez = product_err(k, zs, room)
    close(v["z"], z, ez, "bf16", "z")
    f = OL.keep_factor(m, n, 0.1, 7, 1)
    y = OL.act(z, "gelu") * f
    close(v["y"], y + v["res"], act_err(z, ez, "gelu") * f + 4 * U * (np.abs(y) + np.abs(y + v["res"])), "bf16", "y")
    dh, s1, room = reference(*q["dz"], *q["wt"], n)
    close(v["dh"], dh, product_err(n, s1, room), "bf16", "dh")
    dw, s2, room = reference(*q["dzt"], *q["ht"], m)
    close(v["dw"], dw, product_err(m, s2, room) + 2 * U * np.abs(dw), "f32", "dw")
    xhat = v["x"] * v["rstd"][:, None]
    dgamma = (v["dh"] * xhat).sum(axis=0)
    close(v["dgamma"], dgamma, (m / 4 + 170) * U * np.abs(v["dh"] * xhat).sum(axis=0), "f32", "dgamma")


def test_layer_gradient_points_down(gpu):
    """The 4-bit layer's gradients against the float64 layer's: quantised to 4 bits
    both ways, an element is off by up to a sixth of itself or a twelfth of its
    block's largest (about 0.12 of the spread in the mean square for normal
    values), and a sum of products of two by about sqrt(2) times that, relative to
    its spread: under 0.25 of the norm."""
    m, n, k = 300, 520, 1100
    s = layer(gpu, m, n, k)
    s["res"].zero_()
    layer_pass(s, m, n, k)
    x, w, gamma, dy = (s[name].double() for name in ("x", "master", "gamma", "dy"))
    x, w, gamma = (t.clone().requires_grad_() for t in (x, w, gamma))
    h = x * torch.rsqrt((x * x).mean(1, keepdim=True) + 1e-5) * gamma
    z = h @ w.t()
    keep = torch.from_numpy(OL.keep_factor(m, n, 0.1, 7, 1)).cuda()
    (z * torch.special.ndtr(z) * keep).backward(dy)
    for got, want in ((s["dx"], x.grad), (s["dw"], w.grad), (s["dgamma"], gamma.grad[0])):
        assert float((got.double() - want).norm() / want.norm()) < 0.25


@pytest.mark.parametrize("m,n,k", LAYERS)
def test_two_streams_at_once(gpu, m, n, k):
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    sets, want = [layer(gpu, m, n, k, seed) for seed in (4, 5)], []
    for s in sets:
        layer_pass(s, m, n, k)
        want.append({name: s[name].clone() for name in OUT})
        for name in OUT:
            s[name].zero_()
    torch.cuda.synchronize()
    for _ in range(4):
        for s, stream in zip(sets, streams):
            with torch.cuda.stream(stream):
                s["dw"].zero_()
            layer_pass(s, m, n, k, stream)
    torch.cuda.synchronize()
    for s, w in zip(sets, want):
        assert all(torch.equal(s[name], w[name]) for name in OUT)


@pytest.mark.parametrize("m,n,k", LAYERS)
def test_captured_and_replayed(gpu, m, n, k):
    s = layer(gpu, m, n, k)
    layer_pass(s, m, n, k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s["dw"].zero_()
        layer_pass(s, m, n, k)
    for seed in (6, 7, 8):
        new = layer(gpu, m, n, k, seed)
        for name in IN:
            s[name].copy_(new[name])
        graph.replay()
        torch.cuda.synchronize()
        layer_pass(new, m, n, k)
        torch.cuda.synchronize()
        assert all(torch.equal(s[name], new[name]) for name in OUT), seed


def test_the_copy_between_two_steps(gpu):
    """The step's fp32 master weights quantised after each of two AdamW steps, and the
    product of the copy: what a rank's rows of the next all-gather hold."""
    from rank_step_amd.workloads import HPARAMS
    n, k, m = 96, 200, 24
    g = gen(12)
    p, mo, v = randn(g, n, k, 0.05), torch.zeros(n, k, device=gpu), torch.zeros(n, k, device=gpu)
    grads = randn(g, n, k, 0.1)
    c, sc = torch.empty(n, Q.code_bytes(k), dtype=torch.uint8, device=gpu), torch.empty(n, Q.scale_bytes(k), dtype=torch.uint8, device=gpu)
    a, asc, av, asv = packed(g, m, k)
    y = torch.empty(m, n, device=gpu)
    with B.MtPlan([dict(param_fp32=p, exp_avg=mo, exp_avg_sq=v, grad_slices=grads, slice_stride=n * k, shard_numel=n * k,
                        valid=n * k)], 1, "f32") as plan:
        for step in (1, 2):
            before = p.clone()
            plan.step(HPARAMS, step)
            B.fsdp_mx4_quantize(p, n, k, "f32", c, sc)
            B.fsdp_mx4_product(y, a.t, asc.t, c, sc, m, n, k, y_dtype="f32")
            torch.cuda.synchronize()
            assert not torch.equal(before, p)
            codes, scales = Q.quantize(p.double().cpu().numpy())
            assert np.array_equal(c.cpu().numpy(), codes) and np.array_equal(sc.cpu().numpy(), scales)
            want, s, room = reference(av, asv, codes, scales, k)
            close(y.double().cpu().numpy(), want, product_err(k, s, room), "f32", "y")


@pytest.mark.parametrize("ld", [0, 1, 5, 1 << 40])
def test_the_stride_of_a_single_row_says_nothing(gpu, space, ld):
    k, n = 300, 40
    g = gen(13)
    a, asc, av, asv = packed(g, 1, k)
    b, bsc, bv, bsv = packed(g, n, k)
    y, want = torch.empty(1, n, device=gpu), torch.empty(1, n, device=gpu)
    B.fsdp_mx4_product(want, a.t, asc.t, b.t, bsc.t, 1, n, k, y_dtype="f32", workspace=space)
    B.fsdp_mx4_product(y, a.ptr, asc.ptr, b.ptr, bsc.ptr, 1, n, k, y_dtype="f32", workspace=space, lda=ld, ldas=ld, ldy=ld)
    assert torch.equal(y, want)
    x = randn(g, 1, k)
    out = [torch.empty(1, w, dtype=torch.uint8, device=gpu) for w in (Q.code_bytes(k), Q.scale_bytes(k)) * 2]
    B.fsdp_mx4_quantize(x, 1, k, "f32", out[0], out[1])
    B.fsdp_mx4_quantize(x.data_ptr(), 1, k, "f32", out[2].data_ptr(), out[3].data_ptr(), ldx=ld, ldc=ld, lds=ld)
    assert torch.equal(out[0], out[2]) and torch.equal(out[1], out[3])
    v = [torch.empty(1, k, device=gpu) for _ in range(2)]
    B.fsdp_mx4_dequantize(v[0], out[0], out[1], 1, k, "f32")
    B.fsdp_mx4_dequantize(v[1].data_ptr(), out[0].data_ptr(), out[1].data_ptr(), 1, k, "f32", ldy=ld, ldc=ld, lds=ld)
    assert torch.equal(v[0], v[1])


def test_offsets_past_32_bits(gpu, space):
    """A matrix of 2.2 G elements, its copies and its values, the last rows and
    columns against the same of a small one; and products whose codes, scales and
    outputs lie past 2^32 bytes."""
    rows, cols = 540_032, 4096
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=gpu)
    tail = randn(gen(14), 64, cols).to(torch.bfloat16)
    x[-64:] = tail
    e = lambda r, c: torch.full((r, c), 0x77, dtype=torch.uint8, device=gpu)  # noqa: E731
    c, s, ct, st = e(rows, Q.code_bytes(cols)), e(rows, Q.scale_bytes(cols)), e(cols, Q.code_bytes(rows)), e(cols, Q.scale_bytes(rows))
    B.fsdp_mx4_quantize(x, rows, cols, codes=c, scales=s, codes_t=ct, scales_t=st)
    c2, s2, ct2, st2 = e(64, Q.code_bytes(cols)), e(64, Q.scale_bytes(cols)), e(cols, Q.code_bytes(64)), e(cols, Q.scale_bytes(64))
    B.fsdp_mx4_quantize(tail, 64, cols, codes=c2, scales=s2, codes_t=ct2, scales_t=st2)
    assert torch.equal(c[-64:], c2) and torch.equal(s[-64:], s2) and not bool(c[:-64].any()) and not bool(s[:-64].any())
    blocks = rows // 32
    assert torch.equal(ct[:, -32:], ct2) and torch.equal(st[:, blocks - 2:blocks], st2[:, :2])
    assert not bool(ct[:, :-32].any()) and not bool(st[:, :blocks - 2].any()) and not bool(st[:, blocks:].any())
    x.fill_(1.0)
    B.fsdp_mx4_dequantize(x, c, s, rows, cols)
    v2 = torch.empty_like(tail)
    B.fsdp_mx4_dequantize(v2, c2, s2, 64, cols)
    assert torch.equal(x[-64:], v2) and not bool(x[:-64].any())
    # y [rows, 4096] in bf16 is 4.4 GB; A's codes are read to their end
    b, bs = c2[:32].repeat(128, 1), s2[:32].repeat(128, 1)
    B.fsdp_mx4_product(x, c, s, b, bs, rows, cols, cols, workspace=space)
    y2 = torch.empty(64, cols, dtype=torch.bfloat16, device=gpu)
    B.fsdp_mx4_product(y2, c2, s2, b, bs, 64, cols, cols)
    assert float((x[-64:].float() - y2.float()).abs().max()) <= 2.0 ** -7 * float(y2.float().abs().max())
    assert not bool(x[:-64].any())
    del x, ct, st
    # rows of codes 2^22 bytes apart: the last of 1100 rows lies past 2^32
    big = torch.zeros(1100 << 22, dtype=torch.uint8, device=gpu)
    wide = big.view(1100, 1 << 22)[:, :Q.code_bytes(cols)]
    wide[-64:] = c2
    sc = torch.zeros(1100, Q.scale_bytes(cols), dtype=torch.uint8, device=gpu)
    sc[-64:] = s2
    y = torch.empty(1100, cols, dtype=torch.bfloat16, device=gpu)
    B.fsdp_mx4_product(y, big, sc, b, bs, 1100, cols, cols, lda=1 << 22, workspace=space)
    assert float((y[-64:].float() - y2.float()).abs().max()) <= 2.0 ** -7 * float(y2.float().abs().max())
    assert not bool(y[:-64].any())
