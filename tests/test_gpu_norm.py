"""The norm's calls on the GPU against the float64 oracle.

Each input lies in a buffer whose other elements (before it, after it, and
between its rows) are NaN, so that reading one into a result shows; each output
in a buffer of a fixed pattern that must be whole outside the output afterwards.

Tolerances, with u = 2^-24 (half an fp32 step) and L = 64 + n / 1024, which no
chain of a row's additions is longer than (32 in a lane, 6 over a wave, 16 over
waves; rows that registers do not hold: n / 1024 in a thread):

* mean: its first estimate is off by L u of the mean magnitude and u of itself;
  where it exceeds four times the spread it is corrected by the mean distance
  from that, so L u of the spread, and 2u of itself;
* variance: (L + 8) u of itself (and of the square of the mean's error), so
  half of that in rstd, with 4u for eps, the root and the quotient;
* y: those, 4u of the value for its four operations;
* the gradient's two sums: (L + 8) u of their terms' magnitudes over n; 6u of
  the magnitudes that form dx;
* column sums: each term passes through at most m / 4 + 160 additions (rows of a
  thread, then 16 parts at a time), u of the terms' magnitudes each, and 4u for
  the terms;
* half a step of the output's type, and 2^-133 for subnormal bf16.
"""

import numpy as np
import pytest
import torch

from oracle import norm as ON
from rank_step_amd import binding as B
from tests.test_gpu_linear import HALF, U, Mat, gen, randn

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -133
EPS = 1e-5


def close(got, ref, err, dtype, what):
    tol = err + HALF[dtype] * (np.abs(ref) + err) + TINY
    off = np.abs(got - ref) / tol
    bad = ~(off <= 1)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, worst {np.nanmax(off):.3g} at "
                           f"{np.argwhere(bad)[0].tolist()}, {got[bad][0]} against {ref[bad][0]}")


@pytest.fixture(scope="module")
def space(gpu):
    return torch.empty(B.NORM_WORKSPACE_BYTES, dtype=torch.uint8, device=gpu)


def activations(g, m, n, shift=0.5):
    return randn(g, m, n) * (1 + 0.2 * randn(g, 1, n)) + shift * randn(g, 1, n)


def check_forward(m, n, dtype="bf16", kind="layer", wt="bf16", weight=True, bias=True, stats=True, off=0, pad=0,
                  same=False, eps=EPS, values=None, seed=1):
    g = gen(seed)
    x = Mat(m, n, dtype, activations(g, m, n) if values is None else values, off, pad)
    w = Mat(1, n, wt, 1 + 0.1 * randn(g, 1, n), off) if weight else None
    b = Mat(1, n, wt, 0.1 * randn(g, 1, n), off) if bias else None
    y = x if same else Mat(m, n, dtype, None, off, pad)
    mean = Mat(1, m, "f32", None, off) if stats and kind == "layer" else None
    rstd = Mat(1, m, "f32", None, off) if stats else None
    xv = x.np()
    ptr = lambda t: None if t is None else t.ptr  # noqa: E731
    B.fsdp_norm_forward(y.ptr, x.ptr, m, n, dtype=dtype, kind=kind, weight=ptr(w), bias=ptr(b), w_dtype=wt, eps=eps,
                        mean=ptr(mean), rstd=ptr(rstd), ldy=y.ld, ldx=x.ld)
    torch.cuda.synchronize()
    wv, bv = (None if t is None else t.np()[0] for t in (w, b))
    yv, mv, rv = ON.forward(xv, wv, bv, eps, kind)
    long = 64 + n / 1024
    var = ((xv - mv[:, None]) ** 2).mean(axis=1)  # of the values: 1 / rstd^2 - eps cancels where eps is the larger
    if kind == "layer":
        first = long * U * np.abs(xv).mean(axis=1) + U * np.abs(mv)  # the first estimate's error
        near = mv * mv < 17 * var
        em = 2 * U * np.abs(mv) + (long + 3) * U * (np.sqrt(var) + first) + np.where(near, first, 0)
    else:
        first, em = 0 * mv, 0 * mv
    er = rv * (0.5 * (long + 8) * U * (var + first ** 2 + em ** 2) * rv ** 2 + 4 * U)
    close(rstd.np()[0], rv, er, "f32", "rstd") if rstd else None
    close(mean.np()[0], mv, em, "f32", "mean") if mean else None
    aw = 1.0 if wv is None else np.abs(wv)
    d = np.abs(xv - mv[:, None])
    ey = (em[:, None] * rv[:, None] + d * er[:, None] + 3 * U * d * rv[:, None]) * aw + U * np.abs(yv)
    close(y.np(), yv, ey, dtype, "y")
    for t in (None if same else y, mean, rstd):
        if t is not None:
            t.check_surroundings()


def check_backward(m, n, space, dtype="bf16", kind="layer", wt="bf16", weight=True, residual=False, dx=True, dw=True,
                   db=True, dwt="f32", add=False, off=0, pad=0, same=False, seed=2):
    g = gen(seed)
    x = Mat(m, n, dtype, activations(g, m, n), off, pad)
    dy = Mat(m, n, dtype, randn(g, m, n, 1e-3), off, pad)
    w = Mat(1, n, wt, 1 + 0.1 * randn(g, 1, n), off) if weight else None
    r = Mat(m, n, dtype, randn(g, m, n, 1e-3), off, pad) if residual else None
    out = r if same else Mat(m, n, dtype, None, off, pad) if dx else None
    old = {name: Mat(1, n, dwt, randn(g, 1, n, 1e-2) if add else None, off) for name, want in (("dw", dw), ("db", db)) if want}
    before = {name: t.np()[0] if add else 0.0 for name, t in old.items()}
    xv, dyv, resv = x.np(), dy.np(), r.np() if residual else 0.0
    wv = w.np()[0] if weight else None
    _, mv, rv = ON.forward(xv, None, None, EPS, kind)
    mean = torch.from_numpy(mv).float().cuda() if kind == "layer" else None
    rstd = torch.from_numpy(rv).float().cuda()
    mv, rv = mean.double().cpu().numpy() if kind == "layer" else 0 * mv, rstd.double().cpu().numpy()
    ptr = lambda t: None if t is None else t.ptr  # noqa: E731
    B.fsdp_norm_backward(ptr(out), dy.ptr, x.ptr, m, n, dtype=dtype, kind=kind, weight=ptr(w), w_dtype=wt, mean=mean,
                         rstd=rstd, residual=ptr(r), dw=ptr(old.get("dw")), db=ptr(old.get("db")), dw_dtype=dwt,
                         accumulate=add, workspace=space, lddx=out.ld if out else None, lddy=dy.ld, ldx=x.ld,
                         ldr=r.ld if r else None)
    torch.cuda.synchronize()
    dxv, dwv, dbv = ON.backward(dyv, xv, mv, rv, wv, kind)
    long = 64 + n / 1024
    xhat = np.abs(xv - mv[:, None]) * rv[:, None]
    ag = np.abs(dyv if wv is None else dyv * wv)
    if out is not None:
        m1 = ag.mean(axis=1, keepdims=True) if kind == "layer" else 0.0
        m2 = (ag * xhat).mean(axis=1, keepdims=True)
        e = rv[:, None] * ((long + 8) * U * (m1 + xhat * m2) + 6 * U * (ag + m1 + xhat * m2))
        close(out.np(), dxv + resv, e + 2 * U * np.abs(dxv + resv), dtype, "dx")
        if not same:
            out.check_surroundings()
    for name, v, mag in (("dw", dwv, (np.abs(dyv) * xhat).sum(axis=0)), ("db", dbv, np.abs(dyv).sum(axis=0))):
        if name not in old:
            continue
        v = v + before[name]
        close(old[name].np()[0], v, (m / 4 + 164) * U * mag + 2 * U * np.abs(v), dwt, name)
        if not add:
            old[name].check_surroundings()


# rows shorter than a 16-byte chunk, one chunk, around each division of a row, and too long for registers
WIDTHS = [1, 2, 3, 5, 7, 8, 9, 64, 251, 256, 257, 511, 512, 513, 1024, 1025, 1365, 2048, 2049, 4096, 4097, 8192, 8193,
          11008, 16384, 16385, 32768, 32769, 40001]


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward_widths(gpu, n, dtype):
    other = "f32" if dtype == "bf16" else "bf16"
    check_forward(5, n, dtype, "layer", dtype)
    check_forward(3, n, dtype, "rms", other, bias=False)
    check_forward(2, n, dtype, "layer", other, stats=False, off=3, pad=5)
    check_forward(6, n, dtype, "rms", dtype, off=1, pad=0)


@pytest.mark.parametrize("m", [0, 1, 2, 4, 333, 1000, 8195, 70001])
@pytest.mark.parametrize("n", [24, 100, 1365])
def test_forward_rows(gpu, m, n):
    check_forward(m, n)
    check_forward(m, n, "f32", "rms", "f32", weight=False, bias=False)


@pytest.mark.parametrize("m,n", [(2100, 4096), (4300, 2056), (600, 16384), (520, 33000)])
def test_forward_several_rows_a_workgroup(gpu, m, n):
    check_forward(m, n)
    check_forward(m, n, "bf16", "rms")
    check_forward(m // 2, n // 2, "f32", "layer", "f32", pad=3)


@pytest.mark.parametrize("weight,bias,stats", [(False, False, False), (True, False, True), (False, True, True)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_forward_parts(gpu, weight, bias, stats, kind):
    for n in (40, 520, 5000, 40000):
        check_forward(9, n, "bf16", kind, "f32", weight, bias, stats)
        check_forward(9, n, "f32", kind, "bf16", weight, bias, stats)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("n", [7, 1000, 4096, 9000, 40000])
def test_forward_in_place(gpu, kind, n):
    check_forward(37, n, "bf16", kind, same=True, off=1, pad=3)
    check_forward(37, n, "f32", kind, same=True)


@pytest.mark.parametrize("n", [64, 1365, 4096, 40000])
def test_a_mean_far_from_zero(gpu, n):
    """Rows whose spread is a thousandth of their mean, and constant rows."""
    g = gen(5)
    check_forward(20, n, "f32", values=1000 + randn(g, 20, n))
    check_forward(20, n, "f32", values=torch.full((20, n), 1234.5, device=gpu))
    check_forward(20, n, "bf16", values=torch.full((20, n), -3.0, device=gpu))
    check_forward(20, n, "f32", "rms", values=torch.zeros(20, n, device=gpu))
    check_forward(20, n, "f32", values=1e-20 * randn(g, 20, n))
    check_forward(20, n, "f32", values=1e15 * randn(g, 20, n))


@pytest.mark.parametrize("n", [5, 64, 1365, 4096, 40000])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_nonfinite_values_stay_in_their_rows(gpu, n, kind):
    x = randn(gen(6), 12, n)
    x[3, n - 1], x[5, 0], x[7, n // 2] = float("nan"), float("inf"), float("-inf")
    y = torch.empty_like(x)
    rstd = torch.empty(12, device=gpu)
    B.fsdp_norm_forward(y, x, 12, n, dtype="f32", kind=kind, rstd=rstd)
    rows = torch.tensor([3, 5, 7], device=gpu)
    others = torch.tensor([i for i in range(12) if i not in (3, 5, 7)], device=gpu)
    if kind == "layer":
        assert bool(y[rows].isnan().all())
    else:
        assert bool(y[3].isnan().all()) and bool(y[5, 0].isnan()) and bool(y[7, n // 2].isnan())
    assert bool(y[others].isfinite().all()) and bool(rstd[others].isfinite().all())
    dx, dw = torch.empty_like(x), torch.empty(n, device=gpu)
    mean = torch.zeros(12, device=gpu) if kind == "layer" else None
    B.fsdp_norm_backward(dx, y, x, 12, n, dtype="f32", kind=kind, mean=mean, rstd=torch.ones(12, device=gpu), dw=dw)
    assert bool(dx[3].isnan().all()) and bool(dx[others].isfinite().all())


def test_eps(gpu):
    check_forward(7, 100, "f32", eps=0.0)
    check_forward(7, 100, "f32", eps=1e3)
    x = torch.ones(3, 16, device=gpu)
    B.fsdp_norm_forward(x, x, 3, 16, dtype="f32", eps=0.0)
    assert bool(x.isnan().all())


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_widths(gpu, space, n, dtype):
    other = "f32" if dtype == "bf16" else "bf16"
    check_backward(5, n, space, dtype, "layer", dtype, residual=True)
    check_backward(3, n, space, dtype, "rms", other, dwt="bf16", add=True, db=False)
    check_backward(6, n, None, dtype, "layer", other, off=3, pad=5, add=True)
    check_backward(6, n, space, dtype, "rms", dtype, residual=True, off=1, pad=0, dw=False)


@pytest.mark.parametrize("m", [0, 1, 2, 7, 333, 511, 513, 1000, 8195, 70001])
@pytest.mark.parametrize("n", [24, 100, 1365])
def test_backward_rows(gpu, space, m, n):
    check_backward(m, n, space)
    check_backward(m, n, space, "f32", "rms", "f32", weight=False, add=True, dwt="f32")


@pytest.mark.parametrize("m,n", [(2100, 4096), (4300, 2056), (600, 16384), (520, 33000)])
def test_backward_several_rows_a_workgroup(gpu, space, m, n):
    check_backward(m, n, space, residual=True)
    check_backward(m, n, space, "bf16", "rms", dwt="bf16", add=True)
    check_backward(m // 2, n // 2, space, "f32", "layer", "f32", residual=True, pad=3)


@pytest.mark.parametrize("size", [0, 16, 4 << 10, 64 << 10, 300 << 10, 1 << 20, 8 << 20])
@pytest.mark.parametrize("m,n", [(700, 96), (700, 4096), (300, 20000)])
def test_backward_workspaces(gpu, size, m, n):
    """Room for no part of the sums, for some, for all; what lies behind the workspace stays."""
    buf = torch.full((size + 64,), 0x5A, dtype=torch.uint8, device=gpu)
    ws = buf[:size] if size else None
    check_backward(m, n, ws, residual=True)
    check_backward(m, n, ws, "f32", "rms", dx=False, add=True)
    assert bool((buf[size:] == 0x5A).all())


@pytest.mark.parametrize("dx,dw,db", [(True, False, False), (False, True, False), (False, False, True), (True, True, False),
                                      (True, False, True), (False, True, True)])
def test_backward_parts(gpu, space, dx, dw, db):
    for m, n in ((9, 40), (9, 5000), (9, 40000), (700, 520)):
        check_backward(m, n, space, "bf16", "layer", dx=dx, dw=dw, db=db)
        check_backward(m, n, space, "f32", "rms", weight=False, dx=dx, dw=dw, db=db, dwt="bf16", add=True)


@pytest.mark.parametrize("n", [7, 1000, 4096, 9000, 40000])
def test_backward_residual_in_place(gpu, space, n):
    check_backward(37, n, space, "bf16", residual=True, same=True, off=1, pad=3)
    check_backward(37, n, space, "f32", "rms", residual=True, same=True)


def test_gradients_against_differences(gpu, space):
    """dx, dw and db against central differences of the GPU's own forward pass in
    fp32: with h = 2^-7 the loss of 6 rows of 40 is off by about 240 * 4u of its
    terms (each under 4), 2e-4 over 2h, and by h^2 / 6 of a third derivative
    (under 20), 2e-4."""
    m, n, h = 6, 40, 2.0 ** -7
    for kind in ("layer", "rms"):
        g = gen(9)
        x, dy, w, b = randn(g, m, n), randn(g, m, n), 1 + 0.3 * randn(g, 1, n), randn(g, 1, n)
        y, rstd = torch.empty_like(x), torch.empty(m, device=gpu)
        mean = torch.empty(m, device=gpu) if kind == "layer" else None

        def loss(x, w, b):
            B.fsdp_norm_forward(y, x.contiguous(), m, n, dtype="f32", kind=kind, weight=w.contiguous(),
                                bias=b.contiguous(), w_dtype="f32", mean=mean, rstd=rstd)
            return float((y.double() * dy.double()).sum())

        loss(x, w, b)
        dx, dw, db = torch.empty_like(x), torch.empty(n, device=gpu), torch.empty(n, device=gpu)
        B.fsdp_norm_backward(dx, dy, x, m, n, dtype="f32", kind=kind, weight=w, w_dtype="f32", mean=mean, rstd=rstd,
                             dw=dw, db=db, workspace=space)
        for i, j in ((0, 0), (2, 17), (5, 39)):
            e = torch.zeros_like(x)
            e[i, j] = h
            assert abs((loss(x + e, w, b) - loss(x - e, w, b)) / (2 * h) - float(dx[i, j])) < 4e-4 * 2
            e = torch.zeros_like(w)
            e[0, j] = h
            assert abs((loss(x, w + e, b) - loss(x, w - e, b)) / (2 * h) - float(dw[j])) < 4e-4 * 2
            assert abs((loss(x, w, b + e) - loss(x, w, b - e)) / (2 * h) - float(db[j])) < 4e-4 * 2


def layer(gpu, m, n, dtype, seed=11):
    g = gen(seed)
    tt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    s = dict(x=activations(g, m, n).to(tt), dy=randn(g, m, n).to(tt), w=(1 + 0.1 * randn(g, 1, n)).to(tt),
             b=randn(g, 1, n).to(tt), res=randn(g, m, n).to(tt))
    s |= dict(y=torch.empty_like(s["x"]), dx=torch.empty_like(s["x"]), mean=torch.empty(m, device=gpu),
              rstd=torch.empty(m, device=gpu), dw=torch.empty(n, device=gpu), db=torch.empty(n, device=gpu),
              ws=torch.empty(16 << 20, dtype=torch.uint8, device=gpu))
    return s


def both_passes(s, m, n, dtype, stream=None):
    B.fsdp_norm_forward(s["y"], s["x"], m, n, dtype=dtype, weight=s["w"], bias=s["b"], w_dtype=dtype, mean=s["mean"],
                        rstd=s["rstd"], stream=stream)
    B.fsdp_norm_backward(s["dx"], s["dy"], s["x"], m, n, dtype=dtype, weight=s["w"], w_dtype=dtype, mean=s["mean"],
                         rstd=s["rstd"], residual=s["res"], dw=s["dw"], db=s["db"], workspace=s["ws"], stream=stream)


OUT = ("y", "mean", "rstd", "dx", "dw", "db")
PASSES = [(700, 40, "bf16"), (333, 1365, "f32"), (1500, 4096, "bf16"), (90, 40000, "bf16")]


@pytest.mark.parametrize("m,n,dtype", PASSES)
def test_the_same_bits_again(gpu, m, n, dtype):
    s = layer(gpu, m, n, dtype)
    both_passes(s, m, n, dtype)
    first = {k: s[k].clone() for k in OUT}
    for k in OUT:
        s[k].fill_(float("nan"))
    s["ws"].fill_(0xFF)
    both_passes(s, m, n, dtype)
    assert all(torch.equal(first[k], s[k]) for k in OUT)


@pytest.mark.parametrize("m,n,dtype", PASSES)
def test_two_streams_at_once(gpu, m, n, dtype):
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    sets = [layer(gpu, m, n, dtype, seed) for seed in (11, 12)]
    want = []
    for s in sets:
        both_passes(s, m, n, dtype)
        want.append({k: s[k].clone() for k in OUT})
        for k in OUT:
            s[k].fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, stream in zip(sets, streams):
            both_passes(s, m, n, dtype, stream)
    torch.cuda.synchronize()
    for s, w in zip(sets, want):
        assert all(torch.equal(w[k], s[k]) for k in OUT)


@pytest.mark.parametrize("m,n,dtype", PASSES)
def test_captured_and_replayed(gpu, m, n, dtype):
    s = layer(gpu, m, n, dtype)
    both_passes(s, m, n, dtype)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both_passes(s, m, n, dtype)
    for seed in (21, 22, 23):
        new = layer(gpu, m, n, dtype, seed)
        for k in ("x", "dy", "w", "b", "res"):
            s[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        both_passes(new, m, n, dtype)
        torch.cuda.synchronize()
        assert all(torch.equal(new[k], s[k]) for k in OUT), seed


def test_offsets_past_32_bits(gpu, space):
    """2.2 G elements, bf16: the last rows against the oracle, and the column sums
    of ones exactly."""
    m, n = 540_000, 4096
    x = torch.empty(m, n, dtype=torch.bfloat16, device=gpu)
    tail = activations(gen(3), 64, n).to(torch.bfloat16)
    x[:-64] = 1.0
    x[-64:] = tail
    y = torch.empty_like(x)
    mean, rstd = torch.empty(m, device=gpu), torch.empty(m, device=gpu)
    B.fsdp_norm_forward(y, x, m, n, mean=mean, rstd=rstd)
    small = torch.empty_like(tail)
    sm, sr = torch.empty(64, device=gpu), torch.empty(64, device=gpu)
    B.fsdp_norm_forward(small, tail, 64, n, mean=sm, rstd=sr)
    assert torch.equal(y[-64:], small) and torch.equal(mean[-64:], sm) and torch.equal(rstd[-64:], sr)
    assert not bool(y[:-64].any())
    # dy = 1 everywhere: db counts rows (a power of two times a small number: exact in fp32)
    y.fill_(1.0)
    db = torch.empty(n, device=gpu)
    dx = torch.empty_like(x)
    B.fsdp_norm_backward(dx, y, x, m, n, mean=mean, rstd=rstd, db=db, workspace=space)
    assert bool((db == m).all())
    # the last rows' dx, which rounding alone makes other than 0: few rows may be summed in another order
    dsmall = torch.empty_like(tail)
    B.fsdp_norm_backward(dsmall, torch.ones_like(tail), tail, 64, n, mean=sm, rstd=sr)
    tv, mv, rv = (t.double().cpu().numpy() for t in (tail, sm, sr))
    want = ON.backward(np.ones_like(tv), tv, mv, rv)[0]
    xhat = np.abs(tv - mv[:, None]) * rv[:, None]
    m2 = xhat.mean(axis=1, keepdims=True)
    e = rv[:, None] * ((64 + n / 1024 + 8) * U * (1 + xhat * m2) + 6 * U * (2 + xhat * m2))
    close(dx[-64:].double().cpu().numpy(), want, e, "bf16", "dx")
    close(dsmall.double().cpu().numpy(), want, e, "bf16", "dx of few rows")
