"""The norm's calls refuse what they cannot do (CPU only): every bad argument
comes back with its code before any device work.  The cases carry device
addresses that are never touched."""

import os
import re

import pytest

from rank_step_amd import binding as B
from tests.test_linear_host import Space

X, Y, DX, DY, R, W, BIAS, MEAN, RSTD, DW, DB, WS = (0x10000000 * i for i in range(1, 13))
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def forward(**kw):
    a = dict(y=Y, x=X, m=4, n=8, weight=W, bias=BIAS, mean=MEAN, rstd=RSTD, stream=0)
    a.update(kw)
    B.fsdp_norm_forward(**a)


def backward(**kw):
    a = dict(dx=DX, dy=DY, x=X, m=4, n=8, weight=W, mean=MEAN, rstd=RSTD, residual=R, dw=DW, db=DB, stream=0)
    a.update(kw)
    B.fsdp_norm_backward(**a)


BAD = [
    (forward, dict(x=None), "FSDP_E_ARG"),
    (forward, dict(y=None), "FSDP_E_ARG"),
    (forward, dict(m=-1), "FSDP_E_ARG"),
    (forward, dict(n=-1), "FSDP_E_ARG"),
    (forward, dict(m=(1 << 30) + 1), "FSDP_E_CAPACITY"),
    (forward, dict(n=(1 << 30) + 1), "FSDP_E_CAPACITY"),
    (forward, dict(dtype=2), "FSDP_E_DTYPE"),
    (forward, dict(w_dtype=2), "FSDP_E_DTYPE"),
    (forward, dict(kind=2), "FSDP_E_ARG"),
    (forward, dict(kind=-1), "FSDP_E_ARG"),
    (forward, dict(kind="rms"), "FSDP_E_ARG"),  # with a mean
    (forward, dict(eps=-1e-9), "FSDP_E_ARG"),
    (forward, dict(eps=float("nan")), "FSDP_E_ARG"),
    (forward, dict(eps=float("inf")), "FSDP_E_ARG"),
    (forward, dict(eps=1e39), "FSDP_E_ARG"),  # infinite in fp32
    (forward, dict(ldx=7), "FSDP_E_ARG"),
    (forward, dict(ldy=7), "FSDP_E_ARG"),
    (forward, dict(ldx=1 << 62), "FSDP_E_ARG"),
    (forward, dict(x=X + 1), "FSDP_E_ALIGN"),
    (forward, dict(x=X + 2, dtype="f32"), "FSDP_E_ALIGN"),
    (forward, dict(weight=W + 1), "FSDP_E_ALIGN"),
    (forward, dict(bias=BIAS + 2, w_dtype="f32"), "FSDP_E_ALIGN"),
    (forward, dict(mean=MEAN + 2), "FSDP_E_ALIGN"),
    (forward, dict(rstd=RSTD + 1), "FSDP_E_ALIGN"),
    (forward, dict(y=X + 2), "FSDP_E_ALIAS"),
    (forward, dict(y=X, ldy=9), "FSDP_E_ALIAS"),
    (forward, dict(mean=RSTD), "FSDP_E_ALIAS"),
    (forward, dict(mean=X), "FSDP_E_ALIAS"),
    (forward, dict(rstd=Y + 60), "FSDP_E_ALIAS"),
    (forward, dict(weight=Y), "FSDP_E_ALIAS"),
    (forward, dict(bias=MEAN), "FSDP_E_ALIAS"),
    (backward, dict(dy=None), "FSDP_E_ARG"),
    (backward, dict(x=None), "FSDP_E_ARG"),
    (backward, dict(rstd=None), "FSDP_E_ARG"),
    (backward, dict(mean=None), "FSDP_E_ARG"),
    (backward, dict(kind="rms"), "FSDP_E_ARG"),  # with a mean
    (backward, dict(kind=2), "FSDP_E_ARG"),
    (backward, dict(m=-1), "FSDP_E_ARG"),
    (backward, dict(n=(1 << 30) + 1), "FSDP_E_CAPACITY"),
    (backward, dict(dtype=3), "FSDP_E_DTYPE"),
    (backward, dict(w_dtype=-1), "FSDP_E_DTYPE"),
    (backward, dict(dw_dtype=2), "FSDP_E_DTYPE"),
    (backward, dict(accumulate=2), "FSDP_E_ARG"),
    (backward, dict(lddx=7), "FSDP_E_ARG"),
    (backward, dict(lddy=7), "FSDP_E_ARG"),
    (backward, dict(ldx=7), "FSDP_E_ARG"),
    (backward, dict(ldr=7), "FSDP_E_ARG"),
    (backward, dict(dw=DW + 2), "FSDP_E_ALIGN"),
    (backward, dict(db=DB + 1, dw_dtype="bf16"), "FSDP_E_ALIGN"),
    (backward, dict(rstd=RSTD + 2), "FSDP_E_ALIGN"),
    (backward, dict(workspace=Space(WS + 8, 64)), "FSDP_E_ALIGN"),
    (backward, dict(workspace=Space(0, 64)), "FSDP_E_ARG"),
    (backward, dict(workspace=Space(WS, -1)), "FSDP_E_ARG"),
    (backward, dict(workspace=Space(DX, 64)), "FSDP_E_ALIAS"),
    (backward, dict(workspace=Space(RSTD, 64)), "FSDP_E_ALIAS"),
    (backward, dict(dx=DY), "FSDP_E_ALIAS"),
    (backward, dict(dx=X), "FSDP_E_ALIAS"),
    (backward, dict(dx=R + 2), "FSDP_E_ALIAS"),
    (backward, dict(dx=R, lddx=9), "FSDP_E_ALIAS"),
    (backward, dict(dw=DB), "FSDP_E_ALIAS"),
    (backward, dict(dw=W), "FSDP_E_ALIAS"),
    (backward, dict(db=RSTD), "FSDP_E_ALIAS"),
]


@pytest.mark.parametrize("call,kw,code", BAD)
def test_refusals(call, kw, code):
    with pytest.raises(B.FsdpError) as e:
        call(**kw)
    assert e.value.name == code, str(e.value)


def _wrong_tensors():
    import torch
    b, f = torch.bfloat16, torch.float32

    def t(r, c, dt=b):
        return torch.zeros(r, c, dtype=dt)

    return [
        (forward, dict(x=t(4, 8, f)), "FSDP_E_DTYPE", "x is torch.float32"),
        (forward, dict(y=t(4, 8), dtype="f32"), "FSDP_E_DTYPE", "y is"),
        (forward, dict(weight=t(1, 8, f)), "FSDP_E_DTYPE", "weight is"),
        (forward, dict(bias=t(1, 8), w_dtype="f32"), "FSDP_E_DTYPE", "bias is"),
        (forward, dict(mean=t(1, 4)), "FSDP_E_DTYPE", "mean is"),
        (forward, dict(rstd=t(1, 4, torch.float64)), "FSDP_E_DTYPE", "rstd is"),
        (forward, dict(x=t(8, 4).t()), "FSDP_E_ARG", "not contiguous"),
        (forward, dict(y=t(3, 8)), "FSDP_E_ARG", "room"),
        (forward, dict(weight=t(1, 7)), "FSDP_E_ARG", "room"),
        (forward, dict(rstd=t(1, 3, f)), "FSDP_E_ARG", "room"),
        (forward, dict(x=t(4, 8)), "FSDP_E_ARG", "on cpu"),
        (backward, dict(dx=t(4, 8, f)), "FSDP_E_DTYPE", "dx is"),
        (backward, dict(dw=t(1, 8)), "FSDP_E_DTYPE", "dw is"),  # dw_dtype is f32 unless given
        (backward, dict(db=t(1, 8, f), dw_dtype="bf16"), "FSDP_E_DTYPE", "db is"),
        (backward, dict(residual=t(4, 7)), "FSDP_E_ARG", "room"),
        (backward, dict(dy=t(4, 16)[:, 8:]), "FSDP_E_ARG", "not contiguous"),
        (backward, dict(mean=t(1, 4, f)), "FSDP_E_ARG", "on cpu"),
        (backward, dict(workspace=torch.zeros(64, dtype=torch.uint8)), "FSDP_E_ARG", "on cpu"),
    ]


@pytest.mark.parametrize("i", range(18))
def test_tensors_that_do_not_hold_the_operand(i):
    cases = _wrong_tensors()
    assert len(cases) == 18
    call, kw, code, words = cases[i]
    with pytest.raises(B.FsdpError) as e:
        call(**kw)
    assert e.value.name == code and words in str(e.value), str(e.value)


def test_empty_outputs_are_no_ops():
    """Nothing is queued (there is no device here to queue on), null or not."""
    forward(m=0, x=None, y=None)
    forward(n=0, x=None, y=None, weight=None)
    backward(n=0, dx=None, dy=None, x=None, rstd=None, mean=None, residual=None)
    backward(m=0, dx=None, dy=None, x=None, residual=None, accumulate=True)
    backward(m=0, dw=None, db=None)
    backward(dx=None, dw=None, db=None)


def test_constants():
    text = open(os.path.join(ROOT, "include", "fsdp_norm.h")).read()
    assert re.search(r"FSDP_NORM_WORKSPACE_BYTES \(\(int64_t\)64 << 20\)", text)
    assert B.NORM_WORKSPACE_BYTES == 64 << 20
    for name, value in B.NORMS.items():
        assert re.search(r"FSDP_NORM_%s = %d\b" % (name.upper(), value), text), name
