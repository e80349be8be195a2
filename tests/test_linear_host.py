"""The linear layer's calls refuse what they cannot do (CPU only): every bad
argument comes back with its code before any device work.  The cases carry
device addresses that are never touched."""

import ctypes

import pytest

from rank_step_amd import binding as B

X, W, Y, Z, R, DZ, DB, WS = (0x10000000 * i for i in range(1, 9))
S = 0  # the null stream, never used


def forward(**kw):
    a = dict(y=Y, x=X, w=W, m=4, n=8, k=16, stream=S)
    a.update(kw)
    B.fsdp_linear_forward(**a)


def backward(**kw):
    a = dict(dz=DZ, dy=Y, m=4, n=8, z=Z, act="gelu", db=DB, stream=S)
    a.update(kw)
    B.fsdp_linear_epilogue_backward(**a)


def grad_input(**kw):
    a = dict(dx=X, dz=DZ, w=W, m=4, n=8, k=16, stream=S)
    a.update(kw)
    B.fsdp_linear_grad_input(**a)


def grad_weight(**kw):
    a = dict(dw=W, dz=DZ, x=X, m=4, n=8, k=16, stream=S)
    a.update(kw)
    B.fsdp_linear_grad_weight(**a)


def dropout(**kw):
    a = dict(y=Y, x=X, rows=4, cols=8, dtype="bf16", dropout={"p": 0.5, "seed": 1, "offset": 2}, stream=S)
    a.update(kw)
    B.fsdp_dropout(**a)


P = {"p": 0.5, "seed": 1, "offset": 2}


class Space:
    """A workspace as the binding takes it: an address and a size."""

    def __init__(self, ptr, size):
        self.ptr, self.size = ptr, size

    def data_ptr(self):
        return self.ptr

    def numel(self):
        return self.size

    def element_size(self):
        return 1


BAD = [
    (forward, dict(x=None), "FSDP_E_ARG"),
    (forward, dict(w=None), "FSDP_E_ARG"),
    (forward, dict(y=None), "FSDP_E_ARG"),
    (forward, dict(m=-1), "FSDP_E_ARG"),
    (forward, dict(k=-1), "FSDP_E_ARG"),
    (forward, dict(ldx=15), "FSDP_E_ARG"),
    (forward, dict(ldw=15), "FSDP_E_ARG"),
    (forward, dict(ldy=7), "FSDP_E_ARG"),
    (forward, dict(z=Z, ldz=7), "FSDP_E_ARG"),
    (forward, dict(residual=R, ldr=7), "FSDP_E_ARG"),
    (forward, dict(m=(1 << 30) + 1), "FSDP_E_CAPACITY"),
    (forward, dict(n=1 << 31), "FSDP_E_CAPACITY"),
    (forward, dict(ldx=1 << 62), "FSDP_E_ARG"),
    (forward, dict(w_dtype=0), "FSDP_E_DTYPE"),
    (forward, dict(w_dtype=3), "FSDP_E_DTYPE"),
    (forward, dict(y_dtype=2), "FSDP_E_DTYPE"),
    (forward, dict(w_dtype="e4m3"), "FSDP_E_ARG"),
    (forward, dict(w_scale=R), "FSDP_E_ARG"),
    (forward, dict(w_dtype="e4m3", w_scale=R + 2), "FSDP_E_ALIGN"),
    (forward, dict(act=4), "FSDP_E_ARG"),
    (forward, dict(act=-1), "FSDP_E_ARG"),
    (forward, dict(x=X + 1), "FSDP_E_ALIGN"),
    (forward, dict(y=Y + 2, y_dtype="f32"), "FSDP_E_ALIGN"),
    (forward, dict(bias=R + 1), "FSDP_E_ALIGN"),
    (forward, dict(residual=R + 2, y_dtype="f32"), "FSDP_E_ALIGN"),
    (forward, dict(workspace=Space(WS + 8, 64)), "FSDP_E_ALIGN"),
    (forward, dict(workspace=Space(0, 64)), "FSDP_E_ARG"),
    (forward, dict(workspace=Space(WS, -1)), "FSDP_E_ARG"),
    (forward, dict(dropout={**P, "p": 1.5}), "FSDP_E_ARG"),
    (forward, dict(dropout={**P, "p": -0.1}), "FSDP_E_ARG"),
    (forward, dict(dropout={**P, "p": float("nan")}), "FSDP_E_ARG"),
    (forward, dict(dropout={**P, "offset_dev": R + 4}), "FSDP_E_ALIGN"),
    (forward, dict(y=X), "FSDP_E_ALIAS"),
    (forward, dict(y=X + 4 * 16 * 2 - 2), "FSDP_E_ALIAS"),
    (forward, dict(y=W + 16), "FSDP_E_ALIAS"),
    (forward, dict(z=Y), "FSDP_E_ALIAS"),
    (forward, dict(z=X), "FSDP_E_ALIAS"),
    (forward, dict(bias=Y + 6), "FSDP_E_ALIAS"),
    (forward, dict(residual=Y + 2), "FSDP_E_ALIAS"),
    (forward, dict(residual=Y, ldr=9), "FSDP_E_ALIAS"),
    (forward, dict(residual=Z, z=Z), "FSDP_E_ALIAS"),
    (forward, dict(workspace=Space(Y, 1 << 20)), "FSDP_E_ALIAS"),
    (forward, dict(workspace=Space(X - 1024, 1 << 20)), "FSDP_E_ALIAS"),
    (forward, dict(w_dtype="e4m3", w_scale=Y + 4), "FSDP_E_ALIAS"),
    (forward, dict(dropout={**P, "offset_dev": Y + 8}), "FSDP_E_ALIAS"),
    # columns of one row stride: y takes [8, 16) and x [0, 16) of rows of 32
    (forward, dict(ldx=32, y=X + 16, ldy=32), "FSDP_E_ALIAS"),
    (forward, dict(ldx=32, y=X + 64 - 14, ldy=32), "FSDP_E_ALIAS"),
    (backward, dict(dy=None), "FSDP_E_ARG"),
    (backward, dict(z=None), "FSDP_E_ARG"),
    (backward, dict(n=-1), "FSDP_E_ARG"),
    (backward, dict(act=9), "FSDP_E_ARG"),
    (backward, dict(db_dtype=2), "FSDP_E_DTYPE"),
    (backward, dict(accumulate=2), "FSDP_E_ARG"),
    (backward, dict(db=DB + 2), "FSDP_E_ALIGN"),
    (backward, dict(lddz=7), "FSDP_E_ARG"),
    (backward, dict(dz=Y + 2), "FSDP_E_ALIAS"),
    (backward, dict(dz=Y, lddz=9), "FSDP_E_ALIAS"),
    (backward, dict(db=Y), "FSDP_E_ALIAS"),
    (backward, dict(db=DZ + 16), "FSDP_E_ALIAS"),
    (backward, dict(workspace=Space(DZ, 64)), "FSDP_E_ALIAS"),
    (backward, dict(dropout={**P, "p": 2}), "FSDP_E_ARG"),
    (backward, dict(dropout={**P, "offset_dev": DZ}), "FSDP_E_ALIAS"),
    (grad_input, dict(dx=None), "FSDP_E_ARG"),
    (grad_input, dict(dz=None), "FSDP_E_ARG"),
    (grad_input, dict(w=None), "FSDP_E_ARG"),
    (grad_input, dict(lddx=15), "FSDP_E_ARG"),
    (grad_input, dict(w_dtype="e4m3"), "FSDP_E_ARG"),
    (grad_input, dict(w_dtype=0), "FSDP_E_DTYPE"),
    (grad_input, dict(dx=DZ), "FSDP_E_ALIAS"),
    (grad_input, dict(dx=W), "FSDP_E_ALIAS"),
    (grad_input, dict(workspace=Space(DZ, 1 << 20)), "FSDP_E_ALIAS"),
    (grad_input, dict(k=(1 << 30) + 1), "FSDP_E_CAPACITY"),
    (grad_weight, dict(dw=None), "FSDP_E_ARG"),
    (grad_weight, dict(x=None), "FSDP_E_ARG"),
    (grad_weight, dict(dw_dtype=2), "FSDP_E_DTYPE"),
    (grad_weight, dict(accumulate=-1), "FSDP_E_ARG"),
    (grad_weight, dict(dw=W + 2, dw_dtype="f32"), "FSDP_E_ALIGN"),
    (grad_weight, dict(dw=X), "FSDP_E_ALIAS"),
    (grad_weight, dict(lddz=7), "FSDP_E_ARG"),
    (dropout, dict(x=None), "FSDP_E_ARG"),
    (dropout, dict(y=None), "FSDP_E_ARG"),
    (dropout, dict(dropout=None), "FSDP_E_ARG"),
    (dropout, dict(dtype=2), "FSDP_E_DTYPE"),
    (dropout, dict(dtype="f32", x=X + 2), "FSDP_E_ALIGN"),
    (dropout, dict(y=X + 2), "FSDP_E_ALIAS"),
    (dropout, dict(y=X, ldy=9), "FSDP_E_ALIAS"),
    (dropout, dict(residual=Y + 4), "FSDP_E_ALIAS"),
    (dropout, dict(ldx=7), "FSDP_E_ARG"),
    (dropout, dict(rows=-1), "FSDP_E_ARG"),
    (dropout, dict(dropout={**P, "offset_dev": Y}), "FSDP_E_ALIAS"),
]


@pytest.mark.parametrize("call,kw,code", BAD)
def test_refusals(call, kw, code):
    with pytest.raises(B.FsdpError) as e:
        call(**kw)
    assert e.value.name == code, str(e.value)


def _tensors():
    import torch
    b, f = torch.bfloat16, torch.float32
    return torch, b, f, lambda r, c, dt=b: torch.zeros(r, c, dtype=dt)


def _wrong_tensors():
    """(call, arguments, code, words of the message) of tensors that do not hold
    what the call would read or write there."""
    torch, b, f, t = _tensors()
    from_stride = t(8, 32)
    return [
        (forward, dict(x=t(4, 16, f)), "FSDP_E_DTYPE", "x is torch.float32"),
        (forward, dict(x=t(4, 16, torch.float16)), "FSDP_E_DTYPE", "x is torch.float16"),
        (forward, dict(w=t(8, 16, torch.uint8)), "FSDP_E_DTYPE", "w is"),
        (forward, dict(w=t(8, 16), w_dtype="e4m3", w_scale=R), "FSDP_E_DTYPE", "w is"),
        (forward, dict(w_dtype=2, w_scale=t(1, 1)), "FSDP_E_DTYPE", "w_scale"),
        (forward, dict(y=t(4, 8), y_dtype="f32"), "FSDP_E_DTYPE", "y is"),
        (forward, dict(residual=t(4, 8, f)), "FSDP_E_DTYPE", "residual is"),
        (forward, dict(z=t(4, 8, f)), "FSDP_E_DTYPE", "z is"),
        (forward, dict(bias=t(1, 8, f)), "FSDP_E_DTYPE", "bias is"),
        (backward, dict(db=t(1, 8)), "FSDP_E_DTYPE", "db is"),  # db_dtype is f32 unless given
        (grad_weight, dict(dw=t(8, 16, f)), "FSDP_E_DTYPE", "dw is"),
        (dropout, dict(x=t(4, 8), dtype="f32"), "FSDP_E_DTYPE", "x is"),
        (dropout, dict(dropout={**P, "offset_dev": torch.zeros(1, dtype=torch.int32)}), "FSDP_E_DTYPE", "offset_dev"),
        (forward, dict(x=t(16, 4).t()), "FSDP_E_ARG", "not contiguous"),
        (forward, dict(w=from_stride[:, :16]), "FSDP_E_ARG", "not contiguous"),
        (forward, dict(bias=t(1, 1).expand(1, 8)), "FSDP_E_ARG", "not contiguous"),
        (forward, dict(workspace=torch.zeros(64, 4, dtype=torch.uint8)[:, :2]), "FSDP_E_ARG", "not contiguous"),
        (grad_input, dict(dz=t(4, 16)[:, 8:]), "FSDP_E_ARG", "not contiguous"),
        (dropout, dict(y=t(8, 4).t()), "FSDP_E_ARG", "not contiguous"),
        (forward, dict(x=t(16, 4).t(), ldx=4), "FSDP_E_ARG", "next to each other"),
        (forward, dict(w=from_stride[:, :16], ldw=36), "FSDP_E_ARG", "room"),
        (forward, dict(w=from_stride[1:, :16], ldw=32), "FSDP_E_ARG", "room"),
        (forward, dict(y=t(4, 8)[:, 4:], ldy=8), "FSDP_E_ARG", "room"),
        (forward, dict(x=t(4, 15)), "FSDP_E_ARG", "room"),
        (forward, dict(y=t(3, 8)), "FSDP_E_ARG", "room"),
        (backward, dict(db=t(1, 7, f)), "FSDP_E_ARG", "room"),
        (grad_weight, dict(dw=t(8, 15)), "FSDP_E_ARG", "room"),
        (dropout, dict(residual=t(4, 7)), "FSDP_E_ARG", "room"),
        (forward, dict(x=t(4, 16)), "FSDP_E_ARG", "on cpu"),
        (forward, dict(w=from_stride[:, :16], ldw=32), "FSDP_E_ARG", "on cpu"),
        (forward, dict(workspace=torch.zeros(64, dtype=torch.uint8)), "FSDP_E_ARG", "on cpu"),
        (backward, dict(z=t(4, 8)), "FSDP_E_ARG", "on cpu"),
        (grad_input, dict(w=t(8, 16).view(torch.int16)), "FSDP_E_ARG", "on cpu"),  # the same bits
        (grad_input, dict(w=torch.zeros(8, 16).to(torch.float8_e4m3fn), w_dtype="e4m3", w_scale=R), "FSDP_E_ARG", "on cpu"),
        (dropout, dict(x=torch.nn.Parameter(t(4, 8))), "FSDP_E_ARG", "on cpu"),
        (dropout, dict(dropout={**P, "offset_dev": torch.zeros(1, dtype=torch.int64)}), "FSDP_E_ARG", "on cpu"),
    ]


@pytest.mark.parametrize("i", range(36))
def test_tensors_that_do_not_hold_the_operand(i):
    """A tensor of another type, layout, size or device than the call takes is
    refused, not read as if it were."""
    cases = _wrong_tensors()
    assert len(cases) == 36
    call, kw, code, words = cases[i]
    with pytest.raises(B.FsdpError) as e:
        call(**kw)
    assert e.value.name == code and words in str(e.value), str(e.value)


def test_more_tiles_than_a_launch():
    """Refused before any device work, on every way's path."""
    far = dict(x=1 << 40, w=1 << 42, y=1 << 50)
    big = 1 << 30
    for kw in (dict(m=big, n=big, k=8), dict(m=big, n=big, k=7), dict(m=16, n=big, k=8, w=1 << 44),
               dict(m=big, n=big, k=16, w_dtype="e4m3", w_scale=64)):
        with pytest.raises(B.FsdpError) as e:
            forward(**{**far, **kw})
        assert e.value.name == "FSDP_E_CAPACITY", (kw, str(e.value))


@pytest.mark.parametrize("kw", [dict(w=(1 << 42) + 2), dict(w=(1 << 42) + 1, w_dtype="e4m3", w_scale=64)])
def test_more_tiles_than_a_launch_with_an_operand_to_lay_out(kw):
    """A tall product whose weight is off 16-byte boundaries and fits in the
    workspace: refused before the weight is laid out there."""
    kw = dict(x=1 << 40, m=1 << 30, n=8, k=8, workspace=Space(1 << 52, 1 << 20), **kw)
    with pytest.raises(B.FsdpError) as e:
        forward(y=1 << 50, **kw)
    assert e.value.name == "FSDP_E_CAPACITY", str(e.value)
    kw["dz"] = kw.pop("x")
    with pytest.raises(B.FsdpError) as e:
        grad_input(dx=1 << 50, **kw)
    assert e.value.name == "FSDP_E_CAPACITY", str(e.value)


def test_reserved_and_null_record():
    L = B.lib()
    assert L.fsdp_linear_forward(None, None) == -1
    a = B.Linear(4, 8, 16, X, 16, W, 16, None, None, None, 8, Y, 8, None, 8, None, None, 0, 1, 1, 0, 1)
    assert L.fsdp_linear_forward(ctypes.byref(a), None) == -1
    assert b"reserved" in L.fsdp_last_error()


def test_empty_outputs_are_no_ops():
    """Nothing is queued (there is no device here to queue on), null or not."""
    forward(m=0, x=None, y=None)
    forward(n=0, w=None, y=None)
    grad_input(m=0, dx=None, dz=None)
    grad_input(k=0, dx=None, w=None)
    grad_weight(n=0, dw=None, dz=None)
    grad_weight(k=0, dw=None, x=None)
    backward(n=0, dz=None, dy=None, z=None, db=None)
    backward(m=0, dz=None, dy=None, z=None, db=None)
    backward(m=0, dz=None, dy=None, z=None, accumulate=True)
    backward(dz=None, db=None)
    dropout(rows=0, x=None, y=None)
    dropout(cols=0, x=None, y=None)


def test_exports_and_constants():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "fsdp_linear.h")).read()
    assert re.search(r"FSDP_LINEAR_WORKSPACE_BYTES \(\(int64_t\)64 << 20\)", text)
    assert B.LINEAR_WORKSPACE_BYTES == 64 << 20
    for name, value in B.ACTIVATIONS.items():
        assert re.search(r"FSDP_ACT_%s = %d\b" % (name.upper(), value), text), name
    assert B.WEIGHT_DTYPES["e4m3"] == int(re.search(r"FSDP_DT_E4M3 = (\d+)", text).group(1))


def test_from_plain_c(tmp_path):
    import json
    import os
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("needs a C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = tmp_path / "linear_from_c"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(root, "include"),
                    os.path.join(root, "tests", "c", "linear_from_c.c"), "-o", str(exe), B.lib_path(),
                    "-Wl,-rpath," + os.path.dirname(B.lib_path())], check=True, timeout=120)
    got = json.loads(subprocess.run([str(exe)], capture_output=True, text=True, timeout=60, check=True).stdout)
    assert got["linear"] == ctypes.sizeof(B.Linear) and got["mask"] == ctypes.sizeof(B.DropoutMask)
    assert got["act_at"] == B.Linear.act.offset
    assert got["empty"] == 0 and got["bad"] == -1
    assert got["message"] == "fsdp_linear_forward: unknown activation"
