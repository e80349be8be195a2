"""The 4-bit matrices' calls refuse what they cannot do (CPU only): every bad
argument comes back with its code before any device work.  The cases carry
device addresses that are never touched."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest

from oracle import mx4 as Q
from rank_step_amd import binding as B
from tests.test_linear_host import P, Space

X, Y, Z, R, BIAS, C, S, CT, ST, A, AS, BB, BS, WS = (0x10000000 * i for i in range(1, 15))
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def quantize(**kw):
    a = dict(x=X, rows=4, cols=70, codes=C, scales=S, codes_t=CT, scales_t=ST, stream=0)
    a.update(kw)
    B.fsdp_mx4_quantize(**a)


def dequantize(**kw):
    a = dict(y=Y, codes=C, scales=S, rows=4, cols=70, stream=0)
    a.update(kw)
    B.fsdp_mx4_dequantize(**a)


def product(**kw):
    a = dict(y=Y, a=A, a_scales=AS, b=BB, b_scales=BS, m=4, n=8, k=70, stream=0)
    a.update(kw)
    B.fsdp_mx4_product(**a)


BAD = [
    (quantize, dict(x=None), "FSDP_E_ARG"),
    (quantize, dict(codes=None), "FSDP_E_ARG"),
    (quantize, dict(scales=None), "FSDP_E_ARG"),
    (quantize, dict(codes_t=None), "FSDP_E_ARG"),
    (quantize, dict(scales_t=None), "FSDP_E_ARG"),
    (quantize, dict(codes=None, scales=None, codes_t=None, scales_t=None), "FSDP_E_ARG"),
    (quantize, dict(rows=-1), "FSDP_E_ARG"),
    (quantize, dict(cols=-1), "FSDP_E_ARG"),
    (quantize, dict(rows=(1 << 30) + 1), "FSDP_E_CAPACITY"),
    (quantize, dict(cols=(1 << 30) + 1), "FSDP_E_CAPACITY"),
    (quantize, dict(x_dtype=2), "FSDP_E_DTYPE"),
    (quantize, dict(ldx=69), "FSDP_E_ARG"),
    (quantize, dict(ldc=32), "FSDP_E_ARG"),
    (quantize, dict(ldc=56), "FSDP_E_ALIGN"),
    (quantize, dict(lds=0), "FSDP_E_ARG"),
    (quantize, dict(lds=24), "FSDP_E_ALIGN"),
    (quantize, dict(ldct=0), "FSDP_E_ARG"),
    (quantize, dict(ldst=-16), "FSDP_E_ARG"),
    (quantize, dict(codes=C + 8), "FSDP_E_ALIGN"),
    (quantize, dict(scales=S + 1), "FSDP_E_ALIGN"),
    (quantize, dict(codes_t=CT + 4), "FSDP_E_ALIGN"),
    (quantize, dict(scales_t=ST + 2), "FSDP_E_ALIGN"),
    (quantize, dict(x=X + 1), "FSDP_E_ALIGN"),
    (quantize, dict(x=X + 2, x_dtype="f32"), "FSDP_E_ALIGN"),
    (quantize, dict(codes=X), "FSDP_E_ALIAS"),
    (quantize, dict(codes=S), "FSDP_E_ALIAS"),
    (quantize, dict(codes_t=C + 16), "FSDP_E_ALIAS"),
    (quantize, dict(scales_t=X + 4 * 70 * 2 - 16), "FSDP_E_ALIAS"),
    (dequantize, dict(y=None), "FSDP_E_ARG"),
    (dequantize, dict(codes=None), "FSDP_E_ARG"),
    (dequantize, dict(scales=None), "FSDP_E_ARG"),
    (dequantize, dict(rows=-1), "FSDP_E_ARG"),
    (dequantize, dict(cols=(1 << 30) + 1), "FSDP_E_CAPACITY"),
    (dequantize, dict(y_dtype=2), "FSDP_E_DTYPE"),
    (dequantize, dict(ldy=69), "FSDP_E_ARG"),
    (dequantize, dict(ldc=40), "FSDP_E_ARG"),
    (dequantize, dict(lds=17), "FSDP_E_ALIGN"),
    (dequantize, dict(codes=C + 4), "FSDP_E_ALIGN"),
    (dequantize, dict(y=Y + 1), "FSDP_E_ALIGN"),
    (dequantize, dict(y=C), "FSDP_E_ALIAS"),
    (dequantize, dict(y=S + 2), "FSDP_E_ALIAS"),
    (product, dict(a=None), "FSDP_E_ARG"),
    (product, dict(a_scales=None), "FSDP_E_ARG"),
    (product, dict(b=None), "FSDP_E_ARG"),
    (product, dict(b_scales=None), "FSDP_E_ARG"),
    (product, dict(y=None), "FSDP_E_ARG"),
    (product, dict(m=-1), "FSDP_E_ARG"),
    (product, dict(k=-1), "FSDP_E_ARG"),
    (product, dict(n=(1 << 30) + 1), "FSDP_E_CAPACITY"),
    (product, dict(y_dtype=2), "FSDP_E_DTYPE"),
    (product, dict(act=4), "FSDP_E_ARG"),
    (product, dict(lda=32), "FSDP_E_ARG"),
    (product, dict(ldb=32), "FSDP_E_ARG"),
    (product, dict(ldas=0), "FSDP_E_ARG"),
    (product, dict(ldbs=8), "FSDP_E_ARG"),
    (product, dict(lda=56), "FSDP_E_ALIGN"),
    (product, dict(ldbs=40), "FSDP_E_ALIGN"),
    (product, dict(a=A + 8), "FSDP_E_ALIGN"),
    (product, dict(b_scales=BS + 4), "FSDP_E_ALIGN"),
    (product, dict(lda=(1 << 22) + 16), "FSDP_E_CAPACITY"),
    (product, dict(ldas=(1 << 22) + 16), "FSDP_E_CAPACITY"),
    (product, dict(ldb=(1 << 22) + 16), "FSDP_E_CAPACITY"),
    (product, dict(ldbs=1 << 23), "FSDP_E_CAPACITY"),
    (product, dict(k=(1 << 23) + 1, a_scales=1 << 40, b=1 << 41, b_scales=1 << 42, y=1 << 43), "FSDP_E_CAPACITY"),
    (product, dict(ldy=7), "FSDP_E_ARG"),
    (product, dict(z=Z, ldz=7), "FSDP_E_ARG"),
    (product, dict(residual=R, ldr=7), "FSDP_E_ARG"),
    (product, dict(bias=BIAS + 1), "FSDP_E_ALIGN"),
    (product, dict(y=Y + 2, y_dtype="f32"), "FSDP_E_ALIGN"),
    (product, dict(dropout={**P, "p": 1.5}), "FSDP_E_ARG"),
    (product, dict(dropout={**P, "offset_dev": R + 4}), "FSDP_E_ALIGN"),
    (product, dict(workspace=Space(WS + 8, 64)), "FSDP_E_ALIGN"),
    (product, dict(workspace=Space(0, 64)), "FSDP_E_ARG"),
    (product, dict(y=A), "FSDP_E_ALIAS"),
    (product, dict(y=AS), "FSDP_E_ALIAS"),
    (product, dict(y=BB + 16), "FSDP_E_ALIAS"),
    (product, dict(y=BS), "FSDP_E_ALIAS"),
    (product, dict(z=Y), "FSDP_E_ALIAS"),
    (product, dict(z=BS), "FSDP_E_ALIAS"),
    (product, dict(residual=Y + 2), "FSDP_E_ALIAS"),
    (product, dict(residual=Y, ldr=9), "FSDP_E_ALIAS"),
    (product, dict(bias=Y), "FSDP_E_ALIAS"),
    (product, dict(workspace=Space(A, 1 << 20)), "FSDP_E_ALIAS"),
    (product, dict(workspace=Space(Y, 1 << 20)), "FSDP_E_ALIAS"),
    (product, dict(dropout={**P, "offset_dev": Y + 8}), "FSDP_E_ALIAS"),
]


@pytest.mark.parametrize("call,kw,code", BAD)
def test_refusals(call, kw, code):
    with pytest.raises(B.FsdpError) as e:
        call(**kw)
    assert e.value.name == code, str(e.value)


def _wrong_tensors():
    import torch
    b, f, u = torch.bfloat16, torch.float32, torch.uint8

    def t(r, c, dt=b):
        return torch.zeros(r, c, dtype=dt)

    return [
        (quantize, dict(x=t(4, 70, f)), "FSDP_E_DTYPE", "x is torch.float32"),
        (quantize, dict(codes=t(4, 48)), "FSDP_E_DTYPE", "codes is"),
        (quantize, dict(scales=t(4, 16, torch.int32)), "FSDP_E_DTYPE", "scales is"),
        (quantize, dict(codes=t(4, 47, u)), "FSDP_E_ARG", "room"),
        (quantize, dict(scales=t(3, 16, u)), "FSDP_E_ARG", "room"),
        (quantize, dict(codes_t=t(69, 16, u)), "FSDP_E_ARG", "room"),
        (quantize, dict(x=t(70, 4).t()), "FSDP_E_ARG", "not contiguous"),
        (quantize, dict(scales_t=t(70, 16, u)), "FSDP_E_ARG", "on cpu"),
        (dequantize, dict(y=t(4, 70, f)), "FSDP_E_DTYPE", "y is"),
        (dequantize, dict(y=t(4, 69)), "FSDP_E_ARG", "room"),
        (dequantize, dict(codes=t(4, 96, u)[:, :48]), "FSDP_E_ARG", "not contiguous"),
        (product, dict(a=t(4, 48)), "FSDP_E_DTYPE", "a is"),
        (product, dict(b_scales=t(8, 16, f)), "FSDP_E_DTYPE", "b_scales is"),
        (product, dict(y=t(4, 8), y_dtype="f32"), "FSDP_E_DTYPE", "y is"),
        (product, dict(residual=t(4, 8, f)), "FSDP_E_DTYPE", "residual is"),
        (product, dict(b=t(8, 47, u)), "FSDP_E_ARG", "room"),
        (product, dict(a_scales=t(4, 16, u)), "FSDP_E_ARG", "on cpu"),
        (product, dict(bias=t(1, 7)), "FSDP_E_ARG", "room"),
    ]


@pytest.mark.parametrize("i", range(18))
def test_tensors_that_do_not_hold_the_operand(i):
    cases = _wrong_tensors()
    assert len(cases) == 18
    call, kw, code, words = cases[i]
    with pytest.raises(B.FsdpError) as e:
        call(**kw)
    assert e.value.name == code and words in str(e.value), str(e.value)


def test_more_tiles_than_a_launch():
    far = dict(a=1 << 40, a_scales=1 << 41, b=1 << 42, b_scales=1 << 43, y=1 << 50)
    with pytest.raises(B.FsdpError) as e:
        product(m=1 << 30, n=1 << 30, k=32, **far)
    assert e.value.name == "FSDP_E_CAPACITY", str(e.value)


def test_empty_outputs_are_no_ops():
    """Nothing is queued (there is no device here to queue on), null or not."""
    quantize(rows=0, x=None, codes=None, scales=None, codes_t=None, scales_t=None)
    quantize(cols=0, x=None)
    dequantize(rows=0, y=None, codes=None, scales=None)
    dequantize(cols=0)
    product(m=0, y=None, a=None, a_scales=None)
    product(n=0, y=None, b=None, b_scales=None)


def test_null_record():
    assert B.lib().fsdp_mx4_product(None, None) == -1


def test_constants():
    text = open(os.path.join(ROOT, "include", "fsdp_mx4.h")).read()
    assert re.search(r"FSDP_MX4_WORKSPACE_BYTES \(\(int64_t\)64 << 20\)", text)
    assert B.MX4_WORKSPACE_BYTES == 64 << 20
    for cols in (0, 1, 31, 32, 33, 511, 512, 513, 4096, 11008):
        assert B.mx4_code_bytes(cols) == Q.code_bytes(cols) and B.mx4_scale_bytes(cols) == Q.scale_bytes(cols)


def test_from_plain_c(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("needs a C compiler")
    src = tmp_path / "mx4_from_c.c"
    src.write_text('''#include <stdio.h>
#include <stddef.h>
#include "fsdp_norm.h"
#include "fsdp_mx4.h"
int main(void) {
    fsdp_mx4_operands a = {0};
    a.act = 9;
    a.y_dtype = FSDP_DT_F32;
    printf("%d %d %d %d %d ", (int)sizeof a, (int)offsetof(fsdp_mx4_operands, act), (int)FSDP_MX4_CODE_BYTES(70),
           (int)FSDP_MX4_SCALE_BYTES(513), fsdp_mx4_product(&a, 0));
    printf("%s\\n", fsdp_last_error());
    return fsdp_norm_forward(0, 0, 0, 0, 0, 0, FSDP_DT_F32, FSDP_NORM_RMS, 0, 0, FSDP_DT_F32, 1e-5, 0, 8, 0);
}
''')
    exe = tmp_path / "mx4_from_c"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe),
                    B.lib_path(), "-Wl,-rpath," + os.path.dirname(B.lib_path())], check=True, timeout=120)
    got = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60, check=True).stdout.split(maxsplit=5)
    assert [int(v) for v in got[:5]] == [ctypes.sizeof(B.Mx4Operands), B.Mx4Operands.act.offset, 48, 32, -1]
    assert got[5].strip() == "fsdp_mx4_product: unknown activation"
