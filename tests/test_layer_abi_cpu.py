"""What the root-mean-square norm, dropout and cross attention refuse, through
the C ABI and on tensors: every refusal comes before any GPU call, so made-up
pointers do (CPU)."""
import ctypes
import os
import subprocess

import pytest

import libutil
import ring_allreduce_reduce_amd as ra
from ring_allreduce_reduce_amd import attention as A
from ring_allreduce_reduce_amd import block as B

F16, BF16, F32, F64 = 2, 3, 4, 5
P = [0x100000000 * (i + 1) for i in range(12)]      # far apart, aligned
BAD_ARG, BAD_USE = ra.INVALID_ARGUMENT, ra.INVALID_USAGE
INF = float("inf")


def call(name, args):
    libutil.lib()
    return B._fn(name)(ctypes.byref(args) if args is not None else None, None)


def rms(**kw):
    d = dict(dtype=BF16, param_dtype=BF16, out=0, rows=4, cols=256, x=P[0], ldx=256, residual=P[1], ldr=256, weight=P[2], eps=1e-6,
             sum=P[3], lds=256, y=P[4], ldy=256, scale=None, rstd=P[5])
    return B.ringar_rms_norm_t(**{**d, **kw})


def rms_back(**kw):
    d = dict(dtype=BF16, param_dtype=BF16, rows=4, cols=64, dy=P[0], lddy=64, x=P[1], ldx=64, rstd=P[2], weight=P[3], dsum=P[4],
             ldds=64, dx=P[5], lddx=64, dweight=P[6])
    return B.ringar_rms_norm_backward_t(**{**d, **kw})


def drop(**kw):
    d = dict(dtype=BF16, rows=4, cols=64, x=P[0], ldx=64, residual=P[1], ldr=64, p=0.1, seed=1, offset=2, more_offset=P[2], first_row=0,
             first_col=0, y=P[3], ldy=64)
    return B.ringar_dropout_t(**{**d, **kw})


def strides(*s):
    return A._three(*s)


SIZES = dict(dtype=BF16, batch=2, queries=5, keys=7, heads=4, kv_heads=2, head_dim=64, scale=0.125)
Q_STRIDES, K_STRIDES = (5 * 256, 256, 64), (7 * 128, 128, 64)


def att(**kw):
    d = dict(SIZES, q=P[0], q_strides=strides(*Q_STRIDES), k=P[1], k_strides=strides(*K_STRIDES), v=P[2], v_strides=strides(*K_STRIDES),
             key_lengths=P[3], y=P[4], y_strides=strides(*Q_STRIDES), lse=P[5])
    return A.ringar_cross_attention_t(**{**d, **kw})


def att_back(**kw):
    d = dict(SIZES, dy=P[0], dy_strides=strides(*Q_STRIDES), q=P[1], q_strides=strides(*Q_STRIDES), k=P[2], k_strides=strides(*K_STRIDES),
             v=P[3], v_strides=strides(*K_STRIDES), y=P[4], y_strides=strides(*Q_STRIDES), lse=P[5], key_lengths=P[6], dq=P[7], dk=P[8], dv=P[9])
    return A.ringar_cross_attention_backward_t(**{**d, **kw})


RMS = [(dict(dtype=F64), BAD_ARG), (dict(param_dtype=F16), BAD_ARG), (dict(rows=-1), BAD_ARG), (dict(cols=0), BAD_ARG),
       (dict(cols=1 << 31), BAD_ARG), (dict(out=3), BAD_ARG), (dict(out=-1), BAD_ARG), (dict(eps=-1.0), BAD_ARG),
       (dict(eps=float("nan")), BAD_ARG), (dict(x=None), BAD_ARG), (dict(y=None), BAD_ARG), (dict(residual=None), BAD_ARG),
       (dict(sum=None), BAD_ARG), (dict(x=P[0] + 1), BAD_ARG), (dict(ldx=100), BAD_ARG), (dict(lds=0), BAD_ARG),
       (dict(out=1), BAD_ARG), (dict(out=2, scale=P[6] + 2), BAD_ARG), (dict(out=2, scale=P[4]), BAD_USE), (dict(out=1, scale=P[6], y=P[0]), BAD_USE),
       (dict(y=P[3]), BAD_USE), (dict(y=P[0] + 2), BAD_USE), (dict(sum=P[1] + 16), BAD_USE), (dict(sum=P[2]), BAD_USE),
       (dict(rstd=P[4]), BAD_USE), (dict(y=P[0], sum=P[0]), BAD_USE), (dict(y=P[0], ldy=512), BAD_USE)]
RMS_BACK = [(dict(dtype=F64), BAD_ARG), (dict(rstd=None), BAD_ARG), (dict(dy=None), BAD_ARG), (dict(x=None), BAD_ARG),
            (dict(cols=0), BAD_ARG), (dict(rows=1 << 31), BAD_ARG), (dict(lddx=3), BAD_ARG), (dict(ldds=3), BAD_ARG),
            (dict(dx=P[0]), BAD_USE), (dict(dx=P[1]), BAD_USE), (dict(dweight=P[3]), BAD_USE), (dict(dx=P[4], lddx=72), BAD_USE)]
DROP = [(dict(dtype=F64), BAD_ARG), (dict(p=-0.1), BAD_ARG), (dict(p=1.01), BAD_ARG), (dict(p=float("nan")), BAD_ARG),
        (dict(rows=-1), BAD_ARG), (dict(x=None), BAD_ARG), (dict(y=None), BAD_ARG), (dict(first_col=4), BAD_ARG),
        (dict(first_col=-8), BAD_ARG), (dict(first_row=-1), BAD_ARG), (dict(first_row=(1 << 32) - 3), BAD_ARG),
        (dict(first_col=1 << 31), BAD_ARG), (dict(more_offset=P[2] + 4), BAD_ARG), (dict(ldr=8), BAD_ARG),
        (dict(y=P[0] + 2), BAD_USE), (dict(y=P[1], ldy=72), BAD_USE), (dict(y=P[2]), BAD_USE)]
BOTH = [(dict(dtype=F64), BAD_ARG), (dict(batch=-1), BAD_ARG), (dict(heads=3), BAD_ARG), (dict(kv_heads=0), BAD_ARG),
        (dict(head_dim=0), BAD_ARG), (dict(head_dim=60), BAD_ARG), (dict(head_dim=136), BAD_ARG), (dict(scale=0.0), BAD_ARG),
        (dict(scale=-1.0), BAD_ARG), (dict(scale=INF), BAD_ARG), (dict(scale=float("nan")), BAD_ARG), (dict(q=None), BAD_ARG),
        (dict(k=None), BAD_ARG), (dict(v=None), BAD_ARG), (dict(y=None), BAD_ARG), (dict(q=P[0] + 8), BAD_ARG),
        (dict(k_strides=strides(7 * 128, 132, 64)), BAD_ARG), (dict(v_strides=strides(-8, 128, 64)), BAD_ARG),
        (dict(k_strides=strides(7 << 24, 1 << 24, 64)), BAD_ARG), (dict(key_lengths=P[3] + 2), BAD_ARG),
        (dict(q_strides=strides(1 << 60, 256, 64)), BAD_ARG), (dict(queries=1 << 30, heads=8), BAD_ARG)]
ATT = BOTH + [(dict(y_strides=strides(5 * 256, 256, 32)), BAD_ARG), (dict(y_strides=strides(0, 256, 64)), BAD_ARG),
              (dict(y=P[0]), BAD_USE), (dict(y=P[1] + 64), BAD_USE), (dict(lse=P[4] + 4), BAD_USE), (dict(lse=P[3]), BAD_USE),
              (dict(lse=P[5] + 2), BAD_ARG)]
ATT_BACK = BOTH + [(dict(lse=None), BAD_ARG), (dict(dy=None), BAD_ARG), (dict(dq=P[0]), BAD_USE), (dict(dk=P[9]), BAD_USE),
                   (dict(dv=P[5]), BAD_USE), (dict(dq=P[7] + 4), BAD_ARG)]


@pytest.mark.parametrize("name,make,table", [
    ("ringar_rms_norm", rms, RMS), ("ringar_rms_norm_backward", rms_back, RMS_BACK), ("ringar_dropout", drop, DROP),
    ("ringar_cross_attention", att, ATT), ("ringar_cross_attention_backward", att_back, ATT_BACK)])
def test_refusals(name, make, table):
    assert call(name, None) == BAD_ARG
    for change, code in table:
        assert call(name, make(**change)) == code, (name, change)
        assert ra.ringar_last_error(), change


def test_nothing_to_do_needs_no_gpu():
    assert call("ringar_rms_norm", rms(rows=0, x=None, y=None, residual=None, sum=None, rstd=None)) == ra.SUCCESS
    assert call("ringar_rms_norm_backward", rms_back(rows=0, dweight=None)) == ra.SUCCESS
    assert call("ringar_dropout", drop(rows=0, x=None, y=None)) == ra.SUCCESS
    assert call("ringar_cross_attention", att(batch=0, q=None, y=None)) == ra.SUCCESS
    assert call("ringar_cross_attention", att(queries=0, y=None)) == ra.SUCCESS
    assert call("ringar_cross_attention", att(heads=0, kv_heads=0)) == ra.SUCCESS
    assert call("ringar_cross_attention_backward", att_back(dq=None, dk=None, dv=None)) == ra.SUCCESS
    assert call("ringar_cross_attention_backward", att_back(batch=0)) == ra.SUCCESS


def test_tensor_calls_refuse_what_is_no_operand():
    import torch
    libutil.lib()
    t, q, stats = torch.zeros(4, 8), torch.zeros(1, 2, 3, 8), torch.zeros(4)
    z = torch.randn(4, 8, dtype=torch.complex64).conj().imag
    calls = [lambda: ra.rms_norm(t), lambda: ra.rms_norm_fp8(t), lambda: ra.rms_norm_backward(t, t, stats), lambda: ra.dropout(t, 0.1, 0),
             lambda: ra.dropout_backward(t, 0.1, 0), lambda: ra.cross_attention(q, q, q), lambda: ra.cross_attention_backward(q, q, q, q, q, stats),
             lambda: ra.rms_norm("x"), lambda: ra.rms_norm(z), lambda: ra.rms_norm(t, residual=z), lambda: ra.rms_norm(t, stats=1),
             lambda: ra.dropout(None, 0.1, 0), lambda: ra.dropout(t, 0.1, -1), lambda: ra.dropout(t, 0.1, 1 << 64), lambda: ra.dropout(t, 0.1, 1.5),
             lambda: ra.rms_norm_fp8(t, group=64), lambda: ra.rms_norm_fp8(t, group=True), lambda: ra.rms_norm_fp8(t, group="128"),
             lambda: ra.cross_attention(q, None, q), lambda: ra.cross_attention(q, q, q, stats=None)]
    for i, c in enumerate(calls):
        with pytest.raises(ra.RingarError) as e:
            c()
        assert e.value.code == BAD_ARG, i
    for c in (lambda: ra.dropout(t, "0.1", 0), lambda: ra.rms_norm(t, None, "eps")):
        with pytest.raises(TypeError):
            c()


def test_struct_layouts_match_the_header(tmp_path):
    """sizeof and every field's offset, as a C compiler sees the header."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    types = [B.ringar_rms_norm_t, B.ringar_rms_norm_backward_t, B.ringar_dropout_t, A.ringar_cross_attention_t, A.ringar_cross_attention_backward_t]
    lines, want = [], []
    for t in types:
        n = t.__name__
        lines.append(f'printf("%zu\\n", sizeof({n}));')
        lines += [f'printf("%zu\\n", offsetof({n}, {f[0]}));' for f in t._fields_]
        want += [ctypes.sizeof(t)] + [getattr(t, f[0]).offset for f in t._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "ringar.h"\nint main(void) {' + "\n".join(lines) + "return 0; }\n")
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), "-o", str(tmp_path / "layout"), str(src)], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout.split()]
    assert got == want
