"""What the block operators refuse, through the C ABI: every refusal comes
before any GPU call, so made-up pointers do (CPU)."""
import ctypes

import pytest

import ring_allreduce_reduce_amd as ra
from ring_allreduce_reduce_amd import block as B

import libutil

BF16, F32, F64, I8 = 3, 4, 5, 0
P = [0x100000000 * (i + 1) for i in range(12)]      # far apart, aligned


def call(name, args):
    libutil.lib()
    return B._fn(name)(ctypes.byref(args) if args is not None else None, None)


def norm(**kw):
    d = dict(dtype=BF16, param_dtype=BF16, rows=4, cols=64, x=P[0], ldx=64, weight=P[1], bias=P[2], eps=1e-5, y=P[3],
             ldy=64, mean=P[4], rstd=P[5])
    return B.ringar_layer_norm_t(**{**d, **kw})


def norm_back(**kw):
    d = dict(dtype=BF16, param_dtype=BF16, rows=4, cols=64, dy=P[0], lddy=64, x=P[1], ldx=64, mean=P[2], rstd=P[3],
             weight=P[4], dx=P[5], lddx=64, dweight=P[6], dbias=P[7])
    return B.ringar_layer_norm_backward_t(**{**d, **kw})


def lin(**kw):
    d = dict(dtype=BF16, act=0, rows=4, in_features=64, out_features=32, x=P[0], ldx=64, weight=P[1], ldw=64, bias=P[2],
             residual=None, ldr=0, y=P[4], ldy=32, pre=P[5], ldp=64)
    return B.ringar_linear_t(**{**d, **kw})


def lin_back(**kw):
    d = dict(dtype=BF16, act=4, rows=4, in_features=64, out_features=32, dy=P[0], lddy=32, pre=P[1], ldp=64, x=P[2],
             ldx=64, weight=P[3], ldw=64, dx=P[4], lddx=64, dweight=P[5], lddw=64, dbias=P[6])
    return B.ringar_linear_backward_t(**{**d, **kw})


BAD_ARG, BAD_USE = ra.INVALID_ARGUMENT, ra.INVALID_USAGE

NORM = [(dict(dtype=F64), BAD_ARG), (dict(dtype=I8), BAD_ARG), (dict(param_dtype=2), BAD_ARG), (dict(rows=-1), BAD_ARG),
        (dict(cols=0), BAD_ARG), (dict(cols=1 << 31), BAD_ARG), (dict(x=None), BAD_ARG), (dict(y=None), BAD_ARG),
        (dict(x=P[0] + 1), BAD_ARG), (dict(ldx=63), BAD_ARG), (dict(ldy=0), BAD_ARG), (dict(ldx=-64), BAD_ARG),
        (dict(ldy=1 << 31), BAD_ARG), (dict(eps=-1.0), BAD_ARG), (dict(eps=float("nan")), BAD_ARG),
        (dict(mean=P[4] + 2), BAD_ARG), (dict(y=P[0] + 2), BAD_USE), (dict(y=P[0], ldy=72), BAD_USE),
        (dict(mean=P[1]), BAD_USE), (dict(rstd=P[4] + 4), BAD_USE), (dict(weight=P[3] + 128), BAD_USE)]
NORM_BACK = [(dict(dtype=F64), BAD_ARG), (dict(mean=None), BAD_ARG), (dict(rstd=None), BAD_ARG), (dict(dy=None), BAD_ARG),
             (dict(x=None), BAD_ARG), (dict(lddx=32), BAD_ARG), (dict(dx=P[0]), BAD_USE), (dict(dweight=P[7]), BAD_USE),
             (dict(dbias=P[4]), BAD_USE), (dict(cols=0), BAD_ARG), (dict(rows=1 << 31), BAD_ARG)]
LIN = [(dict(dtype=F64), BAD_ARG), (dict(act=6), BAD_ARG), (dict(act=-1), BAD_ARG), (dict(rows=-1), BAD_ARG),
       (dict(in_features=1 << 31, ldx=1 << 31), BAD_ARG), (dict(out_features=-5), BAD_ARG), (dict(x=None), BAD_ARG),
       (dict(weight=None), BAD_ARG), (dict(y=None), BAD_ARG), (dict(ldx=10), BAD_ARG), (dict(ldw=-64), BAD_ARG),
       (dict(ldy=0), BAD_ARG), (dict(ldp=8), BAD_ARG), (dict(bias=P[2] + 1), BAD_ARG), (dict(y=P[0]), BAD_USE),
       (dict(y=P[5]), BAD_USE), (dict(y=P[1] + 64), BAD_USE), (dict(pre=P[2]), BAD_USE)]
RESIDUAL = [(dict(residual=P[4], ldr=40), BAD_USE), (dict(residual=P[4] + 2, ldr=32), BAD_USE),
            (dict(residual=P[6], ldr=16), BAD_ARG), (dict(residual=P[5], ldr=32), BAD_USE)]
LIN_BACK = [(dict(dtype=F64), BAD_ARG), (dict(act=9), BAD_ARG), (dict(pre=None), BAD_ARG), (dict(dy=None), BAD_ARG),
            (dict(x=None), BAD_ARG), (dict(weight=None), BAD_ARG), (dict(lddw=63), BAD_ARG), (dict(dx=P[2]), BAD_USE),
            (dict(dweight=P[4]), BAD_USE), (dict(dbias=P[1]), BAD_USE), (dict(rows=-3), BAD_ARG)]


@pytest.mark.parametrize("name,make,table", [
    ("ringar_layer_norm", norm, NORM), ("ringar_layer_norm_backward", norm_back, NORM_BACK),
    ("ringar_linear", lin, LIN + RESIDUAL), ("ringar_gated_ffn", lin, LIN),
    ("ringar_linear_backward", lin_back, LIN_BACK), ("ringar_gated_ffn_backward", lin_back, LIN_BACK)])
def test_refusals(name, make, table):
    assert call(name, None) == BAD_ARG
    for change, code in table:
        assert call(name, make(**change)) == code, (name, change)
        assert ra.ringar_last_error(), change


def test_gated_refuses_a_residual_and_too_many_features():
    assert call("ringar_gated_ffn", lin(residual=P[6], ldr=32)) == BAD_ARG
    assert call("ringar_gated_ffn", lin(out_features=1 << 30, ldy=1 << 30, ldp=1 << 31)) == BAD_ARG


def test_nothing_to_do_needs_no_gpu():
    assert call("ringar_layer_norm", norm(rows=0, x=None, y=None)) == ra.SUCCESS
    assert call("ringar_linear", lin(rows=0, x=None, y=None)) == ra.SUCCESS
    assert call("ringar_gated_ffn", lin(out_features=0, weight=None, y=None)) == ra.SUCCESS


def test_tensor_calls_refuse_what_is_not_on_a_gpu():
    import torch
    libutil.lib()
    t = torch.zeros(4, 8)
    stats = torch.zeros(4)
    calls = [lambda: ra.layer_norm(t), lambda: ra.linear(t, t), lambda: ra.gated_ffn(t, t),
             lambda: ra.layer_norm_backward(t, t, stats, stats), lambda: ra.linear_backward(t, t, t, t),
             lambda: ra.gated_ffn_backward(t, t, t, t), lambda: ra.linear(None, t), lambda: ra.layer_norm("x"),
             lambda: ra.linear(t, t, act="swish"), lambda: ra.gated_ffn_backward(t, t, t, t, act=3)]
    for i, call in enumerate(calls):
        with pytest.raises(ra.RingarError) as e:
            call()
        assert e.value.code == BAD_ARG, i


def test_struct_layouts_match_the_header(tmp_path):
    """sizeof and every field's offset, as a C compiler sees the header."""
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = ["ringar_layer_norm_t", "ringar_layer_norm_backward_t", "ringar_linear_t", "ringar_linear_backward_t"]
    lines = []
    for n in names:
        lines.append(f'printf("%zu\\n", sizeof({n}));')
        lines += [f'printf("%zu\\n", offsetof({n}, {f[0]}));' for f in getattr(B, n)._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "ringar.h"\nint main(void) {' + "\n".join(lines) + "return 0; }\n")
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), "-o", str(tmp_path / "layout"), str(src)], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for n in names:
        t = getattr(B, n)
        want.append(ctypes.sizeof(t))
        want += [getattr(t, f[0]).offset for f in t._fields_]
    assert got == want
