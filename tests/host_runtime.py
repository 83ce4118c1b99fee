"""Runs a piece of Python against the library over fake_hip.c, in a process of
its own (the library binds to the first runtime it finds)."""
import os
import subprocess
import sys
import textwrap

HERE = os.path.dirname(os.path.abspath(__file__))

PROLOGUE = """
import ctypes, os, sys
sys.path[:0] = [{root!r}, {here!r}]
fake = ctypes.CDLL({lib!r}, mode=os.RTLD_GLOBAL | os.RTLD_NOW)
import ring_allreduce_reduce_amd as ra
from test_block_abi_cpu import P, call, lin, lin_back, norm, norm_back
from ring_allreduce_reduce_amd import block as B


class Launch(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char_p), ("grid", ctypes.c_uint64 * 3), ("block", ctypes.c_uint64 * 3), ("stream", ctypes.c_uint64)]


fake.fake_launch.restype = ctypes.POINTER(Launch)


def launches():
    # (kernel, blocks, threads of a block) of every launch since the last reset
    out = []
    for i in range(fake.fake_launches()):
        l = fake.fake_launch(i).contents
        out.append((l.name.decode(), list(l.grid), list(l.block)))
    return out


def on(name, args, stream):
    return B._fn(name)(ctypes.byref(args), stream)
"""


def build(folder):
    """fake_hip.c as a shared library in `folder`."""
    out = os.path.join(str(folder), "libfake_hip.so")
    subprocess.run(["gcc", "-O1", "-Wall", "-shared", "-fPIC", "-pthread", os.path.join(HERE, "fake_hip.c"), "-o", out], check=True)
    return out


def run(lib, code):
    """Runs `code` after the prologue; it fails by raising."""
    import libutil
    libutil.lib()
    text = PROLOGUE.format(root=os.path.dirname(HERE), here=HERE, lib=lib) + textwrap.dedent(code)
    r = subprocess.run([sys.executable, "-c", text], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    return r.stdout
