"""Host checks of the dense entries (no GPU): bad arguments come back as status
codes before any CUDA call."""
import ctypes

import numpy as np

from .test_capi_cpu import _lib

FAKE = 1 << 20  # never dereferenced: every case fails, or ends, on the host


def _p(x):
    return None if x is None else ctypes.c_void_p(x)


def _i32(xs):
    return None if xs is None else np.asarray(xs, dtype=np.int32).ctypes.data_as(ctypes.POINTER(ctypes.c_int32))


def _dense(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, layout=None, cq=[0, 10], ck=[0, 10], n=1, hq=4, hkv=2, d=128, qr=10,
             kr=10, causal=1, scale=0.0, out=FAKE, lse=None)
    a.update(kw)
    keep = [np.asarray(x, dtype=np.int32) if x is not None else None for x in (a["cq"], a["ck"])]
    ptr = [None if x is None else x.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)) for x in keep]
    return _lib().dense_attn_varlen(
        _p(a["q"]), _p(a["k"]), _p(a["v"]), a["layout"], ptr[0], ptr[1], a["n"], a["hq"], a["hkv"], a["d"],
        a["qr"], a["kr"], a["causal"], a["scale"], _p(a["out"]), _p(a["lse"]), None)


def _layout(**kw):
    from block_sparse_attention_15_b200 import binding as B
    base = dict(q=(0, 1280, 128), k=(0, 1280, 128), v=(0, 1280, 128), out=(0, 1280, 128))
    base.update(kw)
    lay = B.VsaDenseLayout(*[B.VsaStrides(*base[n]) for n in ("q", "k", "v", "out")])
    return ctypes.byref(lay)


def test_dense_argument_checks():
    assert _dense(q=None) == 1 and _dense(k=None) == 1 and _dense(out=None) == 1
    assert _dense(q=FAKE + 2) == 1 and _dense(out=FAKE + 8) == 1        # misaligned
    assert _dense(cq=None) == 1 and _dense(hq=0) == 1 and _dense(scale=float("nan")) == 1
    assert _dense(n=0) == 2                                              # empty batch
    assert _dense(hq=5) == 2                                             # heads do not divide
    assert _dense(cq=[1, 10]) == 2 and _dense(ck=[0, 11]) == 2          # from 0, within the rows
    assert _dense(cq=[0, 8, 5], ck=[0, 1, 2], n=2) == 2                 # falling
    assert _dense(d=96) == 3 and _dense(d=256) == 3
    assert _dense(qr=1 << 31) == 3                                       # tile coordinates are 32-bit
    assert _dense(layout=_layout(q=(0, 1280, 4))) == 3                   # stride not 16 bytes
    assert _dense(layout=_layout(k=(0, 0, 128))) == 3                    # broadcast heads
    assert _dense(layout=_layout(out=(0, -1280, 128))) == 3


def test_dense_without_rows_is_a_no_op():
    assert _dense(cq=[0, 0], q=None, k=None, v=None, out=None) == 0
