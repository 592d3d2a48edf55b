"""Host checks of the dense entries (no GPU): bad arguments come back as status
codes before any CUDA call."""
import ctypes

import numpy as np

from .test_capi_cpu import _lib

FAKE = 1 << 20  # never dereferenced: every case fails, or ends, on the host


def _p(x):
    return None if x is None else ctypes.c_void_p(x)


def _i32(xs):
    return (ctypes.c_int32 * len(xs))(*xs)


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


def _prefix(**kw):
    a = dict(q=FAKE, kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, lens=FAKE, layout=None, b=2, hq=4, hkv=2, t=1, d=128,
             p=100, s=50, scale=0.0, out=FAKE, lse=None, ws=FAKE, bytes=1 << 30)
    a.update(kw)
    return _lib().shared_prefix_attn(
        _p(a["q"]), _p(a["kp"]), _p(a["vp"]), _p(a["ks"]), _p(a["vs"]), _p(a["lens"]), a["layout"], a["b"],
        a["hq"], a["hkv"], a["t"], a["d"], a["p"], a["s"], a["scale"], _p(a["out"]), _p(a["lse"]), _p(a["ws"]),
        a["bytes"], None)


def _prefix_layout(**kw):
    from block_sparse_attention_15_b200 import binding as B
    base = dict(q=(512, 128, 128), out=(512, 128, 128), k_prefix=(0, 12800, 128), v_prefix=(0, 12800, 128),
                k_suffix=(12800, 6400, 128), v_suffix=(12800, 6400, 128))
    base.update(kw)
    return ctypes.byref(B.VsaPrefixLayout(*[B.VsaStrides(*base[n]) for n, _ in B.VsaPrefixLayout._fields_]))


def test_prefix_argument_checks():
    for n in ("q", "kp", "vp", "ks", "vs", "lens", "out"):
        assert _prefix(**{n: None}) == 1
        assert _prefix(**{n: FAKE + 2}) == 1                             # misaligned
    assert _prefix(b=-1) == 1 and _prefix(t=-1) == 1 and _prefix(p=-1) == 1 and _prefix(s=-1) == 1
    assert _prefix(hkv=0) == 1 and _prefix(scale=float("nan")) == 1
    assert _prefix(hq=5) == 2
    assert _prefix(d=96) == 3 and _prefix(p=1 << 31) == 3 and _prefix(s=1 << 31) == 3
    assert _prefix(b=1 << 20, t=1 << 10) == 3                            # rows are counted in 32 bits
    assert _prefix(b=1 << 16, s=1 << 30) == 3                            # key tiles too
    assert _prefix(layout=_prefix_layout(q=(510, 128, 128))) == 3
    assert _prefix(layout=_prefix_layout(k_suffix=(0, 6400, 128))) == 3  # broadcast suffix
    assert _prefix(layout=_prefix_layout(v_prefix=(0, 12800, 132))) == 3
    assert _prefix(ws=None) == 7 and _prefix(ws=FAKE + 16) == 7
    need = _lib().shared_prefix_attn_workspace_size(2, 4, 2, 1, 128, 100, 50)
    assert need > 0 and _prefix(bytes=need - 1) == 7


def test_prefix_without_rows_is_a_no_op():
    assert _prefix(b=0) == 0 and _prefix(t=0) == 0
    assert _lib().shared_prefix_attn_workspace_size(2, 5, 2, 1, 128, 100, 50) == 0


def _backward(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, out=FAKE, dout=FAKE, lse=FAKE, layout=None, cq=[0, 10], ck=[0, 10], n=1, hq=4,
             hkv=2, d=128, qr=10, kr=10, causal=1, scale=0.0, dq=FAKE, dk=FAKE, dv=FAKE, ws=FAKE, bytes=1 << 20)
    a.update(kw)
    keep = [np.asarray(a[n], dtype=np.int32) for n in ("cq", "ck")]
    ptr = [x.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)) for x in keep]
    return _lib().dense_attn_varlen_backward(
        *[_p(a[n]) for n in ("q", "k", "v", "out", "dout", "lse")], a["layout"], ptr[0], ptr[1], a["n"], a["hq"],
        a["hkv"], a["d"], a["qr"], a["kr"], a["causal"], a["scale"], _p(a["dq"]), _p(a["dk"]), _p(a["dv"]),
        _p(a["ws"]), a["bytes"], None)


def test_backward_argument_checks():
    from block_sparse_attention_15_b200 import binding as B
    for n in ("q", "k", "v", "out", "dout", "dq", "dk", "dv"):
        assert _backward(**{n: None}) == 1 and _backward(**{n: FAKE + 8}) == 1
    assert _backward(lse=None) == 1 and _backward(n=0) == 2 and _backward(hq=5) == 2 and _backward(d=96) == 3
    assert _backward(cq=[0, 11]) == 2 and _backward(ck=[3, 10]) == 2
    cu = _i32([0, 10])
    need = _lib().dense_attn_varlen_backward_workspace_size(cu, cu, 1, 4, 2, 128, 10, 10, 1)
    assert need >= 160 and _lib().dense_attn_varlen_backward_workspace_size(cu, cu, 1, 5, 2, 128, 10, 10, 1) == 0
    assert _backward(ws=None) == 7 and _backward(ws=FAKE + 16) == 7 and _backward(bytes=need - 1) == 7
    good = dict(zip([n for n, _ in B.VsaDenseLayout._fields_], [(0, 1280, 128)] * 8))
    for n in good:
        lay = B.VsaDenseLayout(*[B.VsaStrides(*(good | {n: (0, 1280, 132)})[m]) for m in good])
        assert _backward(layout=ctypes.byref(lay)) == 3
    assert _backward(cq=[0, 0], ck=[0, 0], q=None, dk=None, lse=None, ws=None) == 0


def test_backward_workspace_of_shared_key_tiles():
    """One long sequence of many query heads over one key head has fewer key tiles
    than SMs: room for their partial sums, and no more than 80 MB."""
    f = _lib().dense_attn_varlen_backward_workspace_size

    def partial(hq, hkv, n, causal=1):
        cu = _i32([0, n])
        return f(cu, cu, 1, hq, hkv, 128, n, n, causal) - (4 * hq * n + 255) // 256 * 256

    assert partial(8, 1, 2000) == 16 * 2 * 2000 * 128 * 4               # 16 key tiles, shared by 16 items each
    assert partial(4, 1, 130) == 0 and partial(8, 8, 2000) == 0          # walks of 8 tiles; key tiles enough
    assert partial(40, 8, 8192) == 0
    for n in (130, 2000, 8192, 18000, 40000):
        for hq, hkv in ((8, 1), (16, 2), (64, 8), (12, 12)):
            for causal in (0, 1):
                assert 0 <= partial(hq, hkv, n, causal) <= 80 << 20
