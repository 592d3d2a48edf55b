"""The dense kernels' FMA-pipe exponential (exp2_fma2_any in dense_attn.cuh),
modelled in float32 with its integer steps: the sparse kernels' values where
those are normal numbers, 0 below, NaN kept."""
import os
import re

import numpy as np

from block_sparse_attention_15_b200 import exp2_fit as E


def model(x):
    c = E.coefficients_f32()
    x = np.asarray(x, dtype=np.float32)
    xx = np.where(np.isnan(x), x, np.maximum(x, np.float32(-127.0))).astype(np.float32)  # max.NaN
    t = (xx + E.ROUND_MAGIC).astype(np.float32)
    j = (t - E.ROUND_MAGIC).astype(np.float32)
    f = E._fma32(j, np.float32(-1.0), xx)
    q = E._fma32(E._fma32(E._fma32(f, c[3], c[2]), f, c[1]), f, c[0])
    scale = ((t.view(np.uint32) << np.uint32(23)) + np.uint32(0x3F800000)).view(np.float32)
    return (q * scale).astype(np.float32)


def test_equals_the_sparse_kernels_values():
    rng = np.random.default_rng(3)
    x = np.concatenate([np.linspace(-120, 32, 400001), rng.uniform(-120, 32, 100000),
                        np.arange(-120, 33) + 0.5]).astype(np.float32)
    assert np.array_equal(model(x), E.exp2_model(x))


def test_small_values_and_values_that_are_none():
    x = np.array([-120.5, -126.0, -126.4], dtype=np.float32)
    assert np.allclose(model(x).astype(np.float64), np.exp2(x.astype(np.float64)), rtol=8e-5, atol=2.0 ** -149)
    assert (model([-126.6, -127.0, -150.0, -1e30, -np.inf]) == 0).all()
    with np.errstate(invalid="ignore"):
        assert np.isnan(model([np.nan, -np.nan, np.inf])).all()


def test_source_holds_the_fitted_coefficients():
    path = os.path.join(os.path.dirname(E.__file__), "csrc", "dense_attn.cuh")
    body = open(path).read()
    body = body[body.index("exp2_fma2_any(float"):]
    lits = re.findall(r"pk2\((-?0x1\.[0-9a-f]+p-?\d+)f,", body[:body.index("\n}\n")])
    assert [np.float32(float.fromhex(x)) for x in reversed(lits)] == list(E.coefficients_f32())
