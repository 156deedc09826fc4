"""q8 rows at the ends of float32's range."""

import numpy as np
import pytest
import torch

from ffn_block_gb300 import binding as B
from oracle import q8_oracle as Q

from q8_util import E32, dev, empty, f64, ok, sync

pytestmark = pytest.mark.gpu
TOP = float(np.finfo(np.float32).max)


@pytest.mark.parametrize("C", [40, 41, 1288])
def test_rows_of_the_largest_values_read_back_finite(C):
    rng = np.random.default_rng(C)
    x = rng.uniform(-1, 1, (6, C)).astype(np.float32).astype(np.float64) * TOP
    x[:, 3] = [TOP, -TOP, np.float32(TOP * (1 - 2.0 ** -24)), np.float32(TOP * 0.999), TOP / 2, -TOP]
    x = x.astype(np.float32).astype(np.float64)
    sh, P = B.make_rows(6, C, "f32"), Q.pitch(C)
    q, s, v = empty((6, P), torch.int8), empty(6, torch.float32), empty((6, C), "f32")
    ok(B.rmx_quant_rows_q8(sh, dev(x, "f32"), q, s))
    ok(B.rmx_dequant_rows_q8(sh, q, s, v))
    sync()
    top = np.abs(x).max(1)
    # the scale: top / 127, one rounding, or one unit below it (2^-23)
    assert np.all(np.abs(f64(s) - top / 127) <= top / 127 * 3 * E32)
    got = f64(v)
    assert np.all(np.isfinite(got))
    # half a step; the scale's and the quotient's roundings of up to 127 steps, and the value's own
    assert np.all(np.abs(got - x) <= (top / 127 * (0.5 + 127 * 8 * E32))[:, None])


def test_weights_of_the_largest_values_have_finite_values():
    G, K, N = 2, 70, 5
    w = np.full((G, K, N), TOP)
    w[:, ::2] *= -1
    q, s = empty((G, N, Q.pitch(K)), torch.int8), empty((G, N), torch.float32)
    v = empty((G * N, K), "f32")
    ok(B.rmx_weight_q8(B.make_layer(1, G, K, N, "f32"), dev(w, "f32"), q, s))
    ok(B.rmx_dequant_rows_q8(B.make_rows(G * N, K, "f32"), q, s, v))
    sync()
    assert np.all(np.isfinite(f64(v))) and np.all(np.abs(np.abs(f64(v)) - TOP) <= TOP * 4 * E32)
