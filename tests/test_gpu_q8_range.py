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


@pytest.mark.parametrize("C", [40, 41, 1288])
def test_norm_rows_without_a_finite_norm(C):
    """Scale and integers say what the float32 norm is: NaN and zeros where it holds an infinity or a NaN, 0 and zeros
    where it is zero."""
    x = np.ones((6, C))
    x[0] = 0            # 0 * infinity
    x[1] = 1e-30        # the squares vanish: infinity
    x[2] = 1e25         # the squares pass float32: zero
    x[3], x[3, 1] = 1e-30, 0
    x[4], x[4, 0] = 1e-3, 1e-2
    x[5] = 3
    g = np.ones(C)
    g[0] = 3e38         # row 4: 3e36 before its norm, an infinity after it; row 5: below float32's largest value
    x[5, 0] = 0.5
    sh, P = B.make_rows(6, C, "f32"), Q.pitch(C)
    y, s, rstd = empty((6, C), "f32"), empty(6, torch.float32), empty(6, torch.float32)
    q = torch.full((6, P), 5, dtype=torch.int8, device="cuda")
    ok(B.rmx_rms_norm_q8(sh, 0.0, dev(x, "f32"), None, dev(g, "f32"), None, y, q, s, rstd))
    sync()
    qd, sd = q, s
    y, q, s = f64(y), f64(q), f64(s)
    assert f64(rstd)[0] == np.inf and f64(rstd)[1] == np.inf and f64(rstd)[2] == 0
    for r in range(6):
        if not np.isfinite(y[r]).all():
            assert np.isnan(s[r]) and not q[r].any(), r
        elif not y[r].any():
            assert s[r] == 0 and not q[r].any(), r
        else:
            top = np.abs(y[r]).max()
            # y and the scale: two float32 products each way
            assert abs(s[r] - top / 127) <= top / 127 * 6 * E32, r
            assert np.all(np.abs(q[r, :C] * s[r] - y[r]) <= top / 127 * (0.5 + 127 * 8 * E32)), r
    # n in float32 as (h * gamma) * rstd; row 2's first column is 1e25 * 3e38 times 0
    with np.errstate(all="ignore"):
        n = (x.astype(np.float32) * g.astype(np.float32)) * f64(rstd).astype(np.float32)[:, None]
    finite = np.isfinite(n).all(1)
    assert finite.tolist() == [False, False, False, False, False, True]
    assert np.isfinite(y).all(1).tolist() == finite.tolist()
    assert not y[2, 1:].any() and y[5].any()

    g[0] = 1            # row 2 without the first column's product: the norm of squares past float32 is zero
    ok(B.rmx_rms_norm_q8(sh, 0.0, dev(x, "f32"), None, dev(g, "f32"), None, None, qd, sd, None))
    sync()
    assert f64(sd)[2] == 0 and not f64(qd)[2].any()
