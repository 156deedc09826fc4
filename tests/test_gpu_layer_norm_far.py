"""Layer norm's backward on rows far from zero: it takes h - mean before it multiplies, so what a row holds beyond its
deviations is not rounded with them."""

import numpy as np
import pytest
import torch

from ffn_block_gb300 import binding as B
from oracle import sparse_oracle as O
from tests.sparse_util import DEPTH, E32, TINY, U, dev, empty, f64, full_of, ok, rnd, within

pytestmark = pytest.mark.gpu


# one row length for each way that rows are given to lanes and warps, whole and odd vectors
@pytest.mark.parametrize("C", [7, 40, 100, 250, 500, 513, 1001, 1280, 1288, 4104, 16384])
@pytest.mark.parametrize("R,shift", [(29, 1000.0), (300, 1000.0), (29, 30000.0), (29, -10.0)])
def test_backward_far_from_zero(R, C, shift):
    """Float32 rows of deviation 1.  xh = (h - mean) * rstd rounds twice, each time by 2^-24 of itself at most, wherever
    the row lies; the other terms as in the backward's tests near zero."""
    rng = np.random.default_rng(C)
    h, dy, dh = (rnd(rng.standard_normal((R, C)) + s, "f32") for s in (shift, 0.0, 0.0))
    g = rnd(1 + 0.3 * rng.standard_normal(C), "f32")
    _, mean, rstd = O.layer_norm(h, None, None, 1e-5)
    mean, rstd = (v.astype(np.float32).astype(np.float64) for v in (mean, rstd))
    shape = B.make_rows(R, C, "f32")
    nws = B.rmx_layer_norm_backward_workspace_bytes(shape)
    dr, dg, db, ws = empty((R, C), "f32"), empty((C,), "f32"), empty((C,), "f32"), full_of((nws,), torch.uint8, 255)
    ok(B.rmx_layer_norm_backward(shape, None, dev(dy, "f32"), dev(dh, "f32"), dev(h, "f32"), dev(mean, "f32"), dev(rstd, "f32"),
                                 dev(g, "f32"), dr, None, dg, db, ws, nws))
    rr, gr, br = O.layer_norm_backward(dy, dh, h, mean, rstd, g)
    s = rstd[:, None]
    xh, t = np.abs((h - mean[:, None]) * s), np.abs(dy * g)
    e_x = 2 * E32 * (1 + E32) * xh
    c1, c2 = t.mean(-1, keepdims=True), (t * xh).mean(-1, keepdims=True)   # at least their magnitudes
    e_c1 = (DEPTH + 3) * E32 * c1
    e_c2 = (DEPTH + 4) * E32 * c2 + (t * e_x).mean(-1, keepdims=True)
    e_r = s * (e_c1 + xh * e_c2 + e_x * c2 + 4 * E32 * (t + c1 + xh * c2)) + 2 * E32 * np.abs(rr)
    within(f64(dr), rr, e_r + U["f32"] * (np.abs(rr) + e_r) + TINY["f32"], "dr")
    n = (R + DEPTH) * E32
    e_g = n * np.abs(dy * xh).sum(0) + (np.abs(dy) * e_x).sum(0)
    within(f64(dg), gr, e_g + U["f32"] * (np.abs(gr) + e_g) + TINY["f32"], "dgamma")
    e_b = n * np.abs(dy).sum(0)
    within(f64(db), br, e_b + U["f32"] * (np.abs(br) + e_b) + TINY["f32"], "dbeta")
