"""Dropout and layer norm (with dropout and residual, and its backward) against the float64 oracle."""

import numpy as np
import pytest
import torch

from ffn_block_gb300 import binding as B
from oracle import sparse_oracle as O
from tests.sparse_util import DEPTH, E32, TINY, U, dev, empty, f64, full_of, ok, rnd, state_of, sync, within

pytestmark = pytest.mark.gpu

SEED, OFFSET = 0xFEDCBA9876543210, (3 << 32) | 0x89ABCDEF
# Row lengths: one, odd, parts of a warp, both sides of every rule on lengths, whole and not whole 16-byte vectors.
COLS = [1, 7, 8, 24, 40, 63, 64, 72, 100, 128, 136, 250, 256, 264, 513, 768, 1001, 1280, 1288, 2560, 4097, 4104, 8192, 8200]


def _rows(rng, R, C, dt, shift=0.0):
    return rnd(rng.standard_normal((R, C)) + shift, dt)


# ------------------------------------------------------------------ dropout
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("R,C", [(1, 1), (3, 7), (5, 8), (37, 40), (9, 64), (6, 63), (4, 100), (17, 264), (33, 513), (128, 250),
                                 (700, 1200), (3, 20001), (2, 16392)])
@pytest.mark.parametrize("resid", [True, False])
def test_dropout(dt, R, C, resid):
    rng = np.random.default_rng(C)
    x, r = _rows(rng, R, C, dt), _rows(rng, R, C, dt) if resid else None
    out = empty((R, C), dt)
    ok(B.rmx_dropout(B.make_rows(R, C, dt), B.make_drop(0.3, state_of(SEED, OFFSET)), dev(x, dt),
                     dev(r, dt) if resid else None, out))
    f = O.drop_factor(R, C, 0.3, SEED, OFFSET)
    ref = x * f + (r if resid else 0.0)
    # the factor's own rounding, the product's, the sum's, then the storage type's
    within(f64(out), ref, 2 * E32 * np.abs(x * f) + (E32 + U[dt]) * np.abs(ref) + TINY[dt])
    if not resid:
        assert np.array_equal(f64(out) == 0, (f == 0) | (x == 0))


@pytest.mark.parametrize("p,rate", [(0.0, 1.0), (2.0 ** -18, 1.0), (1.0, 0.0), (1 - 2.0 ** -18, 0.0), (2.0 ** -16, None), (0.5, None)])
def test_dropout_probabilities(p, rate):
    R, C = 64, 512
    x = full_of((R, C), "f32", float("nan") if rate == 0.0 else 3.0)
    out = empty((R, C), "f32")
    ok(B.rmx_dropout(B.make_rows(R, C, "f32"), B.make_drop(p, None if rate is not None else state_of(1, 2)), x, None, out))
    if rate is not None:
        assert torch.equal(out, torch.full_like(out, 3.0 * rate))
    else:
        f = O.drop_factor(R, C, p, 1, 2)
        within(f64(out), 3.0 * f, 4 * E32 * 3.0 * f)


def test_dropout_drops_infinities_and_keeps_them():
    x = empty((2, 64), "bf16")
    x[0], x[1] = float("inf"), float("nan")
    out = empty((2, 64), "bf16")
    ok(B.rmx_dropout(B.make_rows(2, 64, "bf16"), B.make_drop(0.5, state_of(7, 7)), x, None, out))
    keep = O.keep(2, 64, 0.5, 7, 7)
    got = f64(out)
    assert np.all(got[~keep] == 0) and np.all(np.isinf(got[0][keep[0]])) and np.all(np.isnan(got[1][keep[1]]))


def test_dropout_in_place_and_its_backward():
    """out may be x or r; the backward is the same call, and matches differences of <out, g>."""
    rng = np.random.default_rng(5)
    R, C = 21, 72
    x, r, g, v = (rng.standard_normal((R, C)) for _ in range(4))
    shape, drop = B.make_rows(R, C, "f32"), B.make_drop(0.4, state_of(11, 12))
    out = empty((R, C), "f32")
    ok(B.rmx_dropout(shape, drop, dev(x, "f32"), dev(r, "f32"), out))
    a, b = dev(x, "f32"), dev(r, "f32")
    ok(B.rmx_dropout(shape, drop, a, dev(r, "f32"), a))
    ok(B.rmx_dropout(shape, drop, dev(x, "f32"), b, b))
    assert torch.equal(out, a) and torch.equal(out, b)
    dx, up, lo = (empty((R, C), "f32") for _ in range(3))
    ok(B.rmx_dropout(shape, drop, dev(g, "f32"), None, dx))
    h = 0.125
    ok(B.rmx_dropout(shape, drop, dev(x + h * v, "f32"), None, up))
    ok(B.rmx_dropout(shape, drop, dev(x - h * v, "f32"), None, lo))
    diff = ((f64(up) - f64(lo)) * g).sum() / (2 * h)
    # linear in x: each output is off by at most 3 roundings of values up to 5, over 2 h
    assert abs(diff - (f64(dx) * v).sum()) <= 8 * E32 * (5 / h + 5) * np.abs(g).sum()


def test_dropout_rows_of_the_counter():
    """Other offsets and seeds give other bits; the same state gives the same."""
    R, C = 16, 256
    x, outs = full_of((R, C), "f16", 1.0), []
    for s, o in ((1, 1), (1, 2), (2, 1), (1, 1 + (1 << 32)), (1 + (1 << 32), 1), (1, 1)):
        outs.append(empty((R, C), "f16"))
        ok(B.rmx_dropout(B.make_rows(R, C, "f16"), B.make_drop(0.5, state_of(s, o)), x, None, outs[-1]))
        assert np.array_equal(f64(outs[-1]) != 0, O.keep(R, C, 0.5, s, o))
    assert torch.equal(outs[0], outs[5]) and not any(torch.equal(outs[0], t) for t in outs[1:5])


def test_dropout_past_31_bits():
    """Elements past 2^31: rows near the end and in the middle."""
    C, R = 4096, (1 << 19) + 5
    x = torch.ones((R, C), dtype=torch.float16, device="cuda")
    ok(B.rmx_dropout(B.make_rows(R, C, "f16"), B.make_drop(0.5, state_of(3, 4)), x, None, x))
    for row in (0, 12345, (1 << 19) - 1, 1 << 19, R - 1):
        assert np.array_equal(f64(x[row : row + 1]) != 0, O.keep(1, C, 0.5, 3, 4, row0=row))


# ------------------------------------------------------------------ forward
def _forward(R, C, dt, p, resid, shift=0.0, affine=True, eps=1e-5, seed=0):
    rng = np.random.default_rng(seed + C)
    x, r = _rows(rng, R, C, dt, shift), _rows(rng, R, C, dt) if resid else None
    g = rnd(1 + 0.3 * rng.standard_normal(C), dt) if affine else None
    b = rnd(0.3 * rng.standard_normal(C), dt) if affine else None
    h, y, mean, rstd = empty((R, C), dt), empty((R, C), dt), empty((R,), "f32"), empty((R,), "f32")
    d = lambda a: None if a is None else dev(a, dt)  # noqa: E731
    ok(B.rmx_layer_norm(B.make_rows(R, C, dt), eps, B.make_drop(p, state_of(SEED, OFFSET)), d(x), d(r), d(g), d(b), h, y, mean,
                        rstd))
    f = O.drop_factor(R, C, p, SEED, OFFSET) if p else np.ones((R, C))
    hr = x * f + (r if resid else 0.0)
    e_h = 2 * E32 * np.abs(x * f) * (p > 0) + E32 * np.abs(hr) * resid
    yr, mr, sr = O.layer_norm(hr, g, b, eps)
    dv = np.abs(hr - mr[:, None])
    e_m = e_h.mean(-1) + (DEPTH + 2) * E32 * np.abs(hr).mean(-1)
    e_d = e_h + e_m[:, None] + E32 * dv
    var = (dv * dv).mean(-1)
    # a mean that is off by m adds m^2 to the squares' mean
    e_var = (2 * dv * e_d + e_d * e_d).mean(-1) + (DEPTH + 3) * E32 * var
    rel = 0.5 * e_var / (var + eps - np.minimum(e_var, 0.5 * (var + eps))) + 4 * E32
    gm, bm = (1.0 if g is None else np.abs(g)), (0.0 if b is None else np.abs(b))
    e_y = gm * (e_d * sr[:, None] * (1 + rel[:, None]) + dv * sr[:, None] * (rel[:, None] + 3 * E32)) + 2 * E32 * (np.abs(yr) + bm)
    within(f64(h), hr, e_h + U[dt] * np.abs(hr) + TINY[dt], "h")
    within(f64(mean), mr, e_m, "mean")
    within(f64(rstd), sr, sr * rel * (1 + rel), "rstd")
    within(f64(y), yr, e_y + U[dt] * (np.abs(yr) + e_y) + TINY[dt], "y")


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("C", COLS)
def test_layer_norm(dt, C):
    _forward(13, C, dt, 0.3, True)


@pytest.mark.parametrize("p,resid,affine", [(0.0, False, True), (0.0, True, False), (0.5, False, False), (0.9, True, True)])
@pytest.mark.parametrize("C", [40, 333, 1280, 3000])
def test_layer_norm_forms(p, resid, affine, C):
    _forward(70, C, "bf16", p, resid, affine=affine, seed=1)


@pytest.mark.parametrize("R", [1, 2, 31, 33, 257, 5000, 40000])
def test_layer_norm_row_counts(R):
    _forward(R, 64, "f32", 0.25, True, seed=2)


def test_layer_norm_long_rows():
    _forward(3, 16384, "f16", 0.1, True)
    _forward(3, 16383, "bf16", 0.1, True)


def test_layer_norm_far_from_zero():
    """A mean of 1000 with a deviation of 1: the deviations are taken from the mean, not from squares of the values."""
    _forward(20, 1280, "f32", 0.0, False, shift=1000.0)


def test_layer_norm_constant_and_faulty_rows():
    R, C = 6, 1280
    x = full_of((R, C), "f32", 2.0)
    x[1, 77], x[2, 5] = float("inf"), float("nan")
    x[3] = torch.randn(C, device="cuda")
    y, mean, rstd = empty((R, C), "f32"), empty((R,), "f32"), empty((R,), "f32")
    ok(B.rmx_layer_norm(B.make_rows(R, C, "f32"), 1e-5, None, x, None, None, None, None, y, mean, rstd))
    got = f64(y)
    assert np.all(got[[0, 4, 5]] == 0) and np.all(np.isnan(got[[1, 2]])) and np.all(np.isfinite(got[3]))
    assert abs(f64(rstd)[0] - 1 / np.sqrt(1e-5)) < 4 * E32 / np.sqrt(1e-5)
    ok(B.rmx_layer_norm(B.make_rows(R, C, "f32"), 0.0, None, x, None, None, None, None, y, None, rstd))
    assert np.all(np.isnan(f64(y)[0])) and np.isinf(f64(rstd)[0])


def test_layer_norm_sum_in_place():
    rng = np.random.default_rng(9)
    R, C = 50, 1280
    x, r = dev(_rows(rng, R, C, "bf16"), "bf16"), dev(_rows(rng, R, C, "bf16"), "bf16")
    s, d = B.make_rows(R, C, "bf16"), B.make_drop(0.2, state_of(1, 1))
    h, y = empty((R, C), "bf16"), empty((R, C), "bf16")
    ok(B.rmx_layer_norm(s, 1e-5, d, x, r, None, None, h, y, None, None))
    for which in (0, 1):
        a, b, y2 = x.clone(), r.clone(), empty((R, C), "bf16")
        ok(B.rmx_layer_norm(s, 1e-5, d, a, b, None, None, (a, b)[which], y2, None, None))
        assert torch.equal((a, b)[which], h) and torch.equal(y2, y)


def test_layer_norm_equals_dropout_then_norm():
    """The fused dropout draws the bits of the one by itself."""
    R, C = 40, 264
    x, r = (torch.randn((R, C), device="cuda") for _ in range(2))
    s, d = B.make_rows(R, C, "f32"), B.make_drop(0.35, state_of(5, 6))
    h, y, h2, y2 = (empty((R, C), "f32") for _ in range(4))
    ok(B.rmx_layer_norm(s, 1e-5, d, x, r, None, None, h, y, None, None))
    ok(B.rmx_dropout(s, d, x, r, h2))
    ok(B.rmx_layer_norm(s, 1e-5, None, h2, None, None, None, None, y2, None, None))
    assert torch.equal(h, h2) and torch.equal(y, y2)


# ------------------------------------------------------------------ backward
def _backward(R, C, dt, p, resid, affine=True, seed=0, shift=0.5):
    rng = np.random.default_rng(seed + C)
    h, dy = _rows(rng, R, C, dt, shift), _rows(rng, R, C, dt)
    dh = _rows(rng, R, C, dt) if resid else None
    g = rnd(1 + 0.3 * rng.standard_normal(C), dt) if affine else None
    _, mean, rstd = O.layer_norm(h, None, None, 1e-5)
    mean, rstd = mean.astype(np.float32).astype(np.float64), rstd.astype(np.float32).astype(np.float64)
    shape = B.make_rows(R, C, dt)
    nws = B.rmx_layer_norm_backward_workspace_bytes(shape)
    ws = full_of((nws,), torch.uint8, 255)
    dr, dx, dg, db = empty((R, C), dt), empty((R, C), dt) if p else None, empty((C,), dt), empty((C,), dt)
    d = lambda a: None if a is None else dev(a, dt)  # noqa: E731
    ok(B.rmx_layer_norm_backward(shape, B.make_drop(p, state_of(SEED, OFFSET)), d(dy), d(dh), d(h), dev(mean, "f32"),
                                 dev(rstd, "f32"), d(g), dr, dx, dg, db, ws, nws))
    rr, gr, br = O.layer_norm_backward(dy, dh, h, mean, rstd, g)
    s, m = rstd[:, None], np.abs(mean)[:, None]
    xh = np.abs((h - mean[:, None]) * s)
    e_x = E32 * (np.abs(h) * s + 2 * m * s + xh)
    t = np.abs(dy * (1.0 if g is None else g))
    e_c1 = (DEPTH + 3) * E32 * t.mean(-1, keepdims=True)
    e_c2 = (DEPTH + 4) * E32 * (t * xh).mean(-1, keepdims=True) + (t * e_x).mean(-1, keepdims=True)
    c1, c2 = t.mean(-1, keepdims=True), (t * xh).mean(-1, keepdims=True)   # at least their magnitudes
    e_r = s * (e_c1 + xh * e_c2 + e_x * c2 + 4 * E32 * (t + c1 + xh * c2)) + 2 * E32 * np.abs(rr)
    within(f64(dr), rr, e_r + U[dt] * (np.abs(rr) + e_r) + TINY[dt], "dr")
    if p:
        f = O.drop_factor(R, C, p, SEED, OFFSET)
        e = f * e_r + 2 * E32 * np.abs(rr * f)
        within(f64(dx), rr * f, e + U[dt] * (np.abs(rr * f) + e) + TINY[dt], "dx")
    n = (R + DEPTH) * E32
    e_g = n * np.abs(dy * xh).sum(0) + (np.abs(dy) * e_x).sum(0)
    within(f64(dg), gr, e_g + U[dt] * (np.abs(gr) + e_g) + TINY[dt], "dgamma")
    e_b = n * np.abs(dy).sum(0)
    within(f64(db), br, e_b + U[dt] * (np.abs(br) + e_b) + TINY[dt], "dbeta")


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("C", COLS)
def test_layer_norm_backward(dt, C):
    _backward(29, C, dt, 0.3, True)


@pytest.mark.parametrize("p,resid,affine", [(0.0, False, True), (0.0, True, False), (0.5, False, False)])
@pytest.mark.parametrize("C", [40, 333, 1280, 3000])
def test_layer_norm_backward_forms(p, resid, affine, C):
    _backward(70, C, "bf16", p, resid, affine=affine, seed=1)


@pytest.mark.parametrize("R,C", [(1, 64), (2, 1280), (31, 8), (33, 1280), (5000, 64), (40000, 40), (3001, 513), (9000, 1280)])
def test_layer_norm_backward_row_counts(R, C):
    _backward(R, C, "f32", 0.25, True, seed=2)


def test_layer_norm_backward_long_rows():
    _backward(5, 16384, "f16", 0.1, True)
    _backward(5, 16383, "bf16", 0.1, True)
    _backward(400, 16384, "f32", 0.1, True)


def test_layer_norm_backward_differences():
    """<dr, v> against the difference of <y, dy> + <h, dh> along v, and dgamma, dbeta likewise."""
    rng = np.random.default_rng(4)
    R, C, eps = 12, 200, 1e-5
    x, dy, dh, v = rng.standard_normal((4, R, C))
    g, b, vg, vb = rng.standard_normal((4, C))
    shape = B.make_rows(R, C, "f32")

    def f(s, out=None):
        h, y, m, r = empty((R, C), "f32"), empty((R, C), "f32"), empty((R,), "f32"), empty((R,), "f32")
        ok(B.rmx_layer_norm(shape, eps, None, dev(x + s * v, "f32"), None, dev(g + s * vg, "f32"), dev(b + s * vb, "f32"), h, y,
                            m, r))
        if out is not None:
            out.update(h=h, m=m, r=r)
        return (f64(y) * dy).sum() + (f64(h) * dh).sum()

    kept, step = {}, 1e-2
    f(0.0, kept)
    nws = B.rmx_layer_norm_backward_workspace_bytes(shape)
    dr, dg, db, ws = empty((R, C), "f32"), empty((C,), "f32"), empty((C,), "f32"), empty((nws,), torch.uint8)
    ok(B.rmx_layer_norm_backward(shape, None, dev(dy, "f32"), dev(dh, "f32"), kept["h"], kept["m"], kept["r"], dev(g, "f32"), dr,
                                 None, dg, db, ws, nws))
    got = (f64(dr) * v).sum() + (f64(dg) * vg).sum() + (f64(db) * vb).sum()
    # fourth-order differences: outputs are off by some 1e-6 of values near 1, over the step
    diff = (8 * (f(step) - f(-step)) - (f(2 * step) - f(-2 * step))) / (12 * step)
    assert abs(got - diff) < 2e-3 * np.abs(dy).sum() ** 0.5 + 1e-4 * abs(got)


def test_layer_norm_backward_in_place_and_some_gradients():
    rng = np.random.default_rng(6)
    R, C = 37, 1288
    h, dy, dh = (dev(_rows(rng, R, C, "bf16"), "bf16") for _ in range(3))
    mean, rstd = empty((R,), "f32"), empty((R,), "f32")
    mean.copy_(h.float().mean(-1))
    rstd.copy_(1 / h.float().std(-1))
    s, d = B.make_rows(R, C, "bf16"), B.make_drop(0.2, state_of(1, 1))
    nws = B.rmx_layer_norm_backward_workspace_bytes(s)
    ws = empty((nws,), torch.uint8)
    dr, dx, dg, db = empty((R, C), "bf16"), empty((R, C), "bf16"), empty((C,), "bf16"), empty((C,), "bf16")
    ok(B.rmx_layer_norm_backward(s, d, dy, dh, h, mean, rstd, None, dr, dx, dg, db, ws, nws))
    for which in (0, 1):
        a, b, dx2 = dy.clone(), dh.clone(), empty((R, C), "bf16")
        ok(B.rmx_layer_norm_backward(s, d, a, b, h, mean, rstd, None, (a, b)[which], dx2, None, None, ws, nws))
        assert torch.equal((a, b)[which], dr) and torch.equal(dx2, dx)
    for want in ((True, False), (False, True)):
        g2, b2 = (empty((C,), "bf16") if w else None for w in want)
        ok(B.rmx_layer_norm_backward(s, d, dy, dh, h, mean, rstd, None, dr, None, g2, b2, ws, nws))
        assert (g2 is None or torch.equal(g2, dg)) and (b2 is None or torch.equal(b2, db))


def test_layer_norm_backward_of_no_rows():
    s = B.make_rows(0, 24, "bf16")
    dg, db = full_of((24,), "bf16", 7.0), full_of((24,), "bf16", 7.0)
    ok(B.rmx_layer_norm_backward(s, None, None, None, None, None, None, None, None, None, dg, db, None, 0))
    assert not dg.any() and not db.any()


def test_layer_norm_repeats_bit_for_bit():
    R, C = 3001, 513
    h, dy = (torch.randn((R, C), device="cuda") for _ in range(2))
    mean, rstd = h.mean(-1), 1 / h.std(-1)
    s = B.make_rows(R, C, "f32")
    nws = B.rmx_layer_norm_backward_workspace_bytes(s)
    ws, outs = empty((nws,), torch.uint8), []
    for _ in range(3):
        dr, dg, db = empty((R, C), "f32"), empty((C,), "f32"), empty((C,), "f32")
        ok(B.rmx_layer_norm_backward(s, None, dy, None, h, mean, rstd, None, dr, None, dg, db, ws, nws))
        outs.append((dr, dg, db))
    assert all(torch.equal(a, b) for o in outs[1:] for a, b in zip(outs[0], o))
    sync()


@pytest.mark.parametrize("C", [40, 333, 1001, 1280, 4104])
def test_layer_norm_that_drops_everything(C):
    """p = 1: the sum is the residual, whatever x holds, and no gradient reaches x."""
    R = 200
    s, d = B.make_rows(R, C, "bf16"), B.make_drop(1.0)
    x, r, dy = full_of((R, C), "bf16", float("nan")), torch.randn((R, C), device="cuda").bfloat16(), torch.randn((R, C), device="cuda").bfloat16()
    h, y, y2, mean, rstd = empty((R, C), "bf16"), empty((R, C), "bf16"), empty((R, C), "bf16"), empty((R,), "f32"), empty((R,), "f32")
    ok(B.rmx_layer_norm(s, 1e-5, d, x, r, None, None, h, y, mean, rstd))
    ok(B.rmx_layer_norm(s, 1e-5, None, r, None, None, None, None, y2, None, None))
    assert torch.equal(h, r) and torch.equal(y, y2)
    nws = B.rmx_layer_norm_backward_workspace_bytes(s)
    dr, dr2, dx, ws = empty((R, C), "bf16"), empty((R, C), "bf16"), full_of((R, C), "bf16", 1.0), empty((nws,), torch.uint8)
    ok(B.rmx_layer_norm_backward(s, d, dy, None, h, mean, rstd, None, dr, dx, None, None, ws, nws))
    ok(B.rmx_layer_norm_backward(s, None, dy, None, h, mean, rstd, None, dr2, None, None, None, ws, nws))
    assert not dx.any() and torch.equal(dr, dr2)


@pytest.mark.parametrize("R", [3, 5000])
@pytest.mark.parametrize("C", [72, 513, 1280])
def test_layer_norm_with_one_parameter(R, C):
    """gamma without beta and beta without gamma: as with ones and zeros in the other's place.  Either side rounds the
    product twice and the sum once, or product and sum together: 2 |product| + |y| <= 3 |y| + 2 |beta| units each."""
    s = B.make_rows(R, C, "f32")
    x, g = torch.randn((R, C), device="cuda"), torch.randn(C, device="cuda")
    one, zero = torch.ones(C, device="cuda"), torch.zeros(C, device="cuda")
    for a, b in ((None, g), (g, None)):
        y, y2 = empty((R, C), "f32"), empty((R, C), "f32")
        ok(B.rmx_layer_norm(s, 1e-5, None, x, None, a, b, None, y, None, None))
        ok(B.rmx_layer_norm(s, 1e-5, None, x, None, one if a is None else a, zero if b is None else b, None, y2, None, None))
        ref, beta = f64(y2), 0.0 if b is None else np.abs(f64(b))
        within(f64(y), ref, 2 * E32 * (3 * np.abs(ref) + 2 * beta) * (1 + 2.0 ** -20))
