"""Pins of the 8-bit operators' float64 oracle, and the refusals of their
entry points (no GPU)."""

import os

import numpy as np
import pytest

from ffn_block_gb300 import binding as B
from oracle import q8_oracle as Q


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from ffn_block_gb300 import build
        build.build()
    return B.lib()


# ------------------------------------------------------------------ oracle pins

def test_quant_rows_closed_form():
    q, s = Q.quant_rows(np.array([[127.0, -63.5, 0.4, 0.6], [0, 0, 0, 0], [1, np.inf, 2, 3]]))
    assert q.shape == (3, 32) and np.array_equal(q[0, :5], [127, -64, 0, 1, 0]) and s[0] == 1.0
    assert s[1] == 0 and not q[1].any()
    assert np.isnan(s[2]) and not q[2].any()


def test_checkpoint_exponent_is_the_smallest_that_fits():
    x = np.zeros((6, 32))
    x[:, 3] = [127.5, np.nextafter(127.5, 200), 64.0, 63.7, 0.0, np.nan]
    q, e = Q.ckpt_pack(x, "f32")
    assert e[:, 0].tolist() == [0, 1, 0, -1, -126, 127]
    assert q[:, 3].tolist() == [127, 64, 64, 127, 0, 0]
    v = Q.ckpt_values(q, e, 32)
    assert np.isnan(v[5]).all() and np.array_equal(v[4], np.zeros(32))


@pytest.mark.parametrize("dtype,top", [("f16", 65504.0), ("f32", 3.4028234663852886e38), ("bf16", 3.3895313892515355e38)])
def test_checkpoint_of_the_largest_value_stays_finite(dtype, top):
    q, e = Q.ckpt_pack(np.full((1, 32), top), dtype)
    v = Q.ckpt_values(q, e, 32)
    assert np.all(v <= top) and np.all(v >= top * (1 - 2.0 ** -6))


def test_checkpoint_error_is_half_a_step():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((20, 100)) * np.exp(rng.standard_normal((20, 100)))
    q, e = Q.ckpt_pack(x, "f32")
    step = np.repeat(2.0 ** e.astype(float), 32, axis=1)[:, :100]
    assert np.all(np.abs(Q.ckpt_values(q, e, 100) - x) <= step / 2)


def test_rms_gradients_match_differences():
    rng = np.random.default_rng(5)
    R, C, eps = 3, 17, 1e-5
    x, r, g, dn = (rng.standard_normal(s) for s in ((R, C), (R, C), (C,), (R, C)))
    dh = rng.standard_normal((R, C))

    def loss(x, r, g):
        h, _, n = Q.rms_norm(x, r, g, eps)
        return np.sum(n * dn) + np.sum(h * dh)

    h, rstd, _ = Q.rms_norm(x, r, g, eps)
    dx, dg = Q.rms_norm_backward(h, rstd, g, dn, dh)
    t = 1e-5
    for _ in range(4):
        vx, vg = rng.standard_normal((R, C)), rng.standard_normal(C)
        num = (loss(x + t * vx, r, g + t * vg) - loss(x - t * vx, r, g - t * vg)) / (2 * t)
        # central differences: error ~ t^2 third derivatives + rounding / t
        assert abs(num - (np.sum(dx * vx) + np.sum(dg * vg))) < 1e-6 * (1 + abs(num))


def test_linear_and_wgrad_match_loops():
    rng = np.random.default_rng(6)
    M, G, K, N = 3, 2, 5, 4
    a = rng.integers(-127, 128, (M, G, 32)).astype(np.int8)
    w = rng.integers(-127, 128, (G, N, 32)).astype(np.int8)
    sa, sw, b = rng.random((M, G)), rng.random((G, N)), rng.standard_normal((G, N))
    out = Q.linear_q8(a, sa, w, sw, b, None, K)
    x, dy = rng.standard_normal((M, G, K)), rng.standard_normal((M, G, N))
    dw, db = Q.wgrad(x, dy)
    for g in range(G):
        for n in range(N):
            for m in range(M):
                s = sum(int(a[m, g, k]) * int(w[g, n, k]) for k in range(K))
                assert np.isclose(out[m, g, n], s * sa[m, g] * sw[g, n] + b[g, n], rtol=1e-13)
            for k in range(K):
                assert np.isclose(dw[g, k, n], sum(x[m, g, k] * dy[m, g, n] for m in range(M)), rtol=1e-12)
            assert np.isclose(db[g, n], sum(dy[m, g, n] for m in range(M)), rtol=1e-12)


def test_planted_mistakes_are_seen():
    """A wrong oracle is caught by the pins: an exponent one too large, a
    dropped mean term in the norm's backward."""
    x = np.full((1, 32), 64.0)
    q, e = Q.ckpt_pack(x, "f32")
    assert not np.array_equal(Q.ckpt_values(q, e + 1, 32), x)
    rng = np.random.default_rng(7)
    h, g, dn = rng.standard_normal((2, 9)), np.ones(9), rng.standard_normal((2, 9))
    rstd = 1 / np.sqrt(np.mean(h * h, -1))
    dx, _ = Q.rms_norm_backward(h, rstd, g, dn, None)
    # the norm does not change when h is scaled: the gradient is orthogonal to h
    assert np.all(np.abs(np.sum(dx * h, -1)) < 1e-12)
    assert np.all(np.abs(np.sum(rstd[:, None] * dn * g * h, -1)) > 1e-3)


# ------------------------------------------------------------------ refusals

def rows(R=4, C=64, dt="bf16"):
    return B.make_rows(R, C, dt)


BAD_ROWS = [B.rmx_rows(-1, 64, 1), B.rmx_rows(4, 0, 1), B.rmx_rows(4, 64, 3), B.rmx_rows(4, 64, -1),
            B.rmx_rows(1 << 40, 64, 1), B.rmx_rows(4, (1 << 24) + 1, 1)]
BAD_LAYERS = [B.rmx_layer(-1, 1, 8, 8, 1), B.rmx_layer(1, 0, 8, 8, 1), B.rmx_layer(1, 1, 0, 8, 1),
              B.rmx_layer(1, 1, 8, 0, 1), B.rmx_layer(1, 1, 8, 8, 3), B.rmx_layer(1 << 30, 2, 8, 8, 1),
              B.rmx_layer(1, 65536, 8, 8, 1), B.rmx_layer(1, 1, (1 << 20) + 1, 8, 1),
              B.rmx_layer(1, 65535, 8, 1 << 20, 1)]
P, Pm = 0x1000, 0x1008   # an aligned and a misaligned address, never followed
INV, ALN, WS, UNS = B.RMX_ERR_INVALID_ARG, B.RMX_ERR_ALIGNMENT, B.RMX_ERR_WORKSPACE, B.RMX_ERR_UNSUPPORTED


def test_pitch(lib):
    assert [B.rmx_q8_pitch(c) for c in (1, 31, 32, 33, 1280)] == [32, 32, 32, 64, 1280]
    assert B.rmx_q8_pitch(0) == 0 and B.rmx_q8_pitch(-5) == 0 and B.rmx_q8_pitch((1 << 24) + 1) == 0


@pytest.mark.parametrize("bad", range(len(BAD_ROWS)))
def test_bad_row_shapes_are_refused(lib, bad):
    s = BAD_ROWS[bad]
    assert B.rmx_rms_norm_q8(s, 1e-5, P, None, P, None, None, P, P, None) == INV
    assert B.rmx_rms_norm_backward(s, P, None, P, None, None, P, P, P, P, P, 1 << 40) == INV
    assert B.rmx_rms_norm_backward_workspace_bytes(s) == 0
    assert B.rmx_quant_rows_q8(s, P, P, P) == INV
    assert B.rmx_dequant_rows_q8(s, P, P, P) == INV
    assert B.rmx_ckpt8_pack(s, P, P, P) == INV
    assert B.rmx_ckpt8_unpack(s, P, P, P) == INV


@pytest.mark.parametrize("bad", range(len(BAD_LAYERS)))
def test_bad_layers_are_refused(lib, bad):
    l = BAD_LAYERS[bad]
    assert B.rmx_linear_q8(l, P, P, P, P, None, None, P) == INV
    assert B.rmx_weight_q8(l, P, P, P) == INV
    assert B.rmx_ckpt8_wgrad_workspace_bytes(l) == 0
    assert B.rmx_ckpt8_wgrad(l, P, P, P, P, P, P, 1 << 40) == INV


def test_null_and_misaligned_pointers_are_refused(lib):
    s, l = rows(), B.make_layer(2, 2, 40, 24, "f16")
    nb, lb = B.rmx_rms_norm_backward_workspace_bytes(s), B.rmx_ckpt8_wgrad_workspace_bytes(l)
    calls = [
        (lambda *p: B.rmx_rms_norm_q8(s, 1e-5, p[0], None, p[1], None, None, p[2], p[3], None), 4),
        (lambda *p: B.rmx_rms_norm_backward(s, p[0], None, None, p[1], p[2], p[3], p[4], p[5], p[6], p[7], nb), 8),
        (lambda *p: B.rmx_quant_rows_q8(s, *p), 3),
        (lambda *p: B.rmx_dequant_rows_q8(s, *p), 3),
        (lambda *p: B.rmx_ckpt8_pack(s, *p), 3),
        (lambda *p: B.rmx_ckpt8_unpack(s, *p), 3),
        (lambda *p: B.rmx_weight_q8(l, *p), 3),
        (lambda *p: B.rmx_linear_q8(l, p[0], p[1], p[2], p[3], None, None, p[4]), 5),
        (lambda *p: B.rmx_ckpt8_wgrad(l, p[0], p[1], p[2], p[3], None, p[4], lb), 5),
    ]
    for k, (f, n) in enumerate(calls):
        for i in range(n):
            assert f(*[None if j == i else P for j in range(n)]) == INV, (k, i)
            assert f(*[Pm if j == i else P for j in range(n)]) == ALN, (k, i)
    # optional operands: null is fine, a misaligned one is not
    assert B.rmx_rms_norm_q8(s, 1e-5, P, Pm, P, None, None, P, P, None) == ALN
    assert B.rmx_rms_norm_q8(s, 1e-5, P, None, P, Pm, None, P, P, None) == ALN
    assert B.rmx_rms_norm_q8(s, 1e-5, P, None, P, None, None, P, P, Pm) == ALN
    assert B.rmx_linear_q8(l, P, P, P, P, Pm, None, P) == ALN
    assert B.rmx_linear_q8(l, P, P, P, P, None, Pm, P) == ALN
    assert B.rmx_ckpt8_wgrad(l, P, P, P, P, Pm, P, lb) == ALN


def test_contradictory_arguments_are_refused(lib):
    s = rows()
    nb = B.rmx_rms_norm_backward_workspace_bytes(s)
    assert B.rmx_rms_norm_q8(s, 1e-5, P, None, P, P, None, None, None, None) == INV     # no output of the norm
    assert B.rmx_rms_norm_q8(s, 1e-5, P, None, P, None, 0x2000, P, None, None) == INV   # q without scale
    assert B.rmx_rms_norm_q8(s, -1.0, P, None, P, None, None, P, P, None) == INV
    assert B.rmx_rms_norm_q8(s, float("nan"), P, None, P, None, None, P, P, None) == INV
    assert B.rmx_rms_norm_q8(s, 1e-5, P, None, P, None, P, P, P, None) == INV           # y over x
    assert B.rmx_rms_norm_backward(s, P, None, P, P, P, P, P, 0x2000, P, P, nb) == INV  # h and its checkpoint
    assert B.rmx_rms_norm_backward(s, P, None, None, None, None, P, P, P, P, P, nb) == INV
    assert B.rmx_rms_norm_backward(s, P, None, None, P, None, P, P, P, P, P, nb) == INV
    assert B.rmx_rms_norm_backward(s, P, None, 0x2000, None, None, P, P, 0x2000, P, P, nb) == INV  # dx over h


def test_small_workspaces_and_long_rows_are_refused(lib):
    s, l = rows(), B.make_layer(2, 2, 40, 24, "f16")
    assert B.rmx_rms_norm_backward(s, P, None, P, None, None, P, P, 0x2000, P, P,
                                   B.rmx_rms_norm_backward_workspace_bytes(s) - 1) == WS
    assert B.rmx_ckpt8_wgrad(l, P, P, P, P, P, P, B.rmx_ckpt8_wgrad_workspace_bytes(l) - 1) == WS
    long = rows(4, 16385)
    assert B.rmx_rms_norm_q8(long, 1e-5, P, None, P, None, None, P, P, None) == UNS
    assert B.rmx_quant_rows_q8(long, P, P, P) == UNS
    assert B.rmx_rms_norm_backward(long, P, None, P, None, None, P, P, 0x2000, P, P, 1 << 40) == UNS
    assert B.rmx_rms_norm_backward_workspace_bytes(long) == 0


def test_empty_batches_launch_nothing(lib):
    before = B.rmx_launch_count()
    s, l = rows(0), B.make_layer(0, 2, 40, 24, "f16")
    assert B.rmx_rms_norm_q8(s, 1e-5, None, None, None, None, None, P, P, None) == B.RMX_OK
    assert B.rmx_quant_rows_q8(s, None, None, None) == B.RMX_OK
    assert B.rmx_dequant_rows_q8(s, None, None, None) == B.RMX_OK
    assert B.rmx_ckpt8_pack(s, None, None, None) == B.RMX_OK
    assert B.rmx_ckpt8_unpack(s, None, None, None) == B.RMX_OK
    assert B.rmx_linear_q8(l, None, None, None, None, None, None, None) == B.RMX_OK
    assert B.rmx_launch_count() == before
