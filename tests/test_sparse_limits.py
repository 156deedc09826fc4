"""Refusals of the sparse layer's operators: found on the host, before anything is enqueued (no GPU)."""

import os

import pytest

from ffn_block_gb300 import binding as B

P, Q, R, S = 0x1000, 0x2000, 0x3000, 0x4000   # aligned addresses, never followed
ODD = 0x1008
INV, UNS, ALI, WS = B.RMX_ERR_INVALID_ARG, B.RMX_ERR_UNSUPPORTED, B.RMX_ERR_ALIGNMENT, B.RMX_ERR_WORKSPACE
BIG = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def nothing_enqueued():
    if not os.path.exists(B.LIB_PATH):
        from ffn_block_gb300 import build
        build.build()
    before = B.rmx_launch_count()
    yield
    assert B.rmx_launch_count() == before


def test_rows_without_rows():
    none = B.make_rows(0, 40, "bf16")
    d = B.make_drop(0.5, P)
    assert B.rmx_dropout(none, d, None, None, None) == B.RMX_OK
    assert B.rmx_layer_norm(none, 1e-5, d, None, None, None, None, None, None, None, None) == B.RMX_OK
    assert B.rmx_quant_f8(none, "e4m3", None, None, None) == B.RMX_OK
    assert B.rmx_dequant_f8(none, "e5m2", None, None, None) == B.RMX_OK
    r = B.make_routes(0, 2, 8, 64, "bf16")
    assert B.rmx_expert_gather(r, None, None, P, "e4m3") == B.RMX_OK
    assert B.rmx_expert_combine(r, None, None, None, None) == B.RMX_OK
    assert B.rmx_expert_combine_backward(r, None, None, None, None, P, None) == B.RMX_OK
    l = B.make_layer_f8(0, 4, 64, 64, "bf16")
    assert B.rmx_linear_f8(l, None, None, None, None, None, None, None, None) == B.RMX_OK


@pytest.mark.parametrize("bad", [dict(rows=-1, cols=8, dtype="f32"), dict(rows=4, cols=0, dtype="f32"),
                                 dict(rows=4, cols=(1 << 24) + 1, dtype="f32"), dict(rows=(1 << 36) + 1, cols=8, dtype="f32"),
                                 dict(rows=4, cols=8, dtype="tf32"), dict(rows=4, cols=8, dtype=9)])
def test_row_shapes(bad):
    s = B.make_rows(**bad)
    assert B.rmx_dropout(s, None, P, None, Q) == INV
    assert B.rmx_layer_norm(s, 1e-5, None, P, None, None, None, None, Q, None, None) == INV
    assert B.rmx_layer_norm_backward_workspace_bytes(s) == 0
    assert B.rmx_layer_norm_backward(s, None, P, None, Q, P, P, None, R, None, None, None, S, BIG) == INV
    assert B.rmx_quant_f8(s, "e4m3", P, Q, R) == INV
    assert B.rmx_dequant_f8(s, "e4m3", P, Q, R) == INV


def test_rows_longer_than_the_norm_holds():
    s = B.make_rows(4, 16385, "f32")
    assert B.rmx_layer_norm(s, 1e-5, None, P, None, None, None, None, Q, None, None) == UNS
    assert B.rmx_layer_norm_backward(s, None, P, None, Q, P, P, None, R, None, None, None, S, BIG) == UNS
    assert B.rmx_layer_norm_backward_workspace_bytes(s) == 0
    assert B.rmx_layer_norm_backward_workspace_bytes(B.make_rows(4, 16384, "f32")) > 0


@pytest.mark.parametrize("p", [-0.1, 1.5, float("nan"), float("inf")])
def test_probabilities(p):
    s, d = B.make_rows(4, 64, "f32"), B.make_drop(p, P)
    assert B.rmx_dropout(s, d, P, None, Q) == INV
    assert B.rmx_layer_norm(s, 1e-5, d, P, None, None, None, None, Q, None, None) == INV
    assert B.rmx_layer_norm_backward(s, d, P, None, Q, P, P, None, R, None, None, None, S, BIG) == INV


def test_dropout_needs_its_state():
    s = B.make_rows(4, 64, "f32")
    assert B.rmx_dropout(s, B.make_drop(0.5), P, None, Q) == INV
    assert B.rmx_dropout(s, B.make_drop(0.5, ODD), P, None, Q) == ALI
    assert B.rmx_layer_norm(s, 1e-5, B.make_drop(0.5), P, None, None, None, None, Q, None, None) == INV
    # looked at only where dx is asked for; then the workspace is the next thing that is wrong
    args = (P, None, Q, P, P, None, R)
    assert B.rmx_layer_norm_backward(s, B.make_drop(0.5), *args, S, None, None, S, 0) == INV
    assert B.rmx_layer_norm_backward(s, B.make_drop(0.5), *args, None, None, None, S, 0) == WS
    assert B.rmx_layer_norm_backward(s, B.make_drop(1.0), *args, 0x5000, None, None, S, 0) == WS


def test_layer_norm_pointers():
    s = B.make_rows(4, 64, "f32")
    f = lambda **k: B.rmx_layer_norm(s, k.pop("eps", 1e-5), None, *(k.get(n, v) for n, v in  # noqa: E731
                                     dict(x=P, r=None, gamma=None, beta=None, h=None, y=Q, mean=None, rstd=None).items()))
    assert f(eps=-1.0) == INV and f(eps=float("nan")) == INV
    assert f(x=None) == INV and f(y=None) == INV
    assert f(y=P) == INV and f(r=Q) == INV and f(h=Q) == INV
    for n in ("x", "r", "gamma", "beta", "h", "y", "mean", "rstd"):
        assert f(**{n: ODD}) == ALI
    names = dict(dy=P, dh=None, h=Q, mean=P, rstd=P, gamma=None, dr=R, dx=None, dgamma=None, dbeta=None, ws=S)
    g = lambda **k: B.rmx_layer_norm_backward(s, None, *(k.get(n, v) for n, v in names.items()), k.get("n", BIG))  # noqa: E731
    for n in ("dy", "h", "mean", "rstd", "dr", "ws"):
        assert g(**{n: None}) == INV
    for n in names:
        assert g(**{n: ODD}) == ALI
    assert g(dr=Q) == INV and g(dx=Q) == INV and g(dx=R) == INV and g(dx=P) == INV
    assert g(n=B.rmx_layer_norm_backward_workspace_bytes(s) - 1) == WS


@pytest.mark.parametrize("bad", [dict(tokens=-1), dict(k=0), dict(k=65), dict(experts=0), dict(experts=1025),
                                 dict(tokens=1 << 26, k=32)])
def test_routes(bad):
    r = B.make_routes(**{**dict(tokens=8, k=2, experts=4, cols=64, dtype="bf16"), **bad})
    assert B.rmx_expert_sort_workspace_bytes(r) == 0
    assert B.rmx_expert_sort(r, P, Q, R, S, P, BIG) == INV
    assert B.rmx_expert_gather(r, P, Q, R, "e4m3") == INV
    assert B.rmx_expert_combine(r, P, None, Q, R) == INV
    assert B.rmx_expert_combine_backward(r, P, None, Q, R, S, None) == INV


def test_routes_rows():
    for bad in (dict(cols=0), dict(cols=16385), dict(dtype="tf32"), dict(dtype=5)):
        r = B.make_routes(**{**dict(tokens=8, k=2, experts=4, cols=64, dtype="bf16"), **bad})
        assert B.rmx_expert_sort_workspace_bytes(r) > 0     # the sort reads neither
        assert B.rmx_expert_gather(r, P, Q, R, "e4m3") == INV
        assert B.rmx_expert_combine(r, P, None, Q, R) == INV
        assert B.rmx_expert_combine_backward(r, P, None, Q, R, S, None) == INV


def test_routes_pointers():
    r = B.make_routes(8, 2, 4, 64, "bf16")
    n = B.rmx_expert_sort_workspace_bytes(r)
    assert B.rmx_expert_sort(r, P, Q, R, S, P, n - 1) == WS
    for i in range(5):
        args = [P, Q, R, S, P]
        args[i] = None
        assert B.rmx_expert_sort(r, *args, n) == INV
        args[i] = ODD
        assert B.rmx_expert_sort(r, *args, n) == ALI
    assert B.rmx_expert_gather(r, P, Q, None, "e4m3") == INV          # nothing to write
    assert B.rmx_expert_gather(r, P, Q, None, "e4m3", R, None) == INV
    assert B.rmx_expert_gather(r, P, Q, Q, "e4m3") == INV
    assert B.rmx_expert_gather(r, P, Q, R, 2) == INV
    assert B.rmx_expert_gather(r, ODD, Q, R, "e4m3") == ALI
    assert B.rmx_expert_combine(r, P, ODD, Q, R) == ALI
    assert B.rmx_expert_combine(r, P, None, Q, Q) == INV
    assert B.rmx_expert_combine_backward(r, P, None, Q, None, None, S) == INV   # dweight needs y
    assert B.rmx_expert_combine_backward(r, P, None, Q, None, None, None) == INV
    assert B.rmx_expert_combine_backward(r, P, None, Q, R, Q, None) == INV


def test_f8_sizes():
    assert [B.rmx_f8_pitch(c) for c in (0, 1, 128, 129, 1 << 24, (1 << 24) + 1)] == [0, 128, 128, 256, 1 << 24, 0]
    assert [B.rmx_f8_exps(c) for c in (0, 1, 512, 513, 1024)] == [0, 4, 4, 8, 8]
    assert B.rmx_f8_ragged_pitch(0, 8) == 0
    assert B.rmx_f8_ragged_pitch(1, 8) == 128 and B.rmx_f8_ragged_pitch(300, 4) == 128 * (2 + 4)
    assert B.rmx_f8_ragged_pitch(8, 1025) == 0 and B.rmx_f8_ragged_pitch(-1, 4) == 0
    s = B.make_rows(4, 64, "f32")
    assert B.rmx_quant_f8(s, 2, P, Q, R) == INV and B.rmx_dequant_f8(s, -1, P, Q, R) == INV
    for args in ((None, Q, R), (P, None, R), (P, Q, None)):
        assert B.rmx_quant_f8(s, "e4m3", *args) == INV and B.rmx_dequant_f8(s, "e4m3", *args) == INV
    assert B.rmx_quant_f8(s, "e4m3", P, ODD, R) == ALI


@pytest.mark.parametrize("bad", [dict(M=-1), dict(G=0), dict(C=0), dict(dtype="tf32"), dict(order=3), dict(M=(1 << 24) + 1),
                                 dict(M=1 << 24, G=128), dict(C=1 << 24, G=128), dict(order="ragged", G=1025)])
def test_groups(bad):
    g = B.make_groups(**{**dict(M=300, G=4, C=64, dtype="bf16", order="tokens"), **bad})
    off = P if bad.get("order") == "ragged" else None
    assert B.rmx_quant_f8_groups_workspace_bytes(g) == 0
    assert B.rmx_quant_f8_groups(g, "e4m3", off, P, Q, R, None, None, None, None, 0) == INV


def test_groups_arguments():
    g, r = (B.make_groups(300, 4, 64, "bf16", o) for o in ("groups", "ragged"))
    f = B.rmx_quant_f8_groups
    assert f(g, 2, None, P, Q, R, None, None, None, None, 0) == INV
    assert f(g, "e4m3", P, P, Q, R, None, None, None, None, 0) == INV        # offsets without ragged
    assert f(r, "e4m3", None, P, Q, R, None, None, None, None, 0) == INV     # and the other way
    assert f(g, "e4m3", None, P, Q, None, None, None, None, None, 0) == INV
    assert f(g, "e4m3", None, P, None, None, Q, None, None, None, 0) == INV
    assert f(g, "e4m3", None, P, None, None, None, None, None, None, 0) == INV
    assert f(g, "e4m3", None, None, Q, R, None, None, None, None, 0) == INV
    assert f(g, "e4m3", None, P, ODD, R, None, None, None, None, 0) == ALI
    n = B.rmx_quant_f8_groups_workspace_bytes(g)
    assert f(g, "e4m3", None, P, None, None, None, None, Q, R, n - 1) == WS
    assert f(g, "e4m3", None, P, None, None, None, None, Q, None, n) == INV
    huge = B.make_groups(1 << 24, 1, 1 << 24, "bf16", "groups")   # more tiles than a grid counts
    assert B.rmx_quant_f8_groups_workspace_bytes(huge) == 0
    assert f(huge, "e4m3", None, P, Q, R, None, None, None, None, 0) == UNS


@pytest.mark.parametrize("bad", [dict(M=-1), dict(G=0), dict(K=0), dict(N=0), dict(K=(1 << 20) + 1), dict(N=(1 << 20) + 1),
                                 dict(G=65536), dict(dtype="tf32"), dict(a_format=2), dict(b_format=-1),
                                 dict(G=1024, K=(1 << 20) + 0, N=8, M=1 << 21)])
def test_layers(bad):
    l = B.make_layer_f8(**{**dict(M=8, G=4, K=64, N=64, dtype="bf16"), **bad})
    assert B.rmx_linear_f8(l, None, P, P, P, P, None, None, Q) == INV
    assert B.rmx_wgrad_f8(l, None, P, P, P, P, Q) == INV


def test_layer_arguments():
    l = B.make_layer_f8(8, 4, 64, 64, "bf16")
    for i in (0, 1, 2, 3, 6):
        args = [P, P, P, P, None, None, Q]
        args[i] = None
        assert B.rmx_linear_f8(l, None, *args) == INV
        args[i] = ODD
        assert B.rmx_linear_f8(l, None, *args) == ALI
    assert B.rmx_linear_f8(l, None, P, P, P, P, ODD, None, Q) == ALI
    assert B.rmx_linear_f8(l, ODD, P, P, P, P, None, None, Q) == ALI
    for i in range(5):
        args = [P, P, P, P, Q]
        args[i] = None
        assert B.rmx_wgrad_f8(l, None, *args) == INV
    many = B.make_layer_f8(8, 1025, 64, 64, "bf16")                     # experts
    assert B.rmx_linear_f8(many, P, P, P, P, P, None, None, Q) == INV
    assert B.rmx_wgrad_f8(many, P, P, P, P, P, Q) == INV
    wide = B.make_layer_f8(8, 1, 1 << 20, 1 << 20, "bf16")              # past a tensor map's strides
    assert B.rmx_linear_f8(wide, None, P, P, P, P, None, None, Q) == UNS
    long = B.make_layer_f8(1 << 30, 1, 1 << 10, 8, "bf16")
    assert B.rmx_wgrad_f8(long, None, P, P, P, P, Q) == UNS
