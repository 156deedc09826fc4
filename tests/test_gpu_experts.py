"""Routing to experts against the oracle: the sort, the gather (also to 8 bits), the combination and their backward."""

import numpy as np
import pytest
import torch

from ffn_block_gb300 import binding as B
from oracle import sparse_oracle as O
from tests.sparse_util import DEPTH, E32, TINY, U, dev, empty, f64, full_of, ok, rnd, within

pytestmark = pytest.mark.gpu
NAN = float("nan")


def _sort(ids, E):
    T, k = ids.shape
    r = B.make_routes(T, k, E, 1, "f32")
    nws = B.rmx_expert_sort_workspace_bytes(r)
    off, pos, src = (full_of(n, torch.int32, -7) for n in ((E + 1,), (T, k), (T * k,)))
    ws = full_of((nws,), torch.uint8, 255)
    ok(B.rmx_expert_sort(r, dev(ids.astype(np.int32)), off, pos, src, ws, nws))
    return off, pos, src


def _check_sort(ids, E):
    got = _sort(ids, E)
    for a, b in zip(got, O.expert_sort(ids, E)):
        assert np.array_equal(a.cpu().numpy(), b)
    return got


# both sides of the limits of one CTA (2048 slots) and of a cluster (49152), and of a warp's share; experts up to 1024
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 64, 3), (5, 2, 7), (31, 1, 2), (33, 3, 1024), (64, 2, 32), (1024, 8, 64),
                                   (2048, 1, 5), (2049, 1, 5), (8193, 1, 5), (4097, 2, 1024), (1229, 7, 33), (49152, 1, 64),
                                   (49153, 1, 64), (12289, 4, 1024), (65536, 2, 64), (20000, 8, 200)])
def test_sort(T, k, E):
    rng = np.random.default_rng(T)
    _check_sort(rng.integers(0, E, (T, k)), E)
    _check_sort(rng.integers(-1, E + 2, (T, k)), E)          # some dropped
    _check_sort((rng.random((T, k)) ** 6 * E).astype(int), E)  # few experts take most


@pytest.mark.parametrize("T,k,E", [(300, 3, 8), (9000, 2, 40)])
def test_sort_edges(T, k, E):
    _check_sort(np.full((T, k), -1), E)                      # nothing is routed
    _check_sort(np.full((T, k), E), E)
    _check_sort(np.full((T, k), np.iinfo(np.int32).min), E)
    _check_sort(np.full((T, k), E - 1), E)                   # all to one; every choice of a token the same
    ids = np.full((T, k), -1)
    ids[-1, -1] = 0
    _check_sort(ids, E)


def test_sort_of_no_tokens():
    off = full_of((5,), torch.int32, 9)
    ok(B.rmx_expert_sort(B.make_routes(0, 2, 4, 1, "f32"), None, off, None, None, None, 0))
    assert not off.any()


def test_sort_many_slots():
    """More slots than 4096 warps take at 512 each."""
    T, k, E = 1_500_000, 2, 129
    rng = np.random.default_rng(0)
    ids = rng.integers(-1, E, (T, k)).astype(np.int32)
    off, pos, src = (a.cpu().numpy() for a in _sort(ids, E))
    flat = ids.reshape(-1)
    order = np.argsort(np.where(flat < 0, E, flat), kind="stable")
    n = int((flat >= 0).sum())
    assert off[-1] == n and np.array_equal(src[:n], order[:n]) and np.all(src[n:] == -1)
    assert np.array_equal(pos.reshape(-1)[order[:n]], np.arange(n)) and np.all(pos.reshape(-1)[flat < 0] == -1)


SHAPES = [(1, 1, 1), (3, 2, 7), (40, 2, 8), (13, 4, 40), (25, 3, 64), (9, 2, 72), (17, 2, 100), (50, 8, 130), (21, 2, 513),
          (30, 5, 1001), (64, 2, 1280), (11, 3, 4104), (7, 2, 16384), (6, 2, 16383)]


def _case(T, k, C, dt, seed=0):
    rng = np.random.default_rng(seed + C)
    E = 6
    ids = rng.integers(-1, E, (T, k))
    off, pos, src = O.expert_sort(ids, E)
    return rng, B.make_routes(T, k, E, C, dt), int(off[-1]), pos, src


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,k,C", SHAPES)
def test_gather_and_its_backward(dt, T, k, C):
    rng, r, n, pos, src = _case(T, k, C, dt)
    x = rnd(rng.standard_normal((T, C)), dt)
    out = full_of((T * k, C), dt, 5.0)
    ok(B.rmx_expert_gather(r, dev(src), dev(x, dt), out))
    got = f64(out)
    assert np.array_equal(got[:n], x[src[:n] // k]) and np.all(got[n:] == 5.0)
    d = rnd(rng.standard_normal((T * k, C)), dt)
    d[n:] = NAN                                              # rows behind the last expert's are not read
    dx = empty((T, C), dt)
    ok(B.rmx_expert_combine(r, dev(pos), None, dev(d, dt), dx))
    ref = O.combine(pos, None, d)
    mag = O.combine(pos, None, np.abs(d))
    within(f64(dx), ref, k * E32 * mag + U[dt] * np.abs(ref) + TINY[dt])


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,k,C", SHAPES)
def test_combine_and_its_backward(dt, T, k, C):
    rng, r, n, pos, src = _case(T, k, C, dt, 1)
    y, dout = rnd(rng.standard_normal((T * k, C)), dt), rnd(rng.standard_normal((T, C)), dt)
    y[n:] = NAN
    w = rng.random((T, k)).astype(np.float32).astype(np.float64)
    w[pos < 0] = NAN                                         # dropped slots' weights are not used
    out = empty((T, C), dt)
    ok(B.rmx_expert_combine(r, dev(pos), dev(w, "f32"), dev(y, dt), out))
    ref, mag = O.combine(pos, w, y), O.combine(pos, w, np.abs(y))
    within(f64(out), ref, (k + 1) * E32 * mag + U[dt] * np.abs(ref) + TINY[dt], "out")
    ry, rw = O.combine_backward(pos, w, dout, y)
    bound_w = (DEPTH + 2) * E32 * O.combine_backward(pos, w, np.abs(dout), np.abs(y))[1]
    for weights in (True, False):
        dy, dw = full_of((T * k, C), dt, 3.0), full_of((T, k), "f32", NAN)
        ok(B.rmx_expert_combine_backward(r, dev(pos), dev(w, "f32") if weights else None, dev(dout, dt), dev(y, dt), dy, dw))
        want = ry if weights else O.combine_backward(pos, None, dout, y)[0]
        got = f64(dy)
        assert np.all(got[n:] == 3.0)
        within(got[:n], want[:n], (E32 + U[dt]) * np.abs(want[:n]) + TINY[dt], "dy")
        within(f64(dw), rw, bound_w, "dweight")
    # one of them alone, and dy in place of y
    only, inplace = empty((T, k), "f32"), dev(y, dt)
    ok(B.rmx_expert_combine_backward(r, dev(pos), dev(w, "f32"), dev(dout, dt), inplace, None, only))
    assert torch.equal(only, dw)
    ok(B.rmx_expert_combine_backward(r, dev(pos), dev(w, "f32"), dev(dout, dt), inplace, inplace, only))
    assert torch.equal(only, dw)
    dy2 = full_of((T * k, C), dt, 3.0)
    ok(B.rmx_expert_combine_backward(r, dev(pos), dev(w, "f32"), dev(dout, dt), None, dy2, None))
    assert torch.equal(dy2[:n], inplace[:n])


def test_combine_of_dropped_tokens():
    r = B.make_routes(4, 3, 2, 40, "bf16")
    out = full_of((4, 40), "bf16", 9.0)
    pos = full_of((4, 3), torch.int32, -1)
    ok(B.rmx_expert_combine(r, pos, full_of((4, 3), "f32", NAN), full_of((12, 40), "bf16", NAN), out))
    assert not out.any()


def test_indices_out_of_range_are_left_out():
    """Positions and sources that no sort writes are taken as dropped slots: nothing outside the arrays is touched."""
    T, k, C = 8, 2, 72
    r = B.make_routes(T, k, 4, C, "f32")
    bad = torch.tensor([-1, -(1 << 31), 16, (1 << 31) - 1] * 4, dtype=torch.int32, device="cuda")
    x, y = torch.randn((T, C), device="cuda"), torch.randn((T * k, C), device="cuda")
    out = full_of((T * k, C), "f32", 1.0)
    ok(B.rmx_expert_gather(r, bad, x, out))
    assert torch.equal(out, torch.ones_like(out))
    q, e = full_of((T * k, 128), torch.uint8, 3), full_of((T * k, 4), torch.uint8, 3)
    ok(B.rmx_expert_gather(r, bad, x, out, "e4m3", q, e))
    assert torch.equal(out, torch.ones_like(out)) and torch.all(q == 3) and torch.all(e == 3)
    res = empty((T, C), "f32")
    ok(B.rmx_expert_combine(r, bad, None, y, res))
    assert not res.any()
    dw = empty((T, k), "f32")
    ok(B.rmx_expert_combine_backward(r, bad, None, x, y, out, dw))
    assert torch.equal(out, torch.ones_like(out)) and not dw.any()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,k,C", [(3, 2, 7), (40, 2, 128), (13, 4, 136), (30, 5, 1001), (64, 2, 1280)])
def test_gather_to_8_bits(fmt, dt, T, k, C):
    """The same bytes as quantising the gathered rows, with the rows beside them or not."""
    rng, r, n, pos, src = _case(T, k, C, dt, 2)
    x = dev(rnd(rng.standard_normal((T, C)), dt), dt)
    S, P, EP = T * k, B.rmx_f8_pitch(C), B.rmx_f8_exps(C)
    rows = full_of((S, C), dt, 0.0)
    ok(B.rmx_expert_gather(r, dev(src), x, rows))
    q, e = full_of((S, P), torch.uint8, 9), full_of((S, EP), torch.uint8, 9)
    ok(B.rmx_quant_f8(B.make_rows(n, C, dt), fmt, rows, q, e))
    for beside in (True, False):
        q2, e2, out = full_of((S, P), torch.uint8, 9), full_of((S, EP), torch.uint8, 9), full_of((S, C), dt, 0.0)
        ok(B.rmx_expert_gather(r, dev(src), x, out if beside else None, fmt, q2, e2))
        assert torch.equal(q, q2) and torch.equal(e, e2)
        assert not beside or torch.equal(out, rows)


@pytest.mark.parametrize("T,k,E", [(500, 2, 40), (9000, 2, 64), (40000, 2, 64)])
def test_sort_in_a_graph(T, k, E):
    """One CTA, a cluster and three launches, captured and replayed with other experts."""
    r = B.make_routes(T, k, E, 1, "f32")
    nws = B.rmx_expert_sort_workspace_bytes(r)
    ids, off, pos, src = (empty(n, torch.int32) for n in ((T, k), (E + 1,), (T, k), (T * k,)))
    ws, st = empty((nws,), torch.uint8), torch.cuda.Stream()
    ids.random_(0, E)
    ok(B.rmx_expert_sort(r, ids, off, pos, src, ws, nws, st))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        ok(B.rmx_expert_sort(r, ids, off, pos, src, ws, nws, st))
    for _ in range(2):
        ids.random_(-1, E)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            g.replay()
        torch.cuda.synchronize()
        for a, b in zip((off, pos, src), O.expert_sort(ids.cpu().numpy(), E)):
            assert np.array_equal(a.cpu().numpy(), b)
