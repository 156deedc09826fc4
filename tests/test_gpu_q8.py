"""The 8-bit operators on the GPU against their float64 definitions."""

import numpy as np
import pytest
import torch

from ffn_block_gb300 import binding as B
from oracle import q8_oracle as Q

from q8_util import DT, E32, TINY, U, dev, empty, f64, ok, rnd, sync, within

pytestmark = pytest.mark.gpu
EPS = 1e-5

ROW_SHAPES = [(1, 1), (1, 1280), (3, 8), (5, 31), (4, 33), (7, 100), (300, 64), (9, 513), (65, 1280), (11, 1281),
              (6, 2048), (5, 3001), (3, 4096), (2, 8192), (3, 8200), (2, 16384)]
# both sides of every change of threads a row, odd and even
ROW_SHAPES += [(37, 40), (37, 41), (33, 65), (33, 72), (35, 127), (35, 128), (19, 129), (19, 256), (17, 257), (17, 264),
               (9, 512), (9, 520), (5, 1272), (5, 1288), (3, 4097), (3, 4104), (3, 8193)]


def rms_data(R, C, dt, seed=0):
    rng = np.random.default_rng(seed)
    x, r = rnd(rng.standard_normal((R, C)), dt), rnd(rng.standard_normal((R, C)), dt)
    return x, r, rnd(1 + 0.3 * rng.standard_normal(C), dt), rng


def run_rms(x, r, g, dt, want=("h", "y", "q", "rstd"), stream=None):
    R, C = x.shape
    P = Q.pitch(C)
    o = dict(h=empty((R, C), dt) if "h" in want else None, y=empty((R, C), dt) if "y" in want else None,
             q=torch.full((R, P), 77, dtype=torch.int8, device="cuda") if "q" in want else None,
             scale=empty(R, torch.float32) if "q" in want else None,
             rstd=empty(R, torch.float32) if "rstd" in want else None)
    ok(B.rmx_rms_norm_q8(B.make_rows(R, C, dt), EPS, dev(x, dt), None if r is None else dev(r, dt), dev(g, dt),
                         o["h"], o["y"], o["q"], o["scale"], o["rstd"], stream))
    sync()
    return o


def check_rms(o, x, r, g, dt):
    h, rstd, n = Q.rms_norm(x, r, g, EPS)
    C = x.shape[1]
    # mean square: C float32 squares and sums (of one sign: relative), halved by
    # the root; the sum h itself (one rounding); rsqrt (2 ulp); three products.
    # At most 8 * 16 terms are summed in one thread and 5 + 16 more levels join them.
    rel = (160 / 2 + 10) * E32
    if o["h"] is not None:
        within(f64(o["h"]), h, np.abs(h) * (U[dt] + 2 * E32) + TINY[dt], "h")
    if o["rstd"] is not None:
        within(f64(o["rstd"]), rstd, rstd * rel, "rstd")
    if o["y"] is not None:
        within(f64(o["y"]), n, np.abs(n) * (U[dt] + rel) + TINY[dt], "y")
    if o["q"] is not None:
        top = np.max(np.abs(n), axis=1)
        within(f64(o["scale"]), top / 127, top / 127 * rel, "scale")
        q = f64(o["q"])
        assert np.all(q[:, C:] == 0) and np.all(np.abs(q) <= 127)
        step = top / 127
        # half a step from the rounding to integers, and the float32 error of n and of the scale
        within(q[:, :C] * f64(o["scale"])[:, None], n, (step * (0.5 + 127 * 2 * rel))[:, None], "values")


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("R,C", ROW_SHAPES)
def test_rms_norm_q8(R, C, dt):
    x, r, g, _ = rms_data(R, C, dt, R + C)
    check_rms(run_rms(x, r, g, dt), x, r, g, dt)
    check_rms(run_rms(x, None, g, dt, ("q",)), x, None, g, dt)
    check_rms(run_rms(x, None, g, dt, ("y",)), x, None, g, dt)


def test_rms_norm_many_rows():
    x, r, g, _ = rms_data(40_000, 40, "bf16")
    check_rms(run_rms(x, r, g, "bf16"), x, r, g, "bf16")


def test_rms_norm_in_place_sum():
    x, r, g, _ = rms_data(50, 200, "f16")
    for over in (0, 1):
        tx, tr, tg = dev(x, "f16"), dev(r, "f16"), dev(g, "f16")
        y = empty((50, 200), "f16")
        h = (tx, tr)[over]
        ok(B.rmx_rms_norm_q8(B.make_rows(50, 200, "f16"), EPS, tx, tr, tg, h, y, None, None, None))
        sync()
        check_rms(dict(h=h, y=y, q=None, rstd=None), x, r, g, "f16")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rms_norm_special_rows(dt):
    """Zero rows, rows with an infinity or a NaN, rows of tiny and of large values."""
    C = 70
    x, _, g, _ = rms_data(7, C, dt)
    x[0] = 0
    x[1, 3] = np.inf
    x[2, 69] = np.nan
    x[3] = rnd(x[3] * 1e-30, dt)
    x[4] = rnd(x[4] * 1e15, dt)
    o = run_rms(x, None, g, dt, ("y", "q", "rstd"))
    q, s = f64(o["q"]), f64(o["scale"])
    assert s[0] == 0 and not q[0].any() and np.all(f64(o["y"])[0] == 0)
    for r in (1, 2):
        assert np.isnan(s[r]) and not q[r].any()
    assert np.isnan(f64(o["y"])[2]).all()
    fine = [0, 3, 4, 5, 6]
    keep = lambda t: None if t is None else t[fine]
    check_rms(dict(h=None, y=keep(o["y"]), q=keep(o["q"]), scale=keep(o["scale"]), rstd=keep(o["rstd"])), x[fine], None, g, dt)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("R,C", [(1, 1), (5, 33), (64, 1280), (3, 2500), (2, 16384)])
def test_quant_and_dequant_rows(R, C, dt):
    rng = np.random.default_rng(R + C)
    x = rnd(rng.standard_normal((R, C)) * np.exp(3 * rng.standard_normal((R, 1))), dt)
    if R > 3:
        x[1], x[2, 0] = 0, np.inf
    P = Q.pitch(C)
    q, s, v = empty((R, P), torch.int8), empty(R, torch.float32), empty((R, C), dt)
    sh = B.make_rows(R, C, dt)
    ok(B.rmx_quant_rows_q8(sh, dev(x, dt), q, s))
    ok(B.rmx_dequant_rows_q8(sh, q, s, v))
    sync()
    _, rs = Q.quant_rows(x)
    within(f64(s), rs, np.nan_to_num(rs) * 2 * E32 + 2.0 ** -149, "scale")
    assert np.all(f64(q)[:, C:] == 0)
    got = f64(q)[:, :C] * f64(s)[:, None]
    fine = np.isfinite(rs)
    within(got[fine], x[fine], (rs[fine] * (0.5 + 127 * 6 * E32))[:, None], "values")
    within(f64(v), got, np.nan_to_num(np.abs(got)) * (U[dt] + E32) + TINY[dt], "read back")
    assert np.isnan(f64(v)[~fine]).all()


# ------------------------------------------------------------------ RMS norm backward

@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("ck", [True, False], ids=["checkpoint", "stored"])
@pytest.mark.parametrize("R,C", ROW_SHAPES + [(5000, 96), (1300, 1280)])
def test_rms_norm_backward(R, C, ck, dt):
    rng = np.random.default_rng(R * 3 + C)
    h = rnd(rng.standard_normal((R, C)), dt)
    g, dn = rnd(1 + 0.3 * rng.standard_normal(C), dt), rnd(rng.standard_normal((R, C)), dt)
    dh = rnd(rng.standard_normal((R, C)), dt) if C % 2 else None
    q, e = Q.ckpt_pack(h, dt) if R * C < 200_000 else Q_fast_pack(h, dt)
    hv = Q.ckpt_values(q, e, C) if ck else h
    rstd = np.float32(1 / np.sqrt(np.mean(h * h, -1) + EPS)).astype(np.float64)
    sh = B.make_rows(R, C, dt)
    nb = B.rmx_rms_norm_backward_workspace_bytes(sh)
    ws = torch.full((nb,), 0x7F, dtype=torch.uint8, device="cuda")
    dx, dg = empty((R, C), dt), empty(C, dt)
    ok(B.rmx_rms_norm_backward(sh, dev(dn, dt), None if dh is None else dev(dh, dt), None if ck else dev(h, dt),
                               dev(q) if ck else None, dev(e) if ck else None, dev(rstd.astype(np.float32)),
                               dev(g, dt), dx, dg, ws, nb))
    sync()
    rdx, rdg = Q.rms_norm_backward(hv, rstd, g, dn, dh)
    xh = hv * rstd[:, None]
    t = dn * g
    # the mean of C products, three roundings a term and the sum's own
    dot = np.mean(np.abs(t * xh), -1, keepdims=True)
    err = rstd[:, None] * (4 * np.abs(t) + np.abs(xh) * dot * (8 + 160)) * E32
    if dh is not None:
        err = err + np.abs(rdx) * 2 * E32
    within(f64(dx), rdx, np.abs(rdx) * U[dt] + err * (1 + U[dt]) + TINY[dt], "dx")
    # column sums over R rows in a fixed order: at most R additions
    mag = np.sum(np.abs(dn * xh), 0)
    within(f64(dg), rdg, np.abs(rdg) * U[dt] + mag * min(R + 6, 700) * E32 * (1 + U[dt]) + TINY[dt], "dgamma")


def Q_fast_pack(x, dt):
    """The same checkpoint by whole arrays (checked against the definition on its first rows)."""
    R, C = x.shape
    lo, hi = Q.EXP_RANGE[dt]
    p = np.zeros((R, Q.pitch(C)))
    p[:, :C] = x
    grp = p.reshape(R, -1, 32)
    top = np.abs(grp).max(-1)
    m, k = np.frexp(top)
    e = np.where(top > 0, np.clip(k - 7 + (m > 127.5 / 128), lo, hi), lo)
    q = np.clip(np.rint(grp / 2.0 ** e[..., None].astype(float)), -127, 127).reshape(R, -1).astype(np.int8)
    q0, e0 = Q.ckpt_pack(x[:4], dt)
    assert np.array_equal(q[:4], q0) and np.array_equal(e[:4], e0)
    return q, e.astype(np.int8)


def test_rms_norm_backward_in_place_and_empty():
    R, C, dt = 37, 136, "bf16"
    rng = np.random.default_rng(1)
    h, dn, dh = (rnd(rng.standard_normal((R, C)), dt) for _ in range(3))
    g = rnd(1 + 0.3 * rng.standard_normal(C), dt)
    rstd = (1 / np.sqrt(np.mean(h * h, -1) + EPS)).astype(np.float32)
    sh = B.make_rows(R, C, dt)
    nb = B.rmx_rms_norm_backward_workspace_bytes(sh)
    ws = empty(nb, torch.uint8)
    outs = []
    for over in (None, 0, 1):
        tn, th = dev(dn, dt), dev(dh, dt)
        dx = empty((R, C), dt) if over is None else (tn, th)[over]
        dg = empty(C, dt)
        ok(B.rmx_rms_norm_backward(sh, tn, th, dev(h, dt), None, None, dev(rstd), dev(g, dt), dx, dg, ws, nb))
        sync()
        outs.append((dx, dg))
    for dx, dg in outs[1:]:
        assert torch.equal(dx, outs[0][0]) and torch.equal(dg, outs[0][1])
    dg = torch.full((C,), 3.0, dtype=DT[dt], device="cuda")
    ok(B.rmx_rms_norm_backward(B.make_rows(0, C, dt), None, None, None, None, None, None, None, None, dg, None, 0))
    sync()
    assert not dg.any()


# ------------------------------------------------------------------ checkpoints

@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("R,C", [(1, 1), (1, 8), (3, 31), (4, 33), (17, 96), (9, 513), (33, 1280), (2, 20001), (41, 40),
                                 (41, 41), (33, 100), (33, 127), (19, 130), (7, 1000), (8, 32), (3, 256), (65, 64),
                                 (6, 4000), (300, 1)])
def test_checkpoint_is_the_definition(R, C, dt):
    rng = np.random.default_rng(R + C)
    x = rnd(rng.standard_normal((R, C)) * np.exp(2 * rng.standard_normal((R, C))), dt)
    if C > 8:
        x[0, :8] = 0
    P = Q.pitch(C)
    q = torch.full((R, P), 55, dtype=torch.int8, device="cuda")
    e, v = empty((R, P // 32), torch.int8), empty((R, C), dt)
    sh = B.make_rows(R, C, dt)
    ok(B.rmx_ckpt8_pack(sh, dev(x, dt), q, e))
    ok(B.rmx_ckpt8_unpack(sh, q, e, v))
    sync()
    rq, re = Q.ckpt_pack(x, dt)
    assert np.array_equal(e.cpu().numpy(), re)
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(f64(v), Q.ckpt_values(rq, re, C))   # exact in the storage type


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_checkpoint_special_groups(dt):
    fi = torch.finfo(DT[dt])
    tiny = TINY[dt]
    x = np.zeros((8, 64))
    x[0, :] = fi.max
    x[1, 5], x[1, 40] = np.inf, 1.0
    x[2, 31], x[2, 32] = np.nan, -1.0
    x[3, :] = tiny
    x[4, :] = 127.5
    x[5, 0] = -fi.max
    x[6, 63] = fi.tiny
    x = rnd(x, dt)
    q, e, v = empty((8, 64), torch.int8), empty((8, 2), torch.int8), empty((8, 64), dt)
    sh = B.make_rows(8, 64, dt)
    ok(B.rmx_ckpt8_pack(sh, dev(x, dt), q, e))
    ok(B.rmx_ckpt8_unpack(sh, q, e, v))
    sync()
    rq, re = Q.ckpt_pack(x, dt)
    assert np.array_equal(e.cpu().numpy(), re) and np.array_equal(q.cpu().numpy(), rq)
    rv = Q.ckpt_values(rq, re, 64)
    got = f64(v)
    assert np.array_equal(np.isnan(got), np.isnan(rv)) and np.array_equal(got[~np.isnan(rv)], rv[~np.isnan(rv)])
    assert np.isnan(got[1, :32]).all() and got[1, 40] == 1.0 and np.isnan(got[2, :32]).all() and got[2, 32] == -1.0


# ------------------------------------------------------------------ int8 product

def linear_data(M, G, K, N, dt, seed, bias=True, resid=False):
    rng = np.random.default_rng(seed)
    P = Q.pitch(K)
    a, w = np.zeros((M, G, P), np.int8), np.zeros((G, N, P), np.int8)
    a[..., :K] = rng.integers(-127, 128, (M, G, K))
    w[..., :K] = rng.integers(-127, 128, (G, N, K))
    sa = rng.uniform(0.01, 0.03, (M, G)).astype(np.float32)
    sw = (rng.uniform(0.5, 1.5, (G, N)) / (127 * np.sqrt(K))).astype(np.float32)
    b = rnd(rng.standard_normal((G, N)), dt) if bias else None
    r = rnd(rng.standard_normal((M, G, N)), dt) if resid else None
    return a, sa, w, sw, b, r


def run_linear(a, sa, w, sw, b, r, K, dt, out=None, stream=None):
    M, G, _ = a.shape
    N = w.shape[1]
    out = empty((M, G, N), dt) if out is None else out
    ok(B.rmx_linear_q8(B.make_layer(M, G, K, N, dt), dev(a), dev(sa), dev(w), dev(sw),
                       None if b is None else dev(b, dt), None if r is None else dev(r, dt), out, stream))
    sync()
    return out


def check_linear(out, a, sa, w, sw, b, r, K, dt):
    d = lambda t: None if t is None else t.astype(np.float64)
    ref = Q.linear_q8(a, d(sa), w, d(sw), b, r, K)
    prod = np.abs(Q.linear_q8(a, d(sa), w, d(sw), None, None, K))
    # integer sums below 2^24 are exact; two products and two sums follow in float32
    terms = prod + (np.abs(b) if b is not None else 0) + (np.abs(r) if r is not None else 0)
    within(f64(out), ref, np.abs(ref) * U[dt] + terms * 5 * E32 * (1 + U[dt]) + TINY[dt], "out")


LIN_SHAPES = [(1, 1, 1, 1), (1, 3, 64, 32), (2, 1, 31, 17), (5, 2, 33, 65), (8, 4, 250, 123), (17, 3, 1280, 640),
              (33, 2, 96, 300), (64, 5, 200, 129), (100, 1, 513, 257), (128, 2, 128, 256), (129, 2, 64, 520),
              (200, 3, 320, 384), (256, 1, 1000, 512), (300, 2, 72, 40), (1, 2, 4100, 1000), (700, 1, 416, 771)]
# both sides of a CTA alone and a pair, of one token tile and two; more tiles than SMs; few k
LIN_SHAPES += [(96, 1, 130, 129), (97, 1, 70, 128), (97, 2, 70, 129), (192, 1, 128, 256), (193, 1, 129, 257),
               (16, 3, 127, 33), (32, 1, 257, 140), (385, 1, 64, 600), (3, 200, 40, 140), (130, 90, 33, 300)]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,G,K,N", LIN_SHAPES)
def test_linear_q8(M, G, K, N, dt):
    bias, resid = (M + N) % 3 != 0, (M + K) % 2 == 0
    data = linear_data(M, G, K, N, dt, M + K + N, bias, resid)
    check_linear(run_linear(*data, K, dt), *data, K, dt)


# Few tiles of a long K: one, two and four CTAs to a tile, on both sides of each rule (steps of 128 columns,
# tiles); one token, whole and ragged tiles of them; more than one token tile of few channels.
SPLIT_SHAPES = [(1, 1, 1000, 128), (1, 1, 896, 128), (1, 1, 1281, 5120), (1, 1, 1280, 5120), (2, 1, 2023, 300),
                (7, 21, 1504, 96), (96, 1, 1153, 130), (96, 2, 1152, 128), (95, 18, 2048, 128), (33, 19, 2048, 100),
                (16, 36, 1030, 128), (17, 37, 1630, 120), (64, 72, 2060, 64), (96, 40, 2305, 60), (1, 73, 1520, 64),
                (300, 2, 2100, 128), (21, 3, 3104, 48), (1, 1, 3840, 2570), (50, 1, 40000, 200)]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,G,K,N", SPLIT_SHAPES)
def test_linear_q8_few_tiles(M, G, K, N, dt):
    bias, resid = (M + N) % 3 != 0, (M + K) % 2 == 0
    data = linear_data(M, G, K, N, dt, 2 * M + K + N, bias, resid)
    out = run_linear(*data, K, dt)
    check_linear(out, *data, K, dt)
    assert torch.equal(out, run_linear(*data, K, dt))
    # A token without a scale: its row only.
    data[1][M // 2, 0] = np.nan
    bad = run_linear(*data, K, dt)
    assert torch.isnan(bad[M // 2, 0]).all()
    keep = torch.ones((M, G), dtype=torch.bool, device=bad.device)
    keep[M // 2, 0] = False
    assert torch.equal(bad[keep], out[keep])


# Pairs of CTAs: more tiles of up to 96 tokens and 128 channels than SMs (one fewer, one more), one token tile of
# a pair and two, ragged ends of all three.
PAIR_SHAPES = [(97, 38, 64, 256), (97, 39, 64, 256), (97, 60, 70, 129), (112, 80, 33, 200), (192, 80, 128, 256), (193, 40, 129, 257),
               (200, 18, 320, 384), (256, 13, 1000, 512), (385, 20, 64, 600), (700, 3, 416, 771), (1024, 4, 130, 640),
               (300, 25, 4100, 200), (128, 150, 40, 130)]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,G,K,N", PAIR_SHAPES + [(706, 2, 2979, 214), (129, 1, 1100, 257), (385, 9, 1000, 256)])
def test_linear_q8_many_tokens(M, G, K, N, dt):
    bias, resid = (M + G) % 3 != 0, (M + K) % 2 == 0
    data = linear_data(M, G, K, N, dt, M + 3 * K + N, bias, resid)
    check_linear(run_linear(*data, K, dt), *data, K, dt)


def test_linear_q8_few_tiles_in_place_in_a_graph_and_beside_another():
    M, G, K, N, dt = 90, 3, 2100, 400, "bf16"
    data = linear_data(M, G, K, N, dt, 11, True, True)
    ref = run_linear(*data, K, dt)
    args = [dev(t) for t in data[:4]] + [dev(data[4], dt)]
    first = dev(data[5], dt)
    bufs = [first.clone(), first.clone()]
    layer = B.make_layer(M, G, K, N, dt)
    graphs = []
    for buf in bufs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            ok(B.rmx_linear_q8(layer, *args, buf, buf, torch.cuda.current_stream()))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for buf, g, st in zip(bufs, graphs, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                buf.copy_(first)
                g.replay()
    sync()
    assert all(torch.equal(buf, ref) for buf in bufs)


def test_linear_q8_lowest_int8_and_padding():
    """-128 is allowed, and columns past K count for nothing where one operand has zeros there."""
    M, G, K, N = 20, 2, 50, 70
    a, sa, w, sw, b, r = linear_data(M, G, K, N, "f32", 4)
    a[..., :K], w[:, ::2, :K] = -128, -128
    a[..., K:] = 99
    data = (a, sa, w, sw, b, r)
    check_linear(run_linear(*data, K, "f32"), *data, K, "f32")


def test_linear_q8_sums_past_24_bits():
    """Largest sums: every partial sum is rounded to at most 24 bits, by 2^-24 of it at each of K / 16 steps."""
    M, G, K, N = 9, 1, 4096, 33
    a, sa, w, sw, _, _ = linear_data(M, G, K, N, "f32", 5)
    a[..., :K], w[..., :K] = 127, 127
    w[:, ::3] = -127
    w[:, 1::3, ::2] = 126
    out = f64(run_linear(a, sa, w, sw, None, None, K, "f32"))
    ref = Q.linear_q8(a, sa.astype(float), w, sw.astype(float), None, None, K)
    within(out, ref, np.abs(ref) * (K / 16 * 2 * E32 + 5 * E32), "out")


def test_linear_q8_residual_in_place():
    M, G, K, N, dt = 150, 2, 96, 136, "bf16"
    data = linear_data(M, G, K, N, dt, 8, True, True)
    ref = run_linear(*data, K, dt)
    buf = dev(data[5], dt)
    ok(B.rmx_linear_q8(B.make_layer(M, G, K, N, dt), *[dev(t) for t in data[:4]], dev(data[4], dt), buf, buf))
    sync()
    assert torch.equal(buf, ref)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("G,K,N", [(1, 1, 1), (2, 33, 31), (3, 100, 65), (2, 256, 96)])
def test_weight_q8(G, K, N, dt):
    rng = np.random.default_rng(K + N)
    w = rnd(rng.standard_normal((G, K, N)) * np.exp(rng.standard_normal((G, 1, N))), dt)
    if N > 30:
        w[0, :, 3] = 0
        w[0, K // 2, 5] = np.nan
    P = Q.pitch(K)
    q, s = torch.full((G, N, P), 9, dtype=torch.int8, device="cuda"), empty((G, N), torch.float32)
    ok(B.rmx_weight_q8(B.make_layer(1, G, K, N, dt), dev(w, dt), q, s))
    sync()
    rq, rs = Q.weight_q8(w)
    within(f64(s), rs, np.nan_to_num(rs) * 2 * E32, "scale")
    assert np.all(f64(q)[..., K:] == 0)
    got = f64(q)[..., :K] * f64(s)[..., None]
    fine = np.isfinite(rs)
    within(got[fine], np.swapaxes(w, 1, 2)[fine], (rs[fine] * (0.5 + 127 * 6 * E32))[:, None], "values")
    assert np.isnan(f64(s)[~fine]).all() and not f64(q)[~fine].any()


# ------------------------------------------------------------------ weight gradient

@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,G,K,N", [(1, 1, 1, 1), (1, 2, 64, 64), (3, 2, 33, 17), (64, 3, 128, 256), (129, 2, 96, 72),
                                     (200, 1, 81, 243), (77, 4, 40, 130), (300, 2, 256, 512), (513, 1, 136, 264)])
def test_ckpt8_wgrad(M, G, K, N, dt):
    rng = np.random.default_rng(M + K)
    q, e = Q.ckpt_pack(rnd(rng.standard_normal((M * G, K)), dt), dt)
    x = Q.ckpt_values(q, e, K).reshape(M, G, K)
    dy = rnd(rng.standard_normal((M, G, N)), dt)
    l = B.make_layer(M, G, K, N, dt)
    nb = B.rmx_ckpt8_wgrad_workspace_bytes(l)
    dw, db = empty((G, K, N), dt), empty((G, N), dt)
    ws = torch.full((nb,), 0x7F, dtype=torch.uint8, device="cuda")
    ok(B.rmx_ckpt8_wgrad(l, dev(q), dev(e), dev(dy, dt), dw, db, ws, nb))
    sync()
    rw, rb = Q.wgrad(x, dy)
    mw, mb = Q.wgrad(np.abs(x), np.abs(dy))
    # 16-bit products are exact in float32, so only the sums of M terms round;
    # a tensor-core step may drop bits below 2^-23 of its largest partial.
    within(f64(dw), rw, np.abs(rw) * U[dt] + mw * (2 * M + 4) * E32 + TINY[dt], "dw")
    within(f64(db), rb, np.abs(rb) * U[dt] + mb * (M + 4) * E32 + TINY[dt], "db")
    dw2 = empty((G, K, N), dt)
    ok(B.rmx_ckpt8_wgrad(l, dev(q), dev(e), dev(dy, dt), dw2, None, ws, nb))
    sync()
    assert torch.equal(dw, dw2)


def test_ckpt8_wgrad_of_nothing_is_zero():
    l = B.make_layer(0, 2, 10, 12, "bf16")
    dw = torch.ones((2, 10, 12), dtype=torch.bfloat16, device="cuda")
    db = torch.ones((2, 12), dtype=torch.bfloat16, device="cuda")
    ok(B.rmx_ckpt8_wgrad(l, None, None, None, dw, db, None, 0))
    sync()
    assert not dw.any() and not db.any()
