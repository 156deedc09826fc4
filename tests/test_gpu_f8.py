"""8-bit floating rows and their products against the oracle."""

import numpy as np
import pytest
import torch

from ffn_block_gb300 import binding as B
from oracle import sparse_oracle as O
from tests.sparse_util import E32, F8, TINY, U, dev, empty, f64, f8_operand, f8_values, full_of, mma_bound, ok, rnd, sync, within

pytestmark = pytest.mark.gpu
FORMATS = ["e4m3", "e5m2"]


def _spread(rng, shape, dt):
    """Values over many magnitudes, zeros among them."""
    x = rng.standard_normal(shape) * np.exp2(rng.integers(-6, 7, shape[:-1] + (1,)).astype(float))
    x[rng.random(shape) < 0.05] = 0
    return rnd(x, dt)


def _check_rows(q, e, x, fmt, cols):
    vq, ve = O.quant_rows(x, fmt)
    KB = ve.shape[1]
    assert np.array_equal(e.cpu().numpy()[:, :KB], ve) and not e[:, KB:].any()
    assert np.array_equal(f8_values(q, fmt), vq)


# ------------------------------------------------------------------ rows
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("R,C", [(1, 1), (3, 7), (5, 64), (2, 128), (9, 129), (31, 136), (33, 513), (17, 1001), (40, 1280), (300, 640),
                                 (3, 5000)])
def test_quantised_rows(fmt, dt, R, C):
    rng = np.random.default_rng(R * C)
    x = _spread(rng, (R, C), dt)
    P, EP = B.rmx_f8_pitch(C), B.rmx_f8_exps(C)
    q, e = full_of((R, P), torch.uint8, 255), full_of((R, EP), torch.uint8, 255)
    shape = B.make_rows(R, C, dt)
    ok(B.rmx_quant_f8(shape, fmt, dev(x, dt), q, e))
    _check_rows(q, e, x, fmt, C)
    out = empty((R, C), dt)
    ok(B.rmx_dequant_f8(shape, fmt, q, e, out))
    ref = O.round_rows(x, fmt)
    within(f64(out), ref, U[dt] * np.abs(ref) * (dt == "f16") + TINY[dt] * (dt == "f16"))


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_value_reads_back(fmt):
    """All finite bytes under several exponents."""
    b = torch.arange(256, dtype=torch.uint8)
    b[~torch.isfinite(b.view(F8[fmt]).float())] = 0
    q = torch.cat([b[:128], b[128:]]).reshape(1, 256).repeat(5, 1)
    ex = torch.tensor([[0, 1, 0, 0], [127, 127, 0, 0], [130, 100, 0, 0], [239, 238, 0, 0], [255, 127, 0, 0]], dtype=torch.uint8)
    out = empty((5, 256), "f32")
    ok(B.rmx_dequant_f8(B.make_rows(5, 256, "f32"), fmt, q.cuda(), ex.cuda(), out))
    ref = O.row_values(q.view(F8[fmt]).double().numpy(), ex.numpy()[:, :2].astype(np.int64), 256)
    assert np.array_equal(f64(out), np.clip(ref, -np.finfo(np.float32).max, np.finfo(np.float32).max), equal_nan=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_the_ends_of_the_range(fmt, dt):
    """The largest and smallest numbers of the type, subnormals, ties, zeros, infinities and NaN."""
    big, tiny = torch.finfo({"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dt]).max, TINY[dt]
    x = np.zeros((8, 256))
    x[0, :3], x[0, 130] = (big, -big, big / 2), tiny
    x[1, 5], x[1, 200] = tiny, -3 * tiny
    x[2, :4] = O.LARGEST[fmt], -O.LARGEST[fmt], 17.0, 19.0
    x[3, 7], x[3, 255] = np.inf, 1.0
    x[4, 7], x[4, 128] = np.nan, -np.inf
    x[5, :] = np.linspace(-1, 1, 256)
    x[7, :2] = 1.0, 2.0 ** -14
    x = rnd(x, dt)
    q, e = full_of((8, 256), torch.uint8, 1), full_of((8, 4), torch.uint8, 1)
    shape = B.make_rows(8, 256, dt)
    ok(B.rmx_quant_f8(shape, fmt, dev(x, dt), q, e))
    _check_rows(q, e, x, fmt, 256)
    out = empty((8, 256), dt)
    ok(B.rmx_dequant_f8(shape, fmt, q, e, out))
    got, ref = f64(out), O.round_rows(x, fmt)
    assert np.all(np.isnan(got) == np.isnan(ref))
    fine = np.isfinite(ref)
    assert np.all(np.isfinite(got[fine]))
    within(got[fine], np.clip(ref[fine], -big, big), U[dt] * np.abs(ref[fine]) * (dt == "f16") + TINY[dt] / 2)


# ------------------------------------------------------------------ rows and columns
def _layout(order, M, G, C):
    return {"tokens": (M, G, C), "groups": (G, M, C), "ragged": (M, C)}[order]


def _sizes(rng, M, G):
    share = rng.random(G) * (rng.random(G) < 0.8)
    s = rng.multinomial(M, share / share.sum()) if share.sum() else np.zeros(G, int)
    return np.concatenate([[0], np.cumsum(s)])


@pytest.mark.parametrize("order", ["tokens", "groups", "ragged"])
@pytest.mark.parametrize("dt,fmt", [("bf16", "e4m3"), ("f16", "e5m2"), ("f32", "e4m3")])
@pytest.mark.parametrize("M,G,C", [(1, 1, 1), (5, 3, 7), (128, 2, 128), (129, 2, 136), (300, 4, 264), (77, 5, 1001), (260, 1, 130),
                                   (1000, 7, 72)])
def test_rows_and_columns(order, dt, fmt, M, G, C):
    rng = np.random.default_rng(M + C)
    x = _spread(rng, _layout(order, M, G, C), dt)
    off = _sizes(rng, M, G) if order == "ragged" else None
    if order == "ragged" and M > 10:
        off[-1] = max(off[-2], off[-1] - 3)                  # some rows belong to nobody
    gr = B.make_groups(M, G, C, dt, order)
    P, EP = B.rmx_f8_pitch(C), B.rmx_f8_exps(C)
    lead = x.shape[:-1]
    ragged = order == "ragged"
    TP = B.rmx_f8_ragged_pitch(M, G) if ragged else B.rmx_f8_pitch(M)
    TE = (TP // 128 + 3) // 4 * 4 if ragged else B.rmx_f8_exps(M)
    new = lambda: (full_of((*lead, P), torch.uint8, 7), full_of((*lead, EP), torch.uint8, 7),  # noqa: E731
                   full_of(((C, TP) if ragged else (G, C, TP)), torch.uint8, 7),
                   full_of(((C, TE) if ragged else (G, C, TE)), torch.uint8, 7), full_of((G, C), dt, 7.0))
    nws = B.rmx_quant_f8_groups_workspace_bytes(gr)
    ws = full_of((nws,), torch.uint8, 255)
    q, e, qt, et, sums = new()
    dx, doff = dev(x, dt), dev(off.astype(np.int32)) if ragged else None
    ok(B.rmx_quant_f8_groups(gr, fmt, doff, dx, q, e, qt, et, sums, ws, nws))
    # rows: as from rmx_quant_f8
    n = off[-1] if ragged else int(np.prod(lead))
    flat = x.reshape(-1, C)
    _check_rows(q.reshape(-1, P)[:n], e.reshape(-1, EP)[:n], flat[:n], fmt, C)
    assert torch.all(q.reshape(-1, P)[n:] == 7) and torch.all(e.reshape(-1, EP)[n:] == 7)
    kb = 0
    for g in range(G):
        xg = x[off[g] : off[g + 1]] if ragged else x[:, g] if order == "tokens" else x[g]
        within(f64(sums[g]), xg.sum(0), 136 * E32 * np.abs(xg).sum(0) + U[dt] * np.abs(xg.sum(0)) + TINY[dt], "sums")
        nb = -(-xg.shape[0] // 128)
        if ragged:
            if nb:
                vq, ve = O.quant_rows(xg.T, fmt)
                got = qt.reshape(TP // 128, C, 128)[kb : kb + nb].transpose(0, 1).reshape(C, nb * 128).contiguous()
                assert np.array_equal(f8_values(got, fmt), vq)
                assert np.array_equal(et.reshape(-1, C, 4).transpose(0, 1).reshape(C, TE).cpu().numpy()[:, kb : kb + nb], ve)
            kb += nb
        else:
            _check_rows(qt[g], et[g], xg.T, fmt, M)
    if ragged:
        assert torch.all(qt.reshape(TP // 128, C, 128)[kb:] == 7) and torch.all(et.reshape(-1, C, 4).transpose(0, 1).reshape(C, TE)[:, kb:] == 7)
    # each by itself is the same
    a, b = new(), new()
    ok(B.rmx_quant_f8_groups(gr, fmt, doff, dx, a[0], a[1], None, None, None, None, 0))
    ok(B.rmx_quant_f8_groups(gr, fmt, doff, dx, None, None, a[2], a[3], None, None, 0))
    ok(B.rmx_quant_f8_groups(gr, fmt, doff, dx, None, None, None, None, a[4], ws, nws))
    assert all(torch.equal(u, v) for u, v in zip(a, (q, e, qt, et, sums)))
    assert all(torch.all(v == 7) for v in b)


def test_groups_without_rows():
    sums = full_of((3, 40), "bf16", 5.0)
    for order, off in (("tokens", None), ("ragged", torch.zeros(4, dtype=torch.int32, device="cuda"))):
        sums.fill_(5.0)
        gr = B.make_groups(0, 3, 40, "bf16", order)
        ok(B.rmx_quant_f8_groups(gr, "e4m3", off, None, None, None, None, None, sums, None, 0))
        assert not sums.any()
    # experts of which none has rows
    gr = B.make_groups(50, 3, 40, "bf16", "ragged")
    nws = B.rmx_quant_f8_groups_workspace_bytes(gr)
    x, sums = full_of((50, 40), "bf16", 1.0), full_of((3, 40), "bf16", 5.0)
    off = torch.full((4,), 20, dtype=torch.int32, device="cuda")
    ok(B.rmx_quant_f8_groups(gr, "e4m3", off, x, None, None, None, None, sums, empty((nws,), torch.uint8), nws))
    assert not sums.any()


@pytest.mark.parametrize("bad", [[-5, 10, 20, 30], [0, 20, 10, 30], [0, 10, 1000, 2000], [0, (1 << 31) - 1, -(1 << 31), 5]])
def test_offsets_out_of_order_are_taken_as_the_nearest(bad):
    M, G, C = 40, 3, 72
    rng = np.random.default_rng(0)
    x = _spread(rng, (M, C), "f32")
    good = np.clip(np.maximum.accumulate(np.array(bad, np.int64)), 0, M)
    outs = []
    for off in (bad, good):
        off = torch.from_numpy(np.array(off, np.int64).astype(np.int32)).cuda()
        gr = B.make_groups(M, G, C, "f32", "ragged")
        nws = B.rmx_quant_f8_groups_workspace_bytes(gr)
        TP = B.rmx_f8_ragged_pitch(M, G)
        o = (full_of((M, 128), torch.uint8, 1), full_of((M, 4), torch.uint8, 1), full_of((C, TP), torch.uint8, 1),
             full_of((C, (TP // 128 + 3) // 4 * 4), torch.uint8, 1), empty((G, C), "f32"))
        ok(B.rmx_quant_f8_groups(gr, "e4m3", off, dev(x, "f32"), *o, empty((nws,), torch.uint8), nws))
        w, we = f8_operand(np.random.default_rng(1), G * 24, C, "e4m3")[1:]
        out, dw = full_of((M, 24), "f32", 2.0), full_of((G, C, C), "f32", 2.0)
        ok(B.rmx_linear_f8(B.make_layer_f8(M, G, C, 24, "f32"), off, o[0], o[1], w, we, None, None, out))
        ok(B.rmx_wgrad_f8(B.make_layer_f8(M, G, C, C, "f32"), off, o[2], o[3], o[2], o[3], dw))
        outs.append((*o, out, dw))
    sync()
    assert all(torch.equal(a, b) for a, b in zip(*outs))


# ------------------------------------------------------------------ the product
def _product(M, G, K, N, dt, af, bf, bias=True, resid=False, seed=0, spread=2):
    rng = np.random.default_rng(seed + M + 7 * K + 13 * N)
    a, qa, ea = f8_operand(rng, M * G, K, af, spread)
    w, qw, ew = f8_operand(rng, G * N, K, bf, spread)
    a, w = a.reshape(M, G, K), w.reshape(G, N, K)
    scale = np.sqrt(K) * np.abs(a).mean() * np.abs(w).mean()
    b = rnd(rng.standard_normal((G, N)) * scale, dt) if bias else None
    r = rnd(rng.standard_normal((M, G, N)) * scale, dt) if resid else None
    out = full_of((M, G, N), dt, float("nan"))
    ok(B.rmx_linear_f8(B.make_layer_f8(M, G, K, N, dt, af, bf), None, qa, ea, qw, ew, dev(b, dt) if bias else None,
                       dev(r, dt) if resid else None, out))
    sync()
    got = f64(out)
    for g in range(G):
        ref = a[:, g] @ w[g].T + (b[g] if bias else 0.0) + (r[:, g] if resid else 0.0)
        extra = 2 * E32 * (np.abs(ref) + (np.abs(b[g]) if bias else 0.0) + (np.abs(r[:, g]) if resid else 0.0))
        within(got[:, g], ref, mma_bound(a[:, g], w[g], K, dt, ref) + extra, f"group {g}")


def test_product_one_tile():
    _product(16, 1, 128, 128, "f32", "e4m3", "e4m3", bias=False, spread=0)


def test_product_exponents():
    _product(32, 1, 128, 128, "f32", "e4m3", "e4m3", bias=False, spread=6)
    _product(200, 1, 640, 128, "f32", "e4m3", "e4m3", bias=False, spread=6)


# one token to several tiles, one block of k to many, odd everything
@pytest.mark.parametrize("M,G,K,N", [(1, 1, 1, 1), (1, 1, 128, 128), (3, 2, 40, 24), (16, 1, 512, 64), (17, 3, 513, 130), (5, 2, 1280, 256),
                                     (100, 2, 300, 200), (128, 1, 1001, 333), (129, 2, 256, 129), (224, 1, 384, 128), (225, 1, 384, 128),
                                     (500, 3, 129, 257), (64, 5, 2000, 1)])
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_product(M, G, K, N, dt):
    _product(M, G, K, N, dt, "e4m3", "e4m3")


@pytest.mark.parametrize("af", FORMATS)
@pytest.mark.parametrize("bf", FORMATS)
def test_product_formats(af, bf):
    _product(70, 2, 700, 190, "f32", af, bf, bias=False)


@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("resid", [True, False])
def test_product_epilogues(bias, resid):
    _product(45, 2, 300, 140, "bf16", "e4m3", "e4m3", bias, resid)
    _product(400, 40, 256, 512, "bf16", "e4m3", "e4m3", bias, resid)


@pytest.mark.parametrize("M,G,K,N,dt", [(300, 64, 640, 512, "bf16"), (1000, 40, 130, 300, "f16"), (448, 30, 1280, 1280, "f32"),
                                        (257, 20, 2049, 1030, "bf16")])
def test_product_of_pairs(M, G, K, N, dt):
    """Enough tiles that CTA pairs take them, several each."""
    _product(M, G, K, N, dt, "e4m3", "e5m2")


# both sides of the rules on sharing a tile: eight, four and two CTAs to one, uneven shares, residuals
@pytest.mark.parametrize("M,G,K,N", [(1, 1, 4096, 1920), (3, 1, 1100, 300), (7, 2, 4000, 900), (200, 1, 6000, 500), (30, 2, 2000, 2100),
                                     (9, 3, 4099, 1300), (16, 1, 1025, 130), (2, 4, 5000, 2200), (224, 1, 8200, 129)])
def test_product_of_shared_tiles(M, G, K, N):
    _product(M, G, K, N, "f32", "e4m3", "e5m2", bias=True, resid=True, spread=1)
    _product(M, G, K, N, "bf16", "e4m3", "e4m3", bias=False, spread=1)


def test_product_in_place_of_the_residual():
    rng = np.random.default_rng(3)
    M, G, K, N = 90, 2, 256, 136
    _, qa, ea = f8_operand(rng, M * G, K, "e4m3")
    _, qw, ew = f8_operand(rng, G * N, K, "e4m3")
    r = torch.randn((M, G, N), device="cuda").bfloat16()
    out, l = empty((M, G, N), "bf16"), B.make_layer_f8(M, G, K, N, "bf16")
    ok(B.rmx_linear_f8(l, None, qa, ea, qw, ew, None, r, out))
    ok(B.rmx_linear_f8(l, None, qa, ea, qw, ew, None, r, r))
    assert torch.equal(out, r)


def test_product_of_faulty_blocks():
    """A NaN block makes its row (or channel) NaN and no other."""
    rng = np.random.default_rng(4)
    M, K, N = 40, 384, 200
    a, qa, ea = f8_operand(rng, M, K, "e4m3")
    w, qw, ew = f8_operand(rng, N, K, "e4m3")
    ea[7, 1], ew[150, 2] = 255, 255
    out = empty((M, 1, N), "f32")
    ok(B.rmx_linear_f8(B.make_layer_f8(M, 1, K, N, "f32"), None, qa, ea, qw, ew, None, None, out))
    got = f64(out)[:, 0]
    bad = np.zeros((M, N), bool)
    bad[7], bad[:, 150] = True, True
    assert np.array_equal(np.isnan(got), bad)
    ref = a @ w.T
    within(got[~bad], ref[~bad], mma_bound(a, w, K, "f32", ref)[~bad])


@pytest.mark.parametrize("M,G,K,N,dt", [(1, 1, 64, 64, "f32"), (2, 8, 256, 128, "bf16"), (50, 3, 200, 130, "f32"), (128, 32, 512, 256, "bf16"),
                                        (700, 5, 384, 300, "f16"), (3000, 7, 256, 520, "bf16"), (9000, 40, 256, 640, "f32"),
                                        (513, 1024, 128, 40, "f32")])
def test_product_by_expert(M, G, K, N, dt):
    rng = np.random.default_rng(M)
    a, qa, ea = f8_operand(rng, M, K, "e4m3")
    w, qw, ew = f8_operand(rng, G * N, K, "e4m3")
    w = w.reshape(G, N, K)
    off = _sizes(rng, M, G)
    n = off[-1] = max(off[-2], off[-1] - (5 if M > 20 else 0))
    ea[n:], qa[n:] = 255, 0x7F                               # rows behind the last expert's: any bytes
    b = rnd(rng.standard_normal((G, N)) * 10, dt)
    r = rnd(rng.standard_normal((M, N)) * 10, dt)
    out = full_of((M, N), dt, 3.0)
    ok(B.rmx_linear_f8(B.make_layer_f8(M, G, K, N, dt), dev(off.astype(np.int32)), qa, ea, qw, ew, dev(b, dt), dev(r, dt), out))
    sync()
    got = f64(out)
    assert np.all(got[n:] == 3.0)
    for g in range(G):
        s = slice(off[g], off[g + 1])
        ref = a[s] @ w[g].T + b[g] + r[s]
        within(got[s], ref, mma_bound(a[s], w[g], K, dt, ref) + 2 * E32 * (np.abs(ref) + np.abs(b[g]) + np.abs(r[s])), f"expert {g}")


def test_product_by_expert_all_to_one():
    """More rows at one expert than its share."""
    M, G, K, N = 2000, 16, 256, 512
    rng = np.random.default_rng(0)
    a, qa, ea = f8_operand(rng, M, K, "e4m3")
    w, qw, ew = f8_operand(rng, G * N, K, "e4m3")
    off = np.array([0] * 6 + [M] * 11, np.int32)
    out = empty((M, N), "f32")
    ok(B.rmx_linear_f8(B.make_layer_f8(M, G, K, N, "f32"), dev(off), qa, ea, qw, ew, None, None, out))
    sync()
    ref = a @ w.reshape(G, N, K)[5].T
    within(f64(out), ref, mma_bound(a, w.reshape(G, N, K)[5], K, "f32", ref))


# ------------------------------------------------------------------ the weight gradient
@pytest.mark.parametrize("order", ["tokens", "ragged"])
@pytest.mark.parametrize("M,G,K,N,dt", [(1, 1, 1, 1, "f32"), (40, 2, 64, 130, "f32"), (300, 3, 200, 136, "bf16"), (129, 1, 257, 300, "f16"),
                                        (1000, 6, 96, 72, "f32"), (700, 30, 300, 520, "bf16"), (520, 200, 40, 24, "f32"),
                                        (9000, 1, 130, 140, "f32"), (12000, 3, 200, 300, "bf16"), (20001, 2, 24, 500, "f32")])
def test_weight_gradient(order, M, G, K, N, dt):
    rng = np.random.default_rng(M + K)
    ragged = order == "ragged"
    off = _sizes(rng, M, G) if ragged else None
    x, dy = (_spread(rng, _layout(order, M, G, c), "f32") for c in (K, N))
    forms = []
    for v, c, fmt in ((x, K, "e4m3"), (dy, N, "e5m2")):
        TP = B.rmx_f8_ragged_pitch(M, G) if ragged else B.rmx_f8_pitch(M)
        TE = (TP // 128 + 3) // 4 * 4 if ragged else B.rmx_f8_exps(M)
        qt = full_of((c, TP) if ragged else (G, c, TP), torch.uint8, 0x7F)
        et = full_of((c, TE) if ragged else (G, c, TE), torch.uint8, 255)
        ok(B.rmx_quant_f8_groups(B.make_groups(M, G, c, "f32", order), fmt, dev(off.astype(np.int32)) if ragged else None,
                                 dev(v, "f32"), None, None, qt, et, None, None, 0))
        forms += [qt, et]
    dw = full_of((G, K, N), dt, float("nan"))
    ok(B.rmx_wgrad_f8(B.make_layer_f8(M, G, K, N, dt, "e4m3", "e5m2"), dev(off.astype(np.int32)) if ragged else None, *forms, dw))
    sync()
    got = f64(dw)
    for g in range(G):
        xg, yg = ((v[off[g] : off[g + 1]] if ragged else v[:, g]) for v in (x, dy))
        if xg.shape[0] == 0:
            assert not got[g].any()
            continue
        a, b = O.round_rows(xg.T, "e4m3"), O.round_rows(yg.T, "e5m2")
        ref = a @ b.T
        within(got[g], ref, mma_bound(a, b, xg.shape[0] + 127, dt, ref), f"group {g}")


def test_weight_gradient_of_no_rows():
    dw = full_of((2, 24, 40), "bf16", 5.0)
    ok(B.rmx_wgrad_f8(B.make_layer_f8(0, 2, 24, 40, "bf16"), None, None, None, None, None, dw))
    assert not dw.any()


def test_products_repeat_bit_for_bit():
    M, G, K, N = 600, 40, 640, 512
    rng = np.random.default_rng(8)
    _, qa, ea = f8_operand(rng, M * G, K, "e4m3")
    _, qw, ew = f8_operand(rng, G * N, K, "e4m3")
    outs = [empty((M, G, N), "bf16") for _ in range(4)]
    for o in outs:
        ok(B.rmx_linear_f8(B.make_layer_f8(M, G, K, N, "bf16"), None, qa, ea, qw, ew, None, None, o))
    sync()
    assert all(torch.equal(outs[0], o) for o in outs[1:])


def test_sums_of_faulty_columns():
    """A column's sum holds its infinities and NaN, its neighbours' do not; tiny and huge values sum as they are."""
    M, G, C = 200, 1, 64
    x = torch.randn((M, C), device="cuda")
    x[3, 5], x[150, 6] = float("inf"), float("nan")
    x[:, 8] = 2.0 ** -140
    x[:, 9] = 2.0 ** 120
    gr = B.make_groups(M, G, C, "f32", "groups")
    nws = B.rmx_quant_f8_groups_workspace_bytes(gr)
    sums = empty((G, C), "f32")
    ok(B.rmx_quant_f8_groups(gr, "e4m3", None, x, None, None, None, None, sums, empty((nws,), torch.uint8), nws))
    got, v = f64(sums)[0], f64(x)
    assert np.isposinf(got[5]) and np.isnan(got[6])
    fine = np.ones(C, bool)
    fine[5:7] = False
    within(got[fine], v.sum(0)[fine], 136 * E32 * np.abs(v).sum(0)[fine])
