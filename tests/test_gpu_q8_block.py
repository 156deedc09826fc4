"""The 8-bit operators together, as they are used: the block served in int8,
its saved activations kept in 8 bits, a pre-norm layer forward and backward;
streams, graphs, buffer bounds, repeatability, long offsets."""

import numpy as np
import pytest
import torch

from ffn_block_gb300 import binding as B
from ffn_block_gb300 import inputs as I
from ffn_block_gb300.device import RankMixerDevice
from oracle import q8_oracle as Q
from oracle import rmx_oracle as O

from parity_util import NAMES, oracle_outputs, rel_err
from q8_util import DT, E32, TINY, U, dev, empty, f64, ok, rnd, sync, within

pytestmark = pytest.mark.gpu

BLOCKS = [dict(B=4, T=16, D=128, H=256), dict(B=1, T=8, D=64, H=128), dict(B=130, T=8, D=128, H=384),
          dict(B=33, T=8, D=240, H=360), dict(B=3, T=4, D=512, H=2568)]
IDS = lambda d: "B{B}_T{T}_D{D}_H{H}".format(**d)  # noqa: E731


def block(dims, dt, seed=7101):
    shape = I.Shape(dtype=dt, **dims)
    arrays = I.make_inputs(shape, seed=seed, ln_params="random")
    return RankMixerDevice(shape, arrays), arrays


# ------------------------------------------------------------------ the block served in int8

@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dims", BLOCKS, ids=IDS)
def test_forward_q8(dims, dt):
    blk, arrays = block(dims, dt)
    blk.quantize_weights()
    blk.y.fill_(float("nan"))
    blk.forward_q8()
    sync()
    a = I.to_float64(arrays)
    p = {k: a[k] for k in I.PARAM_NAMES}
    ref = Q.block_forward_q8(a["x"], p, *(f64(blk.q8[k]) for k in ("w1", "w1_scale", "wout", "wout_scale")))
    # Rows are quantised from values rounded to the storage type, so some
    # integers differ by one from the definition's: a rounding error d moves a
    # share d / step of them.  16-bit: d about 2^-10 of the row's rms and the
    # step about 2^-5: 3% of the integers, sqrt(0.03) * 2^-5 = 0.6% of the
    # norm, in two products; with the 2e-2 of the block's own 16-bit passes.
    # float32: d about 2^-22, a share of 2^-17, 1e-4 of the norm.
    tol = 5e-4 if dt == "f32" else 3e-2
    y = f64(blk.y)
    assert np.all(np.isfinite(y)) and rel_err(y, ref) <= tol
    # Against the block itself: rounding to int8 is off by step / sqrt(12) rms.
    # out1 and w1: steps of 1/32 and 1/64 of the rms, hidden (long tails): up
    # to 1/12, so about 1%, 0.5% and 2.4% of the products' norms.
    full, _ = O.forward(a["x"], p)
    assert rel_err(y, full) <= 6e-2


def test_forward_q8_refusals_and_empty_batch():
    blk, _ = block(dict(B=4, T=16, D=128, H=256), "bf16")
    blk.quantize_weights()
    for cfg in (B.make_config(4, 9, 81, 162, "bf16"), B.make_config(4, 16, 128, 256, "tf32")):
        assert B.rmx_forward_q8_workspace_bytes(cfg) == 0 and B.rmx_saved8_bytes(cfg) == 0
        assert B.rmx_forward_q8(cfg, blk.x, blk.c_params, blk.c_q8, blk.ws_q8, 1 << 40, blk.y) == B.RMX_ERR_UNSUPPORTED
        assert B.rmx_saved_pack8(cfg, blk.saved, 1 << 40, blk.ws, 1 << 40) == B.RMX_ERR_UNSUPPORTED
    assert B.rmx_forward_q8(blk.cfg, blk.x, blk.c_params, blk.c_q8, blk.ws_q8, blk.ws_q8.numel() - 1,
                            blk.y) == B.RMX_ERR_WORKSPACE
    assert B.rmx_forward_q8(blk.cfg, blk.x, blk.c_params, blk.c_q8, blk.ws_q8, blk.ws_q8.numel(),
                            blk.x) == B.RMX_ERR_INVALID_ARG
    empty_cfg = B.make_config(0, 16, 128, 256, "bf16")
    assert B.rmx_forward_q8(empty_cfg, None, blk.c_params, blk.c_q8, None, 0, None) == B.RMX_OK


def test_forward_q8_needs_no_16_bit_weights():
    blk, _ = block(dict(B=4, T=16, D=128, H=256), "bf16")
    blk.quantize_weights()
    blk.forward_q8()
    sync()
    y = blk.y.clone()
    params = B.make_params({**blk.params, "w1": 0, "wout": 0})
    blk.y.zero_()
    ok(B.rmx_forward_q8(blk.cfg, blk.x, params, blk.c_q8, blk.ws_q8, blk.ws_q8.numel(), blk.y))
    sync()
    assert torch.equal(blk.y, y)


# ------------------------------------------------------------------ saved activations in 8 bits

def saved_tensors(blk):
    """out1, Z, hidden, s2, s1 and the statistics of the saved buffer, by its documented layout."""
    s, e = blk.shape, 4 if blk.shape.dtype == "f32" else 2
    N, up = s.B * s.T, lambda v: (v + 255) // 256 * 256
    tiles = (2 * s.H + 127) // 128
    out, o = {}, 0
    for name, cols, size in (("out1", s.D, e), ("Z", 2 * s.H, e), ("hidden", s.H, e), ("s2", s.D, e), ("stats", 10, 4),
                             ("zstats", 4 * tiles, 4), ("s1", s.D, e)):
        n = N * cols * size
        raw = blk.saved[o:o + n]
        out[name] = raw.view(torch.float32 if name in ("stats", "zstats") else DT[s.dtype]).view(N, cols)
        o = up(o + n)
    return out


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dims", BLOCKS, ids=IDS)
def test_saved_checkpoint_and_backward(dims, dt):
    blk, arrays = block(dims, dt)
    blk.forward()
    sync()
    before = {k: v.clone() for k, v in saved_tensors(blk).items()}
    packed = blk.pack_saved()
    # 33 bytes for 32 elements of two or four bytes, the statistics as they
    # are, and each of the 11 segments rounded up to 256 bytes
    assert packed.numel() < 0.62 * blk.saved.numel() + 11 * 256
    blk.saved.fill_(0xFF)                       # NaN everywhere
    blk.unpack_saved(packed)
    sync()
    after = saved_tensors(blk)
    assert torch.equal(after["stats"], before["stats"])
    for k in ("out1", "Z", "hidden", "s2", "s1"):
        q, e = Q.ckpt_pack(f64(before[k]), dt)
        assert np.array_equal(f64(after[k]), Q.ckpt_values(q, e, after[k].shape[1])), k
    blk.backward()
    sync()
    got, ref = blk.results(), oracle_outputs(arrays)
    # Half a step of a group is at most 1/127.5 of its largest value, uniform:
    # 0.5% rms of it, about 1% of the group's rms (three such tensors in a row
    # on a gradient's way, each through a LayerNorm's backward).
    for k in NAMES:
        if k != "y":
            assert np.all(np.isfinite(got[k])), k
            if np.linalg.norm(ref[k]) > 1e-9 * np.linalg.norm(ref["dx"]):
                assert rel_err(got[k], ref[k]) <= 6e-2, k


def test_saved8_refusals():
    blk, _ = block(dict(B=4, T=16, D=128, H=256), "bf16")
    n8 = B.rmx_saved8_bytes(blk.cfg)
    buf = empty(n8, torch.uint8)
    assert B.rmx_saved_pack8(blk.cfg, blk.saved, blk.saved_bytes, buf, n8 - 1) == B.RMX_ERR_WORKSPACE
    assert B.rmx_saved_pack8(blk.cfg, blk.saved, blk.saved_bytes - 1, buf, n8) == B.RMX_ERR_WORKSPACE
    assert B.rmx_saved_unpack8(blk.cfg, buf, n8 - 1, blk.saved, blk.saved_bytes) == B.RMX_ERR_WORKSPACE
    assert B.rmx_saved_unpack8(blk.cfg, None, n8, blk.saved, blk.saved_bytes) == B.RMX_ERR_INVALID_ARG
    assert B.rmx_saved_pack8(blk.cfg, blk.saved, blk.saved_bytes, buf.data_ptr() + 8, n8) == B.RMX_ERR_ALIGNMENT


# ------------------------------------------------------------------ a pre-norm layer, forward and backward

class Layer:
    """x, r -> h = x + r, n = rms(h) in int8, out = n @ w + b; then the gradients from 8-bit checkpoints."""

    def __init__(self, M, G, K, N, dt, seed=3, make=empty):
        rng = np.random.default_rng(seed)
        self.M, self.G, self.K, self.N, self.dt = M, G, K, N, dt
        R, P = M * G, Q.pitch(K)
        self.rows, self.layer = B.make_rows(R, K, dt), B.make_layer(M, G, K, N, dt)
        self.x, self.r = (dev(rng.standard_normal((R, K)), dt) for _ in range(2))
        self.gamma = dev(1 + 0.3 * rng.standard_normal(K), dt)
        self.w = dev(rng.standard_normal((G, K, N)) / np.sqrt(K), dt)
        self.b = dev(rng.standard_normal((G, N)), dt)
        self.dout = dev(rng.standard_normal((M, G, N)), dt)
        self.dn = dev(rng.standard_normal((R, K)), dt)   # the gradient a data-gradient product hands on
        i8, f4 = torch.int8, torch.float32
        self.wq, self.ws = make((G, N, P), i8), make((G, N), f4)
        self.h, self.n, self.q, self.s, self.rstd = make((R, K), dt), make((R, K), dt), make((R, P), i8), make(R, f4), make(R, f4)
        self.out = make((M, G, N), dt)
        self.hq, self.he, self.nq, self.ne = (make((R, P // d), i8) for d in (1, 32, 1, 32))
        self.dw, self.db, self.dx, self.dg = make((G, K, N), dt), make((G, N), dt), make((R, K), dt), make(K, dt)
        self.nb1 = B.rmx_ckpt8_wgrad_workspace_bytes(self.layer)
        self.nb2 = B.rmx_rms_norm_backward_workspace_bytes(self.rows)
        self.w1, self.w2 = make(self.nb1, torch.uint8), make(self.nb2, torch.uint8)

    def outputs(self):
        return {k: getattr(self, k) for k in ("wq", "ws", "h", "n", "q", "s", "rstd", "out", "hq", "he", "nq", "ne", "dw",
                                              "db", "dx", "dg")}

    def run(self, st=None):
        ok(B.rmx_weight_q8(self.layer, self.w, self.wq, self.ws, st))
        ok(B.rmx_rms_norm_q8(self.rows, 1e-5, self.x, self.r, self.gamma, self.h, self.n, self.q, self.s, self.rstd, st))
        ok(B.rmx_linear_q8(self.layer, self.q, self.s, self.wq, self.ws, self.b, None, self.out, st))
        ok(B.rmx_ckpt8_pack(self.rows, self.h, self.hq, self.he, st))
        ok(B.rmx_ckpt8_pack(self.rows, self.n, self.nq, self.ne, st))
        ok(B.rmx_ckpt8_wgrad(self.layer, self.nq, self.ne, self.dout, self.dw, self.db, self.w1, self.nb1, st))
        ok(B.rmx_rms_norm_backward(self.rows, self.dn, None, None, self.hq, self.he, self.rstd, self.gamma, self.dx,
                                   self.dg, self.w2, self.nb2, st))


SHAPES = [(5, 3, 100, 72, "bf16"), (64, 2, 256, 512, "f16"), (33, 4, 81, 55, "bf16"), (200, 1, 320, 300, "bf16"),
          (20, 2, 64, 40, "f32")]


@pytest.mark.parametrize("M,G,K,N,dt", SHAPES)
def test_layer_forward_and_backward(M, G, K, N, dt):
    L = Layer(M, G, K, N, dt)
    L.run()
    sync()
    x, r, g, w, b = (f64(t) for t in (L.x, L.r, L.gamma, L.w, L.b))
    h, rstd, n = Q.rms_norm(x, r, g, 1e-5)
    out = np.einsum("mgk,gkn->mgn", n.reshape(M, G, K), w) + b
    # int8 rows and channels: half a step (max / 254) uniform on each factor
    noise = np.einsum("mgk,gkn->mgn", (np.abs(n).max(1, keepdims=True) / 127 / np.sqrt(12) * np.ones_like(n)).reshape(M, G, K) ** 2,
                      w ** 2) + np.einsum("mgk,gkn->mgn", n.reshape(M, G, K) ** 2,
                                          (np.abs(w).max(1, keepdims=True) / 127 / np.sqrt(12) * np.ones_like(w)) ** 2)
    err = np.abs(f64(L.out) - out)
    assert np.all(err <= 6 * np.sqrt(noise) + np.abs(out) * 2 * U[dt])          # six sigmas
    # the gradients, from what the checkpoints hold
    nv = Q.ckpt_values(*Q.ckpt_pack(f64(L.n), dt), K)
    hv = Q.ckpt_values(*Q.ckpt_pack(f64(L.h), dt), K)
    dw, db = Q.wgrad(nv.reshape(M, G, K), f64(L.dout))
    mw, mb = Q.wgrad(np.abs(nv).reshape(M, G, K), np.abs(f64(L.dout)))
    within(f64(L.dw), dw, np.abs(dw) * U[dt] + mw * (2 * M + 4) * E32 + TINY[dt], "dw")
    within(f64(L.db), db, np.abs(db) * U[dt] + mb * (M + 4) * E32 + TINY[dt], "db")
    dx, dg = Q.rms_norm_backward(hv, f64(L.rstd), g, f64(L.dn), None)
    assert rel_err(f64(L.dx), dx) <= U[dt] + 1e-5 and rel_err(f64(L.dg), dg) <= U[dt] + 1e-5
    # and against the gradients of the unquantised layer: 1% a checkpoint
    tw, _ = Q.wgrad(n.reshape(M, G, K), f64(L.dout))
    tx, tg = Q.rms_norm_backward(h, rstd, g, f64(L.dn), None)
    for got, ref in ((L.dw, tw), (L.dx, tx), (L.dg, tg)):
        assert rel_err(f64(got), ref) <= 3e-2


@pytest.mark.parametrize("M,G,K,N,dt", SHAPES)
def test_layer_is_repeatable_and_writes_only_its_buffers(M, G, K, N, dt):
    ref = Layer(M, G, K, N, dt)
    ref.run()
    sync()
    raws = []

    def guarded(shape, d):
        t = torch.empty(shape, dtype=DT.get(d, d), device="cuda")
        n = t.numel() * t.element_size()
        raw = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        raws.append((raw, n))
        return raw[4096:4096 + n].view(t.dtype).view(t.shape)

    L = Layer(M, G, K, N, dt, make=guarded)
    for _ in range(2):
        L.run()
        sync()
        for k, v in L.outputs().items():
            assert torch.equal(v, ref.outputs()[k]), k
        for raw, n in raws:
            assert (raw[:4096] == 0xA5).all().item() and (raw[4096 + n:] == 0xA5).all().item()


def test_layers_on_two_streams_at_once():
    ref = [Layer(64, 4, 256, 384, "bf16", seed=s) for s in (1, 2)]
    for L in ref:
        L.run()
    sync()
    both = [Layer(64, 4, 256, 384, "bf16", seed=s) for s in (1, 2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in both]
    for _ in range(5):
        for L, st in zip(both, streams):
            L.run(st)
    for st in streams:
        B.check(B.rmx_check(st))
    for a, b in zip(ref, both):
        for k, v in a.outputs().items():
            assert torch.equal(v, b.outputs()[k]), k


@pytest.mark.parametrize("M,G,K,N,dt", SHAPES[:3])
def test_layer_in_a_graph(M, G, K, N, dt):
    L = Layer(M, G, K, N, dt)
    L.run()
    sync()
    want = {k: v.clone() for k, v in L.outputs().items()}
    graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=st):
        L.run(st)
    for v in L.outputs().values():
        v.zero_()
    for _ in range(2):
        graph.replay()
    sync()
    for k, v in L.outputs().items():
        assert torch.equal(v, want[k]), k
    # new values in the same buffers
    L.x.mul_(0.5)
    graph.replay()
    sync()
    again = {k: v.clone() for k, v in L.outputs().items()}
    L.run()
    sync()
    for k, v in L.outputs().items():
        assert torch.equal(v, again[k]), k
    assert not torch.equal(again["out"], want["out"])


# ------------------------------------------------------------------ offsets past 31 bits

def test_checkpoint_past_2_31_elements():
    R, C = (1 << 20) + 3, 2112
    x = torch.empty((R, C), dtype=torch.bfloat16, device="cuda")
    x.copy_((torch.arange(C, device="cuda") % 251 - 125).to(torch.bfloat16))
    x[-1] *= 3
    q, e = empty((R, C), torch.int8), empty((R, C // 32), torch.int8)
    sh = B.make_rows(R, C, "bf16")
    ok(B.rmx_ckpt8_pack(sh, x, q, e))
    v = torch.zeros_like(x)
    ok(B.rmx_ckpt8_unpack(sh, q, e, v))
    sync()
    for rows in (slice(0, 2), slice(R // 2, R // 2 + 2), slice(R - 2, R)):
        rq, re = Q.ckpt_pack(f64(x[rows]), "bf16")
        assert np.array_equal(q[rows].cpu().numpy(), rq) and np.array_equal(e[rows].cpu().numpy(), re)
        assert np.array_equal(f64(v[rows]), Q.ckpt_values(rq, re, C))


def test_linear_past_2_31_outputs():
    M, G, K, N = 4100, 64, 32, 8200
    g = torch.Generator(device="cuda").manual_seed(0)
    a = torch.randint(-127, 128, (M, G, 32), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-127, 128, (G, N, 32), generator=g, device="cuda", dtype=torch.int8)
    sa, sw = torch.rand((M, G), generator=g, device="cuda"), torch.rand((G, N), generator=g, device="cuda")
    out = empty((M, G, N), "bf16")
    ok(B.rmx_linear_q8(B.make_layer(M, G, K, N, "bf16"), a, sa, w, sw, None, None, out))
    sync()
    for m in (0, 2049, M - 1):
        ref = Q.linear_q8(*(f64(t) for t in (a[m:m + 1], sa[m:m + 1], w, sw)), None, None, K)
        within(f64(out[m:m + 1]), ref, np.abs(ref) * (U["bf16"] + 6 * E32) + TINY["bf16"], m)
