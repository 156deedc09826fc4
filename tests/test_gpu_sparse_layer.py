"""The sparse layer's operators together, as they are used: a layer of experts forward and backward against the oracle
with the same 8-bit roundings; on streams, in graphs, beside other work, at the ends of buffers, past 31-bit offsets."""

import numpy as np
import pytest
import torch

from ffn_block_gb300 import binding as B
from oracle import sparse_oracle as O
from tests.sparse_util import DT, E32, F8, TINY, U, dev, empty, f64, full_of, ok, state_of, sync, within

pytestmark = pytest.mark.gpu
SEED, OFFSET, P_DROP, EPS = 77, 5, 0.2, 1e-5


class Layer:
    """Buffers and calls of one layer: T tokens of C columns, k of E experts with a [C, C] product each."""

    def __init__(self, T, k, E, C, dt, seed=0):
        rng = np.random.default_rng(seed)
        self.T, self.k, self.E, self.C, self.S, self.dt = T, k, E, C, T * k, dt
        n = lambda *s: rng.standard_normal(s)  # noqa: E731
        self.np = dict(x=n(T, C), w=n(E, C, C) / np.sqrt(C), bias=0.1 * n(E, C), gate=rng.random((T, k)), gamma=1 + 0.2 * n(C),
                       beta=0.2 * n(C), dy=n(T, C), expert=rng.integers(-1, E, (T, k)))
        for name, v in self.np.items():
            t = dev(v.astype(np.int32)) if name == "expert" else dev(v, "f32" if name == "gate" else dt)
            setattr(self, name, t)
            if name != "expert":
                self.np[name] = f64(t)
        S, u8 = self.S, torch.uint8
        P, X = B.rmx_f8_pitch(C), B.rmx_f8_exps(C)
        TP = B.rmx_f8_ragged_pitch(S, E)
        TE = (TP // 128 + 3) // 4 * 4
        self.state = state_of(SEED, OFFSET)
        z = lambda *s, d=dt: full_of(s, d, 0)  # noqa: E731
        i32 = torch.int32
        self.off, self.pos, self.src = z(E + 1, d=i32), z(T, k, d=i32), z(S, d=i32)
        self.rows, self.yr, self.c, self.h, self.y, self.mean, self.rstd = (z(S, C), z(S, C), z(T, C), z(T, C), z(T, C),
                                                                            z(T, d="f32"), z(T, d="f32"))
        self.q, self.e, self.qt, self.et = z(S, P, d=u8), z(S, X, d=u8), z(C, TP, d=u8), z(C, TE, d=u8)
        self.dq, self.de, self.dqt, self.det = z(S, P, d=u8), z(S, X, d=u8), z(C, TP, d=u8), z(C, TE, d=u8)
        self.wq, self.we, self.wqt, self.wet = z(E, C, P, d=u8), z(E, C, X, d=u8), z(E, C, P, d=u8), z(E, C, X, d=u8)
        self.dr, self.dc, self.dgamma, self.dbeta = z(T, C), z(T, C), z(C), z(C)
        self.dyr, self.dgate, self.drows, self.dxg = z(S, C), z(T, k, d="f32"), z(S, C), z(T, C)
        self.dw, self.db = z(E, C, C), z(E, C)
        self.routes, self.tok = B.make_routes(T, k, E, C, dt), B.make_rows(T, C, dt)
        self.acts, self.wts = B.make_groups(S, E, C, dt, "ragged"), B.make_groups(C, E, C, dt, "groups")
        self.drop = B.make_drop(P_DROP, self.state)
        need = [B.rmx_expert_sort_workspace_bytes(self.routes), B.rmx_quant_f8_groups_workspace_bytes(self.acts),
                B.rmx_layer_norm_backward_workspace_bytes(self.tok)]
        self.ws = z(max(need), d=u8)

    def forward(self, st=None):
        E, C, S, n, ws = self.E, self.C, self.S, self.ws.numel(), self.ws
        ok(B.rmx_quant_f8_groups(self.wts, "e4m3", None, self.w, self.wq, self.we, self.wqt, self.wet, None, None, 0, st))
        ok(B.rmx_expert_sort(self.routes, self.expert, self.off, self.pos, self.src, ws, n, st))
        ok(B.rmx_expert_gather(self.routes, self.src, self.x, self.rows, stream=st))
        ok(B.rmx_quant_f8_groups(self.acts, "e4m3", self.off, self.rows, self.q, self.e, self.qt, self.et, None, None, 0, st))
        ok(B.rmx_linear_f8(B.make_layer_f8(S, E, C, C, self.dt), self.off, self.q, self.e, self.wqt, self.wet, self.bias, None,
                           self.yr, st))
        ok(B.rmx_expert_combine(self.routes, self.pos, self.gate, self.yr, self.c, st))
        ok(B.rmx_layer_norm(self.tok, EPS, self.drop, self.c, self.x, self.gamma, self.beta, self.h, self.y, self.mean, self.rstd,
                            st))

    def backward(self, st=None):
        E, C, S, n, ws = self.E, self.C, self.S, self.ws.numel(), self.ws
        ok(B.rmx_layer_norm_backward(self.tok, self.drop, self.dy, None, self.h, self.mean, self.rstd, self.gamma, self.dr,
                                     self.dc, self.dgamma, self.dbeta, ws, n, st))
        ok(B.rmx_expert_combine_backward(self.routes, self.pos, self.gate, self.dc, self.yr, self.dyr, self.dgate, st))
        ok(B.rmx_quant_f8_groups(self.acts, "e5m2", self.off, self.dyr, self.dq, self.de, self.dqt, self.det, self.db, ws, n, st))
        ok(B.rmx_linear_f8(B.make_layer_f8(S, E, C, C, self.dt, "e5m2"), self.off, self.dq, self.de, self.wq, self.we, None, None,
                           self.drows, st))
        ok(B.rmx_wgrad_f8(B.make_layer_f8(S, E, C, C, self.dt, "e4m3", "e5m2"), self.off, self.qt, self.et, self.dqt, self.det,
                          self.dw, st))
        ok(B.rmx_expert_combine(self.routes, self.pos, None, self.drows, self.dxg, st))

    def outputs(self):
        return {n: getattr(self, n) for n in ("y", "h", "dr", "dxg", "dgate", "dw", "db", "dgamma", "dbeta")}


def reference(v, T, k, E, C):
    off, pos, src = O.expert_sort(v["expert"], E)
    n = off[-1]
    rows = v["x"][src[:n] // k]
    pad = lambda a: np.concatenate([a, np.zeros((T * k - n, C))])  # noqa: E731
    part = [slice(off[e], off[e + 1]) for e in range(E)]
    yr = np.zeros((n, C))
    for e, p in enumerate(part):
        yr[p] = O.round_rows(rows[p], "e4m3") @ O.round_rows(v["w"][e].T, "e4m3").T + v["bias"][e]
    c = O.combine(pos, v["gate"], pad(yr))
    f = O.drop_factor(T, C, P_DROP, SEED, OFFSET)
    h = c * f + v["x"]
    y, mean, rstd = O.layer_norm(h, v["gamma"], v["beta"], EPS)
    dr, dgamma, dbeta = O.layer_norm_backward(v["dy"], None, h, mean, rstd, v["gamma"])
    dyr, dgate = O.combine_backward(pos, v["gate"], dr * f, pad(yr))
    dyr = dyr[:n]
    drows, dw, db = np.zeros((n, C)), np.zeros((E, C, C)), np.zeros((E, C))
    for e, p in enumerate(part):
        if off[e] == off[e + 1]:
            continue
        drows[p] = O.round_rows(dyr[p], "e5m2") @ O.round_rows(v["w"][e], "e4m3").T
        dw[e] = O.round_rows(rows[p].T, "e4m3") @ O.round_rows(dyr[p].T, "e5m2").T
        db[e] = dyr[p].sum(0)
    return dict(y=y, h=h, dr=dr, dxg=O.combine(pos, None, pad(drows)), dgate=dgate, dw=dw, db=db, dgamma=dgamma, dbeta=dbeta)


@pytest.mark.parametrize("T,k,E,C", [(1, 1, 2, 128), (50, 2, 5, 136), (300, 3, 9, 72), (257, 2, 4, 333), (700, 2, 24, 256)])
def test_layer_against_the_oracle(T, k, E, C):
    """float32 storage.  What reaches an 8-bit rounding is off by some 2^-20 of its value; a value within that of a tie
    (a share of about 2^-16 of them: 2^-20 over a rounding interval of 2^-4) moves by a step of 2^-3 (e4m3) or 2^-2
    (e5m2), so that a tensor of n values may be off by sqrt(2^-16) * 2^-2 = 2^-10 of its norm."""
    l = Layer(T, k, E, C, "f32")
    l.forward()
    l.backward()
    sync()
    for name, ref in reference(l.np, T, k, E, C).items():
        got = f64(l.outputs()[name])
        assert np.linalg.norm(got - ref) <= 2.0 ** -10 * np.linalg.norm(ref) + 1e-12, name


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_layer_in_16_bits(dt):
    """16-bit storage: every intermediate is rounded (2^-9 or 2^-12 rms / sqrt 3 of its value), which moves a share of
    up to 2^-9 / 2^-4 of the 8-bit values by a step of 2^-2: sqrt(2^-5) * 2^-2 / 2 = 2.2% of a norm, in two products
    one after the other in the gradients."""
    T, k, E, C = 400, 2, 6, 256
    l = Layer(T, k, E, C, dt)
    l.forward()
    l.backward()
    sync()
    for name, ref in reference(l.np, T, k, E, C).items():
        got = f64(l.outputs()[name])
        assert np.linalg.norm(got - ref) <= 4.5e-2 * np.linalg.norm(ref), name


def test_layer_gradient_by_differences():
    """Without 8-bit roundings in the way (they have no derivative): the whole layer's dx, dgate and dbias through the
    oracle's chain agree with differences of the loss when the oracle rounds nothing."""
    T, k, E, C = 12, 2, 3, 40
    l = Layer(T, k, E, C, "f32", seed=4)
    v = dict(l.np)
    keep = O.round_rows
    O.round_rows = lambda a, fmt: a
    try:
        g = reference(v, T, k, E, C)
        rng = np.random.default_rng(1)
        for name, grad in (("x", g["dr"] + g["dxg"]), ("gate", g["dgate"]), ("bias", g["db"]), ("w", g["dw"])):
            d = rng.standard_normal(v[name].shape)
            f = lambda s: (reference(dict(v, **{name: v[name] + s * d}), T, k, E, C)["y"] * v["dy"]).sum()  # noqa: E731,B023
            num = (f(1e-5) - f(-1e-5)) / 2e-5
            assert abs(num - (grad * d).sum()) < 1e-5 * np.abs(grad * d).sum() + 1e-7, name
    finally:
        O.round_rows = keep


def _same(a, b):
    return all(torch.equal(a[n], b[n]) for n in a)


def test_layers_on_streams():
    """Three layers on streams of their own at once give what each gives alone."""
    args = [(700, 2, 24, 256, "bf16", 1), (333, 3, 5, 264, "f16", 2), (1000, 1, 8, 1000, "f32", 3)]
    alone = []
    for a in args:
        l = Layer(*a[:5], seed=a[5])
        l.forward()
        l.backward()
        sync()
        alone.append({n: t.clone() for n, t in l.outputs().items()})
    layers = [Layer(*a[:5], seed=a[5]) for a in args]
    streams = [torch.cuda.Stream() for _ in args]
    torch.cuda.synchronize()
    for _ in range(5):
        for l, s in zip(layers, streams):
            l.forward(s)
            l.backward(s)
    torch.cuda.synchronize()
    sync()
    for l, ref in zip(layers, alone):
        assert _same(l.outputs(), ref)


def test_layer_in_graphs():
    """Captured once and replayed with new inputs and a new dropout state; two graphs with buffers of their own at once."""
    args = [(300, 2, 7, 256, "bf16"), (200, 2, 3, 520, "bf16")]
    layers, graphs, streams = [Layer(*a, seed=i) for i, a in enumerate(args)], [], [torch.cuda.Stream() for _ in args]
    for l, s in zip(layers, streams):
        l.forward(s)                       # the first calls, outside a capture
        l.backward(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            l.forward(s)
            l.backward(s)
        graphs.append(g)
    for step in range(3):
        for i, l in enumerate(layers):
            rng = torch.Generator(device="cuda").manual_seed(10 * step + i)
            l.x.copy_(torch.randn(l.x.shape, generator=rng, device="cuda"))
            l.expert.copy_(torch.randint(-1, l.E, l.expert.shape, generator=rng, device="cuda"))
            l.state.copy_(torch.tensor([step, 1000 + i], device="cuda"))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        got = [{n: t.clone() for n, t in l.outputs().items()} for l in layers]
        for l, o in zip(layers, got):
            l.forward()
            l.backward()
            sync()
            assert _same(l.outputs(), o)


# ------------------------------------------------------------------ beside other work
def _whole(rng, rows, K):
    """Rows of whole numbers of at most 8, exponents 127: every partial sum of K < 2^18 products is exact."""
    P, X = B.rmx_f8_pitch(K), B.rmx_f8_exps(K)
    v = torch.zeros((rows, P), device="cuda")
    v[:, :K] = torch.randint(-8, 9, (rows, K), generator=rng, device="cuda").float()
    return v[:, :K], v.to(torch.float8_e4m3fn).view(torch.uint8), torch.full((rows, X), 127, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("M,G,K,N", [(64, 130, 1000, 300), (16, 200, 700, 640), (5, 3, 4000, 500), (300, 90, 128, 256),
                                     (448, 40, 1000, 520), (1000, 4, 1040, 640), (225, 160, 40, 257)])
def test_product_beside_other_work(M, G, K, N):
    rng = torch.Generator(device="cuda").manual_seed(M + K)
    a, qa, ea = _whole(rng, M * G, K)
    w, qw, ew = _whole(rng, G * N, K)
    ref = torch.einsum("mgk,gnk->mgn", a.double().view(M, G, K), w.double().view(G, N, K)).float()
    layer, out = B.make_layer_f8(M, G, K, N, "f32"), empty((M, G, N), "f32")
    big, st = torch.zeros(1 << 26, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(30):
        if i % 3:
            with torch.cuda.stream(st):
                big.add_(1.0)
        out.fill_(float("nan"))
        ok(B.rmx_linear_f8(layer, None, qa, ea, qw, ew, None, None, out))
        sync()
        assert torch.equal(out, ref), i


@pytest.mark.parametrize("dt,R,C", [("bf16", 9000, 1280), ("bf16", 7001, 1001), ("f32", 3000, 2560), ("f16", 2000, 4097), ("bf16", 5000, 256)])
def test_layer_norm_beside_other_work(dt, R, C):
    s, d = B.make_rows(R, C, dt), B.make_drop(0.1, state_of(1, 2))
    x, r, dy = (torch.randn((R, C), device="cuda").to(DT[dt]) for _ in range(3))
    g = torch.randn(C, device="cuda").to(DT[dt])
    nws = B.rmx_layer_norm_backward_workspace_bytes(s)
    h, y, dr, dx, dg, db = (empty((R, C), dt) for _ in range(4)), None, None, None, None, None
    h, y, dr, dx = h
    dg, db, mean, rstd, ws = empty((C,), dt), empty((C,), dt), empty((R,), "f32"), empty((R,), "f32"), empty((nws,), torch.uint8)
    big, st = torch.zeros(1 << 26, device="cuda"), torch.cuda.Stream()
    first = None
    for i in range(12):
        if i:
            with torch.cuda.stream(st):
                big.add_(1.0)
        for t in (h, y, dr, dx, dg, db, mean, rstd):
            t.fill_(float("nan"))
        ok(B.rmx_layer_norm(s, EPS, d, x, r, g, g, h, y, mean, rstd))
        ok(B.rmx_layer_norm_backward(s, d, dy, None, h, mean, rstd, g, dr, dx, dg, db, ws, nws))
        sync()
        now = [t.clone() for t in (h, y, mean, rstd, dr, dx, dg, db)]
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now)), i


# ------------------------------------------------------------------ the ends of buffers
class Guarded:
    """Tensors between two runs of 256 bytes that nothing may write."""

    def __init__(self):
        self.all = []

    def __call__(self, shape, dt, fill=0):
        d = DT.get(dt, dt)
        n = int(np.prod(shape)) * torch.empty((), dtype=d).element_size()
        raw = torch.full((256 + n + 256 + 15,), 0xA5, dtype=torch.uint8, device="cuda")
        t = raw[256 : 256 + n].view(d).view(shape)
        t.fill_(fill)
        self.all.append((raw, n))
        return t

    def check(self):
        for raw, n in self.all:
            assert torch.all(raw[:256] == 0xA5) and torch.all(raw[256 + n :] == 0xA5)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,E,C", [(7, 2, 3, 1), (9, 3, 4, 65), (13, 2, 5, 517), (5, 2, 3, 1001), (33, 1, 2, 1288)])
def test_nothing_past_the_buffers(dt, T, k, E, C):
    z = Guarded()
    S, u8, i32 = T * k, torch.uint8, torch.int32
    x, y, c = z((T, C), dt), z((S, C), dt), z((T, C), dt)
    for t in (x, y, c):
        t.copy_(torch.randn(t.shape, device="cuda"))
    r, ids = B.make_routes(T, k, E, C, dt), z((T, k), i32)
    ids.copy_(torch.randint(-1, E, (T, k), device="cuda"))
    off, pos, src = z((E + 1,), i32), z((T, k), i32), z((S,), i32)
    n = B.rmx_expert_sort_workspace_bytes(r)
    ok(B.rmx_expert_sort(r, ids, off, pos, src, z((n,), u8), n))
    P, X = B.rmx_f8_pitch(C), B.rmx_f8_exps(C)
    rows, q, e, gate, dgate = z((S, C), dt), z((S, P), u8), z((S, X), u8), z((T, k), "f32", 1), z((T, k), "f32")
    ok(B.rmx_expert_gather(r, src, x, rows, "e4m3", q, e))
    ok(B.rmx_expert_gather(r, src, x, rows))
    ok(B.rmx_expert_combine(r, pos, gate, y, c))
    ok(B.rmx_expert_combine_backward(r, pos, gate, c, y, rows, dgate))
    tok, d = B.make_rows(T, C, dt), B.make_drop(0.3, state_of(1, 1))
    h, o, m, s, g = z((T, C), dt), z((T, C), dt), z((T,), "f32"), z((T,), "f32"), z((C,), dt, 1)
    ok(B.rmx_layer_norm(tok, EPS, d, x, c, g, g, h, o, m, s))
    n = B.rmx_layer_norm_backward_workspace_bytes(tok)
    ok(B.rmx_layer_norm_backward(tok, d, x, c, h, m, s, g, z((T, C), dt), z((T, C), dt), z((C,), dt), z((C,), dt), z((n,), u8), n))
    ok(B.rmx_dropout(tok, d, x, c, o))
    ok(B.rmx_dequant_f8(B.make_rows(S, C, dt), "e4m3", q, e, rows))
    gr = B.make_groups(S, E, C, dt, "ragged")
    TP, n = B.rmx_f8_ragged_pitch(S, E), B.rmx_quant_f8_groups_workspace_bytes(gr)
    qt, et = z((C, TP), u8), z((C, (TP // 128 + 3) // 4 * 4), u8)
    ok(B.rmx_quant_f8_groups(gr, "e4m3", off, y, q, e, qt, et, z((E, C), dt), z((n,), u8), n))
    wts = B.make_groups(C, E, C, dt, "groups")
    w, wq, we, wqt, wet = z((E, C, C), dt, 0.01), z((E, C, P), u8), z((E, C, X), u8), z((E, C, P), u8), z((E, C, X), u8)
    ok(B.rmx_quant_f8_groups(wts, "e4m3", None, w, wq, we, wqt, wet, None, None, 0))
    l = B.make_layer_f8(S, E, C, C, dt)
    ok(B.rmx_linear_f8(l, off, q, e, wqt, wet, z((E, C), dt), rows, z((S, C), dt)))
    ok(B.rmx_wgrad_f8(l, off, qt, et, qt, et, z((E, C, C), dt)))
    tokens = B.make_groups(T, k, C, dt, "tokens")
    tq, te = z((k, C, B.rmx_f8_pitch(T)), u8), z((k, C, B.rmx_f8_exps(T)), u8)
    ok(B.rmx_quant_f8_groups(tokens, "e4m3", None, y, q, e, tq, te, None, None, 0))
    ok(B.rmx_linear_f8(B.make_layer_f8(T, k, C, C, dt), None, q, e, wqt, wet, None, None, z((T, k, C), dt)) if k <= E else 0)
    ok(B.rmx_wgrad_f8(B.make_layer_f8(T, k, C, C, dt), None, tq, te, tq, te, z((k, C, C), dt)))
    sync()
    z.check()


# ------------------------------------------------------------------ offsets past 31 bits
def test_rows_past_31_bits():
    """Sorted rows, their 8-bit forms and normalised rows whose elements pass 2^31."""
    T, k, C, dt = (1 << 18) + 5, 2, 4104, "bf16"
    S = T * k
    assert S * C > 1 << 31
    r = B.make_routes(T, k, 2, C, dt)
    src = torch.arange(S - 1, -1, -1, dtype=torch.int32, device="cuda")
    x = torch.randn((T, C), device="cuda", dtype=torch.bfloat16)
    rows = empty((S, C), dt)
    q, e = empty((S, B.rmx_f8_pitch(C)), torch.uint8), empty((S, B.rmx_f8_exps(C)), torch.uint8)
    ok(B.rmx_expert_gather(r, src, x, rows, "e4m3", q, e))
    at = [0, 1, S // 2, S - 2, S - 1]
    for i in at:
        assert torch.equal(rows[i], x[(S - 1 - i) // k])
    few = rows[at].contiguous()
    q2, e2 = empty((5, q.shape[1]), torch.uint8), empty((5, e.shape[1]), torch.uint8)
    ok(B.rmx_quant_f8(B.make_rows(5, C, dt), "e4m3", few, q2, e2))
    assert torch.equal(q[at], q2) and torch.equal(e[at], e2)
    back = empty((5, C), dt)
    ok(B.rmx_dequant_f8(B.make_rows(S, C, dt), "e4m3", q, e, rows))
    ok(B.rmx_dequant_f8(B.make_rows(5, C, dt), "e4m3", q2, e2, back))
    assert torch.equal(rows[at], back)
    pos = torch.arange(S, dtype=torch.int32, device="cuda").view(T, k)
    out = empty((T, C), dt)
    ok(B.rmx_expert_combine(r, pos, None, rows, out))
    ok(B.rmx_expert_combine_backward(r, pos, None, x, rows, rows, empty((T, k), "f32")))
    for t in (0, T // 2, T - 1):
        assert torch.equal(rows[2 * t], x[t]) and torch.equal(rows[2 * t + 1], x[t])
    # the same rows normalised in place, and as rows of an odd length
    for C2 in (C, 4101):
        R = S * C // C2
        s, m, v = B.make_rows(R, C2, dt), empty((R,), "f32"), empty((R,), "f32")
        h = rows.view(-1)[: R * C2].view(R, C2)
        y = empty((R, C2), dt)
        ok(B.rmx_layer_norm(s, EPS, None, h, None, None, None, None, y, m, v))
        for i in (0, R // 2 + 1, R - 1):
            y1 = empty((1, C2), dt)
            ok(B.rmx_layer_norm(B.make_rows(1, C2, dt), EPS, None, h[i].clone(), None, None, None, None, y1, None, None))
            assert torch.equal(y[i : i + 1], y1), i
    sync()


def test_products_past_31_bits():
    M, K, N = 540_000, 128, 4096
    rng = torch.Generator(device="cuda").manual_seed(1)
    a, qa, ea = _whole(rng, M, K)
    w, qw, ew = _whole(rng, N, K)
    out = empty((M, 1, N), "bf16")
    assert out.numel() > 1 << 31
    ok(B.rmx_linear_f8(B.make_layer_f8(M, 1, K, N, "bf16"), None, qa, ea, qw, ew, None, None, out))
    off = torch.tensor([0, 10, M - 7], dtype=torch.int32, device="cuda")
    at = [0, 9, 10, M // 2, M - 8, M - 7, M - 1]
    ref = (a[at].double() @ w.double().t()).bfloat16()
    assert torch.equal(out[at, 0], ref)
    out.fill_(3.0)
    w2, qw2, ew2 = torch.cat([w, w]), torch.cat([qw, qw]), torch.cat([ew, ew])
    ok(B.rmx_linear_f8(B.make_layer_f8(M, 2, K, N, "bf16"), off, qa, ea, qw2, ew2, None, None, out))
    sync()
    assert torch.equal(out[at[:5], 0], ref[:5]) and torch.all(out[at[5:]] == 3.0)
    del out, w2
    # columns of rows past 2^31 elements
    x = torch.randint(-8, 9, (M, N), generator=rng, device="cuda", dtype=torch.int8).bfloat16()
    gr = B.make_groups(M, 2, N, "bf16", "ragged")
    TP, nws = B.rmx_f8_ragged_pitch(M, 2), B.rmx_quant_f8_groups_workspace_bytes(gr)
    qt, et = empty((N, TP), torch.uint8), empty((N, (TP // 128 + 3) // 4 * 4), torch.uint8)
    sums = empty((2, N), "bf16")
    ok(B.rmx_quant_f8_groups(gr, "e4m3", off, x, None, None, qt, et, sums, empty((nws,), torch.uint8), nws))
    sync()
    last = qt.view(TP // 128, N, 128)[1 + (M - 17 + 127) // 128 - 1]     # the second group's last block
    rows = x[10 + (M - 17 - 1) // 128 * 128 : M - 7].float()
    top = rows.abs().amax(0)
    step = torch.exp2(torch.ceil(torch.log2(top / 448)))
    assert torch.equal(last.view(torch.float8_e4m3fn).float()[:, : rows.shape[0]].t() * step, rows)
    assert torch.equal(sums[0].float(), x[:10].float().sum(0).bfloat16().float())
