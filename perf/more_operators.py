"""What is measured of the sparse layer's operators: their cases, plain forms and calls.

Four operators around a layer whose rows go to a few of many experts, each in
its plain form (elementary torch operations in float32, rounded once at the
end) and as the library's own calls:

  norm      h = drop(x) + r; y = (h - mean) * rstd * gamma + beta, with the row
            statistics; and its backward from the stored sum (dr, dx, dgamma,
            dbeta)
  dropout   out = drop(x) + r
  route     (token, choice) slots sorted by expert, the tokens' rows gathered in
            that order, and the experts' rows added up again with the router's
            weights; in training also both backward passes
  f8        product of 8-bit floating rows: out = X W + bias, X quantised in the
            call; in training also dX = dY W^T, dW = X^T dY and db, with all
            operands quantised in the call

Dropout.  The keep bits come from Philox4x32-10 (Salmon, Moraes, Dror, Shaw,
"Parallel random numbers: as easy as 1, 2, 3", 2011): the counter is (column /
8, row, offset), the key the seed; each of the four words gives two elements 16
bits, the lower half first.  An element is kept where its 16 bits are at least
round(65536 p), and is multiplied by 65536 / (65536 - round(65536 p)).

8-bit rows.  A row is cut into blocks of 128 columns along the contraction.  A
block keeps q * 2^e, q in e4m3 (largest value 448) or e5m2 (57344), e the
smallest exponent >= -127 with max|block| <= largest * 2^e, one byte e + 127 a
block.  Rows are padded with zeros to whole blocks.
"""

import math

import numpy as np
import torch

own = False

EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
MASK = 0xFFFFFFFF


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # One sample's tokens, served: launch latency.
        dict(name="norm one sample", op="norm", rows=64, cols=1280, dtype="bf16", p=0.0, resid=True),
        # Every row of the production block (B = 1024, T = 64, D = 1280), trained with dropout.
        dict(name="norm production", op="norm", rows=65536, cols=1280, dtype="bf16", p=0.1, resid=True),
        # The same rows' backward.
        dict(name="norm_bwd production", op="norm_bwd", rows=65536, cols=1280, dtype="bf16", p=0.1, resid=True),
        # Odd row length, float32, no other gradient.
        dict(name="norm_bwd odd f32", op="norm_bwd", rows=3001, cols=513, dtype="f32", p=0.25, resid=False),
        # The rows of the ragged block (1000 x 40 x 1200).
        dict(name="dropout ragged f16", op="dropout", rows=40000, cols=1200, dtype="f16", p=0.5, resid=True),
        # A small float32 batch, alone.
        dict(name="dropout small f32", op="dropout", rows=128, cols=250, dtype="f32", p=0.2, resid=False),
        # One sample served by two of 32 experts a token.
        dict(name="route one sample", op="route", tokens=64, k=2, experts=32, cols=1280, dtype="bf16", holes=False,
             train=False),
        # A production batch in training, a few slots dropped by the router.
        dict(name="route production", op="route", tokens=65536, k=2, experts=64, cols=1280, dtype="bf16", holes=True,
             train=True),
        # Odd sizes: rows of 1001 columns, four of 24 experts.
        dict(name="route odd f16", op="route", tokens=5003, k=4, experts=24, cols=1001, dtype="f16", holes=True,
             train=True),
        # A sample served by the per-token layer: its weights are streamed once.
        dict(name="f8 one sample", op="f8", M=1, G=64, K=1280, N=5120, dtype="bf16", ragged=False, bias=True,
             train=False, grad="e4m3"),
        # The first layer of the production block.
        dict(name="f8 production", op="f8", M=1024, G=64, K=1280, N=5120, dtype="bf16", ragged=False, bias=True,
             train=False, grad="e4m3"),
        # 32 experts' training step on 16384 tokens with two experts each.
        dict(name="f8 experts training", op="f8", M=32768, G=32, K=1280, N=2560, dtype="bf16", ragged=True, bias=True,
             train=True, grad="e5m2"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "dropout", "route", "f8", "f8"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    p = rng.choice([0.0, 0.1, 0.25, 0.5])
    if op in ("norm", "norm_bwd", "dropout"):
        cols = _log(rng, 16, 8192)
        if rng.random() < 0.6:
            cols = max(16, cols // 8 * 8)
        most = 40_000_000 if dtype == "f32" else 80_000_000
        return dict(op=op, rows=_log(rng, 1, max(2, min(65536, most // cols))), cols=cols, dtype=dtype,
                    p=0.3 if op == "dropout" and p == 0 else p, resid=rng.random() < 0.6)
    if op == "route":
        experts, cols = _log(rng, 2, 256), _log(rng, 16, 4096)
        if rng.random() < 0.6:
            cols = max(16, cols // 8 * 8)
        k = rng.randint(1, min(8, experts))
        most = 80_000_000 // (cols * k)
        return dict(op=op, tokens=_log(rng, 1, max(2, min(65536, most))), k=k, experts=experts, cols=cols, dtype=dtype,
                    holes=rng.random() < 0.5, train=rng.random() < 0.6)
    K, N = _log(rng, 48, 3840), _log(rng, 48, 5120)
    if rng.random() < 0.6:
        K, N = max(48, K // 16 * 16), max(48, N // 16 * 16)
    ragged, G = rng.random() < 0.6, _log(rng, 1, 64)
    M = _log(rng, 1, 32768 if ragged else 1024)
    train = ragged and rng.random() < 0.5
    while (M if ragged else M * G) * K * N * (3 if train else 1) > 32768 * 1280 * 2560 * 3 or G * K * N > 200_000_000:
        G, M = max(1, G // 2), max(1, M // 2)
    return dict(op=op, M=M, G=G, K=K, N=N, dtype="bf16" if dtype == "f32" else dtype, ragged=ragged,
                bias=rng.random() < 0.6, train=train, grad=rng.choice(["e4m3", "e5m2"]))


# ------------------------------------------------------------------ formats
def _pitch(cols):
    return (cols + 127) // 128 * 128


def _pow2(e):
    """2^e for an integer tensor, in float64 and exact."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _quantise(x, fmt):
    """x [..., C] float32 -> its 8-bit values q [..., P] (as float8) and exponents e [..., P / 128]."""
    C, P = x.shape[-1], _pitch(x.shape[-1])
    if P != C:
        x = torch.nn.functional.pad(x, (0, P - C))
    b = x.reshape(*x.shape[:-1], P // 128, 128)
    m, k = torch.frexp(b.abs().amax(-1))           # max = m * 2^k, m in [0.5, 1)
    e = k - (9 if fmt == "e4m3" else 16) + (m > 0.875).to(k.dtype)
    e = torch.where(m > 0, e, torch.full_like(e, -127)).clamp_min(-127)
    q = (b * _pow2(-e).float().unsqueeze(-1)).to(F8[fmt])
    return q.reshape(x.shape), e


def _values(q, e, cols):
    v = q.float().reshape(*e.shape, 128) * _pow2(e).float().unsqueeze(-1)
    return v.reshape(q.shape)[..., :cols]


def _round8(x, fmt):
    """The values that the 8-bit rows of x [..., C] stand for, in float32."""
    return _values(*_quantise(x, fmt), x.shape[-1])


# ------------------------------------------------------------------ dropout
def _philox(c, k0, k1):
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((b >> 32) & MASK) ^ c[1] ^ k0, b & MASK, ((a >> 32) & MASK) ^ c[3] ^ k1, a & MASK]
        k0, k1 = (k0 + 0x9E3779B9) & MASK, (k1 + 0xBB67AE85) & MASK
    return c


def _factor(case, rng):
    """What dropout multiplies each element by: 0 or the scale, float32 [rows, cols]; None where p is 0."""
    t = round(case["p"] * 65536)
    if t == 0:
        return None
    R, C = case["rows"], case["cols"]
    groups = (C + 7) // 8
    row = torch.arange(R, device="cuda").unsqueeze(1)
    col = torch.arange(groups, device="cuda").unsqueeze(0)
    seed, off = rng[0], rng[1]
    zero = torch.zeros((R, groups), dtype=torch.int64, device="cuda")
    words = _philox([col + zero, row + zero, (off & MASK) + zero, ((off >> 32) & MASK) + zero],
                    seed & MASK, (seed >> 32) & MASK)
    keep = torch.empty((R, groups, 8), dtype=torch.bool, device="cuda")
    for j, w in enumerate(words):
        keep[..., 2 * j] = (w & 0xFFFF) >= t
        keep[..., 2 * j + 1] = (w >> 16) >= t
    return keep.reshape(R, groups * 8)[:, :C].float() * (65536 / (65536 - t))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, shape, dt):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)


def prepare(case, seed):
    g, dt, op = _gen(seed), DTYPES[case["dtype"]], case["op"]
    s = dict(case)
    empty = lambda *shape, dtype=dt: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    zeros = lambda *shape, dtype=dt: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
    if op in ("norm", "norm_bwd", "dropout"):
        R, C = case["rows"], case["cols"]
        s["rng"] = torch.randint(0, 1 << 62, (2,), generator=g, device="cuda")
        x = _randn(g, (R, C), dt)
        if op == "dropout":
            s.update(x=x, r=_randn(g, (R, C), dt) if case["resid"] else None, out=empty(R, C))
            return s
        s["gamma"] = (1 + 0.2 * torch.randn(C, generator=g, device="cuda")).to(dt)
        if op == "norm":
            s["beta"] = (0.2 * torch.randn(C, generator=g, device="cuda")).to(dt)
            s.update(x=x, r=_randn(g, (R, C), dt) if case["resid"] else None)
            s.update(h=empty(R, C), y=empty(R, C), mean=empty(R, dtype=torch.float32), rstd=empty(R, dtype=torch.float32))
            return s
        # the sum that the forward kept, with the statistics of its rows
        s["h"] = (x.float() + 0.25).to(dt)
        h = s["h"].double()
        s["mean"] = h.mean(-1).float()
        s["rstd"] = torch.rsqrt((h - h.mean(-1, keepdim=True)).square().mean(-1) + EPS).float()
        del h, x
        s["dy"] = _randn(g, (R, C), dt)
        s["dh"] = _randn(g, (R, C), dt) if case["resid"] else None
        # scratch: up to 1024 partial rows of two float32 column sums
        s.update(dr=empty(R, C), dx=empty(R, C) if case["p"] > 0 else None, dgamma=empty(C), dbeta=empty(C),
                 ws=empty(1024 * 2 * (C + 64) * 4 + 4096, dtype=torch.uint8))
        return s
    if op == "route":
        T, k, E, C = (case[n] for n in ("tokens", "k", "experts", "cols"))
        S = T * k
        # a router's scores, some experts more popular than others
        score = torch.randn((T, E), generator=g, device="cuda") + 0.6 * torch.randn(E, generator=g, device="cuda")
        w, ids = torch.topk(torch.softmax(score, -1), k)
        s["weight"] = (w / w.sum(-1, keepdim=True)).contiguous()
        s["expert"] = ids.to(torch.int32).contiguous()
        if case["holes"]:
            s["expert"][torch.rand((T, k), generator=g, device="cuda") < 0.03] = -1
        s.update(x=_randn(g, (T, C), dt), y=_randn(g, (S, C), dt))
        i32 = lambda *shape: empty(*shape, dtype=torch.int32)  # noqa: E731
        # rows behind the last expert's stay what they are: zeros here
        s.update(offsets=i32(E + 1), position=i32(T, k), source=i32(S), rows=zeros(S, C), out=empty(T, C),
                 ws=empty(4 * (E + 32) * (S // 256 + 512) + 65536, dtype=torch.uint8))
        if case["train"]:
            s.update(dout=_randn(g, (T, C), dt), drows=_randn(g, (S, C), dt), dy=zeros(S, C),
                     dweight=empty(T, k, dtype=torch.float32), dx=empty(T, C))
        return s
    M, G, K, N = (case[n] for n in "MGKN")
    u8 = lambda *shape: empty(*shape, dtype=torch.uint8)  # noqa: E731
    ex = lambda c: (_pitch(c) // 128 + 3) // 4 * 4  # noqa: E731
    lead = (M,) if case["ragged"] else (M, G)
    s["x"] = _randn(g, (*lead, K), dt)
    # a few columns with larger values, as activations have
    s["x"][..., ::61] *= 8
    if case["ragged"]:
        cpu = np.random.default_rng(seed)
        share = np.exp(0.6 * cpu.standard_normal(G)) * (cpu.random(G) < 0.95)
        sizes = cpu.multinomial(M, share / share.sum()) if share.sum() > 0 else np.array([M] + [0] * (G - 1))
        s["sizes"] = [int(v) for v in sizes]
        s["offsets"] = torch.tensor([0, *np.cumsum(sizes)], dtype=torch.int32, device="cuda")
    s["bias"] = _randn(g, (G, N), dt) if case["bias"] else None
    w = torch.randn((G, K, N), generator=g, device="cuda") / math.sqrt(K)
    s.update(out=empty(*lead, N), q=u8(*lead, _pitch(K)), e=u8(*lead, ex(K)))
    if not case["train"]:
        # serving: the weights are in 8 bits, [G, N, P], laid out once
        q, e = _quantise(w.transpose(1, 2).contiguous(), "e4m3")
        s["w"] = q.view(torch.uint8)
        s["we"] = torch.zeros((G, N, ex(K)), dtype=torch.uint8, device="cuda")
        s["we"][..., : e.shape[-1]] = (e + 127).to(torch.uint8)
        return s
    s["w"] = w.to(dt)
    s["dy"] = _randn(g, (M, N), dt)
    tp = (M // 128 + min(G, M)) * 128  # rows of every expert in whole blocks of 128
    s.update(qt=u8(K, tp), et=u8(K, (tp // 128 + 3) // 4 * 4), dq=u8(M, _pitch(N)), de=u8(M, ex(N)),
             dqt=u8(N, tp), det=u8(N, (tp // 128 + 3) // 4 * 4),
             wq=u8(G, K, _pitch(N)), we=u8(G, K, ex(N)), wqt=u8(G, N, _pitch(K)), wet=u8(G, N, ex(K)),
             dx=empty(M, K), dw=empty(G, K, N), db=empty(G, N),
             ws=empty(4 * (tp // 128) * (N + 64) + 65536, dtype=torch.uint8))
    return s


# ------------------------------------------------------------------ one pass
def _plain_norm(s):
    f, C = _factor(s, s["rng"]), s["cols"]
    if s["op"] == "norm":
        h = s["x"].float() if f is None else s["x"].float() * f
        h = h if s["r"] is None else h + s["r"].float()
        mean = h.mean(-1, keepdim=True)
        d = h - mean
        rstd = torch.rsqrt(d.square().mean(-1, keepdim=True) + EPS)
        y = d * rstd * s["gamma"].float() + s["beta"].float()
        dt = s["x"].dtype
        return {"h": h.to(dt), "y": y.to(dt), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    dt = s["dy"].dtype
    xh = (s["h"].float() - s["mean"].unsqueeze(1)) * s["rstd"].unsqueeze(1)
    dy = s["dy"].float()
    t = dy * s["gamma"].float()
    dr = s["rstd"].unsqueeze(1) * (t - t.sum(-1, keepdim=True) / C - xh * ((t * xh).sum(-1, keepdim=True) / C))
    if s["dh"] is not None:
        dr = dr + s["dh"].float()
    out = {"dr": dr.to(dt)}
    if f is not None:
        out["dx"] = (dr * f).to(dt)
    out["dgamma"] = (dy * xh).double().sum(0).to(dt)
    out["dbeta"] = dy.double().sum(0).to(dt)
    return out


def _plain_route(s):
    T, k, E, C, S = s["tokens"], s["k"], s["experts"], s["cols"], s["tokens"] * s["k"]
    dt = s["x"].dtype
    expert = s["expert"].reshape(-1).long()
    key = torch.where((expert >= 0) & (expert < E), expert, torch.full_like(expert, E))
    source = torch.sort(key, stable=True).indices
    counts = (key.unsqueeze(0) == torch.arange(E, device="cuda").unsqueeze(1)).sum(1)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(counts, 0)])
    place = torch.empty_like(source)
    place[source] = torch.arange(S, device="cuda")
    live = place < offsets[E]
    row_live = (torch.arange(S, device="cuda") < offsets[E]).unsqueeze(1)
    position = torch.where(live, place, torch.full_like(place, -1))
    out = {"offsets": offsets.int(), "position": position.int().reshape(T, k),
           "source": torch.where(row_live[:, 0], source, torch.full_like(source, -1)).int()}
    out["rows"] = torch.where(row_live, s["x"][source // k], torch.zeros((), dtype=dt, device="cuda"))
    w = torch.where(live.reshape(T, k), s["weight"], torch.zeros((), device="cuda"))
    acc = torch.zeros((T, C), dtype=torch.float32, device="cuda")
    dx = torch.zeros_like(acc)
    dweight = torch.empty_like(s["weight"])
    for j in range(k):
        at, ok = place.reshape(T, k)[:, j], live.reshape(T, k)[:, j : j + 1]
        y = torch.where(ok, s["y"][at].float(), 0.0)
        acc += w[:, j : j + 1] * y
        if s["train"]:
            dweight[:, j] = (s["dout"].float() * y).sum(-1)
            dx += torch.where(ok, s["drows"][at].float(), 0.0)
    out["out"] = acc.to(dt)
    if s["train"]:
        dy = s["weight"].reshape(-1)[source].unsqueeze(1) * s["dout"][source // k].float()
        out["dy"] = torch.where(row_live, dy, 0.0).to(dt)
        out["dweight"], out["dx"] = dweight, dx.to(dt)
    return out


def _plain_f8(s):
    dt, grad = s["x"].dtype, s["grad"]
    bias = None if s["bias"] is None else s["bias"].float()
    if not s["ragged"]:
        x = _round8(s["x"].float(), "e4m3").transpose(0, 1)                # [G, M, K]
        w = _values(s["w"].view(F8["e4m3"]), s["we"][..., : _pitch(s["K"]) // 128].int() - 127, s["K"])
        out = torch.bmm(x, w.transpose(1, 2))
        out = out if bias is None else out + bias.unsqueeze(1)
        return {"out": out.transpose(0, 1).to(dt)}
    out = torch.empty(s["out"].shape, dtype=dt, device="cuda")
    if s["train"]:
        dx = torch.empty(s["dx"].shape, dtype=dt, device="cuda")
        dw, db = torch.zeros_like(s["dw"]), torch.zeros_like(s["db"])
    r = 0
    for e, n in enumerate(s["sizes"]):
        x = s["x"][r : r + n].float()
        if s["train"]:
            wf = s["w"][e].float()
            w = _round8(wf.t().contiguous(), "e4m3")                        # [N, K]
        else:
            w = _values(s["w"][e].view(F8["e4m3"]), s["we"][e, :, : _pitch(s["K"]) // 128].int() - 127, s["K"])
        c = _round8(x, "e4m3") @ w.t()
        out[r : r + n] = (c if bias is None else c + bias[e]).to(dt)
        if s["train"] and n:
            dy = s["dy"][r : r + n].float()
            dx[r : r + n] = (_round8(dy, grad) @ _round8(wf, "e4m3").t()).to(dt)
            dw[e] = (_round8(x.t().contiguous(), "e4m3") @ _round8(dy.t().contiguous(), grad).t()).to(dt)
            db[e] = dy.double().sum(0).to(dt)
        r += n
    return {"out": out, "dx": dx, "dw": dw, "db": db} if s["train"] else {"out": out}


def _own_f8(B, s):
    M, G, K, N, dt = s["M"], s["G"], s["K"], s["N"], s["dtype"]
    off = s.get("offsets")
    fwd = B.make_layer_f8(M, G, K, N, dt, "e4m3", "e4m3")
    if not s["train"]:
        rows = B.make_rows(M if s["ragged"] else M * G, K, dt)
        B.check(B.rmx_quant_f8(rows, "e4m3", s["x"], s["q"], s["e"]))
        B.check(B.rmx_linear_f8(fwd, off, s["q"], s["e"], s["w"], s["we"], s["bias"], None, s["out"]))
        return {"out": s["out"]}
    ws, nws = s["ws"], s["ws"].numel()
    weights, acts, grads = (B.make_groups(*v, dt, order) for v, order in
                            (((K, G, N), "groups"), ((M, G, K), "ragged"), ((M, G, N), "ragged")))
    B.check(B.rmx_quant_f8_groups(weights, "e4m3", None, s["w"], s["wq"], s["we"], s["wqt"], s["wet"], None, ws, nws))
    B.check(B.rmx_quant_f8_groups(acts, "e4m3", off, s["x"], s["q"], s["e"], s["qt"], s["et"], None, ws, nws))
    B.check(B.rmx_linear_f8(fwd, off, s["q"], s["e"], s["wqt"], s["wet"], s["bias"], None, s["out"]))
    B.check(B.rmx_quant_f8_groups(grads, s["grad"], off, s["dy"], s["dq"], s["de"], s["dqt"], s["det"], s["db"], ws,
                                  nws))
    back = B.make_layer_f8(M, G, N, K, dt, s["grad"], "e4m3")
    B.check(B.rmx_linear_f8(back, off, s["dq"], s["de"], s["wq"], s["we"], None, None, s["dx"]))
    wgrad = B.make_layer_f8(M, G, K, N, dt, "e4m3", s["grad"])
    B.check(B.rmx_wgrad_f8(wgrad, off, s["qt"], s["et"], s["dqt"], s["det"], s["dw"]))
    return {"out": s["out"], "dx": s["dx"], "dw": s["dw"], "db": s["db"]}


def run(state):
    s, op = state, state["op"]
    if not own:
        if op in ("norm", "norm_bwd"):
            return _plain_norm(s)
        if op == "dropout":
            f = _factor(s, s["rng"])
            v = s["x"].float() * f
            return {"out": (v if s["r"] is None else v + s["r"].float()).to(s["x"].dtype)}
        return _plain_route(s) if op == "route" else _plain_f8(s)
    from ffn_block_gb300 import binding as B
    if op == "f8":
        return _own_f8(B, s)
    if op == "route":
        r = B.make_routes(s["tokens"], s["k"], s["experts"], s["cols"], s["dtype"])
        B.check(B.rmx_expert_sort(r, s["expert"], s["offsets"], s["position"], s["source"], s["ws"], s["ws"].numel()))
        B.check(B.rmx_expert_gather(r, s["source"], s["x"], s["rows"], "e4m3", None, None))
        B.check(B.rmx_expert_combine(r, s["position"], s["weight"], s["y"], s["out"]))
        out = {n: s[n] for n in ("offsets", "position", "source", "rows", "out")}
        if s["train"]:
            B.check(B.rmx_expert_combine_backward(r, s["position"], s["weight"], s["dout"], s["y"], s["dy"],
                                                  s["dweight"]))
            B.check(B.rmx_expert_combine(r, s["position"], None, s["drows"], s["dx"]))
            out.update({n: s[n] for n in ("dy", "dweight", "dx")})
        return out
    shape = B.make_rows(s["rows"], s["cols"], s["dtype"])
    drop = B.make_drop(s["p"], s["rng"])
    if op == "dropout":
        B.check(B.rmx_dropout(shape, drop, s["x"], s["r"], s["out"]))
        return {"out": s["out"]}
    if op == "norm":
        B.check(B.rmx_layer_norm(shape, EPS, drop, s["x"], s["r"], s["gamma"], s["beta"], s["h"], s["y"], s["mean"],
                                 s["rstd"]))
        return {n: s[n] for n in ("h", "y", "mean", "rstd")}
    B.check(B.rmx_layer_norm_backward(shape, drop, s["dy"], s["dh"], s["h"], s["mean"], s["rstd"], s["gamma"], s["dr"],
                                      s["dx"], s["dgamma"], s["dbeta"], s["ws"], s["ws"].numel()))
    return {n: s[n] for n in ("dr", "dx", "dgamma", "dbeta") if s[n] is not None}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, e = case["op"], 4 if case["dtype"] == "f32" else 2
    if op in ("norm", "norm_bwd", "dropout"):
        R, C = case["rows"], case["cols"]
        n, res = R * C, 1 if case["resid"] else 0
        if op == "dropout":   # x (, r) in; out
            return {"bytes": n * e * (2 + res), "flops": 2 * n}
        if op == "norm":      # x (, r) in; h, y, two statistics out
            return {"bytes": n * e * (3 + res) + 2 * C * e + 8 * R, "flops": 8 * n}
        drop = 1 if case["p"] > 0 else 0  # dy (, dh), h in; dr (, dx) out
        return {"bytes": n * e * (3 + res + drop) + 3 * C * e + 8 * R, "flops": 12 * n}
    if op == "route":
        T, k, C = case["tokens"], case["k"], case["cols"]
        S = T * k
        b = 4 * S + 8 * S + 4 * case["experts"]      # ids in; the order and its inverse out
        b += T * C * e + S * C * e                   # gather
        b += S * C * e + 4 * S + T * C * e           # combine
        if case["train"]:
            b += T * C * e + 2 * S * C * e + 4 * S   # dout, y in; dy, dweight out
            b += S * C * e + T * C * e               # drows in; dx out
        return {"bytes": b, "flops": 2 * S * C * (3 if case["train"] else 1)}
    M, G, K, N = (case[n] for n in "MGKN")
    R = M if case["ragged"] else M * G
    b = R * (K + N) * e + (G * N * e if case["bias"] else 0)
    if not case["train"]:
        return {"bytes": b + G * N * (K + -(-K // 128)), "flops": 2 * R * K * N}
    b += G * K * N * e                               # the weights, once
    b += R * (N + K) * e + G * K * N * e + G * N * e  # dy in; dx, dw, db out
    return {"bytes": b, "flops": 6 * R * K * N}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_factor(case, s):
    """Dropout's factors in float64, by the words of the generator on the host."""
    t = int(np.rint(case["p"] * 65536.0))
    if t == 0:
        return 1.0
    R, C = case["rows"], case["cols"]
    seed, off = (int(v) for v in s["rng"].tolist())
    n = -(-C // 8)
    lo, sh = np.uint64(MASK), np.uint64(32)
    word = [np.tile(np.arange(n, dtype=np.uint64), R), np.repeat(np.arange(R, dtype=np.uint64), n),
            np.uint64(off & MASK), np.uint64(off >> 32)]
    key = [seed & MASK, seed >> 32]
    for _ in range(10):
        p0, p1 = word[0] * np.uint64(0xD2511F53), word[2] * np.uint64(0xCD9E8D57)
        word = [(p1 >> sh) ^ word[1] ^ np.uint64(key[0]), p1 & lo, (p0 >> sh) ^ word[3] ^ np.uint64(key[1]), p0 & lo]
        key = [(key[0] + 0x9E3779B9) & MASK, (key[1] + 0xBB67AE85) & MASK]
    halves = np.stack([np.broadcast_to(w, R * n).astype(np.uint32) for w in word], -1).view(np.uint16)  # little-endian
    keep = torch.from_numpy((halves.reshape(R, n * 8)[:, :C] >= t).astype(np.uint8)).cuda()
    return keep.double() / ((65536 - t) / 65536)


def _exact8(x, fmt):
    """x [R, C] float64 rounded to the 8-bit rows' values."""
    top, bits, low = (448.0, 3, -6) if fmt == "e4m3" else (57344.0, 2, -14)
    out = torch.empty_like(x)
    for c in range(0, x.shape[-1], 128):
        b = x[..., c : c + 128]
        amax = b.abs().amax(-1, keepdim=True)
        e = torch.floor(torch.log2((amax / top).clamp_min(1e-300)) - 1e-9).clamp(-127, 127)
        e = torch.where(amax > top * _pow2(e), e + 1, e).clamp(-127, 127)
        unit = _pow2(e)
        v = b / unit
        step = torch.floor(torch.log2(v.abs().clamp_min(1e-300)) + 1e-12).clamp_min(low) - bits
        step = _pow2(step)
        out[..., c : c + 128] = torch.round(v / step) * step * unit
    return out


def _exact_weights(q, e, cols):
    v = q.view(F8["e4m3"]).double()[..., :cols]
    return v * _pow2(e.long() - 127).repeat_interleave(128, -1)[..., :cols]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    d = lambda t: None if t is None else t.double()  # noqa: E731
    if op in ("norm", "norm_bwd", "dropout"):
        f = _exact_factor(case, s)
        if op == "dropout":
            return {"out": s["x"].double() * f + (0.0 if s["r"] is None else s["r"].double())}
        if op == "norm":
            h = s["x"].double() * f + (0.0 if s["r"] is None else s["r"].double())
            mean = h.sum(-1) / case["cols"]
            rstd = 1 / ((h - mean[:, None]).pow(2).sum(-1) / case["cols"] + EPS).sqrt()
            return {"h": h, "y": (h - mean[:, None]) * rstd[:, None] * d(s["gamma"]) + d(s["beta"]), "mean": mean,
                    "rstd": rstd}
        # y_i = gamma_i (h_i - mu) rho: dr_j = rho (g_j - sum_i g_i / C - xh_j sum_i g_i xh_i / C), g = gamma dy
        rho, mu, dy = d(s["rstd"])[:, None], d(s["mean"])[:, None], d(s["dy"])
        xh = (d(s["h"]) - mu) * rho
        g1 = torch.einsum("rc,c->r", dy, d(s["gamma"]))[:, None] / case["cols"]
        g2 = torch.einsum("rc,rc,c->r", dy, xh, d(s["gamma"]))[:, None] / case["cols"]
        dr = (dy * d(s["gamma"]) - g1 - xh * g2) * rho
        dr = dr if s["dh"] is None else dr + d(s["dh"])
        out = {"dr": dr} if case["p"] == 0 else {"dr": dr, "dx": dr * f}
        out["dgamma"], out["dbeta"] = torch.einsum("rc,rc->c", dy, xh), dy.sum(0)
        return out
    if op == "route":
        T, k, E, C = (case[n] for n in ("tokens", "k", "experts", "cols"))
        ids = s["expert"].cpu().numpy().reshape(-1)
        # the slots in order, expert by expert
        order = np.concatenate([np.flatnonzero(ids == e) for e in range(E)])
        offsets = np.concatenate([[0], np.cumsum([np.count_nonzero(ids == e) for e in range(E)])])
        n, S = len(order), T * k
        source, position = np.full(S, -1, np.int32), np.full(S, -1, np.int32)
        source[:n] = order
        position[order] = np.arange(n)
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        at = dev(order.astype(np.int64))
        out = {"offsets": dev(offsets.astype(np.int32)), "position": dev(position.reshape(T, k)), "source": dev(source)}
        rows = torch.zeros((S, C), dtype=torch.float64, device="cuda")
        rows[:n] = d(s["x"])[at // k]
        w = d(s["weight"]).reshape(-1)[at][:, None]
        acc = lambda v: torch.zeros((T, C), dtype=torch.float64, device="cuda").index_add_(0, at // k, v)  # noqa: E731
        y = d(s["y"][:n])
        out.update(rows=rows, out=acc(w * y))
        if case["train"]:
            dy, dweight = torch.zeros_like(rows), torch.zeros(S, dtype=torch.float64, device="cuda")
            up = d(s["dout"])[at // k]
            dy[:n] = w * up
            dweight[at] = torch.einsum("rc,rc->r", up, y)
            out.update(dy=dy, dweight=dweight.reshape(T, k), dx=acc(d(s["drows"][:n])))
        return out
    M, G, K, N = (case[n] for n in "MGKN")
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    res = {"out": out}
    if case["train"]:
        for n in ("dx", "dw", "db"):
            res[n] = torch.zeros(s[n].shape, dtype=torch.float64, device="cuda")
    starts = [0, *np.cumsum(s["sizes"]).tolist()] if case["ragged"] else None
    for g in range(G):
        pick = slice(starts[g], starts[g + 1]) if case["ragged"] else (slice(None), g)
        x = d(s["x"][pick])
        if x.shape[0] == 0:
            continue
        w = _exact8(d(s["w"][g]).t().contiguous(), "e4m3") if case["train"] else _exact_weights(s["w"][g], s["we"][g], K)
        out[pick] = _exact8(x, "e4m3") @ w.t() + (0.0 if s["bias"] is None else d(s["bias"][g]))
        if case["train"]:
            dy = d(s["dy"][pick])
            res["dx"][pick] = _exact8(dy, case["grad"]) @ _exact8(d(s["w"][g]), "e4m3").t()
            xt, dyt = _exact8(x.t().contiguous(), "e4m3"), _exact8(dy.t().contiguous(), case["grad"])
            res["dw"][g] = xt @ dyt.t()
            res["db"][g] = dy.sum(0)
    return res
