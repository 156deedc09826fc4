"""What is measured of the 8-bit operators: their cases, plain forms and calls.

Five operators around an 8-bit per-token layer, each in its plain form
(elementary torch operations in float32, rounded once at the end) and as the
library's own call:

  rms     h = x + r; n = h / sqrt(mean(h^2) + eps) * gamma, quantised to int8
          with one float32 scale per row, and read back as the values it
          stands for
  rms_bwd gradients of the norm (dx, dgamma) from an 8-bit checkpoint of h
  linear  C[m,g] = (A[m,g] @ W[g]) * sa[m,g] * sw[g] + bias[g] (+ resid), A
          and W int8, one scale per token and per channel
  ckpt    an activation packed into an 8-bit checkpoint and unpacked again
  wgrad   dW[g] = X[:,g]^T @ dY[:,g] and db[g] = sum dY[:,g], X read from its
          8-bit checkpoint

Formats.  int8 rows are padded with zeros to a pitch of a multiple of 32
bytes.  `q8 rows`: value = q * scale[row], scale = max|row| / 127.  `8-bit
checkpoint`: value = q * 2^e with one int8 exponent e per 32 columns, the
smallest e for which no value of the group rounds past 127 steps, held in a
range that keeps every value exact in the storage type.
"""

import math

import torch

own = False

EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EXP_RANGE = {"f32": (-126, 121), "bf16": (-126, 121), "f16": (-24, 9)}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # One token of a decode step: launch latency.
        dict(name="rms one token", op="rms", rows=1, cols=1280, dtype="bf16", resid=True),
        # Every row of the production block (B = 1024, T = 64, D = 1280).
        dict(name="rms production", op="rms", rows=65536, cols=1280, dtype="bf16", resid=True),
        # The same rows in training, the sum kept as a checkpoint.
        dict(name="rms_bwd production", op="rms_bwd", rows=65536, cols=1280, dtype="bf16", resid=True),
        # Odd row length, strict float32, one gradient only.
        dict(name="rms_bwd odd f32", op="rms_bwd", rows=3001, cols=513, dtype="f32", resid=False),
        # One sample served: the whole 8-bit w1 is streamed for 64 tokens.
        dict(name="linear one sample", op="linear", M=1, G=64, K=1280, N=5120, dtype="bf16", bias=True, resid=False),
        # A serving batch of the mid block's second layer.
        dict(name="linear batch 48", op="linear", M=48, G=32, K=1536, N=512, dtype="bf16", bias=True, resid=True),
        # The second layer of the ragged block, with its residual.
        dict(name="linear ragged f16", op="linear", M=1000, G=40, K=3600, N=1200, dtype="f16", bias=True, resid=True),
        # The first layer of the production block: the largest product.
        dict(name="linear production", op="linear", M=1024, G=64, K=1280, N=5120, dtype="bf16", bias=True, resid=False),
        # The production block's activations kept for the backward.
        dict(name="ckpt production", op="ckpt", rows=65536, cols=1280, dtype="bf16"),
        # Odd rows of a small strict float32 block.
        dict(name="ckpt odd f32", op="ckpt", rows=1024, cols=333, dtype="f32"),
        # Weight gradient of the production block's first layer.
        dict(name="wgrad production", op="wgrad", M=1024, G=64, K=1280, N=5120, dtype="bf16"),
        # Weight gradient of a small odd layer.
        dict(name="wgrad odd f16", op="wgrad", M=203, G=9, K=81, N=243, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rms", "rms_bwd", "linear", "linear", "ckpt", "wgrad"])
    if op in ("rms", "rms_bwd", "ckpt"):
        cols = _log(rng, 16, 8192)
        if rng.random() < 0.6:
            cols = max(16, cols // 8 * 8)
        rows = _log(rng, 1, max(2, min(65536, 80_000_000 // cols)))
        dtype = rng.choice(["bf16", "f16"] if op == "rms" else ["bf16", "f16", "f32"])
        c = dict(op=op, rows=rows, cols=cols, dtype=dtype)
        if op != "ckpt":
            c["resid"] = rng.random() < 0.5
        return c
    M, G = _log(rng, 1, 1024), _log(rng, 1, 64)
    K, N = _log(rng, 48, 3840), _log(rng, 48, 5120)
    if rng.random() < 0.6:
        K, N = max(48, K // 16 * 16), max(48, N // 16 * 16)
    while M * G * K * N > 1024 * 64 * 1280 * 5120 or G * K * N > 64 * 1280 * 5120:
        G = max(1, G // 2)
    c = dict(op=op, M=M, G=G, K=K, N=N, dtype=rng.choice(["bf16", "f16", "f32"]))
    if op == "wgrad" and c["dtype"] == "f32":
        c["dtype"] = "bf16"
    if op == "linear":
        c["bias"], c["resid"] = rng.random() < 0.7, rng.random() < 0.4
    return c


# ------------------------------------------------------------------ formats
def _pitch(cols):
    return (cols + 31) // 32 * 32


def _pad(x, pitch):
    """x [..., C] as a contiguous [..., pitch] tensor with zeros behind C."""
    out = torch.zeros(*x.shape[:-1], pitch, dtype=x.dtype, device=x.device)
    out[..., : x.shape[-1]] = x
    return out


def _ck_pack(x, dtype):
    """Checkpoint of x [R, C] (already in float32/64): int8 [R, P] and int8 exponents [R, P / 32]."""
    lo, hi = EXP_RANGE[dtype]
    g = _pad(x, _pitch(x.shape[-1])).reshape(x.shape[0], -1, 32)
    amax = g.abs().amax(-1)
    m, k = torch.frexp(amax)                   # amax = m * 2^k, m in [0.5, 1)
    e = k - 7 + (m > 127.5 / 128).to(k.dtype)  # amax / 2^e <= 127.5
    e = torch.where(amax > 0, e, torch.full_like(e, lo)).clamp(lo, hi)
    q = torch.round(torch.ldexp(g, -e.unsqueeze(-1))).clamp(-127, 127)
    return q.reshape(x.shape[0], -1).to(torch.int8), e.to(torch.int8)


def _ck_values(q, e, cols, f):
    """The values a checkpoint stands for, in the float type f."""
    v = torch.ldexp(q.to(f).reshape(q.shape[0], -1, 32), e.to(torch.int32).unsqueeze(-1))
    return v.reshape(q.shape[0], -1)[:, :cols]


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, shape, dt):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)


def prepare(case, seed):
    g, dt, op = _gen(seed), DTYPES[case["dtype"]], case["op"]
    s = dict(case)
    empty = lambda *shape, dtype=dt: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    if op in ("rms", "rms_bwd", "ckpt"):
        R, C = case["rows"], case["cols"]
        P = _pitch(C)
        s["x"] = _randn(g, (R, C), dt)
        if op == "ckpt":
            # a few columns with larger values, as activations have
            s["x"][:, :: 61] *= 12
            s.update(q=empty(R, P, dtype=torch.int8), e=empty(R, P // 32, dtype=torch.int8), out=empty(R, C))
            return s
        s["gamma"] = (1 + 0.2 * torch.randn(C, generator=g, device="cuda")).to(dt)
        if op == "rms":
            s["r"] = _randn(g, (R, C), dt) if case["resid"] else None
            s.update(h=empty(R, C), q=empty(R, P, dtype=torch.int8), scale=empty(R, dtype=torch.float32),
                     rstd=empty(R, dtype=torch.float32), n=empty(R, C))
            return s
        h = s.pop("x").float()
        s["q"], s["e"] = _ck_pack(h, case["dtype"])
        s["rstd"] = torch.rsqrt(h.square().mean(-1) + EPS)
        del h
        s["dn"] = _randn(g, (R, C), dt)
        s["dh"] = _randn(g, (R, C), dt) if case["resid"] else None
        # scratch: up to 512 partial rows of float32 column sums
        s.update(dx=empty(R, C), dgamma=empty(C), ws=empty(512 * C * 4 + 4096, dtype=torch.uint8))
        return s
    M, G, K, N = (case[k] for k in "MGKN")
    P = _pitch(K)
    if op == "linear":
        ints = lambda *shape: _pad(torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8), P)  # noqa: E731
        s["a"], s["w"] = ints(M, G, K), ints(G, N, K)
        s["sa"] = 0.01 + 0.02 * torch.rand(M, G, generator=g, device="cuda")
        s["sw"] = (0.5 + torch.rand(G, N, generator=g, device="cuda")) / (127 * math.sqrt(K))
        s["bias"] = _randn(g, (G, N), dt) if case["bias"] else None
        s["res"] = _randn(g, (M, G, N), dt) if case["resid"] else None
        s["out"] = empty(M, G, N)
        return s
    q, e = _ck_pack(torch.randn((M * G, K), generator=g, device="cuda"), case["dtype"])
    s["q"], s["e"] = q.reshape(M, G, P), e.reshape(M, G, P // 32)
    s["dy"] = _randn(g, (M, G, N), dt)
    K8, N8 = (K + 7) // 8 * 8, (N + 7) // 8 * 8
    # scratch: the unpacked activation, padded copies of dy and dW, partial column sums
    nbytes = 2 * (M * G * (K8 + N8) + G * K8 * N8) + 4 * 64 * G * N8 + 65536
    s.update(dw=empty(G, K, N), db=empty(G, N), ws=empty(nbytes, dtype=torch.uint8))
    return s


# ------------------------------------------------------------------ one pass
def _rms_math(x, r, gamma, f):
    h = x.to(f) if r is None else x.to(f) + r.to(f)
    rstd = torch.rsqrt(h.square().mean(-1) + EPS)
    n = h * rstd.unsqueeze(-1) * gamma.to(f)
    scale = n.abs().amax(-1) / 127
    q = torch.round(n / torch.where(scale > 0, scale, torch.ones_like(scale)).unsqueeze(-1)).clamp(-127, 127)
    return h, rstd, scale, q * scale.unsqueeze(-1)


def _rms_bwd_math(h, rstd, gamma, dn, dh, f):
    xhat = h * rstd.to(f).unsqueeze(-1)
    dn = dn.to(f)
    t = dn * gamma.to(f)
    dx = rstd.to(f).unsqueeze(-1) * (t - xhat * (t * xhat).mean(-1, keepdim=True))
    return dx if dh is None else dx + dh.to(f), (dn * xhat).sum(0)


def _linear_math(s, f):
    K = s["K"]
    c = torch.bmm(s["a"][..., :K].permute(1, 0, 2).to(f), s["w"][..., :K].transpose(1, 2).to(f)).permute(1, 0, 2)
    c = c * s["sa"].to(f).unsqueeze(-1) * s["sw"].to(f)
    if s["bias"] is not None:
        c = c + s["bias"].to(f)
    return c if s["res"] is None else c + s["res"].to(f)


def _wgrad_math(s, f):
    M, G, K = s["M"], s["G"], s["K"]
    x = _ck_values(s["q"].reshape(M * G, -1), s["e"].reshape(M * G, -1), K, f).reshape(M, G, K)
    dy = s["dy"].to(f)
    return torch.bmm(x.permute(1, 2, 0), dy.permute(1, 0, 2)), dy.sum(0)


def run(state):
    s, op = state, state["op"]
    dt = DTYPES[s["dtype"]]
    if own:
        return _run_own(s, op)
    f = torch.float32
    if op == "rms":
        h, rstd, scale, v = _rms_math(s["x"], s["r"], s["gamma"], f)
        return {"h": h.to(dt), "rstd": rstd, "scale": scale, "n": v.to(dt)}
    if op == "rms_bwd":
        dx, dg = _rms_bwd_math(_ck_values(s["q"], s["e"], s["cols"], f), s["rstd"], s["gamma"], s["dn"], s["dh"], f)
        return {"dx": dx.to(dt), "dgamma": dg.to(dt)}
    if op == "linear":
        return {"c": _linear_math(s, f).to(dt)}
    if op == "ckpt":
        return {"x": _ck_values(*_ck_pack(s["x"].to(f), s["dtype"]), s["cols"], f).to(dt)}
    dw, db = _wgrad_math(s, f)
    return {"dw": dw.to(dt), "db": db.to(dt)}


def _run_own(s, op):
    from ffn_block_gb300 import binding as B

    if op in ("rms", "rms_bwd", "ckpt"):
        rows = B.make_rows(s["rows"], s["cols"], s["dtype"])
        if op == "rms":
            B.check(B.rmx_rms_norm_q8(rows, EPS, s["x"], s["r"], s["gamma"], s["h"], None, s["q"], s["scale"], s["rstd"]))
            B.check(B.rmx_dequant_rows_q8(rows, s["q"], s["scale"], s["n"]))
            return {"h": s["h"], "rstd": s["rstd"], "scale": s["scale"], "n": s["n"]}
        if op == "rms_bwd":
            B.check(B.rmx_rms_norm_backward(rows, s["dn"], s["dh"], None, s["q"], s["e"], s["rstd"], s["gamma"], s["dx"],
                                            s["dgamma"], s["ws"], s["ws"].numel()))
            return {"dx": s["dx"], "dgamma": s["dgamma"]}
        B.check(B.rmx_ckpt8_pack(rows, s["x"], s["q"], s["e"]))
        B.check(B.rmx_ckpt8_unpack(rows, s["q"], s["e"], s["out"]))
        return {"x": s["out"]}
    layer = B.make_layer(s["M"], s["G"], s["K"], s["N"], s["dtype"])
    if op == "linear":
        B.check(B.rmx_linear_q8(layer, s["a"], s["sa"], s["w"], s["sw"], s["bias"], s["res"], s["out"]))
        return {"c": s["out"]}
    B.check(B.rmx_ckpt8_wgrad(layer, s["q"], s["e"], s["dy"], s["dw"], s["db"], s["ws"], s["ws"].numel()))
    return {"dw": s["dw"], "db": s["db"]}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, e = case["op"], 4 if case["dtype"] == "f32" else 2
    if op in ("rms", "rms_bwd", "ckpt"):
        R, C = case["rows"], case["cols"]
        n = R * C
        q = n + R * -(-C // 32)  # an 8-bit checkpoint with its exponents
        streams = 1 if case.get("resid") else 0
        if op == "rms":    # x (, r) in; h, int8, its values, two row statistics out
            return {"bytes": n * e * (3 + streams) + n + C * e + 8 * R, "flops": 8 * n}
        if op == "rms_bwd":  # dn (, dh), checkpoint in; dx, dgamma out
            return {"bytes": n * e * (2 + streams) + q + 2 * C * e + 4 * R, "flops": 10 * n}
        return {"bytes": 2 * n * e + q, "flops": 4 * n}
    M, G, K, N = (case[k] for k in "MGKN")
    if op == "linear":
        b = M * G * K + G * N * K + 4 * G * (M + N) + M * G * N * e * (2 if case["resid"] else 1)
        return {"bytes": b + (G * N * e if case["bias"] else 0), "flops": 2 * M * G * K * N}
    return {"bytes": M * G * (K + -(-K // 32)) + M * G * N * e + G * K * N * e + G * N * e, "flops": 2 * M * G * K * N}


# ------------------------------------------------------------------ the definitions in 64 bits
def _power(e):
    return torch.pow(torch.tensor(2.0, dtype=torch.float64, device=e.device), e.double())


def _exact_ck(q, e, cols):
    return (q.double() * _power(e).repeat_interleave(32, -1))[..., :cols]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    d = lambda t: None if t is None else t.double()  # noqa: E731
    if op == "rms":
        x, r, g = d(s["x"]), d(s["r"]), d(s["gamma"])
        h = x if r is None else x + r
        ms = (h * h).sum(-1) / case["cols"] + EPS
        n = h / ms.sqrt()[:, None] * g
        scale = n.abs().max(-1).values / 127
        v = (n / scale.clamp_min(1e-300)[:, None]).round() * scale[:, None]
        return {"h": h, "rstd": 1 / ms.sqrt(), "scale": scale, "n": v}
    if op == "rms_bwd":
        # y = gamma * h * rho with rho = mean(h^2)^(-1/2) as kept in rstd:
        # dx_j = rho * gamma_j * dn_j - rho^3 * h_j / C * sum_i(gamma_i * dn_i * h_i)
        h, rho, g, dn = _exact_ck(s["q"], s["e"], case["cols"]), d(s["rstd"])[:, None], d(s["gamma"]), d(s["dn"])
        dot = torch.einsum("rc,rc,c->r", dn, h, g)[:, None]
        dx = rho * g * dn - rho**3 * h * dot / case["cols"]
        return {"dx": dx if s["dh"] is None else dx + d(s["dh"]), "dgamma": torch.einsum("rc,rc,r->c", dn, h, rho[:, 0])}
    if op == "ckpt":
        x, out = d(s["x"]), torch.empty_like(s["x"], dtype=torch.float64)
        lo, hi = EXP_RANGE[case["dtype"]]
        for c in range(0, case["cols"], 32):
            v = x[:, c:c + 32]
            top = v.abs().max(-1).values
            # 1e-9: a power of two's logarithm may come out a hair above the integer
            e = torch.ceil(torch.log2(top.clamp_min(1e-300) / 127.5) - 1e-9).clamp(lo, hi)
            step = _power(e)[:, None]
            out[:, c:c + 32] = (v / step).round().clamp(-127, 127) * step
        return {"x": out}
    M, G, K = case["M"], case["G"], case["K"]
    if op == "linear":
        out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
        for g in range(G):
            c = d(s["a"][:, g, :K]) @ d(s["w"][g, :, :K]).t()
            c = c * d(s["sa"][:, g])[:, None] * d(s["sw"][g])[None, :]
            if s["bias"] is not None:
                c += d(s["bias"][g])
            if s["res"] is not None:
                c += d(s["res"][:, g])
            out[:, g] = c
        return {"c": out}
    dw = torch.empty(s["dw"].shape, dtype=torch.float64, device="cuda")
    for g in range(G):
        dw[g] = _exact_ck(s["q"][:, g], s["e"][:, g], K).t() @ d(s["dy"][:, g])
    return {"dw": dw, "db": d(s["dy"]).sum(0)}
