"""Plain float64 definitions of the 8-bit operators (numpy).

Written out from the formulas; shares no code with the CUDA path.  Arrays are
float64 unless they hold integers.
"""

import numpy as np

GROUP = 32
EXP_RANGE = {"f32": (-126, 121), "bf16": (-126, 121), "f16": (-24, 9)}
NAN_EXP = 127


def pitch(cols: int) -> int:
    return -(-cols // GROUP) * GROUP


def quant_rows(x):
    """q8 rows of x [R, C]: int8 [R, pitch], scale [R]."""
    R, C = x.shape
    q = np.zeros((R, pitch(C)), np.int8)
    scale = np.zeros(R)
    for r in range(R):
        if not np.all(np.isfinite(x[r])):
            scale[r] = np.nan
            continue
        top = np.max(np.abs(x[r]))
        if top > 0:
            scale[r] = top / 127.0
            q[r, :C] = np.rint(x[r] / scale[r])
    return q, scale


def rms_norm(x, r, gamma, eps):
    """h, rstd and the normalised rows."""
    h = x if r is None else x + r
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=-1) + eps)
    return h, rstd, h * rstd[:, None] * gamma


def rms_norm_backward(h, rstd, gamma, dn, dh):
    xh = h * rstd[:, None]
    t = dn * gamma
    dx = rstd[:, None] * (t - xh * np.mean(t * xh, axis=-1, keepdims=True))
    return (dx if dh is None else dx + dh), np.sum(dn * xh, axis=0)


def ckpt_pack(x, dtype):
    """8-bit checkpoint of x [R, C]: int8 [R, pitch], exponents [R, pitch / 32]."""
    R, C = x.shape
    P = pitch(C)
    lo, hi = EXP_RANGE[dtype]
    q = np.zeros((R, P), np.int8)
    e = np.zeros((R, P // GROUP), np.int8)
    for r in range(R):
        for g in range(P // GROUP):
            v = x[r, g * GROUP:min(C, (g + 1) * GROUP)]
            if not np.all(np.isfinite(v)):
                e[r, g] = NAN_EXP
                continue
            top = np.max(np.abs(v))
            k = lo
            while k < hi and top / 2.0 ** k > 127.5:
                k += 1
            e[r, g] = k
            q[r, g * GROUP:g * GROUP + len(v)] = np.clip(np.rint(v / 2.0 ** k), -127, 127)
    return q, e


def ckpt_values(q, e, cols):
    e = e.astype(np.float64)
    step = np.where(e == NAN_EXP, np.nan, 2.0 ** e)
    return (q.astype(np.float64) * np.repeat(step, GROUP, axis=-1))[..., :cols]


def weight_q8(w):
    """w [G, K, N] -> int8 [G, N, pitch(K)], scale [G, N]."""
    G, K, N = w.shape
    q = np.zeros((G, N, pitch(K)), np.int8)
    scale = np.zeros((G, N))
    for g in range(G):
        q[g], scale[g] = quant_rows(np.ascontiguousarray(w[g].T))
    return q, scale


def linear_q8(a, sa, w, sw, bias, resid, K):
    """a [M, G, P], w [G, N, P] int8 -> [M, G, N]."""
    s = np.einsum("mgk,gnk->mgn", a[..., :K].astype(np.float64), w[..., :K].astype(np.float64), optimize=True)
    out = s * sa[:, :, None] * sw[None]
    if bias is not None:
        out = out + bias
    return out if resid is None else out + resid


def wgrad(x, dy):
    """x [M, G, K], dy [M, G, N] -> dw [G, K, N], db [G, N]."""
    return np.einsum("mgk,mgn->gkn", x, dy, optimize=True), dy.sum(0)


def block_forward_q8(x, p, w1q, w1s, woutq, wouts):
    """The RankMixer block's forward with int8 contractions: out1 and hidden
    quantised per row, the weights given as int8 [T, N, pitch] and scales."""
    from . import rmx_oracle as O
    B, T, D = x.shape
    H = p["lnx_w"].shape[0]
    n0, _ = O.layer_norm(x, p["gamma0"], p["beta0"], 1e-3)
    out1, _ = O.layer_norm(O.token_mixer(n0) + x, p["gamma1"], p["beta1"], 1e-3)

    def product(a, wq, ws, bias, resid):
        K = a.shape[-1]
        q, s = quant_rows(a.reshape(B * T, K))
        return linear_q8(q.reshape(B, T, -1), s.reshape(B, T), wq, ws, bias, resid, K)

    Z = product(out1, w1q, w1s, p["b1"], None)
    U, G = Z[..., :H], Z[..., H:]
    u, _ = O.layer_norm(U, p["lnx_w"], p["lnx_b"], 1e-5)
    g, _ = O.layer_norm(G, p["lng_w"], p["lng_b"], 1e-5)
    s2 = product(u * O.silu(g), woutq, wouts, p["bout"], out1)
    return O.layer_norm(s2, p["gamma2"], p["beta2"], 1e-3)[0]
