"""Row passes of the 8-bit operators with more rows than their grids hold at once, so that every block takes several in
its loop: all rows against the definitions in float64 (torch, on whole arrays)."""

import numpy as np
import pytest
import torch

from ffn_block_gb300 import binding as B
from oracle import q8_oracle as Q

from q8_util import DT, E32, TINY, U, empty, ok, sync

pytestmark = pytest.mark.gpu
EPS = 1e-5


def randn(shape, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(DT[dt])


def near(got, ref, bound, what):
    over = (got.double() - ref).abs() - bound
    assert bool((over <= 0).all()), (what, float(over.max()), int((over > 0).sum()))


def pack(x, dt):
    """8-bit checkpoint of x (float64) by whole arrays."""
    R, C = x.shape
    lo, hi = Q.EXP_RANGE[dt]
    p = torch.zeros((R, Q.pitch(C)), dtype=torch.float64, device="cuda")
    p[:, :C] = x
    grp = p.view(R, -1, 32)
    m, k = torch.frexp(grp.abs().amax(-1))
    e = (k - 7 + (m > 127.5 / 128).int()).clamp(lo, hi)
    e = torch.where(m > 0, e, torch.full_like(e, lo))
    step = torch.exp2(e.double())[..., None]
    q = (grp / step).round().clamp(-127, 127)
    return q.view(R, -1).to(torch.int8), e.to(torch.int8), (q * step).view(R, -1)[:, :C]


# lanes and warps a row: 8, 16 and 32 lanes of one warp, four warps, sixteen with two and four blocks each; whole
# vectors and odd rows
@pytest.mark.parametrize("R,C,dt", [(160_000, 40, "bf16"), (160_000, 41, "f16"), (90_000, 100, "bf16"), (45_000, 300, "f16"),
                                    (45_000, 1001, "bf16"), (12_000, 1500, "bf16"), (12_000, 1501, "f32"),
                                    (6_000, 5000, "f16"), (6_000, 9000, "bf16"), (5_500, 9001, "bf16")])
def test_rms_norm(R, C, dt):
    x, r, g = randn((R, C), dt, 1), randn((R, C), dt, 2), (1 + 0.3 * randn(C, "f32", 3)).to(DT[dt])
    P = Q.pitch(C)
    h, y, q = empty((R, C), dt), empty((R, C), dt), empty((R, P), torch.int8)
    s, rstd, v = empty(R, torch.float32), empty(R, torch.float32), empty((R, C), dt)
    sh = B.make_rows(R, C, dt)
    ok(B.rmx_rms_norm_q8(sh, EPS, x, r, g, h, y, q, s, rstd))
    ok(B.rmx_dequant_rows_q8(sh, q, s, v))
    sync()
    rel = (160 / 2 + 10) * E32      # as counted in the tests of single rows
    for a in range(0, R, 16384):
        o = slice(a, a + 16384)
        rh = x[o].double() + r[o].double()
        rr = 1 / (rh.square().mean(-1) + EPS).sqrt()
        n = rh * rr[:, None] * g.double()
        step = n.abs().amax(-1) / 127
        near(h[o], rh, rh.abs() * (U[dt] + 2 * E32) + TINY[dt], "h")
        near(rstd[o], rr, rr * rel, "rstd")
        near(y[o], n, n.abs() * (U[dt] + rel) + TINY[dt], "y")
        near(s[o], step, step * rel, "scale")
        assert not q[o, C:].any()
        val = q[o, :C].double() * s[o].double()[:, None]
        near(val, n, (step * (0.5 + 127 * 2 * rel))[:, None], "values")
        near(v[o], val, val.abs() * (U[dt] + E32) + TINY[dt], "read back")


@pytest.mark.parametrize("ck", [True, False], ids=["checkpoint", "stored"])
@pytest.mark.parametrize("R,C,dt", [(40_000, 40, "bf16"), (40_000, 41, "f16"), (20_000, 96, "bf16"), (20_000, 101, "f32"),
                                    (15_000, 300, "f16"), (4_000, 1400, "bf16"), (2_000, 2501, "bf16"), (2_000, 5000, "f16"),
                                    (1_000, 9000, "bf16")])
def test_rms_norm_backward(R, C, dt, ck):
    h, dn, dh = randn((R, C), dt, 4), randn((R, C), dt, 5), randn((R, C), dt, 6)
    g = (1 + 0.3 * randn(C, "f32", 7)).to(DT[dt])
    q, e, hv = pack(h.double(), dt)
    if not ck:
        hv = h.double()
    rstd = (1 / (h.double().square().mean(-1) + EPS).sqrt()).float()
    sh = B.make_rows(R, C, dt)
    nb = B.rmx_rms_norm_backward_workspace_bytes(sh)
    ws = torch.full((nb,), 0x7F, dtype=torch.uint8, device="cuda")
    dx, dg = empty((R, C), dt), empty(C, dt)
    ok(B.rmx_rms_norm_backward(sh, dn, dh, None if ck else h, q if ck else None, e if ck else None, rstd, g, dx, dg,
                               ws, nb))
    sync()
    rho = rstd.double()[:, None]
    xh, t = hv * rho, dn.double() * g.double()
    ref = rho * (t - xh * (t * xh).mean(-1, keepdim=True)) + dh.double()
    dot = (t * xh).abs().mean(-1, keepdim=True)
    err = rho * (4 * t.abs() + xh.abs() * dot * (8 + 160)) * E32 + ref.abs() * 2 * E32
    near(dx, ref, ref.abs() * U[dt] + err * (1 + U[dt]) + TINY[dt], "dx")
    # additions one after another: a thread's rows (at most 18 here), the lanes and sets of a block, up to 456 blocks
    mag, rg = (dn.double() * xh).abs().sum(0), (dn.double() * xh).sum(0)
    near(dg, rg, rg.abs() * U[dt] + mag * 700 * E32 * (1 + U[dt]) + TINY[dt], "dgamma")


@pytest.mark.parametrize("R,C,dt", [(700_000, 40, "bf16"), (700_000, 41, "f16"), (400_000, 100, "bf16"), (30_000, 1001, "bf16"),
                                    (40_000, 1000, "f32")])
def test_checkpoint(R, C, dt):
    x = randn((R, C), dt, 8) * torch.exp(randn((R, 1), "f32", 9)).to(DT[dt])
    q, e = empty((R, Q.pitch(C)), torch.int8), empty((R, Q.pitch(C) // 32), torch.int8)
    v, sh = empty((R, C), dt), B.make_rows(R, C, dt)
    ok(B.rmx_ckpt8_pack(sh, x, q, e))
    ok(B.rmx_ckpt8_unpack(sh, q, e, v))
    sync()
    for a in range(0, R, 1 << 17):
        o = slice(a, a + (1 << 17))
        rq, re, rv = pack(x[o].double(), dt)
        assert torch.equal(q[o], rq) and torch.equal(e[o], re) and torch.equal(v[o].double(), rv)
    few = slice(0, 3)
    nq, ne = Q.ckpt_pack(x[few].double().cpu().numpy(), dt)      # the whole-array form against the definition
    assert np.array_equal(q[few].cpu().numpy(), nq) and np.array_equal(e[few].cpu().numpy(), ne)


@pytest.mark.parametrize("C,dt", [(40, "bf16"), (300, "f16")])
def test_quantised_rows_and_weights(C, dt):
    R = 120_000 if C == 40 else 50_000
    x = randn((R, C), dt, 10)
    q, s = empty((R, Q.pitch(C)), torch.int8), empty(R, torch.float32)
    ok(B.rmx_quant_rows_q8(B.make_rows(R, C, dt), x, q, s))
    G, N = 70, 130
    w = randn((G, C, N), dt, 11)
    wq, ws = empty((G, N, Q.pitch(C)), torch.int8), empty((G, N), torch.float32)
    ok(B.rmx_weight_q8(B.make_layer(1, G, C, N, dt), w, wq, ws))
    sync()
    for val, sc, ref in ((q, s, x.double()), (wq.view(G * N, -1), ws.view(-1), w.double().transpose(1, 2).reshape(G * N, C))):
        top = ref.abs().amax(-1) / 127
        near(sc, top, top * 2 * E32, "scale")
        near(val[:, :C].double() * sc.double()[:, None], ref, (top * (0.5 + 127 * 6 * E32))[:, None], "values")
        assert not val[:, C:].any()
