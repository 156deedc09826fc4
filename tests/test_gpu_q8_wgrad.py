"""The weight gradient with its fused column sums where a CTA or pair takes several tiles, summed ones (the first row
of tiles) and others in turn, on a ring that the contraction does not fill a whole number of times."""

import numpy as np
import pytest
import torch

from ffn_block_gb300 import binding as B

from q8_util import DT, dev, empty, ok, sync

pytestmark = pytest.mark.gpu

# (samples, tokens, inputs, outputs): pairs of CTAs (inputs past 128) and CTAs alone, extents of whole 64s (stages of
# interleaved pieces) and others, padded rows, contractions of 2, 3, 8 and 11 steps of 64
SHAPES = [(72, 40, 640, 512), (448, 30, 768, 512), (70, 40, 600, 520), (450, 30, 777, 515), (700, 20, 520, 700),
          (136, 200, 128, 320), (130, 200, 96, 300), (513, 160, 72, 270)]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("M,G,K,N", SHAPES)
def test_wgrad_of_many_tiles(M, G, K, N, dt):
    """Integers: every product and partial sum is exact, so dw and db are the integers rounded once; with another
    stream keeping the memory system busy in some of the runs."""
    g = torch.Generator(device="cuda").manual_seed(M + K)
    P = B.rmx_q8_pitch(K)
    q = torch.randint(-3, 4, (M, G, P), generator=g, device="cuda", dtype=torch.int8)
    q[..., K:] = 0
    e = torch.zeros((M, G, P // 32), dtype=torch.int8, device="cuda")
    dy = torch.randint(-4, 5, (M, G, N), generator=g, device="cuda").to(DT[dt])
    rw = torch.bmm(q[..., :K].double().permute(1, 2, 0), dy.double().permute(1, 0, 2)).to(DT[dt])
    rb = dy.double().sum(0).to(DT[dt])
    layer = B.make_layer(M, G, K, N, dt)
    nb = B.rmx_ckpt8_wgrad_workspace_bytes(layer)
    ws, dw, db = empty(nb, torch.uint8), empty((G, K, N), dt), empty((G, N), dt)
    big, st = torch.zeros(1 << 26, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(12):
        if i % 3:
            with torch.cuda.stream(st):
                big.add_(1.0)
        ws.fill_(0x7F)
        dw.fill_(float("nan"))
        db.fill_(float("nan"))
        ok(B.rmx_ckpt8_wgrad(layer, q, e, dy, dw, db, ws, nb))
        sync()
        assert torch.equal(dw, rw) and torch.equal(db, rb), i
    torch.cuda.synchronize()
    assert np.isfinite(float(big[0]))


def test_wgrad_scales_of_groups():
    """The same with a checkpoint of mixed exponents: powers of two leave the sums exact."""
    M, G, K, N, dt = 90, 50, 300, 520, "f16"
    rng = np.random.default_rng(9)
    P = B.rmx_q8_pitch(K)
    q = np.zeros((M, G, P), np.int8)
    q[..., :K] = rng.integers(-1, 2, (M, G, K))
    e = rng.integers(-2, 3, (M, G, P // 32)).astype(np.int8)
    dy = rng.integers(-1, 2, (M, G, N)).astype(np.float64)
    x = (q * np.repeat(2.0 ** e.astype(float), 32, axis=-1))[..., :K]
    layer = B.make_layer(M, G, K, N, dt)
    nb = B.rmx_ckpt8_wgrad_workspace_bytes(layer)
    dw, db = empty((G, K, N), dt), empty((G, N), dt)
    ok(B.rmx_ckpt8_wgrad(layer, dev(q), dev(e), dev(dy, dt), dw, db, empty(nb, torch.uint8), nb))
    sync()
    # sums of at most 90 terms of up to 4 in quarters: below 512 and a whole number of quarters, so 11 bits hold them
    rw = np.einsum("mgk,mgn->gkn", x, dy, optimize=True)
    assert np.abs(rw).max() < 512
    assert np.array_equal(dw.double().cpu().numpy(), rw) and np.array_equal(db.double().cpu().numpy(), dy.sum(0))
