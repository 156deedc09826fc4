"""The int8 product while other work keeps the memory system busy: what one warp, copy or CTA hands to another
arrives whole, so every run gives the exact integers."""

import numpy as np
import pytest
import torch

from ffn_block_gb300 import binding as B

from q8_util import empty, ok, sync

pytestmark = pytest.mark.gpu


# CTAs alone, several tiles each, and two and four CTAs to a tile
ALONE = [(64, 130, 1000, 300), (96, 100, 1024, 520), (16, 200, 700, 640), (5, 40, 1000, 5000)]
SPLIT = [(90, 6, 1024, 600), (16, 70, 1030, 100), (1, 1, 1040, 4500), (96, 18, 1024, 200)]
# several tiles a pair
PAIRS = [(192, 90, 128, 256), (100, 100, 1000, 300), (400, 40, 1000, 520), (97, 160, 40, 257), (1024, 4, 1040, 640)]


@pytest.mark.parametrize("M,G,K,N", ALONE + SPLIT + PAIRS)
def test_linear_beside_other_work(M, G, K, N):
    g = torch.Generator(device="cuda").manual_seed(M + K)
    P = B.rmx_q8_pitch(K)
    a = torch.randint(-127, 128, (M, G, P), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-127, 128, (G, N, P), generator=g, device="cuda", dtype=torch.int8)
    one_a, one_w = torch.ones((M, G), device="cuda"), torch.ones((G, N), device="cuda")
    # K * 127^2 < 2^24: every partial sum is an integer that float32 holds
    assert K * 127 * 127 < 2 ** 24
    af, wf = a[..., :K].double(), w[..., :K].double()
    ref = torch.stack([af[:, i] @ wf[i].t() for i in range(G)], dim=1).float()
    layer, out = B.make_layer(M, G, K, N, "f32"), empty((M, G, N), "f32")
    big, st = torch.zeros(1 << 26, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(40):
        if i % 3:
            with torch.cuda.stream(st):
                big.add_(1.0)
        out.fill_(float("nan"))
        ok(B.rmx_linear_q8(layer, a, one_a, w, one_w, None, None, out))
        sync()
        assert torch.equal(out, ref), i
    torch.cuda.synchronize()
    assert np.isfinite(float(big[0]))
