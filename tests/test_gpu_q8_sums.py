"""Integer sums of the int8 product: exact while no partial sum passes 2^24, and off by a counted bound where one does,
also where the terms cancel."""

import numpy as np
import pytest
import torch

from ffn_block_gb300 import binding as B
from oracle import q8_oracle as Q

from q8_util import dev, empty, f64, ok, sync

pytestmark = pytest.mark.gpu


def product(a, w, K):
    M, G, _ = a.shape
    N = w.shape[1]
    out = empty((M, G, N), "f32")
    one = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    ok(B.rmx_linear_q8(B.make_layer(M, G, K, N, "f32"), dev(a), one(M, G), dev(w), one(G, N), None, None, out))
    sync()
    return f64(out)


def operands(M, G, K, N, seed, lo=-128, hi=127):
    rng = np.random.default_rng(seed)
    a, w = np.zeros((M, G, Q.pitch(K)), np.int8), np.zeros((G, N, Q.pitch(K)), np.int8)
    a[..., :K], w[..., :K] = rng.integers(lo, hi + 1, (M, G, K)), rng.integers(lo, hi + 1, (G, N, K))
    return a, w, rng


# one CTA to a tile, several, pairs
@pytest.mark.parametrize("M,G,N", [(20, 80, 130), (3, 1, 200), (200, 45, 260)])
def test_sums_of_1024_products_are_exact(M, G, N):
    K = 1024
    a, w, _ = operands(M, G, K, N, M)
    a[0], w[:, 0] = -128, -128                       # 2^24 itself
    w[:, 1, ::2], w[:, 1, 1::2] = 127, -128          # large terms that cancel
    a[M // 2] = np.where(np.arange(K) < K // 2, 127, -128)
    ref = np.einsum("mgk,gnk->mgn", a.astype(np.float64), w.astype(np.float64), optimize=True)
    assert ref[0, 0, 0] == 2 ** 24
    assert np.array_equal(product(a, w, K), ref)


@pytest.mark.parametrize("M,G,K,N", [(20, 80, 4096, 130), (150, 45, 3001, 260), (9, 2, 8000, 100)])
def test_cancelling_sums_are_off_by_the_largest_partial_sum(M, G, K, N):
    a, w, rng = operands(M, G, K, N, K, 90, 127)
    half = K // 2 // 16 * 16
    w[..., half:K] = -w[..., half:K]                 # up to half * 127^2, then down again
    a64, w64 = a.astype(np.float64), w.astype(np.float64)
    out = product(a, w, K)
    ref = np.einsum("mgk,gnk->mgn", a64, w64, optimize=True)
    up = np.einsum("mgk,gnk->mgn", a64[..., :half], w64[..., :half], optimize=True)
    assert up.max() > 2 ** 24 and np.abs(ref).min() < 2 ** 24
    # The largest partial sum is the ascent's (or the result, past it); shares of K that several CTAs sum up apart
    # are no larger.  Each step of 16 columns rounds or cuts the sum so far to 24 bits, each share's sum once more.
    largest = np.maximum(up, np.abs(ref)) + 16 * 127 * 127
    assert np.all(np.abs(out - ref) <= (np.ceil(K / 16) + 4) * 2.0 ** -23 * largest)
