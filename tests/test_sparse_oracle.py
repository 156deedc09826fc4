"""Pins of the sparse layer's oracle (CPU): published vectors, torch's own arithmetic, differences."""

import numpy as np
import pytest
import torch

from oracle import sparse_oracle as O

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


@pytest.mark.parametrize("counter,key,words", [
    # The known answers that Random123 publishes for philox4x32-10.
    ([0, 0, 0, 0], [0, 0], [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
    ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
     [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]),
])
def test_philox_known_answers(counter, key, words):
    assert O.philox(counter, key) == words


def test_keep_bits_by_hand():
    seed, offset = 0x0123456789ABCDEF, (5 << 32) | 77
    k = O.keep(3, 19, 0.3, seed, offset, row0=(7 << 32) + 1)
    t = O.drop_threshold(0.3)
    for r in range(3):
        row = (7 << 32) + 1 + r
        for c in range(19):
            w = O.philox([c // 8 | (row >> 32) << 24, row & O.MASK, 77, 5], [seed & O.MASK, seed >> 32])[c % 8 // 2]
            assert k[r, c] == ((w >> (16 * (c % 2)) & 0xFFFF) >= t)


def test_keep_rate():
    k = O.keep(2000, 512, 0.25, 99, 3)
    n, p = k.size, 0.75
    assert abs(k.mean() - p) < 5 * np.sqrt(p * (1 - p) / n)
    # neighbours are not related: of pairs, p^2 are both kept
    assert abs((k[:, 1:] & k[:, :-1]).mean() - p * p) < 5 * np.sqrt(p * p / n)


@pytest.mark.parametrize("gamma", [True, False])
def test_layer_norm_against_torch_and_differences(gamma):
    rng = np.random.default_rng(0)
    h, dy, dh = rng.standard_normal((3, 7, 33))
    g = 1 + 0.3 * rng.standard_normal(33) if gamma else None
    b = rng.standard_normal(33) if gamma else None
    y, mean, rstd = O.layer_norm(h, g, b, 1e-5)
    T = lambda a: None if a is None else torch.from_numpy(a).requires_grad_()  # noqa: E731
    th, tg, tb = T(h), T(g), T(b)
    ty = torch.nn.functional.layer_norm(th, (33,), tg, tb, 1e-5)
    assert np.allclose(y, ty.detach().numpy(), atol=1e-12)
    ty.backward(torch.from_numpy(dy))
    dr, dg, db = O.layer_norm_backward(dy, None, h, mean, rstd, g)
    assert np.allclose(dr, th.grad.numpy(), atol=1e-12)
    if gamma:
        assert np.allclose(dg, tg.grad.numpy(), atol=1e-12) and np.allclose(db, tb.grad.numpy(), atol=1e-12)
    d = rng.standard_normal(h.shape)
    f = lambda s: (O.layer_norm(h + s * d, g, b, 1e-5)[0] * dy).sum() + ((h + s * d) * dh).sum()  # noqa: E731
    dr = O.layer_norm_backward(dy, dh, h, mean, rstd, g)[0]
    assert abs((f(1e-5) - f(-1e-5)) / 2e-5 - (dr * d).sum()) < 1e-6 * np.abs(dr * d).sum()


def test_expert_sort_by_numpy():
    rng = np.random.default_rng(1)
    ids = rng.integers(-2, 9, (40, 3))
    off, pos, src = O.expert_sort(ids, 7)
    flat = ids.reshape(-1)
    live = np.flatnonzero((flat >= 0) & (flat < 7))
    order = live[np.argsort(flat[live], kind="stable")]
    assert np.array_equal(src[: order.size], order) and np.all(src[order.size :] == -1)
    assert off[-1] == order.size and np.array_equal(np.diff(off), [np.sum(flat == e) for e in range(7)])
    assert np.array_equal(src[pos.reshape(-1)[live]], live) and np.all(pos.reshape(-1)[(flat < 0) | (flat >= 7)] == -1)


def test_combine_gradient_by_differences():
    rng = np.random.default_rng(2)
    _, pos, _ = O.expert_sort(rng.integers(-1, 4, (11, 3)), 4)
    w, y, dout = rng.standard_normal((11, 3)), rng.standard_normal((33, 5)), rng.standard_normal((11, 5))
    dy, dw = O.combine_backward(pos, w, dout, y)
    vw, vy = rng.standard_normal(w.shape), rng.standard_normal(y.shape)
    f = lambda s: (O.combine(pos, w + s * vw, y + s * vy) * dout).sum()  # noqa: E731
    assert abs((f(1e-6) - f(-1e-6)) / 2e-6 - ((dw * vw).sum() + np.nansum(dy * vy))) < 1e-6


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_f8_values_are_torchs(fmt):
    """Every value, every midpoint between two and both neighbours of a midpoint round as torch rounds."""
    v = torch.arange(256, dtype=torch.uint8).view(F8[fmt]).double().numpy()
    v = np.unique(v[np.isfinite(v)])
    mid = (v[1:] + v[:-1]) / 2
    x = np.concatenate([v, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)])
    assert np.array_equal(O.to_f8(x, fmt), torch.from_numpy(x).float().to(F8[fmt]).double().numpy())


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_block_exponents(fmt):
    top = O.LARGEST[fmt]
    for b in (0, 1, 100, 127, 200, 254):
        at = top * 2.0 ** (b - 127)
        assert O.block_exp(at, fmt) == b and O.block_exp(at * (1 + 2.0 ** -40), fmt) in (b + 1, 0 if b == 254 else b + 1)
    assert O.block_exp(0.0, fmt) == 0


def test_quantised_rows_are_close():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((20, 300)) * np.exp(rng.standard_normal((20, 1)) * 5)
    for fmt, half in (("e4m3", 2.0 ** -4), ("e5m2", 2.0 ** -3)):
        q, e = O.quant_rows(x, fmt)
        v = O.row_values(q, e, 300)
        tiny = 2.0 ** (np.repeat(e, 128, 1)[:, :300] - 127 + O.LOWEST[fmt] - O.MANTISSA[fmt] - 1)
        assert np.all(np.abs(v - x) <= np.maximum(half * np.abs(x), tiny))
        assert np.all(q[:, 300:] == 0)
    x[3, 130] = np.inf
    q, e = O.quant_rows(x, "e4m3")
    assert e[3, 1] == 255 and np.all(np.isnan(O.row_values(q, e, 300)[3, 128:256])) and np.all(e[3, [0, 2]] < 255)
