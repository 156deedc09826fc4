"""Shared by the tests of the sparse layer's operators: device arrays, 8-bit rows, error bounds.

Bounds count roundings, as in q8_util.  A sum in a tree of additions of depth n is
off by at most n * 2^-24 times the sum of the terms' magnitudes; the row passes'
trees are at most 64 deep (20 pairs a lane, a lane's pair, 5 steps of a warp, 16
warps)."""

import numpy as np
import torch

from ffn_block_gb300 import binding as B
from tests.q8_util import DT, E32, TINY, U, dev, empty, f64, ok, rnd, sync, within  # noqa: F401

DEPTH = 64
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def state_of(seed, offset):
    return torch.from_numpy(np.array([seed, offset], np.uint64).view(np.int64)).cuda()


def full_of(shape, dt, value):
    return torch.full(shape, value, dtype=DT.get(dt, dt), device="cuda")


def f8_values(q, fmt):
    """8-bit floating bytes (a uint8 tensor) as float64."""
    return q.view(F8[fmt]).float().double().cpu().numpy()


def f8_bytes(values, fmt):
    """Values of the format as bytes (on the CPU)."""
    return torch.from_numpy(np.asarray(values, np.float64)).float().to(F8[fmt]).view(torch.uint8)


def f8_operand(rng, rows, cols, fmt, spread=2):
    """Random 8-bit rows with their padding: values [rows, cols] near 1 (so that products fit float16), bytes [rows, P],
    exponents [rows, EP]."""
    P, EP = B.rmx_f8_pitch(cols), B.rmx_f8_exps(cols)
    v = np.zeros((rows, P))
    top = 448 if fmt == "e4m3" else 57344
    x = np.clip(rng.standard_normal((rows, cols)) * (100 if fmt == "e4m3" else 1000), -top, top)
    v[:, :cols] = f8_bytes(x, fmt).view(F8[fmt]).double()
    e = np.zeros((rows, EP), np.int64)
    mid = 127 - (7 if fmt == "e4m3" else 10)
    e[:, : P // 128] = rng.integers(mid - spread, mid + 1 + spread, (rows, P // 128))
    step = 2.0 ** (e[:, : P // 128].astype(np.float64) - 127)
    values = (v.reshape(rows, -1, 128) * step[..., None]).reshape(rows, P)[:, :cols]
    return values, f8_bytes(v, fmt).cuda(), torch.from_numpy(e.astype(np.uint8)).cuda()


def mma_bound(a, b, K, dtype, ref):
    """Bound of a product a [m, K] @ b [n, K]^T: 32 terms at a time enter the float32 sum, aligned to the largest of
    them and the sum with at least 23 bits kept, so that each of them and the sum may lose 2^-23 of the largest:
    2^-23 (K / 32 + 32) sum |terms| over the whole of K; then one rounding."""
    mag = np.abs(a) @ np.abs(b).T
    return 2.0 ** -23 * (K / 32 + 32) * mag + U[dtype] * np.abs(ref) + TINY[dtype]
