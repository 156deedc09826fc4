"""Shared by the tests of the 8-bit operators: devices arrays, error bounds.

Bounds count roundings.  U[t] is half a unit in the last place of type t,
relative to the value (a rounding to nearest is off by at most that much).
float32 sums of n terms are off by at most n * 2^-24 times the sum of the
terms' magnitudes, whatever the order.
"""

import numpy as np
import torch

from ffn_block_gb300 import binding as B

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
# Smallest subnormal of the storage type: a result below its normal range is
# off by half of it.
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}
E32 = 2.0 ** -24


def rnd(a, dtype):
    """float64 array rounded to the storage type, as float64."""
    return torch.from_numpy(np.asarray(a, np.float64)).to(DT[dtype]).double().numpy()


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t.to(DT[dtype]) if dtype else t).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def empty(shape, dt):
    return torch.empty(shape, dtype=DT.get(dt, dt), device="cuda")


def within(got, ref, bound, what=""):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    ok = ~np.isnan(ref)
    over = np.abs(got - ref)[ok] - np.broadcast_to(bound, ref.shape)[ok]
    assert over.size == 0 or np.max(over) <= 0, (what, float(np.max(over)), int(np.sum(over > 0)))


def ok(status, what=""):
    B.check(status, what)


def sync():
    B.check(B.rmx_check())
