"""A whole block step while another stream keeps the memory system busy: the same bits as alone."""

import numpy as np
import pytest
import torch

from ffn_block_gb300 import binding as B
from ffn_block_gb300 import inputs as I
from ffn_block_gb300.device import RankMixerDevice

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,dims", [("bf16", dict(B=256, T=32, D=512, H=1536)), ("f16", dict(B=100, T=40, D=1200, H=2400)),
                                     ("f32", dict(B=64, T=16, D=256, H=512)), ("tf32", dict(B=64, T=16, D=256, H=512)),
                                     # the general form of norm0's backward (T not a multiple of 8, padded rows)
                                     ("bf16", dict(B=700, T=10, D=1200, H=1800)), ("f16", dict(B=700, T=10, D=630, H=1260))],
                         ids=["bf16", "f16", "f32", "tf32", "general", "padded"])
def test_step_beside_other_work(dt, dims):
    shape = I.Shape(dtype=dt, **dims)
    blk = RankMixerDevice(shape, I.make_inputs(shape, seed=11, ln_params="random"))
    blk.step()
    B.check(B.rmx_check())
    want = {k: v.clone() for k, v in dict(blk.grads, y=blk.y, dx=blk.dx).items()}
    assert all(torch.isfinite(v).all() for v in want.values())
    big, st = torch.zeros(1 << 26, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(30):
        with torch.cuda.stream(st):
            for _ in range(1 + i % 3):
                big.add_(1.0)
        for v in (blk.y, blk.dx, *blk.grads.values()):
            v.fill_(float("nan"))
        blk.step()
        B.check(B.rmx_check())
        for k, v in dict(blk.grads, y=blk.y, dx=blk.dx).items():
            assert torch.equal(v, want[k]), (i, k)
    torch.cuda.synchronize()
    assert np.isfinite(float(big[0]))
