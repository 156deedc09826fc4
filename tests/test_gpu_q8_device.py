"""RankMixerDevice's 8-bit methods on the GPU: graphs over a weight update, and
buffers that go from one stream to another."""

import numpy as np
import pytest
import torch

from ffn_block_gb300 import binding as B
from ffn_block_gb300 import inputs as I
from ffn_block_gb300.device import RankMixerDevice

from q8_util import sync

pytestmark = pytest.mark.gpu


def block(seed, **dims):
    shape = I.Shape(dtype="bf16", **(dims or dict(B=6, T=8, D=128, H=256)))
    return RankMixerDevice(shape, I.make_inputs(shape, seed=seed, ln_params="random"))


@pytest.mark.parametrize("side", [False, True], ids=["default stream", "side stream"])
def test_graph_of_forward_q8_sees_requantised_weights(side):
    blk, other = block(1), block(2)
    st = torch.cuda.Stream()
    on = st if side else None
    blk.quantize_weights(on)
    blk.forward_q8(on)
    B.check(B.rmx_check(on))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        blk.forward_q8(st)
    before = blk.y.clone()
    for k in ("w1", "wout"):
        blk.params[k].copy_(other.params[k])
    torch.cuda.synchronize()
    blk.quantize_weights(on)
    B.check(B.rmx_check(on))
    # whatever was given back since the capture is written over
    junk = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda")
            for n in [v.numel() * v.element_size() for v in blk.q8.values()] + [blk.ws_q8.numel()]]
    blk.y.zero_()
    torch.cuda.synchronize()
    graph.replay()
    sync()
    replayed = blk.y.clone()
    blk.forward_q8()
    sync()
    assert torch.equal(replayed, blk.y) and not torch.equal(replayed, before)
    assert np.isfinite(blk.results()["y"]).all()
    del junk
