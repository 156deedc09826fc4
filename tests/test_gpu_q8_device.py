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
    assert torch.isfinite(blk.y).all()
    del junk


def checkpoint(blk):
    blk.forward()
    sync()
    packed = blk.pack_saved()
    sync()
    return packed


def test_pack_on_another_stream_than_the_current_one():
    """Memory that the current stream's pending work still writes is not handed to pack_saved on `stream`."""
    blk = block(3, B=64, T=8, D=128, H=256)
    want = checkpoint(blk).clone()
    st = torch.cuda.Stream()
    sync()
    late = torch.empty_like(want)
    torch.cuda._sleep(20_000_000)       # about 10 ms of the current stream
    late.fill_(0x77)
    del late
    packed = blk.pack_saved(st)
    sync()
    torch.cuda.synchronize()
    assert torch.equal(packed, want)


@pytest.mark.parametrize("handle", [False, True], ids=["stream", "its handle"])
def test_packed_may_be_dropped_while_another_stream_reads_it(handle):
    blk = block(4, B=64, T=8, D=128, H=256)
    packed = checkpoint(blk)
    blk.saved.zero_()
    blk.unpack_saved(packed)
    sync()
    want, n = blk.saved.clone(), packed.numel()
    blk.saved.zero_()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)
    blk.unpack_saved(packed, st.cuda_stream if handle else st)
    del packed
    junk = [torch.full((n,), 0x77, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(blk.saved, want)
    del junk


def test_8_bit_methods_on_a_side_stream():
    a, b = block(5), block(5)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    for blk, on in ((a, None), (b, st)):
        for _ in range(2):
            blk.quantize_weights(on)
            blk.forward_q8(on)
        blk.y8 = blk.y
        blk.y = torch.empty_like(blk.y)
        torch.cuda.synchronize()
        blk.forward(on)
        packed = blk.pack_saved(on)
        blk.unpack_saved(packed, on)
        del packed
        blk.backward(on)
        B.check(B.rmx_check(on))
    assert torch.equal(a.y8, b.y8)
    ra, rb = a.results(), b.results()
    assert all(np.array_equal(ra[k], rb[k]) for k in ra)
