"""Buffers of RankMixerDevice's 8-bit methods, with the library's calls faked (no GPU)."""

import contextlib
import os

import pytest
import torch

from ffn_block_gb300 import binding as B
from ffn_block_gb300 import inputs as I
from ffn_block_gb300.device import RankMixerDevice


@pytest.fixture
def blk(monkeypatch):
    """A block in host memory; the calls that would launch kernels only note their pointers."""
    if not os.path.exists(B.LIB_PATH):
        from ffn_block_gb300 import build
        build.build()
    shape = I.Shape(dtype="bf16", B=2, T=4, D=32, H=64)
    blk = RankMixerDevice(shape, I.make_inputs(shape, seed=1), device="cpu")
    blk.calls = []

    def fake(name):
        def call(*a):
            blk.calls.append((name, tuple(B._ptr(v) if hasattr(v, "data_ptr") else v for v in a)))
            return B.RMX_OK
        return call

    # Streams: torch's current one is "current" unless a context says otherwise.
    blk.allocated, blk.recorded, current = [], [], ["current"]

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: blk.allocated.append(current[-1]) or empty(*a, **k))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda s, device=None: ("external", s))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: blk.recorded.append((t.data_ptr(), s)))
    for name in ("rmx_weight_q8", "rmx_forward_q8", "rmx_saved_pack8", "rmx_saved_unpack8"):
        monkeypatch.setattr(B, name, fake(name))
    return blk


def test_weights_are_quantised_again_in_place(blk):
    """A captured forward_q8 holds the pointers of the first call."""
    blk.quantize_weights()
    first = {k: v.data_ptr() for k, v in blk.q8.items()}
    c_q8, ws = blk.c_q8, blk.ws_q8.data_ptr()
    keep = list(blk.q8.values()), blk.ws_q8      # so that a new buffer cannot get an old one's place
    blk.quantize_weights()
    assert {k: v.data_ptr() for k, v in blk.q8.items()} == first
    assert blk.c_q8 is c_q8 and blk.ws_q8.data_ptr() == ws
    writes = [c[1][2:4] for c in blk.calls]
    assert writes == 2 * [(first["w1"], first["w1_scale"]), (first["wout"], first["wout_scale"])]
    del keep


class Stream:
    cuda_stream = 0x4000


@pytest.mark.parametrize("stream,expect", [(None, "default"), (0, "default"), (1, "default"), (0x4000, ("external", 0x4000)),
                                           (Stream, Stream)])
def test_buffers_belong_to_the_stream_that_uses_them(blk, stream, expect):
    blk.quantize_weights(stream)
    packed = blk.pack_saved(stream)
    assert blk.allocated == 6 * [expect]        # two weights, two scales, the workspace, the checkpoint
    assert blk.recorded == []
    blk.unpack_saved(packed, stream)
    assert blk.recorded == [(packed.data_ptr(), expect)]
