"""Device buffers of one RankMixer block, kept in torch CUDA memory.

torch provides the memory and the streams; every step of the block runs in
librmx.so through the C ABI (``binding``).
"""

from __future__ import annotations

import numpy as np
import torch

from . import binding as B
from .inputs import PARAM_NAMES, Shape

TORCH_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "tf32": torch.float32}


def _upload(a: np.ndarray, dt: torch.dtype, device) -> torch.Tensor:
    # Values are already rounded to the storage type, so the cast is exact.
    return torch.from_numpy(np.ascontiguousarray(a)).to(device).to(dt).contiguous()


def _ptr_or_none(t: torch.Tensor):
    return t if t.numel() > 0 else None


class RankMixerDevice:
    """Parameters, input, upstream gradient and every output of one block."""

    def __init__(self, shape: Shape, arrays: dict, device="cuda"):
        self.shape = shape
        self.device = torch.device(device)
        self.cfg = B.make_config(shape.B, shape.T, shape.D, shape.H, shape.dtype)
        dt = TORCH_DTYPES[shape.dtype]
        self.dtype = dt
        self.params = {n: _upload(arrays[n], dt, self.device) for n in PARAM_NAMES}
        self.x = _upload(arrays["x"], dt, self.device)
        self.dy = _upload(arrays["dy"], dt, self.device)
        self.y = torch.empty_like(self.x)
        self.dx = torch.empty_like(self.x)
        self.grads = {n: torch.empty_like(self.params[n]) for n in PARAM_NAMES}
        self.saved_bytes = B.rmx_saved_bytes(self.cfg)
        self.ws_bytes = B.rmx_workspace_bytes(self.cfg)
        self.saved = torch.empty(max(self.saved_bytes, 1), dtype=torch.uint8, device=self.device)
        self.ws = torch.empty(max(self.ws_bytes, 1), dtype=torch.uint8, device=self.device)
        self.c_params = B.make_params(self.params)
        self.c_grads = B.make_grads(self.grads)
        self.q8 = None  # int8 weights and their scales, from the first quantize_weights

    def forward(self, stream=None) -> None:
        B.check(B.rmx_forward(self.cfg, _ptr_or_none(self.x), self.c_params, self.saved, self.saved_bytes,
                              _ptr_or_none(self.y), stream), "rmx_forward")

    def backward(self, stream=None) -> None:
        B.check(B.rmx_backward(self.cfg, _ptr_or_none(self.x), _ptr_or_none(self.dy), self.saved,
                               self.saved_bytes, self.c_params, _ptr_or_none(self.dx), self.c_grads,
                               self.ws, self.ws_bytes, stream), "rmx_backward")

    def step(self, stream=None) -> None:
        self.forward(stream)
        self.backward(stream)

    # ---------------------------------------------------------------- 8 bits
    # Buffers that these methods make are taken from the pool of the stream
    # that fills them: what torch's current stream has freed, its pending work
    # may still use.

    def _torch_stream(self, stream):
        """The torch stream of a `stream` argument (None: the legacy default stream)."""
        if stream is None or (isinstance(stream, int) and stream in (0, 1)):  # 1: cudaStreamLegacy
            return torch.cuda.default_stream(self.device)
        return torch.cuda.ExternalStream(stream, device=self.device) if isinstance(stream, int) else stream

    def quantize_weights(self, stream=None) -> None:
        """int8 copies of w1 and wout for forward_q8 (once per weight update).

        The first call makes the buffers, every later one writes them again in
        place, so a graph captured from forward_q8 stays valid.  As with the
        parameters themselves, the caller orders an update after the work that
        still reads the old copies."""
        if self.q8 is None:
            with torch.cuda.stream(self._torch_stream(stream)):
                self._make_q8_buffers()
        s = self.shape
        for name, K, N in (("w1", s.D, 2 * s.H), ("wout", s.H, s.D)):
            B.check(B.rmx_weight_q8(B.make_layer(max(s.B, 1), s.T, K, N, s.dtype), self.params[name], self.q8[name],
                                    self.q8[name + "_scale"], stream), "rmx_weight_q8")

    def _make_q8_buffers(self) -> None:
        s = self.shape
        self.q8 = {}
        for name, K, N in (("w1", s.D, 2 * s.H), ("wout", s.H, s.D)):
            self.q8[name] = torch.empty((s.T, N, B.rmx_q8_pitch(K)), dtype=torch.int8, device=self.device)
            self.q8[name + "_scale"] = torch.empty((s.T, N), dtype=torch.float32, device=self.device)
        self.c_q8 = B.make_q8_weights(self.q8["w1"], self.q8["w1_scale"], self.q8["wout"], self.q8["wout_scale"])
        self.ws_q8 = torch.empty(max(B.rmx_forward_q8_workspace_bytes(self.cfg), 1), dtype=torch.uint8,
                                 device=self.device)

    def forward_q8(self, stream=None) -> None:
        """The forward for serving: int8 contractions, nothing saved."""
        B.check(B.rmx_forward_q8(self.cfg, _ptr_or_none(self.x), self.c_params, self.c_q8, self.ws_q8,
                                 self.ws_q8.numel(), _ptr_or_none(self.y), stream), "rmx_forward_q8")

    def pack_saved(self, stream=None) -> torch.Tensor:
        """The saved activations of the last forward as 8-bit checkpoints."""
        with torch.cuda.stream(self._torch_stream(stream)):
            out = torch.empty(max(B.rmx_saved8_bytes(self.cfg), 1), dtype=torch.uint8, device=self.device)
        B.check(B.rmx_saved_pack8(self.cfg, self.saved, self.saved_bytes, out, out.numel(), stream), "rmx_saved_pack8")
        return out

    def unpack_saved(self, packed: torch.Tensor, stream=None) -> None:
        """Checkpoints of pack_saved back into the saved buffer, for backward().

        `packed` may be dropped at once: its memory is not used for anything
        else before `stream` has read it."""
        B.check(B.rmx_saved_unpack8(self.cfg, packed, packed.numel(), self.saved, self.saved_bytes, stream),
                "rmx_saved_unpack8")
        packed.record_stream(self._torch_stream(stream))

    def results(self) -> dict:
        """y, dx and every gradient as float64 numpy arrays (synchronises)."""
        torch.cuda.synchronize(self.device)
        out = {"y": self.y, "dx": self.dx}
        out.update({n: self.grads[n] for n in PARAM_NAMES})
        return {k: v.detach().float().cpu().numpy().astype(np.float64) for k, v in out.items()}
