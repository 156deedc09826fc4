"""Pointers need 16-byte alignment and no more: with every buffer 16 bytes past a 32-byte boundary the 8-bit operators
give the bits that they give on one."""

import numpy as np
import pytest
import torch

from ffn_block_gb300 import binding as B
from tests.sparse_util import DT, f8_operand, full_of, ok, sync

pytestmark = pytest.mark.gpu
EDGE = 64


class Places:
    """Device buffers that start `by` bytes past a 64-byte boundary, EDGE bytes of 0xA5 before and behind each."""

    def __init__(self, by):
        self.by, self.raw = by, []

    def __call__(self, shape, dt):
        dt = DT.get(dt, dt)
        n = int(np.prod(shape)) * torch.empty((), dtype=dt).element_size()
        raw = full_of((EDGE + self.by + n + EDGE,), torch.uint8, 0xA5)
        assert raw.data_ptr() % 64 == 0
        self.raw.append((raw, EDGE + self.by, n))
        return raw[EDGE + self.by : EDGE + self.by + n].view(dt).reshape(shape)

    def of(self, t):
        out = self(t.shape, t.dtype)
        out.copy_(t)
        return out

    def edges_are_left(self):
        return all(bool((r[:a] == 0xA5).all()) and bool((r[a + n :] == 0xA5).all()) for r, a, n in self.raw)


def _both(run):
    """What `run` returns with buffers on 64-byte boundaries and with all of them 16 bytes behind one."""
    outs = []
    for by in (0, 16):
        new = Places(by)
        outs.append(run(new))
        sync()
        assert new.edges_are_left()
    assert all(torch.equal(a, b) for a, b in zip(*outs))


# whole and odd rows and columns, one block of rows and several, last blocks of one row
@pytest.mark.parametrize("order", ["tokens", "groups", "ragged"])
@pytest.mark.parametrize("dt,fmt", [("bf16", "e4m3"), ("f16", "e5m2"), ("f32", "e4m3")])
@pytest.mark.parametrize("M,G,C", [(1, 1, 1), (128, 2, 128), (129, 3, 264), (77, 5, 1001), (520, 4, 136)])
def test_rows_and_columns(order, dt, fmt, M, G, C):
    ragged = order == "ragged"
    g = torch.Generator().manual_seed(M + C)
    x = torch.randn({"tokens": (M, G, C), "groups": (G, M, C), "ragged": (M, C)}[order], generator=g).to(DT[dt]).cuda()
    off = (torch.arange(G + 1, dtype=torch.int32) * M // G).cuda() if ragged else None
    gr = B.make_groups(M, G, C, dt, order)
    P, EP = B.rmx_f8_pitch(C), B.rmx_f8_exps(C)
    TP = B.rmx_f8_ragged_pitch(M, G) if ragged else B.rmx_f8_pitch(M)
    TE = (TP // 128 + 3) // 4 * 4 if ragged else B.rmx_f8_exps(M)
    nws = B.rmx_quant_f8_groups_workspace_bytes(gr)

    def run(new):
        lead = x.shape[:-1]
        outs = [new((*lead, P), torch.uint8), new((*lead, EP), torch.uint8), new((C, TP) if ragged else (G, C, TP), torch.uint8),
                new((C, TE) if ragged else (G, C, TE), torch.uint8), new((G, C), dt)]
        ok(B.rmx_quant_f8_groups(gr, fmt, new.of(off) if ragged else None, new.of(x), *outs, new((nws,), torch.uint8), nws))
        alone = [new(outs[2].shape, torch.uint8), new(outs[3].shape, torch.uint8)]     # the columns without the sums
        ok(B.rmx_quant_f8_groups(gr, fmt, new.of(off) if ragged else None, new.of(x), None, None, *alone, None, None, 0))
        assert torch.equal(alone[0], outs[2]) and torch.equal(alone[1], outs[3])
        return outs

    _both(run)


def test_rows_and_products():
    """The other calls that read or write 8-bit rows."""
    rng = np.random.default_rng(1)
    M, G, K, N = 150, 3, 264, 136
    a, ea = f8_operand(rng, M * G, K, "e4m3")[1:]
    w, ew = f8_operand(rng, G * N, K, "e4m3")[1:]
    at, eat = f8_operand(rng, G * K, M, "e4m3")[1:]
    bt, ebt = f8_operand(rng, G * N, M, "e5m2")[1:]
    x, bias = torch.randn((M * G, K), device="cuda").bfloat16(), torch.randn((G, N), device="cuda").bfloat16()
    resid = torch.randn((M, G, N), device="cuda").bfloat16()
    routes, src = B.make_routes(M, G, 5, K, "bf16"), torch.randperm(M * G, device="cuda", dtype=torch.int32)

    def run(new):
        q, e, back = new(a.shape, torch.uint8), new(ea.shape, torch.uint8), new(x.shape, "bf16")
        rows = B.make_rows(M * G, K, "bf16")
        ok(B.rmx_quant_f8(rows, "e4m3", new.of(x), q, e))
        ok(B.rmx_dequant_f8(rows, "e4m3", q, e, back))
        gq, ge, out, dw = new(a.shape, torch.uint8), new(ea.shape, torch.uint8), new((M, G, N), "bf16"), new((G, K, N), "bf16")
        ok(B.rmx_expert_gather(routes, new.of(src), new.of(x[:M]), None, "e5m2", gq, ge))
        ok(B.rmx_linear_f8(B.make_layer_f8(M, G, K, N, "bf16"), None, new.of(a), new.of(ea), new.of(w), new.of(ew), new.of(bias),
                           new.of(resid), out))
        ok(B.rmx_wgrad_f8(B.make_layer_f8(M, G, K, N, "bf16", "e4m3", "e5m2"), None, new.of(at), new.of(eat), new.of(bt),
                          new.of(ebt), dw))
        return [q, e, back, gq, ge, out, dw]

    _both(run)
