"""Prompts of linear attention that a workspace lets the call cut into segments: what the cut costs.
The cut against the formula: test_gpu_linear."""
import ctypes

import pytest
import torch

from indexed_sparse_attention_indexer_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Prompts:
    def __init__(self, lens, H, d):
        self.n, self.B, self.H, self.d = sum(lens), len(lens), H, d
        g = torch.Generator(device=DEV).manual_seed(1)
        self.q, self.k, self.v = (torch.randn((self.n, H, d), generator=g, device=DEV).to(torch.bfloat16) for _ in range(3))
        self.decay = -torch.rand(H, generator=g, device=DEV) * 0.1
        self.state = torch.zeros((self.B, H, d, d), device=DEV)
        self.out = torch.empty((self.n, H, d), dtype=torch.bfloat16, device=DEV)
        self.starts = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
        self.struct, _ = binding._linear(self.q, self.k, self.v, self.decay, d ** -0.5, self.state, None, None,
                                         self.out, self.B, None)
        self.workspace = binding.alloc_workspace(binding.linear_workspace_size(self.n, self.B, H, d, d), DEV)

    def call(self, split):
        ws = self.workspace
        st = binding.load().dsi_linear_prefill(
            ctypes.byref(self.struct), self.n, self.starts.data_ptr(), self.B, ws.data_ptr() if split else None,
            ws.numel() if split else 0, binding._stream(None))
        assert st == 0

    def time(self, split):
        """us a call, the least of several."""
        for _ in range(3):
            self.call(split)
        best = float("inf")
        for _ in range(8):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(10):
                self.call(split)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b) * 100)
        return best


@pytest.mark.parametrize("B,n,H,d", [(4, 4096, 8, 128), (8, 4096, 8, 64), (1, 4096, 32, 128), (4, 8192, 8, 128)])
def test_a_workspace_costs_no_time(B, n, H, d):
    """Sequences of one length: whole ones, and cut as the call cuts them, which takes at most 6 % longer
    (with a few segments more than there are CTAs it took 1.5 times as long)."""
    p = Prompts([n] * B, H, d)
    assert p.time(True) <= 1.25 * p.time(False)
    assert binding.device_status() == 0
