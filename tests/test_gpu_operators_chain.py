"""Head norms with rotation, dense and window attention together, as a model's layers use them:
a prompt's latent rows into a paged cache, its window attention, then decode steps of which one
call norms and rotates the new tokens' keys into the cache and rotates their queries, and the
attention calls read both.  Every stage is compared with its formula in 64 bits, from what the
stage before stored (the tolerances are those of the operators' own tests)."""
import math

import pytest
import torch

from indexed_sparse_attention_indexer_gb300 import binding
from tests.test_gpu_dense_mla import SCALE, reference as attention_reference, spots
from tests.test_gpu_norm_rope import check_bf16, reference as rope_reference

pytestmark = pytest.mark.gpu
DEV = "cuda"
NORM = dict(norm="rms", norm_dim=512)
ROPE = dict(rope_offset=512, interleaved=True)


class Model:
    """Two layers' worth of state over one paged pool: the first attends to everything, the
    second to a window with sinks."""

    def __init__(self, lens, T, H, page, fp8, room, seed):
        self.g = torch.Generator().manual_seed(seed)
        self.B, self.T, self.H, self.page, self.fp8 = len(lens), T, H, page, fp8
        wide = (max(lens) + room + page - 1) // page
        pages = self.B * wide + 3
        self.table = torch.randperm(pages, generator=self.g)[:self.B * wide].view(self.B, wide).to(torch.int32).to(DEV)
        dtype = torch.uint8 if fp8 else torch.bfloat16
        # what no call has written yet is NaN (0x7F in E4M3; scales too)
        self.pool = torch.full((pages, page, 576), 0x7F if fp8 else math.nan, dtype=dtype, device=DEV)
        if fp8:
            self.pool = self.pool.view(torch.float8_e4m3fn)
        self.scales = torch.full((pages, page, 5), math.nan, device=DEV) if fp8 else None
        self.lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.cache = binding.Cache(None, self.pool, self.lens, block_table=self.table, page_size=page,
                                   latent_scale=self.scales)
        self.rope = binding.rope_table(wide * page, 64, device=DEV)
        self.weight = torch.empty(512).uniform_(0.5, 1.5, generator=self.g).to(DEV)

    def new(self, n, heads):
        return torch.randn((n, heads, 576), generator=self.g).to(torch.bfloat16).to(DEV)

    def slots(self, b, pos):
        return self.table.long()[b, pos // self.page] * self.page + pos % self.page

    def heads(self, x, dst):
        return binding.Heads(x, weight=self.weight, out=self.pool, out_scale=self.scales, dst_rows=dst, **NORM)

    # what attention_reference reads of a case
    def rows(self, b, pos):
        at = self.slots(torch.tensor(b, device=DEV), pos.to(DEV))
        c = self.pool.view(torch.uint8 if self.fp8 else torch.bfloat16).view(-1, 576)[at]
        if self.fp8:
            sc = self.scales.view(-1, 5)[at].repeat_interleave(128, dim=-1)[:, :576]
            c = (c.view(torch.float8_e4m3fn).float() * sc).to(torch.bfloat16)
        return c.double().cpu()

    def check_rows(self, x, b, pos):
        """The cache rows of tokens x at (b, pos)."""
        z, M = rope_reference(x, "rms", self.weight, None, 512, self.rope, pos, 512, True, 1e-6)
        z, M = z[:, 0], M[:, 0]
        got = torch.cat([self.rows(int(i), p[None]) for i, p in zip(b, pos)])
        if not self.fp8:
            return check_bf16(got, z, M)
        # half an E4M3 step of the code (2^-4 relative, 2^-10 of the scale for subnormals), the
        # scale's and the product's rounding to bf16 (2^-8), the fp32 arithmetic
        s = torch.nn.functional.pad(z, (0, 64)).unflatten(-1, (5, 128)).abs().amax(-1) / 448
        s = s.repeat_interleave(128, dim=-1)[:, :576]
        tol = z.abs() * (2.0 ** -4 + 2.0 ** -7) + 2.0 ** -9 * s + 2.0 ** -14 * M
        assert bool(((got - z).abs() <= tol).all())

    def check_attention(self, q, out, lse, views):
        self.q = q.cpu()
        for r, b, pos in views:
            ref, tol, rl, tl = attention_reference(self, r, b, pos, SCALE)
            assert bool(((out[r].double().cpu() - ref).abs() <= tol).all()), r
            assert bool(((lse[r].double().cpu() - rl).abs() <= tl).all()), r


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,page", [(1, 128, 64), (2, 16, 16), (3, 20, 24)])
def test_prompt_then_steps(fp8, T, H, page):
    lens, window, sink = [130, 1, 63], 50, 3
    m = Model(lens, T, H, page, fp8, room=12, seed=T)
    b = torch.cat([torch.full((n,), i) for i, n in enumerate(lens)]).to(DEV)
    pos = torch.cat([torch.arange(n) for n in lens]).to(DEV)
    x = m.new(pos.numel(), 1)
    binding.norm_rope(None, m.heads(x, m.slots(b, pos)), m.rope, pos, **ROPE)
    # the first sequence's prompt: its queries rotated in place, then the window
    q = m.new(130, H)
    raw = q.clone()
    binding.norm_rope(binding.Heads(q, out=q), None, m.rope, pos[:130].contiguous(), **ROPE)
    first = binding.Cache(None, m.pool, None, block_table=m.table[:1], page_size=page, latent_scale=m.scales)
    out, lse = binding.window_mla_prefill(q, first, 0, window, sink, SCALE)
    torch.cuda.synchronize()
    m.check_rows(x, b, pos)
    check_bf16(q, *rope_reference(raw, None, None, None, 576, m.rope, pos[:130], 512, True, 1e-6))
    m.check_attention(q, out, lse, [(t, 0, spots(t + 1, window, sink)) for t in range(0, 130, 7)])
    # decode: T tokens a sequence and step, keys into the cache and queries in one launch
    for _ in range(3):
        m.lens += T
        pos = (m.lens.long()[:, None] - T + torch.arange(T, device=DEV)).reshape(-1)
        b = torch.arange(m.B, device=DEV).repeat_interleave(T)
        x, raw = m.new(m.B * T, 1), m.new(m.B * T, H)
        q, _ = binding.norm_rope(binding.Heads(raw), m.heads(x, m.slots(b, pos)), m.rope, pos, **ROPE)
        dense = binding.dense_mla_decode(q, m.cache, SCALE, tokens_per_seq=T)
        near = binding.window_mla_decode(q, m.cache, window, sink, SCALE, tokens_per_seq=T)
        torch.cuda.synchronize()
        assert binding.device_status() == 0
        m.check_rows(x, b, pos)
        check_bf16(q, *rope_reference(raw, None, None, None, 576, m.rope, pos, 512, True, 1e-6))
        seen = [(r, int(b[r]), int(pos[r]) + 1) for r in range(m.B * T)]
        m.check_attention(q, *dense, [(r, i, torch.arange(n)) for r, i, n in seen])
        m.check_attention(q, *near, [(r, i, spots(n, window, sink)) for r, i, n in seen])


@pytest.mark.parametrize("fp8", [False, True])
def test_captured_step(fp8):
    """A whole step in one graph on a stream of its own: lengths, positions and cache slots advance
    on the device, so that replays go on from each other."""
    T, H, page, window, sink = 1, 128, 64, 100, 4
    lens = [700, 3, 64]
    m = Model(lens, T, H, page, fp8, room=80, seed=9)
    b = torch.cat([torch.full((n,), i) for i, n in enumerate(lens)]).to(DEV)
    pos = torch.cat([torch.arange(n) for n in lens]).to(DEV)
    x = m.new(pos.numel(), 1)
    binding.norm_rope(None, m.heads(x, m.slots(b, pos)), m.rope, pos, **ROPE)
    seqs = torch.arange(m.B, device=DEV)
    pos, dst = torch.zeros(m.B, dtype=torch.int64, device=DEV), torch.zeros(m.B, dtype=torch.int64, device=DEV)
    x, raw = m.new(m.B, 1), m.new(m.B, H)
    queries, keys = binding.Heads(raw), m.heads(x, dst)
    wsp = [binding.alloc_workspace(binding.dense_mla_workspace_size(m.B, H), DEV) for _ in range(2)]
    outs = [(torch.empty((m.B, H, 512), dtype=torch.bfloat16, device=DEV), torch.empty((m.B, H), device=DEV))
            for _ in range(2)]

    def step():
        pos.copy_(m.lens)
        m.lens.add_(1)
        dst.copy_(m.slots(seqs, pos))
        binding.norm_rope(queries, keys, m.rope, pos, **ROPE)
        binding.dense_mla_decode(queries.out, m.cache, SCALE, out=outs[0][0], lse=outs[0][1], workspace=wsp[0])
        binding.window_mla_decode(queries.out, m.cache, window, sink, SCALE, out=outs[1][0], lse=outs[1][1],
                                  workspace=wsp[1])

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        for _ in range(66):                          # over a page's end in every sequence
            x.copy_(m.new(m.B, 1))
            raw.copy_(m.new(m.B, H))
            graph.replay()
    stream.synchronize()
    assert binding.device_status() == 0
    assert m.lens.tolist() == [n + 67 for n in lens]
    m.check_rows(x, seqs, pos)
    n = (pos + 1).tolist()
    m.check_attention(queries.out, *outs[0], [(i, i, torch.arange(n[i])) for i in range(m.B)])
    m.check_attention(queries.out, *outs[1], [(i, i, spots(n[i], window, sink)) for i in range(m.B)])
