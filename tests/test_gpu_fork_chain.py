"""A hybrid model's two kinds of layers over a batch that goes on from one common prefix, as they would be
used together: the prefix's tokens through the linear layer into one state slot and, normed and rotated, onto
latent pages; every request's own prompt from that slot into a slot of its own; then steps in which all
requests share the prefix's pages and each updates its own state and pages.  Every stage is compared with its
formula in 64 bits, from what the stage before stored (tolerances: the operators' own tests)."""
import math

import pytest
import torch

from indexed_sparse_attention_indexer_gb300 import binding
from tests.test_gpu_dense_mla import SCALE
from tests.test_gpu_linear import Case
from tests.test_gpu_operators_chain import Model
from tests.test_gpu_prefix_mla import Shared

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROPE = dict(rope_offset=512, interleaved=True)
DK, DV = 64, 96


def linear_case(q, k, v, log_decay, scale, lens, state, ins, outs):
    """What Case.reference and Case.check read, of tensors on the device."""
    c = Case.__new__(Case)
    c.q, c.k, c.v, c.log_decay, c.scale, c.lens, c.lead = q.cpu(), k.cpu(), v.cpu(), log_decay.cpu(), scale, lens, 0
    c.H, c.Hk, c.dk, c.dv = q.shape[1], k.shape[1], q.shape[2], v.shape[2]
    c.state, c.in_slots, c.out_slots = state.cpu(), ins.cpu(), outs.cpu()
    return c


class Linear:
    """The linear layer: decays, a pool of states and calls that are checked."""

    def __init__(self, H, Hk, slots, g):
        self.H, self.Hk, self.g = H, Hk, g
        self.log_decay = -torch.exp2(-torch.linspace(1.0, 9.0, H)).to(DEV)
        self.state = torch.full((slots, H, DK, DV), math.nan, device=DEV)
        self.scale = DK ** -0.5

    def tokens(self, n):
        x = torch.randn((n, self.H * DK + self.Hk * (DK + DV)), generator=self.g).to(torch.bfloat16).to(DEV)
        q, k, v = x.split([self.H * DK, self.Hk * DK, self.Hk * DV], dim=1)
        return q.view(n, self.H, DK), k.view(n, self.Hk, DK), v.view(n, self.Hk, DV)

    def prompt(self, lens, ins, outs):
        q, k, v = self.tokens(sum(lens))
        ins, outs = (torch.tensor(s, dtype=torch.int32, device=DEV) for s in (ins, outs))
        starts = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
        before = self.state.clone()
        out = binding.linear_prefill(q, k, v, self.log_decay, self.scale, starts, self.state, ins, outs)
        linear_case(q, k, v, self.log_decay, self.scale, lens, before, ins, outs).check(out, self.state)

    def step(self, T, slots):
        q, k, v = self.tokens(T * slots.numel())
        before = self.state.clone()
        out = binding.linear_decode(q, k, v, self.log_decay, self.scale, self.state, T, slots)
        linear_case(q, k, v, self.log_decay, self.scale, [T] * slots.numel(), before, slots, slots).check(
            out, self.state, "decode")


def attention_case(m, prefix_len, lens, T, H, q):
    """What Shared.check reads: sequence 0 of the model is the prefix, the others the requests."""
    c = Shared.__new__(Shared)
    c.P, c.T, c.H, c.lens, c.q = prefix_len, T, H, lens, q.cpu()

    class Rows:
        def __init__(self, first):
            self.first, self.s_max = first, 1 << 30

        def rows(self, b, pos):
            return m.rows(self.first + b, pos)

    c.first, c.own = Rows(0), Rows(1)
    return c


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,page", [(1, 16, 64), (2, 32, 16), (1, 128, 24)])
def test_fork_then_steps(fp8, T, H, page):
    prefix, own = 300, [70, 0, 129, 5]
    m = Model([prefix] + own, T, H, page, fp8, room=10, seed=T)
    lin = Linear(8, 4, 6, m.g)
    # the prefix, once: its linear state into slot 5, its latent rows onto its pages
    lin.prompt([prefix], [-1], [5])
    pos = torch.arange(prefix, device=DEV)
    binding.norm_rope(None, m.heads(m.new(prefix, 1), m.slots(torch.zeros_like(pos), pos)), m.rope, pos, **ROPE)
    # the requests' own prompts: every state goes on from slot 5, which stays
    kept = lin.state[5].clone()
    lin.prompt(own, [5] * 4, [0, 1, 2, 3])
    assert torch.equal(lin.state[5], kept)
    b = torch.cat([torch.full((n,), i + 1) for i, n in enumerate(own)]).to(DEV)
    at = torch.cat([torch.arange(n) for n in own]).to(DEV)                # in the request's own pages
    binding.norm_rope(None, m.heads(m.new(b.numel(), 1), m.slots(b, at)), m.rope, at, **ROPE)
    first = binding.Cache(None, m.pool, m.lens[:1], block_table=m.table[:1], page_size=page, latent_scale=m.scales)
    cache = binding.Cache(None, m.pool, m.lens[1:], block_table=m.table[1:], page_size=page, latent_scale=m.scales)
    slots = torch.arange(4, dtype=torch.int32, device=DEV)
    for _ in range(3):
        m.lens[1:] += T
        at = (m.lens[1:].long()[:, None] - T + torch.arange(T, device=DEV)).reshape(-1)
        b = torch.arange(1, 5, device=DEV).repeat_interleave(T)
        q, _ = binding.norm_rope(binding.Heads(m.new(4 * T, H)), m.heads(m.new(4 * T, 1), m.slots(b, at)), m.rope, at, **ROPE)
        out, lse = binding.prefix_mla_decode(q, first, cache, SCALE, tokens_per_seq=T)
        torch.cuda.synchronize()
        attention_case(m, prefix, m.lens[1:].tolist(), T, H, q).check(out, lse)
        lin.step(T, slots)
    assert torch.equal(lin.state[5], kept)


def test_captured_steps():
    """A step of both layers in one graph; lengths and cache slots advance on the device, so that
    replays go on from each other."""
    H, page, prefix, own = 16, 64, 700, [3, 64, 0]
    m = Model([prefix] + own, 1, H, page, False, room=80, seed=9)
    lin = Linear(4, 4, 4, m.g)
    lin.prompt([prefix], [-1], [3])
    lin.prompt([1, 1, 1], [3, 3, 3], [0, 1, 2])
    b = torch.cat([torch.full((n,), i) for i, n in enumerate([prefix] + own)]).to(DEV)
    at = torch.cat([torch.arange(n) for n in [prefix] + own]).to(DEV)
    binding.norm_rope(None, m.heads(m.new(b.numel(), 1), m.slots(b, at)), m.rope, at, **ROPE)
    first = binding.Cache(None, m.pool, m.lens[:1], block_table=m.table[:1], page_size=page)
    own_lens = m.lens[1:]
    cache = binding.Cache(None, m.pool, own_lens, block_table=m.table[1:], page_size=page)
    seqs, slots = torch.arange(1, 4, device=DEV), torch.arange(3, dtype=torch.int32, device=DEV)
    pos, dst = (torch.zeros(3, dtype=torch.int64, device=DEV) for _ in range(2))
    x, raw = m.new(3, 1), m.new(3, H)
    queries, keys = binding.Heads(raw), m.heads(x, dst)
    lq, lk, lv = lin.tokens(3)
    lout = torch.empty((3, 4, DV), dtype=torch.bfloat16, device=DEV)
    out, lse = torch.empty((3, H, 512), dtype=torch.bfloat16, device=DEV), torch.empty((3, H), device=DEV)
    wsp = binding.alloc_workspace(binding.prefix_mla_workspace_size(3, H), DEV)

    def step():
        pos.copy_(own_lens)
        own_lens.add_(1)
        dst.copy_(m.slots(seqs, pos))
        binding.norm_rope(queries, keys, m.rope, pos, **ROPE)
        binding.prefix_mla_decode(queries.out, first, cache, SCALE, out=out, lse=lse, workspace=wsp)
        binding.linear_decode(lq, lk, lv, lin.log_decay, lin.scale, lin.state, 1, slots, out=lout)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        for i in range(66):                          # over a page's end in every sequence
            x.copy_(m.new(3, 1))
            raw.copy_(m.new(3, H))
            if i == 65:
                stream.synchronize()
                before = lin.state.clone()
            graph.replay()
    stream.synchronize()
    assert m.lens.tolist() == [prefix] + [n + 67 for n in own]
    attention_case(m, prefix, own_lens.tolist(), 1, H, queries.out).check(out, lse)
    linear_case(lq, lk, lv, lin.log_decay, lin.scale, [1] * 3, before, slots, slots).check(lout, lin.state, "decode")
