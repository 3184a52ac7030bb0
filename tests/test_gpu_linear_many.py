"""Prefills of linear attention over hundreds and thousands of sequences, most of them decoding rows.

The long sequences have to come out as in a call of their own, the rows of one token as from the decode
call, bit for bit (both are held against 64 bits in test_gpu_linear)."""
import math

import pytest
import torch

from indexed_sparse_attention_indexer_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"


def inputs(n, H, d, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q, k, v = (torch.randn((n, H, d), generator=g, device=DEV).to(torch.bfloat16) for _ in range(3))
    return q, k, v, -torch.rand(H, generator=g, device=DEV) * 0.2


def starts_of(lens):
    return torch.tensor([0] + list(lens), device=DEV).cumsum(0).to(torch.int32)


LONG = [dict(B=257, at={0: 9}), dict(B=257, at={256: 300}), dict(B=300, at={7: 130, 8: 9, 299: 40}), dict(B=2048, at={2047: 200, 31: 9}),
        dict(B=2049, at={2048: 77, 2047: 10, 1: 129}), dict(B=2049, at={}), dict(B=5003, at={5002: 9, 2500: 600, 2501: 9, 4: 12, 0: 128}),
        dict(B=5000, at={i: 9 + i % 140 for i in range(11, 5000, 37)}), dict(B=40000, at={39999: 9, 20000: 400}),
        dict(B=70001, at={i: 9 for i in range(0, 70001, 4999)} | {35000: 260}), dict(B=4500, at={i: 9 for i in range(1000, 3600)}),
        dict(B=3000, at={}, empty=3), dict(B=3000, at={i: 30 for i in range(2900, 3000)}, empty=2)]


@pytest.mark.parametrize("kw", LONG, ids=lambda kw: f"{kw['B']}-{len(kw['at'])}-{kw.get('empty', 0)}")
@pytest.mark.parametrize("H,d", [(1, 8), (5, 72)])
def test_long_sequences_among_many_short_ones(kw, H, d):
    B, at, empty = kw["B"], kw["at"], kw.get("empty", 0)
    lens = [at.get(b, 0 if empty and b % empty == 0 else 1) for b in range(B)]
    starts = starts_of(lens)
    q, k, v, decay = inputs(sum(lens), H, d, seed=B)
    state = torch.randn((B, H, d, d), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    first = state.clone()
    out = binding.linear_prefill(q, k, v, decay, 0.3, starts, state)
    assert binding.device_status() == 0
    one = torch.tensor([b for b in range(B) if lens[b] == 1], dtype=torch.int64, device=DEV)
    rows = starts[:-1].long()[one]
    want = first.clone()
    slots = one.to(torch.int32)
    y = binding.linear_decode(q[rows], k[rows], v[rows], decay, 0.3, want, in_slots=slots)
    assert torch.equal(out[rows], y) and torch.equal(state[one], want[one])
    for lo in range(0, len(at), 200):
        part = sorted(at)[lo:lo + 200]
        rows = torch.cat([torch.arange(int(starts[b]), int(starts[b + 1]), device=DEV) for b in part])
        slots = torch.tensor(part, dtype=torch.int32, device=DEV)
        want = first.clone()
        y = binding.linear_prefill(q[rows], k[rows], v[rows], decay, 0.3, starts_of([lens[b] for b in part]), want,
                                   in_slots=slots)
        assert torch.equal(out[rows], y) and torch.equal(state[slots.long()], want[slots.long()])
    assert binding.device_status() == 0


def test_a_cta_that_finds_nothing_for_long():
    """Long sequences wherever the first CTA's pieces are not: it goes through 5000 rounds and has none.  With
    a decay to nothing out_i = scale (q_i . k_i) v_i: the weight and out are rounded to bf16."""
    G, rounds, d = torch.cuda.get_device_properties(0).multi_processor_count, 5000, 8
    i = torch.arange(G * rounds, device=DEV)
    lens = torch.where((i % (2 * G) == 0) | (i % (2 * G) == 2 * G - 1), 1, 9)
    starts = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), lens.cumsum(0)]).to(torch.int32)
    q, k, v, decay = inputs(int(starts[-1]), 1, d)
    out = binding.linear_prefill(q, k, v, torch.full_like(decay, -math.inf), 0.5, starts)
    assert binding.device_status() == 0
    q, k, v = q.double(), k.double(), v.double()
    want = 0.5 * (q * k).sum(-1, keepdim=True) * v
    far = 0.5 * (q * k).abs().sum(-1, keepdim=True) * v.abs()
    assert bool(((out.double() - want).abs() <= 2.0 ** -7 * want.abs() + (d + 4) * 2.0 ** -22 * far + 1e-37).all())


@pytest.mark.parametrize("B,H,d", [(65536, 16, 8), (2048, 16, 16)])
def test_short_rows_cost_what_they_do_as_a_step(B, H, d):
    """The search for long sequences is not what the call takes its time for."""
    def least(call):
        for _ in range(3):
            call()
        times = []
        for _ in range(10):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            torch.cuda.synchronize()
            torch.cuda._sleep(200000)         # (the host is ahead)
            a.record()
            call()
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    q, k, v, decay = inputs(B, H, d)
    out, starts = torch.empty_like(v), starts_of([1] * B)
    prefill = least(lambda: binding.linear_prefill(q, k, v, decay, 0.3, starts, out=out))
    step = least(lambda: binding.linear_decode(q, k, v, decay, 0.3, out=out))
    assert prefill <= 1.4 * step + 0.02       # ms: a launch or two (measured: 1.10 and 1.15 times)
