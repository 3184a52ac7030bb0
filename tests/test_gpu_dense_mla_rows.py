"""Attention over the whole latent cache and over windows: rows do not depend on the entry that
computes them or on what else is in the call, and rows that see something infinite say so."""
import math

import pytest
import torch

from indexed_sparse_attention_indexer_gb300 import binding
from tests.test_gpu_dense_mla import SCALE, Case, check, decode_views

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H", [(4, 32), (1, 128), (3, 20), (5, 128)])
def test_decode_and_prefill_give_the_same_bits(T, H, fp8):
    """The last tokens of one sequence through either entry: the same groups, tiles and order."""
    n, window, sink = 333, 100, 3
    case = Case([n], T, H, 64, fp8, seed=8)
    cache = case.device()
    a, la = binding.window_mla_decode(case.d_q, cache, window, sink, SCALE, tokens_per_seq=T)
    b, lb = binding.window_mla_prefill(case.d_q, cache, n - T, window, sink, SCALE)
    torch.cuda.synchronize()
    check(case, a, la, decode_views(case, window, sink))
    assert torch.equal(a, b) and torch.equal(la, lb)


def _without_workspace(case, cache, T, H):
    out = torch.empty((case.q.shape[0], H, 512), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((case.q.shape[0], H), device=DEV)
    assert binding.load().dsi_dense_mla_decode(binding._ptr(case.d_q), cache.ref(), T, H, SCALE, binding._ptr(out),
                                               binding._ptr(lse), None, 0, binding._stream(None)) == 0
    return out, lse


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H", [(1, 128), (2, 48)])
def test_rows_do_not_depend_on_the_others(T, H, fp8):
    """A sequence alone or among others.  Without a workspace nothing is split: the same bits.  With one
    a sequence may be split elsewhere: the formula's bounds hold either way."""
    lens = [2500, 40, 333, 0, 1000]
    case = Case(lens, T, H, 64, fp8, seed=9, garbage=False)
    cache = case.device()
    out, lse = _without_workspace(case, cache, T, H)
    split, split_lse = binding.dense_mla_decode(case.d_q, cache, SCALE, tokens_per_seq=T)
    check(case, out, lse, decode_views(case))
    check(case, split, split_lse, decode_views(case))
    for b in range(len(lens)):
        rows = slice(b * T, b * T + T)
        q = case.d_q[rows].contiguous()
        alone = Case([1], T, H, seed=0)
        alone.q, alone.d_q = q, q
        one = binding.Cache(None, case.d_latent, case.seq_lens[b:b + 1], block_table=case.d_table[b:b + 1],
                            page_size=64, latent_scale=cache.latent_scale)
        o, l = _without_workspace(alone, one, T, H)
        torch.cuda.synchronize()
        assert torch.equal(o, out[rows]) and torch.equal(l, lse[rows])
        o, l = binding.dense_mla_decode(q, one, SCALE, tokens_per_seq=T)
        torch.cuda.synchronize()
        split[rows], split_lse[rows] = o, l
    check(case, split, split_lse, decode_views(case))


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_partly_visible_row_that_is_not_finite(bad):
    """Seen by the later tokens of a step only: their outputs and their lse are NaN, whichever dim it is
    in; the earlier tokens' are those of a cache without it, bit for bit."""
    for dim in (5, 300, 520, 575):
        case = Case([200, 200], 4, 16, seed=11, garbage=False)
        clean, clean_lse = binding.dense_mla_decode(case.q.to(DEV), case.device(), SCALE, tokens_per_seq=4)
        case.latent[0, 198, dim] = bad              # position 198: tokens 2 and 3
        out, lse = binding.dense_mla_decode(case.q.to(DEV), case.device(), SCALE, tokens_per_seq=4)
        torch.cuda.synchronize()
        keep = torch.tensor([0, 1, 4, 5, 6, 7], device=DEV)
        assert torch.equal(out[keep], clean[keep]) and torch.equal(lse[keep], clean_lse[keep])
        assert bool(torch.isnan(out[2:4]).all()) and bool(torch.isnan(lse[2:4]).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("sink", [0, 130])
def test_a_row_that_leaves_the_window(sink, fp8):
    """Not finite and seen by the first tokens of a step only, at the window's lower edge: theirs alone."""
    n, T, H, window = 900, 4, 16, 333
    lo = n - T + 1 - window                          # the first token's first position
    for dim in (7, 400, 570):
        case = Case([n, 50], T, H, 64, fp8, seed=21, garbage=False)
        clean, clean_lse = binding.window_mla_decode(case.q.to(DEV), case.device(), window, sink, SCALE,
                                                     tokens_per_seq=T)
        at = int(case.phys(0, torch.tensor([lo + 1])))                 # tokens 0 and 1
        if fp8:
            case.latent.view(torch.uint8).view(-1, 576)[at, dim] = 0x7F
        else:
            case.latent.view(-1, 576)[at, dim] = math.inf
        out, lse = binding.window_mla_decode(case.q.to(DEV), case.device(), window, sink, SCALE, tokens_per_seq=T)
        torch.cuda.synchronize()
        assert torch.equal(out[2:], clean[2:]) and torch.equal(lse[2:], clean_lse[2:])
        assert bool(torch.isnan(out[:2]).all()) and bool(torch.isnan(lse[:2]).all())
        assert binding.device_status() == 0


@pytest.mark.parametrize("lens", [[70, 300], [9000, 70]], ids=["whole", "split"])
def test_logits_that_are_all_minus_infinity(lens):
    """A head whose query makes every logit -inf weighs nothing: zeros, and an lse of -inf."""
    case = Case(lens, 1, 32, 64, seed=23, garbage=False)
    case.latent[..., 10] = case.latent[..., 10].abs() + 0.5
    cache = case.device()
    clean, clean_lse = (t.clone() for t in binding.dense_mla_decode(case.d_q, cache, SCALE))
    case.d_q[0, 5, 10] = case.d_q[1, 31, 10] = -math.inf
    out, lse = binding.dense_mla_decode(case.d_q, cache, SCALE)
    torch.cuda.synchronize()
    hit = torch.zeros((2, 32), dtype=torch.bool, device=DEV)
    hit[0, 5] = hit[1, 31] = True
    assert bool((out[hit] == 0).all()) and bool((lse[hit] == -math.inf).all())
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])


def test_the_checked_library():
    """The build with bounds checks gives the same bits."""
    case = Case([2000, 5, 0], 2, 48, 16, True, seed=22, garbage=False)
    cache = case.device()
    for call in (lambda c: binding.dense_mla_decode(case.d_q, cache, SCALE, tokens_per_seq=2, checked=c),
                 lambda c: binding.window_mla_decode(case.d_q, cache, 70, 3, SCALE, tokens_per_seq=2, checked=c)):
        a, b = call(False), call(True)
        torch.cuda.synchronize()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    table, pos = binding.rope_table(3000, 64, device=DEV), torch.arange(6, device=DEV)
    a, b = (binding.norm_rope(binding.Heads(case.d_q, "rms"), None, table, pos, rope_offset=512, checked=c)[0]
            for c in (False, True))
    torch.cuda.synchronize()
    assert torch.equal(a, b) and binding.device_status() == 0 and binding.device_status(checked=True) == 0


def test_a_first_call_that_is_captured():
    """A process whose first calls of the library are captured into a graph."""
    import os
    import subprocess
    import sys
    code = """
import torch
from indexed_sparse_attention_indexer_gb300 import binding as B
q = torch.randn((3, 16, 576), device="cuda").bfloat16()
lat = torch.randn((3, 3000, 576), device="cuda").bfloat16()
lens = torch.tensor([3000, 5, 700], dtype=torch.int32, device="cuda")
cache, pos = B.Cache(None, lat, lens), torch.arange(3, device="cuda")
table = B.rope_table(10, 64)
heads = B.Heads(q)
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    r, _ = B.norm_rope(heads, None, table, pos, rope_offset=512)
    out, lse = B.dense_mla_decode(r, cache, 0.04)
graph.replay()
torch.cuda.synchronize()
got = out.clone(), lse.clone()
r, _ = B.norm_rope(B.Heads(q), None, table, pos, rope_offset=512)
want = B.dense_mla_decode(r, cache, 0.04)
torch.cuda.synchronize()
assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and B.device_status() == 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
