"""dsi_norm_rope: dims that the rotation does not touch depend on nothing but themselves and the norm.

An infinity, a NaN or an infinite weight in such a dim stays in it: no other dim of the vector
changes by a bit (without a norm, or outside its dims), and what passes through keeps its bits, the
sign of a zero among them."""
import math

import pytest
import torch

from indexed_sparse_attention_indexer_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"

# d, heads, rope_offset, rope_dim: one unit of dims a lane (32, 64, 128, 256) and several
SHAPES = [(32, 2, 16, 16), (64, 5, 0, 32), (64, 1, 24, 16), (128, 3, 0, 64), (128, 2, 64, 64),
          (256, 2, 96, 64), (512, 1, 0, 64), (80, 2, 0, 32), (96, 1, 32, 64), (576, 1, 512, 64), (1024, 2, 8, 512)]


def _call(x, norm, weight, bias, norm_dim, ro, rd, il):
    n = x.shape[0]
    table = binding.rope_table(300, rd, device=DEV)
    pos = torch.arange(n, device=DEV) * 7 % 300
    out, _ = binding.norm_rope(binding.Heads(x, norm, weight, bias, norm_dim), None, table, pos, rope_offset=ro,
                               interleaved=il)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    return out


def _bits(t):
    return t.contiguous().view(torch.int16)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,heads,ro,rd", SHAPES)
@pytest.mark.parametrize("norm", [None, "rms", "layer"])
def test_special_values_stay_where_they_are(norm, d, heads, ro, rd, interleaved):
    """Outside the rotation and the norm: every vector has one special value in such a dim."""
    g = torch.Generator().manual_seed(d + ro)
    # the norm covers the first 8 dims, or the rotated ones where they come first
    nd = None if norm is None else 8 if ro >= 8 else rd
    free = [i for i in range(d) if not ro <= i < ro + rd and (norm is None or i >= nd)]
    n = 41
    x = torch.randn((n, heads, d), generator=g).to(torch.bfloat16)
    w = torch.empty(nd).uniform_(0.5, 1.5, generator=g).to(DEV) if norm else None
    b = torch.empty(nd).uniform_(-1, 1, generator=g).to(DEV) if norm == "layer" else None
    clean = _call(x.to(DEV), norm, w, b, nd, ro, rd, interleaved)
    free = torch.tensor(free)
    assert torch.equal(_bits(clean[..., free.to(DEV)]), _bits(x[..., free].to(DEV)))
    at = free[torch.randint(0, free.numel(), (n, heads), generator=g)]
    special = torch.tensor([math.inf, -math.inf, math.nan, -0.0, 3e38]).to(torch.bfloat16)
    value = special[torch.arange(n * heads).view(n, heads) % 5]
    dirty = x.scatter(2, at[..., None], value[..., None])
    got = _call(dirty.to(DEV), norm, w, b, nd, ro, rd, interleaved).cpu()
    touched = torch.zeros((n, heads, d), dtype=torch.bool).scatter(2, at[..., None], True)
    assert torch.equal(_bits(got)[~touched], _bits(clean.cpu())[~touched])
    there = got.gather(2, at[..., None])[..., 0]
    nan = torch.isnan(value)
    assert bool(torch.isnan(there[nan]).all()) and torch.equal(_bits(there[~nan]), _bits(value[~nan]))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,ro,rd", [(128, 0, 64), (128, 64, 64), (64, 16, 32), (80, 0, 32), (576, 512, 64)])
def test_infinite_weights_and_biases_stay_in_their_dims(d, ro, rd, interleaved):
    """A normed dim outside the rotation with an infinite weight or bias: that dim alone."""
    g = torch.Generator().manual_seed(d)
    x = torch.randn((9, 2, d), generator=g).to(torch.bfloat16).to(DEV)
    w = torch.empty(d).uniform_(0.5, 1.5, generator=g).to(DEV)
    b = torch.empty(d).uniform_(-1, 1, generator=g).to(DEV)
    free = [i for i in range(d) if not ro <= i < ro + rd]
    at = free[len(free) // 3]
    keep = torch.arange(d, device=DEV) != at
    for norm, which in (("rms", "weight"), ("layer", "weight"), ("layer", "bias")):
        bias = b if norm == "layer" else None
        good = _call(x, norm, w, bias, d, ro, rd, interleaved)
        w2, b2 = w.clone(), b.clone()
        (w2 if which == "weight" else b2)[at] = math.inf
        got = _call(x, norm, w2, b2 if norm == "layer" else None, d, ro, rd, interleaved)
        assert torch.equal(_bits(got[..., keep]), _bits(good[..., keep])), (norm, which)
        assert bool(torch.isinf(got[..., at]).all())


def test_an_infinity_in_a_normed_vector():
    """RMS norm of a vector with an infinity: 1 / sqrt(inf) = 0, so zeros, and NaN in that dim alone
    where the rotation does not mix it with others."""
    x = torch.randn((4, 3, 128), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    x[:, :, 70] = math.inf
    for ro, il in ((0, False), (0, True)):
        got = _call(x, "rms", None, None, 128, ro, 64, il)
        keep = torch.arange(128, device=DEV) != 70
        assert bool((got[..., keep] == 0).all()) and bool(torch.isnan(got[..., 70]).all())
