"""dsi_norm_rope where a warp takes many vectors one after another: the ring of copies wraps, the
maxima of a vector's scale groups follow those of the one before, destinations and positions are
looked up ahead, and the last warps' steps end early.  Every value, code and scale is compared with
the formula in 64 bits.

Tolerances: those of the operator's other tests (fp32 arithmetic within 2^-15 M).  A code has to lie
between the codes of z - e and z + e, divided by the stored scale, with e = 2^-15 M + 2^-20 |z| for the
arithmetic and the division or reciprocal: rounding to E4M3 is monotone."""
import pytest
import torch

from indexed_sparse_attention_indexer_gb300 import binding
from tests.test_gpu_norm_rope import check_bf16, reference

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _inputs(n, heads, d, norm, nd, seed, bias=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, heads, d), generator=g)
    x = (x * torch.exp(torch.empty((n, 1, 1)).uniform_(-3, 3, generator=g))).to(torch.bfloat16).to(DEV)
    w = torch.empty(nd).uniform_(-1.5, 1.5, generator=g).to(DEV) if norm else None
    b = torch.empty(nd).uniform_(-1, 1, generator=g).to(DEV) if norm == "layer" and bias else None
    return x, w, b, torch.randint(0, 3000, (n,), generator=g).to(DEV), g


def _scattered(n, g, skipped):
    """Destinations in a pool of n + 50 rows, every `skipped`-th of them negative."""
    rows = torch.randperm(n + 50, generator=g)[:n]
    rows[3::skipped] = -1
    return rows


def _check_codes(codes, scale, z, M):
    """codes E4M3 and scale (fp64, one a dim) against z: see the top of the file."""
    live = scale > 0
    s = torch.where(live, scale, torch.ones_like(scale))
    e = 2.0 ** -15 * M + 2.0 ** -20 * z.abs()
    lo, hi = (((z + k * e) / s).clamp(-448, 448).float().to(torch.float8_e4m3fn).float() for k in (-1, 1))
    got = codes.float()
    assert bool((((got >= lo) & (got <= hi)) | ~live).all())
    assert bool((got[~live] == 0).all())
    # and hardly any of them needs the interval: errors of some 2^-22 M, spread evenly, carry a code
    # over a midpoint where it is that near, about 2^-22 / 2^-5 of the codes (steps are 2^-4 to 2^-3 of z)
    near = (z / s).clamp(-448, 448).float().to(torch.float8_e4m3fn).float()
    assert float((got != near)[live].float().mean()) < 1e-3


def _untouched(pool, rows, value):
    left = torch.ones(pool.shape[0], dtype=torch.bool)
    left[rows[rows >= 0]] = False
    assert bool((pool.view(torch.uint8)[left.to(DEV)] == value).all())


@pytest.mark.parametrize("norm,interleaved", [("rms", True), ("layer", False), (None, True)])
def test_latent_rows_to_fp8(norm, interleaved):
    n, d = 20001, 576
    x, w, b, pos, g = _inputs(n, 1, d, norm, 512, 1)
    x[77], x[20000] = 0, 0                       # all-zero vectors between others
    rows = _scattered(n, g, 9)
    table = binding.rope_table(3000, 64, device=DEV)
    codes = torch.full((n + 50, d), 0x11, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    scales = torch.full((n + 50, 5), -1.0, device=DEV)
    binding.norm_rope(None, binding.Heads(x, norm, w, b, 512, out=codes, out_scale=scales, dst_rows=rows.to(DEV)),
                      table, pos, rope_offset=512, interleaved=interleaved)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    z, M = reference(x, norm, w, b, 512, table, pos, 512, interleaved, 1e-6)
    keep = rows >= 0
    z, M = z[keep, 0], M[keep, 0]
    got = scales[rows[keep].to(DEV)].cpu().double()
    s = torch.nn.functional.pad(z, (0, 64)).unflatten(-1, (5, 128)).abs().amax(-1) / 448
    assert bool(((got - s).abs() <= 2.0 ** -23 * s + 2.0 ** -15 * M / 448).all())
    _check_codes(codes[rows[keep].to(DEV)].cpu(), got.repeat_interleave(128, dim=-1)[:, :d], z, M)
    _untouched(codes, rows, 0x11)
    left = torch.ones(n + 50, dtype=torch.bool)
    left[rows[keep]] = False
    assert bool((scales[left.to(DEV)] == -1).all())


@pytest.mark.parametrize("n,heads,d,group", [(30001, 1, 128, 32), (30001, 3, 128, 64), (9001, 5, 256, 128),
                                             (20003, 2, 96, 32), (6001, 1, 960, 32)])
def test_keys_to_mxfp8(n, heads, d, group):
    """One unit a lane (d of 128 and 256), three and four."""
    rd = 64 if d != 96 else 96
    x, w, b, pos, g = _inputs(n, heads, d, "layer", d, 2)
    rows = _scattered(n, g, 11)
    table = binding.rope_table(3000, rd, device=DEV)
    codes = torch.full((n + 50, heads, d), 0x11, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    scales = torch.full((n + 50, heads, d // group), 9, dtype=torch.uint8, device=DEV)
    binding.norm_rope(None, binding.Heads(x, "layer", w, b, out=codes, out_scale=scales, dst_rows=rows.to(DEV)),
                      table, pos)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    z, M = reference(x, "layer", w, b, d, table, pos, 0, False, 1e-6)
    keep = rows >= 0
    z, M = z[keep], M[keep]
    big = z.unflatten(-1, (d // group, group)).abs().amax(-1)
    X = torch.floor(torch.log2(big)) - 8
    got = scales[rows[keep].to(DEV)].cpu().double() - 127
    # the exponent can differ only where the maximum sits at a power of two, within the fp32 error
    edge = (torch.log2(big) - torch.round(torch.log2(big))).abs() < 2.0 ** -14 * (M / big)
    assert bool(((got == X) | (edge & ((got - X).abs() <= 1))).all())
    _check_codes(codes[rows[keep].to(DEV)].cpu(), torch.pow(2.0, got).repeat_interleave(group, dim=-1), z, M)
    _untouched(codes, rows, 0x11)
    _untouched(scales, rows, 9)


@pytest.mark.parametrize("norm", ["rms", "layer", None])
@pytest.mark.parametrize("n,hq,hk,d,ro,rd,interleaved", [
    (6007, 5, 2, 96, 0, 96, False),              # three units a lane
    (5003, 7, 1, 200, 8, 64, True),              # four
    (7411, 1, 0, 1024, 0, 512, False),           # two
    (30011, 3, 1, 64, 0, 32, True),              # one
    (20011, 2, 3, 80, 48, 32, False)])
def test_bf16_rows(norm, n, hq, hk, d, ro, rd, interleaved):
    q, qw, qb, pos, _ = _inputs(n, hq, d, norm, d, 3)
    k, kw, kb, _, g = _inputs(n, max(hk, 1), d, norm, d, 4, bias=False)
    rows = _scattered(n, g, 7)
    table = binding.rope_table(3000, rd, device=DEV)
    pool = torch.full((n + 50, hk, d), 7.0, dtype=torch.bfloat16, device=DEV)
    out, _ = binding.norm_rope(
        binding.Heads(q, norm, qw, qb),
        binding.Heads(k, norm, kw, kb, out=pool, dst_rows=rows.to(DEV)) if hk else None,
        table, pos, rope_offset=ro, interleaved=interleaved)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    check_bf16(out, *reference(q, norm, qw, qb, d, table, pos, ro, interleaved, 1e-6))
    if hk:
        keep = rows >= 0
        z, M = reference(k, norm, kw, kb, d, table, pos, ro, interleaved, 1e-6)
        check_bf16(pool[rows[keep].to(DEV)], z[keep], M[keep])
        left = torch.ones(n + 50, dtype=torch.bool)
        left[rows[keep]] = False
        assert bool((pool[left.to(DEV)] == 7).all())


def test_in_place_over_many_steps():
    """x as out: vectors are copied ahead of the ones that are being written."""
    q, w, _, pos, _ = _inputs(30011, 3, 128, "rms", 128, 5)
    table = binding.rope_table(3000, 64, device=DEV)
    expect, _ = binding.norm_rope(binding.Heads(q, "rms", w), None, table, pos)
    binding.norm_rope(binding.Heads(q, "rms", w, out=q), None, table, pos)
    torch.cuda.synchronize()
    assert torch.equal(q, expect)
