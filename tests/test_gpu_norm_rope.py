"""Head norms with position rotation (dsi_norm_rope) against the formulas in 64 bits.

Tolerances.  The kernel computes in fp32 and rounds once.  A result z is off by
  - the final rounding: half a step, 2^-8 |z| for bf16 (finfo.eps / 2), 2^-4 |z| or half of the
    smallest subnormal step, 2^-10 of the scale, for E4M3;
  - the fp32 arithmetic.  A norm's sum has at most 32 * 16 terms in one lane's chain and five
    shuffle steps, all of one sign (squares) or bounded by the sum of magnitudes (means): a
    relative error below (64 + 5) * 2^-24 < 2^-17; rsqrt, the products and the rotation's two
    products and sum add less than 8 * 2^-24.  Every one of these errors is relative to terms
    no larger than M = r * max|x| * max|w| + max|b| (normed dims) or max|x| (the others), twice
    that in a rotation of two dims: below 2^-15 M in all.
"""
import math

import pytest
import torch

from indexed_sparse_attention_indexer_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"


def reference(x, norm, weight, bias, norm_dim, table, pos, ro, interleaved, eps):
    """(z [n, h, d], M [n, h, 1]) in fp64."""
    y = x.double().cpu().clone()
    M = y.abs().amax(-1, keepdim=True)
    if norm is not None:
        v = y[..., :norm_dim]
        big = v.abs().amax(-1, keepdim=True)
        if norm == "layer":
            v = v - v.mean(-1, keepdim=True)
        r = 1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
        v = v * r
        w = weight.double().cpu() if weight is not None else torch.ones(norm_dim, dtype=torch.float64)
        v = v * w
        Mn = r * big * w.abs().max()
        if bias is not None:
            v = v + bias.double().cpu()
            Mn = Mn + bias.double().cpu().abs().max()
        y[..., :norm_dim] = v
        rest = y[..., norm_dim:].abs().amax(-1, keepdim=True) if norm_dim < y.shape[-1] else torch.zeros_like(Mn)
        M = torch.maximum(Mn, rest)
    rd = table.shape[1]
    cs = table.double().cpu()[pos.cpu()][:, None]
    i = torch.arange(rd // 2)
    a, b = (ro + 2 * i, ro + 2 * i + 1) if interleaved else (ro + i, ro + i + rd // 2)
    ya, yb, c, s = y[..., a], y[..., b], cs[..., :rd // 2], cs[..., rd // 2:]
    z = y.clone()
    z[..., a], z[..., b] = ya * c - yb * s, ya * s + yb * c
    return z, M


def check_bf16(got, z, M):
    err = (got.double().cpu() - z).abs()
    tol = 2.0 ** -8 * z.abs() + 2.0 ** -15 * M
    assert bool((err <= tol).all()), float((err / tol).max())


def _side(g, n, heads, d, norm, norm_dim, weight=True, bias=None, pad=0):
    x = torch.randn((n, heads * d + pad), generator=g)
    x = (x * torch.exp(torch.empty((n, 1)).uniform_(-3, 3, generator=g))).to(torch.bfloat16).to(DEV)
    x = x[:, :heads * d].view(n, heads, d) if pad == 0 else x[:, :heads * d].unflatten(1, (heads, d))
    w = torch.empty(norm_dim).uniform_(-1.5, 1.5, generator=g).to(DEV) if weight and norm else None
    b = torch.empty(norm_dim).uniform_(-1, 1, generator=g).to(DEV) if norm == "layer" and bias is not False else None
    return x, w, b


CASES = [
    # n, hq, hk, d, norm_q, norm_k, norm_dim, rope_offset, rope_dim, interleaved
    (1, 1, 1, 16, "rms", "rms", 16, 0, 16, False),
    (1, 64, 1, 128, "rms", "layer", 128, 0, 64, False),
    (5, 3, 2, 128, None, "layer", 128, 64, 64, True),
    (33, 40, 8, 96, "rms", "rms", 96, 0, 96, False),
    (7, 5, 1, 80, "layer", None, 80, 0, 80, True),
    (9, 2, 3, 80, "rms", "layer", 40, 40, 32, False),
    (129, 0, 1, 576, None, "rms", 512, 512, 64, True),
    (130, 4, 1, 576, None, "layer", 512, 512, 64, False),
    (3, 7, 7, 1024, "rms", "layer", 1024, 0, 1024, False),
    (2, 1, 2, 1016, "layer", "rms", 8, 8, 16, False),
    (1000, 17, 1, 24, "rms", None, 24, 8, 16, True),
    (4099, 6, 2, 64, "layer", "rms", 64, 0, 32, False),
]


@pytest.mark.parametrize("case", CASES, ids=[f"n{c[0]}_h{c[1]}+{c[2]}_d{c[3]}" for c in CASES])
@pytest.mark.parametrize("pad", [0, 8])
def test_matches_formulas(case, pad):
    n, hq, hk, d, nq, nk, nd, ro, rd, il = case
    g = torch.Generator().manual_seed(n + d + pad)
    table = binding.rope_table(5000, rd, device=DEV)
    pos = torch.randint(0, 5000, (n,), generator=g).to(DEV)
    pos[0] = 4999
    q, qw, qb = _side(g, n, hq, d, nq, nd, pad=pad)
    k, kw, kb = _side(g, n, hk, d, nk, nd, weight=pad == 0, pad=pad)
    qo, ko = binding.norm_rope(
        binding.Heads(q, nq, qw, qb, nd) if hq else None, binding.Heads(k, nk, kw, kb, nd),
        table, pos, rope_offset=ro, interleaved=il, eps=1e-5)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    if hq:
        check_bf16(qo, *reference(q, nq, qw, qb, nd, table, pos, ro, il, 1e-5))
    check_bf16(ko, *reference(k, nk, kw, kb, nd, table, pos, ro, il, 1e-5))


def test_in_place_and_special_rows():
    """x as out; an all-zero vector (eps alone under the root), a constant one (no variance), large
    and tiny values, position 0 (no rotation)."""
    g = torch.Generator().manual_seed(4)
    n, h, d = 6, 2, 128
    x, w, b = _side(g, n, h, d, "layer", d)
    x[0], x[1], x[2], x[3] = 0, 3.0, x[2] * 1e15, x[3] * 1e-18
    pos = torch.zeros(n, dtype=torch.int64, device=DEV)
    pos[2:] = torch.arange(n - 2, device=DEV) * 100
    table = binding.rope_table(1000, 64, device=DEV)
    for norm, bias in (("rms", None), ("layer", b), (None, None)):
        y = x.clone()
        z, M = reference(x, norm, w if norm else None, bias, d, table, pos, 0, False, 1e-6)
        binding.norm_rope(binding.Heads(y, norm, w if norm else None, bias, out=y), None, table, pos)
        torch.cuda.synchronize()
        check_bf16(y, z, M)
    # zero rows of an RMS norm stay zero; position 0 leaves an unnormed vector bit for bit
    assert torch.equal(y[1], x[1])


def test_cache_rows():
    """dst_rows scatters into a pool: negative entries skip, rows out of range and positions out of
    the table are skipped and reported, other rows stay as they were."""
    g = torch.Generator().manual_seed(5)
    n, d, pages, page = 40, 128, 4, 16
    k, w, b = _side(g, n, 1, d, "layer", d)
    rows = torch.randperm(pages * page, generator=g)[:n]
    rows[3], rows[11] = -1, -(1 << 40)
    pos = torch.arange(n) * 3
    table = binding.rope_table(3 * n, 64, device=DEV)
    z, M = reference(k, "layer", w, b, d, table, pos, 0, False, 1e-6)

    def run(rows, pos):
        pool = torch.full((pages, page, d), 7.0, dtype=torch.bfloat16, device=DEV)
        binding.norm_rope(None, binding.Heads(k, "layer", w, b, out=pool, dst_rows=rows.to(DEV)), table,
                          pos.to(DEV))
        torch.cuda.synchronize()
        return pool.view(-1, d), binding.device_status()

    pool, status = run(rows, pos)
    assert status == 0
    keep = rows >= 0
    check_bf16(pool[rows[keep].to(DEV)], z[keep, 0], M[keep, 0])
    others = torch.ones(pages * page, dtype=torch.bool)
    others[rows[keep]] = False
    assert bool((pool[others.to(DEV)] == 7).all())
    # out of range: reported once, the good rows still written
    far, late = rows.clone(), pos.clone()
    far[5], late[6], late[7] = pages * page, 3 * n, -1
    pool2, status = run(far, late)
    assert status == binding.DSI_ERR_BOUNDS and binding.device_status() == 0
    good = keep.clone()
    good[5:8] = False
    assert torch.equal(pool2[rows[good].to(DEV)], pool[rows[good].to(DEV)])
    skipped = rows[5:8][rows[5:8] >= 0].to(DEV)
    assert bool((pool2[skipped] == 7).all())
    # a skipped row's position does not matter
    late = pos.clone()
    late[3] = 1 << 50
    assert run(rows, late)[1] == 0


def _e4m3_close(codes, scale, z, M):
    """Codes times scales against z, clamped where the scale makes it saturate."""
    lim = 448.0 * scale
    zc = torch.maximum(torch.minimum(z, lim), -lim)
    err = (codes.double() * scale - zc).abs()
    # half an E4M3 step of the clamped value, half a subnormal step of the scale, and the fp32
    # arithmetic (which can also carry a value over a midpoint: covered by the same bound)
    tol = 2.0 ** -4 * zc.abs() * (1 + 2.0 ** -14) + 2.0 ** -10 * scale + 2.0 ** -15 * M
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,heads", [(1, 1), (67, 1), (19, 3)])
def test_mxfp8_out(group, n, heads):
    g = torch.Generator().manual_seed(n + group)
    d = 128
    k, w, b = _side(g, n, heads, d, "layer", d)
    if n > 2:
        k[1] = 0
    pos = torch.randint(0, 900, (n,), generator=g).to(DEV)
    table = binding.rope_table(900, 64, device=DEV)
    rows = torch.randperm(n + 5, generator=g)[:n].to(DEV)
    codes = torch.full((n + 5, heads, d), 0x11, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    scales = torch.full((n + 5, heads, d // group), 9, dtype=torch.uint8, device=DEV)
    w2 = None if n == 1 else w
    binding.norm_rope(None, binding.Heads(k, "layer", w2, b, out=codes, out_scale=scales, dst_rows=rows), table, pos)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    z, M = reference(k, "layer", w2, b, d, table, pos, 0, False, 1e-6)
    big = z.unflatten(-1, (d // group, group)).abs().amax(-1)
    X = torch.floor(torch.log2(big)) - 8
    got = scales[rows].cpu().double() - 127
    # the exponent can differ only where the maximum sits at a power of two, within the fp32 error
    edge = (torch.log2(big) - torch.round(torch.log2(big))).abs() < 2.0 ** -14 * (M / big)
    assert bool(((got == X) | (edge & ((got - X).abs() <= 1))).all())
    s = torch.pow(2.0, got).repeat_interleave(group, dim=-1)
    _e4m3_close(codes[rows].cpu().float(), s, z, M)
    left = torch.ones(n + 5, dtype=torch.bool)
    left[rows.cpu()] = False
    assert bool((codes.view(torch.uint8)[left.to(DEV)] == 0x11).all()) and bool((scales[left.to(DEV)] == 9).all())


@pytest.mark.parametrize("n,d", [(1, 576), (131, 576), (10, 200)])
def test_fp8_tiles_out(n, d):
    g = torch.Generator().manual_seed(n + d)
    nd, ro = (512, 512) if d == 576 else (128, 136)
    k, w, _ = _side(g, n, 1, d, "rms", nd)
    if n > 2:
        k[1] = 0                       # all-zero tiles: scale 0, codes 0
    pos = torch.randint(0, 900, (n,), generator=g).to(DEV)
    table = binding.rope_table(900, 64, device=DEV)
    tiles = (d + 127) // 128
    codes = torch.zeros((n, d), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    scales = torch.full((n, tiles), -1.0, device=DEV)
    binding.norm_rope(None, binding.Heads(k, "rms", w, None, nd, out=codes, out_scale=scales), table, pos,
                      rope_offset=ro, interleaved=True)
    torch.cuda.synchronize()
    z, M = reference(k, "rms", w, None, nd, table, pos, ro, True, 1e-6)
    z, M = z[:, 0], M[:, 0]
    pad = torch.nn.functional.pad(z, (0, tiles * 128 - d)).unflatten(-1, (tiles, 128))
    s = pad.abs().amax(-1) / 448
    assert bool(((scales.cpu().double() - s).abs() <= 2.0 ** -23 * s + 2.0 ** -15 * M / 448).all())
    _e4m3_close(codes.cpu().float(), scales.cpu().double().repeat_interleave(128, dim=-1)[:, :d], z, M)
    if n > 2:
        assert bool((scales[1] == 0).all()) and bool((codes.view(torch.uint8)[1] & 0x7F == 0).all())


def test_streams_and_graph():
    """On another stream than the current one, and captured into a graph whose inputs change."""
    g = torch.Generator().manual_seed(9)
    n, d = 50, 128
    q, w, _ = _side(g, n, 8, d, "rms", d)
    k, kw, kb = _side(g, n, 1, d, "layer", d)
    pos = torch.arange(n, device=DEV)
    table = binding.rope_table(200, 64, device=DEV)
    qs, ks = binding.Heads(q, "rms", w), binding.Heads(k, "layer", kw, kb)
    binding.norm_rope(qs, ks, table, pos)
    torch.cuda.synchronize()
    first = qs.out.clone(), ks.out.clone()
    side = torch.cuda.Stream()
    qs.out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    binding.norm_rope(qs, ks, table, pos, stream=side)
    side.synchronize()
    assert torch.equal(qs.out, first[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.norm_rope(qs, ks, table, pos)
    pos.add_(100)
    graph.replay()
    torch.cuda.synchronize()
    z, M = reference(q, "rms", w, None, d, table, pos, 0, False, 1e-6)
    check_bf16(qs.out, z, M)
    assert not torch.equal(ks.out, first[1])


def test_many_rows():
    """More vectors than the resident grid, odd counts on both sides, offsets past 2^31 bytes."""
    g = torch.Generator(device=DEV).manual_seed(3)
    n, hq, d = 70001, 129, 128            # queries of 2.3 GB
    q = torch.randn((n, hq, d), generator=g, device=DEV, dtype=torch.bfloat16)
    pos = torch.randint(0, 300, (n,), generator=g, device=DEV)
    table = binding.rope_table(300, 64, device=DEV)
    out, _ = binding.norm_rope(binding.Heads(q, "rms"), None, table, pos)
    torch.cuda.synchronize()
    pick = torch.tensor([0, 1, n // 2, n - 1], device=DEV)
    z, M = reference(q[pick], "rms", None, None, d, table, pos[pick], 0, False, 1e-6)
    check_bf16(out[pick], z, M)
    assert math.isfinite(float(out[-1].float().sum()))
