"""Layouts that the entry points of norms with rotation and of attention over the whole latent cache
take and that a model's buffers have: head-major and interleaved vectors, buffers that start at any
16 bytes, pages of any multiple of 8, long steps through the decode entry."""
import pytest
import torch

from indexed_sparse_attention_indexer_gb300 import binding
from tests.test_gpu_dense_mla import SCALE, Case, check, decode_views
from tests.test_gpu_norm_rope import check_bf16, reference

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("norm", [None, "rms", "layer"])
@pytest.mark.parametrize("n,heads,d,rd", [(37, 5, 128, 64), (1, 3, 96, 96), (300, 2, 576, 64)])
def test_head_major_vectors(n, heads, d, rd, norm):
    """x and out as [heads, n, d] in memory, either or both."""
    g = torch.Generator().manual_seed(n)
    base = torch.randn((heads, n, d), generator=g).to(torch.bfloat16).to(DEV)
    w = torch.empty(d).uniform_(0.5, 1.5, generator=g).to(DEV) if norm else None
    b = torch.empty(d).uniform_(-1, 1, generator=g).to(DEV) if norm == "layer" else None
    table, pos = binding.rope_table(500, rd, device=DEV), torch.randint(0, 500, (n,), generator=g).to(DEV)
    x = base.transpose(0, 1)
    z, M = reference(x, norm, w, b, d, table, pos, 0, False, 1e-6)
    plain, _ = binding.norm_rope(binding.Heads(x, norm, w, b), None, table, pos)
    out = torch.full((heads, n + 2, d), 7.0, dtype=torch.bfloat16, device=DEV)
    binding.norm_rope(binding.Heads(x, norm, w, b, out=out.transpose(0, 1)), None, table, pos)
    torch.cuda.synchronize()
    check_bf16(plain, z, M)
    assert torch.equal(out[:, :n].transpose(0, 1), plain) and bool((out[:, n:] == 7).all())
    binding.norm_rope(binding.Heads(x, norm, w, b, out=x), None, table, pos)      # in place
    torch.cuda.synchronize()
    assert torch.equal(x, plain)


def test_projection_in_place():
    """Queries and keys side by side in one projection's rows, both normed and rotated where they are;
    what lies between them stays."""
    n, hq, hk, d = 517, 7, 2, 96
    g = torch.Generator().manual_seed(3)
    rows = torch.randn((n, (hq + hk + 1) * d), generator=g).to(torch.bfloat16).to(DEV)
    q, rest, k = rows.split([hq * d, d, hk * d], dim=1)
    q, k = q.unflatten(1, (hq, d)), k.unflatten(1, (hk, d))
    w = torch.empty(d).uniform_(0.5, 1.5, generator=g).to(DEV)
    table, pos = binding.rope_table(900, d, device=DEV), torch.arange(n, device=DEV)
    zq, zk = (reference(t.clone(), "rms", w, None, d, table, pos, 0, True, 1e-6) for t in (q, k))
    before = rest.clone()
    binding.norm_rope(binding.Heads(q, "rms", w, out=q), binding.Heads(k, "rms", w, out=k), table, pos,
                      interleaved=True)
    torch.cuda.synchronize()
    check_bf16(q, *zq)
    check_bf16(k, *zk)
    assert torch.equal(rest, before)


def _shifted(t, elements):
    """The same values `elements` elements into a buffer."""
    buf = torch.empty(t.numel() + 64, dtype=t.dtype, device=DEV)
    assert buf.data_ptr() % 256 == 0
    v = buf[elements:elements + t.numel()].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,T,H", [([700, 5, 0, 130], 2, 33), ([9000, 70], 1, 128)], ids=["whole", "split"])
def test_buffers_at_16_bytes(lens, T, H, fp8):
    """Queries, latent rows and outputs that start 16 bytes into an allocation: the same bits."""
    case = Case(lens, T, H, 64, fp8, seed=31, garbage=False)
    cache = case.device()
    want = binding.dense_mla_decode(case.d_q, cache, SCALE, tokens_per_seq=T)
    check(case, *want, decode_views(case))
    q = _shifted(case.d_q, 8)
    lat = _shifted(case.d_latent.view(torch.uint8), 16).view(case.d_latent.dtype)
    out = _shifted(torch.full_like(want[0], 7.0), 8)
    lse = _shifted(torch.full_like(want[1], 7.0), 1)
    moved = binding.Cache(None, lat, case.seq_lens, block_table=case.d_table, page_size=64,
                          latent_scale=cache.latent_scale)
    binding.dense_mla_decode(q, moved, SCALE, tokens_per_seq=T, out=out, lse=lse)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and binding.device_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [8, 40, 96, 200, 256])
def test_page_sizes(page, fp8):
    """The pages' order and size do not matter: the bits of a contiguous cache."""
    lens, H = [777, 64, 1, 0, 401], 24
    case = Case(lens, 1, H, page, fp8, seed=32, garbage=False)
    cache = case.device()
    flat = Case(lens, 1, H, 0, fp8, seed=0, garbage=False, s_max=case.s_max)
    pos = torch.arange(case.s_max)
    for b, n in enumerate(lens):
        at = case.phys(b, pos[:n])
        flat.latent.view(torch.uint8)[b, :n] = case.latent.view(torch.uint8).view(-1, case.latent.view(torch.uint8).shape[-1])[at]
        if fp8:
            flat.scales[b, :n] = case.scales.view(-1, 5)[at]
    flat.q = case.q
    whole = flat.device()
    for window, sink in ((None, 0), (100, 5)):
        if window is None:
            got, want = (binding.dense_mla_decode(case.d_q, c, SCALE) for c in (cache, whole))
        else:
            got, want = (binding.window_mla_decode(case.d_q, c, window, sink, SCALE) for c in (cache, whole))
        torch.cuda.synchronize()
        check(case, *got, decode_views(case, window, sink))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("fp8", [False, True])
def test_long_steps(fp8):
    """300 tokens of each sequence through the decode entry, some of them before its first position."""
    T, H = 300, 8
    case = Case([900, 300, 299, 17, 0], T, H, 16, fp8, seed=33)
    views = decode_views(case)
    cache = case.device([(b, pos) for _, b, pos in views])
    out, lse = binding.dense_mla_decode(case.d_q, cache, SCALE, tokens_per_seq=T)
    torch.cuda.synchronize()
    check(case, out, lse, views[::29] + views[600:606] + views[896:904] + views[-3:])
