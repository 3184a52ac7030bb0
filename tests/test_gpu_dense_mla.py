"""Attention over the whole latent cache and over windows of it with sinks (dsi_dense_mla_decode,
dsi_window_mla_decode, dsi_window_mla_prefill) against the formulas in 64 bits.

Tolerances, per element, with A = sum_s p_s |v_s| / sum_s p_s (the average of magnitudes) and
L = max_s scale * sum |q||c|:
  - a logit is an fp32 sum of 576 products, in pieces: off by less than 576 * 2^-23 L < 2^-13 L in
    natural units, so a weight by less than a factor 1 + 2^-12 L (with the fp32 maximum, exp2 and
    sum: 2^-20), and the output by 2 * 2^-12 L A;
  - weights are rounded to bf16 before they multiply the values (half a step, 2^-8 relative), the
    same rounded weights are summed for the denominator: 2^-8 (A + |out|);
  - the output is rounded to bf16: 2^-8 |out|.
lse sums the unrounded weights: off by 2^-12 L + 2^-20 (1 + |lse|).
"""
import math

import pytest
import torch

from indexed_sparse_attention_indexer_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 1.0 / math.sqrt(576)


class Case:
    """A cache (contiguous or paged, bf16 or FP8) whose rows outside the visible range hold NaN."""

    def __init__(self, lens, T, H, page=0, fp8=False, seed=0, s_max=None, q_std=1.5, garbage=True):
        g = torch.Generator().manual_seed(seed)
        B = len(lens)
        self.lens, self.T, self.H, self.page, self.fp8 = list(lens), T, H, page, fp8
        longest = max(max(lens), 1)
        self.s_max = s_max or longest
        if page:
            wide = max(1, (self.s_max + page - 1) // page)
            need = [(min(max(n, 0), wide * page) + page - 1) // page for n in lens]
            shape = (sum(need) + 2, page)
            ids = torch.randperm(shape[0], generator=g).to(torch.int32)
            table = torch.full((B, wide), -7, dtype=torch.int32)
            at = 0
            for b, k in enumerate(need):
                table[b, :k] = ids[at:at + k]
                at += k
            self.table = table
            self.s_max = wide * page
        else:
            shape, self.table = (B, self.s_max), None
        x = torch.randn(shape + (576,), generator=g).to(torch.bfloat16)
        self.scales = None
        if fp8:
            self.scales = torch.empty(shape + (5,)).uniform_(1 / 128, 1 / 32, generator=g)
            x = (x.float() * 64).clamp(-448, 448).to(torch.float8_e4m3fn)
        self.q = (torch.randn((B * T, H, 576), generator=g) * q_std).to(torch.bfloat16)
        self.latent = x
        self.garbage = garbage

    def phys(self, b, pos):
        if self.table is None:
            return b * self.s_max + pos
        return self.table[b].long()[pos // self.page] * self.page + pos % self.page

    def rows(self, b, pos):
        c = self.latent.view(torch.uint8 if self.fp8 else torch.bfloat16).view(-1, 576)[self.phys(b, pos)]
        if self.fp8:
            sc = self.scales.view(-1, 5)[self.phys(b, pos)].repeat_interleave(128, dim=-1)[:, :576]
            c = (c.view(torch.float8_e4m3fn).float() * sc).to(torch.bfloat16)
        return c.double()

    def device(self, keep=None):
        """Device tensors; rows that no query sees (keep: [(b, positions)]) become NaN."""
        lat = self.latent.clone()
        if self.garbage and keep is not None:
            seen = torch.zeros(lat.view(torch.uint8).view(-1, 576 * (1 if self.fp8 else 2)).shape[0], dtype=torch.bool)
            for b, pos in keep:
                seen[self.phys(b, pos)] = True
            raw = lat.view(torch.uint8).view(seen.numel(), -1)
            raw[~seen] = 0x7F if self.fp8 else 0xFF          # NaN in both formats
        sc = None
        if self.fp8:
            sc = self.scales.clone()
            if self.garbage and keep is not None:
                sc.view(-1, 5)[~seen] = math.inf
            sc = sc.to(DEV)
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device=DEV)
        self.d_latent = lat.view(torch.uint8).to(DEV).view(lat.dtype)
        self.d_table = self.table.to(DEV) if self.table is not None else None
        self.d_q = self.q.to(DEV)
        return binding.Cache(None, self.d_latent, self.seq_lens, block_table=self.d_table,
                             page_size=self.page, latent_scale=sc)


def spots(n, window, sink):
    lo = max(0, n - window)
    return torch.cat([torch.arange(min(sink, lo)), torch.arange(lo, n)])


def reference(case, r, b, pos, scale):
    """(out [H, 512], tol, lse [H], lse tol) of query row r over positions pos of sequence b."""
    H = case.H
    if pos.numel() == 0:
        z = torch.zeros((H, 512), dtype=torch.float64)
        return z, z, torch.full((H,), -math.inf, dtype=torch.float64), torch.zeros(H, dtype=torch.float64)
    c, q = case.rows(b, pos).to(DEV), case.q[r].double().to(DEV)
    l = q @ c.T * scale
    L = (q.abs() @ c.abs().T * abs(scale)).amax(-1)
    lse = torch.logsumexp(l, dim=-1)
    p = torch.exp(l - lse[:, None])
    v = c[:, :512]
    out, A = p @ v, p @ v.abs()
    tol = 2.0 ** -8 * (A + 2 * out.abs()) + 2.0 ** -11 * L[:, None] * A
    return out.cpu(), tol.cpu(), lse.cpu(), (2.0 ** -12 * L + 2.0 ** -20 * (1 + lse.abs())).cpu()


def check(case, out, lse, views, scale=SCALE):
    """views: (row, sequence, positions) of every query row that is compared."""
    assert binding.device_status() == 0
    worst = 0.0
    for r, b, pos in views:
        ref, tol, rl, tl = reference(case, r, b, pos, scale)
        got = out[r].double().cpu()
        if pos.numel() == 0:
            assert bool((got == 0).all()) and (lse is None or bool((lse[r].cpu() == -math.inf).all()))
            continue
        err = (got - ref).abs()
        assert bool((err <= tol).all()), f"row {r}: {float((err / tol).max())} of the tolerance"
        worst = max(worst, float((err / tol).max()))
        if lse is not None:
            el = (lse[r].double().cpu() - rl).abs()
            assert bool((el <= tl).all()), f"row {r} lse: {float(el.max())}"
    return worst


def decode_views(case, window=None, sink=0):
    v = []
    for b, n in enumerate(case.lens):
        for t in range(case.T):
            k = min(max(0, n - (case.T - 1 - t)), case.s_max)
            v.append((b * case.T + t, b, spots(k, window if window is not None else k + 1, sink)))
    return v


def run_decode(case, window=None, sink=0, scale=SCALE, views=None, **kw):
    views = views or decode_views(case, window, sink)
    cache = case.device([(b, pos) for _, b, pos in views])
    if window is None:
        out, lse = binding.dense_mla_decode(case.d_q, cache, scale, tokens_per_seq=case.T, **kw)
    else:
        out, lse = binding.window_mla_decode(case.d_q, cache, window, sink, scale,
                                             tokens_per_seq=case.T, **kw)
    torch.cuda.synchronize()
    check(case, out, lse, views, scale)
    return out, lse


DENSE = {
    # lens, T, H, page, fp8
    "one_token": ([1], 1, 1, 0, False),
    "tile_edges": ([63, 64, 65, 127, 128, 129], 1, 128, 0, False),
    "empty_and_short": ([0, 5, 0, 1, 300], 1, 128, 64, False),
    "heads_16": ([2048], 1, 16, 0, False),
    "heads_17": ([700, 33], 1, 17, 16, False),
    "heads_100_page24": ([500, 129, 24, 25], 1, 100, 24, False),
    "heads_3_page8": ([77, 8, 9, 1000], 1, 3, 8, False),
    "page_128": ([1000, 128, 300], 1, 128, 128, False),
    "two_tokens": ([500, 1, 2, 64], 2, 64, 0, False),
    "four_tokens_128": ([300, 3, 0, 67], 4, 128, 64, False),
    "five_tokens_30": ([300, 4, 61], 5, 30, 16, False),
    "nine_tokens_16": ([130, 8], 9, 16, 0, False),
    "long_single": ([20000], 1, 128, 64, False),
    "long_ragged": ([9000, 17, 4097, 640, 0, 12345], 1, 128, 64, False),
    "fp8": ([300, 64, 1, 0, 900], 1, 128, 64, True),
    "fp8_heads_20": ([513, 70], 3, 20, 0, True),
    "fp8_long": ([8000, 100], 1, 64, 24, True),
    "many_short": ([i % 7 for i in range(300)], 1, 8, 8, False),
    "many_mid": ([64 * (i % 5) + i % 3 for i in range(200)], 1, 128, 64, False),
}


@pytest.mark.parametrize("name", sorted(DENSE))
def test_dense_decode(name):
    lens, T, H, page, fp8 = DENSE[name]
    case = Case(lens, T, H, page, fp8, seed=len(name))
    a = run_decode(case)
    b = run_decode(case)                             # the same from one call to the next
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("name", ["tile_edges", "four_tokens_128", "long_ragged", "fp8", "many_mid"])
def test_dense_decode_without_workspace(name):
    """The C entry without a workspace: no split."""
    lens, T, H, page, fp8 = DENSE[name]
    case = Case(lens, T, H, page, fp8, seed=3)
    views = decode_views(case)
    cache = case.device([(b, pos) for _, b, pos in views])
    out = torch.empty((len(lens) * T, H, 512), dtype=torch.bfloat16, device=DEV)
    lib = binding.load()
    st = lib.dsi_dense_mla_decode(binding._ptr(case.d_q), cache.ref(), T, H, SCALE, binding._ptr(out), None,
                                  None, 0, binding._stream(None))
    assert st == 0
    torch.cuda.synchronize()
    check(case, out, None, views)


WINDOW = {
    # lens, T, H, page, fp8, window, sink
    "w1": ([1, 5, 64, 65, 200], 1, 128, 0, False, 1, 0),
    "w64_s1": ([1, 64, 65, 66, 128, 129, 500], 1, 128, 64, False, 64, 1),
    "w63_s4": ([1000, 63, 67, 68], 1, 128, 64, False, 63, 4),
    "w100_s64": ([1000, 164, 165, 163, 100], 1, 16, 16, False, 100, 64),
    "w100_s70": ([1000, 170, 171, 10], 1, 64, 0, False, 100, 70),
    "w1024_s4": ([5000, 1028, 1024, 3], 1, 128, 64, False, 1024, 4),
    "sinks_past_history": ([50, 500], 1, 32, 8, False, 7, 5000),
    "w_past_history": ([50, 500], 1, 32, 8, False, 1 << 40, 1 << 41),
    "four_tokens": ([700, 130, 2, 0], 4, 16, 24, False, 65, 3),
    "three_tokens_128": ([700, 130, 2, 0], 3, 128, 64, False, 129, 3),
    "fp8": ([700, 130, 2, 0], 2, 64, 64, True, 129, 3),
    "many": ([31 * i % 900 for i in range(170)], 1, 128, 64, False, 200, 4),
}


@pytest.mark.parametrize("name", sorted(WINDOW))
def test_window_decode(name):
    lens, T, H, page, fp8, window, sink = WINDOW[name]
    case = Case(lens, T, H, page, fp8, seed=len(name))
    a = run_decode(case, window, sink)
    b = run_decode(case, window, sink)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


PREFILL = {
    # T, q_offset, extra rows, H, page, fp8, window, sink
    "first_token": (1, 0, 5, 128, 0, False, 10, 0),
    "from_zero": (200, 0, 0, 128, 64, False, 64, 4),
    "chunk": (130, 1000, 100, 128, 64, False, 257, 16),
    "heads_16": (77, 300, 3, 16, 16, False, 33, 70),
    "heads_5": (61, 64, 0, 5, 8, False, 1, 1),
    "dense_causal": (150, 10, 0, 32, 0, False, 160, 0),
    "fp8": (70, 129, 60, 64, 24, True, 100, 2),
    "many_groups": (700, 0, 0, 64, 64, False, 40, 0),
}


@pytest.mark.parametrize("name", sorted(PREFILL))
def test_window_prefill(name):
    T, off, extra, H, page, fp8, window, sink = PREFILL[name]
    case = Case([off + T], T, H, page, fp8, seed=len(name), s_max=off + T + extra)
    views = [(t, 0, spots(off + t + 1, window, sink)) for t in range(T)]
    cache = case.device([(0, pos) for _, _, pos in views])
    runs = []
    for _ in range(2):
        runs.append(binding.window_mla_prefill(case.d_q, cache, off, window, sink, SCALE))
        torch.cuda.synchronize()
    check(case, *runs[0], views[:: max(1, T // 60)] + views[-3:])
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])


def test_decode_equals_prefill_rows():
    """The same rows through the decode and the prefill entry, and packed with others or not."""
    case = Case([333], 4, 32, 64, seed=8)
    cache = case.device()
    a, la = binding.window_mla_decode(case.d_q, cache, 100, 3, SCALE, tokens_per_seq=4)
    b, lb = binding.window_mla_prefill(case.d_q, cache, 329, 100, 3, SCALE)
    torch.cuda.synchronize()
    views = decode_views(case, 100, 3)
    check(case, a, la, views)
    check(case, b, lb, views)


def test_clamped_and_negative_lengths():
    """A length above the cache's rows counts as all of them, a negative one as none."""
    case = Case([500, -3, 90], 2, 16, seed=5, s_max=96)
    run_decode(case)
    case = Case([500, -3, 90], 1, 128, 16, seed=5, s_max=96)
    run_decode(case, 50, 2)


@pytest.mark.parametrize("scale,q_std", [(0.0, 1.0), (-SCALE, 1.5), (SCALE, 30.0), (1e-30, 1.0)])
def test_scales(scale, q_std):
    """No, negative, tiny and very peaked logits (the running maximum moves far and often)."""
    case = Case([900, 65], 1, 128, 64, seed=6, q_std=q_std)
    run_decode(case, scale=scale)


def test_rising_logits():
    """Every tile holds larger logits than the ones before: the accumulator is rescaled each time."""
    case = Case([2000], 1, 128, 0, seed=7)
    ramp = torch.linspace(0.01, 3.0, 2000)[:, None]
    base = torch.randn((1, 576), generator=torch.Generator().manual_seed(1))
    case.latent = (base * ramp + 0.05 * case.latent.float()[0]).to(torch.bfloat16)[None]
    case.q = (base * 2 + 0.1 * case.q.float()).to(torch.bfloat16)
    run_decode(case)
    case.q = -case.q
    run_decode(case)


def test_non_finite_rows():
    """A NaN row that only the later tokens of a step see makes their outputs NaN and leaves the
    earlier tokens alone; a row that every token sees reaches every token; other sequences and
    rows behind them are untouched."""
    for bad in (math.nan, math.inf):
        case = Case([200, 200], 4, 16, seed=11, garbage=False)
        views = decode_views(case)
        case.latent[0, 198, 5] = bad              # position 198: seen by tokens 2 and 3
        cache = case.device()
        out, lse = binding.dense_mla_decode(case.d_q, cache, SCALE, tokens_per_seq=4)
        torch.cuda.synchronize()
        check(case, out, lse, [v for v in views if v[0] not in (2, 3)])
        assert bool(torch.isnan(out[2:4]).any(-1).all())
        assert not bool(torch.isfinite(lse[2:4].sum(-1)).any()) or bad == math.inf
        case = Case([200], 1, 16, seed=12, garbage=False)
        case.latent[0, 70, 500] = bad
        out, _ = binding.dense_mla_decode(case.d_q if hasattr(case, "d_q") else case.q.to(DEV), case.device(), SCALE)
        torch.cuda.synchronize()
        assert bool(torch.isnan(out).any(-1).all())


def test_bad_pages_are_reported():
    """A page id outside the pool under a visible position: reported, read as zeros; the other
    sequences' results do not change."""
    for T, H, fp8 in ((1, 128, False), (2, 16, False), (1, 32, True)):
        case = Case([300, 300, 300], T, H, 16, fp8, seed=13, garbage=False)
        cache = case.device()
        good = binding.dense_mla_decode(case.d_q, cache, SCALE, tokens_per_seq=T)[0].clone()
        assert binding.device_status() == 0
        for page in (-1, 1 << 30, -(1 << 31)):
            case.d_table[1, 3] = page
            case.d_table[1, 18] = page             # the last page: inside a partial tile
            out, _ = binding.dense_mla_decode(case.d_q, cache, SCALE, tokens_per_seq=T)
            torch.cuda.synchronize()
            assert binding.device_status() == binding.DSI_ERR_BOUNDS
            assert torch.equal(out[:T], good[:T]) and torch.equal(out[2 * T:], good[2 * T:])
            assert bool(torch.isfinite(out.float()).all())


def test_outputs_are_only_written_where_they_belong():
    case = Case([100, 0, 50], 1, 5, 8, seed=14)
    cache = case.device([(b, pos) for _, b, pos in decode_views(case)])
    big = torch.full((5, 5, 512), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((5, 5), 7.0, device=DEV)
    binding.dense_mla_decode(case.d_q, cache, SCALE, out=big[1:4], lse=lse[1:4])
    torch.cuda.synchronize()
    check(case, big[1:4], lse[1:4], decode_views(case))
    assert bool((big[0] == 7).all()) and bool((big[4] == 7).all()) and bool((lse[0] == 7).all()) and bool((lse[4] == 7).all())


def test_graphs_and_streams():
    """Two captured steps with a workspace each replayed at once on two streams, with new lengths
    and queries, against direct calls."""
    cases = [Case([3000, 40, 900], 1, 128, 64, seed=20, garbage=False),
             Case([5000], 2, 16, 16, seed=21, garbage=False)]
    caches = [c.device() for c in cases]
    graphs, outs = [], []
    for c, cache in zip(cases, caches):
        wsp = binding.alloc_workspace(binding.dense_mla_workspace_size(c.q.shape[0], c.H), DEV)
        out = torch.empty((c.q.shape[0], c.H, 512), dtype=torch.bfloat16, device=DEV)
        lse = torch.empty((c.q.shape[0], c.H), device=DEV)
        call = lambda: binding.dense_mla_decode(c.d_q, cache, SCALE, tokens_per_seq=c.T, out=out,
                                                lse=lse, workspace=wsp)
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append(graph)
        outs.append((out, lse, wsp))
    cases[0].lens = [1500, 0, 897]
    cases[0].seq_lens.copy_(torch.tensor(cases[0].lens, dtype=torch.int32))
    for c in cases:
        c.q = c.q.flip(0)
        c.d_q.copy_(c.q.to(DEV))
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for c, (out, lse, _) in zip(cases, outs):
        check(c, out, lse, decode_views(c))
    # direct, on a stream that is not the current one; buffers of the call's own
    c = cases[1]
    streams[0].wait_stream(torch.cuda.current_stream())
    out, lse = binding.dense_mla_decode(c.d_q, caches[1], SCALE, tokens_per_seq=2, stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(out, outs[1][0])


def test_long_offsets():
    """A pool whose rows lie past 2^32 bytes, and positions past 2^16 in one sequence."""
    pages, page = 66000, 64                       # 4.9 GB of latent rows
    pool = torch.zeros((pages, page, 576), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(2)
    table = torch.arange(pages - 1, pages - 2001, -1, dtype=torch.int32, device=DEV)[None].contiguous()
    pool[-2000:] = torch.randn((2000, page, 576), generator=g, device=DEV).to(torch.bfloat16)
    lens = torch.tensor([2000 * page - 5], dtype=torch.int32, device=DEV)
    q = torch.randn((1, 128, 576), generator=g, device=DEV).to(torch.bfloat16)
    cache = binding.Cache(None, pool, lens, block_table=table, page_size=page)
    out, lse = binding.dense_mla_decode(q, cache, SCALE)
    torch.cuda.synchronize()
    c = pool[-2000:].flip(0).reshape(-1, 576)[:2000 * page - 5].double()
    l = q[0].double() @ c.T * SCALE
    ref = torch.softmax(l, dim=-1) @ c[:, :512]
    # averages of 1.3e5 nearly independent values: 2^-8 of the average magnitude and of the result
    A = torch.softmax(l, dim=-1) @ c[:, :512].abs()
    L = (q[0].double().abs() @ c.abs().T * SCALE).amax(-1)[:, None]
    assert bool(((out[0].double() - ref).abs() <= 2.0 ** -8 * (A + 2 * ref.abs()) + 2.0 ** -11 * L * A).all())
    assert binding.device_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens", [[70, 300], [9000, 70]], ids=["whole", "split"])
def test_non_finite_queries(lens, fp8):
    """A head whose query holds NaN gets NaN outputs and a NaN lse, the others what they get without."""
    case = Case(lens, 1, 32, 64, fp8, seed=15, garbage=False)
    cache = case.device()
    good, good_lse = (t.clone() for t in binding.dense_mla_decode(case.d_q, cache, SCALE))
    case.d_q[0, 5, 7] = math.nan
    case.d_q[1, 31, 570] = math.nan
    out, lse = binding.dense_mla_decode(case.d_q, cache, SCALE)
    torch.cuda.synchronize()
    bad = torch.zeros((2, 32), dtype=torch.bool, device=DEV)
    bad[0, 5] = bad[1, 31] = True
    assert bool(torch.isnan(out[bad]).all()) and bool(torch.isnan(lse[bad]).all())
    assert torch.equal(out[~bad], good[~bad]) and torch.equal(lse[~bad], good_lse[~bad])


@pytest.mark.parametrize("where", ["latent", "rope", "scale"])
def test_non_finite_fp8_rows(where):
    """A row that only the later tokens of a step see, with a NaN code or an infinite scale."""
    case = Case([200, 200], 4, 16, 16, True, seed=16, garbage=False)
    views = decode_views(case)
    at = int(case.phys(0, torch.tensor([198])))
    case.latent.view(torch.uint8).view(-1, 576)[at, :] = 0x31             # (no zero codes: inf * 0 is NaN)
    if where == "scale":
        case.scales.view(-1, 5)[at, 1] = math.inf
    else:
        case.latent.view(torch.uint8).view(-1, 576)[at, 300 if where == "latent" else 560] = 0xFF
    cache = case.device()
    out, lse = binding.dense_mla_decode(case.d_q, cache, SCALE, tokens_per_seq=4)
    torch.cuda.synchronize()
    check(case, out, lse, [v for v in views if v[0] not in (2, 3)])
    assert bool(torch.isnan(out[2:4]).any(-1).all())


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("name", ["one_tile", "two_tiles", "window_two_tiles", "window_three_tiles", "mixed"])
def test_many_short_groups(name, fp8):
    """Many groups of one to three tiles for every pair of SMs: query slices and tiles take turns
    in the ring, and every one of its slots has to be seen by all who wait for it."""
    T, H, page, window, sink, lens = {
        "one_tile": (1, 128, 0, None, 0, [1 + 7 * i % 64 for i in range(700)]),
        "two_tiles": (1, 128, 16, None, 0, [65 + 11 * i % 64 for i in range(700)]),
        "window_two_tiles": (850, 64, 16, 40, 0, [1000]),
        "window_three_tiles": (850, 64, 16, 59, 4, [2855]),
        "mixed": (1, 128, 64, None, 0, [(1, 70, 130, 0, 64, 200, 65)[i % 7] for i in range(700)]),
    }[name]
    case = Case(lens, T, H, page, fp8, seed=17)
    if T == 1:
        views = decode_views(case)
    else:
        views = [(t, 0, spots(lens[0] - T + t + 1, window, sink)) for t in range(T)]
    cache = case.device([(b, pos) for _, b, pos in views])
    runs = []
    for _ in range(20):
        if T == 1:
            runs.append(binding.dense_mla_decode(case.d_q, cache, SCALE))
        else:
            runs.append(binding.window_mla_prefill(case.d_q, cache, lens[0] - T, window, sink, SCALE))
    torch.cuda.synchronize()
    check(case, *runs[0], views[::13] + views[-5:])
    for out, lse in runs[1:]:
        assert torch.equal(out, runs[0][0]) and torch.equal(lse, runs[0][1])
