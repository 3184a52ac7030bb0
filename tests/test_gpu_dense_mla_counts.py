"""Attention over the whole latent cache and over windows, with every tile of positions visible in
the results: a tile that is left out, counted twice, or weighted by another tile's logits changes
them by far more than a rounding.

Rows hold small whole numbers.  Value dims are marks: position p has ones at dim (p // 64) % 256 and
256 + (5 (p // 64) + 3) % 192 (its tile, one mark in each half of the value dims) and at 448 + p % 64
(where it is in its tile).  The scale is ln 2 and queries are zeros and ones over rope dims of both
halves and one mark dim, so that a logit is a whole number of powers of two: the weights are
2^g, exactly representable in bf16.

Tolerances.  The logits' sums are exact; times the scale in log2 units (two roundings, 2^-23) an
exponent of at most 12 is off by less than 12 * 2^-23 and a weight by 2^-20 relative (exp2 included:
2^-19).  A weight keeps its bf16 value, a power of two (half a step is 2^-9, far more than 2^-19).
A row's fp32 sum of weights has 32 terms in a tree, then at most 150 tiles in one run and 76 pieces,
each a rounding of 2^-24: below 2^-16 with the weights' own error.  The products with the values add up in at
most 4 * 150 steps of a run, each off by at most a last place (2^-23, should the tensor core cut off):
below 2^-13.  So the output is off by its own rounding, 2^-8 |out|, and 2^-13 |out|; lse by 2^-16 and
its own 2^-22 (1 + |lse|).
A tile that is lost changes the dim of its mark by at least an eighth (at most 8 tiles share a dim) and
lse by about 1 / tiles, 5e-4 at the longest."""
import math

import pytest
import torch

from indexed_sparse_attention_indexer_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = math.log(2.0)


class Marks:
    """lens, query rows, and a cache of marked rows (contiguous, or pages in any order)."""

    def __init__(self, lens, rows, H, page, fp8, seed, first_page=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.lens, self.H, self.page, self.fp8 = lens, H, page, fp8
        B, longest = len(lens), max(lens)
        if page:
            wide = (longest + page - 1) // page
            shape = (first_page + B * wide, page)
            self.table = (first_page + torch.randperm(B * wide, generator=g, device=DEV).view(B, wide)).to(torch.int32)
            self.at = self.table.long().repeat_interleave(page, dim=1) * page + torch.arange(wide * page, device=DEV) % page
        else:
            wide, shape, self.table = longest, (B, longest), None
            self.at = torch.arange(B * longest, device=DEV).view(B, longest)
        n = self.at.shape[1]
        p = torch.arange(n, device=DEV)
        # (uint8 codes: -2 .. 2 in the rope dims, marks of one)
        self.pool = torch.zeros(shape + (576,), dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEV)
        if fp8:
            self.pool = self.pool.view(torch.float8_e4m3fn)
        self.scales = None
        if fp8:                                  # code times tile scale is exact: powers of two
            self.scales = torch.ones(shape + (5,), device=DEV)
        flat = self.pool.view(torch.uint8 if fp8 else torch.bfloat16).view(-1, 576)
        for b in range(B):
            c = torch.zeros((n, 576), device=DEV)
            tile = p // 64
            c[p, tile % 256] = 1
            c[p, 256 + (5 * tile + 3) % 192] = 1
            c[p, 448 + p % 64] = 1
            c[:, 512:] = torch.randint(-2, 3, (n, 64), generator=g, device=DEV).float()
            if fp8:
                sc = torch.pow(2.0, torch.randint(-3, 4, (n, 5), generator=g, device=DEV).float())
                self.scales.view(-1, 5)[self.at[b]] = sc
                c = (c / sc.repeat_interleave(128, dim=1)[:, :576]).to(torch.float8_e4m3fn).view(torch.uint8)
            flat[self.at[b]] = c.to(flat.dtype)
        h = torch.arange(H, device=DEV)
        q = torch.zeros((rows, H, 576), device=DEV)
        for r in range(rows):
            q[r, h, (11 * h + r) % 448] = 1                  # a tile's mark
            q[r, h, 512 + (h + 3 * r) % 32] = 1              # the rope dims of either half
            q[r, h, 544 + (7 * h + r) % 32] = 1
        self.q = q.to(torch.bfloat16)
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.cache = binding.Cache(None, self.pool, self.seq_lens, block_table=self.table, page_size=page,
                                   latent_scale=self.scales)

    def rows(self, b, pos):
        c = self.pool.view(torch.uint8 if self.fp8 else torch.bfloat16).view(-1, 576)[self.at[b, pos]]
        if self.fp8:
            c = c.view(torch.float8_e4m3fn).double() * self.scales.view(-1, 5)[self.at[b, pos]].double() \
                .repeat_interleave(128, dim=1)[:, :576]
        return c.double()

    def check(self, out, lse, views):
        torch.cuda.synchronize()
        assert binding.device_status() == 0
        for r, b, pos in views:
            pos = pos.to(DEV)
            if pos.numel() == 0:
                assert bool((out[r] == 0).all()) and bool((lse[r] == -math.inf).all())
                continue
            c = self.rows(b, pos)
            w = torch.pow(2.0, self.q[r].double() @ c.T)
            total = w.sum(-1, keepdim=True)
            ref, rl = w @ c[:, :512] / total, torch.log(total[:, 0])
            err, el = (out[r].double() - ref).abs(), (lse[r].double() - rl).abs()
            assert bool((err <= (2.0 ** -8 + 2.0 ** -13) * ref).all()), (r, float((err / ref.clamp(min=1e-30)).max()))
            assert bool((el <= 2.0 ** -16 + 2.0 ** -22 * (1 + rl.abs())).all()), (r, float(el.max()))


def _spots(n, window=None, sink=0):
    lo = 0 if window is None else max(0, n - window)
    return torch.cat([torch.arange(min(sink, lo)), torch.arange(lo, n)])


def test_the_measure_sees_a_lost_tile():
    """The bounds of this file against the longest case with one of its 2000 tiles left out, counted
    twice, or weighted by its neighbour's logits: on the formulas alone."""
    m = Marks([127995], 1, 8, 64, False, 1)
    c = m.rows(0, torch.arange(127995, device=DEV))
    w = torch.pow(2.0, m.q[0].double() @ c.T)
    ref, rl = w @ c[:, :512] / w.sum(-1, keepdim=True), torch.log(w.sum(-1))
    for what in ("lost", "twice", "other"):
        for tile in (0, 1, 999, 1998):
            w2 = w.clone()
            here = slice(64 * tile, 64 * tile + 64)
            w2[:, here] = {"lost": 0 * w[:, here], "twice": 2 * w[:, here],
                           "other": w[:, 64 * tile + 64: 64 * tile + 64 + w[:, here].shape[1]]
                           if tile < 1998 else w[:, :64]}[what]
            out = w2 @ c[:, :512] / w2.sum(-1, keepdim=True)
            far = ((out - ref).abs() / ((2.0 ** -8 + 2.0 ** -13) * ref.clamp(min=1e-30))).amax(-1)    # of each head
            assert bool((far > 8).all()) if what != "other" else bool((far > 2).any()), (what, tile)
            if what != "other":
                assert bool(((torch.log(w2.sum(-1)) - rl).abs() > 4 * (2.0 ** -16 + 2.0 ** -22 * (1 + rl))).all())


DECODE = {
    # lens, T, H, page, fp8, window, sink
    "single": ([20000], 1, 128, 64, False, None, 0),
    "single_few_heads": ([20000], 1, 8, 0, False, None, 0),
    "single_fp8": ([20000], 1, 128, 64, True, None, 0),
    "ragged": ([9000, 17, 4097, 640, 0, 12345, 63, 64, 65], 1, 128, 64, False, None, 0),
    "ragged_fp8": ([9000, 17, 4097, 640, 0, 12345, 63, 64, 65], 1, 128, 24, True, None, 0),
    "few_heads_batch": ([9000 - 37 * i for i in range(40)], 1, 16, 0, False, None, 0),
    "few_heads_batch_fp8": ([9000 - 37 * i for i in range(40)], 1, 8, 16, True, None, 0),
    "three_tokens": ([5000, 2, 0, 777], 3, 128, 64, False, None, 0),
    "four_tokens_fp8": ([5000, 2, 0, 777], 4, 32, 64, True, None, 0),
    "batch": ([4000 + 64 * (i % 9) for i in range(64)], 1, 128, 0, False, None, 0),
    "batch_fp8": ([4000 + 64 * (i % 9) for i in range(64)], 1, 128, 0, True, None, 0),
    "window": ([5000 - 11 * i for i in range(90)], 1, 128, 64, False, 1024, 4),
    "window_fp8": ([5000 - 11 * i for i in range(90)], 1, 64, 64, True, 1024, 70),
    "window_tokens_fp8": ([900, 130, 2, 0], 4, 16, 16, True, 129, 3),
}


@pytest.mark.parametrize("name", sorted(DECODE))
def test_decode_counts_every_position_once(name):
    lens, T, H, page, fp8, window, sink = DECODE[name]
    m = Marks(lens, len(lens) * T, H, page, fp8, len(name))
    if window is None:
        out, lse = binding.dense_mla_decode(m.q, m.cache, SCALE, tokens_per_seq=T)
    else:
        out, lse = binding.window_mla_decode(m.q, m.cache, window, sink, SCALE, tokens_per_seq=T)
    m.check(out, lse, [(b * T + t, b, _spots(max(0, n - T + 1 + t), window, sink))
                       for b, n in enumerate(lens) for t in range(T)])


PREFILL = {
    # T, q_offset, H, page, fp8, window (None: dense causal), sink
    "causal": (1500, 0, 128, 64, False, None, 0),
    "causal_fp8": (1500, 0, 32, 24, True, None, 0),
    "causal_chunk": (600, 3333, 64, 0, False, None, 0),
    "causal_few_heads": (1111, 0, 8, 16, False, None, 0),
    "window": (1500, 700, 128, 64, False, 511, 16),
    "window_fp8": (777, 1001, 32, 0, True, 511, 70),
}


@pytest.mark.parametrize("name", sorted(PREFILL))
def test_prefill_counts_every_position_once(name):
    T, off, H, page, fp8, window, sink = PREFILL[name]
    m = Marks([off + T], T, H, page, fp8, len(name))
    out, lse = binding.window_mla_prefill(m.q, m.cache, off, window or off + T, sink, SCALE)
    rows = sorted(set(range(0, T, 37)) | {0, 1, 62, 63, 64, 65, T - 2, T - 1})
    m.check(out, lse, [(t, 0, _spots(off + t + 1, window, sink)) for t in rows])


@pytest.mark.parametrize("fp8", [False, True])
def test_long_offsets_count_every_tile(fp8):
    """128,000 positions in pages past 2^32 bytes of the pool: output and lse."""
    m = Marks([127995], 1, 128, 64, fp8, 5, first_page=118000 if fp8 else 60000)
    assert m.pool[m.table.min():].data_ptr() - m.pool.data_ptr() > 1 << 32
    out, lse = binding.dense_mla_decode(m.q, m.cache, SCALE)
    m.check(out, lse, [(0, 0, torch.arange(127995))])
    out, lse = binding.window_mla_decode(m.q, m.cache, 100001, 130, SCALE)
    m.check(out, lse, [(0, 0, _spots(127995, 100001, 130))])
