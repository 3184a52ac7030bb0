"""Attention over a prefix that the batch shares and over the sequences' own rows
(dsi_prefix_mla_decode) against the formula in 64 bits, with the tolerances of
test_gpu_dense_mla (the two parts' fp32 sums are joined in fp32: no further rounding to bf16)."""
import math

import pytest
import torch

from indexed_sparse_attention_indexer_gb300 import binding
from tests.test_gpu_dense_mla import DEV, SCALE, Case

pytestmark = pytest.mark.gpu


class Shared:
    """A prefix and a batch's own rows; what nobody sees is NaN."""

    def __init__(self, prefix, lens, T, H, page=0, fp8=False, seed=0, prefix_page=None, q_std=1.5, garbage=True,
                 prefix_max=None, s_max=None):
        self.P, self.T, self.H, self.fp8 = prefix, T, H, fp8
        self.first = Case([prefix], 1, H, page if prefix_page is None else prefix_page, fp8, seed=seed + 1000,
                          s_max=prefix_max, garbage=garbage)
        self.own = Case(lens, T, H, page, fp8, seed=seed, s_max=s_max, q_std=q_std, garbage=garbage)
        self.lens, self.q = self.own.lens, self.own.q

    def seen(self, r):
        b, t = divmod(r, self.T)
        n = min(max(0, self.lens[b] - (self.T - 1 - t)), self.own.s_max)     # as for the dense call
        return b, min(max(0, self.P), self.first.s_max), n

    def device(self):
        R = len(self.lens) * self.T
        self.prefix = self.first.device([(0, torch.arange(self.seen(0)[1] if R else 0))])
        keep = [(b, torch.arange(n)) for b, _, n in map(self.seen, range(R))]
        self.cache = self.own.device(keep)
        self.d_q = self.own.d_q
        return self

    def run(self, scale=SCALE, **kw):
        return binding.prefix_mla_decode(self.d_q, self.prefix, self.cache, scale, tokens_per_seq=self.T, **kw)

    def reference(self, r, scale=SCALE):
        b, p, n = self.seen(r)
        c = torch.cat([self.first.rows(0, torch.arange(p)), self.own.rows(b, torch.arange(n))]).to(DEV)
        q = self.q[r].double().to(DEV)
        l = q @ c.T * scale
        L = (q.abs() @ c.abs().T * abs(scale)).amax(-1)
        lse = torch.logsumexp(l, dim=-1)
        w, v = torch.exp(l - lse[:, None]), c[:, :512]
        out, A = w @ v, w @ v.abs()
        return (out, 2.0 ** -8 * (A + 2 * out.abs()) + 2.0 ** -11 * L[:, None] * A, lse,
                2.0 ** -12 * L + 2.0 ** -20 * (1 + lse.abs()))

    def check(self, out, lse, rows=None, scale=SCALE):
        assert binding.device_status() == 0
        for r in range(len(self.lens) * self.T) if rows is None else rows:
            _, p, n = self.seen(r)
            if p + n == 0:
                assert bool((out[r] == 0).all()) and (lse is None or bool((lse[r] == -math.inf).all()))
                continue
            ref, tol, rl, tl = self.reference(r, scale)
            err = (out[r].double() - ref).abs()
            assert bool((err <= tol).all()), f"row {r}: {float((err / tol).max())} of the tolerance"
            if lse is not None:
                assert bool(((lse[r].double() - rl).abs() <= tl).all()), f"row {r} lse"


CASES = {
    # prefix, lens, T, H, page, fp8, prefix page
    "one_row": (1, [1], 1, 1, 0, False, None),
    "nothing_at_all": (0, [0, 3, 0], 1, 16, 0, False, None),
    "prefix_alone": (100, [0, 0], 1, 128, 0, False, None),
    "no_prefix": (0, [70, 5, 300], 1, 16, 64, False, None),
    "tile_edges_128": (128, [63, 64, 65, 1], 1, 128, 0, False, None),
    "tile_edges_63": (63, [63, 64, 65, 1, 0], 1, 32, 64, False, None),
    "tile_edges_65": (65, [128, 129, 127], 1, 32, 16, False, None),
    "heads_16_long": (5000, [40, 1, 777, 300, 0, 64, 65, 2, 9], 1, 16, 64, False, None),
    "heads_16_many": (2000, [i % 130 for i in range(70)], 1, 16, 0, False, None),
    "heads_17": (500, [33, 70, 2, 600], 1, 17, 16, False, None),
    "heads_100": (300, [33, 0, 2], 1, 100, 24, False, None),
    "heads_3_many": (700, [i % 9 for i in range(90)], 1, 3, 8, False, None),
    "heads_1": (900, [5] * 200, 1, 1, 0, False, None),
    "own_longer": (64, [3000, 9, 1500], 1, 64, 64, False, None),
    "two_tokens": (600, [500, 1, 2, 64, 0], 2, 64, 0, False, None),
    "four_tokens_128": (300, [300, 3, 0, 67], 4, 128, 64, False, None),
    "five_tokens_30": (411, [300, 4, 61], 5, 30, 16, False, None),
    "three_tokens_50": (1000, [2, 90, 0, 400, 17], 3, 50, 64, False, None),
    "nine_tokens_16": (130, [130, 8], 9, 16, 0, False, None),
    "batch_128_heads": (3000, [200, 0, 64, 129, 1000, 5, 77], 1, 128, 64, False, None),
    "other_pages": (1000, [200, 30, 64], 1, 32, 16, False, 128),
    "prefix_contiguous": (777, [200, 30, 64], 1, 32, 16, False, 0),
    "prefix_paged": (777, [200, 30, 64], 1, 32, 0, False, 64),
    "one_sequence": (9000, [100], 1, 16, 64, False, None),
    "fp8": (500, [300, 64, 1, 0, 900], 1, 128, 64, True, None),
    "fp8_heads_16": (3000, [100, 64, 1, 0, 300] * 5, 1, 16, 64, True, None),
    "fp8_tokens": (513, [70, 300, 2], 3, 20, 0, True, 24),
    # (long enough for the prefix to be converted once)
    "fp8_converted": (4005, [37 * i % 200 for i in range(20)], 1, 128, 64, True, None),
    "fp8_converted_tokens": (4700, [53 * i % 90 for i in range(18)], 2, 64, 24, True, 0),
    "fp8_converted_heads_20": (6001, [0, 1, 2] * 26, 1, 20, 0, True, 16),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_prefix_decode(name):
    prefix, lens, T, H, page, fp8, pp = CASES[name]
    case = Shared(prefix, lens, T, H, page, fp8, seed=len(name), prefix_page=pp).device()
    a = case.run()
    b = case.run()
    torch.cuda.synchronize()
    case.check(*a)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_same_as_dense_on_shared_pages():
    """dsi_dense_mla_decode over block tables that begin with the prefix's pages sees the same rows."""
    H, page, P = 16, 16, 640                         # whole pages of prefix
    case = Shared(P, [100, 3, 64, 700], 1, H, page, seed=4).device()
    out, lse = case.run()
    wide = P // page + case.own.table.shape[1]
    pool = torch.cat([case.first.d_latent, case.own.d_latent])
    table = torch.cat([case.first.d_table[:, :P // page].expand(4, -1),
                       torch.where(case.own.d_table >= 0, case.own.d_table + case.first.d_latent.shape[0],
                                   case.own.d_table)], dim=1).contiguous()
    assert table.shape[1] == wide
    cache = binding.Cache(None, pool, case.own.seq_lens + P, block_table=table, page_size=page)
    d_out, d_lse = binding.dense_mla_decode(case.d_q, cache, SCALE)
    torch.cuda.synchronize()
    case.check(out, lse)
    case.check(d_out, d_lse)


def test_pages_of_one_pool():
    """Prefix and sequences on pages of one pool, as forks of one request leave them."""
    g = torch.Generator().manual_seed(3)
    page, P, lens, H = 64, 700, [90, 0, 130], 16
    pool = torch.randn((20, page, 576), generator=g).to(torch.bfloat16)
    ids = torch.randperm(20, generator=g).to(torch.int32)
    ptab, otab = ids[None, :11].contiguous(), torch.stack([ids[11:14], ids[14:17], ids[17:20]])
    q = torch.randn((3, H, 576), generator=g).to(torch.bfloat16)
    d = pool.to(DEV)
    prefix = binding.Cache(None, d, torch.tensor([P], dtype=torch.int32, device=DEV), block_table=ptab.to(DEV), page_size=page)
    cache = binding.Cache(None, d, torch.tensor(lens, dtype=torch.int32, device=DEV), block_table=otab.to(DEV), page_size=page)
    out, lse = binding.prefix_mla_decode(q.to(DEV), prefix, cache, SCALE)
    torch.cuda.synchronize()
    rows = lambda t, n: pool[t.long()].reshape(-1, 576)[:n].double()              # noqa: E731
    for b, n in enumerate(lens):
        c = torch.cat([rows(ptab[0], P), rows(otab[b], n)])
        l = q[b].double() @ c.T * SCALE
        w = torch.softmax(l, -1)
        A = w @ c[:, :512].abs()
        L = (q[b].double().abs() @ c.abs().T * SCALE).amax(-1)
        ref = w @ c[:, :512]
        tol = 2.0 ** -8 * (A + 2 * ref.abs()) + 2.0 ** -11 * L[:, None] * A
        assert bool(((out[b].double().cpu() - ref).abs() <= tol).all())
        assert bool(((lse[b].double().cpu() - torch.logsumexp(l, -1)).abs() <= 2.0 ** -12 * L + 2.0 ** -18).all())


def test_clamped_and_negative_lengths():
    case = Shared(5000, [500, -3, 90], 2, 16, seed=5, s_max=96, prefix_max=320).device()
    case.check(*case.run())
    case = Shared(-7, [500, -3, 90], 1, 128, 16, seed=5, s_max=96, prefix_max=320).device()
    case.check(*case.run())


@pytest.mark.parametrize("scale,q_std", [(0.0, 1.0), (-SCALE, 1.5), (SCALE, 30.0), (1e-30, 1.0)])
def test_scales(scale, q_std):
    case = Shared(900, [65, 200, 0], 1, 32, 64, seed=6, q_std=q_std).device()
    case.check(*case.run(scale), scale=scale)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_non_finite_rows(bad):
    """A row of the prefix reaches every token; an own row the sequence's tokens that see it."""
    case = Shared(300, [200, 200], 4, 16, seed=11, garbage=False)
    case.own.latent[0, 198, 5] = bad                  # seen by tokens 2 and 3 of sequence 0
    out, lse = case.device().run()
    torch.cuda.synchronize()
    case.check(out, lse, [0, 1, 4, 5, 6, 7])
    assert bool(torch.isnan(out[2:4]).any(-1).all())
    case = Shared(300, [200, 0], 1, 16, seed=12, garbage=False)
    case.first.latent[0, 70, 500] = bad
    out, _ = case.device().run()
    torch.cuda.synchronize()
    assert bool(torch.isnan(out).any(-1).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_non_finite_queries(fp8):
    """A head whose query holds NaN has NaN outputs; the others, in its tile too, what they get without."""
    case = Shared(900, [70, 300, 0, 5, 64, 700, 1, 2], 1, 16, 64, fp8, seed=15, garbage=False).device()
    good, good_lse = (t.clone() for t in case.run())
    case.d_q[0, 5, 7] = math.nan
    case.d_q[5, 15, 570] = math.nan
    out, lse = case.run()
    torch.cuda.synchronize()
    hit = torch.zeros((8, 16), dtype=torch.bool, device=DEV)
    hit[0, 5] = hit[5, 15] = True
    assert bool(torch.isnan(out[hit]).all()) and bool(torch.isnan(lse[hit]).all())
    assert torch.equal(out[~hit], good[~hit]) and torch.equal(lse[~hit], good_lse[~hit])


def test_bad_pages_are_reported():
    for fp8 in (False, True):
        case = Shared(300, [300, 300, 300], 1, 16, 16, fp8, seed=13, garbage=False).device()
        good = case.run()[0].clone()
        assert binding.device_status() == 0
        keep = case.own.d_table.clone()
        for page in (-1, 1 << 30, -(1 << 31)):
            case.own.d_table[1, 3] = page
            case.own.d_table[1, 18] = page
            out, _ = case.run()
            torch.cuda.synchronize()
            assert binding.device_status() == binding.DSI_ERR_BOUNDS
            assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2]) and bool(out.isfinite().all())
            case.own.d_table.copy_(keep)
            kept = int(case.first.d_table[0, 7])
            case.first.d_table[0, 7] = page
            out, _ = case.run()
            torch.cuda.synchronize()
            assert binding.device_status() == binding.DSI_ERR_BOUNDS and bool(out.isfinite().all())
            case.first.d_table[0, 7] = kept
        out, _ = case.run()
        torch.cuda.synchronize()
        assert binding.device_status() == 0 and torch.equal(out, good)


def test_outputs_are_only_written_where_they_belong():
    case = Shared(200, [100, 0, 50], 1, 5, 8, seed=14).device()
    big = torch.full((5, 5, 512), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((5, 5), 7.0, device=DEV)
    case.run(out=big[1:4], lse=lse[1:4])
    torch.cuda.synchronize()
    case.check(big[1:4], lse[1:4])
    assert bool((big[[0, 4]] == 7).all()) and bool((lse[[0, 4]] == 7).all())
    out, none = case.run(want_lse=False)
    assert none is None and torch.equal(out, big[1:4])


def test_graphs_and_streams():
    """Captured steps with a workspace each, replayed at once on two streams with new lengths and
    queries; the workspace holds anything at first."""
    cases = [Shared(3000, [300, 40, 90], 1, 128, 64, seed=20, garbage=False).device(),
             Shared(2000, [50, 64, 7, 900], 2, 16, 16, seed=21, garbage=False).device()]
    graphs, outs = [], []
    for c in cases:
        R = c.q.shape[0]
        wsp = binding.alloc_workspace(binding.prefix_mla_workspace_size(R, c.H), DEV).fill_(0xFF)
        out = torch.empty((R, c.H, 512), dtype=torch.bfloat16, device=DEV)
        lse = torch.empty((R, c.H), device=DEV)
        c.run(out=out, lse=lse, workspace=wsp)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.run(out=out, lse=lse, workspace=wsp)
        graphs.append(graph)
        outs.append((out, lse, wsp))
    cases[0].lens = cases[0].own.lens = [150, 0, 87]
    cases[0].own.seq_lens.copy_(torch.tensor(cases[0].lens, dtype=torch.int32))
    cases[1].P = 1111
    cases[1].first.seq_lens.fill_(1111)
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
        c.check(out, lse)
    out, lse = cases[1].run(stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(out, outs[1][0]) and torch.equal(lse, outs[1][1])


def test_long_prefix():
    """Positions past 2^16 and pages past 2^32 bytes, every position with a say."""
    pages, page, P, H, B = 66000, 64, 100000, 8, 20
    pool = torch.zeros((pages, page, 576), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(2)
    used = (P + page - 1) // page
    table = torch.arange(pages - 1, pages - 1 - used, -1, dtype=torch.int32, device=DEV)[None].contiguous()
    pool[-used:] = torch.randn((used, page, 576), generator=g, device=DEV).to(torch.bfloat16)
    prefix = binding.Cache(None, pool, torch.tensor([P], dtype=torch.int32, device=DEV), block_table=table, page_size=page)
    own = torch.randn((B, 40, 576), generator=g, device=DEV).to(torch.bfloat16)
    cache = binding.Cache(None, own, torch.full((B,), 40, dtype=torch.int32, device=DEV))
    q = torch.randn((B, H, 576), generator=g, device=DEV).to(torch.bfloat16)
    out, lse = binding.prefix_mla_decode(q, prefix, cache, SCALE)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    shared = pool[-used:].flip(0).reshape(-1, 576)[:P].double()
    for b in range(B):
        c = torch.cat([shared, own[b].double()])
        l = q[b].double() @ c.T * SCALE
        w = torch.softmax(l, -1)
        ref, A = w @ c[:, :512], w @ c[:, :512].abs()
        L = (q[b].double().abs() @ c.abs().T * SCALE).amax(-1)
        assert bool(((out[b].double() - ref).abs() <= 2.0 ** -8 * (A + 2 * ref.abs()) + 2.0 ** -11 * L[:, None] * A).all())
        assert bool(((lse[b].double() - torch.logsumexp(l, -1)).abs() <= 2.0 ** -12 * L + 2.0 ** -16).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H", [16, 128])
def test_every_tile_counts(fp8, H):
    """A tile that is lost, doubled or wrongly weighted shows in the lse: with queries of zero every
    position weighs the same, and the lse is the logarithm of their number to fp32."""
    P, lens = 5000, [700, 64, 0, 129, 1, 333, 65, 2]
    case = Shared(P, lens, 1, H, 64, fp8, seed=30)
    case.own.q.zero_()
    case.q = case.own.q
    out, lse = case.device().run()
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        assert bool(((lse[b].double() - math.log(P + n)).abs() <= 2.0 ** -20 * (1 + math.log(P + n))).all())
    case.check(out, lse)


def test_checked_library():
    case = Shared(900, [70, 300, 0, 5], 1, 16, 64, seed=31).device()
    out, lse = case.run()
    again = case.run(checked=True)
    torch.cuda.synchronize()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1]) and binding.device_status(checked=True) == 0


def test_converted_fp8_prefix_edges():
    """A prefix that is converted once: its length on the device shorter than its table, bad pages, a NaN code, and
    what stays in the workspace from the call before."""
    H, B, page = 128, 24, 64
    case = Shared(3001, [5] * B, 1, H, page, True, seed=40, prefix_max=4096, garbage=False)
    case.first.latent.view(torch.uint8)[case.first.table[0, 20].item(), 3, 17] = 0x7F      # NaN at position 1283
    wsp = binding.alloc_workspace(binding.prefix_mla_workspace_size(B, H), DEV).fill_(0xFF)
    out, lse = case.device().run(workspace=wsp)
    torch.cuda.synchronize()
    assert bool(out.isnan().all()) and bool(lse.isnan().all()) and binding.device_status() == 0
    case.P = 1283                                     # up to that position
    case.first.seq_lens.fill_(1283)
    out, lse = case.run(workspace=wsp)
    torch.cuda.synchronize()
    case.check(out, lse, range(0, B, 5))
    good = out.clone()
    kept = int(case.first.d_table[0, 7])
    case.first.d_table[0, 7] = 1 << 29
    out, _ = case.run(workspace=wsp)
    torch.cuda.synchronize()
    assert binding.device_status() == binding.DSI_ERR_BOUNDS and bool(out.isfinite().all())
    case.first.d_table[0, 7] = kept
    out, _ = case.run(workspace=wsp)
    torch.cuda.synchronize()
    assert binding.device_status() == 0 and torch.equal(out, good)
