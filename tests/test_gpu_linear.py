"""Linear attention with a decay for each head (dsi_linear_prefill, dsi_linear_decode) against the
formula in 64 bits.

With w_ij = exp(g (i - j)) q_i . k_j, M_i = scale (sum_j exp(g (i - j)) (|q_i| . |k_j|) |v_j| +
exp(g (i + 1)) |S_0|^T |q_i|) (the same sums of magnitudes) and N_S the state's sum of magnitudes, tolerances per element:
  decode: every step rounds the state twice and its decay once, an output sums dk products:
    (dk + 4 n + 16) 2^-24 M_i and half a bf16 step of the output, 2^-8 |out|;
    state (4 n + 16) 2^-24 N_S;
  prefill: the weights within 128 tokens and the state that they find are rounded to bf16 (2^-8 of each), the
    values entering the state split in two bf16 parts (2^-16), fp32 sums of at most n + dk terms that
    the tensor core may cut off rather than round (2^-22 a term), exponentials of arguments down to
    -150 whose angle is rounded in fp32 (150 * 2^-24 < 2^-16):
    2^-8 (|out| + scale (sum over the token's 128 |w_ij| |v_j| + exp(..) |S|^T |q_i|)) + (2^-14 + (n + dk) 2^-22) M_i;
    state (2^-14 + n 2^-22) N_S.
"""
import ctypes
import math

import pytest
import torch

from indexed_sparse_attention_indexer_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"
BLOCK = 128


def decays(H, kind, g):
    if kind == "mixed":                       # exp(-1/2) to one in a thousand a token
        return -torch.exp2(-torch.linspace(1.0, 10.0, H)[torch.randperm(H, generator=g)])
    if kind == "none":
        return torch.zeros(H)
    if kind == "near":                        # one in 10^5 to one in 10^7
        return -torch.logspace(-5, -7, H)
    # strong ones, some to nothing
    return torch.tensor([(-math.inf, -90.0, -20.0, -3.0)[i % 4] for i in range(H)])


class Case:
    """Inputs as views of one projection, rows around the sequences and unused slots filled with NaN."""

    def __init__(self, lens, H, Hk=None, dk=128, dv=128, kind="mixed", state=True, seed=0, lead=3, tail=2,
                 fork=False, heads_first=False):
        g = torch.Generator().manual_seed(seed)
        Hk = Hk or H
        self.lens, self.H, self.Hk, self.dk, self.dv = list(lens), H, Hk, dk, dv
        self.lead, n = lead, sum(lens) + lead + tail
        self.n = n
        wide = H * dk + Hk * (dk + dv)
        x = torch.randn((n, wide), generator=g) * torch.empty((n, 1)).uniform_(0.3, 3.0, generator=g)
        x = x.to(torch.bfloat16)
        x[:lead] = math.nan
        x[n - tail:] = math.nan
        q, k, v = x.split([H * dk, Hk * dk, Hk * dv], dim=1)
        self.q, self.k, self.v = q.view(n, H, dk), k.view(n, Hk, dk), v.view(n, Hk, dv)
        d = x.to(DEV)
        dq, dk_, dv_ = d.split([H * dk, Hk * dk, Hk * dv], dim=1)
        self.dq, self.dk_, self.dv_ = dq.view(n, H, dk), dk_.view(n, Hk, dk), dv_.view(n, Hk, dv)
        if heads_first:                       # [heads, tokens, dims] in memory
            self.dq, self.dk_, self.dv_ = (t.transpose(0, 1).contiguous().transpose(0, 1)
                                           for t in (self.dq, self.dk_, self.dv_))
        self.log_decay = decays(H, kind, g)
        self.scale = dk ** -0.5
        starts = [lead]
        for m in lens:
            starts.append(starts[-1] + m)
        self.starts = torch.tensor(starts, dtype=torch.int32, device=DEV)
        B = len(lens)
        self.B = B
        self.state = self.in_slots = self.out_slots = None
        if state:
            order = torch.randperm(2 * B + 3, generator=g).to(torch.int32)
            self.state = torch.full((2 * B + 3, H, dk, dv), math.nan)
            ins = order[:1].expand(B).clone() if fork else order[:B].clone()
            for i, s in enumerate(ins.tolist()):
                self.state[s] = torch.randn((H, dk, dv), generator=g) * 2
            if B > 2 and not fork:
                ins[2] = -1
            self.in_slots, self.out_slots = ins, order[B:2 * B].clone()
            if B > 3:
                self.out_slots[3] = -5

    def reference(self, b):
        """out, its tolerance in prefill and decode, and the state with the same, of sequence b."""
        n, at = self.lens[b], self.lead + sum(self.lens[:b])
        H, dk = self.H, self.dk
        q = self.q[at:at + n].double().to(DEV).transpose(0, 1)
        rep = H // self.Hk
        k = self.k[at:at + n].double().to(DEV).transpose(0, 1).repeat_interleave(rep, 0)
        v = self.v[at:at + n].double().to(DEV).transpose(0, 1).repeat_interleave(rep, 0)
        g = self.log_decay.double().to(DEV)
        src = -1 if self.state is None else int(self.in_slots[b])
        s0 = (self.state[src].double().to(DEV) if src >= 0
              else torch.zeros((H, dk, self.dv), dtype=torch.float64, device=DEV))

        def power(m):                        # exp(g m), 1 for m = 0 whatever g is
            m = m.double()
            e = torch.exp(g.view(-1, *[1] * m.dim()) * m)
            return torch.where(m == 0, torch.ones_like(e), e)

        i = torch.arange(n, device=DEV)
        far = i[:, None] - i
        lam = power(far.clamp(min=0)) * (far >= 0)
        w = lam * (q @ k.transpose(1, 2))
        since = power(i + 1)[..., None]
        out = self.scale * (w @ v + since * (q @ s0))
        M = self.scale * ((lam * (q.abs() @ k.abs().transpose(1, 2))) @ v.abs() + since * (q.abs() @ s0.abs()))
        near = (i[:, None] // BLOCK == i // BLOCK)
        A = (w.abs() * near) @ v.abs()
        for c in range(0, n, BLOCK):         # what the state that a block finds adds
            left = power((c - 1 - i[:c]).clamp(min=0))[..., None]
            s = power(torch.tensor(float(c), device=DEV))[:, None, None] * s0 + (k[:, :c] * left).transpose(1, 2) @ v[:, :c]
            rows = slice(c, min(n, c + BLOCK))
            A[:, rows] += power(i[rows] - c + 1)[..., None] * (q[:, rows].abs() @ s.abs())
        left = power(n - 1 - i)[..., None]
        all_ = power(torch.tensor(float(n), device=DEV))[:, None, None]
        new = all_ * s0 + (k * left).transpose(1, 2) @ v
        N = all_ * s0.abs() + (k.abs() * left).transpose(1, 2) @ v.abs()
        tol = {"prefill": 2.0 ** -8 * (out.abs() + self.scale * A) + (2.0 ** -14 + (n + dk) * 2.0 ** -22) * M,
               "decode": 2.0 ** -8 * out.abs() + (dk + 4 * n + 16) * 2.0 ** -24 * M}
        tol_s = {"prefill": (2.0 ** -14 + n * 2.0 ** -22) * N, "decode": (4 * n + 16) * 2.0 ** -24 * N}
        tiny = 1e-37                          # what fp32 and bf16 flush
        return (out.transpose(0, 1), {x: t.transpose(0, 1) + tiny for x, t in tol.items()}, new,
                {x: t + tiny for x, t in tol_s.items()})

    def prefill(self, workspace=None, stream=None, out=None):
        """Out (rows behind the sequences marked) and the states after a call."""
        state = self.state.to(DEV) if self.state is not None else None
        if out is None:
            out = torch.full((self.n, self.H, self.dv), 7.0, dtype=torch.bfloat16, device=DEV)
        move = lambda t: t.to(DEV) if t is not None else None                    # noqa: E731
        binding.linear_prefill(self.dq, self.dk_, self.dv_, self.log_decay.to(DEV), self.scale, self.starts,
                               state=state, in_slots=move(self.in_slots), out_slots=move(self.out_slots),
                               out=out, workspace=workspace, stream=stream)
        return out, state

    def check(self, out, state, form="prefill"):
        assert binding.device_status() == 0
        at = self.lead
        written = set()
        for b, n in enumerate(self.lens):
            ref, tol, new, tol_s = self.reference(b)
            err = (out[at:at + n].double() - ref).abs()
            assert bool((err <= tol[form]).all()), (b, float((err / tol[form]).max()))
            at += n
            if state is not None and int(self.out_slots[b]) >= 0:
                written.add(int(self.out_slots[b]))
                err = (state[int(self.out_slots[b])].double() - new).abs()
                assert bool((err <= tol_s[form]).all()), (b, float((err / tol_s[form]).max()))
        assert bool((out[:self.lead] == 7).all()) and bool((out[at:] == 7).all())
        if state is not None:                 # the other slots are as they were, bit for bit
            rest = [s for s in range(state.shape[0]) if s not in written]
            assert torch.equal(state[rest].view(torch.int32), self.state[rest].to(DEV).view(torch.int32))


PREFILLS = [
    dict(lens=[1], H=2), dict(lens=[127], H=3), dict(lens=[128], H=1), dict(lens=[129], H=2),
    dict(lens=[700], H=4, kind="none"), dict(lens=[513], H=4, kind="strong"), dict(lens=[900], H=3, kind="near"),
    dict(lens=[0], H=2), dict(lens=[5, 0, 300, 1, 128, 77], H=6, Hk=2),
    dict(lens=[40, 260, 0, 9], H=4, fork=True), dict(lens=[333], H=2, state=False),
    dict(lens=[200, 31], H=2, dk=64, dv=64), dict(lens=[300], H=2, dk=96, dv=80), dict(lens=[257], H=2, dk=8, dv=8),
    dict(lens=[140], H=3, dk=72, dv=128), dict(lens=[140], H=3, dk=128, dv=24), dict(lens=[390], H=4, Hk=1, dk=40, dv=104),
    dict(lens=[150, 150], H=5, heads_first=True), dict(lens=[130] * 40, H=8), dict(lens=[1500], H=1),
    dict(lens=[7, 8, 9, 0, 10, 200, 1], H=3), dict(lens=[1] * 30 + [700], H=4, Hk=2, fork=True), dict(lens=[8], H=2), dict(lens=[9], H=2),
    dict(lens=[3, 9, 8, 2, 1, 0] * 50, H=1, dk=96), dict(lens=[5, 4000, 2], H=1, dv=40),
    dict(lens=[7 * i % 41 for i in range(300)], H=2, dk=64, dv=64), dict(lens=[i % 3 * 100 for i in range(256)], H=1, dk=32, dv=16),
]


@pytest.mark.parametrize("kw", PREFILLS, ids=str)
def test_prefill(kw):
    c = Case(**kw)
    c.check(*c.prefill())


# long sequences of few heads, which a workspace lets the call cut into segments
LONG = [
    dict(lens=[9000], H=1), dict(lens=[4000], H=2, kind="none", dk=64, dv=64), dict(lens=[4097], H=2, kind="near"),
    dict(lens=[7000, 0, 8000, 1, 129], H=2), dict(lens=[5000, 2500], H=2, fork=True), dict(lens=[3500], H=2, state=False),
    dict(lens=[4000], H=4, kind="strong", dk=96, dv=40), dict(lens=[128 * 25], H=1), dict(lens=[3333], H=3, Hk=1),
]


@pytest.mark.parametrize("kw", LONG, ids=str)
def test_long_prefill(kw):
    """Cut into segments and whole (without a workspace), each against the formula."""
    c = Case(**kw)
    heads = (c.H, c.dk, c.dv)
    assert binding.linear_workspace_size(c.n, c.B, *heads) > 256
    a = c.prefill()
    c.check(*a)
    again = c.prefill()
    assert torch.equal(a[0], again[0])
    out = torch.full((c.n, c.H, c.dv), 7.0, dtype=torch.bfloat16, device=DEV)
    state = c.state.to(DEV) if c.state is not None else None
    s, _ = binding._linear(c.dq, c.dk_, c.dv_, c.log_decay.to(DEV), c.scale, state,
                           None if state is None else c.in_slots.to(DEV), None if state is None else c.out_slots.to(DEV),
                           out, c.B, None)
    keep = [c.log_decay.to(DEV)] + ([] if state is None else [c.in_slots.to(DEV), c.out_slots.to(DEV)])
    s.log_decay = keep[0].data_ptr()
    if state is not None:
        s.in_slots, s.out_slots = keep[1].data_ptr(), keep[2].data_ptr()
    st = binding.load().dsi_linear_prefill(ctypes.byref(s), c.n, c.starts.data_ptr(), c.B, None, 0, binding._stream(None))
    assert st == 0
    torch.cuda.synchronize()
    c.check(out, state)


@pytest.mark.parametrize("where", ["q", "k", "v"])
def test_long_values_that_are_not_finite(where):
    """As below, over the segments of a cut sequence."""
    c = Case([4000, 300], H=2, lead=0, tail=0, seed=12)
    clean = c.prefill()[0]
    x = {"q": c.dq, "k": c.dk_, "v": c.dv_}[where]
    x[1500, 1, 5] = math.nan
    out, state = c.prefill()
    assert binding.device_status() == 0
    hit = torch.zeros(out.shape, dtype=torch.bool, device=DEV)
    hit[1500:1501 if where == "q" else 4000, 1] = True
    assert torch.equal(out[~hit], clean[~hit])
    ok = out.isfinite()
    if where == "v":
        assert not bool(ok[1500:4000, 1, 5].any())
    else:
        assert not bool(ok[hit.any(-1)].all(-1).any())
    assert bool(state[int(c.out_slots[0])][0].isfinite().all()) and bool(state[int(c.out_slots[1])].isfinite().all())
    assert bool(state[int(c.out_slots[0])][1].isfinite().all()) == (where == "q")


def test_long_starts_that_go_back():
    """More tokens in sequences than there are rows: reported, and nothing beyond the workspace."""
    c = Case([3000, 1000], H=1, lead=0, tail=0, seed=13)
    want = c.prefill()[0]
    size = binding.linear_workspace_size(c.n, 8, 1, 128, 128)
    ws = torch.full((size + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
    starts = torch.tensor([0, 3000, 0, 4000, 0, 4000, 0, 4000, 0], dtype=torch.int32, device=DEV)
    out = torch.zeros_like(want)
    binding.linear_prefill(c.dq, c.dk_, c.dv_, c.log_decay.to(DEV), c.scale, starts, out=out, workspace=ws[:size])
    assert binding.device_status() == binding.DSI_ERR_BOUNDS
    assert bool((ws[size:] == 0x5A).all())


@pytest.mark.parametrize("kw", [
    dict(B=1, T=1, H=1), dict(B=1, T=1, H=16), dict(B=5, T=1, H=7), dict(B=4, T=4, H=6, Hk=3), dict(B=3, T=5, H=4),
    dict(B=2, T=9, H=2, kind="strong"), dict(B=3, T=1, H=4, dk=64, dv=64), dict(B=3, T=2, H=4, dk=96, dv=80),
    dict(B=3, T=3, H=2, dk=8, dv=8), dict(B=2, T=1, H=3, dk=120, dv=32), dict(B=2, T=2, H=3, dk=16, dv=40),
    dict(B=64, T=1, H=32), dict(B=2, T=150, H=2, kind="near"), dict(B=4, T=2, H=4, heads_first=True)], ids=str)
def test_decode(kw):
    B, T = kw.pop("B"), kw.pop("T")
    c = Case([T] * B, lead=0, tail=0, **kw)
    state = c.state.to(DEV)
    out = binding.linear_decode(c.dq, c.dk_, c.dv_, c.log_decay.to(DEV), c.scale, state, tokens_per_seq=T,
                                in_slots=c.in_slots.to(DEV), out_slots=c.out_slots.to(DEV))
    c.check(out, state, "decode")


def test_in_place_slots_by_default():
    """Without slots sequence b updates slot b; with in_slots alone, the slot that it starts from."""
    c = Case([3, 3], H=4, lead=0, tail=0, seed=3)
    dec = c.log_decay.to(DEV)
    pool = torch.stack([c.state[int(s)] for s in c.in_slots] + [torch.full_like(c.state[0], math.nan)]).to(DEV)
    a, b, d = pool.clone(), pool.clone(), pool.flip(0).contiguous()
    out = binding.linear_decode(c.dq, c.dk_, c.dv_, dec, c.scale, a, tokens_per_seq=3)
    out2 = binding.linear_decode(c.dq, c.dk_, c.dv_, dec, c.scale, d, tokens_per_seq=3,
                                 in_slots=torch.tensor([2, 1], dtype=torch.int32, device=DEV))
    out3 = binding.linear_prefill(c.dq, c.dk_, c.dv_, dec, c.scale, c.starts, state=b)
    assert torch.equal(out, out2) and torch.equal(a[:2].flip(0), d[1:]) and bool(d[0].isnan().all())
    c.out_slots = torch.tensor([0, 1], dtype=torch.int32)
    for i in range(2):
        ref, tol, new, tol_s = c.reference(i)
        for o, s, form in ((out, a, "decode"), (out3, b, "prefill")):
            assert bool(((o[3 * i:3 * i + 3].double() - ref).abs() <= tol[form]).all())
            assert bool(((s[i].double() - new).abs() <= tol_s[form]).all())
    assert bool(a[2].isnan().all()) and bool(b[2].isnan().all())


def test_prompt_in_pieces_is_the_prompt():
    """A prompt, the same in two calls that pass the state on, and token by token."""
    c = Case([391], H=4, lead=0, tail=0, state=False, seed=5)
    dec = c.log_decay.to(DEV)
    ref, tol, new, tol_s = c.reference(0)
    for cuts in ([391], [128, 263], [1, 200, 190], [390, 1]):
        state = torch.zeros((1, 4, 128, 128), device=DEV)
        outs, at = [], 0
        for m in cuts:
            rows = slice(at, at + m)
            starts = torch.tensor([0, m], dtype=torch.int32, device=DEV)
            outs.append(binding.linear_prefill(c.dq[rows], c.dk_[rows], c.dv_[rows], dec, c.scale, starts, state=state))
            at += m
        # (blocks begin elsewhere: the sums of magnitudes bound every way of dividing them)
        err = (torch.cat(outs).double() - ref).abs()
        assert bool((err <= 4 * tol["prefill"]).all())
        assert bool(((state[0].double() - new).abs() <= len(cuts) * tol_s["prefill"]).all())
    state = torch.zeros((1, 4, 128, 128), device=DEV)
    outs = [binding.linear_decode(c.dq[i:i + 1], c.dk_[i:i + 1], c.dv_[i:i + 1], dec, c.scale, state) for i in range(391)]
    assert bool(((torch.cat(outs).double() - ref).abs() <= tol["decode"]).all())
    assert bool(((state[0].double() - new).abs() <= tol_s["decode"]).all())


@pytest.mark.parametrize("where", ["q", "k", "v"])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("at", [0, 70, 127, 200])
def test_values_that_are_not_finite(where, value, at):
    """A q reaches its own token; a k or v its head's tokens from its own on and the state, never
    earlier tokens, other heads or other sequences (of which one follows directly)."""
    c = Case([260, 90], H=3, lead=0, tail=0, seed=11, kind="mixed")
    x = {"q": c.dq, "k": c.dk_, "v": c.dv_}[where]
    {"q": c.q, "k": c.k, "v": c.v}[where][at, 1, 5] = 0.0       # the reference's
    clean = c.prefill()[0]
    x[at, 1, 5] = value
    out, state = c.prefill()
    assert binding.device_status() == 0
    ok = torch.isfinite(out.float())
    hit = torch.zeros_like(ok)
    if where == "q":
        hit[at, 1] = True
    else:
        hit[at:260, 1] = True
    if where == "v":                                            # its own dim at least
        assert not bool(ok[at:260, 1, 5].any())
        assert bool(state[int(c.out_slots[0])][1][:, 5].isfinite().logical_not().all())
    else:
        assert not bool(ok[hit.any(-1)].all(-1).any())
    assert bool(ok[~hit].all())
    assert torch.equal(out[~hit], clean[~hit])
    s = int(c.out_slots[0])
    assert bool(state[s][[0, 2]].isfinite().all()) and bool(state[int(c.out_slots[1])].isfinite().all())


def test_bad_slots_and_starts_are_reported():
    c = Case([20, 30], H=2, lead=0, tail=0, seed=2)
    want_out, want = c.prefill()
    assert binding.device_status() == 0
    slots = c.state.shape[0]
    bad = c.in_slots.clone()
    bad[1] = slots
    keep, c.in_slots = c.in_slots, bad
    out, state = c.prefill()
    assert binding.device_status() == binding.DSI_ERR_BOUNDS
    assert torch.equal(out[:20], want_out[:20]) and bool(out.isfinite().all())
    c.in_slots = keep
    bad = c.out_slots.clone()
    bad[0] = 1 << 30
    c.out_slots, keep = bad, c.out_slots
    out, state = c.prefill()
    assert binding.device_status() == binding.DSI_ERR_BOUNDS
    assert torch.equal(out, want_out) and torch.equal(state[int(keep[1])], want[int(keep[1])])
    assert bool(state[int(keep[0])].isnan().all())
    c.out_slots = keep
    for starts in ([-4, 20, 50], [0, 20, 51], [0, 20, 19]):
        c.starts = torch.tensor(starts, dtype=torch.int32, device=DEV)
        out, state = c.prefill()
        assert binding.device_status() == binding.DSI_ERR_BOUNDS
        assert torch.equal(out[:20], want_out[:20])
    assert bool((out[20:] == 7).all())


def test_streams_and_captures():
    """The same call on a stream of its own, captured and replayed: bit for bit the same."""
    c = Case([700, 31, 0, 260], H=4, seed=8)
    out, state = c.prefill()
    c.check(out, state)
    step = Case([2] * 3, H=4, lead=0, tail=0, seed=9)
    dec, ins, outs = step.log_decay.to(DEV), step.in_slots.to(DEV), step.out_slots.to(DEV)
    pool = step.state.to(DEV)
    y = binding.linear_decode(step.dq, step.dk_, step.dv_, dec, step.scale, pool, 2, ins, outs)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    again = c.prefill(stream=stream)
    stream.synchronize()
    assert torch.equal(out, again[0])
    o2 = torch.full_like(out, 7.0)
    s2, p2, y2 = c.state.to(DEV), step.state.to(DEV), torch.empty_like(y)
    dec2, ins2, outs2 = c.log_decay.to(DEV), c.in_slots.to(DEV), c.out_slots.to(DEV)
    ws = binding.alloc_workspace(binding.linear_workspace_size(c.n, c.B, c.H, 128, 128), DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        binding.linear_prefill(c.dq, c.dk_, c.dv_, dec2, c.scale, c.starts, s2, ins2, outs2, o2, ws)
        binding.linear_decode(step.dq, step.dk_, step.dv_, dec, step.scale, p2, 2, ins, outs, y2)
    for _ in range(3):
        o2.fill_(7.0)
        s2.copy_(c.state)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o2, out) and torch.equal(s2.view(torch.int32), state.view(torch.int32))
        assert torch.equal(y2, y) and torch.equal(p2.view(torch.int32), pool.view(torch.int32))


@pytest.mark.parametrize("lens,H", [([300, 5], 3), ([4000], 1)])
def test_checked_library(lens, H):
    """The bounds-checked build gives the same bits."""
    c = Case(lens, H=H, lead=0, tail=0, seed=21)
    out, state = c.prefill()
    again = c.state.to(DEV)
    out2 = binding.linear_prefill(c.dq, c.dk_, c.dv_, c.log_decay.to(DEV), c.scale, c.starts, again, c.in_slots.to(DEV),
                                  c.out_slots.to(DEV), checked=True)
    assert torch.equal(out, out2) and torch.equal(state.view(torch.int32), again.view(torch.int32))
    args = (c.dq[:4], c.dk_[:4], c.dv_[:4], c.log_decay.to(DEV), c.scale)
    a, b = (torch.ones((2, H, 128, 128), device=DEV) for _ in range(2))
    assert torch.equal(binding.linear_decode(*args, a, 2), binding.linear_decode(*args, b, 2, checked=True))
    assert torch.equal(a, b) and binding.device_status() == 0 and binding.device_status(checked=True) == 0


def test_offsets_past_32_bits():
    """Rows and slots that lie past 2^32 bytes: the same bits as close together."""
    n, wide = 33100, 65536                        # 4.3 GB of token rows
    g = torch.Generator(device=DEV).manual_seed(4)
    near = torch.randn((n, 3, 64), generator=g, device=DEV).to(torch.bfloat16)
    far = torch.empty((n, wide), dtype=torch.bfloat16, device=DEV)
    far[:, :192] = near.view(n, 192)
    far = far[:, :192].view(n, 3, 64)
    dec = torch.tensor([-0.01], device=DEV)
    starts = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    outs, states = [], []
    for x in (near, far):
        state = torch.zeros((1, 1, 64, 64), device=DEV)
        out = torch.empty((n, wide), dtype=torch.bfloat16, device=DEV)[:, :64].view(n, 1, 64) if x is far else None
        outs.append(binding.linear_prefill(x[:, :1], x[:, 1:2], x[:, 2:], dec, 0.125, starts, state, out=out))
        states.append(state)
    assert torch.equal(outs[0], outs[1]) and torch.equal(states[0], states[1])
    del far, outs
    slots = 70000                                 # 4.6 GB of states
    pool = torch.zeros((slots, 1, 128, 128), device=DEV)
    pool[-2:] = torch.randn((2, 1, 128, 128), generator=g, device=DEV)
    small = pool[-2:].clone()
    q, k, v = (torch.randn((2, 1, 128), generator=g, device=DEV).to(torch.bfloat16) for _ in range(3))
    at = torch.tensor([slots - 1, slots - 2], dtype=torch.int32, device=DEV)
    a = binding.linear_decode(q, k, v, dec, 0.1, pool, in_slots=at)
    b = binding.linear_decode(q, k, v, dec, 0.1, small, in_slots=at - (slots - 2))
    assert torch.equal(a, b) and torch.equal(pool[-2:], small) and not bool(pool[:-2].any())
    assert binding.device_status() == 0
