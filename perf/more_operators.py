"""Cases that measure the operators with which a hybrid model serves requests that go on from a common
prefix: attention over latent rows that a whole batch shares, and linear attention with a decay for each
head, whose state takes the place of a cache, over prompts and for a step's tokens.

``own`` false: plain torch in 32 bits.  ``own`` true: the library's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
D_QK, D_LATENT = 576, 512
TILES = 5                                   # scales of an FP8 latent row: tiles of 128 dims
SCALE = 1.0 / math.sqrt(D_QK)
BLOCK = 128                                 # tokens that the plain linear attention takes together


def listed():
    return [
        # a few requests on one device of several (16 heads), a prefix of 2048 positions: latency
        dict(name="prefix_few_2048", op="prefix", batch=4, tokens=1, heads=16, prefix=2048, suffix=40,
             page=0, fp8=False),
        # the decode batch that the layer is quoted on, its history one shared document; every sequence
        # with an answer of its own of any length, on the same pages
        dict(name="prefix_batch_32768", op="prefix", batch=64, tokens=1, heads=128, prefix=32768,
             suffix=777, page=64, fp8=False),
        # the same batch where eight devices share the heads
        dict(name="prefix_batch_16_heads", op="prefix", batch=64, tokens=1, heads=16, prefix=32768,
             suffix=1024, page=64, fp8=False),
        # the longest prefix, an odd number of positions, kept apart from the sequences' rows
        dict(name="prefix_long_131071", op="prefix", batch=48, tokens=1, heads=32, prefix=131071,
             suffix=300, page=0, fp8=False),
        # a speculative step of two tokens over FP8 pages
        dict(name="prefix_two_tokens_fp8", op="prefix", batch=17, tokens=2, heads=64, prefix=8191,
             suffix=500, page=64, fp8=True),
        # a prompt of 8192 tokens
        dict(name="linear_prompt_8192", op="prompt", lengths="one", batch=1, tokens=8192, heads=64,
             kv_heads=64, dk=128, dv=128, start="none"),
        # prompts of any length, among them an empty one and one of one token, that go on from the state
        # of a common prefix
        dict(name="linear_prompts_ragged", op="prompt", lengths="ragged", batch=24, tokens=4096, heads=16,
             kv_heads=16, dk=128, dv=128, start="fork"),
        # a long document with few heads
        dict(name="linear_long_few_heads", op="prompt", lengths="one", batch=1, tokens=32768, heads=8,
             kv_heads=8, dk=64, dv=64, start="none"),
        # a chunk of a longer prompt, shared key heads, odd sizes
        dict(name="linear_chunk_odd", op="prompt", lengths="one", batch=1, tokens=777, heads=12,
             kv_heads=4, dk=96, dv=80, start="own"),
        # a single sequence's next token: latency
        dict(name="linear_step_single", op="step", batch=1, tokens=1, heads=16, kv_heads=16, dk=128,
             dv=128),
        # a step of the decode batch
        dict(name="linear_step_batch", op="step", batch=64, tokens=1, heads=64, kv_heads=64, dk=128,
             dv=128),
        # a step of four candidate tokens with narrow heads
        dict(name="linear_step_four_tokens", op="step", batch=24, tokens=4, heads=32, kv_heads=8, dk=64,
             dv=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "prompt", "prompt", "step"])
    if op == "prefix":
        heads = rng.choice([1, 3, 8, 16, 16, 32, 64, 128])
        batch, tokens = _log(rng, 1, 128), rng.choice([1, 1, 1, 2, 4])
        most = min(131072, max(64, 64 * 128 * 32768 // (batch * tokens * heads)))
        return dict(op=op, batch=batch, tokens=tokens, heads=heads, prefix=_log(rng, 1, most),
                    suffix=_log(rng, 1, min(4096, 131072 // batch)),
                    page=rng.choice([0, 0, 16, 24, 64, 64, 128]), fp8=rng.random() < 0.3)
    kv = rng.randint(1, 16)
    heads = kv * rng.choice([1, 1, 1, 2, 4])
    dk = rng.choice([64, 128, 128, 8 * rng.randint(2, 16)])
    dv = dk if rng.random() < 0.6 else 8 * rng.randint(2, 16)
    if op == "step":
        return dict(op=op, batch=_log(rng, 1, 64), tokens=rng.choice([1, 1, 2, 4]), heads=heads,
                    kv_heads=kv, dk=dk, dv=dv)
    lengths = rng.choice(["one", "ragged"])
    batch = 1 if lengths == "one" else _log(rng, 2, 48)
    most = min(32768, 64 * 8192 // (heads * batch))
    return dict(op=op, lengths=lengths, batch=batch, tokens=_log(rng, 1, max(2, most)), heads=heads,
                kv_heads=kv, dk=dk, dv=dv, start=rng.choice(["none", "own", "fork"]))


# ----------------------------------------------------------------------------- inputs

def _spread(n, longest):
    """n lengths from 1 to the longest, spread over their logarithm, one of them empty."""
    if n == 1:
        return [longest]
    r = [int(round(math.exp(math.log(max(1, longest)) * ((7 * i) % n) / (n - 1)))) for i in range(n)]
    if n >= 8:
        r[3] = 0
    return r


def _lengths(case):
    if case["op"] == "prompt" and case["lengths"] == "one":
        return [case["tokens"]]
    return _spread(case["batch"], case["suffix"] if case["op"] == "prefix" else case["tokens"])


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return _prepare_prefix(case, g) if case["op"] == "prefix" else _prepare_linear(case, g)


def _rows(shape, fp8, g):
    """Latent rows and their scales (None for bf16)."""
    x = torch.randn(shape + (D_QK,), generator=g, device=DEV, dtype=torch.bfloat16)
    if not fp8:
        return x, None
    return ((x * 64).clamp(-448, 448).to(torch.float8_e4m3fn),
            torch.empty(shape + (TILES,), device=DEV).uniform_(1 / 128, 1 / 32, generator=g))


def _prepare_prefix(case, g):
    B, T, H, P, page = case["batch"], case["tokens"], case["heads"], case["prefix"], case["page"]
    lens = _lengths(case)
    st = dict(case=case, prefix_table=None, table=None,
              prefix_len=torch.tensor([P], dtype=torch.int32, device=DEV),
              seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    if page:
        # prefix and sequences live on pages of one pool, in any order
        need = [(n + page - 1) // page for n in [P] + lens]
        pool = sum(need) + 3
        ids = torch.randperm(pool, generator=g, device=DEV).to(torch.int32).cpu()
        table = torch.full((B + 1, max(max(need), 1)), -1, dtype=torch.int32)
        at = 0
        for b, k in enumerate(need):
            table[b, :k] = ids[at:at + k]
            at += k
        st["prefix_table"] = table[:1].to(DEV)
        st["table"] = table[1:, :max(max(need[1:]), 1)].contiguous().to(DEV)
        st["latent"], st["scale"] = st["prefix_latent"], st["prefix_scale"] = _rows((pool, page), case["fp8"], g)
    else:
        st["prefix_latent"], st["prefix_scale"] = _rows((1, P), case["fp8"], g)
        st["latent"], st["scale"] = _rows((B, max(max(lens), 1)), case["fp8"], g)
    st["q"] = (torch.randn((B * T, H, D_QK), generator=g, device=DEV) * 1.5).to(torch.bfloat16)
    st["out"] = torch.empty((B * T, H, D_LATENT), dtype=torch.bfloat16, device=DEV)
    st["lse"] = torch.empty((B * T, H), device=DEV)
    if own:
        from indexed_sparse_attention_indexer_gb300 import binding
        st["prefix_cache"] = binding.Cache(None, st["prefix_latent"], st["prefix_len"], page_size=page,
                                           block_table=st["prefix_table"], latent_scale=st["prefix_scale"])
        st["cache"] = binding.Cache(None, st["latent"], st["seq_lens"], page_size=page,
                                    block_table=st["table"], latent_scale=st["scale"])
        st["workspace"] = binding.alloc_workspace(binding.prefix_mla_workspace_size(B * T, H), DEV)
    return st


def _prepare_linear(case, g):
    B, H, Hk, dk, dv = case["batch"], case["heads"], case["kv_heads"], case["dk"], case["dv"]
    step = case["op"] == "step"
    lens = [case["tokens"]] * B if step else _lengths(case)
    n = sum(lens)
    # queries, keys and values leave one projection side by side
    qkv = torch.randn((n, H * dk + Hk * (dk + dv)), generator=g, device=DEV)
    qkv = (qkv * torch.empty((n, 1), device=DEV).uniform_(0.3, 3.0, generator=g)).to(torch.bfloat16)
    q, k, v = qkv.split([H * dk, Hk * dk, Hk * dv], dim=1)
    # decays of exp(-1/2) to about one in a thousand a token, those of the heads in any order
    steps = torch.linspace(1.0, 10.0, H, device=DEV)[torch.randperm(H, generator=g, device=DEV)]
    start = "own" if step else case["start"]
    st = dict(case=case, q=q.view(n, H, dk), k=k.view(n, Hk, dk), v=v.view(n, Hk, dv), lens=lens,
              log_decay=-torch.exp2(-steps), scale=dk ** -0.5, start=start,
              out=torch.empty((n, H, dv), dtype=torch.bfloat16, device=DEV),
              seq_starts=torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32))
    # the states' slots: a step updates a sequence's own, a prompt leaves the one that it starts from
    slots = 2 * B + 1
    order = torch.randperm(slots, generator=g, device=DEV).to(torch.int32)
    st["state"] = torch.randn((slots, H, dk, dv), generator=g, device=DEV) * 2.0
    st["out_slots"] = order[:B].contiguous()
    st["in_slots"] = (st["out_slots"] if step else
                      {"none": torch.full_like(order[:B], -1), "own": order[B:2 * B].contiguous(),
                       "fork": order[B:B + 1].expand(B).contiguous()}[start])
    if own:
        from indexed_sparse_attention_indexer_gb300 import binding
        st["workspace"] = None if step else binding.alloc_workspace(
            binding.linear_workspace_size(n, B, H, dk, dv), DEV)
    return st


# ----------------------------------------------------------------------------- one pass

def run(st):
    op = st["case"]["op"]
    if op == "prefix":
        return _own_prefix(st) if own else _plain_prefix(st)
    if own:
        _own_linear(st)
    elif op == "prompt":
        _plain_prompt(st)
    else:
        _plain_step(st)
    return {"out": st["out"], "state": st["state"]}


def _own_prefix(st):
    from indexed_sparse_attention_indexer_gb300 import binding
    return binding.prefix_mla_decode(st["q"], st["prefix_cache"], st["cache"], SCALE,
                                     tokens_per_seq=st["case"]["tokens"], out=st["out"], lse=st["lse"],
                                     workspace=st["workspace"])


def _own_linear(st):
    from indexed_sparse_attention_indexer_gb300 import binding
    kw = dict(in_slots=st["in_slots"], out_slots=st["out_slots"], out=st["out"])
    if st["case"]["op"] == "step":
        binding.linear_decode(st["q"], st["k"], st["v"], st["log_decay"], st["scale"], st["state"],
                              tokens_per_seq=st["case"]["tokens"], **kw)
    else:
        binding.linear_prefill(st["q"], st["k"], st["v"], st["log_decay"], st["scale"], st["seq_starts"],
                               state=st["state"], workspace=st["workspace"], **kw)


def _values(latent, scale, at):
    """Latent rows `at` (of all rows) as they take part: an FP8 row is code * tile scale rounded to bf16."""
    if scale is None:
        return latent.view(-1, D_QK)[at].float()
    c = latent.view(torch.uint8).view(-1, D_QK)[at].view(torch.float8_e4m3fn).float()
    sc = scale.view(-1, TILES)[at].repeat_interleave(128, dim=-1)[..., :D_QK]
    return (c * sc).to(torch.bfloat16).float()


def _plain_prefix(st):
    case = st["case"]
    B, T, H, P, page = case["batch"], case["tokens"], case["heads"], case["prefix"], case["page"]
    pos = torch.arange(P, device=DEV)
    if page:
        pos = st["prefix_table"][0, pos // page].long() * page + pos % page
    shared = _values(st["prefix_latent"], st["prefix_scale"], pos)
    S = max(1, max(_lengths(case)))
    pos = torch.arange(S, device=DEV).expand(B, S)
    seq = torch.arange(B, device=DEV)[:, None]
    if page:
        at = st["table"][seq, pos // page].long().clamp(min=0) * page + pos % page
    else:
        at = seq * S + pos
    c = _values(st["latent"], st["scale"], at)
    t = torch.arange(T, device=DEV)
    n = st["seq_lens"].long()[:, None] - (T - 1 - t)[None, :]
    ok = (torch.arange(S, device=DEV) < n[..., None]).repeat_interleave(H, dim=1)        # [B, T * H, S]
    q = st["q"].float().view(B, T * H, D_QK)
    # one product of all rows with the shared positions, one of each sequence with its own
    first = torch.matmul(q.view(-1, D_QK), shared.t()).view(B, T * H, P) * SCALE
    second = (torch.matmul(q, c.transpose(1, 2)) * SCALE).masked_fill(~ok, -math.inf)
    top = torch.maximum(first.amax(-1, keepdim=True), second.amax(-1, keepdim=True))
    first, second = torch.exp(first - top), torch.exp(second - top)
    total = first.sum(-1, keepdim=True) + second.sum(-1, keepdim=True)
    out = torch.matmul(first.view(-1, P), shared[:, :D_LATENT]).view(B, T * H, D_LATENT)
    out = (out + torch.matmul(second, c[..., :D_LATENT])) / total
    st["out"].copy_(out.view(B * T, H, D_LATENT))
    st["lse"].copy_((top + torch.log(total)).view(B * T, H))
    return st["out"], st["lse"]


def _first_states(st):
    """The states [B, H, dk, dv] that the sequences start from."""
    slots = st["in_slots"].long()
    return st["state"][slots.clamp(min=0)] * (slots >= 0)[:, None, None, None]


def _power(g, n):
    """exp(g n) for g [H] and whole numbers n, the angles in 64 bits: [H, *n.shape]."""
    return torch.exp(g.double().view(-1, *[1] * n.dim()) * n.double()).float()


def _plain_prompt(st):
    case = st["case"]
    B, H, dk, dv = case["batch"], case["heads"], case["dk"], case["dv"]
    g, group = st["log_decay"], case["heads"] // case["kv_heads"]
    n = st["seq_starts"][1:].long() - st["seq_starts"][:-1].long()
    blocks = (max(1, max(st["lens"])) + BLOCK - 1) // BLOCK
    L = blocks * BLOCK
    # every sequence padded to whole blocks, keys and values of nothing behind its end
    i = torch.arange(L, device=DEV)
    ok = i < n[:, None]
    at = torch.where(ok, st["seq_starts"][:-1].long()[:, None] + i, torch.zeros_like(i))
    take = lambda x: (x[at] * ok[..., None, None]).float().transpose(1, 2)               # noqa: E731
    q, k, v = take(st["q"]), take(st["k"]), take(st["v"])
    k, v = k.repeat_interleave(group, dim=1), v.repeat_interleave(group, dim=1)
    first = _first_states(st)
    qb, kb, vb = (x.unflatten(2, (blocks, BLOCK)) for x in (q, k, v))
    # within a block
    r = torch.arange(BLOCK, device=DEV)
    apart = r[:, None] - r
    decay = torch.where(apart >= 0, _power(g, apart.clamp(min=0)), 0.0)[None, :, None]
    out = torch.matmul(torch.matmul(qb, kb.transpose(-1, -2)) * decay, vb)
    # what each block adds to the state, and the state that it finds
    left = _power(g, BLOCK - 1 - r)[None, :, None, :, None]
    adds = torch.matmul((kb * left).transpose(-1, -2), vb).flatten(-2)                    # [B, H, blocks, dk * dv]
    e = torch.arange(blocks, device=DEV)
    gap = e[:, None] - 1 - e
    carry = torch.where(gap >= 0, _power(g, BLOCK * gap.clamp(min=0)), 0.0)
    found = torch.matmul(carry, adds) + _power(g, BLOCK * e)[..., None] * first.flatten(-2)[:, :, None]
    since = _power(g, r + 1)[None, :, None, :, None]
    out = out + torch.matmul(qb, found.unflatten(-1, (dk, dv))) * since
    out = out.flatten(2, 3).transpose(1, 2) * st["scale"]
    st["out"][at[ok]] = out[ok].to(torch.bfloat16)
    # the state behind every sequence's last token
    left = _power(g, (n[:, None] - 1 - i).clamp(min=0)).transpose(0, 1)[..., None]
    last = torch.matmul((k * left).transpose(-1, -2), v) + _power(g, n).t()[..., None, None] * first
    st["state"][st["out_slots"].long()] = last


def _plain_step(st):
    case = st["case"]
    B, T, H, g = case["batch"], case["tokens"], case["heads"], st["log_decay"]
    group = H // case["kv_heads"]
    q = st["q"].float().unflatten(0, (B, T)).transpose(1, 2)
    k = st["k"].float().unflatten(0, (B, T)).transpose(1, 2).repeat_interleave(group, dim=1)
    v = st["v"].float().unflatten(0, (B, T)).transpose(1, 2).repeat_interleave(group, dim=1)
    s, t = _first_states(st), torch.arange(T, device=DEV)
    apart = t[:, None] - t
    decay = torch.where(apart >= 0, _power(g, apart.clamp(min=0)), 0.0)
    out = torch.matmul(torch.matmul(q, k.transpose(-1, -2)) * decay, v)
    out = (out + torch.matmul(q, s) * _power(g, t + 1)[..., None]) * st["scale"]
    st["out"].copy_(out.transpose(1, 2).flatten(0, 1))
    left = _power(g, T - 1 - t)[..., None]
    st["state"][st["out_slots"].long()] = (
        torch.matmul((k * left).transpose(-1, -2), v)
        + torch.exp(g.double() * T).float()[:, None, None] * s)


# ----------------------------------------------------------------------------- counts

def work(case):
    B, T, H = case["batch"], case["tokens"], case["heads"]
    lens = _lengths(case) if case["op"] != "step" else [T] * B
    if case["op"] == "prefix":
        row = D_QK + 4 * TILES if case["fp8"] else 2 * D_QK
        pairs = B * T * case["prefix"] + sum(max(0, n - t) for n in lens for t in range(T))
        return {"bytes": (case["prefix"] + sum(lens)) * row + B * T * H * (2 * D_QK + 2 * D_LATENT + 4),
                "flops": 2 * pairs * H * (D_QK + D_LATENT)}
    Hk, dk, dv, n = case["kv_heads"], case["dk"], case["dv"], sum(lens)
    # token by token: the state decayed and added to (three operations an entry), then read (two)
    start = {"none": 0, "fork": 1, "own": B}["own" if case["op"] == "step" else case["start"]]
    return {"bytes": 2 * n * (H * (dk + dv) + Hk * (dk + dv)) + 4 * (start + B) * H * dk * dv + 4 * H,
            "flops": 5 * n * H * dk * dv}


# ----------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return _exact_prefix(st) if case["op"] == "prefix" else _exact_linear(st)


def _exact_rows(latent, scale, at):
    if scale is None:
        return latent.flatten(0, 1)[at].double()
    c = latent.flatten(0, 1).view(torch.uint8)[at].view(torch.float8_e4m3fn).double()
    for t in range(TILES):
        c[:, 128 * t:128 * t + 128] *= scale.flatten(0, 1)[at, t].double()[:, None]
    return c.to(torch.bfloat16).double()


def _exact_prefix(st):
    case = st["case"]
    T, H, P, page = case["tokens"], case["heads"], case["prefix"], case["page"]
    spots = torch.arange(P, device=DEV)
    at = st["prefix_table"][0].long()[spots // page] * page + spots % page if page else spots
    shared = _exact_rows(st["prefix_latent"], st["prefix_scale"], at)
    out, lse = [], []
    for b, n in enumerate(_lengths(case)):
        spots = torch.arange(n, device=DEV)
        wide = max(1, max(_lengths(case)))
        at = st["table"][b].long()[spots // page] * page + spots % page if page else b * wide + spots
        c = torch.cat([shared, _exact_rows(st["latent"], st["scale"], at)])
        for t in range(T):
            see = P + max(0, n - (T - 1 - t))
            logits = st["q"][b * T + t].double() @ c[:see].t() / math.sqrt(D_QK)
            lse.append(torch.logsumexp(logits, dim=-1))
            out.append(torch.softmax(logits, dim=-1) @ c[:see, :D_LATENT])
    return torch.stack(out), torch.stack(lse)


def _exact_linear(st):
    """Every token's sum over those before it, a head at a time."""
    case = st["case"]
    H, dv = case["heads"], case["dv"]
    if sum(n * n for n in st["lens"]) * H * (case["dk"] + dv) > 6e12:
        return None
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    state = st["state"].double()
    decay = st["log_decay"].double()
    at = 0
    for b, n in enumerate(st["lens"]):
        src, dst = int(st["in_slots"][b]), int(st["out_slots"][b])
        new = torch.zeros(st["state"].shape[1:], dtype=torch.float64, device=DEV)
        for h in range(H):
            hk = h * case["kv_heads"] // H
            s0 = st["state"][src, h].double() if src >= 0 else torch.zeros_like(new[h])
            q, k, v = (st[x][at:at + n, y].double() for x, y in (("q", h), ("k", hk), ("v", hk)))
            i = torch.arange(n, device=DEV, dtype=torch.float64)
            for lo in range(0, n, 4096):
                rows = i[lo:lo + 4096]
                far = rows[:, None] - i[:lo + len(rows)]
                w = torch.exp(decay[h] * far.clamp(min=0)) * (far >= 0)
                y = (q[lo:lo + 4096] @ k[:lo + len(rows)].t() * w) @ v[:lo + len(rows)]
                y = y + torch.exp(decay[h] * (rows + 1))[:, None] * (q[lo:lo + 4096] @ s0)
                out[at + lo:at + lo + len(rows), h] = y * st["scale"]
            new[h] = torch.exp(decay[h] * n) * s0 + (k * torch.exp(decay[h] * (n - 1 - i))[:, None]).t() @ v
        state[dst] = new
        at += n
    return {"out": out, "state": state}
