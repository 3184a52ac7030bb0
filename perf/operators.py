"""Cases that measure the cache-side operators of the attention layer: head norms with the position
rotation written into a cache, attention over a whole latent cache, and attention over a sliding
window of it with the first positions visible.

``own`` false: plain torch in 32 bits.  ``own`` true: the library's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
D_QK, D_LATENT = 576, 512
TILES = 5                                   # scales of an FP8 latent row: tiles of 128 dims
SCALE = 1.0 / math.sqrt(D_QK)
EPS = 1e-6


def listed():
    return [
        # one step of a decode batch: index queries and the new index key of every sequence, the
        # keys quantised into their rows of a paged MXFP8 cache
        dict(name="rope_index_step_mxfp8", op="rope", rows=64, hq=64, hk=1, d=128, norm_dim=128,
             rope_offset=0, rope_dim=64, norm_q="rms", norm_k="layer", interleaved=False,
             k_out="mxfp8", far=32768),
        # the same of a prefill of 8192 tokens into a bf16 cache
        dict(name="rope_index_prefill", op="rope", rows=8192, hq=64, hk=1, d=128, norm_dim=128,
             rope_offset=0, rope_dim=64, norm_q="none", norm_k="layer", interleaved=False,
             k_out="bf16", far=8192),
        # latent rows of long prompts (an odd number of tokens) into a paged FP8 cache: the latent
        # dims normed, the rope dims rotated
        dict(name="rope_latent_fp8", op="rope", rows=65537, hq=0, hk=1, d=576, norm_dim=512,
             rope_offset=512, rope_dim=64, norm_q="none", norm_k="rms", interleaved=True,
             k_out="fp8", far=131072),
        # grouped query heads with fewer key heads, the whole head normed and rotated
        dict(name="rope_grouped_heads", op="rope", rows=1537, hq=40, hk=8, d=96, norm_dim=96,
             rope_offset=0, rope_dim=96, norm_q="rms", norm_k="rms", interleaved=False,
             k_out="bf16", far=4096),
        # a single sequence's next token with few heads: latency
        dict(name="dense_single_2048", op="dense", batch=1, tokens=1, s=2048, heads=16, page=0,
             fp8=False, ragged=False),
        # the decode batch that the layer is quoted on, over its whole history
        dict(name="dense_batch_32768", op="dense", batch=64, tokens=1, s=32768, heads=128, page=0,
             fp8=False, ragged=False),
        # sequences of any length from one token up, on pages, some of them new
        dict(name="dense_ragged_paged", op="dense", batch=48, tokens=1, s=65536, heads=128, page=64,
             fp8=False, ragged=True),
        # a speculative step of two tokens over an FP8 cache
        dict(name="dense_two_tokens_fp8", op="dense", batch=17, tokens=2, s=8191, heads=64, page=64,
             fp8=True, ragged=True),
        # hybrid layers: the decode batch over the last 1024 positions and four sinks
        dict(name="window_batch_1024", op="window", batch=64, tokens=1, s=32768, heads=128, page=64,
             fp8=False, ragged=False, window=1024, sink=4, prefill=False),
        # a step of four candidate tokens with few heads and a short window
        dict(name="window_step_4x16", op="window", batch=24, tokens=4, s=5000, heads=16, page=16,
             fp8=False, ragged=True, window=129, sink=1, prefill=False),
        # a prompt's prefill over a window of 1024
        dict(name="window_prefill_4096", op="window", batch=1, tokens=4096, s=4096, heads=128,
             page=64, fp8=False, ragged=False, window=1024, sink=16, prefill=True),
        # a chunk of a longer prompt over an FP8 cache, odd sizes
        dict(name="window_chunk_fp8", op="window", batch=1, tokens=777, s=9001, heads=32, page=0,
             fp8=True, ragged=False, window=511, sink=70, prefill=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "dense", "dense", "window", "window"])
    if op == "rope":
        kind = rng.choice(["index", "latent", "heads"])
        if kind == "index":
            c = dict(rows=_log(rng, 1, 8192), hq=rng.randint(1, 64), hk=1, d=128, norm_dim=128,
                     rope_offset=rng.choice([0, 64]), rope_dim=64, k_out=rng.choice(["bf16", "mxfp8"]))
        elif kind == "latent":
            c = dict(rows=_log(rng, 1, 65537), hq=0, hk=1, d=576, norm_dim=512, rope_offset=512,
                     rope_dim=64, k_out=rng.choice(["bf16", "fp8"]))
        else:
            d = rng.choice([32, 64, 80, 96, 128, 192, 256])
            hk = rng.randint(1, 8)
            c = dict(rows=_log(rng, 1, 2048), hq=hk * rng.randint(1, 8), hk=hk, d=d, norm_dim=d,
                     rope_offset=0, rope_dim=rng.choice([d, d // 32 * 16]), k_out="bf16")
        return dict(op="rope", norm_q=rng.choice(["none", "rms", "layer"]),
                    norm_k=rng.choice(["rms", "layer"]), interleaved=rng.random() < 0.5,
                    far=_log(rng, 4096, 131072), **c)
    heads = rng.choice([1, 3, 8, 16, 32, 64, 128, 128])
    page = rng.choice([0, 0, 16, 24, 64, 64, 128])
    fp8 = rng.random() < 0.3
    if op == "dense":
        s = _log(rng, 1, 65536)
        batch = max(1, min(_log(rng, 1, 128), 2097152 // s))
        return dict(op=op, batch=batch, tokens=rng.choice([1, 1, 1, 2, 4]) if batch * s <= 524288 else 1,
                    s=s, heads=heads, page=page, fp8=fp8, ragged=rng.random() < 0.5)
    window, sink = _log(rng, 1, 1024), rng.choice([0, 1, 4, 16, 100])
    if rng.random() < 0.5:
        tokens = _log(rng, 1, 2048)
        return dict(op=op, batch=1, tokens=tokens, s=tokens + _log(rng, 1, 32768), heads=heads,
                    page=page, fp8=fp8, ragged=False, window=window, sink=sink, prefill=True)
    return dict(op=op, batch=_log(rng, 1, 128), tokens=rng.choice([1, 1, 2, 4]), s=_log(rng, 4, 16384),
                heads=heads, page=page, fp8=fp8, ragged=rng.random() < 0.5, window=window, sink=sink,
                prefill=False)


# ----------------------------------------------------------------------------- inputs

def _lengths(case):
    """History lengths: all s, or spread over 1..s by their logarithm, with one empty sequence."""
    B, s = case["batch"], case["s"]
    if not case["ragged"]:
        return [s] * B
    n = [int(round(math.exp(math.log(s) * ((7 * i) % B) / max(1, B - 1)))) for i in range(B)]
    if B >= 8:
        n[3] = 0
    return n


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return _prepare_rope(case, g) if case["op"] == "rope" else _prepare_attention(case, g)


def _prepare_rope(case, g):
    n, hq, hk, d, rd = case["rows"], case["hq"], case["hk"], case["d"], case["rope_dim"]
    nd, far = case["norm_dim"], case["far"]
    # queries and keys leave one projection side by side
    qk = torch.randn((n, (hq + hk) * d), generator=g, device=DEV)
    qk = (qk * torch.empty((n, 1), device=DEV).uniform_(0.2, 5.0, generator=g)).to(torch.bfloat16)
    inv = 10000.0 ** (-torch.arange(0, rd, 2, device=DEV, dtype=torch.float64) / rd)
    ang = torch.arange(far, device=DEV, dtype=torch.float64)[:, None] * inv
    table = torch.cat([ang.cos(), ang.sin()], dim=1).to(torch.float32)
    pool = n + 64
    st = dict(case=case, q=qk[:, :hq * d].view(n, hq, d), k=qk[:, hq * d:].view(n, hk, d), table=table,
              positions=torch.randint(0, far, (n,), generator=g, device=DEV),
              rows=torch.randperm(pool, generator=g, device=DEV)[:n],
              qw=torch.empty(nd, device=DEV).uniform_(0.5, 1.5, generator=g),
              kw=torch.empty(nd, device=DEV).uniform_(0.5, 1.5, generator=g),
              qb=torch.empty(nd, device=DEV).uniform_(-0.2, 0.2, generator=g),
              kb=torch.empty(nd, device=DEV).uniform_(-0.2, 0.2, generator=g),
              q_out=torch.empty((n, hq, d), device=DEV, dtype=torch.bfloat16))
    if case["k_out"] == "bf16":
        st["cache"] = torch.zeros((pool, hk, d), device=DEV, dtype=torch.bfloat16)
        st["scales"] = None
    else:
        st["cache"] = torch.zeros((pool, hk, d), device=DEV, dtype=torch.uint8).view(torch.float8_e4m3fn)
        st["scales"] = (torch.zeros((pool, hk, d // 32), device=DEV, dtype=torch.uint8)
                        if case["k_out"] == "mxfp8" else
                        torch.zeros((pool, hk, (d + 127) // 128), device=DEV))
    if own:
        from indexed_sparse_attention_indexer_gb300 import binding
        norm = {"none": None, "rms": "rms", "layer": "layer"}
        st["q_side"] = binding.Heads(
            st["q"], norm=norm[case["norm_q"]], weight=st["qw"] if case["norm_q"] != "none" else None,
            bias=st["qb"] if case["norm_q"] == "layer" else None, norm_dim=nd, out=st["q_out"]) if hq else None
        st["k_side"] = binding.Heads(
            st["k"], norm=norm[case["norm_k"]], weight=st["kw"],
            bias=st["kb"] if case["norm_k"] == "layer" else None, norm_dim=nd, out=st["cache"],
            out_scale=st["scales"], dst_rows=st["rows"])
    return st


def _prepare_attention(case, g):
    B, T, H, s, page = case["batch"], case["tokens"], case["heads"], case["s"], case["page"]
    lens = _lengths(case)
    if page:
        need = [(n + page - 1) // page for n in lens]
        shape, wide = (sum(need) + 3, page), max(max(need), 1)
        ids = torch.randperm(shape[0], generator=g, device=DEV).to(torch.int32)
        table = torch.full((B, wide), -1, dtype=torch.int32)
        at, ids_host = 0, ids.cpu()
        for b, k in enumerate(need):
            table[b, :k] = ids_host[at:at + k]
            at += k
        table = table.to(DEV)
    else:
        shape, table = (B, s), None
    if case["fp8"]:
        x = torch.randn(shape + (D_QK,), generator=g, device=DEV, dtype=torch.bfloat16)
        latent = (x * 64).clamp(-448, 448).to(torch.float8_e4m3fn)
        del x
        latent_scale = torch.empty(shape + (TILES,), device=DEV).uniform_(1 / 128, 1 / 32, generator=g)
    else:
        latent = torch.randn(shape + (D_QK,), generator=g, device=DEV, dtype=torch.bfloat16)
        latent_scale = None
    q = (torch.randn((B * T, H, D_QK), generator=g, device=DEV) * 1.5).to(torch.bfloat16)
    st = dict(case=case, q=q, latent=latent, latent_scale=latent_scale, table=table,
              seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV), longest=max(lens),
              out=torch.empty((B * T, H, D_LATENT), dtype=torch.bfloat16, device=DEV),
              lse=torch.empty((B * T, H), device=DEV))
    if own:
        from indexed_sparse_attention_indexer_gb300 import binding
        st["cache"] = binding.Cache(None, latent, st["seq_lens"], block_table=table, page_size=page,
                                    latent_scale=latent_scale)
        st["workspace"] = binding.alloc_workspace(binding.dense_mla_workspace_size(B * T, H), DEV)
    return st


# ----------------------------------------------------------------------------- one pass

def run(st):
    case = st["case"]
    if case["op"] == "rope":
        if own:
            _own_rope(st)
        else:
            _plain_rope(st)
        return {"q": st["q_out"], "cache": st["cache"], "scales": st["scales"]}
    if own:
        return _own_attention(st)
    return _plain_attention(st)


def _own_rope(st):
    from indexed_sparse_attention_indexer_gb300 import binding
    case = st["case"]
    binding.norm_rope(st["q_side"], st["k_side"], st["table"], st["positions"],
                      rope_offset=case["rope_offset"], interleaved=case["interleaved"], eps=EPS)


def _own_attention(st):
    from indexed_sparse_attention_indexer_gb300 import binding
    case = st["case"]
    kw = dict(out=st["out"], lse=st["lse"], workspace=st["workspace"])
    if case["op"] == "dense":
        return binding.dense_mla_decode(st["q"], st["cache"], SCALE, tokens_per_seq=case["tokens"], **kw)
    if case["prefill"]:
        return binding.window_mla_prefill(st["q"], st["cache"], case["s"] - case["tokens"],
                                          case["window"], case["sink"], SCALE, **kw)
    return binding.window_mla_decode(st["q"], st["cache"], case["window"], case["sink"], SCALE,
                                     tokens_per_seq=case["tokens"], **kw)


def _plain_heads(x, kind, w, b, st):
    case = st["case"]
    nd, ro, rd = case["norm_dim"], case["rope_offset"], case["rope_dim"]
    y = x.float()
    if kind != "none":
        v = y[..., :nd]
        if kind == "layer":
            v = v - v.mean(-1, keepdim=True)
        v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * w
        if kind == "layer":
            v = v + b
        y = torch.cat([v, y[..., nd:]], dim=-1)
    cs = st["table"][st["positions"]][:, None, :]
    c, s = cs[..., :rd // 2], cs[..., rd // 2:]
    r = y[..., ro:ro + rd]
    if case["interleaved"]:
        a, b2 = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b2 * s, a * s + b2 * c], dim=-1).flatten(-2)
    else:
        a, b2 = r[..., :rd // 2], r[..., rd // 2:]
        r = torch.cat([a * c - b2 * s, a * s + b2 * c], dim=-1)
    return torch.cat([y[..., :ro], r, y[..., ro + rd:]], dim=-1)


def _plain_rope(st):
    case = st["case"]
    if case["hq"]:
        st["q_out"].copy_(_plain_heads(st["q"], case["norm_q"], st["qw"], st["qb"], st))
    z = _plain_heads(st["k"], case["norm_k"], st["kw"], st["kb"], st)
    rows, d = st["rows"], case["d"]
    if case["k_out"] == "bf16":
        st["cache"][rows] = z.to(torch.bfloat16)
        return
    codes = st["cache"].view(torch.uint8)
    if case["k_out"] == "mxfp8":
        v = z.unflatten(-1, (d // 32, 32))
        big = v.abs().amax(-1)
        e = (torch.frexp(big).exponent - 1 - 8).clamp(-127, 127)
        e = torch.where(big > 0, e, torch.full_like(e, -127))
        v = torch.ldexp(v, -e[..., None]).clamp(-448, 448).flatten(-2)
        st["scales"][rows] = (e + 127).to(torch.uint8)
    else:
        tiles = (d + 127) // 128
        pad = torch.nn.functional.pad(z, (0, tiles * 128 - d)).unflatten(-1, (tiles, 128))
        sc = pad.abs().amax(-1) / 448
        v = torch.where(sc[..., None] > 0, pad / sc[..., None], torch.zeros_like(pad))
        v = v.clamp(-448, 448).flatten(-2)[..., :d]
        st["scales"][rows] = sc
    codes[rows] = v.to(torch.float8_e4m3fn).view(torch.uint8)


def _cache_rows(st, pos, seq):
    """Latent rows [*pos.shape, 576] at positions pos of sequences seq (same shapes)."""
    case = st["case"]
    if st["table"] is not None:
        page = case["page"]
        at = st["table"][seq, pos // page].long().clamp(min=0) * page + pos % page
    else:
        at = seq * case["s"] + pos
    c = st["latent"].view(torch.uint8 if case["fp8"] else torch.bfloat16).view(-1, D_QK)[at]
    if not case["fp8"]:
        return c.float()
    # an FP8 row takes part as code * tile scale rounded to bf16
    sc = st["latent_scale"].view(-1, TILES)[at]
    sc = sc.repeat_interleave(128, dim=-1)[..., :D_QK]
    return (c.view(torch.float8_e4m3fn).float() * sc).to(torch.bfloat16).float()


def _visible(st):
    """Visible length and sequence of every query row."""
    case = st["case"]
    T, B = case["tokens"], case["batch"]
    if case.get("prefill"):
        n = torch.arange(case["s"] - T + 1, case["s"] + 1, device=DEV)
        return n, torch.zeros_like(n)
    t = torch.arange(T, device=DEV)
    n = (st["seq_lens"].long()[:, None] - (T - 1 - t)[None, :]).clamp(min=0).flatten()
    return n, torch.arange(B, device=DEV).repeat_interleave(T)


def _softmax_rows(logits, ok, values):
    """Attention of logits [R, H, S] where ok [R, 1, S] over values [R, S, 512]."""
    logits = logits.masked_fill(~ok, -math.inf)
    top = logits.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(logits - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, values) / torch.where(total > 0, total, torch.ones_like(total))
    return out, (top + torch.log(total)).squeeze(-1)


def _plain_attention(st):
    case = st["case"]
    B, T, H = case["batch"], case["tokens"], case["heads"]
    n, seq = _visible(st)
    if case["op"] == "dense":
        # the T tokens of a sequence read its rows together
        S = max(1, st["longest"])
        pos = torch.arange(S, device=DEV).expand(B, S)
        c = _cache_rows(st, pos, torch.arange(B, device=DEV)[:, None].expand(B, S))
        q = st["q"].float().view(B, T * H, D_QK)
        ok = (torch.arange(S, device=DEV)[None, None, :] < n.view(B, T, 1)).repeat_interleave(H, dim=1)
    else:
        # every token reads its own window, and the sinks before it
        W, ns = case["window"], case["sink"]
        w = n[:, None] - W + torch.arange(W, device=DEV)
        k = torch.arange(ns, device=DEV).expand(n.numel(), ns)
        pos = torch.cat([k, w], dim=1)
        ok = torch.cat([(k < n[:, None] - W), (w >= 0)], dim=1)
        pos = torch.where(ok, pos, torch.zeros_like(pos))
        c = _cache_rows(st, pos, seq[:, None].expand_as(pos))
        q, ok = st["q"].float(), ok[:, None, :]
    out, lse = _softmax_rows(torch.matmul(q, c.transpose(1, 2)) * SCALE, ok, c[..., :D_LATENT])
    st["out"].copy_(out.view(B * T, H, D_LATENT))
    st["lse"].copy_(lse.view(B * T, H))
    return st["out"], st["lse"]


# ----------------------------------------------------------------------------- counts

def _seen(case, n):
    """Positions that a row of visible length n attends to."""
    if case["op"] == "dense":
        return n
    return min(n, case["window"]) + max(0, min(case["sink"], n - case["window"]))


def work(case):
    if case["op"] == "rope":
        n, d, hk = case["rows"], case["d"], case["hk"]
        vectors = n * (case["hq"] + hk)
        out = {"bf16": 2 * d, "mxfp8": d + d // 32, "fp8": d + 4 * ((d + 127) // 128)}[case["k_out"]]
        return {"bytes": vectors * 2 * d + n * case["hq"] * 2 * d + n * hk * out
                + n * (4 * case["rope_dim"] + 8 + 8), "flops": vectors * d * 6}
    T, H = case["tokens"], case["heads"]
    row = D_QK + 4 * TILES if case["fp8"] else 2 * D_QK
    if case.get("prefill"):
        q0 = case["s"] - T
        pairs = sum(_seen(case, q0 + t + 1) for t in range(T))
        lo = max(0, q0 + 1 - case["window"])
        rows = case["s"] - lo + min(case["sink"], lo)
    else:
        pairs = rows = 0
        for n in _lengths(case):
            seen = [_seen(case, max(0, n - t)) for t in range(T)]
            pairs += sum(seen)
            if case["op"] == "dense":
                rows += n
            else:
                lo = max(0, n - (T - 1) - case["window"])
                rows += n - lo + min(case["sink"], lo)
    R = case["batch"] * T
    return {"bytes": rows * row + R * H * (2 * D_QK + 2 * D_LATENT + 4),
            "flops": 2 * pairs * H * (D_QK + D_LATENT)}


# ----------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return _exact_rope(st) if case["op"] == "rope" else _exact_attention(st)


def _exact_side(x, kind, w, b, st):
    case = st["case"]
    nd, ro, rd = case["norm_dim"], case["rope_offset"], case["rope_dim"]
    z = x.double().clone()
    if kind == "rms":
        power = z[..., :nd].pow(2).sum(-1) / nd
        z[..., :nd] = z[..., :nd] / (power + EPS).sqrt().unsqueeze(-1) * w.double()
    elif kind == "layer":
        m = z[..., :nd].sum(-1, keepdim=True) / nd
        var = (z[..., :nd] - m).pow(2).sum(-1, keepdim=True) / nd
        z[..., :nd] = (z[..., :nd] - m) / (var + EPS).sqrt() * w.double() + b.double()
    half = torch.arange(rd // 2, device=DEV)
    ia, ib = (ro + 2 * half, ro + 2 * half + 1) if case["interleaved"] else (ro + half, ro + half + rd // 2)
    turn = torch.complex(st["table"][:, :rd // 2].double(), st["table"][:, rd // 2:].double())
    turned = torch.complex(z[..., ia], z[..., ib]) * turn[st["positions"]].unsqueeze(1)
    z[..., ia], z[..., ib] = turned.real, turned.imag
    return z


def _exact_rope(st):
    case = st["case"]
    q = _exact_side(st["q"], case["norm_q"], st["qw"], st["qb"], st)
    z = _exact_side(st["k"], case["norm_k"], st["kw"], st["kb"], st)
    d, scales = case["d"], None
    if case["k_out"] == "mxfp8":
        v = z.unflatten(-1, (d // 32, 32))
        e = torch.floor(torch.log2(v.abs().amax(-1, keepdim=True))) - 8
        z = (v * torch.pow(2.0, -e)).clamp(-448, 448).flatten(-2).float().to(torch.float8_e4m3fn).double()
    elif case["k_out"] == "fp8":
        scales = torch.zeros(st["scales"].shape, device=DEV, dtype=torch.float64)
        parts, sc = [], []
        for at in range(0, d, 128):
            v = z[..., at:at + 128]
            sc.append(v.abs().amax(-1) / 448)
            parts.append(v / sc[-1].unsqueeze(-1))
        z = torch.cat(parts, dim=-1).float().to(torch.float8_e4m3fn).double()
        scales[st["rows"]] = torch.stack(sc, dim=-1)
    cache = torch.zeros(st["cache"].shape, device=DEV, dtype=torch.float64)
    cache[st["rows"]] = z
    return {"q": q, "cache": cache, "scales": scales}


def _exact_attention(st):
    case = st["case"]
    T, H, R = case["tokens"], case["heads"], case["batch"] * case["tokens"]
    out = torch.zeros((R, H, D_LATENT), device=DEV, dtype=torch.float64)
    lse = torch.full((R, H), -math.inf, device=DEV, dtype=torch.float64)
    lens = _lengths(case)
    step = 64 if case.get("prefill") else 1         # query rows that are taken together
    for r0 in range(0, R, step):
        r1 = min(R, r0 + step)
        if case.get("prefill"):
            b, see = 0, [case["s"] - T + 1 + r for r in range(r0, r1)]
        else:
            b, see = r0 // T, [max(0, lens[r0 // T] - (T - 1 - r0 % T))]
        if max(see) == 0:
            continue
        W = case.get("window", case["s"] + 1)
        lo = max(0, min(see) - W)
        spots = torch.cat([torch.arange(min(case.get("sink", 0), lo), device=DEV),
                           torch.arange(lo, max(see), device=DEV)])
        if case["page"]:
            at = st["table"][b].long()[spots // case["page"]] * case["page"] + spots % case["page"]
        else:
            at = spots + b * case["s"]
        c = st["latent"].flatten(0, 1).view(torch.uint8 if case["fp8"] else torch.bfloat16)[at]
        if case["fp8"]:
            c = c.view(torch.float8_e4m3fn).double()
            for t in range(TILES):
                c[:, 128 * t:128 * t + 128] *= st["latent_scale"].flatten(0, 1)[at, t].double()[:, None]
            c = c.to(torch.bfloat16)
        c = c.double()
        n = torch.tensor(see, device=DEV)[:, None, None]
        ok = (spots < n) & ((spots >= n - W) | (spots < case.get("sink", 0)))
        logits = torch.where(ok, torch.einsum("rhd,sd->rhs", st["q"][r0:r1].double(), c) / math.sqrt(D_QK),
                             -math.inf)
        lse[r0:r1] = torch.logsumexp(logits, dim=-1)
        out[r0:r1] = torch.einsum("rhs,sd->rhd", torch.softmax(logits, dim=-1), c[:, :D_LATENT])
    return out, lse
