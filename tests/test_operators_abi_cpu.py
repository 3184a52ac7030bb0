"""Host checks of the cache-side operators (head norms with rotation, attention over the whole
latent cache or a window of it): refusals before any launch, and the structs' layout."""
import ctypes
import os
import subprocess

import pytest
import torch

from indexed_sparse_attention_indexer_gb300 import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20   # an aligned, never dereferenced stand-in for a device pointer
E, U, OK = binding.DSI_ERR_INVALID_ARG, binding.DSI_ERR_UNSUPPORTED, binding.DSI_OK


@pytest.fixture(scope="module", params=[False, True], ids=["release", "checked"])
def L(request):
    if not os.path.exists(binding.lib_path(request.param)):
        pytest.skip("library not built (run __graft_entry__.build())")
    return binding.load(request.param)


def test_heads_struct_layout(tmp_path):
    prog = tmp_path / "layout.c"
    prog.write_text(
        '#include <stdio.h>\n#include <stddef.h>\n#include "dsi.h"\n'
        'int main(void){ printf("size %zu\\n", sizeof(dsi_heads));'
        + "".join(f'printf("{f} %zu\\n", offsetof(dsi_heads, {f}));'
                  for f, _ in binding.DsiHeads._fields_) + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)], check=True)
    got = dict(x.split() for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                                 check=True).stdout.splitlines())
    assert int(got["size"]) == ctypes.sizeof(binding.DsiHeads)
    for f, _ in binding.DsiHeads._fields_:
        assert int(got[f]) == getattr(binding.DsiHeads, f).offset, f


def _heads(**kw):
    h = binding.DsiHeads()
    h.x, h.ld_row, h.ld_head, h.n_heads, h.norm, h.norm_dim = FAKE, 512, 128, 4, 1, 128
    h.out_dtype, h.weight, h.bias, h.out = 0, FAKE, None, FAKE
    h.ld_out_row, h.ld_out_head, h.out_scale, h.dst_rows = 512, 128, None, None
    h.out_rows, h.out_group = 100, 0
    for k, v in kw.items():
        setattr(h, k, v)
    return h


def _rope(L, q, k=None, n=7, d=128, eps=1e-6, table=FAKE, rows=64, pos=FAKE, off=0, rd=64, il=0):
    return L.dsi_norm_rope(ctypes.byref(q) if q is not None else None,
                           ctypes.byref(k) if k is not None else None, n, d, eps, table, rows, pos,
                           off, rd, il, None)


def test_norm_rope_refusals(L):
    for bad in (dict(x=None), dict(out=None), dict(x=FAKE + 2), dict(out=FAKE + 8), dict(weight=FAKE + 4),
                dict(n_heads=-1), dict(ld_row=100), dict(ld_row=516), dict(ld_head=120), dict(ld_head=132),
                dict(ld_out_row=516), dict(ld_out_head=64), dict(bias=FAKE),        # bias without LAYER
                dict(out_rows=6), dict(out_rows=-1),
                dict(out_dtype=2), dict(out_dtype=1), dict(out_dtype=1, out_scale=FAKE + 2)):
        assert _rope(L, _heads(**bad)) == E, bad
        assert _rope(L, None, _heads(**bad)) == E, bad
        assert _rope(L, _heads(n_heads=0), _heads(**bad)) == E, bad
    for bad in (dict(norm=3), dict(norm_dim=4), dict(norm_dim=0), dict(norm_dim=136), dict(norm_dim=60),
                dict(out_dtype=7, out_scale=FAKE), dict(out_dtype=2, out_scale=FAKE, out_group=48)):
        assert _rope(L, _heads(**bad)) == U, bad
    h = _heads()
    for bad in (dict(n=-1), dict(table=None), dict(pos=None), dict(rows=0), dict(eps=-1.0),
                dict(eps=float("nan")), dict(off=-8), dict(off=72), dict(rd=-16), dict(table=FAKE + 4)):
        assert _rope(L, h, **bad) == E, bad
    for bad in (dict(d=0), dict(d=130), dict(d=1032), dict(off=4), dict(rd=8), dict(rd=24), dict(rd=0)):
        assert _rope(L, h, **bad) == U, bad
    wide = _heads(ld_row=4096, ld_head=576, ld_out_row=4096, ld_out_head=576, norm_dim=512,
                  out_dtype=2, out_scale=FAKE, out_group=128)
    assert _rope(L, wide, d=576) == U                      # the group does not divide d
    assert _rope(L, h, n=0) == OK                           # nothing to launch
    assert _rope(L, None, None) == OK
    assert _rope(L, _heads(n_heads=0, x=None), None) == OK


def test_heads_checks():
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    H = binding.Heads
    for kw in (dict(norm="batch"), dict(weight=torch.ones(32)), dict(weight=torch.ones(64).bfloat16()),
               dict(dst_rows=torch.zeros(3, dtype=torch.int32)), dict(dst_rows=torch.zeros(2, dtype=torch.int64)),
               dict(out=torch.zeros((3, 2, 32), dtype=torch.bfloat16)),
               dict(out=torch.zeros((3, 3, 64), dtype=torch.bfloat16)),
               dict(out=torch.zeros((3, 2, 64))),
               dict(out=torch.zeros((3, 2, 64), dtype=torch.bfloat16), out_scale=torch.zeros((3, 2, 1))),
               dict(out=torch.zeros((3, 2, 64), dtype=torch.float8_e4m3fn)),
               dict(out=torch.zeros((3, 2, 64), dtype=torch.float8_e4m3fn), out_scale=torch.zeros((3, 2, 2))),
               dict(out=torch.zeros((3, 2, 64), dtype=torch.float8_e4m3fn),
                    out_scale=torch.zeros((2, 2, 2), dtype=torch.uint8))):
        with pytest.raises(ValueError):
            H(x, **kw)
    with pytest.raises(ValueError):
        H(x.float())
    with pytest.raises(ValueError):
        H(torch.zeros((3, 64, 2), dtype=torch.bfloat16).transpose(1, 2))
    a = H(x)
    assert a.out.shape == x.shape and a.struct.out_rows == 3 and a.struct.ld_row == 128
    # a page pool stands for its rows
    b = H(x[:, :1], out=torch.zeros((5, 16, 64), dtype=torch.bfloat16))
    assert b.struct.out_rows == 80 and b.struct.ld_out_row == 64


def test_norm_rope_binding_checks(L):
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    h, table, pos = binding.Heads(x), torch.zeros((9, 64)), torch.zeros(3, dtype=torch.int64)
    other = binding.Heads(torch.zeros((4, 2, 64), dtype=torch.bfloat16))
    for args in ((None, None, table, pos), (h, other, table, pos), (h, None, table.double(), pos),
                 (h, None, table.t(), pos), (h, None, table, pos.int()), (h, None, table, pos[:2])):
        with pytest.raises(ValueError):
            binding.norm_rope(*args)
    # no rows: nothing is launched
    empty = binding.Heads(torch.zeros((0, 2, 64), dtype=torch.bfloat16))
    assert binding.norm_rope(empty, None, table, pos[:0])[0].shape == (0, 2, 64)


def test_rope_table():
    t = binding.rope_table(70000, 64, device="cpu")
    assert t.shape == (70000, 64) and t.dtype == torch.float32
    a = torch.tensor(69999.0, dtype=torch.float64) * 10000.0 ** (-2.0 * 5 / 64)
    assert abs(float(t[69999, 5]) - float(a.cos())) < 1e-6 and abs(float(t[69999, 37]) - float(a.sin())) < 1e-6


def _cache(**kw):
    c = binding.DsiCache()
    c.k_idx, c.latent, c.seq_lens, c.batch, c.s_max = None, FAKE, FAKE, 4, 1024
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _dense(L, c, q=FAKE, T=1, H=128, scale=0.04, out=FAKE, lse=None, ws=None, wsb=0):
    return L.dsi_dense_mla_decode(q, ctypes.byref(c) if c is not None else None, T, H, scale, out, lse, ws, wsb, None)


def test_dense_and_window_refusals(L):
    need = L.dsi_dense_mla_workspace_size(4, 128)
    assert need >= 256 and L.dsi_dense_mla_workspace_size(0, 128) == 256
    calls = [
        lambda c, window=100, sink=4, T=1, off=0, **kw: _dense(L, c, T=T, **kw),
        lambda c, window=100, sink=4, T=1, off=0, q=FAKE, H=128, scale=0.04, out=FAKE, lse=None, ws=None, wsb=0:
            L.dsi_window_mla_decode(q, ctypes.byref(c) if c is not None else None, T, H, window, sink, scale,
                                    out, lse, ws, wsb, None),
        lambda c, window=100, sink=4, T=1, off=0, q=FAKE, H=128, scale=0.04, out=FAKE, lse=None, ws=None, wsb=0:
            L.dsi_window_mla_prefill(q, ctypes.byref(c) if c is not None else None, T, H, off, window, sink,
                                     scale, out, lse, ws, wsb, None),
    ]
    for i, f in enumerate(calls):
        base = dict(batch=1) if i == 2 else {}
        mk = lambda **kw: _cache(**dict(base, **kw))
        assert f(None) == E
        for kw in (dict(q=None), dict(out=None), dict(q=FAKE + 8), dict(out=FAKE + 2), dict(lse=FAKE + 2),
                   dict(scale=float("nan")), dict(ws=FAKE + 16, wsb=need), dict(T=-1)):
            assert f(mk(), **kw) == E, (i, kw)
        for kw in (dict(H=0), dict(H=129), dict(H=-1)):
            assert f(mk(), **kw) == U, (i, kw)
        assert f(mk(), ws=FAKE, wsb=need - 1) == binding.DSI_ERR_WORKSPACE
        for kw in (dict(latent=None), dict(latent=FAKE + 8), dict(batch=-1), dict(s_max=0),
                   dict(latent_dtype=1), dict(latent_dtype=1, latent_scale=FAKE + 2),
                   dict(block_table=FAKE, page_size=0, max_pages=16, num_pages=9),
                   dict(block_table=FAKE, page_size=64, max_pages=15, num_pages=9)):
            assert f(mk(**kw)) == E, (i, kw)
        for kw in (dict(latent_dtype=2), dict(s_max=1 << 31),
                   dict(block_table=FAKE, page_size=12, max_pages=1, s_max=12, num_pages=9),
                   dict(block_table=FAKE, page_size=64, max_pages=16, num_pages=1 << 25)):
            assert f(mk(**kw)) == U, (i, kw)
    dec, pre = calls[1], calls[2]
    assert _dense(L, _cache(), T=0) == E and _dense(L, _cache(seq_lens=None)) == E
    assert _dense(L, _cache(batch=1 << 30), T=4) == U                # 2^32 query rows
    assert _dense(L, _cache(batch=1 << 21, s_max=1 << 10)) == U       # 2^31 cache rows
    for f in (dec, pre):
        c = _cache(batch=1)
        assert f(c, window=0) == E and f(c, window=-5) == E and f(c, sink=-1) == E
    assert pre(_cache(batch=2)) == E and pre(_cache(batch=1), off=-1) == E
    assert pre(_cache(batch=1), T=8, off=1020) == E                   # beyond s_max
    assert _dense(L, _cache(batch=0)) == OK and pre(_cache(batch=1), T=0) == OK


def test_dense_binding_checks(L):
    lat = torch.zeros((2, 64, 576), dtype=torch.bfloat16)
    cache = binding.Cache(None, lat, torch.zeros(2, dtype=torch.int32))
    q = torch.zeros((2, 8, 576), dtype=torch.bfloat16)
    for bad in (q.float(), q[:, :, :512], q.transpose(0, 1), q[:1]):
        with pytest.raises(ValueError):
            binding.dense_mla_decode(bad, cache, 0.04)
        with pytest.raises(ValueError):
            binding.window_mla_decode(bad, cache, 10, 1, 0.04)
    for kw in (dict(out=torch.zeros((2, 8, 512))), dict(out=torch.zeros((2, 8, 576), dtype=torch.bfloat16)),
               dict(lse=torch.zeros((2, 7))), dict(lse=torch.zeros((2, 8), dtype=torch.float64)),
               dict(tokens_per_seq=2)):
        with pytest.raises(ValueError):
            binding.dense_mla_decode(q, cache, 0.04, **kw)
    with pytest.raises(ValueError):
        binding.dense_mla_decode(q, binding.Cache(torch.zeros((2, 64, 64), dtype=torch.bfloat16), None), 0.04)
    with pytest.raises(ValueError):
        binding.window_mla_prefill(q.float(), cache, 0, 10, 1, 0.04)


def test_prefill_offset_at_the_end_of_64_bits(L):
    """q_offset + T past 2^63 is past s_max like any other."""
    c = _cache(batch=1, k_idx=FAKE, d=128)
    for off in ((1 << 63) - 1, (1 << 63) - 8):
        assert L.dsi_window_mla_prefill(FAKE, ctypes.byref(c), 8, 16, off, 10, 1, 0.04, FAKE, None, None, 0, None) == E
        assert L.dsi_index_score(FAKE, FAKE, ctypes.byref(c), 8, 64, 0, off, FAKE, 1024, None) == E
        assert L.dsi_sparse_mla_prefill(FAKE, ctypes.byref(c), FAKE, 8, 16, 16, off, 0.04, FAKE, None, None, 0, None) == E


def test_largest_sizes_are_refused(L):
    """Past what 32-bit positions and block counts hold."""
    c = dict(block_table=FAKE, page_size=8, num_pages=100)
    for pages, st in ((1 << 28, U), ((1 << 28) - 127, U)):
        assert _dense(L, _cache(max_pages=pages, s_max=8 * pages, **c)) == st
    h = dict(dst_rows=FAKE)
    assert _rope(L, _heads(n_heads=1, **h), n=(1 << 31) + 1) == U
    assert _rope(L, _heads(n_heads=1 << 20, **h), n=(1 << 20) + 1) == U
    assert _rope(L, None, _heads(n_heads=(1 << 31) - 1, **h), n=1 << 31) == U


def test_dense_binding_checks_the_cache(L):
    """What the cache's struct would misread is refused before any launch."""
    bf, i32 = dict(dtype=torch.bfloat16), dict(dtype=torch.int32)
    q, lat, lens = torch.zeros((2, 8, 576), **bf), torch.zeros((2, 64, 576), **bf), torch.zeros(2, **i32)
    f8, sc = torch.zeros((2, 64, 576), dtype=torch.uint8).view(torch.float8_e4m3fn), torch.zeros((2, 64, 5))
    table = torch.zeros((2, 1), **i32)
    C = binding.Cache
    for cache in (C(None, lat.half(), lens), C(None, lat.float(), lens), C(None, torch.zeros((2, 64, 512), **bf), lens),
                  C(None, torch.zeros((2, 128, 576), **bf)[:, ::2], lens), C(None, lat, lens.long()), C(None, lat, lens[:1]),
                  C(None, lat, torch.zeros(4, **i32)[::2]), C(None, f8, lens), C(None, f8, lens, latent_scale=sc[:1]),
                  C(None, f8, lens, latent_scale=sc.double()), C(None, f8, lens, latent_scale=sc[..., :4]),
                  C(None, lat, lens, block_table=table.long(), page_size=64),
                  C(None, lat, lens, block_table=torch.zeros((2, 2), **i32)[:, ::2], page_size=64),
                  C(None, lat, lens, block_table=table, page_size=128),
                  C(torch.zeros((3, 64, 64), **bf), lat, torch.zeros(3, **i32), block_table=torch.zeros((3, 1), **i32), page_size=64),
                  C(None, lat, torch.zeros(2, device="meta", **i32))):
        with pytest.raises(ValueError):
            binding.dense_mla_decode(q, cache, 0.04)
    for good in (C(None, lat, lens), C(None, f8, lens, latent_scale=sc), C(None, lat, lens, block_table=table, page_size=64),
                 C(torch.zeros((2, 64, 64), **bf), lat, lens)):
        assert good.latent_fault() == ""
    for kw in (dict(window=1 << 63, n_sink=0), dict(window=5, n_sink=1 << 64), dict(window=-(1 << 63) - 1, n_sink=0)):
        with pytest.raises(ValueError):
            binding.window_mla_decode(q, C(None, lat, lens), scale=0.04, **kw)
    with pytest.raises(ValueError):
        binding.window_mla_prefill(q, C(None, lat[:1], None), 1 << 64, 5, 0, 0.04)


def test_norm_rope_binding_range(L):
    x, table, pos = torch.zeros((3, 2, 128), dtype=torch.bfloat16), torch.zeros((9, 64)), torch.zeros(3, dtype=torch.int64)
    for off in (1 << 32, -(1 << 32), 72, -8):
        with pytest.raises(ValueError):
            binding.norm_rope(binding.Heads(x), None, table, pos, rope_offset=off)
