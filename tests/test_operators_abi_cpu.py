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
