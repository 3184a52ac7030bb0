"""Host checks of the linear attention calls: refusals before any launch, and the struct's layout."""
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


def test_struct_layout(tmp_path):
    prog = tmp_path / "layout.c"
    prog.write_text(
        '#include <stdio.h>\n#include <stddef.h>\n#include "dsi.h"\n'
        'int main(void){ printf("size %zu\\n", sizeof(dsi_linear));'
        + "".join(f'printf("{f} %zu\\n", offsetof(dsi_linear, {f}));'
                  for f, _ in binding.DsiLinear._fields_) + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)], check=True)
    got = dict(x.split() for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                                 check=True).stdout.splitlines())
    assert int(got["size"]) == ctypes.sizeof(binding.DsiLinear)
    for f, _ in binding.DsiLinear._fields_:
        assert int(got[f]) == getattr(binding.DsiLinear, f).offset, f


def _args(**kw):
    a = binding.DsiLinear()
    a.q, a.k, a.v, a.out = FAKE, FAKE + 4096, FAKE + 8192, FAKE + 65536
    a.ld_q_row = a.ld_k_row = a.ld_v_row = a.ld_out_row = 512
    a.ld_q_head = a.ld_k_head = a.ld_v_head = a.ld_out_head = 128
    a.n_heads, a.n_kv_heads, a.dk, a.dv = 4, 4, 128, 128
    a.log_decay, a.scale, a.state, a.n_slots = FAKE, 1.0, FAKE, 8
    a.in_slots, a.out_slots = FAKE, FAKE
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BAD = [dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(log_decay=None), dict(q=FAKE + 2),
       dict(k=FAKE + 8), dict(v=FAKE + 4), dict(out=FAKE + 65544), dict(out=FAKE), dict(out=FAKE + 4096),
       dict(out=FAKE + 8192), dict(ld_q_row=120), dict(ld_k_row=516), dict(ld_v_head=64), dict(ld_out_row=513),
       dict(ld_out_head=0), dict(n_heads=0), dict(n_kv_heads=0), dict(n_kv_heads=3), dict(n_heads=-4),
       dict(scale=float("nan")), dict(state=FAKE + 8), dict(n_slots=-1), dict(state=None), dict(in_slots=FAKE + 2),
       dict(out_slots=FAKE + 1), dict(log_decay=FAKE + 2), dict(in_slots=None, n_slots=2)]


def test_refusals(L):
    step = lambda a, B=3, T=1: L.dsi_linear_decode(ctypes.byref(a) if a else None, B, T, None)       # noqa: E731
    full = lambda a, n=9, B=3, starts=FAKE, ws=None, size=0: L.dsi_linear_prefill(                    # noqa: E731
        ctypes.byref(a) if a else None, n, starts, B, ws, size, None)
    for bad in BAD:
        assert step(_args(**bad)) == E, bad
        assert full(_args(**bad)) == E, bad
    for bad in (dict(dk=0), dict(dk=12), dict(dk=136), dict(dv=0), dict(dv=20), dict(dv=256), dict(dk=-8)):
        assert step(_args(**bad)) == U and full(_args(**bad)) == U, bad
    assert step(None) == E and full(None) == E
    assert step(_args(), B=-1) == E and step(_args(), T=0) == E and step(_args(), T=-2) == E
    assert full(_args(), n=-1) == E and full(_args(), B=-1) == E
    assert full(_args(), starts=None) == E and full(_args(), starts=FAKE + 2) == E
    assert full(_args(), n=1 << 31) == U and step(_args(), B=1 << 30) == U
    assert step(_args(n_slots=1 << 30), B=1 << 16, T=1 << 15) == U
    assert full(_args(), ws=FAKE + 64, size=1 << 30) == E
    need = L.dsi_linear_workspace_size(9, 3, 4, 128, 128)
    assert need >= 256 and full(_args(), ws=FAKE, size=need - 1) == binding.DSI_ERR_WORKSPACE
    # nothing to launch
    assert step(_args(), B=0) == OK and full(_args(), B=0) == OK and full(_args(q=None, k=None), n=0, B=0) == OK
    assert L.dsi_linear_workspace_size(0, 3, 4, 128, 128) == 256
    assert L.dsi_linear_workspace_size(9, -1, 4, 128, 128) == 256


def test_binding_checks(L):
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)                                          # noqa: E731
    q, k, v, dec = z(6, 4, 64), z(6, 2, 64), z(6, 2, 32), z(4, t=torch.float32)
    st, starts, slots = z(5, 4, 64, 32, t=torch.float32), z(4, t=torch.int32), z(3, t=torch.int32)
    bad = [dict(q=q.float()), dict(q=z(6, 256)), dict(k=z(5, 2, 64)), dict(k=z(6, 2, 32)), dict(v=z(6, 4, 32)),
           dict(log_decay=z(4)), dict(log_decay=z(3, t=torch.float32)), dict(state=z(5, 4, 32, 64, t=torch.float32)),
           dict(state=z(5, 4, 64, 32)), dict(state=st.transpose(0, 1)), dict(in_slots=z(3, t=torch.int64)),
           dict(in_slots=z(2, t=torch.int32)), dict(state=None), dict(out=z(6, 2, 32)), dict(out=z(6, 4, 32, t=torch.float32)),
           dict(out=z(6, 32, 4).transpose(1, 2)), dict(q=z(6, 64, 4).transpose(1, 2))]
    for kw in bad:
        args = dict(q=q, k=k, v=v, log_decay=dec, scale=1.0, state=st, in_slots=slots, out_slots=slots) | kw
        with pytest.raises(ValueError):
            binding.linear_decode(tokens_per_seq=2, **args)
        with pytest.raises(ValueError):
            binding.linear_prefill(seq_starts=starts, **args)
    args = dict(q=q, k=k, v=v, log_decay=dec, scale=1.0)
    for T in (0, -1, 4):
        with pytest.raises(ValueError):
            binding.linear_decode(tokens_per_seq=T, **args)
    for s in (starts.long(), z(2, 2, t=torch.int32), z(8, t=torch.int32)[::2], z(0, t=torch.int32)):
        with pytest.raises(ValueError):
            binding.linear_prefill(seq_starts=s, **args)
    # nothing to launch
    none = dict(q=q[:0], k=k[:0], v=v[:0], log_decay=dec, scale=1.0)
    assert binding.linear_decode(**none).shape == (0, 4, 32)
    assert binding.linear_prefill(seq_starts=starts[:1], **none).shape == (0, 4, 32)
