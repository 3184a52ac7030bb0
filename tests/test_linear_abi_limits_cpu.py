"""Host checks of the linear attention calls: pitches that the copies' maps cannot hold, tokens past what is counted."""
import ctypes

import pytest

from indexed_sparse_attention_indexer_gb300 import binding
from tests.test_linear_abi_cpu import FAKE, L, _args  # noqa: F401


@pytest.mark.parametrize("name", [f"ld_{x}_{y}" for x in "qkv" for y in ("row", "head")])
def test_wide_pitches_are_refused(L, name):                                       # noqa: F811
    """Before anything is launched: a prefill of several sequences launches its short ones first."""
    for heads in (1, 4):
        a = _args(n_heads=heads, n_kv_heads=heads, **{name: 1 << 39})
        assert L.dsi_linear_prefill(ctypes.byref(a), 309, FAKE, 3, None, 0, None) == binding.DSI_ERR_UNSUPPORTED
        assert L.dsi_linear_prefill(ctypes.byref(a), 309, FAKE, 0, None, 0, None) == binding.DSI_ERR_UNSUPPORTED
        a = _args(q=None, k=None, v=None, out=None, **{name: 1 << 39})            # nothing to read
        assert L.dsi_linear_prefill(ctypes.byref(a), 0, FAKE, 0, None, 0, None) == binding.DSI_OK


def test_token_counts_that_leave_no_room_are_refused(L):                          # noqa: F811
    """Chunks and groups of tokens are counted in 32 bits past the last token."""
    a = _args(n_heads=1, n_kv_heads=1, n_slots=1 << 20)
    U = binding.DSI_ERR_UNSUPPORTED
    for n in ((1 << 31) - 1, (1 << 31) - 100, (1 << 31) - 1023):
        assert L.dsi_linear_prefill(ctypes.byref(a), n, FAKE, 0, None, 0, None) == U
    assert L.dsi_linear_prefill(ctypes.byref(a), (1 << 31) - 1024, FAKE, 0, None, 0, None) == binding.DSI_OK
    for B, T in ((1, (1 << 31) - 1), (1, (1 << 31) - 3), (3, 715827882)):
        assert L.dsi_linear_decode(ctypes.byref(a), B, T, None) == U
