"""Host checks of dsi_norm_rope with x as out: vectors are copied ahead of those being written, so each
has to be written where it was read."""
import os

import pytest
import torch

from indexed_sparse_attention_indexer_gb300 import binding
from tests.test_operators_abi_cpu import FAKE, _heads, _rope

E = binding.DSI_ERR_INVALID_ARG


@pytest.fixture(scope="module", params=[False, True], ids=["release", "checked"])
def L(request):
    if not os.path.exists(binding.lib_path(request.param)):
        pytest.skip("library not built (run __graft_entry__.build())")
    return binding.load(request.param)


def test_in_place_refusals(L):
    for bad in (dict(dst_rows=FAKE), dict(ld_out_row=1024), dict(ld_row=1024), dict(ld_out_head=256),
                dict(out_dtype=binding.DSI_FP8_E4M3, out_scale=2 * FAKE),
                dict(out_dtype=binding.DSI_MXFP8_E4M3, out_scale=2 * FAKE)):
        assert _rope(L, _heads(**bad)) == E, bad
        assert _rope(L, None, _heads(**bad)) == E, bad
        assert _rope(L, _heads(out=2 * FAKE), _heads(**bad)) == E, bad
        assert _rope(L, _heads(**bad), n=0) == binding.DSI_OK          # nothing is written


def test_in_place_with_slots(L):
    """x as out and rows that change places, as the binding passes them on."""
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    h = binding.Heads(x, out=x, dst_rows=torch.tensor([1, 0, 3, 2]))
    assert h.struct.x == h.struct.out and _rope(L, h.struct, d=64, n=4) == E
