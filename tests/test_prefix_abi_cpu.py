"""Host checks of the shared-prefix attention call: refusals before any launch."""
import ctypes
import os

import pytest
import torch

from indexed_sparse_attention_indexer_gb300 import binding

FAKE = 1 << 20   # an aligned, never dereferenced stand-in for a device pointer
E, U, OK, W = (binding.DSI_ERR_INVALID_ARG, binding.DSI_ERR_UNSUPPORTED, binding.DSI_OK, binding.DSI_ERR_WORKSPACE)


@pytest.fixture(scope="module", params=[False, True], ids=["release", "checked"])
def L(request):
    if not os.path.exists(binding.lib_path(request.param)):
        pytest.skip("library not built (run __graft_entry__.build())")
    return binding.load(request.param)


def _cache(batch=4, **kw):
    c = binding.DsiCache()
    c.latent, c.seq_lens, c.batch, c.s_max = FAKE, FAKE, batch, 1024
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def test_refusals(L):
    need = L.dsi_prefix_mla_workspace_size(4, 128)
    assert need >= 256 and L.dsi_prefix_mla_workspace_size(0, 128) == 256 == L.dsi_prefix_mla_workspace_size(4, -1)
    ref = lambda c: ctypes.byref(c) if c is not None else None                                  # noqa: E731

    def call(prefix=None, cache=None, q=FAKE, T=1, H=128, scale=0.04, out=FAKE, lse=None, ws=FAKE, size=need, **kw):
        p = _cache(1) if prefix is None else prefix
        c = _cache() if cache is None else cache
        return L.dsi_prefix_mla_decode(q, None if p == 0 else ref(p), None if c == 0 else ref(c), T, H, scale, out,
                                       lse, ws, size, None)

    for kw in (dict(q=None), dict(out=None), dict(q=FAKE + 8), dict(out=FAKE + 2), dict(lse=FAKE + 2), dict(prefix=0),
               dict(cache=0), dict(scale=float("nan")), dict(ws=FAKE + 16), dict(T=0), dict(T=-1)):
        assert call(**kw) == E, kw
    for H in (0, 129, -1):
        assert call(H=H) == U
    assert call(ws=None, size=0) == W and call(size=need - 1) == W
    for n in (0, 2, -1):
        assert call(prefix=_cache(n)) == E
    for kw in (dict(latent=None), dict(latent=FAKE + 8), dict(s_max=0), dict(seq_lens=None), dict(latent_dtype=1),
               dict(latent_dtype=1, latent_scale=FAKE + 2), dict(block_table=FAKE, page_size=0, max_pages=16, num_pages=9),
               dict(block_table=FAKE, page_size=64, max_pages=15, num_pages=9)):
        assert call(prefix=_cache(1, **kw)) == E and call(cache=_cache(**kw)) == E, kw
    for kw in (dict(latent_dtype=2), dict(s_max=1 << 31), dict(block_table=FAKE, page_size=12, max_pages=1, s_max=12, num_pages=9),
               dict(block_table=FAKE, page_size=64, max_pages=16, num_pages=1 << 25), dict(latent_dtype=1, latent_scale=FAKE)):
        assert call(prefix=_cache(1, **kw)) == U and call(cache=_cache(**kw)) == U, kw
    assert call(cache=_cache(-1)) == E and call(cache=_cache(1 << 30), T=4) == U
    assert call(cache=_cache(1 << 21, s_max=1 << 10)) == U                # 2^31 cache rows
    assert call(cache=_cache(1 << 30, s_max=1), H=1) == U == call(cache=_cache(1 << 23, s_max=1), H=128)   # 2^30 outputs
    assert call(cache=_cache(0), ws=None, size=0) == OK


def test_binding_checks(L):
    bf, i32 = dict(dtype=torch.bfloat16), dict(dtype=torch.int32)
    own = binding.Cache(None, torch.zeros((2, 64, 576), **bf), torch.zeros(2, **i32))
    shared = binding.Cache(None, torch.zeros((1, 64, 576), **bf), torch.zeros(1, **i32))
    q = torch.zeros((2, 8, 576), **bf)
    for bad in (q.float(), q[:, :, :512], q.transpose(0, 1), q[:1]):
        with pytest.raises(ValueError):
            binding.prefix_mla_decode(bad, shared, own, 0.04)
    for kw in (dict(out=torch.zeros((2, 8, 512))), dict(lse=torch.zeros((2, 7))), dict(tokens_per_seq=2)):
        with pytest.raises(ValueError):
            binding.prefix_mla_decode(q, shared, own, 0.04, **kw)
    for kw in (dict(prefix=binding.Cache(None, torch.zeros((1, 64, 512), **bf), torch.zeros(1, **i32)), cache=own),
               dict(prefix=binding.Cache(None, torch.zeros((1, 64, 576), **bf), torch.zeros(1, dtype=torch.int64)), cache=own),
               dict(prefix=shared, cache=binding.Cache(None, torch.zeros((2, 64, 576)), torch.zeros(2, **i32)))):
        with pytest.raises(ValueError):
            binding.prefix_mla_decode(q, scale=0.04, **kw)
    # nothing to launch
    none = binding.Cache(None, torch.zeros((0, 64, 576), **bf), torch.zeros(0, **i32))
    assert binding.prefix_mla_decode(q[:0], shared, none, 0.04)[0].shape == (0, 8, 512)
