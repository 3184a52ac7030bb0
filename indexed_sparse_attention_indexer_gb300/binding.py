"""ctypes binding of libdsi (include/dsi.h): argument marshalling only.

Every function here hands device pointers of torch tensors to the C ABI and
allocates the outputs with torch; all computation happens in the library's
CUDA kernels.  A missing library raises ``RuntimeError`` — there is no CPU
fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIBS = {}

DSI_OK, DSI_ERR_INVALID_ARG, DSI_ERR_UNSUPPORTED, DSI_ERR_CUDA = 0, 1, 2, 3
DSI_ERR_TIMEOUT, DSI_ERR_BOUNDS, DSI_ERR_WORKSPACE = 4, 5, 6
DSI_BF16, DSI_FP8_E4M3, DSI_MXFP8_E4M3 = 0, 1, 2
NORMS = {None: 0, "rms": 1, "layer": 2}
D_QK, D_LATENT = 576, 512

c_void_p, c_int32, c_int64, c_float, c_size_t = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                                                 ctypes.c_float, ctypes.c_size_t)


class DsiCache(ctypes.Structure):
    """Mirror of ``struct dsi_cache``."""
    _fields_ = [("k_idx", c_void_p), ("k_dtype", c_int32), ("d", c_int32), ("k_scale", c_void_p),
                ("latent", c_void_p), ("block_table", c_void_p), ("page_size", c_int32),
                ("max_pages", c_int32), ("seq_lens", c_void_p), ("batch", c_int32),
                ("s_max", c_int64), ("num_pages", c_int64), ("k_group", c_int32),
                ("latent_dtype", c_int32), ("latent_scale", c_void_p)]


class DsiHeads(ctypes.Structure):
    """Mirror of ``struct dsi_heads``."""
    _fields_ = [("x", c_void_p), ("ld_row", c_int64), ("ld_head", c_int64), ("n_heads", c_int32),
                ("norm", c_int32), ("norm_dim", c_int32), ("out_dtype", c_int32),
                ("weight", c_void_p), ("bias", c_void_p), ("out", c_void_p),
                ("ld_out_row", c_int64), ("ld_out_head", c_int64), ("out_scale", c_void_p),
                ("dst_rows", c_void_p), ("out_rows", c_int64), ("out_group", c_int32)]


class DsiLinear(ctypes.Structure):
    """Mirror of ``struct dsi_linear``."""
    _fields_ = [("q", c_void_p), ("k", c_void_p), ("v", c_void_p), ("out", c_void_p),
                ("ld_q_row", c_int64), ("ld_q_head", c_int64), ("ld_k_row", c_int64),
                ("ld_k_head", c_int64), ("ld_v_row", c_int64), ("ld_v_head", c_int64),
                ("ld_out_row", c_int64), ("ld_out_head", c_int64), ("n_heads", c_int32),
                ("n_kv_heads", c_int32), ("dk", c_int32), ("dv", c_int32), ("log_decay", c_void_p),
                ("scale", c_float), ("state", c_void_p), ("n_slots", c_int64), ("in_slots", c_void_p),
                ("out_slots", c_void_p)]


# name -> (restype, argtypes); the exported surface of include/dsi.h
SIGNATURES = {
    "dsi_index_score": (c_int32, [c_void_p, c_void_p, ctypes.POINTER(DsiCache), c_int32, c_int32,
                                  c_int32, c_int64, c_void_p, c_int64, c_void_p]),
    "dsi_topk": (c_int32, [c_void_p, c_int64, c_int32, c_void_p, c_int64, c_int32, c_void_p,
                           c_void_p, c_void_p]),
    "dsi_index_topk_prefill": (c_int32, [c_void_p, c_void_p, ctypes.POINTER(DsiCache), c_int32,
                                         c_int32, c_int64, c_int32, c_void_p, c_void_p,
                                         c_void_p]),
    "dsi_sparse_mla_decode": (c_int32, [c_void_p, ctypes.POINTER(DsiCache), c_void_p, c_int32,
                                        c_int32, c_int32, c_float, c_void_p, c_void_p, c_void_p,
                                        c_size_t, c_void_p]),
    "dsi_sparse_mla_prefill": (c_int32, [c_void_p, ctypes.POINTER(DsiCache), c_void_p, c_int32,
                                         c_int32, c_int32, c_int64, c_float, c_void_p, c_void_p,
                                         c_void_p, c_size_t, c_void_p]),
    "dsi_indexed_attention": (c_int32, [c_void_p, c_void_p, c_void_p, ctypes.POINTER(DsiCache),
                                        c_int32, c_int32, c_int32, c_int32, c_int64, c_float,
                                        c_int32, c_void_p, c_void_p, c_void_p, c_void_p,
                                        c_void_p, c_size_t, c_void_p]),
    "dsi_indexed_attention_multi": (c_int32, [c_void_p, c_void_p, c_void_p, ctypes.POINTER(DsiCache),
                                              c_int32, c_int32, c_int32, c_int32, c_float, c_void_p,
                                              c_void_p, c_void_p, c_void_p, c_void_p, c_size_t,
                                              c_void_p]),
    "dsi_indexed_attention_static": (c_int32, [c_void_p, c_void_p, c_void_p,
                                               ctypes.POINTER(DsiCache), c_int32, c_int32,
                                               c_int32, c_int32, c_int64, c_float, c_int32,
                                               c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
    "dsi_mxfp8_quantize": (c_int32, [c_void_p, c_int64, c_int32, c_int64, c_int32, c_void_p,
                                     c_void_p, c_void_p, c_void_p]),
    "dsi_latent_fp8_append": (c_int32, [c_void_p, c_int64, c_int64, c_void_p, c_void_p, c_void_p,
                                        c_void_p]),
    "dsi_dense_mla_decode": (c_int32, [c_void_p, ctypes.POINTER(DsiCache), c_int32, c_int32,
                                       c_float, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "dsi_window_mla_decode": (c_int32, [c_void_p, ctypes.POINTER(DsiCache), c_int32, c_int32,
                                        c_int64, c_int64, c_float, c_void_p, c_void_p, c_void_p,
                                        c_size_t, c_void_p]),
    "dsi_window_mla_prefill": (c_int32, [c_void_p, ctypes.POINTER(DsiCache), c_int32, c_int32,
                                         c_int64, c_int64, c_int64, c_float, c_void_p, c_void_p,
                                         c_void_p, c_size_t, c_void_p]),
    "dsi_prefix_mla_decode": (c_int32, [c_void_p, ctypes.POINTER(DsiCache), ctypes.POINTER(DsiCache), c_int32,
                                        c_int32, c_float, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "dsi_prefix_mla_workspace_size": (c_size_t, [c_int32, c_int32]),
    "dsi_dense_mla_workspace_size": (c_size_t, [c_int32, c_int32]),
    "dsi_norm_rope": (c_int32, [ctypes.POINTER(DsiHeads), ctypes.POINTER(DsiHeads), c_int64,
                                c_int32, c_float, c_void_p, c_int64, c_void_p, c_int32, c_int32,
                                c_int32, c_void_p]),
    "dsi_linear_prefill": (c_int32, [ctypes.POINTER(DsiLinear), c_int64, c_void_p, c_int32, c_void_p,
                                     c_size_t, c_void_p]),
    "dsi_linear_decode": (c_int32, [ctypes.POINTER(DsiLinear), c_int32, c_int32, c_void_p]),
    "dsi_linear_workspace_size": (c_size_t, [c_int64, c_int32, c_int32, c_int32, c_int32]),
    "dsi_workspace_size": (c_size_t, [c_int32, c_int32, c_int32, c_int32, c_int64, c_int32]),
    "dsi_layer_workspace_size": (c_size_t, [ctypes.POINTER(DsiCache), c_int32, c_int32, c_int32,
                                            c_int32, c_int64, c_int32]),
    "dsi_get_device_status": (c_int32, [c_void_p]),
    "dsi_selftest_wait_timeout": (c_int32, [ctypes.c_uint64, c_void_p]),
    "dsi_status_string": (ctypes.c_char_p, [c_int32]),
    "dsi_version": (c_int32, []),
    "dsi_launch_count": (ctypes.c_uint64, []),
}


class DsiError(RuntimeError):
    def __init__(self, fn: str, status: int, lib=None):
        msg = lib.dsi_status_string(status).decode() if lib is not None else str(status)
        super().__init__(f"{fn} failed: {msg} (status {status})")
        self.status = status


def lib_path(checked: bool = False) -> str:
    return os.path.join(_PKG, "libdsi_checked.so" if checked else "libdsi.so")


def load(checked: bool = False):
    """Load (once) and return the library with typed entry points."""
    key = bool(checked)
    if key in _LIBS:
        return _LIBS[key]
    path = lib_path(checked)
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built: run __graft_entry__.build() (no CPU fallback)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _LIBS[key] = lib
    return lib


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _rows_contiguous(t: torch.Tensor, name: str):
    """The C ABI takes a row pitch: elements within a row must be contiguous."""
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be 2-D with contiguous rows")


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(lib, fn: str, status: int):
    if status != DSI_OK:
        raise DsiError(fn, status, lib)


class Cache:
    """Device tensors of one cache plus the ``dsi_cache`` struct that points at them."""

    def __init__(self, k_idx: Optional[torch.Tensor], latent: Optional[torch.Tensor],
                 seq_lens: Optional[torch.Tensor] = None, k_scale: Optional[torch.Tensor] = None,
                 block_table: Optional[torch.Tensor] = None, page_size: int = 0,
                 latent_scale: Optional[torch.Tensor] = None):
        self.k_idx, self.latent, self.seq_lens = k_idx, latent, seq_lens
        self.k_scale, self.block_table, self.page_size = k_scale, block_table, page_size
        self.latent_scale = latent_scale
        ref = k_idx if k_idx is not None else latent
        s = DsiCache()
        s.k_idx = k_idx.data_ptr() if k_idx is not None else None
        s.d = int(k_idx.shape[-1]) if k_idx is not None else 0
        s.k_dtype = DSI_BF16
        s.k_group = 0
        if k_idx is not None and k_idx.dtype == torch.float8_e4m3fn:
            # uint8 scales [.., d/G] are MXFP8 group scales; fp32 [..] per-position scales
            if k_scale is not None and k_scale.dtype == torch.uint8:
                s.k_dtype = DSI_MXFP8_E4M3
                s.k_group = s.d // int(k_scale.shape[-1])
            else:
                s.k_dtype = DSI_FP8_E4M3
        s.k_scale = k_scale.data_ptr() if k_scale is not None else None
        s.latent = latent.data_ptr() if latent is not None else None
        # an E4M3 latent cache is FP8 with per-tile scales
        s.latent_dtype = DSI_FP8_E4M3 if (latent is not None and latent.dtype == torch.float8_e4m3fn) else DSI_BF16
        s.latent_scale = latent_scale.data_ptr() if latent_scale is not None else None
        if block_table is not None:
            s.block_table = block_table.data_ptr()
            s.page_size = int(page_size)
            s.max_pages = int(block_table.shape[1])
            s.batch = int(block_table.shape[0])
            s.s_max = s.max_pages * s.page_size
            s.num_pages = int(ref.shape[0])
        else:
            s.block_table = None
            s.batch = int(ref.shape[0])
            s.s_max = int(ref.shape[1])
            s.num_pages = 0
        s.seq_lens = seq_lens.data_ptr() if seq_lens is not None else None
        self.struct = s
        self._fault: Optional[str] = None

    def latent_fault(self) -> str:
        """What keeps the dense and window calls from reading this cache as its struct says, or ""
        (looked for once: the struct's pointers are those of the tensors given at first)."""
        if self._fault is None:
            self._fault = self._find_latent_fault()
        return self._fault

    def _find_latent_fault(self) -> str:
        lat, s = self.latent, self.struct
        if lat is None or lat.dim() < 3 or lat.shape[-1] != D_QK:
            return f"the latent cache is [batch, s_max, {D_QK}] or [pages, page_size, {D_QK}]"
        if lat.dtype not in (torch.bfloat16, torch.float8_e4m3fn) or not lat.is_contiguous():
            return "the latent cache is contiguous, bf16 or E4M3"
        rows = s.num_pages * s.page_size if self.block_table is not None else s.batch * s.s_max
        if lat.numel() != rows * D_QK:
            return "the latent cache has other rows than the index keys"
        f8, sc = lat.dtype == torch.float8_e4m3fn, self.latent_scale
        if f8 and (sc is None or sc.dtype != torch.float32 or not sc.is_contiguous() or sc.numel() != rows * 5):
            return "E4M3 latent rows have contiguous fp32 scales [.., 5]"
        for t, n, name in ((self.seq_lens, s.batch, "seq_lens"),
                           (self.block_table, s.batch * s.max_pages, "block_table")):
            if t is not None and (t.dtype != torch.int32 or not t.is_contiguous() or t.numel() != n):
                return f"{name} is a contiguous int32 tensor with an entry for every sequence"
        for t in (sc if f8 else None, self.seq_lens, self.block_table):
            if t is not None and t.device != lat.device:
                return "the cache's tensors must be on one device"
        return ""

    @classmethod
    def of(cls, ws) -> "Cache":
        """Cache of a workload whose tensors are on the device."""
        return cls(ws.k_idx, ws.latent, ws.seq_lens, ws.k_scale, ws.block_table, ws.page_size,
                   getattr(ws, "latent_scale", None))

    def ref(self):
        return ctypes.byref(self.struct)


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _i64(v) -> int:
    """An integer argument that the library takes in 64 bits."""
    v = int(v)
    _need(-(1 << 63) <= v < 1 << 63, "an integer argument is past 64 bits")
    return v


def _raw_stream(stream, device: torch.device) -> int:
    """The cudaStream_t of ``stream``, or of the device's current stream."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)   # no stream object is made
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _launch(fn, device: torch.device, stream, *args) -> int:
    """A library call with the tensors' device current (kernels launch on the current device)."""
    if device.index == torch.cuda.current_device():
        return fn(*args, _raw_stream(stream, device))
    with torch.cuda.device(device):
        return fn(*args, _raw_stream(stream, device))


class Heads:
    """Queries or keys of ``norm_rope``: the tensors plus the ``dsi_heads`` struct that points
    at them (it can be kept and used again while the tensors live).

    ``x [n, heads, d]`` bf16 (any row and head strides that are multiples of 8 and at least d); ``norm`` None, "rms" or "layer" over
    the first ``norm_dim`` dims (all of them unless given) with fp32 ``weight`` / ``bias``.
    ``out`` is a bf16 tensor ``[rows, heads, d]`` (``x`` itself for in place; a new one, made on
    the current stream, unless given) or an E4M3 one, packed, with ``out_scale``: uint8 ``[rows, heads, d / group]`` makes it
    MXFP8, fp32 ``[rows, heads, ceil(d / 128)]`` FP8 with tile scales.  The ``heads`` dim may be
    left out of ``out`` and ``out_scale`` when there is one head, and page pools
    ``[pages, page_size, ...]`` may stand for their rows.  ``dst_rows`` (int64 ``[n]``): the out
    row of each row; negative skips it.
    """

    def __init__(self, x: torch.Tensor, norm: Optional[str] = None,
                 weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                 norm_dim: Optional[int] = None, out: Optional[torch.Tensor] = None,
                 out_scale: Optional[torch.Tensor] = None, dst_rows: Optional[torch.Tensor] = None):
        _need(x.dim() == 3 and x.dtype == torch.bfloat16, "x is a bf16 [n, heads, d] tensor")
        n, heads, d = (int(v) for v in x.shape)
        _need(x.stride(2) == 1 or d == 1 or x.numel() == 0, "the dims of x must be contiguous")
        _need(norm in NORMS, f"norm is one of {list(NORMS)}")
        nd = d if norm_dim is None else int(norm_dim)
        for t, name in ((weight, "weight"), (bias, "bias")):
            _need(t is None or (t.dtype == torch.float32 and t.is_contiguous() and t.numel() == nd),
                  f"{name} is a contiguous fp32 [norm_dim] tensor")
        _need(dst_rows is None or (dst_rows.dtype == torch.int64 and dst_rows.is_contiguous()
                                   and dst_rows.numel() == n), "dst_rows is an int64 [n] tensor")
        if out is None:
            out = torch.empty((n, heads, d), dtype=torch.bfloat16, device=x.device)
        for t in (weight, bias, out, out_scale, dst_rows):
            _need(t is None or t.device == x.device, "all tensors must be on one device")
        s = DsiHeads()
        s.x, s.n_heads, s.norm, s.norm_dim = x.data_ptr() or None, heads, NORMS[norm], nd
        # a dim of size one has no pitch that matters
        s.ld_head = int(x.stride(1)) if heads > 1 else d
        s.ld_row = int(x.stride(0)) if n > 1 else d
        s.weight = weight.data_ptr() if weight is not None else None
        s.bias = bias.data_ptr() if bias is not None else None
        s.dst_rows = dst_rows.data_ptr() if dst_rows is not None else None
        s.out = out.data_ptr() or None
        _need(int(out.shape[-1]) == d, "out has the dims of x")
        if out.dtype == torch.bfloat16 and out.dim() == 3 and int(out.shape[1]) == heads:
            _need(out_scale is None, "a bf16 out has no scales")
            _need(out.stride(2) == 1 or d == 1 or out.numel() == 0, "the dims of out must be contiguous")
            rows = int(out.shape[0])
            s.ld_out_head = int(out.stride(1)) if heads > 1 else d
            s.ld_out_row = int(out.stride(0)) if rows > 1 else d
            s.out_dtype = DSI_BF16
        else:
            _need(out.is_contiguous(), "a page pool or E4M3 codes must be contiguous")
            _need(heads <= 1 or int(out.shape[-2]) == heads, "out has the heads of x")
            rows = out.numel() // (heads * d) if heads else 0
            s.ld_out_row, s.ld_out_head = max(1, heads) * d, d
            if out.dtype == torch.bfloat16:
                _need(out_scale is None, "a bf16 out has no scales")
                s.out_dtype = DSI_BF16
            else:
                _need(out.dtype == torch.float8_e4m3fn, "out is bf16 or E4M3 codes")
                _need(out_scale is not None and out_scale.is_contiguous(),
                      "E4M3 codes need a contiguous out_scale")
                per = int(out_scale.shape[-1])
                _need(out_scale.numel() == rows * heads * per,
                      "out_scale has a row for every vector of out")
                if out_scale.dtype == torch.uint8:
                    _need(per > 0 and d % per == 0, "MXFP8 scales are [rows, heads, d / group]")
                    s.out_dtype, s.out_group = DSI_MXFP8_E4M3, d // per
                else:
                    _need(out_scale.dtype == torch.float32 and per == (d + 127) // 128,
                          "FP8 scales are fp32 [rows, heads, ceil(d / 128)]")
                    s.out_dtype = DSI_FP8_E4M3
                s.out_scale = out_scale.data_ptr() or None
        s.out_rows = rows
        self.x, self.weight, self.bias, self.out = x, weight, bias, out
        self.out_scale, self.dst_rows, self.n, self.d, self.struct = out_scale, dst_rows, n, d, s
        self.device, self._ref = x.device, ctypes.byref(s)

    def ref(self):
        return self._ref


# ----------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ----------------------------------------------------------------------------

def index_score(q_idx, w, cache: Cache, decode: bool, q_offset: int = 0, scores=None,
                ld: Optional[int] = None, stream=None, checked: bool = False):
    lib = load(checked)
    rows, H_i = int(q_idx.shape[0]), int(q_idx.shape[1])
    if ld is None:
        ld = cache.struct.s_max if decode else q_offset + rows
    if scores is None:
        scores = torch.empty((rows, ld), dtype=torch.float32, device=q_idx.device)
    st = lib.dsi_index_score(_ptr(q_idx), _ptr(w), cache.ref(), rows, H_i, int(bool(decode)),
                             int(q_offset), _ptr(scores), int(ld), _stream(stream))
    _check(lib, "dsi_index_score", st)
    return scores


def index_topk_prefill(q_idx, w, cache: Cache, K: int, q_offset: int = 0, idx=None, count=None,
                       stream=None, checked: bool = False):
    """Fused prefill indexer: the causal Top-K indices of every query token,
    computed without writing the score matrix."""
    lib = load(checked)
    T, H_i = int(q_idx.shape[0]), int(q_idx.shape[1])
    if idx is None:
        idx = torch.empty((T, K), dtype=torch.int32, device=q_idx.device)
    if count is None:
        count = torch.empty((T,), dtype=torch.int32, device=q_idx.device)
    st = lib.dsi_index_topk_prefill(_ptr(q_idx), _ptr(w), cache.ref(), T, H_i, int(q_offset),
                                    int(K), _ptr(idx), _ptr(count), _stream(stream))
    _check(lib, "dsi_index_topk_prefill", st)
    return idx, count


def mxfp8_quantize(x, group: int = 32, dst_rows=None, codes=None, scales=None, stream=None,
                   checked: bool = False):
    """MXFP8 codes (float8_e4m3fn) and E8M0 scale bytes (uint8) of bf16 rows
    ``x [n, d]``; with ``dst_rows`` (int64 [n]) row i goes to row dst_rows[i]
    of the given ``codes``/``scales`` (an append into a cache)."""
    lib = load(checked)
    n, d = int(x.shape[0]), int(x.shape[1])
    _rows_contiguous(x, "x")
    if codes is None:
        codes = torch.empty((n, d), dtype=torch.float8_e4m3fn, device=x.device)
    if scales is None:
        scales = torch.empty((n, d // group), dtype=torch.uint8, device=x.device)
    st = lib.dsi_mxfp8_quantize(_ptr(x), n, d, int(x.stride(0)), int(group), _ptr(dst_rows),
                                _ptr(codes), _ptr(scales), _stream(stream))
    _check(lib, "dsi_mxfp8_quantize", st)
    return codes, scales


def latent_fp8_append(x, dst_rows=None, codes=None, scales=None, stream=None,
                      checked: bool = False):
    """FP8 latent codes (float8_e4m3fn [*, 576]) and fp32 tile scales ([*, 5]) of
    bf16 latent rows ``x [n, 576]``; with ``dst_rows`` (int64 [n]) row i goes to
    row dst_rows[i] of the given ``codes``/``scales`` (an append into a cache)."""
    lib = load(checked)
    n = int(x.shape[0])
    _rows_contiguous(x, "x")
    if int(x.shape[1]) != D_QK:
        raise ValueError(f"latent rows are {D_QK} wide, got {int(x.shape[1])}")
    if codes is None:
        codes = torch.empty((n, D_QK), dtype=torch.float8_e4m3fn, device=x.device)
    if scales is None:
        scales = torch.empty((n, 5), dtype=torch.float32, device=x.device)
    st = lib.dsi_latent_fp8_append(_ptr(x), n, int(x.stride(0)), _ptr(dst_rows), _ptr(codes),
                                   _ptr(scales), _stream(stream))
    _check(lib, "dsi_latent_fp8_append", st)
    return codes, scales


def dense_mla_workspace_size(rows: int, n_heads: int, checked: bool = False) -> int:
    """Bytes of workspace with which the dense and window calls split long histories."""
    return int(load(checked).dsi_dense_mla_workspace_size(rows, n_heads))


def _dense(fn: str, q, cache: Cache, args, rows: int, scale, out, lse, want_lse, workspace, stream,
           checked, prefix: Optional[Cache] = None):
    """Checks and buffers shared by the dense, window and prefix calls; new buffers belong to the
    stream that the kernels run on."""
    lib = load(checked)
    if q.dtype != torch.bfloat16 or q.dim() != 3 or not q.is_contiguous() or q.shape[2] != D_QK:
        raise ValueError(f"q is a contiguous bf16 [rows, heads, {D_QK}] tensor")
    device = q.device
    for c in (cache,) if prefix is None else (cache, prefix):
        fault = c.latent_fault()
        if fault:
            raise ValueError(fault)
        if c.latent.device != device:
            raise ValueError("the cache has no latent rows on q's device")
    n, H, _ = q.shape
    if n != rows:
        raise ValueError(f"q has {n} rows, the call {rows}")
    if out is not None and (out.dtype != torch.bfloat16 or out.shape != (n, H, D_LATENT) or
                            not out.is_contiguous() or out.device != device):
        raise ValueError(f"out is a contiguous bf16 [rows, heads, {D_LATENT}] tensor")
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (n, H) or
                            not lse.is_contiguous() or lse.device != device):
        raise ValueError("lse is a contiguous fp32 [rows, heads] tensor")
    if workspace is not None and (workspace.device != device or not workspace.is_contiguous()):
        raise ValueError("workspace is a contiguous tensor on q's device")
    if n == 0 or H == 0:
        return (out if out is not None else q.new_empty((n, H, D_LATENT)),
                lse if lse is not None or not want_lse else q.new_empty((n, H), dtype=torch.float32))
    if out is None or workspace is None or (lse is None and want_lse):
        on = stream
        if on is not None and not hasattr(on, "cuda_stream"):
            on = torch.cuda.ExternalStream(int(on), device=device)
        with torch.cuda.device(device), torch.cuda.stream(on):
            if workspace is None:
                size = lib.dsi_dense_mla_workspace_size if prefix is None else lib.dsi_prefix_mla_workspace_size
                workspace = alloc_workspace(size(n, H), device)
            if out is None:
                out = torch.empty((n, H, D_LATENT), dtype=torch.bfloat16, device=device)
            if lse is None and want_lse:
                lse = torch.empty((n, H), dtype=torch.float32, device=device)
    caches = (cache.ref(),) if prefix is None else (prefix.ref(), cache.ref())
    st = _launch(getattr(lib, fn), device, stream, q.data_ptr(), *caches, *args, scale,
                 out.data_ptr(), lse.data_ptr() if lse is not None else None, workspace.data_ptr(),
                 workspace.numel() * workspace.element_size())
    if st:
        raise DsiError(fn, st, lib)
    return out, lse


def dense_mla_decode(q, cache: Cache, scale: float, tokens_per_seq: int = 1, out=None, lse=None,
                     want_lse=True, workspace=None, stream=None, checked: bool = False):
    """Attention of the newest tokens over the whole latent cache: ``dsi_dense_mla_decode``.
    ``q`` bf16 ``[batch * tokens_per_seq, heads, 576]``; returns (out, lse)."""
    T = int(tokens_per_seq)
    return _dense("dsi_dense_mla_decode", q, cache, (T, int(q.shape[1])), cache.struct.batch * T, scale,
                  out, lse, want_lse, workspace, stream, checked)


def window_mla_decode(q, cache: Cache, window: int, n_sink: int, scale: float,
                      tokens_per_seq: int = 1, out=None, lse=None, want_lse=True, workspace=None,
                      stream=None, checked: bool = False):
    """The newest tokens over their last ``window`` positions and the first ``n_sink``:
    ``dsi_window_mla_decode``."""
    T = int(tokens_per_seq)
    return _dense("dsi_window_mla_decode", q, cache, (T, int(q.shape[1]), _i64(window), _i64(n_sink)),
                  cache.struct.batch * T, scale, out, lse, want_lse, workspace, stream, checked)


def window_mla_prefill(q, cache: Cache, q_offset: int, window: int, n_sink: int, scale: float,
                       out=None, lse=None, want_lse=True, workspace=None, stream=None,
                       checked: bool = False):
    """Tokens ``q_offset ...`` of one sequence, each over its last ``window`` positions and the
    first ``n_sink``: ``dsi_window_mla_prefill``."""
    T = int(q.shape[0])
    return _dense("dsi_window_mla_prefill", q, cache, (T, int(q.shape[1]), _i64(q_offset), _i64(window),
                                                       _i64(n_sink)),
                  T, scale, out, lse, want_lse, workspace, stream, checked)


def prefix_mla_workspace_size(rows: int, n_heads: int, checked: bool = False) -> int:
    """Bytes of workspace of ``prefix_mla_decode``."""
    return int(load(checked).dsi_prefix_mla_workspace_size(rows, n_heads))


def prefix_mla_decode(q, prefix: Cache, cache: Cache, scale: float, tokens_per_seq: int = 1, out=None,
                      lse=None, want_lse=True, workspace=None, stream=None, checked: bool = False):
    """Attention of the newest tokens over a prefix that the whole batch shares (a cache of one
    sequence, read once for all) and over the sequences' own rows: ``dsi_prefix_mla_decode``.
    ``q`` bf16 ``[batch * tokens_per_seq, heads, 576]``; returns (out, lse)."""
    T = int(tokens_per_seq)
    return _dense("dsi_prefix_mla_decode", q, cache, (T, int(q.shape[1])), cache.struct.batch * T, scale,
                  out, lse, want_lse, workspace, stream, checked, prefix)


def rope_table(n_positions: int, rope_dim: int, theta: float = 10000.0, device="cuda"):
    """fp32 ``[n_positions, rope_dim]`` table of ``norm_rope``: cosines, then sines, of
    position * theta^(-2 i / rope_dim), the angles in fp64."""
    i = torch.arange(0, rope_dim, 2, dtype=torch.float64, device=device)
    ang = torch.arange(n_positions, dtype=torch.float64, device=device)[:, None] * theta ** (-i / rope_dim)
    return torch.cat([ang.cos(), ang.sin()], dim=1).to(torch.float32)


def norm_rope(queries: Optional[Heads], keys: Optional[Heads], table, positions,
              rope_offset: int = 0, interleaved: bool = False, eps: float = 1e-6, stream=None,
              checked: bool = False):
    """Head norms and position rotation of new tokens' queries and keys in one launch (keys
    into their cache rows): ``dsi_norm_rope``.  ``table`` fp32 ``[positions, rope_dim]`` (see
    ``rope_table``), ``positions`` int64 ``[n]``.  Returns the two sides' outs."""
    lib = load(checked)
    side = queries if queries is not None else keys
    _need(side is not None, "queries, keys or both")
    n, device = side.n, side.device
    if queries is not None and keys is not None and (n != keys.n or side.d != keys.d or device != keys.device):
        raise ValueError("queries and keys have the same rows, dims and device")
    if table.dtype != torch.float32 or table.dim() != 2 or not table.is_contiguous():
        raise ValueError("table is a contiguous fp32 [positions, rope_dim] tensor")
    if positions.dtype != torch.int64 or positions.numel() != n or not positions.is_contiguous():
        raise ValueError("positions is an int64 [n] tensor")
    if table.device != device or positions.device != device:
        raise ValueError("all tensors must be on one device")
    if n:
        rows, rope_dim = table.shape
        _need(0 <= rope_offset <= side.d - rope_dim, "the rotated dims are dims of x")
        st = _launch(lib.dsi_norm_rope, device, stream,
                     queries.ref() if queries is not None else None, keys.ref() if keys is not None else None,
                     n, side.d, eps, table.data_ptr(), rows, positions.data_ptr(), rope_offset, rope_dim,
                     bool(interleaved))
        if st:
            raise DsiError("dsi_norm_rope", st, lib)
    return (queries.out if queries is not None else None), (keys.out if keys is not None else None)


def linear_workspace_size(n_tokens: int, batch: int, n_heads: int, dk: int, dv: int,
                          checked: bool = False) -> int:
    """Bytes of workspace with which ``linear_prefill`` splits its work over the device."""
    return int(load(checked).dsi_linear_workspace_size(int(n_tokens), int(batch), int(n_heads), int(dk),
                                                       int(dv)))


def _on(stream, device: torch.device):
    """Context in which new tensors belong to the stream that the kernels run on."""
    if stream is not None and not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


def _linear(q, k, v, log_decay, scale, state, in_slots, out_slots, out, batch: int, stream):
    """The checked ``dsi_linear`` struct of the linear attention calls, and out (a new one belongs to
    the stream that the kernels run on)."""
    bf16, fp32, device = torch.bfloat16, torch.float32, q.get_device()
    qs, ks, vs = q.shape, k.shape, v.shape
    for t, shape, name in ((q, qs, "q"), (k, ks, "k"), (v, vs, "v")):
        if len(shape) != 3 or t.dtype is not bf16:
            raise ValueError(f"{name} is a bf16 [tokens, heads, dims] tensor")
    n, H, dk = qs
    Hk, dv = ks[1], vs[2]
    if ks != (n, Hk, dk) or vs != (n, Hk, dv):
        raise ValueError("q, k and v have the same tokens, k the dims of q, v the heads of k")
    if log_decay.dtype is not fp32 or log_decay.shape != (H,) or not log_decay.is_contiguous():
        raise ValueError("log_decay is a contiguous fp32 [heads] tensor")
    if out is None:
        where = None
    elif out.dtype is not bf16 or out.shape != (n, H, dv):
        raise ValueError("out is a bf16 [tokens, heads, dv] tensor")
    else:
        where = out.get_device()
    same = k.get_device() == device and v.get_device() == device and log_decay.get_device() == device
    at_state = slots = at_in = at_out = None
    if state is not None:
        if state.dtype is not fp32 or state.shape[1:] != (H, dk, dv) or not state.is_contiguous():
            raise ValueError("state is a contiguous fp32 [slots, heads, dk, dv] tensor")
        at_state, slots = state.data_ptr(), state.shape[0]
        same = same and state.get_device() == device
    for t, name in ((in_slots, "in_slots"), (out_slots if out_slots is not in_slots else None, "out_slots")):
        if t is not None:
            if state is None or t.dtype is not torch.int32 or t.shape != (batch,) or not t.is_contiguous():
                raise ValueError(f"{name} is a contiguous int32 [batch] tensor beside a state")
            same = same and t.get_device() == device
    if in_slots is not None:
        at_in = in_slots.data_ptr()
    if out_slots is not None:
        at_out = out_slots.data_ptr()
    if not same or (where is not None and where != device):
        raise ValueError("all tensors must be on one device")
    q_row, q_head, q_dim = q.stride()
    k_row, k_head, k_dim = k.stride()
    v_row, v_head, v_dim = v.stride()
    if out is None:
        if n == 0 or H == 0 or dv == 0:
            out = q.new_empty((n, H, dv))
        else:
            with torch.cuda.device(q.device), _on(stream, q.device):
                out = torch.empty((n, H, dv), dtype=bf16, device=q.device)
    o_row, o_head, o_dim = out.stride()
    if n and not q_dim == k_dim == v_dim == o_dim == 1:
        raise ValueError("the dims of a head must be contiguous")
    # a dim of size one has no pitch that matters
    if n <= 1:
        q_row = k_row = dk
        v_row = o_row = dv
    if H <= 1:
        q_head, o_head = dk, dv
    if Hk <= 1:
        k_head, v_head = dk, dv
    return DsiLinear(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), q_row, q_head, k_row, k_head, v_row,
                     v_head, o_row, o_head, H, Hk, dk, dv, log_decay.data_ptr(), scale, at_state, slots or 0, at_in,
                     at_out), out


def linear_prefill(q, k, v, log_decay, scale: float, seq_starts, state=None, in_slots=None, out_slots=None,
                   out=None, workspace=None, stream=None, checked: bool = False):
    """Linear attention with a decay for each head over prompts laid end to end: ``dsi_linear_prefill``.

    ``q [n, heads, dk]``, ``k [n, kv_heads, dk]``, ``v [n, kv_heads, dv]`` bf16 (any row and head strides
    that are multiples of 8), ``log_decay`` fp32 ``[heads]``, ``seq_starts`` int32 ``[batch + 1]``.
    ``state`` fp32 ``[slots, heads, dk, dv]``: sequence b starts from slot ``in_slots[b]`` (b unless given;
    negative: zeros) and leaves its state in ``out_slots[b]`` (the in slot unless given; negative:
    nowhere).  Returns out ``[n, heads, dv]`` bf16."""
    lib = load(checked)
    _need(seq_starts.dim() == 1 and seq_starts.dtype == torch.int32 and seq_starts.is_contiguous() and
          seq_starts.numel() >= 1 and seq_starts.device == q.device,
          "seq_starts is a contiguous int32 [batch + 1] tensor on q's device")
    batch = seq_starts.numel() - 1
    s, out = _linear(q, k, v, log_decay, scale, state, in_slots, out_slots, out, batch, stream)
    device = q.device
    if workspace is not None:
        _need(workspace.device == device and workspace.is_contiguous(), "workspace is a contiguous tensor on q's device")
    elif batch and s.n_heads:
        with torch.cuda.device(device), _on(stream, device):
            workspace = alloc_workspace(
                lib.dsi_linear_workspace_size(q.shape[0], batch, s.n_heads, s.dk, s.dv), device)
    if batch:
        st = _launch(lib.dsi_linear_prefill, device, stream, ctypes.byref(s), q.shape[0], seq_starts.data_ptr(),
                     batch, workspace.data_ptr() if workspace is not None else None,
                     workspace.numel() * workspace.element_size() if workspace is not None else 0)
        if st:
            raise DsiError("dsi_linear_prefill", st, lib)
    return out


def linear_decode(q, k, v, log_decay, scale: float, state=None, tokens_per_seq: int = 1, in_slots=None,
                  out_slots=None, out=None, stream=None, checked: bool = False):
    """The same for ``tokens_per_seq`` new tokens of every sequence, rows in the sequences' order:
    ``dsi_linear_decode``."""
    lib = load(checked)
    T = int(tokens_per_seq)
    _need(T >= 1 and q.dim() == 3 and q.shape[0] % T == 0, "q has tokens_per_seq rows for every sequence")
    batch = q.shape[0] // T
    s, out = _linear(q, k, v, log_decay, scale, state, in_slots, out_slots, out, batch, stream)
    if batch:
        st = _launch(lib.dsi_linear_decode, q.device, stream, ctypes.byref(s), batch, T)
        if st:
            raise DsiError("dsi_linear_decode", st, lib)
    return out


def topk(scores, K: int, row_len=None, q_offset: int = 0, idx=None, count=None, stream=None,
         checked: bool = False):
    lib = load(checked)
    rows, ld = int(scores.shape[0]), int(scores.stride(0)) if scores.dim() == 2 else 0
    if idx is None:
        idx = torch.empty((rows, K), dtype=torch.int32, device=scores.device)
    if count is None:
        count = torch.empty((rows,), dtype=torch.int32, device=scores.device)
    st = lib.dsi_topk(_ptr(scores), ld, rows, _ptr(row_len), int(q_offset), int(K), _ptr(idx),
                      _ptr(count), _stream(stream))
    _check(lib, "dsi_topk", st)
    return idx, count


def sparse_mla_decode(q, cache: Cache, idx, scale: float, out=None, lse=None, want_lse=True,
                      workspace=None, stream=None, checked: bool = False):
    lib = load(checked)
    B, H = int(q.shape[0]), int(q.shape[1])
    K = int(idx.shape[1])
    if out is None:
        out = torch.empty((B, H, D_LATENT), dtype=torch.bfloat16, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    wsz = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib.dsi_sparse_mla_decode(_ptr(q), cache.ref(), _ptr(idx), B, H, K, float(scale),
                                   _ptr(out), _ptr(lse), _ptr(workspace), wsz, _stream(stream))
    _check(lib, "dsi_sparse_mla_decode", st)
    return out, lse


def sparse_mla_prefill(q, cache: Cache, idx, q_offset: int, scale: float, out=None, lse=None,
                       want_lse=True, workspace=None, stream=None, checked: bool = False):
    lib = load(checked)
    T, H = int(q.shape[0]), int(q.shape[1])
    K = int(idx.shape[1])
    if out is None:
        out = torch.empty((T, H, D_LATENT), dtype=torch.bfloat16, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    wsz = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib.dsi_sparse_mla_prefill(_ptr(q), cache.ref(), _ptr(idx), T, H, K, int(q_offset),
                                    float(scale), _ptr(out), _ptr(lse), _ptr(workspace), wsz,
                                    _stream(stream))
    _check(lib, "dsi_sparse_mla_prefill", st)
    return out, lse


def workspace_size(rows: int, n_heads_idx: int, n_heads: int, K: int, s_max: int,
                   decode: bool, checked: bool = False) -> int:
    return int(load(checked).dsi_workspace_size(rows, n_heads_idx, n_heads, K, s_max,
                                                 int(bool(decode))))


def layer_workspace_size(cache: "Cache", rows: int, n_heads_idx: int, n_heads: int, K: int,
                         q_offset: int, decode: bool, checked: bool = False) -> int:
    """Exact workspace bytes of one fused-layer call (no score rows when a
    prefill takes the fused indexer)."""
    return int(load(checked).dsi_layer_workspace_size(cache.ref(), rows, n_heads_idx, n_heads, K,
                                                       int(q_offset), int(bool(decode))))


def alloc_workspace(nbytes: int, device) -> torch.Tensor:
    # torch's caching allocator returns 512-byte aligned blocks
    return torch.empty((max(256, nbytes),), dtype=torch.uint8, device=device)


def indexed_attention(q_idx, w, q, cache: Cache, K: int, scale: float, decode: bool,
                      q_offset: int = 0, out=None, lse=None, idx=None, count=None,
                      workspace=None, want_lse=True, want_idx=True, stream=None,
                      checked: bool = False):
    """The whole layer (indexer -> Top-K -> sparse MLA) through ``dsi_indexed_attention``."""
    lib = load(checked)
    rows, H_i, H = int(q_idx.shape[0]), int(q_idx.shape[1]), int(q.shape[1])
    dev = q.device
    if workspace is None:
        workspace = alloc_workspace(
            layer_workspace_size(cache, rows, H_i, H, K, q_offset, decode, checked), dev)
    if out is None:
        out = torch.empty((rows, H, D_LATENT), dtype=torch.bfloat16, device=dev)
    if lse is None and want_lse:
        lse = torch.empty((rows, H), dtype=torch.float32, device=dev)
    if idx is None and want_idx:
        idx = torch.empty((rows, K), dtype=torch.int32, device=dev)
    if count is None and want_idx:
        count = torch.empty((rows,), dtype=torch.int32, device=dev)
    st = lib.dsi_indexed_attention(_ptr(q_idx), _ptr(w), _ptr(q), cache.ref(), rows, H_i, H, int(K),
                                   int(q_offset), float(scale), int(bool(decode)), _ptr(idx),
                                   _ptr(count), _ptr(out), _ptr(lse), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream(stream))
    _check(lib, "dsi_indexed_attention", st)
    return out, lse, idx, count


def indexed_attention_multi(q_idx, w, q, cache: Cache, tokens_per_seq: int, K: int, scale: float,
                            out=None, lse=None, idx=None, count=None, workspace=None,
                            want_lse=True, want_idx=True, stream=None, checked: bool = False):
    """A multi-token decode step through ``dsi_indexed_attention_multi``: rows
    come ``tokens_per_seq`` to a sequence (row r is candidate r % T of
    sequence r // T)."""
    lib = load(checked)
    rows, H_i, H = int(q_idx.shape[0]), int(q_idx.shape[1]), int(q.shape[1])
    dev = q.device
    if workspace is None:
        workspace = alloc_workspace(workspace_size(rows, H_i, H, K, cache.struct.s_max, True,
                                                   checked), dev)
    if out is None:
        out = torch.empty((rows, H, D_LATENT), dtype=torch.bfloat16, device=dev)
    if lse is None and want_lse:
        lse = torch.empty((rows, H), dtype=torch.float32, device=dev)
    if idx is None and want_idx:
        idx = torch.empty((rows, K), dtype=torch.int32, device=dev)
    if count is None and want_idx:
        count = torch.empty((rows,), dtype=torch.int32, device=dev)
    st = lib.dsi_indexed_attention_multi(_ptr(q_idx), _ptr(w), _ptr(q), cache.ref(),
                                         int(tokens_per_seq), H_i, H, int(K), float(scale),
                                         _ptr(idx), _ptr(count), _ptr(out), _ptr(lse),
                                         _ptr(workspace),
                                         workspace.numel() * workspace.element_size(),
                                         _stream(stream))
    _check(lib, "dsi_indexed_attention_multi", st)
    return out, lse, idx, count


def device_status(stream=None, checked: bool = False) -> int:
    """Synchronise the stream and read/clear the device status word."""
    lib = load(checked)
    return int(lib.dsi_get_device_status(_stream(stream)))


def selftest_wait_timeout(limit_ns: int, stream=None, checked: bool = False) -> None:
    """Launch the bounded-wait self-test (one warp waits on a barrier nothing
    completes, for ``limit_ns``); ``device_status()`` then reports the timeout."""
    lib = load(checked)
    _check(lib, "dsi_selftest_wait_timeout", lib.dsi_selftest_wait_timeout(int(limit_ns),
                                                                          _stream(stream)))


def launch_count(checked: bool = False) -> int:
    """Kernels the library has launched in this process."""
    return int(load(checked).dsi_launch_count())


def layer(ws, workspace=None, stream=None, checked: bool = False, **kw):
    """Run the whole layer on a device-resident workload."""
    return indexed_attention(ws.q_idx, ws.w, ws.q, Cache.of(ws), ws.K, ws.scale,
                             ws.mode == "decode", ws.q_offset, workspace=workspace,
                             stream=stream, checked=checked, **kw)
