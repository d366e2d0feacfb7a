"""paged_fp8_kv_02_gb300 -- decode attention over a paged FP8 (e4m3) KV cache
for NVIDIA GB300 (sm_103a).

A thin Python binding over the C ABI in ``include/pfkv.h`` (``libpfkv.so``).
Every function below has the name of the C entry point without the ``pfkv_``
prefix and only marshals arguments: tensors become device pointers, the current
torch CUDA stream becomes the ``stream`` argument, and a negative status raises
``PfkvError``.  PyTorch supplies device memory and streams; all arithmetic runs
in the library's CUDA kernels.  There is no fallback: if ``libpfkv.so`` is
missing or fails to load, importing the binding's functions raises.
"""
from __future__ import annotations

import array
import ctypes
import os
import threading

from . import _build

__all__ = [
    "PfkvError", "load", "lib_path", "kv_append_fp8", "kv_append_bf16",
    "kv_append_fp8_scaled", "kv_append_fp8_block", "page_key_bounds", "select_pages_workspace_size", "select_pages",
    "paged_sparse_decode_attn",
    "paged_decode_workspace_size", "paged_decode_attn", "paged_decode_attn_noalloc", "paged_decode_attn_scaled",
    "paged_prefill_workspace_size", "paged_prefill_attn",
    "Rotary", "rotary_embed", "rotary_append_fp8", "verify_drafts", "PagedArrays", "copy_pages",
    "SCALE_TENSOR", "SCALE_HEAD", "SCALE_TOKEN", "SCALE_BLOCK",
    "mla_decode_workspace_size",
    "mla_decode_attn", "validate_tables", "verify_page_tags", "workspace_status", "selftest_barrier_timeout",
    "last_error", "version",
    "CACHE_FP8_E4M3", "CACHE_BF16", "DEVERR", "REQ_TAG_MISMATCH", "REQ_BAD_INDEX",
    "REQ_BAD_TOKEN", "REQ_NO_MASS",
    "PagePool", "block_hash", "slots_from_table",
]

CACHE_FP8_E4M3 = 0
CACHE_BF16 = 1
DEVERR = {
    "WAIT_TIMEOUT": 0x01, "BAD_PAGE": 0x02, "BAD_CONTEXT": 0x04, "WORKSPACE": 0x08,
    "BAD_TOPK": 0x10, "BAD_SLOT": 0x20,
}

REQ_TAG_MISMATCH = 0x1  # verify_page_tags: a page the request reads carries another tag
REQ_BAD_INDEX = 0x2     # verify_page_tags: a page id or context length out of range; verify_drafts: q_start
REQ_BAD_TOKEN = 0x4     # verify_drafts: a drafted token outside the vocabulary
REQ_NO_MASS = 0x8       # verify_drafts: no weight to draw a token with

_lock = threading.Lock()
_lib = None


class PfkvError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} failed with status {code}: {msg}")
        self.code = code


def lib_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libpfkv.so (building it first if it is absent and allowed)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB
        if not os.path.exists(path):
            if not build_if_missing:
                raise OSError(f"libpfkv not built: {path}")
            _build.build_pfkv()
        L = ctypes.CDLL(path)
        vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        sig = {
            "pfkv_kv_append_fp8": (i32, [vp, vp, vp, vp, vp, i32, i32, i32, i32, i64, f32, f32, vp]),
            "pfkv_kv_append_bf16": (i32, [vp, vp, vp, vp, vp, i32, i32, i32, i32, i64, vp]),
            "pfkv_kv_append_fp8_scaled": (i32, [vp, vp, vp, vp, vp, i32, i32, i32, i32, i64, i32, vp, vp,
                                                vp]),
            "pfkv_kv_append_fp8_block": (i32, [vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32,
                                               i32, i64, vp]),
            "pfkv_rotary_init": (i32, [vp, vp, vp, i32, i32, i32, i32]),
            "pfkv_rotary_embed": (i32, [vp, i64, vp, i64, vp, vp, i32, i32, i32, vp]),
            "pfkv_rotary_append_fp8": (i32, [vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, vp, i32, i32, i32,
                                             i32, i32, i64, i32, vp, vp, vp]),
            "pfkv_verify_drafts": (i32, [vp, vp, vp, i64, vp, i64, i32, vp, vp, vp, i32, i32, i32, vp, vp, vp]),
            "pfkv_copy_pages": (i32, [vp, i32, vp, i32, i64, vp, vp]),
            "pfkv_page_key_bounds": (i32, [vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, i64, vp]),
            "pfkv_select_pages_workspace_size": (sz, [i32, i32, i32]),
            "pfkv_select_pages": (i32, [vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i64, i32, i32,
                                        i32, vp, sz, vp, vp]),
            "pfkv_paged_sparse_decode_attn": (i32, [vp, vp, vp, vp, i32, vp, vp, vp, i32, vp, i32, vp, i32, i32,
                                                    i32, i32, i32, i64, f32, vp, vp, vp]),
            "pfkv_paged_decode_workspace_size": (sz, [i32, i32, i32, i32, i32, i64]),
            "pfkv_paged_decode_attn": (i32, [vp, vp, vp, vp, i32, vp, i32, vp, i32, i32, i32, i32, i32,
                                             i64, f32, f32, f32, i32, vp, sz, vp, vp]),
            "pfkv_paged_decode_attn_noalloc": (i32, [vp, vp, vp, vp, i32, vp, i32, vp, i32, i32, i32, i32,
                                                     i32, i64, f32, f32, f32, i32, i64, vp, vp, vp]),
            "pfkv_paged_decode_attn_scaled": (i32, [vp, vp, vp, vp, i32, vp, vp, vp, i32, vp, i32, i32, i32,
                                                    i32, i32, i64, f32, i32, vp, sz, vp, vp]),
            "pfkv_paged_prefill_workspace_size": (sz, [i32, i32, i32, i32, i32, i32, i32]),
            "pfkv_paged_prefill_attn": (i32, [vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, i64,
                                              i32, i32, f32, f32, f32, i32, vp, sz, vp, vp]),
            "pfkv_mla_decode_workspace_size": (sz, [i32, i32, i32, i32]),
            "pfkv_mla_decode_attn": (i32, [vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, i32,
                                           i64, f32, f32, vp, sz, vp, vp]),
            "pfkv_validate_tables": (i32, [vp, i32, vp, i32, i32, i64, vp, i32, vp, i32, vp, vp]),
            "pfkv_verify_page_tags": (i32, [vp, vp, i32, vp, i32, i32, vp, i64, vp, vp]),
            "pfkv_workspace_status": (i32, [vp, vp, vp]),
            "pfkv_pool_create": (vp, [i64, i32]),
            "pfkv_pool_destroy": (None, [vp]),
            "pfkv_pool_num_free": (i64, [vp]),
            "pfkv_pool_refcount": (i32, [vp, ctypes.c_int32]),
            "pfkv_pool_page_tags": (i32, [vp, vp]),
            "pfkv_pool_map_request": (i32, [vp, vp, i32, vp, vp, i32, vp]),
            "pfkv_pool_release": (i32, [vp, vp, i32]),
            "pfkv_pool_fork": (i32, [vp, vp, i32]),
            "pfkv_pool_resize": (i32, [vp, vp, vp, i32, i32]),
            "pfkv_pool_make_writable": (i32, [vp, vp, vp, i32, i32, vp, vp]),
            "pfkv_pool_compact": (i32, [vp, i64, vp, vp, vp]),
            "pfkv_block_hash": (ctypes.c_uint64, [ctypes.c_uint64, vp, i32]),
            "pfkv_slots_from_table": (i32, [vp, i32, i32, i32, i32, vp]),
            "pfkv_selftest_barrier_timeout": (i32, [vp, vp]),
            "pfkv_last_error": (ctypes.c_char_p, []),
            "pfkv_version": (ctypes.c_char_p, []),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
        return _lib


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _stream(stream):
    import torch
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _check(fn: str, rc: int):
    if rc != 0:
        raise PfkvError(fn, rc, last_error())


def last_error() -> str:
    return load().pfkv_last_error().decode()


def version() -> str:
    return load().pfkv_version().decode()


# ---------------------------------------------------------------- append
def kv_append_fp8(k_new, v_new, k_cache, v_cache, slot_mapping, k_scale: float, v_scale: float = 1.0,
                  stream=None):
    """Quantise bf16 rows k_new/v_new [T][H][D] to e4m3 and scatter them into
    k_cache/v_cache [pages][H][P][D] (uint8) at slot_mapping [T] (int64).
    For one latent tensor pass v_new = v_cache = None."""
    T, H, D = k_new.shape
    pages, _, P, _ = k_cache.shape
    rc = load().pfkv_kv_append_fp8(_ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                   _ptr(slot_mapping), T, H, D, P, pages, float(k_scale),
                                   float(v_scale), _stream(stream))
    _check("kv_append_fp8", rc)


def kv_append_bf16(k_new, v_new, k_cache, v_cache, slot_mapping, stream=None):
    T, H, D = k_new.shape
    pages, _, P, _ = k_cache.shape
    rc = load().pfkv_kv_append_bf16(_ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                    _ptr(slot_mapping), T, H, D, P, pages, _stream(stream))
    _check("kv_append_bf16", rc)


SCALE_TENSOR = 0
SCALE_HEAD = 1
SCALE_TOKEN = 2
SCALE_BLOCK = 3


def kv_append_fp8_scaled(k_new, v_new, k_cache, v_cache, slot_mapping, granularity: int, k_scales,
                         v_scales=None, stream=None):
    """kv_append_fp8 with float32 device scales: SCALE_TENSOR [1] / SCALE_HEAD
    [H] are read; SCALE_TOKEN [pages][H][P] receives each appended row's
    scale (its amax / 448)."""
    T, H, D = k_new.shape
    pages, _, P, _ = k_cache.shape
    rc = load().pfkv_kv_append_fp8_scaled(_ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                          _ptr(slot_mapping), T, H, D, P, pages, int(granularity),
                                          _ptr(k_scales), _ptr(v_scales), _stream(stream))
    _check("kv_append_fp8_scaled", rc)


def _want(name: str, t, dtype, shape, device: int) -> int:
    """Device address of a tensor that has to be just this; ValueError otherwise."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on the call's device "
                     f"{device}, got {t.dtype} {tuple(t.shape)} on {t.device}")


def _count(name: str, v) -> int:
    """A count for a 32-bit argument, which would be cut to its low bits otherwise."""
    if -0x80000000 <= v <= 0x7FFFFFFF:
        return int(v)
    raise ValueError(f"{name}: {v} does not fit 32 bits")


def _bound(v) -> int:
    """An upper bound for a 32-bit argument: larger ones say no more than the largest."""
    return _count("max_new_len", v if v <= 0x7FFFFFFF else 0x7FFFFFFF)


def _on(device: int, f, *args):
    """f(*args) with `device` the current one."""
    import torch
    if device == torch._C._cuda_getDevice():
        return f(*args)
    with torch.cuda.device(device):
        return f(*args)


def _call(fn: str, device: int, stream, *args):
    """One entry point on a device: its current stream unless one is given."""
    import torch
    if device < 0:
        raise ValueError("expected CUDA tensors")
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(device)
    elif stream.device.index != device:
        raise ValueError(f"{fn}: the stream belongs to {stream.device}, the tensors to device {device}")
    else:
        handle = stream.cuda_stream
    _check(fn, _on(device, getattr(_lib or load(), "pfkv_" + fn), *args, handle))


def kv_append_fp8_block(k_new, v_new, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, new_start,
                        max_new_len: int, stream=None):
    """Quantise the last n_b = new_start[b+1] - new_start[b] tokens of every
    request (rows new_start[b].. of k_new/v_new bf16 [T][H][D]) into the pages
    of its block table, with one power-of-two scale per (page, KV head) in
    k_scales/v_scales float32 [pages][H]; a scale grows, and the page's earlier
    codes move to it, when new rows need it.  context_lens int32 [B] counts the
    new tokens; new_start int32 [B+1]; max_new_len bounds every n_b.  For K
    alone pass v_new = v_cache = v_scales = None."""
    import torch
    dev = k_new.get_device()
    T, H, D = k_new.shape
    pages, _, P, _ = k_cache.shape
    B, maxp = block_tables.shape
    cache, scales = (pages, H, P, D), (pages, H)
    v = [None, None, None]
    if not (v_new is None and v_cache is None and v_scales is None):
        if v_new is None or v_cache is None or v_scales is None:
            raise ValueError("v_new, v_cache and v_scales: all or none")
        v = [_want("v_new", v_new, torch.bfloat16, k_new.shape, dev), _want("v_cache", v_cache, torch.uint8, cache, dev),
             _want("v_scales", v_scales, torch.float32, scales, dev)]
    _call("kv_append_fp8_block", dev, stream, _want("k_new", k_new, torch.bfloat16, (T, H, D), dev), v[0],
          _want("k_cache", k_cache, torch.uint8, cache, dev), v[1],
          _want("k_scales", k_scales, torch.float32, scales, dev), v[2],
          _want("block_tables", block_tables, torch.int32, (B, maxp), dev), maxp,
          _want("context_lens", context_lens, torch.int32, (B,), dev),
          _want("new_start", new_start, torch.int32, (B + 1,), dev), B, T, _bound(max_new_len), H, D, P, pages)


# ------------------------------------------------------------ rotary positions
class _RotaryStruct(ctypes.Structure):
    _fields_ = [("first", ctypes.c_int32), ("num_pairs", ctypes.c_int32), ("neighbours", ctypes.c_int32),
                ("num_axes", ctypes.c_int32), ("turns", ctypes.c_uint64 * 128), ("axis", ctypes.c_uint8 * 128)]


class Rotary:
    """A model's rotary positions (``pfkv_rotary_init``), on the host: pair i
    turns by frequencies[i] radians per position on axis axes[i] (None: one
    axis).  The pairs are channels (first + i, first + n + i), or with
    ``neighbours`` (first + 2i, first + 2i + 1).  num_axes: rows of the
    positions, by default one more than the largest axis named."""

    def __init__(self, frequencies, axes=None, first: int = 0, neighbours: bool = False, num_axes: int = None):
        import numpy as np
        f, fp = _host(frequencies, np.float64)
        if f.ndim != 1:
            raise ValueError("frequencies: expected one number per pair")
        ap = None
        if axes is not None:
            x = np.asarray(axes)
            if x.shape != f.shape or not np.issubdtype(x.dtype, np.integer):
                raise ValueError("axes: expected one whole number per pair")
            if x.size and not (0 <= x.min() and x.max() < 128):
                raise ValueError("axes: out of range")
            x, ap = _host(x, np.int32)
            if num_axes is None and x.size:
                num_axes = int(x.max()) + 1
        self._struct = _RotaryStruct()
        self.num_axes = 1 if num_axes is None else _count("num_axes", num_axes)
        _check("rotary_init", load().pfkv_rotary_init(ctypes.byref(self._struct), fp, ap, f.shape[0], self.num_axes,
                                                      _count("first", first), 1 if neighbours else 0))

    @property
    def _ptr(self) -> int:
        """Address of the description, taken when it is passed: a copied or
        unpickled object has a description of its own."""
        return ctypes.addressof(self._struct)


def _rows(name: str, t, dtype, shape, device: int):
    """Address of a tensor [tokens][...] and the elements between two tokens;
    what belongs to one token is contiguous.  ValueError otherwise."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device:
        if t.is_contiguous():
            return t.data_ptr(), shape[1] * shape[2] if len(shape) == 3 else shape[1]
        if t[0].is_contiguous() and shape[0] > 1:
            return t.data_ptr(), t.stride(0)
    raise ValueError(f"{name}: expected a {dtype} tensor of shape {tuple(shape)} on the call's device {device}, "
                     f"contiguous within a token, got {t.dtype} {tuple(t.shape)}, strides {tuple(t.stride())}, on {t.device}")


def _positions(t, rotary: Rotary, tokens: int, device: int) -> int:
    import torch
    shape = (tokens,) if rotary.num_axes == 1 and t.dim() == 1 else (rotary.num_axes, tokens)
    return _want("positions", t, torch.int32, shape, device)


def rotary_embed(out, x, positions, rotary: Rotary, stream=None):
    """Turn bf16 rows x [T][H][D] by their token's positions int32 [axes][T]
    ([T] for one axis) into out, which may be x itself.  Both may be parts of
    wider rows (any stride between tokens that is a multiple of 8), of the same
    ones too where the parts lie beside each other."""
    import torch
    dev = x.get_device()
    T, H, D = x.shape
    o, os = _rows("out", out, torch.bfloat16, (T, H, D), dev)
    i, is_ = _rows("x", x, torch.bfloat16, (T, H, D), dev)
    _call("rotary_embed", dev, stream, o, os, i, is_, _positions(positions, rotary, T, dev), rotary._ptr, T, H, D)


def rotary_append_fp8(q_out, q, k_new, v_new, k_cache, v_cache, slot_mapping, positions, rotary: Rotary,
                      granularity: int, k_scales, v_scales=None, stream=None):
    """rotary_embed of the queries q [T][Hq][D] into q_out and of the keys k_new
    [T][H][D] on their way through kv_append_fp8_scaled, with v_new, in one
    launch: caches uint8 [pages][H][P][D], slot_mapping int64 [T]; SCALE_TENSOR
    [1] / SCALE_HEAD [H] are read, SCALE_TOKEN [pages][H][P] is written.  q_out
    = q = None: no queries.  v_new = v_cache = v_scales = None: keys only."""
    import torch
    dev = k_new.get_device()
    T, H, D = k_new.shape
    pages, _, P, _ = k_cache.shape
    cache, dt = (pages, H, P, D), torch.bfloat16
    scales = {SCALE_TENSOR: (1,), SCALE_HEAD: (H,), SCALE_TOKEN: (pages, H, P)}.get(granularity, k_scales.shape)
    o = os = i = is_ = Hq = 0
    if q is not None or q_out is not None:
        if q is None or q_out is None:
            raise ValueError("q_out and q: both or none")
        Hq = q.shape[1]
        o, os = _rows("q_out", q_out, dt, (T, Hq, D), dev)
        i, is_ = _rows("q", q, dt, (T, Hq, D), dev)
    k, ks = _rows("k_new", k_new, dt, (T, H, D), dev)
    v = vs = vc = vsc = 0
    if not (v_new is None and v_cache is None and v_scales is None):
        if v_new is None or v_cache is None or v_scales is None:
            raise ValueError("v_new, v_cache and v_scales: all or none")
        v, vs = _rows("v_new", v_new, dt, (T, H, D), dev)
        vc = _want("v_cache", v_cache, torch.uint8, cache, dev)
        vsc = _want("v_scales", v_scales, torch.float32, scales, dev)
    _call("rotary_append_fp8", dev, stream, o, os, i, is_, k, ks, v, vs,
          _want("k_cache", k_cache, torch.uint8, cache, dev), vc,
          _want("slot_mapping", slot_mapping, torch.int64, (T,), dev), _positions(positions, rotary, T, dev), rotary._ptr,
          T, Hq, H, D, P, pages, int(granularity), _want("k_scales", k_scales, torch.float32, scales, dev), vsc)


# ---------------------------------------------------------- block-sparse decode
def page_key_bounds(bounds, bound_scales, k_cache, block_tables, context_lens, new_start, max_new_len: int,
                    stream=None):
    """Channelwise bounds of the keys of every page that holds one of a
    request's last new_start[b+1] - new_start[b] tokens: bounds int8
    [pages][H][2][128] (lower, upper) in units of bound_scales float32
    [pages][H] times the page's K scale, from the e4m3 k_cache uint8
    [pages][H][P][128].  max_new_len bounds the counts.  A page shared by
    requests has to hold the same number of rows for each, as full pages do."""
    import torch
    dev = k_cache.get_device()
    pages, H, P, D = k_cache.shape
    B, maxp = block_tables.shape
    _call("page_key_bounds", dev, stream, _want("bounds", bounds, torch.int8, (pages, H, 2, D), dev),
          _want("bound_scales", bound_scales, torch.float32, (pages, H), dev),
          _want("k_cache", k_cache, torch.uint8, (pages, H, P, D), dev),
          _want("block_tables", block_tables, torch.int32, (B, maxp), dev), maxp,
          _want("context_lens", context_lens, torch.int32, (B,), dev),
          _want("new_start", new_start, torch.int32, (B + 1,), dev), B, _bound(max_new_len), H, D, P, pages)


def select_pages_workspace_size(batch: int, num_kv_heads: int, max_pages_per_seq: int) -> int:
    """Bytes of scratch that select_pages needs on the current device."""
    return int(load().pfkv_select_pages_workspace_size(batch, num_kv_heads, max_pages_per_seq))


def select_pages(selected, q, bounds, bound_scales, block_tables, context_lens, page_size: int, sink_pages: int = 1,
                 recent_pages: int = 1, k_scales=None, workspace=None, unit_status=None, stream=None):
    """List the pages each (request, KV head) attends: selected int32
    [B][Hkv][top_pages] receives logical page numbers in ascending order, -1
    past a shorter context's last.  q bf16 [B][Hq][128]; bounds and
    bound_scales from page_key_bounds; k_scales float32 [pages][Hkv] for a
    cache with scales per block.  The first sink_pages and last recent_pages
    pages are always listed.  unit_status: optional int32 [B][Hkv].  Returns
    the workspace used (allocated with torch when not given and needed)."""
    import torch
    dev = q.get_device()
    B, Hq, D = q.shape
    pages, Hkv = bound_scales.shape
    maxp, top = block_tables.shape[1], selected.shape[2]
    nbytes = 0
    if workspace is None:
        if dev < 0:
            raise ValueError("expected CUDA tensors")
        nbytes = _on(dev, (_lib or load()).pfkv_select_pages_workspace_size, B, Hkv, maxp)
        if nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
            if stream is not None:  # a caller that drops it gives it back while that stream may still use it
                workspace.record_stream(stream)
    else:
        nbytes = workspace.numel()
    _call("select_pages", dev, stream, _want("selected", selected, torch.int32, (B, Hkv, top), dev),
          _want("q", q, torch.bfloat16, (B, Hq, D), dev), _want("bounds", bounds, torch.int8, (pages, Hkv, 2, D), dev),
          _want("bound_scales", bound_scales, torch.float32, (pages, Hkv), dev),
          None if k_scales is None else _want("k_scales", k_scales, torch.float32, (pages, Hkv), dev),
          _want("block_tables", block_tables, torch.int32, (B, maxp), dev), maxp,
          _want("context_lens", context_lens, torch.int32, (B,), dev), B, Hq, Hkv, D, _count("page_size", page_size), pages,
          top, _count("sink_pages", sink_pages), _count("recent_pages", recent_pages),
          None if workspace is None else _want("workspace", workspace, torch.uint8, (nbytes,), dev), nbytes,
          None if unit_status is None else _want("unit_status", unit_status, torch.int32, (B, Hkv), dev))
    return workspace


def paged_sparse_decode_attn(out, q, k_cache, v_cache, granularity: int, k_scales, v_scales, selected, block_tables,
                             context_lens, softmax_scale: float, lse_out=None, unit_status=None, stream=None):
    """One decode step over the pages listed for each (request, KV head):
    out/q bf16 [B][Hq][128]; caches uint8 (e4m3) [pages][Hkv][P][128]; scales
    float32 of SCALE_TENSOR [1], SCALE_HEAD [Hkv] or SCALE_BLOCK [pages][Hkv];
    selected int32 [B][Hkv][top_pages], as select_pages writes it (distinct
    logical pages in any order; entries < 0 are padding, in any places).  lse_out: optional float32
    [B][Hq]; unit_status: optional int32 [B][Hkv]."""
    import torch
    dev = q.get_device()
    B, Hq, D = q.shape
    pages, Hkv, P, _ = k_cache.shape
    maxp, top = block_tables.shape[1], selected.shape[2]
    cache = (pages, Hkv, P, D)
    scales = {SCALE_TENSOR: (1,), SCALE_HEAD: (Hkv,), SCALE_BLOCK: (pages, Hkv)}.get(granularity, k_scales.shape)
    _call("paged_sparse_decode_attn", dev, stream, _want("out", out, torch.bfloat16, (B, Hq, D), dev),
          _want("q", q, torch.bfloat16, (B, Hq, D), dev), _want("k_cache", k_cache, torch.uint8, cache, dev),
          _want("v_cache", v_cache, torch.uint8, cache, dev), int(granularity),
          _want("k_scales", k_scales, torch.float32, scales, dev),
          _want("v_scales", v_scales, torch.float32, scales, dev),
          _want("selected", selected, torch.int32, (B, Hkv, top), dev), top,
          _want("block_tables", block_tables, torch.int32, (B, maxp), dev), maxp,
          _want("context_lens", context_lens, torch.int32, (B,), dev), B, Hq, Hkv, D, P, pages, float(softmax_scale),
          None if lse_out is None else _want("lse_out", lse_out, torch.float32, (B, Hq), dev),
          None if unit_status is None else _want("unit_status", unit_status, torch.int32, (B, Hkv), dev))


# ---------------------------------------------------------------- decode
def paged_decode_workspace_size(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int = 128,
                                kv_split_tokens: int = 0, max_total_chunks: int = 0) -> int:
    return int(load().pfkv_paged_decode_workspace_size(batch, num_q_heads, num_kv_heads, head_dim,
                                                       kv_split_tokens, max_total_chunks))


def paged_decode_attn(out, q, k_cache, v_cache, block_tables, context_lens, k_scale: float,
                      v_scale: float, softmax_scale: float, kv_split_tokens: int = 0, workspace=None,
                      lse_out=None, stream=None, max_total_chunks: int = 0):
    """out/q bf16 [B][Hq][D]; caches uint8 (e4m3) or bf16 [pages][Hkv][P][D];
    block_tables int32 [B][max_pages]; context_lens int32 [B].  Returns the
    workspace used (allocated with torch when not given)."""
    import torch
    B, Hq, D = q.shape
    pages, Hkv, P, _ = k_cache.shape
    dt = CACHE_BF16 if k_cache.dtype == torch.bfloat16 else CACHE_FP8_E4M3
    if workspace is None:
        n = paged_decode_workspace_size(B, Hq, Hkv, D, kv_split_tokens, max_total_chunks)
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    rc = load().pfkv_paged_decode_attn(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), dt,
                                       _ptr(block_tables), block_tables.shape[1], _ptr(context_lens), B,
                                       Hq, Hkv, D, P, pages, float(k_scale), float(v_scale),
                                       float(softmax_scale), int(kv_split_tokens), _ptr(workspace),
                                       workspace.numel(), _ptr(lse_out), _stream(stream))
    _check("paged_decode_attn", rc)
    return workspace


def paged_decode_attn_scaled(out, q, k_cache, v_cache, granularity: int, k_scales, v_scales,
                             block_tables, context_lens, softmax_scale: float, kv_split_tokens: int = 0,
                             workspace=None, lse_out=None, stream=None, max_total_chunks: int = 0):
    """paged_decode_attn over an e4m3 cache with float32 device scales of the
    given granularity (SCALE_TENSOR [1], SCALE_HEAD [Hkv], SCALE_TOKEN
    [pages][Hkv][P], SCALE_BLOCK [pages][Hkv]).  Returns the workspace used."""
    import torch
    B, Hq, D = q.shape
    pages, Hkv, P, _ = k_cache.shape
    if granularity == SCALE_BLOCK:
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            _want(name, t, torch.float32, (pages, Hkv), q.get_device())
    if workspace is None:
        n = paged_decode_workspace_size(B, Hq, Hkv, D, kv_split_tokens, max_total_chunks)
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    rc = load().pfkv_paged_decode_attn_scaled(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                              int(granularity), _ptr(k_scales), _ptr(v_scales),
                                              _ptr(block_tables), block_tables.shape[1],
                                              _ptr(context_lens), B, Hq, Hkv, D, P, pages,
                                              float(softmax_scale), int(kv_split_tokens),
                                              _ptr(workspace), workspace.numel(), _ptr(lse_out),
                                              _stream(stream))
    _check("paged_decode_attn_scaled", rc)
    return workspace


def paged_decode_attn_noalloc(out, q, k_cache, v_cache, block_tables, context_lens, k_scale: float,
                              v_scale: float, softmax_scale: float, kv_split_tokens: int = 0,
                              max_total_chunks: int = 0, lse_out=None, status_out=None, stream=None):
    """paged_decode_attn without a workspace: for callers that cannot allocate
    device memory on the decode path.  The library's fixed 64 MiB device
    scratch is used instead (shared by all calls; order calls that could
    overlap).  status_out: optional int32 device tensor of one element."""
    import torch
    B, Hq, D = q.shape
    pages, Hkv, P, _ = k_cache.shape
    dt = CACHE_BF16 if k_cache.dtype == torch.bfloat16 else CACHE_FP8_E4M3
    rc = load().pfkv_paged_decode_attn_noalloc(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), dt,
                                               _ptr(block_tables), block_tables.shape[1], _ptr(context_lens),
                                               B, Hq, Hkv, D, P, pages, float(k_scale), float(v_scale),
                                               float(softmax_scale), int(kv_split_tokens),
                                               int(max_total_chunks), _ptr(lse_out), _ptr(status_out),
                                               _stream(stream))
    _check("paged_decode_attn_noalloc", rc)


def paged_prefill_workspace_size(batch: int, num_q_heads: int, num_kv_heads: int, max_q_len: int,
                                 max_context_len: int, kv_split_tokens: int = 0, head_dim: int = 128) -> int:
    return int(load().pfkv_paged_prefill_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, max_q_len,
                                                        max_context_len, kv_split_tokens))


def paged_prefill_attn(out, q, k_cache, v_cache, block_tables, context_lens, q_start, max_q_len: int,
                       max_context_len: int, k_scale: float, v_scale: float, softmax_scale: float,
                       kv_split_tokens: int = 0, workspace=None, lse_out=None, stream=None):
    """Several new query tokens per request, causal among themselves: q/out
    bf16 [q_start[B]][Hq][D]; q_start int32 [B+1]; caches uint8 (e4m3)
    [pages][Hkv][P][D].  Returns the workspace used."""
    import torch
    T, Hq, D = q.shape
    pages, Hkv, P, _ = k_cache.shape
    B = context_lens.shape[0]
    if workspace is None:
        n = paged_prefill_workspace_size(B, Hq, Hkv, max_q_len, max_context_len, kv_split_tokens, D)
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)
    rc = load().pfkv_paged_prefill_attn(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                        block_tables.shape[1], _ptr(context_lens), _ptr(q_start), B, Hq, Hkv, D,
                                        P, pages, int(max_q_len), int(max_context_len), float(k_scale),
                                        float(v_scale), float(softmax_scale), int(kv_split_tokens),
                                        _ptr(workspace), workspace.numel(), _ptr(lse_out), _stream(stream))
    _check("paged_prefill_attn", rc)
    return workspace


def verify_drafts(next_tokens, accepted, target_probs, draft_probs, tokens, uniforms, q_start, context_lens=None,
                  request_status=None, stream=None):
    """Which drafted tokens stay after a verification pass over the rows
    q_start int32 [B+1] (a request's last known token, then its drafts):
    next_tokens int32 [T] receives the token that follows each row (accepted
    ones, a drawn one, then -1) and accepted int32 [B] their number.
    target_probs float32, bfloat16 or float16 [T][V] is the target's
    distribution of the token after each row; draft_probs likewise the draft's,
    or None where drafts were not sampled; tokens int32 [T]; uniforms float32
    [T] in [0, 1).  Rows of probabilities may lie further apart than V.
    context_lens: optional int32 [B] that loses the rejected tokens;
    request_status: optional int32 [B].  What is written overlaps no other
    tensor of the call (tokens is not next_tokens)."""
    import torch
    dev = target_probs.get_device()
    T, V = target_probs.shape
    B = q_start.shape[0] - 1
    dt = target_probs.dtype
    kind = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}.get(dt)
    if kind is None:
        raise ValueError(f"target_probs: expected float32, bfloat16 or float16, got {dt}")
    p, ps = _rows("target_probs", target_probs, dt, (T, V), dev)
    q, qs = (None, 0) if draft_probs is None else _rows("draft_probs", draft_probs, dt, (T, V), dev)
    i32 = torch.int32
    _call("verify_drafts", dev, stream, _want("next_tokens", next_tokens, i32, (T,), dev),
          _want("accepted", accepted, i32, (B,), dev), p, ps, q, qs, kind, _want("tokens", tokens, i32, (T,), dev),
          _want("uniforms", uniforms, torch.float32, (T,), dev), _want("q_start", q_start, i32, (B + 1,), dev), B, T, V,
          None if context_lens is None else _want("context_lens", context_lens, i32, (B,), dev),
          None if request_status is None else _want("request_status", request_status, i32, (B,), dev))


def mla_decode_workspace_size(batch: int, num_heads: int, d_latent: int = 512, topk: int = 0) -> int:
    return int(load().pfkv_mla_decode_workspace_size(batch, num_heads, d_latent, topk))


def mla_decode_attn(out, q, ckv_cache, block_tables, context_lens, topk_idx, ckv_scale: float,
                    softmax_scale: float, d_latent: int = 512, workspace=None, lse_out=None, stream=None):
    """out bf16 [B][H][d_latent]; q bf16 [B][H][Dqk]; ckv_cache uint8 [pages][P][Dqk];
    topk_idx int32 [B][k] or None."""
    import torch
    B, H, Dqk = q.shape
    pages, P, _ = ckv_cache.shape
    k = 0 if topk_idx is None else topk_idx.shape[1]
    if workspace is None:
        workspace = torch.empty(mla_decode_workspace_size(B, H, d_latent, k), dtype=torch.uint8,
                                device=q.device)
    rc = load().pfkv_mla_decode_attn(_ptr(out), _ptr(q), _ptr(ckv_cache), _ptr(block_tables),
                                     block_tables.shape[1], _ptr(context_lens), _ptr(topk_idx), k, B, H,
                                     d_latent, Dqk - d_latent, P, pages, float(ckv_scale),
                                     float(softmax_scale), _ptr(workspace), workspace.numel(),
                                     _ptr(lse_out), _stream(stream))
    _check("mla_decode_attn", rc)
    return workspace


def validate_tables(block_tables, context_lens, page_size: int, num_pages: int, err_word,
                    topk_idx=None, slot_mapping=None, stream=None):
    B = context_lens.shape[0]
    k = 0 if topk_idx is None else topk_idx.shape[1]
    ns = 0 if slot_mapping is None else slot_mapping.shape[0]
    rc = load().pfkv_validate_tables(_ptr(block_tables), block_tables.shape[1], _ptr(context_lens), B,
                                     page_size, num_pages, _ptr(topk_idx), k, _ptr(slot_mapping), ns,
                                     _ptr(err_word), _stream(stream))
    _check("validate_tables", rc)


def verify_page_tags(block_tables, table_tags, context_lens, page_size: int, page_tags, request_status,
                     stream=None):
    """Page-tag integrity check before decode: request_status[b] (int32, device) receives 0 or an
    OR of REQ_TAG_MISMATCH / REQ_BAD_INDEX.  table_tags (uint32 or int32 bits) has the shape of
    block_tables; page_tags holds one tag per physical page."""
    B = context_lens.shape[0]
    if tuple(table_tags.shape) != tuple(block_tables.shape):
        raise ValueError("table_tags must have the shape of block_tables")
    rc = load().pfkv_verify_page_tags(_ptr(block_tables), _ptr(table_tags), block_tables.shape[1],
                                      _ptr(context_lens), B, page_size, _ptr(page_tags), page_tags.shape[0],
                                      _ptr(request_status), _stream(stream))
    _check("verify_page_tags", rc)


def selftest_barrier_timeout(status, stream=None):
    """Run the bounded-wait self-test; `status` is an int32 device tensor of one element."""
    _check("selftest_barrier_timeout", load().pfkv_selftest_barrier_timeout(_ptr(status), _stream(stream)))


def workspace_status(workspace, stream=None) -> int:
    v = ctypes.c_int32(0)
    rc = load().pfkv_workspace_status(_ptr(workspace), ctypes.byref(v), _stream(stream))
    _check("workspace_status", rc)
    return int(v.value)


# ----------------------------------------------------------------- page copies
class _PagedArrayStruct(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("page_bytes", ctypes.c_int64), ("page_stride", ctypes.c_int64)]


class PagedArrays:
    """The tensors that hold a cache's pages, in all layers: K, V, scales,
    bounds, latents, each [pages][...] with what belongs to a page contiguous.
    Described once, for copy_pages; the tensors are kept, and have to keep
    their memory."""

    def __init__(self, tensors):
        self.tensors = list(tensors)
        if not self.tensors:
            raise ValueError("no tensors")
        self.device = device = self.tensors[0].get_device()
        self.num_pages = pages = self.tensors[0].shape[0] if self.tensors[0].dim() else 0
        numbers = array.array("q")
        for k, t in enumerate(self.tensors):
            if device < 0 or t.get_device() != device:
                raise ValueError(f"tensor {k}: on {t.device}, the first one on device {device}")
            size = t.nbytes
            if size and t.dim() and t.shape[0] == pages:
                page = size // pages
                if t.is_contiguous():
                    numbers.extend((t.data_ptr(), page, page))
                    continue
                if t[0].is_contiguous():
                    numbers.extend((t.data_ptr(), page, t.stride(0) * t.element_size() if pages > 1 else page))
                    continue
            raise ValueError(f"tensor {k}: expected [{pages}][...], contiguous within a page, got {tuple(t.shape)} with "
                             f"strides {tuple(t.stride())}")
        self._arrays = (_PagedArrayStruct * len(self.tensors)).from_buffer(numbers)
        self._ptr = ctypes.addressof(self._arrays)


def copy_pages(arrays: PagedArrays, pairs, pair_status=None, stream=None):
    """Copy page pairs[i][0] to page pairs[i][1] in every array (pairs int32
    [n][2] on 8 bytes; a pair with a negative entry is padding).  No page may be the
    destination of two pairs, or of one and the source of another: its bytes
    are unspecified then.  The pairs of one PagePool.compact, or of
    make_writable calls without a fork, a cut, a release or a compact between
    them, may share a call; others take one each, in the order of the pool's
    calls.  pair_status: optional int32 [n]."""
    import torch
    dev = arrays.device
    n = pairs.shape[0]
    _call("copy_pages", dev, stream, arrays._ptr, len(arrays._arrays), _want("pairs", pairs, torch.int32, (n, 2), dev), n,
          arrays.num_pages, None if pair_status is None else _want("pair_status", pair_status, torch.int32, (n,), dev))


# ------------------------------------------------------ page pool (host side)
def _host(a, dtype):
    import numpy as np
    a = np.ascontiguousarray(a, dtype=dtype)
    return a, a.ctypes.data_as(ctypes.c_void_p)


class PagePool:
    """Host page pool with reference counts, generation tags and a block-hash
    prefix cache (``pfkv_pool_*``).  Arrays are numpy, on the host."""

    def __init__(self, num_pages: int, page_size: int):
        self._h = load().pfkv_pool_create(num_pages, page_size)
        if not self._h:
            raise PfkvError("pool_create", -1, last_error())
        self.num_pages, self.page_size = num_pages, page_size

    def close(self):
        if self._h:
            load().pfkv_pool_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __reduce_ex__(self, protocol):
        raise TypeError("a PagePool is not copied or pickled: the copy would free the same pool")

    def num_free(self) -> int:
        return int(load().pfkv_pool_num_free(self._h))

    def refcount(self, page: int) -> int:
        return int(load().pfkv_pool_refcount(self._h, page))

    def page_tags(self):
        import numpy as np
        out = np.zeros(self.num_pages, np.uint32)
        _check("pool_page_tags", load().pfkv_pool_page_tags(self._h, out.ctypes.data_as(ctypes.c_void_p)))
        return out

    def map_request(self, tokens, max_pages: int):
        """-> (block-table row int32 [max_pages], tags uint32 [max_pages], cached token count)."""
        import numpy as np
        t, tp = _host(tokens, np.int32)
        row = np.zeros(max_pages, np.int32)
        tags = np.zeros(max_pages, np.uint32)
        cached = ctypes.c_int(0)
        rc = load().pfkv_pool_map_request(self._h, tp, t.shape[0], row.ctypes.data_as(ctypes.c_void_p),
                                          tags.ctypes.data_as(ctypes.c_void_p), max_pages, ctypes.byref(cached))
        _check("pool_map_request", rc)
        return row, tags, int(cached.value)

    def release(self, row, n_pages: int):
        import numpy as np
        r, rp = _host(row, np.int32)
        if not 0 <= n_pages <= r.shape[0]:
            raise ValueError(f"n_pages {n_pages} outside the row's {r.shape[0]} entries")
        _check("pool_release", load().pfkv_pool_release(self._h, rp, n_pages))

    def fork(self, row, n_pages: int):
        """One more holder for each of the row's first n_pages pages."""
        import numpy as np
        r, rp = _host(row, np.int32)
        if not 0 <= n_pages <= r.shape[0]:
            raise ValueError(f"n_pages {n_pages} outside the row's {r.shape[0]} entries")
        _check("pool_fork", load().pfkv_pool_fork(self._h, rp, n_pages))

    @staticmethod
    def _row(row, tags):
        """Addresses of a row and its tags, which the call changes in place."""
        import numpy as np
        for name, a, dtype in (("row", row, np.int32), ("tags", tags, np.uint32)):
            if not isinstance(a, np.ndarray) or a.dtype != dtype or a.ndim != 1 or not a.flags.c_contiguous or not a.flags.writeable:
                raise ValueError(f"{name}: expected a writable contiguous {np.dtype(dtype)} array, which is changed in place")
        if row.shape != tags.shape:
            raise ValueError("row and tags: expected the same length")
        return row.ctypes.data_as(ctypes.c_void_p), tags.ctypes.data_as(ctypes.c_void_p), row.shape[0]

    def resize(self, row, tags, n_tokens: int):
        """Grow or cut a request (row and tags of map_request, changed in
        place) to the pages of n_tokens tokens."""
        rp, tp, n = self._row(row, tags)
        _check("pool_resize", load().pfkv_pool_resize(self._h, rp, tp, n, _count("n_tokens", n_tokens)))

    def make_writable(self, row, tags, first_token: int):
        """Give a request (row and tags changed in place) pages of its own from
        token first_token on -> int32 [0 or 1][2], the page to copy before it
        is written (copy_pages, which says what pairs may share a call)."""
        import numpy as np
        rp, tp, n = self._row(row, tags)
        pair, k = np.zeros((1, 2), np.int32), ctypes.c_int(0)
        _check("pool_make_writable", load().pfkv_pool_make_writable(
            self._h, rp, tp, n, _count("first_token", first_token), pair.ctypes.data_as(ctypes.c_void_p), ctypes.byref(k)))
        return pair[:k.value]

    def compact(self, max_moves: int = None):
        """Move held pages to the lowest free ids -> (int32 [n][2] pages to copy,
        with a copy_pages of their own; int32 [num_pages] new id of every page).
        The holders' rows follow:
        row[row >= 0] = remap[row[row >= 0]], tags from page_tags()."""
        import numpy as np
        most = self.num_pages if max_moves is None else min(max_moves, self.num_pages)
        pairs, remap = np.zeros((max(most, 0), 2), np.int32), np.zeros(self.num_pages, np.int32)
        k = ctypes.c_int64(0)
        _check("pool_compact", load().pfkv_pool_compact(self._h, most, pairs.ctypes.data_as(ctypes.c_void_p),
                                                        remap.ctypes.data_as(ctypes.c_void_p), ctypes.byref(k)))
        return pairs[:k.value].copy(), remap


def block_hash(parent: int, tokens) -> int:
    import numpy as np
    t, tp = _host(tokens, np.int32)
    return int(load().pfkv_block_hash(ctypes.c_uint64(parent), tp, t.shape[0]))


def slots_from_table(row, page_size: int, first_token: int, n_tokens: int):
    import numpy as np
    r, rp = _host(row, np.int32)
    out = np.zeros(n_tokens, np.int64)
    _check("slots_from_table", load().pfkv_slots_from_table(rp, r.shape[0], page_size, first_token, n_tokens,
                                                            out.ctypes.data_as(ctypes.c_void_p)))
    return out
