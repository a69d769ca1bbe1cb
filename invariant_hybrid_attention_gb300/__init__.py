"""Python binding of the g4attn C ABI (include/g4attn.h): argument marshalling only.

Every step of the attention path runs in the CUDA kernels of libg4attn.so, loaded with
ctypes from this directory. There is no Python, PyTorch or CPU implementation to fall back
on: if the library is missing or a call fails, an exception says so.

The functions take torch tensors (device memory and streams come from PyTorch) and pass
their raw pointers; names follow the C entry points.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libg4attn.so")

G4_OK, G4_ERR_INVALID, G4_ERR_UNSUPPORTED, G4_ERR_CUDA, G4_ERR_TIMEOUT, G4_ERR_DEVICE, G4_ERR_SCRATCH = range(7)
G4_SLIDING, G4_GLOBAL = 0, 1
PAGE_SIZE = 16
DECODE_STATIC_SCRATCH_BYTES = 32 << 20   # the static scratch of g4attn_decode_static, per device

EXPORTS = ("g4attn_rope_apply", "g4attn_prefill", "g4attn_prefill_stage", "g4attn_prefill_attend",
           "g4attn_prefill_normed", "g4attn_prefill_vision", "g4attn_kv_append_normed", "g4attn_decode_normed",
           "g4attn_decode_exact", "g4attn_decode_exact_workspace_bytes",
           "g4attn_kv_append", "g4attn_decode_workspace_bytes",
           "g4attn_decode", "g4attn_decode_static", "g4attn_provenance", "g4attn_status_sync", "g4attn_status_string",
           "g4attn_set_wait_limit_ns", "g4attn_wait_limit_ns", "g4attn_prefill_partial", "g4attn_merge_partials",
           "g4attn_kv8_page_bytes", "g4attn_kv8_append", "g4attn_kv8_unpack", "g4attn_kv8_prefill",
           "g4attn_kv8_decode_workspace_bytes", "g4attn_kv8_decode", "g4attn_evict_pages",
           "g4attn_kv4_page_bytes", "g4attn_kv4_append", "g4attn_kv4_unpack", "g4attn_kv4_prefill",
           "g4attn_kv4_decode_workspace_bytes", "g4attn_kv4_decode", "g4attn_plan_pages")
DEFAULT_WAIT_LIMIT_NS = 2_000_000_000   # the kernels' bounded waits give up after 2 s by default


class g4attn_layer(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("window", ctypes.c_int32), ("rope_theta", ctypes.c_float),
                ("rope_partial", ctypes.c_float), ("softmax_scale", ctypes.c_float), ("kv_shared", ctypes.c_int32)]


class g4attn_norms(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("v_norm", ctypes.c_int32),
                ("eps", ctypes.c_float)]


class g4attn_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_rot", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32)]
    tensors = None   # make_cache: what k, v and k_rot point into
    room = None      # see _room16


class g4attn_cache8(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32)]
    tensor = None    # make_cache8: what pages points into (None: a raw address)
    room = None      # its bytes and its device


class g4attn_cache4(ctypes.Structure):
    _fields_ = g4attn_cache8._fields_
    tensor = None
    room = None


class g4attn_page_group(ctypes.Structure):
    _fields_ = [("window", ctypes.c_int32), ("num_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32)] + [
        (name, ctypes.c_void_p) for name in ("free_pages", "pool", "out_pool", "page_table", "first_page", "out_first_page",
                                             "lost", "out_lost", "freed", "n_freed", "seq_len", "slots", "out_n_freed")]
    tensors = None   # make_page_group: what the fields point into
    room = None      # its requests, rows (None: no slots) and device


class G4Error(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} (status {status})")
        self.status = status


_lib = None


def load(path: Optional[str] = None):
    """Loads libg4attn.so (built by __graft_entry__.build() or build.build()). Raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libg4attn.so not found at {p}: build it first (the library has no fallback path)")
    lib = ctypes.CDLL(p)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    L, C = ctypes.POINTER(g4attn_layer), ctypes.POINTER(g4attn_cache)
    N, C8 = ctypes.POINTER(g4attn_norms), ctypes.POINTER(g4attn_cache8)
    C4, G = ctypes.POINTER(g4attn_cache4), ctypes.POINTER(g4attn_page_group)
    sigs = {
        "g4attn_rope_apply": (I32, [L, P, P, I32, I32, P, P]),
        "g4attn_prefill": (I32, [L, P, P, P, I32, P, P, P, I32, C, P, I32, P, P]),
        "g4attn_prefill_stage": (I32, [L, P, P, P, I32, P, P, P, I32, C, P, I32, P, P]),
        "g4attn_prefill_attend": (I32, [L, P, I32, P, P, P, I32, C, P, I32, P, P]),
        "g4attn_prefill_normed": (I32, [L, N, P, P, P, I32, P, P, P, I32, C, P, I32, P, P]),
        "g4attn_prefill_vision": (I32, [L, N, P, P, P, I32, P, P, P, I32, P, C, P, I32, P, P]),
        "g4attn_kv_append_normed": (I32, [L, N, P, P, I32, P, P, P, I32, C, P, I32, P]),
        "g4attn_decode_normed": (I32, [L, N, P, P, P, P, I32, C, P, I32, P, P, SZ, P]),
        "g4attn_decode_exact": (I32, [L, N, P, P, P, P, I32, C, P, I32, P, P, SZ, P]),
        "g4attn_decode_exact_workspace_bytes": (SZ, [I32]),
        "g4attn_kv_append": (I32, [L, P, P, I32, P, P, P, I32, C, P, I32, P]),
        "g4attn_decode_workspace_bytes": (SZ, [L, I32, I32]),
        "g4attn_decode": (I32, [L, P, P, P, P, I32, C, P, I32, P, P, SZ, P]),
        "g4attn_decode_static": (I32, [L, P, P, P, P, I32, C, P, I32, P, P]),
        "g4attn_provenance": (I32, [L, ctypes.c_char_p, SZ]),
        "g4attn_status_sync": (I32, [P]),
        "g4attn_status_string": (ctypes.c_char_p, [I32]),
        "g4attn_set_wait_limit_ns": (I32, [ctypes.c_uint64]),
        "g4attn_wait_limit_ns": (ctypes.c_uint64, []),
        "g4attn_prefill_partial": (I32, [L, P, I32, P, P, P, I32, P, P, C, P, I32, P, P, P]),
        "g4attn_merge_partials": (I32, [L, I32, ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(ctypes.c_void_p),
                                        I32, P, P, I32, P, P]),
        "g4attn_kv8_page_bytes": (SZ, [L]),
        "g4attn_kv8_append": (I32, [L, N, P, P, I32, P, P, P, I32, C8, P, I32, P]),
        "g4attn_kv8_unpack": (I32, [L, P, P, I32, C8, P, C, P, I32, P]),
        "g4attn_kv8_prefill": (I32, [L, N, P, P, P, I32, P, P, P, I32, P, C8, P, C, P, I32, P, P]),
        "g4attn_kv8_decode_workspace_bytes": (SZ, [L, I32, I32, I32]),
        "g4attn_kv8_decode": (I32, [L, N, P, P, P, P, P, I32, C8, P, I32, P, P, P, SZ, P]),
        "g4attn_evict_pages": (I32, [P, P, P, I32, I32, I32, I32, I32, P, P, P, P, P, P]),
        "g4attn_kv4_page_bytes": (SZ, [L]),
        "g4attn_kv4_append": (I32, [L, N, P, P, I32, P, P, P, I32, C4, P, I32, P]),
        "g4attn_kv4_unpack": (I32, [L, P, P, I32, C4, P, C, P, I32, P]),
        "g4attn_kv4_prefill": (I32, [L, N, P, P, P, I32, P, P, P, I32, P, C4, P, C, P, I32, P, P]),
        "g4attn_kv4_decode_workspace_bytes": (SZ, [L, I32, I32, I32]),
        "g4attn_kv4_decode": (I32, [L, N, P, P, P, P, P, I32, C4, P, I32, P, P, P, SZ, P]),
        "g4attn_plan_pages": (I32, [P, P, I32, I32, G, I32, P, P, P, P, P, P]),
    }
    for name, (res, args) in sigs.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    _lib = lib
    return lib


def status_string(status: int) -> str:
    try:
        return load().g4attn_status_string(int(status)).decode()
    except Exception:  # noqa: BLE001 - used while formatting errors
        return "unknown"


def sliding_layer(window: int = 1024, softmax_scale: Optional[float] = None, tp: int = 1) -> g4attn_layer:
    """The sliding layer, or (tp > 1) one tensor-parallel rank's slice of it: 32/tp query heads,
    16/tp KV heads."""
    return g4attn_layer(G4_SLIDING, 32 // tp, 16 // tp, 256, int(window), 1.0e4, 1.0,
                        1.0 / math.sqrt(256) if softmax_scale is None else float(softmax_scale), 0)


def global_layer(softmax_scale: Optional[float] = None, tp: int = 1) -> g4attn_layer:
    """The global K==V layer, or (tp > 1) one rank's slice: 32/tp query heads and max(1, 4/tp) KV
    heads (at tp = 8 two ranks hold the same KV head)."""
    return g4attn_layer(G4_GLOBAL, 32 // tp, max(1, 4 // tp), 512, 0, 1.0e6, 0.25,
                        1.0 / math.sqrt(512) if softmax_scale is None else float(softmax_scale), 1)


def make_cache(k, v, num_pages: int, k_rot=None) -> g4attn_cache:
    cache = g4attn_cache(_ptr(k), _ptr(v), _ptr(k_rot), int(num_pages), PAGE_SIZE)
    cache.tensors = (k, v, k_rot)
    return cache


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        if torch.cuda.is_initialized():   # the current stream's address without a Stream object: 0.3 us, not 3
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _check(status: int, what: str):
    if status != G4_OK:
        raise G4Error(status, what)


def g4attn_rope_apply(layer: g4attn_layer, x, pos, out=None, stream=None):
    """out[r][h] = RoPE(x[r][h], pos[r]); x [T, H, D] bf16, pos int32 [T] (device)."""
    out = x if out is None else out
    T, H = int(x.shape[0]), int(x.shape[1])
    _check(load().g4attn_rope_apply(ctypes.byref(layer), _ptr(x), _ptr(pos), T, H, _ptr(out), _stream(stream)),
           "g4attn_rope_apply")
    return out


def g4attn_kv_append(layer, k, v, q_start, q_len, ctx_start, cache: g4attn_cache, page_table, stream=None):
    T, B = int(k.shape[0]), int(q_start.shape[0])
    _check(load().g4attn_kv_append(ctypes.byref(layer), _ptr(k), _ptr(v), T, _ptr(q_start), _ptr(q_len),
                                   _ptr(ctx_start), B, ctypes.byref(cache), _ptr(page_table),
                                   int(page_table.shape[1]), _stream(stream)), "g4attn_kv_append")


def g4attn_prefill(layer, q, k, v, q_start, q_len, ctx_start, cache: g4attn_cache, page_table, out, stream=None):
    T, B = int(q.shape[0]), int(q_start.shape[0])
    _check(load().g4attn_prefill(ctypes.byref(layer), _ptr(q), _ptr(k), _ptr(v), T, _ptr(q_start), _ptr(q_len),
                                 _ptr(ctx_start), B, ctypes.byref(cache), _ptr(page_table), int(page_table.shape[1]),
                                 _ptr(out), _stream(stream)), "g4attn_prefill")
    return out


def g4attn_prefill_stage(layer, q, k, v, q_start, q_len, ctx_start, cache: g4attn_cache, page_table, out,
                         stream=None):
    T, B = int(q.shape[0]), int(q_start.shape[0])
    _check(load().g4attn_prefill_stage(ctypes.byref(layer), _ptr(q), _ptr(k), _ptr(v), T, _ptr(q_start),
                                       _ptr(q_len), _ptr(ctx_start), B, ctypes.byref(cache), _ptr(page_table),
                                       int(page_table.shape[1]), _ptr(out), _stream(stream)), "g4attn_prefill_stage")
    return out


def g4attn_prefill_attend(layer, q, q_start, q_len, ctx_start, cache: g4attn_cache, page_table, out, stream=None):
    """The attention step of a prefill: q the raw query rows (rotated in the kernel), or None when
    g4attn_prefill_stage staged the roped queries in out."""
    T, B = int(out.shape[0]), int(q_start.shape[0])
    _check(load().g4attn_prefill_attend(ctypes.byref(layer), _ptr(q), T, _ptr(q_start), _ptr(q_len), _ptr(ctx_start),
                                        B, ctypes.byref(cache), _ptr(page_table), int(page_table.shape[1]),
                                        _ptr(out), _stream(stream)), "g4attn_prefill_attend")
    return out


def g4attn_decode_workspace_bytes(layer, B: int, max_pages: int) -> int:
    return int(load().g4attn_decode_workspace_bytes(ctypes.byref(layer), int(B), int(max_pages)))


def g4attn_decode(layer, q, k_new, v_new, seq_len, cache: g4attn_cache, page_table, out, workspace, stream=None):
    B = int(q.shape[0])
    nbytes = workspace.numel() * workspace.element_size()
    _check(load().g4attn_decode(ctypes.byref(layer), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(seq_len), B,
                                ctypes.byref(cache), _ptr(page_table), int(page_table.shape[1]), _ptr(out),
                                _ptr(workspace), nbytes, _stream(stream)), "g4attn_decode")
    return out


def g4attn_decode_static(layer, q, k_new, v_new, seq_len, cache: g4attn_cache, page_table, out, stream=None):
    """g4attn_decode with the library's static scratch instead of a workspace: for callers that
    cannot allocate device memory at decode time. Allocates nothing (this wrapper included).
    Raises G4Error(G4_ERR_SCRATCH) when the step needs more than DECODE_STATIC_SCRATCH_BYTES.
    Calls that may overlap on the GPU (unordered streams) share the scratch and race."""
    B = int(q.shape[0])
    _check(load().g4attn_decode_static(ctypes.byref(layer), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(seq_len), B,
                                       ctypes.byref(cache), _ptr(page_table), int(page_table.shape[1]), _ptr(out),
                                       _stream(stream)), "g4attn_decode_static")
    return out


def g4attn_provenance(layer) -> str:
    buf = ctypes.create_string_buffer(2048)
    n = load().g4attn_provenance(ctypes.byref(layer), buf, len(buf))
    if n < 0:
        raise G4Error(G4_ERR_UNSUPPORTED, "g4attn_provenance")
    return buf.value.decode()


def g4attn_status_sync(stream=None) -> int:
    return int(load().g4attn_status_sync(_stream(stream)))


def make_norms(q_weight=None, k_weight=None, v_norm: bool = False, eps: float = 1e-6) -> g4attn_norms:
    """Per-head norm arguments: q_weight / k_weight are bf16 [head_dim] device tensors or None."""
    return g4attn_norms(_ptr(q_weight), _ptr(k_weight), 1 if v_norm else 0, float(eps))


def g4attn_prefill_normed(layer, norms: g4attn_norms, q, k, v, q_start, q_len, ctx_start, cache: g4attn_cache,
                          page_table, out, stream=None):
    T, B = int(q.shape[0]), int(q_start.shape[0])
    _check(load().g4attn_prefill_normed(ctypes.byref(layer), ctypes.byref(norms), _ptr(q), _ptr(k), _ptr(v), T,
                                        _ptr(q_start), _ptr(q_len), _ptr(ctx_start), B, ctypes.byref(cache),
                                        _ptr(page_table), int(page_table.shape[1]), _ptr(out), _stream(stream)),
           "g4attn_prefill_normed")
    return out


def g4attn_prefill_vision(layer, norms, q, k, v, q_start, q_len, ctx_start, span, cache: g4attn_cache,
                          page_table, out, stream=None):
    """g4attn_prefill_normed with image spans: span is an int32 [T, 2] device tensor (or None),
    row t's image [s0, s1) of absolute positions, s1 <= s0 for a text row. norms may be None."""
    T, B = int(q.shape[0]), int(q_start.shape[0])
    nrm = None if norms is None else ctypes.byref(norms)
    _check(load().g4attn_prefill_vision(ctypes.byref(layer), nrm, _ptr(q), _ptr(k), _ptr(v), T,
                                        _ptr(q_start), _ptr(q_len), _ptr(ctx_start), B, _ptr(span),
                                        ctypes.byref(cache), _ptr(page_table), int(page_table.shape[1]), _ptr(out),
                                        _stream(stream)),
           "g4attn_prefill_vision")
    return out


def g4attn_kv_append_normed(layer, norms: g4attn_norms, k, v, q_start, q_len, ctx_start, cache: g4attn_cache,
                            page_table, stream=None):
    T, B = int(k.shape[0]), int(q_start.shape[0])
    _check(load().g4attn_kv_append_normed(ctypes.byref(layer), ctypes.byref(norms), _ptr(k), _ptr(v), T,
                                          _ptr(q_start), _ptr(q_len), _ptr(ctx_start), B, ctypes.byref(cache),
                                          _ptr(page_table), int(page_table.shape[1]), _stream(stream)),
           "g4attn_kv_append_normed")


def g4attn_decode_normed(layer, norms: g4attn_norms, q, k_new, v_new, seq_len, cache: g4attn_cache, page_table,
                         out, workspace, stream=None):
    B = int(q.shape[0])
    _check(load().g4attn_decode_normed(ctypes.byref(layer), ctypes.byref(norms), _ptr(q), _ptr(k_new), _ptr(v_new),
                                       _ptr(seq_len), B, ctypes.byref(cache), _ptr(page_table),
                                       int(page_table.shape[1]), _ptr(out), _ptr(workspace),
                                       int(workspace.numel() * workspace.element_size()), _stream(stream)),
           "g4attn_decode_normed")
    return out


def g4attn_decode_exact_workspace_bytes(B: int) -> int:
    return int(load().g4attn_decode_exact_workspace_bytes(int(B)))


def g4attn_decode_exact(layer, norms, q, k_new, v_new, seq_len, cache: g4attn_cache, page_table, out, workspace,
                        stream=None):
    """One decode step through the prefill kernels: the rows' bits equal a prefill's. norms may be
    None; workspace holds at least g4attn_decode_exact_workspace_bytes(B) bytes."""
    B = int(q.shape[0])
    nrm = None if norms is None else ctypes.byref(norms)
    _check(load().g4attn_decode_exact(ctypes.byref(layer), nrm, _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(seq_len), B,
                                      ctypes.byref(cache), _ptr(page_table), int(page_table.shape[1]), _ptr(out),
                                      _ptr(workspace), int(workspace.numel() * workspace.element_size()),
                                      _stream(stream)),
           "g4attn_decode_exact")
    return out


def g4attn_set_wait_limit_ns(ns: int) -> None:
    """Bound of every protocol wait in kernels launched from now on (0 .. 2e9 ns; default 2 s)."""
    _check(load().g4attn_set_wait_limit_ns(int(ns)), "g4attn_set_wait_limit_ns")


def g4attn_wait_limit_ns() -> int:
    return int(load().g4attn_wait_limit_ns())


def g4attn_prefill_partial(layer, q, q_start, q_len, ctx_start, key_begin, key_end, cache: g4attn_cache, page_table,
                           o_part, ml_part, stream=None):
    """A global layer's attention restricted to each sequence's keys key_begin .. key_end-1 (int32 [B]
    device tensors): writes the un-normalised fp32 output o_part [T, Hq, 512] and the softmax state
    ml_part [T, Hq, 2] (max in log2 units, sum) of every sequence row."""
    T, B = int(q.shape[0]), int(q_start.shape[0])
    _check(load().g4attn_prefill_partial(ctypes.byref(layer), _ptr(q), T, _ptr(q_start), _ptr(q_len), _ptr(ctx_start),
                                         B, _ptr(key_begin), _ptr(key_end), ctypes.byref(cache), _ptr(page_table),
                                         int(page_table.shape[1]), _ptr(o_part), _ptr(ml_part), _stream(stream)),
           "g4attn_prefill_partial")


def g4attn_merge_partials(layer, o_parts, ml_parts, q_start, q_len, out, stream=None):
    """Merges the partials (lists of device tensors, in rank order) into out [T, Hq, 512] bf16."""
    n = len(o_parts)
    arr_o = (ctypes.c_void_p * n)(*[_ptr(t) for t in o_parts])
    arr_m = (ctypes.c_void_p * n)(*[_ptr(t) for t in ml_parts])
    T, B = int(out.shape[0]), int(q_start.shape[0])
    _check(load().g4attn_merge_partials(ctypes.byref(layer), n, arr_o, arr_m, T, _ptr(q_start), _ptr(q_len), B,
                                        _ptr(out), _stream(stream)), "g4attn_merge_partials")
    return out


# ---- the 8-bit paged cache ----------------------------------------------------------------------------
# The kernels take dense tensors of one type on the current device; these calls check that, since a
# raw pointer cannot say otherwise, and that a cache's tensors hold the pages that it is said to have. A small
# step's kernels run for 6 us, so the checks are one pass over the arguments, with torch's names looked up once,
# and what a cache descriptor points into is looked at once per descriptor.

_names = None   # (bfloat16, int32, float32, the current device, a device's current raw stream)


def _torch_names():
    global _names
    import torch
    _names = (torch.bfloat16, torch.int32, torch.float32, torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)
    return _names


def _make_quant(what: str, kind, pages, num_pages: int):
    cache = kind(_ptr(pages), int(num_pages), PAGE_SIZE)
    if not isinstance(pages, int):
        if not pages.is_contiguous():
            raise ValueError(f"{what}: pages must be dense")
        cache.tensor, cache.room = pages, (pages.nbytes, pages.get_device())
    return cache


def make_cache8(pages, num_pages: int) -> g4attn_cache8:
    """pages: a dense tensor (or a raw address, which nothing checks) of num_pages pages."""
    return _make_quant("make_cache8", g4attn_cache8, pages, num_pages)


# bytes of a page and KV head of a quantised cache, by its kind and head_dim
_BLOCK = {g4attn_cache8: {256: 8224, 512: 10272}, g4attn_cache4: {256: 4368, 512: 5456}}


def _room16(what: str, cache: g4attn_cache):
    """Bytes that k and v each hold at least, those of k_rot, and the one device of all three (-2: several, None: raw
    addresses alone); kept in the descriptor."""
    given = [t for t in cache.tensors or () if t is not None and not isinstance(t, int)]
    if not all(t.is_contiguous() for t in given):
        raise ValueError(f"{what}: the bf16 cache's tensors must be dense")
    sizes = [1 << 62 if t is None or isinstance(t, int) else t.nbytes for t in cache.tensors or (None,) * 3]
    at = {t.get_device() for t in given}
    cache.room = (min(sizes[0], sizes[1]), sizes[2], None if not at else at.pop() if len(at) == 1 else -2)
    return cache.room


def _refuse_pool(what: str, name: str, room, need, at, here: int):
    if any(n > r for n, r in zip(need, room)):
        raise ValueError(f"{what}: {name} has {room} bytes, its pages take {need}")
    place = {-1: "the CPU", -2: "several devices"}.get(at, f"cuda:{at}")
    raise ValueError(f"{what}: {name} is on {place}, not on the current CUDA device")


def _pointers(what: str, stream, specs, layer=None, cache=None, bf16_cache=None):
    """The addresses of a call's tensors, given as (name, tensor, dtype, shape), and of its stream (None: the
    current one). None and raw addresses pass unchecked; the first one is a tensor. cache, bf16_cache: descriptors
    whose tensors have to hold their pages of the layer's heads, on the same device."""
    _, _, _, device, raw_stream = _names
    here = specs[0][1].get_device()
    if here >= 0:
        here = device()
    if cache is not None and cache.room is not None:
        room, at = cache.room
        need = cache.num_pages * layer.n_kv_heads * _BLOCK[cache.__class__].get(layer.head_dim, 0)
        if need > room or (at != here and here >= 0):
            _refuse_pool(what, f"the {8 if cache.__class__ is g4attn_cache8 else 4}-bit cache", (room,), (need,), at, here)
    if bf16_cache is not None:
        room, rot_room, at = bf16_cache.room or _room16(what, bf16_cache)
        blocks = bf16_cache.num_pages * layer.n_kv_heads
        need = blocks * 32 * layer.head_dim
        if need > room or blocks * 4096 > rot_room or (at != here and here >= 0 and at is not None):
            _refuse_pool(what, "the bf16 cache", (room, rot_room), (need, blocks * 4096), at, here)
    out = []
    for name, t, dtype, shape in specs:
        if t is None or t.__class__ is int:
            out.append(t)
            continue
        if t.dtype is not dtype or t.shape != shape or t.get_device() != here or here < 0 or not t.is_contiguous():
            _refuse(what, specs, here)
        out.append(t.data_ptr())
    out.append(raw_stream(here) if stream is None else _stream(stream))
    return out


def _refuse(what: str, specs, here: int):
    given = [x for x in specs if x[1] is not None and x[1].__class__ is not int]
    for name, t, dtype, shape in given:
        if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{what}: {name} must be a dense {dtype} tensor of shape {tuple(shape)}, got "
                             f"{t.dtype} {tuple(t.shape)}{'' if t.is_contiguous() else ' (strided)'}")
    name, t = next((name, t) for name, t, _, _ in given if here < 0 or t.get_device() != here)
    raise ValueError(f"{what}: {name} is on {t.device}, not on the current CUDA device")


def _opt(s):
    return None if s is None else ctypes.byref(s)


def g4attn_kv8_page_bytes(layer) -> int:
    return int(load().g4attn_kv8_page_bytes(ctypes.byref(layer)))


def g4attn_kv8_append(layer, norms, k, v, q_start, q_len, ctx_start, cache: g4attn_cache8, page_table, stream=None):
    """g4attn_kv_append_normed into an 8-bit cache; norms may be None. Rows are turned by their held index: a
    sequence that lost pages is continued by g4attn_kv8_decode with pos instead."""
    bf, i32, _, _, _ = _names or _torch_names()
    T, B, width = k.shape[0], q_start.shape[0], page_table.shape[-1]
    kv, rows = (T, layer.n_kv_heads, layer.head_dim), (B,)
    k, v, q_start, q_len, ctx_start, page_table, stream = _pointers("g4attn_kv8_append", stream, (
        ("k", k, bf, kv), ("v", v, bf, kv), ("q_start", q_start, i32, rows), ("q_len", q_len, i32, rows),
        ("ctx_start", ctx_start, i32, rows), ("page_table", page_table, i32, (B, width))),
        layer, cache)
    _check((_lib or load()).g4attn_kv8_append(ctypes.byref(layer), _opt(norms), k, v, T, q_start, q_len, ctx_start, B,
                                              ctypes.byref(cache), page_table, width, stream), "g4attn_kv8_append")


def g4attn_kv8_unpack(layer, key_begin, key_end, cache: g4attn_cache8, page_table, out: g4attn_cache, out_table,
                      stream=None):
    """Reads keys key_begin[b] .. key_end[b]-1 back as bf16 pages of `out` (through out_table)."""
    _, i32, _, _, _ = _names or _torch_names()
    B, width = key_begin.shape[0], page_table.shape[-1]
    rows, table = (B,), (B, width)
    key_begin, key_end, page_table, out_table, stream = _pointers("g4attn_kv8_unpack", stream, (
        ("key_begin", key_begin, i32, rows), ("key_end", key_end, i32, rows), ("page_table", page_table, i32, table),
        ("out_table", out_table, i32, table)), layer, cache, out)
    _check((_lib or load()).g4attn_kv8_unpack(ctypes.byref(layer), key_begin, key_end, B, ctypes.byref(cache),
                                              page_table, ctypes.byref(out), out_table, width, stream),
           "g4attn_kv8_unpack")


def g4attn_kv8_prefill(layer, norms, q, k, v, q_start, q_len, ctx_start, cache: g4attn_cache8, page_table,
                       scratch: g4attn_cache, scratch_table, out, span=None, stream=None):
    """A prefill (or chunk) over an 8-bit cache; scratch: a bf16 cache for the keys its rows see. Not for
    sequences that lost pages (see g4attn_kv8_append)."""
    bf, i32, _, _, _ = _names or _torch_names()
    T, B, width = q.shape[0], q_start.shape[0], page_table.shape[-1]
    qo, kv = (T, layer.n_q_heads, layer.head_dim), (T, layer.n_kv_heads, layer.head_dim)
    rows, table = (B,), (B, width)
    qp, k, v, q_start, q_len, ctx_start, span, page_table, scratch_table, op, stream = _pointers(
        "g4attn_kv8_prefill", stream, (
            ("q", q, bf, qo), ("k", k, bf, kv), ("v", v, bf, kv), ("q_start", q_start, i32, rows),
            ("q_len", q_len, i32, rows), ("ctx_start", ctx_start, i32, rows), ("span", span, i32, (T, 2)),
            ("page_table", page_table, i32, table), ("scratch_table", scratch_table, i32, table), ("out", out, bf, qo)),
        layer, cache, scratch)
    _check((_lib or load()).g4attn_kv8_prefill(ctypes.byref(layer), _opt(norms), qp, k, v, T, q_start, q_len, ctx_start,
                                               B, span, ctypes.byref(cache), page_table, ctypes.byref(scratch),
                                               scratch_table, width, op, stream), "g4attn_kv8_prefill")
    return out


def g4attn_kv8_decode_workspace_bytes(layer, B: int, max_pages: int, page_weights: bool = False) -> int:
    return int(load().g4attn_kv8_decode_workspace_bytes(ctypes.byref(layer), int(B), int(max_pages),
                                                        1 if page_weights else 0))


def g4attn_kv8_decode(layer, norms, q, k_new, v_new, seq_len, cache: g4attn_cache8, page_table, out, workspace,
                      pos=None, page_weights=None, stream=None):
    """One decode step over an 8-bit cache. k_new None: the newest token is in the cache already; pos:
    RoPE positions of sequences that lost pages; page_weights: accumulated per page (global layers)."""
    bf, i32, f32, _, _ = _names or _torch_names()
    B, width = q.shape[0], page_table.shape[-1]
    qo, kv = (B, layer.n_q_heads, layer.head_dim), (B, layer.n_kv_heads, layer.head_dim)
    rows, table = (B,), (B, width)
    q, k_new, v_new, seq_len, pos, page_table, page_weights, op, work, stream = _pointers("g4attn_kv8_decode", stream, (
        ("q", q, bf, qo), ("k_new", k_new, bf, kv), ("v_new", v_new, bf, kv), ("seq_len", seq_len, i32, rows),
        ("pos", pos, i32, rows), ("page_table", page_table, i32, table), ("page_weights", page_weights, f32, table),
        ("out", out, bf, qo), ("workspace", workspace, workspace.dtype, workspace.shape)),
        layer, cache)
    _check((_lib or load()).g4attn_kv8_decode(ctypes.byref(layer), _opt(norms), q, k_new, v_new, seq_len, pos, B,
                                              ctypes.byref(cache), page_table, width, page_weights, op, work,
                                              workspace.nbytes, stream), "g4attn_kv8_decode")
    return out


def g4attn_evict_pages(seq_len, page_table, page_weights, keep_pages: int, first_pages: int, last_pages: int,
                       out_seq_len, out_table, out_weights, freed, n_freed, stream=None):
    """Evicts each sequence's lightest pages down to keep_pages; the out_ tensors may be the inputs. The sequence
    goes on by g4attn_kv8_decode with pos."""
    _, i32, f32, _, _ = _names or _torch_names()
    B, width = seq_len.shape[0], page_table.shape[-1]
    rows, table = (B,), (B, width)
    seq_len, page_table, page_weights, out_seq_len, out_table, out_weights, freed, n_freed, stream = _pointers(
        "g4attn_evict_pages", stream, (
            ("seq_len", seq_len, i32, rows), ("page_table", page_table, i32, table),
            ("page_weights", page_weights, f32, table), ("out_seq_len", out_seq_len, i32, rows),
            ("out_table", out_table, i32, table), ("out_weights", out_weights, f32, table),
            ("freed", freed, i32, table), ("n_freed", n_freed, i32, rows)))
    _check((_lib or load()).g4attn_evict_pages(seq_len, page_table, page_weights, B, width, int(keep_pages),
                                               int(first_pages), int(last_pages), out_seq_len, out_table, out_weights,
                                               freed, n_freed, stream), "g4attn_evict_pages")


# ---- the 4-bit paged cache ------------------------------------------------------------------------------

def make_cache4(pages, num_pages: int) -> g4attn_cache4:
    """pages: a dense tensor (or a raw address, which nothing checks) of num_pages pages."""
    return _make_quant("make_cache4", g4attn_cache4, pages, num_pages)


def g4attn_kv4_page_bytes(layer) -> int:
    return int(load().g4attn_kv4_page_bytes(ctypes.byref(layer)))


def g4attn_kv4_append(layer, norms, k, v, q_start, q_len, ctx_start, cache: g4attn_cache4, page_table, stream=None):
    """g4attn_kv_append_normed into a 4-bit cache; norms may be None. Rows are turned by their held index: a
    sequence that lost pages is continued by g4attn_kv4_decode with pos instead."""
    bf, i32, _, _, _ = _names or _torch_names()
    T, B, width = k.shape[0], q_start.shape[0], page_table.shape[-1]
    kv, rows = (T, layer.n_kv_heads, layer.head_dim), (B,)
    k, v, q_start, q_len, ctx_start, page_table, stream = _pointers("g4attn_kv4_append", stream, (
        ("k", k, bf, kv), ("v", v, bf, kv), ("q_start", q_start, i32, rows), ("q_len", q_len, i32, rows),
        ("ctx_start", ctx_start, i32, rows), ("page_table", page_table, i32, (B, width))),
        layer, cache)
    _check((_lib or load()).g4attn_kv4_append(ctypes.byref(layer), _opt(norms), k, v, T, q_start, q_len, ctx_start, B,
                                              ctypes.byref(cache), page_table, width, stream), "g4attn_kv4_append")


def g4attn_kv4_unpack(layer, key_begin, key_end, cache: g4attn_cache4, page_table, out: g4attn_cache, out_table,
                      stream=None):
    """Reads keys key_begin[b] .. key_end[b]-1 back as bf16 pages of `out` (through out_table)."""
    _, i32, _, _, _ = _names or _torch_names()
    B, width = key_begin.shape[0], page_table.shape[-1]
    rows, table = (B,), (B, width)
    key_begin, key_end, page_table, out_table, stream = _pointers("g4attn_kv4_unpack", stream, (
        ("key_begin", key_begin, i32, rows), ("key_end", key_end, i32, rows), ("page_table", page_table, i32, table),
        ("out_table", out_table, i32, table)), layer, cache, out)
    _check((_lib or load()).g4attn_kv4_unpack(ctypes.byref(layer), key_begin, key_end, B, ctypes.byref(cache),
                                              page_table, ctypes.byref(out), out_table, width, stream),
           "g4attn_kv4_unpack")


def g4attn_kv4_prefill(layer, norms, q, k, v, q_start, q_len, ctx_start, cache: g4attn_cache4, page_table,
                       scratch: g4attn_cache, scratch_table, out, span=None, stream=None):
    """A prefill (or chunk) over a 4-bit cache; scratch: a bf16 cache for the keys its rows see. Not for
    sequences that lost pages (see g4attn_kv4_append)."""
    bf, i32, _, _, _ = _names or _torch_names()
    T, B, width = q.shape[0], q_start.shape[0], page_table.shape[-1]
    qo, kv = (T, layer.n_q_heads, layer.head_dim), (T, layer.n_kv_heads, layer.head_dim)
    rows, table = (B,), (B, width)
    qp, k, v, q_start, q_len, ctx_start, span, page_table, scratch_table, op, stream = _pointers(
        "g4attn_kv4_prefill", stream, (
            ("q", q, bf, qo), ("k", k, bf, kv), ("v", v, bf, kv), ("q_start", q_start, i32, rows),
            ("q_len", q_len, i32, rows), ("ctx_start", ctx_start, i32, rows), ("span", span, i32, (T, 2)),
            ("page_table", page_table, i32, table), ("scratch_table", scratch_table, i32, table), ("out", out, bf, qo)),
        layer, cache, scratch)
    _check((_lib or load()).g4attn_kv4_prefill(ctypes.byref(layer), _opt(norms), qp, k, v, T, q_start, q_len, ctx_start,
                                               B, span, ctypes.byref(cache), page_table, ctypes.byref(scratch),
                                               scratch_table, width, op, stream), "g4attn_kv4_prefill")
    return out


def g4attn_kv4_decode_workspace_bytes(layer, B: int, max_pages: int, page_weights: bool = False) -> int:
    return int(load().g4attn_kv4_decode_workspace_bytes(ctypes.byref(layer), int(B), int(max_pages),
                                                        1 if page_weights else 0))


def g4attn_kv4_decode(layer, norms, q, k_new, v_new, seq_len, cache: g4attn_cache4, page_table, out, workspace,
                      pos=None, page_weights=None, stream=None):
    """One decode step over a 4-bit cache. k_new None: the newest token is in the cache already; pos:
    RoPE positions of sequences that lost pages; page_weights: accumulated per page (global layers)."""
    bf, i32, f32, _, _ = _names or _torch_names()
    B, width = q.shape[0], page_table.shape[-1]
    qo, kv = (B, layer.n_q_heads, layer.head_dim), (B, layer.n_kv_heads, layer.head_dim)
    rows, table = (B,), (B, width)
    q, k_new, v_new, seq_len, pos, page_table, page_weights, op, work, stream = _pointers("g4attn_kv4_decode", stream, (
        ("q", q, bf, qo), ("k_new", k_new, bf, kv), ("v_new", v_new, bf, kv), ("seq_len", seq_len, i32, rows),
        ("pos", pos, i32, rows), ("page_table", page_table, i32, table), ("page_weights", page_weights, f32, table),
        ("out", out, bf, qo), ("workspace", workspace, workspace.dtype, workspace.shape)),
        layer, cache)
    _check((_lib or load()).g4attn_kv4_decode(ctypes.byref(layer), _opt(norms), q, k_new, v_new, seq_len, pos, B,
                                              ctypes.byref(cache), page_table, width, page_weights, op, work,
                                              workspace.nbytes, stream), "g4attn_kv4_decode")
    return out


# ---- the page plan --------------------------------------------------------------------------------------

def make_page_group(window: int, page_table, free_pages, pool, out_pool, seq_len, slots=None, first_page=None,
                    out_first_page=None, lost=None, out_lost=None, freed=None, n_freed=None,
                    out_n_freed=None) -> g4attn_page_group:
    """One layer kind's pages (window 0: a global one), as int32 tensors (slots: int64) on one device that the group
    keeps. page_table [B, columns], free_pages [physical pages], pool [2]; slots [T]; the others [B] (freed as
    page_table). out_n_freed None: n_freed itself where out_lost is lost, so that the pages of an eviction come back once;
    else an array of the group's own, group.tensors["out_n_freed"], which is the n_freed of the state in out_lost."""
    import torch
    B, width = page_table.shape
    if n_freed is not None and out_n_freed is None:
        in_place = lost is not None and out_lost is not None and lost.data_ptr() == out_lost.data_ptr()
        out_n_freed = n_freed if in_place else torch.zeros_like(n_freed)
    tensors = dict(free_pages=free_pages, pool=pool, out_pool=out_pool, page_table=page_table, first_page=first_page,
                   out_first_page=out_first_page, lost=lost, out_lost=out_lost, freed=freed, n_freed=n_freed,
                   seq_len=seq_len, slots=slots, out_n_freed=out_n_freed)
    shapes = dict(free_pages=(free_pages.numel(),), pool=(2,), out_pool=(2,), page_table=(B, width), freed=(B, width),
                  slots=(None if slots is None else slots.numel(),))
    for name, t in tensors.items():
        if t is None:
            continue
        dtype, shape = torch.int64 if name == "slots" else torch.int32, shapes.get(name, (B,))
        if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous() or t.device != page_table.device:
            raise ValueError(f"make_page_group: {name} must be a dense {dtype} tensor of shape {shape} on "
                             f"{page_table.device}, got {t.dtype} {tuple(t.shape)} on {t.device}"
                             f"{'' if t.is_contiguous() else ' (strided)'}")
    group = g4attn_page_group(int(window), free_pages.numel(), width, *(_ptr(t) for t in tensors.values()))
    group.tensors = tensors
    group.room = (B, None if slots is None else slots.numel(), page_table.get_device())
    return group


def g4attn_plan_pages(ctx_len, new_len, groups, out_ctx_len, q_start, q_len, ctx_start, positions, stream=None):
    """Plans one serving step of B requests and T = len(positions) rows over one or two page groups: who is served,
    page tables, slots, positions. out_ctx_len may be ctx_len. A prefill takes q_start, q_len and ctx_start;
    g4attn_kv4_decode a group's seq_len, and ctx_start as pos (positions goes by rows, pos by requests)."""
    _, i32, _, _, _ = _names or _torch_names()
    B, T, n = ctx_len.shape[0], positions.shape[0], len(groups)
    rows = (B,)
    *pointers, stream = _pointers("g4attn_plan_pages", stream, (
        ("ctx_len", ctx_len, i32, rows), ("new_len", new_len, i32, rows), ("out_ctx_len", out_ctx_len, i32, rows),
        ("q_start", q_start, i32, rows), ("q_len", q_len, i32, rows), ("ctx_start", ctx_start, i32, rows),
        ("positions", positions, i32, (T,))))
    here = ctx_len.get_device()
    for g in groups:
        if g.room is not None and g.room != (B, T, here) and g.room != (B, None, here):
            raise ValueError(f"g4attn_plan_pages: a group of {g.room[0]} requests, {g.room[1]} rows on device "
                             f"{g.room[2]} in a call of {B} requests, {T} rows on device {here}")
    array = groups if isinstance(groups, ctypes.Array) else (g4attn_page_group * n)(*groups)
    _check((_lib or load()).g4attn_plan_pages(pointers[0], pointers[1], B, T, array, n, *pointers[2:], stream),
           "g4attn_plan_pages")
