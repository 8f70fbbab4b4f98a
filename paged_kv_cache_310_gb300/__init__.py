"""Python binding of libpagedkv.so -- the paged KV cache hot path on one GB300.

Argument marshalling only: every step runs in the library's CUDA kernels.  PyTorch
supplies device memory and the current stream.  The calls mirror the C ABI in
``include/pagedkv.h``:

* :func:`paged_kv_append`        -- new tokens' K/V into their cache slots
* :func:`paged_block_copy`       -- copy-on-write block copies
* :func:`paged_attention_decode` -- single-token decode attention through block tables
* :func:`paged_kv_gather`        -- the block-table gather alone (indexing checks)

and, for caches held in 4 bits (uint8 pools, 5 bytes for 8 values):

* :func:`paged_kv4_append`       -- new tokens' K/V rounded to 4 bits into their slots
* :func:`paged_kv4_expand`       -- 4-bit blocks widened into blocks of another pool
* :func:`paged_attention_decode_kv4` -- single-token decode attention over a 4-bit pool

and, to shorten sequences by what attention uses least:

* :func:`paged_attention_weights` -- a decode step's attention weights, added per token
* :func:`paged_kv_evict`         -- the heaviest and the most recent rows kept, in fresh blocks

and, for models with rotary positions and sliding windows:

* :func:`paged_qk_rotary`        -- queries and keys normed per head and rotated by position
* :func:`paged_kv_append_rotary` -- the same on the way into the cache (and V as it is)
* :func:`rotary_frequencies`     -- frequencies, also of rotations scaled for long contexts
* :func:`paged_attention_decode_window`, :func:`paged_attention_prefill_window` -- attention over
  the last tokens and the first few
* :func:`paged_attention_prefill_window_plan` -- the kernel that the latter takes

If the library has not been built the import still succeeds, but every call raises:
there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
import struct
import threading

import torch

__all__ = [
    "PagedKVError", "CacheDesc", "DecodeConfig", "DecodePlan", "paged_attention_plan", "library", "library_path", "cache_desc",
    "paged_kv_append", "paged_block_copy", "paged_attention_decode",
    "paged_attention_workspace_bytes", "paged_attention_decode_no_alloc", "paged_attention_no_alloc_limit",
    "paged_kv_gather", "paged_block_swap_out", "paged_block_swap_in", "paged_attention_prefill", "device_error", "declared_functions",
    "PATH_AUTO", "PATH_CUDA_CORE", "PATH_TENSOR_CORE",
    "paged_kv4_append", "paged_kv4_expand", "paged_attention_decode_kv4", "paged_attention_decode_kv4_workspace_bytes",
    "paged_attention_weights", "paged_attention_weights_workspace_bytes", "paged_kv_evict",
    "paged_qk_rotary", "paged_kv_append_rotary", "rotary_frequencies",
    "paged_attention_decode_window", "paged_attention_prefill_window", "paged_attention_prefill_window_plan",
    "PreparedCall", "prepare_kv_append", "prepare_block_copy", "prepare_attention_decode", "set_wait_limit",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libpagedkv.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "pagedkv.h")

F32, F16, BF16, KV4 = 0, 1, 2, 3
DTYPE_CODE = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
PATH_AUTO, PATH_CUDA_CORE, PATH_TENSOR_CORE = 0, 1, 2

STATUS = {0: "PKV_OK", 1: "PKV_ERR_INVALID_ARG", 2: "PKV_ERR_UNSUPPORTED", 3: "PKV_ERR_WORKSPACE",
          4: "PKV_ERR_CUDA", 5: "PKV_ERR_DEVICE_INDEX", 6: "PKV_ERR_DEVICE_TIMEOUT", 7: "PKV_ERR_OUT_OF_BLOCKS"}


class PagedKVError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


class CacheDesc(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class DecodeConfig(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int32), ("partition_tokens", ctypes.c_int32)]


class DecodePlan(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int32), ("partition_tokens", ctypes.c_int32),
                ("max_partitions", ctypes.c_int32), ("kernel_launches", ctypes.c_int32),
                ("workspace_bytes", ctypes.c_size_t), ("kv_heads_per_item", ctypes.c_int32)]


class WindowPlan(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int32), ("tokens_per_item", ctypes.c_int32), ("ctas_per_item", ctypes.c_int32)]


class RotaryScaling(ctypes.Structure):
    _fields_ = [("rule", ctypes.c_int32), ("factor", ctypes.c_double), ("original_len", ctypes.c_double),
                ("fast_turns", ctypes.c_double), ("slow_turns", ctypes.c_double)]


_lock = threading.Lock()
_lib = None


def declared_functions(header: str = HEADER) -> list[str]:
    """Names of the functions include/pagedkv.h declares."""
    text = open(header).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b((?:paged|pkv)_\w+)\s*\(", text)))


def library():
    """The loaded libpagedkv.so (raises if it was never built)."""
    global _lib
    if _lib is not None:  # set once, complete
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(library_path):
            raise PagedKVError(4, f"{library_path} is missing: build it with __graft_entry__.build()")
        lib = ctypes.CDLL(library_path)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        desc_p, cfg_p = ctypes.POINTER(CacheDesc), ctypes.POINTER(DecodeConfig)
        sig = {
            "paged_kv_append": [vp, vp, vp, i32, vp, vp, desc_p, vp],
            "paged_block_copy": [vp, vp, i32, vp, vp, desc_p, vp],
            "paged_attention_workspace_bytes": [i32, i32, i32, desc_p, cfg_p],
            "paged_attention_plan": [i32, i32, i32, desc_p, cfg_p, ctypes.POINTER(DecodePlan)],
            "paged_attention_decode": [vp, vp, vp, vp, i32, vp, i32, i32, i32, ctypes.c_float, vp, i32,
                                       vp, sz, desc_p, cfg_p, vp],
            "paged_kv4_append": [vp, vp, i32, vp, i32, vp, vp, desc_p, vp],
            "paged_attention_decode_kv4_workspace_bytes": [i32, i32, i32, i32, desc_p],
            "paged_attention_decode_kv4": [vp, i32, vp, vp, vp, i32, vp, i32, i32, i32, ctypes.c_float, vp, i32,
                                           vp, sz, desc_p, vp],
            "paged_attention_weights_workspace_bytes": [i32, i32, i32, desc_p],
            "paged_attention_weights": [vp, i32, vp, vp, i32, vp, vp, i32, i32, i32, ctypes.c_float, vp, vp, i64, vp, sz,
                                        desc_p, vp],
            "paged_kv_evict": [vp, vp, i64, vp, i32, vp, vp, i32, vp, i32, i32, i32, i32, vp, vp, vp, desc_p, vp],
            "paged_kv4_expand": [vp, i32, vp, vp, desc_p, vp, vp, desc_p, vp],
            "paged_rotary_frequencies": [vp, i32, ctypes.c_double, ctypes.POINTER(RotaryScaling),
                                         ctypes.POINTER(ctypes.c_float)],
            "paged_qk_rotary": [vp, i64, vp, i64, vp, i32, i32, i32, i32, i32, vp, vp, i64, vp, i64, vp],
            "paged_kv_append_rotary": [vp, i64, vp, i64, vp, i64, vp, vp, i32, i32, vp, vp, i64, vp, vp, desc_p, vp],
            "paged_attention_decode_window": [vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, ctypes.c_float, vp, i32,
                                              desc_p, vp],
            "paged_attention_prefill_window": [vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, i32, ctypes.c_float,
                                               vp, i32, desc_p, vp],
            "paged_attention_prefill_window_plan": [i32, i32, i32, i32, i32, i32, desc_p, ctypes.POINTER(WindowPlan)],
            "paged_kv_gather": [vp, vp, vp, i32, vp, i32, i32, vp, vp, desc_p, vp],
            "paged_block_swap_out": [vp, i32, vp, vp, vp, vp, desc_p, vp],
            "paged_attention_prefill": [vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, ctypes.c_float, vp, i32,
                                        vp, sz, desc_p, vp],
            "paged_attention_prefill_workspace_bytes": [i32, i32, i32, desc_p],
            "paged_block_swap_in": [vp, i32, vp, vp, vp, vp, desc_p, vp],
            "paged_attention_decode_no_alloc": [vp, vp, vp, vp, i32, vp, i32, i32, i32, ctypes.c_float, vp,
                                                i32, desc_p, cfg_p, vp],
            "paged_attention_no_alloc_limit": [],
            "paged_kv_device_error": [vp],
            "paged_kv_selftest_wait_timeout": [ctypes.c_uint64, vp],
            "paged_kv_set_wait_limit": [ctypes.c_uint64],
            "paged_kv_last_error": [],
            "paged_kv_version": [],
        }
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        lib.paged_attention_workspace_bytes.restype = sz
        lib.paged_attention_no_alloc_limit.restype = sz
        lib.paged_attention_prefill_workspace_bytes.restype = sz
        lib.paged_attention_decode_kv4_workspace_bytes.restype = sz
        lib.paged_attention_weights_workspace_bytes.restype = sz
        lib.paged_kv_last_error.restype = ctypes.c_char_p
        lib.paged_kv_version.restype = ctypes.c_char_p
        _lib = lib
        return lib


def _check(status: int) -> None:
    if status != 0:
        raise PagedKVError(status, library().paged_kv_last_error().decode())


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (t.device.type != "cuda" or not t.is_contiguous()):
            raise PagedKVError(1, "tensors must be contiguous CUDA tensors")


def cache_desc(k_cache: torch.Tensor) -> CacheDesc:
    """Descriptor of a pool shaped [num_blocks, num_kv_heads, block_size, head_dim], or of a
    4-bit pool: uint8, [num_blocks, num_kv_heads, block_size, head_dim * 5 / 8]."""
    if k_cache.dim() != 4:
        raise PagedKVError(1, "cache must be [num_blocks, num_kv_heads, block_size, head_dim]")
    nb, hkv, bs, d = k_cache.shape
    if k_cache.dtype == torch.uint8:
        if d % 5:
            raise PagedKVError(1, "rows of a 4-bit pool hold head_dim * 5 / 8 bytes")
        return CacheDesc(nb, bs, hkv, d // 5 * 8, KV4)
    if k_cache.dtype not in DTYPE_CODE:
        raise PagedKVError(2, f"cache dtype {k_cache.dtype}")
    return CacheDesc(nb, bs, hkv, d, DTYPE_CODE[k_cache.dtype])


class PreparedCall:
    """One library call whose arguments were checked and marshalled once.

    Calling it enqueues the same work again on `stream` (a torch.cuda.Stream or a raw
    cudaStream_t handle; default: the device's current stream), with none of the
    per-call argument checks and ctypes conversions of the plain functions -- what a
    serving loop that replays the same buffers every step wants.  The tensors it was
    made from stay referenced by it; their contents may change between calls, their
    storage must not (no reallocation, resize or reshaping in place)."""

    __slots__ = ("_fn", "_args", "_device", "_keep")

    def __init__(self, fn, args, device, keep):
        self._fn, self._args, self._device, self._keep = fn, tuple(args), device, keep

    def __call__(self, stream=None) -> None:
        if stream is None:
            handle = torch.cuda.current_stream(self._device).cuda_stream
        else:
            handle = stream if isinstance(stream, int) else stream.cuda_stream
        status = self._fn(*self._args, ctypes.c_void_p(handle))
        if status != 0:
            raise PagedKVError(status, library().paged_kv_last_error().decode())


def _run(prepared: PreparedCall) -> None:
    prepared()


def _append_call(k, v, slot_mapping, k_cache, v_cache) -> PreparedCall:
    _need_cuda(k, v, slot_mapping, k_cache, v_cache)
    if slot_mapping.dtype != torch.int64 or k.dtype != k_cache.dtype or v.dtype != k_cache.dtype:
        raise PagedKVError(1, "slot_mapping must be int64 and k/v must have the cache dtype")
    if k.shape != v.shape or k.dim() != 3 or k.shape[0] != slot_mapping.numel() \
            or tuple(k.shape[1:]) != (k_cache.shape[1], k_cache.shape[3]) or k_cache.shape != v_cache.shape:
        raise PagedKVError(1, "shape mismatch between k, v, slot_mapping and the caches")
    desc = cache_desc(k_cache)
    args = (_ptr(k), _ptr(v), _ptr(slot_mapping), slot_mapping.numel(), _ptr(k_cache), _ptr(v_cache),
            ctypes.byref(desc))
    return PreparedCall(library().paged_kv_append, args, k_cache.device, (k, v, slot_mapping, k_cache, v_cache, desc))


def paged_kv_append(k, v, slot_mapping, k_cache, v_cache) -> None:
    """k, v [T, Hkv, D] -> k_cache/v_cache rows given by slot_mapping (int64 [T])."""
    _run(_append_call(k, v, slot_mapping, k_cache, v_cache))


def prepare_kv_append(k, v, slot_mapping, k_cache, v_cache) -> PreparedCall:
    """paged_kv_append with its arguments bound once (see PreparedCall)."""
    return _append_call(k, v, slot_mapping, k_cache, v_cache)


def _block_copy_call(src_dst_pairs, k_cache, v_cache, host_pairs) -> PreparedCall:
    _need_cuda(src_dst_pairs, k_cache, v_cache)
    if src_dst_pairs.dtype != torch.int64 or (src_dst_pairs.numel() % 2):
        raise PagedKVError(1, "src_dst_pairs must be int64 [n, 2]")
    if host_pairs is not None:
        host_pairs = host_pairs.to(torch.int64).contiguous()
        if host_pairs.device.type != "cpu" or host_pairs.numel() != src_dst_pairs.numel():
            raise PagedKVError(1, "host_pairs must be a CPU copy of src_dst_pairs")
    desc = cache_desc(k_cache)
    n = src_dst_pairs.numel() // 2
    args = (_ptr(src_dst_pairs), _ptr(host_pairs), n, _ptr(k_cache), _ptr(v_cache), ctypes.byref(desc))
    return PreparedCall(library().paged_block_copy, args, k_cache.device,
                        (src_dst_pairs, host_pairs, k_cache, v_cache, desc))


def paged_block_copy(src_dst_pairs, k_cache, v_cache, host_pairs: torch.Tensor | None = None) -> None:
    """Copy block src to block dst for each row of src_dst_pairs (device int64 [n, 2]).

    host_pairs (CPU int64 [n, 2], optional) lets the library validate the pairs.
    """
    _run(_block_copy_call(src_dst_pairs, k_cache, v_cache, host_pairs))


def prepare_block_copy(src_dst_pairs, k_cache, v_cache, host_pairs: torch.Tensor | None = None) -> PreparedCall:
    """paged_block_copy with its arguments bound once (see PreparedCall); the pairs are
    validated against host_pairs, when given, at every call."""
    return _block_copy_call(src_dst_pairs, k_cache, v_cache, host_pairs)


def _swap_buffers(ids, k_cache, host_k, host_v):
    _need_cuda(ids, k_cache)
    if ids.dtype != torch.int64:
        raise PagedKVError(1, "block ids must be int64")
    shape = (ids.numel(),) + tuple(k_cache.shape[1:])
    for h in (host_k, host_v):
        if tuple(h.shape) != shape or h.dtype != k_cache.dtype or not h.is_contiguous():
            raise PagedKVError(1, f"swap buffers must be contiguous {shape} in the cache dtype")


def paged_block_swap_out(block_ids, k_cache, v_cache, host_k, host_v) -> None:
    """host_k/v[i] <- pool block block_ids[i] (device int64 ids; pinned host buffers)."""
    _swap_buffers(block_ids, k_cache, host_k, host_v)
    desc = cache_desc(k_cache)
    _check(library().paged_block_swap_out(_ptr(block_ids), block_ids.numel(), _ptr(k_cache), _ptr(v_cache),
                                          _ptr(host_k), _ptr(host_v), ctypes.byref(desc), _stream(k_cache)))


def paged_block_swap_in(block_ids, host_k, host_v, k_cache, v_cache) -> None:
    """pool block block_ids[i] <- host_k/v[i]."""
    _swap_buffers(block_ids, k_cache, host_k, host_v)
    desc = cache_desc(k_cache)
    _check(library().paged_block_swap_in(_ptr(block_ids), block_ids.numel(), _ptr(host_k), _ptr(host_v),
                                         _ptr(k_cache), _ptr(v_cache), ctypes.byref(desc), _stream(k_cache)))


def _config(path: int, partition_tokens: int) -> DecodeConfig:
    return DecodeConfig(int(path), int(partition_tokens))


def paged_attention_workspace_bytes(num_seqs, num_q_heads, max_context_len, k_cache, *, path=PATH_AUTO,
                                    partition_tokens=0) -> int:
    desc = cache_desc(k_cache)
    cfg = _config(path, partition_tokens)
    return int(library().paged_attention_workspace_bytes(num_seqs, num_q_heads, max_context_len,
                                                         ctypes.byref(desc), ctypes.byref(cfg)))


def paged_attention_plan(num_seqs, num_q_heads, max_context_len, k_cache, *, path=PATH_AUTO,
                         partition_tokens=0) -> dict:
    """The path, partition size, partition count, kernel launches and workspace bytes
    paged_attention_decode uses for these sizes."""
    desc = cache_desc(k_cache)
    cfg = _config(path, partition_tokens)
    plan = DecodePlan()
    _check(library().paged_attention_plan(num_seqs, num_q_heads, max_context_len, ctypes.byref(desc),
                                          ctypes.byref(cfg), ctypes.byref(plan)))
    return {f: getattr(plan, f) for f, _ in DecodePlan._fields_}


_ws_cache: dict = {}


def _workspace(device, nbytes: int) -> torch.Tensor | None:
    if nbytes == 0:
        return None
    key = (device.type, device.index)
    ws = _ws_cache.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
        _ws_cache[key] = ws
    return ws


def paged_attention_decode(q, k_cache, v_cache, block_tables, context_lens, scale, out, *,
                           max_context_len: int | None = None, workspace: torch.Tensor | None = None,
                           path: int = PATH_AUTO, partition_tokens: int = 0) -> torch.Tensor:
    """out[s, h] = softmax(scale * q[s, h] . K_j) V_j over the context_lens[s] tokens of s.

    q [S, Hq, D]; caches [NB, Hkv, bs, D]; block_tables int32 [S, max_blocks];
    context_lens int32 [S]; out [S, Hq, D] in q's dtype or float32.
    max_context_len: host upper bound on context_lens (computed with a device sync
    when omitted).  workspace: uint8 device buffer, allocated and cached when omitted.
    """
    _run(_decode_call(q, k_cache, v_cache, block_tables, context_lens, scale, out, max_context_len,
                      workspace, path, partition_tokens))
    return out


def prepare_attention_decode(q, k_cache, v_cache, block_tables, context_lens, scale, out, *,
                             max_context_len: int, workspace: torch.Tensor | None = None,
                             path: int = PATH_AUTO, partition_tokens: int = 0) -> PreparedCall:
    """paged_attention_decode with its arguments bound once (see PreparedCall).
    max_context_len stays the bound of every later call."""
    if max_context_len is None:
        raise PagedKVError(1, "max_context_len is required for a prepared decode")
    return _decode_call(q, k_cache, v_cache, block_tables, context_lens, scale, out, max_context_len, workspace,
                        path, partition_tokens)


def _decode_call(q, k_cache, v_cache, block_tables, context_lens, scale, out, max_context_len, workspace, path,
                 partition_tokens) -> PreparedCall:
    _need_cuda(q, k_cache, v_cache, block_tables, context_lens, out, workspace)
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise PagedKVError(1, "block_tables and context_lens must be int32")
    if q.dim() != 3 or out.shape != q.shape or q.dtype != k_cache.dtype or v_cache.shape != k_cache.shape \
            or v_cache.dtype != k_cache.dtype or q.shape[2] != k_cache.shape[3]:
        raise PagedKVError(1, "shape/dtype mismatch between q, out and the caches")
    S, Hq, _ = q.shape
    if context_lens.numel() != S or block_tables.dim() != 2 or block_tables.shape[0] != S:
        raise PagedKVError(1, "block_tables must be [S, max_blocks] and context_lens [S]")
    if out.dtype not in DTYPE_CODE:
        raise PagedKVError(2, f"out dtype {out.dtype}")
    if max_context_len is None:
        max_context_len = int(context_lens.max()) if S else 0
    desc = cache_desc(k_cache)
    cfg = _config(path, partition_tokens)
    lib = library()
    need = int(lib.paged_attention_workspace_bytes(S, Hq, max_context_len, ctypes.byref(desc),
                                                   ctypes.byref(cfg)))
    if workspace is None:
        workspace = _workspace(q.device, need)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = (_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), block_tables.shape[1], _ptr(context_lens),
            S, Hq, max_context_len, ctypes.c_float(float(scale)), _ptr(out), DTYPE_CODE[out.dtype], _ptr(workspace),
            ws_bytes, ctypes.byref(desc), ctypes.byref(cfg))
    return PreparedCall(lib.paged_attention_decode, args, q.device,
                        (q, k_cache, v_cache, block_tables, context_lens, out, workspace, desc, cfg))


def paged_attention_decode_no_alloc(q, k_cache, v_cache, block_tables, context_lens, scale, out, *,
                                    max_context_len: int, path: int = PATH_AUTO,
                                    partition_tokens: int = 0) -> torch.Tensor:
    """paged_attention_decode without a workspace argument, for callers that cannot
    allocate device memory: the scratch is the library's built-in array of
    ``paged_attention_no_alloc_limit()`` bytes per GPU, shared by every call (calls
    that overlap on the GPU race on it).

    max_context_len (a host bound on context_lens) is required here: working it out
    from the device tensor would run a reduction that allocates its result."""
    _need_cuda(q, k_cache, v_cache, block_tables, context_lens, out)
    if q.dim() != 3 or out.shape != q.shape or q.dtype != k_cache.dtype or block_tables.dtype != torch.int32 \
            or context_lens.dtype != torch.int32:
        raise PagedKVError(1, "shape/dtype mismatch between q, out, the caches and the tables")
    if max_context_len is None:
        raise PagedKVError(1, "max_context_len is required: computing it on the device would allocate")
    S, Hq, _ = q.shape
    desc = cache_desc(k_cache)
    cfg = _config(path, partition_tokens)
    _check(library().paged_attention_decode_no_alloc(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), block_tables.shape[1], _ptr(context_lens), S, Hq,
        max_context_len, float(scale), _ptr(out), DTYPE_CODE[out.dtype], ctypes.byref(desc), ctypes.byref(cfg),
        _stream(q)))
    return out


def paged_attention_no_alloc_limit() -> int:
    """Bytes of the built-in workspace array used by paged_attention_decode_no_alloc."""
    return int(library().paged_attention_no_alloc_limit())


def paged_attention_prefill(q, k_cache, v_cache, block_tables, context_lens, query_start, scale, out, *,
                            max_context_len: int | None = None,
                            workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Causal attention of several new tokens per sequence (prefill / chunked prefill).

    q, out [T, Hq, D]: sequence s's new tokens are rows query_start[s]..query_start[s+1]-1,
    the last ones of its context_lens[s] tokens (K/V already appended).  query_start:
    int32 [S+1] on the device.
    """
    _need_cuda(q, k_cache, v_cache, block_tables, context_lens, query_start, out, workspace)
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32 or query_start.dtype != torch.int32:
        raise PagedKVError(1, "block_tables, context_lens and query_start must be int32")
    if q.dim() != 3 or out.shape != q.shape or q.dtype != k_cache.dtype or q.shape[2] != k_cache.shape[3]:
        raise PagedKVError(1, "shape/dtype mismatch between q, out and the caches")
    T, Hq, _ = q.shape
    S = context_lens.numel()
    if query_start.numel() != S + 1 or block_tables.shape[0] != S:
        raise PagedKVError(1, "query_start must be [S+1] and block_tables [S, max_blocks]")
    if out.dtype not in DTYPE_CODE:
        raise PagedKVError(2, f"out dtype {out.dtype}")
    if max_context_len is None:
        max_context_len = int(context_lens.max()) if S else 0
    desc = cache_desc(k_cache)
    lib = library()
    need = int(lib.paged_attention_prefill_workspace_bytes(S, Hq, T, ctypes.byref(desc)))
    if workspace is None:
        workspace = _workspace(q.device, need)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.paged_attention_prefill(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                       block_tables.shape[1], _ptr(context_lens), _ptr(query_start), S, Hq, T,
                                       max_context_len, float(scale), _ptr(out), DTYPE_CODE[out.dtype],
                                       _ptr(workspace), ws_bytes, ctypes.byref(desc), _stream(q)))
    return out


def paged_kv_gather(k_cache, v_cache, block_tables, context_lens, k_out, v_out, *,
                    max_context_len: int | None = None) -> None:
    """k_out/v_out [S, Hkv, max_len, D] <- each sequence's rows through its block table."""
    _need_cuda(k_cache, v_cache, block_tables, context_lens, k_out, v_out)
    S = context_lens.numel()
    if max_context_len is None:
        max_context_len = k_out.shape[2]
    if k_out.shape != (S, k_cache.shape[1], max_context_len, k_cache.shape[3]) or v_out.shape != k_out.shape \
            or k_out.dtype != k_cache.dtype or v_out.dtype != k_cache.dtype:
        raise PagedKVError(1, "k_out/v_out must be [S, Hkv, max_len, D] in the cache dtype")
    desc = cache_desc(k_cache)
    _check(library().paged_kv_gather(_ptr(k_cache), _ptr(v_cache), _ptr(block_tables), block_tables.shape[1],
                                     _ptr(context_lens), S, max_context_len, _ptr(k_out), _ptr(v_out),
                                     ctypes.byref(desc), _stream(k_cache)))


# ---- 4-bit caches and eviction: the tensors of a call share one device, which need not be
# the current one, and a workspace that is not given comes from PyTorch's allocator at every
# call (ordered on the call's stream and, inside a capture, kept by the graph).  These calls
# are short on the GPU, so the binding passes plain integers and asks PyTorch little.

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # handle alone: 2 us less than the Stream object
_get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device  # CUDA is up: there are tensors on it


_INT32_MAX = 2 ** 31 - 1


def _count(n: int) -> int:
    """A number of tokens that may be past any sequence's (a window, sinks, recent rows) as 32 bits hold
    it, where ctypes would keep the low 32 bits of a larger one; negative ones are for the library to refuse."""
    return max(-1, min(n, _INT32_MAX))


def _one_device(first, *rest) -> int:
    """The index of the CUDA device that all the (contiguous) tensors are on."""
    device = first.get_device()
    if device < 0 or not first.is_contiguous():
        raise PagedKVError(1, "tensors must be contiguous CUDA tensors")
    for t in rest:
        if t is not None and (t.get_device() != device or not t.is_contiguous()):
            raise PagedKVError(1, "tensors must be contiguous CUDA tensors on one device")
    return device


def _call(fn, device: int, *args) -> None:
    """fn(*args, stream) with `device` current, on that device's current stream."""
    stream = _raw_stream(device) if _raw_stream else torch.cuda.current_stream(device).cuda_stream
    if device == _get_device():
        status = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, stream)
    if status:
        _check(status)


@functools.lru_cache(maxsize=512)
def _desc_of(shape, dtype):
    """A descriptor (never changed) of a pool of this shape and dtype, and a reference to it."""
    desc = cache_desc(torch.empty(shape, dtype=dtype, device="meta"))
    return desc, ctypes.byref(desc)


def _kv4_desc(k_cache, v_cache):
    if k_cache.dtype != torch.uint8 or v_cache.dtype != torch.uint8 or k_cache.shape != v_cache.shape:
        raise PagedKVError(1, "the 4-bit pools must be uint8 and of one shape")
    return _desc_of(k_cache.shape, torch.uint8)


def _dtype_code(t, what) -> int:
    code = DTYPE_CODE.get(t.dtype)
    if code is None:
        raise PagedKVError(2, f"{what} dtype {t.dtype}")
    return code


def _scratch(workspace, need: int, device: int):
    """(address, bytes) of a call's workspace, and the tensor that holds it."""
    if workspace is None:
        if not need:
            return 0, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=torch.device("cuda", device))
        return workspace.data_ptr(), need, workspace
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def paged_kv4_append(k, v, slot_mapping, k_cache, v_cache) -> None:
    """k, v [T, Hkv, D] (f32, f16 or bf16) rounded to 4 bits -> the rows of the 4-bit pools
    (uint8 [NB, Hkv, bs, D * 5 / 8]) given by slot_mapping (int64 [T]; negative: skipped)."""
    device = _one_device(k, v, slot_mapping, k_cache, v_cache)
    desc, desc_ref = _kv4_desc(k_cache, v_cache)
    if slot_mapping.dtype != torch.int64 or v.dtype != k.dtype:
        raise PagedKVError(1, "slot_mapping must be int64 and k and v of one dtype")
    tokens = slot_mapping.numel()
    if k.shape != v.shape or tuple(k.shape) != (tokens, desc.num_kv_heads, desc.head_dim):
        raise PagedKVError(1, "shape mismatch between k, v, slot_mapping and the caches")
    _call(library().paged_kv4_append, device, k.data_ptr(), v.data_ptr(), _dtype_code(k, "k/v"),
          slot_mapping.data_ptr(), tokens, k_cache.data_ptr(), v_cache.data_ptr(), desc_ref)


def paged_kv4_expand(src_dst_pairs, k_cache, v_cache, k_out, v_out) -> None:
    """Block dst of the pools k_out/v_out [NB', Hkv, bs, D] (f32, f16 or bf16) becomes the
    values of block src of the 4-bit pools, for each row of src_dst_pairs (int64 [n, 2])."""
    device = _one_device(src_dst_pairs, k_cache, v_cache, k_out, v_out)
    _, desc_ref = _kv4_desc(k_cache, v_cache)
    if src_dst_pairs.dtype != torch.int64 or src_dst_pairs.dim() != 2 or src_dst_pairs.shape[1] != 2:
        raise PagedKVError(1, "src_dst_pairs must be int64 [n, 2]")
    if v_out.dtype != k_out.dtype or v_out.shape != k_out.shape:
        raise PagedKVError(1, "k_out and v_out must be of one dtype and shape")
    _dtype_code(k_out, "out pool")
    _call(library().paged_kv4_expand, device, src_dst_pairs.data_ptr(), src_dst_pairs.shape[0], k_cache.data_ptr(),
          v_cache.data_ptr(), desc_ref, k_out.data_ptr(), v_out.data_ptr(), _desc_of(k_out.shape, k_out.dtype)[1])


def paged_attention_decode_kv4_workspace_bytes(num_seqs, num_q_heads, max_context_len, q_dtype, k_cache) -> int:
    """q_dtype: torch.float32, torch.float16 or torch.bfloat16."""
    return int(library().paged_attention_decode_kv4_workspace_bytes(
        num_seqs, num_q_heads, max_context_len, DTYPE_CODE[q_dtype], _kv4_desc(k_cache, k_cache)[1]))


def paged_attention_decode_kv4(q, k_cache, v_cache, block_tables, context_lens, scale, out, *,
                               max_context_len: int | None = None,
                               workspace: torch.Tensor | None = None) -> torch.Tensor:
    """out[s, h] = softmax(scale * q[s, h] . K_j) V_j over the context_lens[s] tokens of s, with
    K and V held in 4-bit pools (uint8 [NB, Hkv, bs, D * 5 / 8]).

    q [S, Hq, D] f32, f16 or bf16; block_tables int32 [S, max_blocks]; context_lens int32
    [S]; out [S, Hq, D] in q's dtype or float32.  max_context_len: host upper bound on
    context_lens (computed with a device sync when omitted).  workspace: uint8 device buffer
    of paged_attention_decode_kv4_workspace_bytes, allocated for the call when omitted.
    """
    device = _one_device(q, k_cache, v_cache, block_tables, context_lens, out, workspace)
    desc, desc_ref = _kv4_desc(k_cache, v_cache)
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise PagedKVError(1, "block_tables and context_lens must be int32")
    if q.dim() != 3 or out.shape != q.shape or q.shape[2] != desc.head_dim:
        raise PagedKVError(1, "shape mismatch between q, out and the caches")
    S, Hq, _ = q.shape
    if context_lens.numel() != S or block_tables.dim() != 2 or block_tables.shape[0] != S:
        raise PagedKVError(1, "block_tables must be [S, max_blocks] and context_lens [S]")
    q_code, out_code = _dtype_code(q, "q"), _dtype_code(out, "out")
    if max_context_len is None:
        max_context_len = int(context_lens.max()) if S else 0
    lib = library()
    need = 0
    if workspace is None:
        need = lib.paged_attention_decode_kv4_workspace_bytes(S, Hq, max_context_len, q_code, desc_ref)
    ws, ws_bytes, workspace = _scratch(workspace, need, device)
    _call(lib.paged_attention_decode_kv4, device, q.data_ptr(), q_code, k_cache.data_ptr(), v_cache.data_ptr(),
          block_tables.data_ptr(), block_tables.shape[1], context_lens.data_ptr(), S, Hq, max_context_len, float(scale),
          out.data_ptr(), out_code, ws, ws_bytes, desc_ref)
    return out


def paged_attention_weights_workspace_bytes(num_seqs, num_q_heads, max_context_len, k_cache) -> int:
    return int(library().paged_attention_weights_workspace_bytes(num_seqs, num_q_heads, max_context_len,
                                                                 _desc_of(k_cache.shape, k_cache.dtype)[1]))


def paged_attention_weights(q, k_cache, block_tables, context_lens, scale, weights, *,
                            weights_out: torch.Tensor | None = None, tracked_lens: torch.Tensor | None = None,
                            max_context_len: int | None = None,
                            workspace: torch.Tensor | None = None) -> torch.Tensor:
    """weights_out[s, g, j] = weights[s, g, j] + the softmax weights that the query heads of KV
    head g give token j, for j < context_lens[s]; other rows are left as they are.

    q [S, Hq, D] in the pool's dtype (a 4-bit pool takes f32, f16 or bf16); weights and
    weights_out float32 [S, Hkv, W], W >= max_context_len; weights_out defaults to weights
    (in place).  tracked_lens (int32 [S], optional): rows j >= tracked_lens[s] start at 0.
    max_context_len: host upper bound on context_lens (computed with a device sync when
    omitted).  workspace: uint8 device buffer, allocated for the call when omitted.
    """
    out = weights if weights_out is None else weights_out
    device = _one_device(q, k_cache, block_tables, context_lens, weights, out, tracked_lens, workspace)
    desc, desc_ref = _desc_of(k_cache.shape, k_cache.dtype)
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32 \
            or (tracked_lens is not None and tracked_lens.dtype != torch.int32):
        raise PagedKVError(1, "block_tables, context_lens and tracked_lens must be int32")
    if q.dim() != 3 or q.shape[2] != desc.head_dim:
        raise PagedKVError(1, "q must be [S, Hq, D] with the cache's head_dim")
    S, Hq, _ = q.shape
    if context_lens.numel() != S or block_tables.dim() != 2 or block_tables.shape[0] != S \
            or (tracked_lens is not None and tracked_lens.numel() != S):
        raise PagedKVError(1, "block_tables must be [S, max_blocks], context_lens and tracked_lens [S]")
    if weights.dtype != torch.float32 or out.dtype != torch.float32 or weights.dim() != 3 \
            or out.shape != weights.shape or tuple(weights.shape[:2]) != (S, desc.num_kv_heads):
        raise PagedKVError(1, "weights and weights_out must be float32 [S, Hkv, W]")
    q_code = _dtype_code(q, "q")
    if max_context_len is None:
        max_context_len = int(context_lens.max()) if S else 0
    lib = library()
    need = 0
    if workspace is None:
        need = lib.paged_attention_weights_workspace_bytes(S, Hq, max_context_len, desc_ref)
    ws, ws_bytes, workspace = _scratch(workspace, need, device)
    _call(lib.paged_attention_weights, device, q.data_ptr(), q_code, k_cache.data_ptr(), block_tables.data_ptr(),
          block_tables.shape[1], context_lens.data_ptr(), 0 if tracked_lens is None else tracked_lens.data_ptr(), S, Hq,
          max_context_len, float(scale), weights.data_ptr(), out.data_ptr(), weights.shape[2], ws, ws_bytes, desc_ref)
    return out


def paged_kv_evict(weights, block_tables, context_lens, keep_lens, new_tables, k_cache, v_cache, weights_out, kept, *,
                   recent: int = 0, max_context_len: int | None = None) -> None:
    """Shorten each sequence to k = min(keep_lens[s], context_lens[s]) rows: per KV head, the
    last min(recent, k) and the heaviest others (ties: lowest row first), in order, moved
    into the blocks of new_tables (int32 [S, max_new_blocks]; blocks that no listed sequence
    reads).  kept[s, g, i] is the row that became row i, weights_out[s, g, i] its weight;
    places past k are left as they are.

    weights, weights_out float32 [S, Hkv, W] (not overlapping); kept int32 [S, Hkv,
    max_keep]; block_tables, context_lens, keep_lens int32; the pools are of any dtype.
    max_context_len: host upper bound on context_lens (computed with a device sync when
    omitted).
    """
    device = _one_device(weights, block_tables, context_lens, keep_lens, new_tables, k_cache, v_cache, weights_out, kept)
    desc, desc_ref = _desc_of(k_cache.shape, k_cache.dtype)
    if v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype:
        raise PagedKVError(1, "the caches must be of one shape and dtype")
    for t in (block_tables, context_lens, keep_lens, new_tables, kept):
        if t.dtype != torch.int32:
            raise PagedKVError(1, "block_tables, context_lens, keep_lens, new_tables and kept must be int32")
    S, heads = context_lens.numel(), desc.num_kv_heads
    if keep_lens.numel() != S or block_tables.dim() != 2 or block_tables.shape[0] != S or new_tables.dim() != 2 \
            or new_tables.shape[0] != S or kept.dim() != 3 or tuple(kept.shape[:2]) != (S, heads):
        raise PagedKVError(1, "tables must be [S, blocks], lengths [S] and kept [S, Hkv, max_keep]")
    if weights.dtype != torch.float32 or weights_out.dtype != torch.float32 or weights.dim() != 3 \
            or weights_out.shape != weights.shape or tuple(weights.shape[:2]) != (S, heads):
        raise PagedKVError(1, "weights and weights_out must be float32 [S, Hkv, W]")
    if max_context_len is None:
        max_context_len = int(context_lens.max()) if S else 0
    _call(library().paged_kv_evict, device, weights.data_ptr(), weights_out.data_ptr(), weights.shape[2],
          block_tables.data_ptr(), block_tables.shape[1], context_lens.data_ptr(), keep_lens.data_ptr(), _count(recent),
          new_tables.data_ptr(), new_tables.shape[1], S, max_context_len, kept.shape[2], kept.data_ptr(),
          k_cache.data_ptr(), v_cache.data_ptr(), desc_ref)


# ---- rotary positions

_ROTARY_RULES = {None: 0, "linear": 1, "base": 2, "parts": 3}


def rotary_frequencies(rotary_dim: int, base: float = 10000.0, *, scaling: str | None = None, factor: float = 1.0,
                       original_len: float = 0.0, fast_turns: float = 32.0, slow_turns: float = 1.0):
    """(inv_freq, factor) of a rotation: float64 [rotary_dim / 2] on the CPU, inv_freq[i] =
    base^(-2 i / rotary_dim), and the factor of cosines and sines.  scaling for contexts
    `factor` times as long: "linear" divides every frequency, "base" raises the base so that
    the lowest one is divided, "parts" divides those that make up to slow_turns within
    original_len, keeps those with fast_turns or more, and blends in between, linearly in the turns.

    A checkpoint wants the rule it was trained with.  Many rules by parts blend linearly in the
    dimension's index instead, whose frequencies differ from these by up to a factor of 3, and some
    (fast_turns 4) leave cosines and sines alone (pass factor=1 to the calls then).  The calls take
    any frequencies and factor: compute those of another rule by its own definition."""
    if scaling not in _ROTARY_RULES:
        raise PagedKVError(1, f"scaling {scaling!r}")
    if not 0 < rotary_dim <= _INT32_MAX:
        raise PagedKVError(1, f"rotary_dim {rotary_dim}")
    out = torch.empty(rotary_dim // 2, dtype=torch.float64)
    rule = RotaryScaling(_ROTARY_RULES[scaling], factor, original_len, fast_turns, slow_turns)
    f = ctypes.c_float()
    _check(library().paged_rotary_frequencies(out.data_ptr() or 8, rotary_dim, base, ctypes.byref(rule), ctypes.byref(f)))
    return out, f.value


def _token_rows(t, what, dtype, device, tokens, head_dim):
    """(address, token stride, heads) of a [T, H, head_dim] tensor whose tokens may lie apart."""
    if t.dim() != 3 or t.dtype is not dtype or t.get_device() != device:
        raise PagedKVError(1, f"{what} must be [T, heads, {head_dim}] of one dtype on one CUDA device")
    n, heads, d = t.shape
    if n != tokens or d != head_dim:
        raise PagedKVError(1, f"{what} must be [T, heads, {head_dim}]")
    if t.is_contiguous():
        return t.data_ptr(), heads * d, heads
    apart, head, one = t.stride()
    if one != 1 or (head != d and heads > 1):
        raise PagedKVError(1, f"{what}: the heads of a token must lie one after the other")
    return t.data_ptr(), apart if n > 1 else heads * d, heads


_pack_rotary = struct.Struct("@PiiffPP").pack  # pkv_rotary, field by field: quicker than a ctypes.Structure


def _rotary(inv_freq, interleaved, factor, q_weight, k_weight, eps, dtype, device, head_dim) -> bytes:
    """The C struct of a rotation."""
    pairs = freq = qw = kw = 0
    if inv_freq is not None:
        pairs, freq = inv_freq.numel(), inv_freq.data_ptr()
        if inv_freq.dtype is not torch.float64 or inv_freq.get_device() != device or not inv_freq.is_contiguous():
            raise PagedKVError(1, "inv_freq must be a contiguous float64 tensor on the call's device")
    if q_weight is not None:
        qw = _norm_weight(q_weight, dtype, device, head_dim)
    if k_weight is not None:
        kw = _norm_weight(k_weight, dtype, device, head_dim)
    return _pack_rotary(freq, 2 * pairs, 1 if interleaved else 0, factor, eps, qw, kw)


def _norm_weight(w, dtype, device, head_dim) -> int:
    if w.dtype is not dtype or w.get_device() != device or not w.is_contiguous() or w.numel() != head_dim:
        raise PagedKVError(1, "norm weights must be contiguous, [head_dim], of the tensors' dtype and device")
    return w.data_ptr()


def paged_qk_rotary(q, k, positions, q_out, k_out, inv_freq, *, interleaved: bool = False, factor: float = 1.0,
                    q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
                    eps: float = 1e-6) -> None:
    """q_out, k_out <- q [T, Hq, D] and k [T, Hkv, D] normed per head (where a weight [D] is
    given) and rotated by positions (int32 [T]; negative: padding, left as it is).

    inv_freq (float64 [R / 2], device, or None): the first R = 2 * numel dimensions of a head
    turn, R a multiple of 16: dimension i with i + R / 2, or 2i with 2i + 1 if interleaved.
    factor multiplies cosines and sines.  Tokens may lie apart (views of a fused
    projection); q_out may be q and k_out may be k.
    """
    device, dtype, tokens = positions.get_device(), q.dtype, positions.numel()
    if device < 0 or not positions.is_contiguous() or positions.dtype != torch.int32:
        raise PagedKVError(1, "positions must be a contiguous int32 CUDA tensor")
    d = q.shape[-1] if q.dim() else 0
    qp, qs, hq = _token_rows(q, "q", dtype, device, tokens, d)
    kp, ks, hkv = _token_rows(k, "k", dtype, device, tokens, d)
    qop, qos, hqo = _token_rows(q_out, "q_out", dtype, device, tokens, d)
    kop, kos, hko = _token_rows(k_out, "k_out", dtype, device, tokens, d)
    if (hqo, hko) != (hq, hkv):
        raise PagedKVError(1, "q_out and k_out must have the shapes of q and k")
    rotary = _rotary(inv_freq, interleaved, factor, q_weight, k_weight, eps, dtype, device, d)
    _call(library().paged_qk_rotary, device, qp, qs, kp, ks, positions.data_ptr(), tokens, hq, hkv, d,
          _dtype_code(q, "q"), rotary, qop, qos, kop, kos)


def paged_kv_append_rotary(q, k, v, positions, slot_mapping, k_cache, v_cache, q_out, inv_freq, *,
                           interleaved: bool = False, factor: float = 1.0, q_weight: torch.Tensor | None = None,
                           k_weight: torch.Tensor | None = None, eps: float = 1e-6) -> torch.Tensor:
    """paged_qk_rotary and paged_kv_append in one pass: q normed and rotated -> q_out, k
    normed and rotated and v as it is -> the cache rows given by slot_mapping (int64 [T]).
    Tokens with a negative slot or position are padding.  q, k, v, q_out have the pools'
    dtype (f32, f16 or bf16); the other arguments are those of paged_qk_rotary."""
    device, dtype, tokens = _one_device(k_cache, v_cache, positions, slot_mapping), k_cache.dtype, positions.numel()
    desc, desc_ref = _desc_of(k_cache.shape, dtype)
    if desc.dtype == KV4:
        raise PagedKVError(2, "4-bit pools: paged_qk_rotary, then paged_kv4_append")
    if v_cache.shape != k_cache.shape or v_cache.dtype != dtype:
        raise PagedKVError(1, "the caches must be of one shape and dtype")
    if positions.dtype != torch.int32 or slot_mapping.dtype != torch.int64 or slot_mapping.numel() != tokens:
        raise PagedKVError(1, "positions must be int32 [T] and slot_mapping int64 [T]")
    d = desc.head_dim
    qp, qs, hq = _token_rows(q, "q", dtype, device, tokens, d)
    kp, ks, hk = _token_rows(k, "k", dtype, device, tokens, d)
    vp, vs, hv = _token_rows(v, "v", dtype, device, tokens, d)
    qop, qos, hqo = _token_rows(q_out, "q_out", dtype, device, tokens, d)
    if hqo != hq or hk != desc.num_kv_heads or hv != hk:
        raise PagedKVError(1, "q_out must have q's shape, k and v the caches' KV heads")
    rotary = _rotary(inv_freq, interleaved, factor, q_weight, k_weight, eps, dtype, device, d)
    _call(library().paged_kv_append_rotary, device, qp, qs, kp, ks, vp, vs, positions.data_ptr(), slot_mapping.data_ptr(),
          tokens, hq, rotary, qop, qos, k_cache.data_ptr(), v_cache.data_ptr(), desc_ref)
    return q_out


# ---- sliding windows

def _window_args(q, k_cache, v_cache, block_tables, context_lens, out, more, max_context_len):
    """Checks that both windowed calls make; (device, descriptor reference, out's dtype code,
    rows and heads of q, sequences, table width, bound of the lengths)."""
    device = _one_device(q, k_cache, v_cache, block_tables, context_lens, out, more)
    dtype, pool, rows, tables = k_cache.dtype, k_cache.shape, q.shape, block_tables.shape
    desc, desc_ref = _desc_of(pool, dtype)
    if desc.dtype == KV4:
        raise PagedKVError(2, "windows over 4-bit pools")
    if block_tables.dtype is not torch.int32 or context_lens.dtype is not torch.int32:
        raise PagedKVError(1, "block_tables and context_lens must be int32")
    if len(rows) != 3 or rows[2] != desc.head_dim or out.shape != rows or q.dtype is not dtype or v_cache.dtype is not dtype \
            or v_cache.shape != pool:
        raise PagedKVError(1, "shape/dtype mismatch between q, out and the caches")
    S = context_lens.numel()
    if len(tables) != 2 or tables[0] != S:
        raise PagedKVError(1, "block_tables must be [S, max_blocks]")
    if max_context_len is None:
        max_context_len = int(context_lens.max()) if S else 0
    elif not -1 <= max_context_len <= _INT32_MAX:
        raise PagedKVError(1, f"max_context_len {max_context_len}")
    return device, desc_ref, _dtype_code(out, "out"), rows[0], rows[1], S, tables[1], max_context_len


def paged_attention_decode_window(q, k_cache, v_cache, block_tables, context_lens, scale, out, *, window: int,
                                  sinks: int = 0, max_context_len: int | None = None) -> torch.Tensor:
    """out[s, h] = softmax(scale * q[s, h] . K_j) V_j over the last `window` of the
    context_lens[s] tokens of s and its first `sinks` (of any size; past the sequence they change nothing).

    Tensors as in paged_attention_decode; table entries of blocks that hold no such token are
    not read (-1 will do).  max_context_len: host upper bound on context_lens (computed with a
    device sync when omitted).  One kernel, no workspace.
    """
    device, desc_ref, out_code, T, Hq, S, width, longest = _window_args(q, k_cache, v_cache, block_tables, context_lens, out,
                                                                        None, max_context_len)
    if T != S:
        raise PagedKVError(1, "context_lens must be [S]")
    _call(library().paged_attention_decode_window, device, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
          block_tables.data_ptr(), width, context_lens.data_ptr(), S, Hq, longest, _count(window), _count(sinks),
          float(scale), out.data_ptr(), out_code, desc_ref)
    return out


def paged_attention_prefill_window(q, k_cache, v_cache, block_tables, context_lens, query_start, scale, out, *,
                                   window: int, sinks: int = 0, max_context_len: int | None = None) -> torch.Tensor:
    """paged_attention_prefill with a window: the new token at position p attends to the
    positions j <= p with j > p - window or j < sinks.  Tensors as there; table entries of blocks
    that hold no token attended to are not read.  No workspace."""
    device, desc_ref, out_code, T, Hq, S, width, longest = _window_args(q, k_cache, v_cache, block_tables, context_lens, out,
                                                                        query_start, max_context_len)
    if query_start.dtype is not torch.int32 or query_start.numel() != S + 1:
        raise PagedKVError(1, "query_start must be int32 [S+1]")
    _call(library().paged_attention_prefill_window, device, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
          block_tables.data_ptr(), width, context_lens.data_ptr(), query_start.data_ptr(), S, Hq, T, longest, _count(window),
          _count(sinks), float(scale), out.data_ptr(), out_code, desc_ref)
    return out


_WINDOW_KERNELS = ("rows", "shared_tiles", "tile_pairs")


def paged_attention_prefill_window_plan(num_seqs, num_q_heads, num_query_tokens, max_context_len, k_cache, *, window: int,
                                        sinks: int = 0) -> dict:
    """The kernel ("rows", "shared_tiles" or "tile_pairs"), new tokens per item and CTAs per item that
    paged_attention_prefill_window uses for these sizes."""
    desc, plan = cache_desc(k_cache), WindowPlan()
    for n in (num_seqs, num_q_heads, num_query_tokens, max_context_len):
        if not -1 <= n <= _INT32_MAX:
            raise PagedKVError(1, f"size {n}")
    _check(library().paged_attention_prefill_window_plan(num_seqs, num_q_heads, num_query_tokens, max_context_len,
                                                         _count(window), _count(sinks), ctypes.byref(desc), ctypes.byref(plan)))
    return dict(kernel=_WINDOW_KERNELS[plan.kernel], tokens_per_item=plan.tokens_per_item, ctas_per_item=plan.ctas_per_item)


def selftest_wait_timeout(limit_ns: int = 50_000_000) -> None:
    """Run the bounded-wait self-test kernel on the current stream (see the header)."""
    stream = torch.cuda.current_stream()
    _check(library().paged_kv_selftest_wait_timeout(int(limit_ns), ctypes.c_void_p(stream.cuda_stream)))


def set_wait_limit(limit_ns: int = 0) -> None:
    """Bound of the decode and prefill kernels' pipeline waits for later launches
    (0 = the default 2 s).  A tiny bound forces their abort path; see the header."""
    _check(library().paged_kv_set_wait_limit(int(limit_ns)))


def device_error(device=None) -> int:
    """Synchronise the current stream and read-and-clear the device error flag (0 = none)."""
    stream = torch.cuda.current_stream(device)
    return int(library().paged_kv_device_error(ctypes.c_void_p(stream.cuda_stream)))
