"""Thin binding of libsvp.so (include/svp.h), by ctypes and, for the calls on
4-bit caches, the gather, score and eviction calls, those on selected pages,
page assignment and log probabilities, by a small extension module
(csrc/calls.cpp).

Argument marshalling only: shape/dtype/device checks, raw device pointers,
the current CUDA stream, and a zero-filled workspace tensor kept per device.
Every step of the computation runs in the library's CUDA kernels; there is
no fallback of any kind -- if libsvp.so is missing or no GPU is present the
calls raise.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

import numpy as np

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsvp.so")

SVP_OK, SVP_ERR_INVALID_ARG, SVP_ERR_UNSUPPORTED, SVP_ERR_CUDA, SVP_ERR_WORKSPACE = (
    0, -1, -2, -3, -4)
SVP_F32, SVP_BF16, SVP_FP8_E4M3, SVP_FP4_E2M1 = 0, 1, 2, 3
PATH_AUTO, PATH_CUDA_CORES, PATH_TENSOR_CORES, PATH_TCGEN05 = 0, 1, 2, 3
DEV_BAD_BLOCK_ID, DEV_BAD_SEQ_LEN, DEV_BAD_TOKEN, DEV_TIMEOUT = 1, 2, 4, 8
DEV_NO_PAGES = 16
EXPORTED = ("paged_decode_attention", "paged_decode_attention_noalloc",
            "paged_tree_attention",
            "paged_decode_workspace_size",
            "kv_append", "kv_gather", "paged_score_update", "kv_evict",
            "kv_page_bounds", "paged_page_scores", "paged_select_pages",
            "paged_sparse_attention", "kv_assign_pages", "kv_append_slots",
            "token_logprobs",
            "spec_accept", "spec_accept_ex", "spec_accept_tree",
            "svp_read_device_status",
            "svp_step_create", "svp_step_host_buffer", "svp_step_launch",
            "svp_step_wait", "svp_step_stream", "svp_step_destroy",
            "svp_status_string", "svp_last_launch_count")


class SvpDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("num_q_heads", ctypes.c_int),
                ("num_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("block_size", ctypes.c_int),
                ("max_blocks_per_seq", ctypes.c_int),
                ("num_blocks", ctypes.c_int), ("dtype", ctypes.c_int),
                ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t),
                ("split_pages", ctypes.c_int),
                ("kernel_path", ctypes.c_int),
                ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float)]


class SvpAcceptOpts(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("allowed", ctypes.c_void_p),
                ("greedy", ctypes.c_int)]


class SvpStepDesc(ctypes.Structure):
    _fields_ = [("dims", SvpDims), ("q_len", ctypes.c_int),
                ("n_sink", ctypes.c_int), ("window", ctypes.c_int),
                ("scale", ctypes.c_float), ("k_cache", ctypes.c_void_p),
                ("v_cache", ctypes.c_void_p), ("num_draft", ctypes.c_int),
                ("vocab", ctypes.c_int), ("temperature", ctypes.c_float),
                ("greedy", ctypes.c_int), ("use_mask", ctypes.c_int),
                ("tree_nodes", ctypes.c_int)]


STEP_FIELDS = ("q", "k_new", "v_new", "block_table", "seq_lens",
               "target_logits", "draft_logits", "draft_tokens", "uniforms",
               "out", "lse", "out_tokens", "n_accepted", "allowed",
               "tree_mask", "parents", "node_tokens", "out_nodes")


class SvpError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn} returned {status} ({msg})")
        self.status = status


_lock = threading.Lock()
_lib = None


_variants = {}


def load_library(path: str = LIB_PATH):
    """Load libsvp.so (raises if it has not been built).  Another path loads
    a separately built copy of the library (its own kernels and device
    state), e.g. a test build."""
    global _lib
    with _lock:
        if path == LIB_PATH and _lib is not None:
            return _lib
        if path in _variants:
            return _variants[path]
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(path)
        vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        dims_p = ctypes.POINTER(SvpDims)
        lib.paged_decode_attention.argtypes = [dims_p, vp, vp, vp, vp, vp, i32,
                                               i32, i32, f32, vp, vp, vp]
        lib.paged_decode_attention.restype = i32
        lib.paged_decode_attention_noalloc.argtypes = [dims_p, vp, vp, vp, vp,
                                                       vp, i32, i32, i32, f32,
                                                       vp, vp, vp]
        lib.paged_decode_attention_noalloc.restype = i32
        lib.paged_tree_attention.argtypes = [dims_p, vp, vp, vp, vp, vp, i32,
                                             vp, f32, vp, vp, vp]
        lib.paged_tree_attention.restype = i32
        lib.paged_decode_workspace_size.argtypes = [dims_p, i32, i32, i32]
        lib.paged_decode_workspace_size.restype = sz
        lib.kv_append.argtypes = [dims_p, vp, vp, vp, vp, vp, vp, i32, vp]
        lib.kv_append.restype = i32
        lib.kv_gather.argtypes = [dims_p, vp, vp, vp, vp, vp, i32, vp, vp, vp]
        lib.kv_gather.restype = i32
        lib.paged_score_update.argtypes = [dims_p, vp, vp, vp, vp, vp, i32, i32,
                                           i32, vp, f32, i32, vp, vp]
        lib.paged_score_update.restype = i32
        lib.kv_evict.argtypes = [dims_p, vp, vp, vp, vp, vp, i32, i32, i32, vp,
                                 i32, vp, vp, vp]
        lib.kv_evict.restype = i32
        lib.kv_page_bounds.argtypes = [dims_p, vp, vp, vp, i32, vp, vp]
        lib.paged_page_scores.argtypes = [dims_p, vp, vp, vp, vp, i32, f32, vp, vp]
        lib.paged_select_pages.argtypes = [i32, i32, i32, vp, vp, i32, i32, i32,
                                           vp, vp]
        lib.paged_sparse_attention.argtypes = [dims_p, vp, vp, vp, vp, vp, i32,
                                               vp, i32, vp, f32, vp, vp, vp]
        lib.kv_assign_pages.argtypes = [i32, i32, i32, vp, vp, vp, vp, vp, i32,
                                        vp, i32, vp, vp]
        lib.kv_append_slots.argtypes = [dims_p, vp, vp, vp, vp, vp, i32, vp]
        lib.token_logprobs.argtypes = [i32, i32, i32, vp, vp, i32, f32, vp, vp,
                                       vp, vp, vp, vp, vp]
        for name in EXPORTED[EXPORTED.index("kv_page_bounds"):
                             EXPORTED.index("token_logprobs") + 1]:
            getattr(lib, name).restype = i32
        lib.spec_accept.argtypes = [i32, i32, i32, vp, vp, vp, vp, vp, vp, vp]
        lib.spec_accept.restype = i32
        lib.spec_accept_ex.argtypes = ([i32, i32, i32] + [vp] * 4 +
                                       [ctypes.POINTER(SvpAcceptOpts)] +
                                       [vp] * 3)
        lib.spec_accept_ex.restype = i32
        lib.spec_accept_tree.argtypes = [i32, i32, i32] + [vp] * 9
        lib.spec_accept_tree.restype = i32
        lib.svp_step_create.argtypes = [ctypes.POINTER(SvpStepDesc),
                                         ctypes.POINTER(vp)]
        lib.svp_step_create.restype = i32
        lib.svp_step_host_buffer.argtypes = [vp, i32, i32, ctypes.POINTER(sz)]
        lib.svp_step_host_buffer.restype = vp
        lib.svp_step_launch.argtypes = [vp, i32]
        lib.svp_step_launch.restype = i32
        lib.svp_step_wait.argtypes = [vp, i32]
        lib.svp_step_wait.restype = i32
        lib.svp_step_stream.argtypes = [vp]
        lib.svp_step_stream.restype = vp
        lib.svp_step_destroy.argtypes = [vp]
        lib.svp_step_destroy.restype = i32
        lib.svp_read_device_status.argtypes = [vp, ctypes.POINTER(i32)]
        lib.svp_read_device_status.restype = i32
        lib.svp_status_string.argtypes = [i32]
        lib.svp_status_string.restype = ctypes.c_char_p
        lib.svp_last_launch_count.argtypes = []
        lib.svp_last_launch_count.restype = i32
        if path == LIB_PATH:
            _lib = lib
        else:
            _variants[path] = lib
        return lib


def _check(fn, status):
    if status != SVP_OK:
        msg = _lib.svp_status_string(status).decode()
        raise SvpError(fn, status, msg)


def _stream_handle(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SVP_F32
    if t.dtype == torch.bfloat16:
        return SVP_BF16
    raise TypeError(f"q/k/v must be float32 or bfloat16, got {t.dtype}")


_FP8_TYPES = (torch.uint8, getattr(torch, "float8_e4m3fn", torch.uint8))


def fp4_row_bytes(head_dim: int) -> int:
    """Bytes of a 4-bit cache row: head_dim/2 of E2M1 codes (element 2i in the
    low nibble of byte i), then head_dim/16 E4M3 scales.  A 4-bit cache is a
    uint8 tensor [num_blocks, Hkv, 16, fp4_row_bytes(head_dim)]."""
    return head_dim // 2 + head_dim // 16


_FP4_DIMS = {fp4_row_bytes(d): d for d in (64, 128)}


def _head_dim(cache):
    """head_dim of a cache: its last dimension, or what a 4-bit row holds
    (36 and 72 bytes are no FP8 head_dim)."""
    n = cache.shape[-1]
    return _FP4_DIMS.get(n, n) if cache.dtype == torch.uint8 else n


def _is_fp4(cache):
    return cache.dtype == torch.uint8 and cache.shape[-1] in _FP4_DIMS


def _cache_code(k_cache, q_dtype):
    """dtype code of a call: the cache's; an FP8 E4M3 cache (uint8 codes or
    float8_e4m3fn) and a 4-bit cache (uint8 rows of fp4_row_bytes) pair with
    bf16 q / out / new rows."""
    if k_cache.dtype in _FP8_TYPES:
        _need(q_dtype == torch.bfloat16,
              "an FP8 or FP4 cache takes bf16 q, out and new rows")
        return SVP_FP4_E2M1 if _is_fp4(k_cache) else SVP_FP8_E4M3
    _need(k_cache.dtype == q_dtype, "q and the caches must share a dtype")
    return _dtype_code(k_cache)


def _need(cond, what):
    if not cond:
        raise ValueError(what)


def _cuda_contig(t, name):
    _need(t.is_cuda, f"{name} must be a CUDA tensor")
    _need(t.is_contiguous(), f"{name} must be contiguous")


def make_dims(q_shape, k_cache, block_table, dtype_code, workspace=None,
              split_pages=0, kernel_path=0, k_scale=1.0, v_scale=1.0):
    B, _, Hq, D = q_shape
    nb, Hkv, bs, D2 = k_cache.shape
    d = SvpDims()
    d.batch, d.num_q_heads, d.num_kv_heads, d.head_dim = B, Hq, Hkv, D
    d.block_size, d.max_blocks_per_seq, d.num_blocks = bs, block_table.shape[1], nb
    d.dtype = dtype_code
    d.split_pages = int(split_pages)
    d.kernel_path = int(kernel_path)
    d.k_scale = float(k_scale)
    d.v_scale = float(v_scale)
    if workspace is not None:
        d.workspace = ctypes.c_void_p(workspace.data_ptr())
        d.workspace_bytes = workspace.numel() * workspace.element_size()
    return d


_ws_cache: dict = {}


def workspace_for(dims: SvpDims, q_len: int, n_sink: int, window: int,
                  device) -> torch.Tensor:
    """A workspace of at least the required size, kept per device and
    reused (calls that share it must not overlap on the GPU).  None for a
    request the library rejects."""
    lib = load_library()
    need = int(lib.paged_decode_workspace_size(ctypes.byref(dims), q_len,
                                               n_sink, window))
    if need == 0:  # an invalid request: the call itself reports the status
        return None
    key = torch.device(device).index or 0
    ws = _ws_cache.get(key)
    if ws is None or ws.numel() < need:
        ws = torch.zeros(need, dtype=torch.uint8, device=device)
        _ws_cache[key] = ws
    return ws


def paged_decode_attention(q, k_cache, v_cache, block_table, seq_lens,
                           q_len=None, n_sink=0, window=0, scale=None,
                           out=None, lse=None, workspace=None, split_pages=0,
                           kernel_path=PATH_AUTO, stream=None, k_scale=1.0,
                           v_scale=1.0):
    """out [B, q_len, Hq, D] (q's dtype) and lse [B, q_len, Hq] fp32 of paged
    decode/verify attention (include/svp.h: paged_decode_attention).  FP8
    E4M3 caches (uint8 codes or float8_e4m3fn) and 4-bit caches (uint8 rows of
    fp4_row_bytes(D)) take bf16 q and their k_scale / v_scale."""
    if _is_fp4(k_cache):
        _need(q_len is None or q_len == q.shape[1], "q.shape[1] must equal q_len")
        r = (_calls or _load_calls()).attention_fp4(
            q, k_cache, v_cache, block_table, seq_lens, n_sink, window, None,
            scale, out, lse, workspace, split_pages, kernel_path, _raw(stream),
            k_scale, v_scale)
        return r if type(r) is tuple else _check("paged_decode_attention", r)
    return _attention(q, k_cache, v_cache, block_table, seq_lens, q_len,
                      n_sink, window, None, scale, out, lse, workspace,
                      split_pages, kernel_path, stream, k_scale, v_scale)


def paged_tree_attention(q, k_cache, v_cache, block_table, seq_lens,
                         tree_mask, scale=None, out=None, lse=None,
                         workspace=None, split_pages=0, kernel_path=PATH_AUTO,
                         stream=None, k_scale=1.0, v_scale=1.0):
    """Draft-tree verify attention (include/svp.h: paged_tree_attention).
    tree_mask: int32 (or uint32) [B, q_len] on the GPU, bit k of entry
    (b, i) set iff node k is an ancestor of node i or i itself."""
    if _is_fp4(k_cache):
        _need(tree_mask is not None, "tree_mask must be int32/uint32 [B, q_len]")
        r = (_calls or _load_calls()).attention_fp4(
            q, k_cache, v_cache, block_table, seq_lens, 0, 0, tree_mask, scale,
            out, lse, workspace, split_pages, kernel_path, _raw(stream), k_scale,
            v_scale)
        return r if type(r) is tuple else _check("paged_tree_attention", r)
    _cuda_contig(tree_mask, "tree_mask")
    _need(tree_mask.dtype in (torch.int32, getattr(torch, "uint32", torch.int32))
          and tuple(tree_mask.shape) == tuple(q.shape[:2]),
          "tree_mask must be int32/uint32 [B, q_len]")
    return _attention(q, k_cache, v_cache, block_table, seq_lens, None, 0, 0,
                      tree_mask, scale, out, lse, workspace, split_pages,
                      kernel_path, stream, k_scale, v_scale)


def _attention(q, k_cache, v_cache, block_table, seq_lens, q_len, n_sink,
               window, tree_mask, scale, out, lse, workspace, split_pages,
               kernel_path, stream, k_scale=1.0, v_scale=1.0):
    lib = load_library()
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache"),
                 (block_table, "block_table"), (seq_lens, "seq_lens")):
        _cuda_contig(t, n)
    code = _cache_code(k_cache, q.dtype)
    _need(v_cache.dtype == k_cache.dtype, "k_cache and v_cache must share a dtype")
    _need(k_cache.shape == v_cache.shape and k_cache.dim() == 4,
          "k_cache/v_cache must be [num_blocks, Hkv, block_size, D]")
    _need(block_table.dtype == torch.int32 and block_table.dim() == 2,
          "block_table must be int32 [B, max_blocks]")
    _need(seq_lens.dtype == torch.int32 and seq_lens.dim() == 1,
          "seq_lens must be int32 [B]")
    B, ql, Hq, D = q.shape
    q_len = ql if q_len is None else q_len
    _need(ql == q_len, "q.shape[1] must equal q_len")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, q_len, Hq), dtype=torch.float32, device=q.device)
    _cuda_contig(out, "out")
    _cuda_contig(lse, "lse")
    dims = make_dims(q.shape, k_cache, block_table, code, None, split_pages,
                     kernel_path, k_scale, v_scale)
    if workspace is None:
        workspace = workspace_for(dims, q_len, n_sink, window, q.device)
    if workspace is not None:
        dims.workspace = ctypes.c_void_p(workspace.data_ptr())
        dims.workspace_bytes = workspace.numel() * workspace.element_size()
    if tree_mask is None:
        st = lib.paged_decode_attention(
            ctypes.byref(dims), q.data_ptr(), k_cache.data_ptr(),
            v_cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
            int(q_len), int(n_sink), int(window), float(scale),
            out.data_ptr(), lse.data_ptr(), _stream_handle(stream, q.device))
        _check("paged_decode_attention", st)
    else:
        st = lib.paged_tree_attention(
            ctypes.byref(dims), q.data_ptr(), k_cache.data_ptr(),
            v_cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
            int(q_len), tree_mask.data_ptr(), float(scale), out.data_ptr(),
            lse.data_ptr(), _stream_handle(stream, q.device))
        _check("paged_tree_attention", st)
    return out, lse


# ---- the 4-bit cache, gather, score and eviction calls: csrc/calls.cpp checks
# their arguments, makes their outputs and calls the library ----
CALLS_PATH = os.path.join(_HERE, "svp_calls.so")
_calls = None


def _load_calls():
    """The marshalling module (raises if it has not been built)."""
    global _calls
    if _calls is None:
        load_library()
        if not os.path.exists(CALLS_PATH):
            raise RuntimeError(
                f"{CALLS_PATH} is missing: build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'`")
        import importlib.util
        spec = importlib.util.spec_from_file_location("svp_calls", CALLS_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        built = getattr(module, "torch_version", "of another version")
        if built != torch.__version__:
            raise RuntimeError(
                f"{CALLS_PATH} was built for torch {built}, this is "
                f"{torch.__version__}: build it again with "
                "`python -c 'import __graft_entry__ as g; g.build()'`")
        _calls = module
    return _calls


def _raw(stream):
    return None if stream is None else stream.cuda_stream


def kv_append(k_new, v_new, k_cache, v_cache, block_table=None, seq_lens=None,
              stream=None, k_scale=1.0, v_scale=1.0, slots=None):
    """Scatter k_new/v_new [B, n_new, Hkv, D] into the paged caches in place
    (include/svp.h: kv_append).  seq_lens are the lengths after the append.
    Into FP8 and 4-bit caches the bf16 rows are quantised with k_scale /
    v_scale.

    With slots (int64 [n_rows], as kv_assign_pages makes them, instead of
    block_table and seq_lens) the rows are packed, [n_rows, Hkv, D], and row i
    goes to slot slots[i]; a negative slot stores nothing (include/svp.h:
    kv_append_slots)."""
    if slots is not None:
        _need(block_table is None and seq_lens is None,
              "kv_append takes either slots or block_table and seq_lens")
        st = (_calls or _load_calls()).append_slots(
            k_new, v_new, k_cache, v_cache, slots, _raw(stream), k_scale, v_scale)
        return None if st is None else _check("kv_append_slots", st)
    _need(block_table is not None and seq_lens is not None,
          "kv_append takes block_table and seq_lens, or slots")
    if _is_fp4(k_cache):
        st = (_calls or _load_calls()).append_fp4(
            k_new, v_new, k_cache, v_cache, block_table, seq_lens, _raw(stream),
            k_scale, v_scale)
        return None if st is None else _check("kv_append", st)
    lib = load_library()
    for t, n in ((k_new, "k_new"), (v_new, "v_new"), (k_cache, "k_cache"),
                 (v_cache, "v_cache"), (block_table, "block_table"),
                 (seq_lens, "seq_lens")):
        _cuda_contig(t, n)
    code = _cache_code(k_cache, k_new.dtype)
    _need(v_new.dtype == k_new.dtype and v_cache.dtype == k_cache.dtype,
          "k_new/v_new and k_cache/v_cache must pair up")
    B, n_new, Hkv, D = k_new.shape
    dims = make_dims((B, n_new, Hkv, D), k_cache, block_table, code,
                     k_scale=k_scale, v_scale=v_scale)
    st = lib.kv_append(ctypes.byref(dims), k_new.data_ptr(), v_new.data_ptr(),
                       k_cache.data_ptr(), v_cache.data_ptr(),
                       block_table.data_ptr(), seq_lens.data_ptr(), int(n_new),
                       _stream_handle(stream, k_cache.device))
    _check("kv_append", st)


def _any_cache_code(cache):
    if _is_fp4(cache):
        return SVP_FP4_E2M1
    return SVP_FP8_E4M3 if cache.dtype in _FP8_TYPES else _dtype_code(cache)


def kv_gather(k_cache, v_cache, block_table, seq_lens, n_rows, starts=None,
              k_out=None, v_out=None, stream=None, k_scale=1.0, v_scale=1.0):
    """The inverse of kv_append (include/svp.h: kv_gather): k and v
    [B, n_rows, Hkv, D] (fp32 of an fp32 cache, else bf16), the values at
    logical positions starts[b] .. starts[b] + n_rows - 1 (int32 [B]; without
    it the newest n_rows); zeros outside the sequence."""
    r = (_calls or _load_calls()).gather(
        k_cache, v_cache, block_table, seq_lens, n_rows, starts, k_out, v_out,
        _raw(stream), k_scale, v_scale)
    return r if type(r) is tuple else _check("kv_gather", r)


def paged_score_update(q, k_cache, lse, block_table, seq_lens, scores,
                       n_fresh=None, n_sink=0, window=0, tree_mask=None,
                       scale=None, k_scale=1.0, stream=None):
    """Adds to scores [num_blocks, Hkv, 16] fp32, in place, the attention
    weight that every cached key received from the query rows q
    [B, q_len, Hq, D], lse [B, q_len, Hq] being what the attention call with
    the same arguments returned (include/svp.h: paged_score_update).  The
    newest n_fresh positions (default: q_len) start from zero.  Returns
    scores.

    No page may stand twice among the sequences of one call: its scores are
    read and written back once for each, and one update would be lost.
    Sequences that share pages (a common prefix) are updated in calls of their
    own, one after another; a shared page's scores then count them all.

    Rows whose lse is -inf add nothing.  After a verification,
    lse.masked_fill_((arange(q_len) > n_accepted[:, None])[..., None], -inf)
    leaves the rejected drafts' rows out; the next step's rows then start from
    zero where those stood."""
    st = (_calls or _load_calls()).score_update(
        q, k_cache, lse, block_table, seq_lens, scores, n_fresh, n_sink, window,
        tree_mask, scale, k_scale, _raw(stream))
    return scores if st is None else _check("paged_score_update", st)


def kv_evict(k_cache, v_cache, scores, block_table, seq_lens, budget, n_sink=0,
             n_recent=0, dst_block_table=None, kept=None, new_lens=None,
             stream=None):
    """Every (sequence, kv head) longer than `budget` keeps its first n_sink
    rows, its newest n_recent and the best-scored others, in order, as the
    first rows of dst_block_table's pages (default: in place); scores move
    along (include/svp.h: kv_evict).  Returns (kept [B, Hkv, budget] int32
    positions, -1 padded, new_lens [B] int32).

    In place, a sequence's pages are its own and its block table has room for
    the budget.  Sequences that share pages go to pages of their own: the
    source pages, scores included, are then only read."""
    r = (_calls or _load_calls()).evict(
        k_cache, v_cache, scores, block_table, seq_lens, budget, n_sink,
        n_recent, dst_block_table, kept, new_lens, _raw(stream))
    return r if type(r) is tuple else _check("kv_evict", r)


def kv_page_bounds(k_cache, block_table, seq_lens, bounds, n_new=None,
                   stream=None):
    """Elementwise smallest and largest K of every page that holds one of the
    newest n_new positions of a sequence (default: of every page), per kv head,
    into bounds [num_blocks, Hkv, 2, D] bf16, in place (include/svp.h:
    kv_page_bounds).  Called after each append with its n_new, before
    paged_page_scores.  Returns bounds."""
    st = (_calls or _load_calls()).page_bounds(
        k_cache, block_table, seq_lens, bounds, n_new, _raw(stream))
    return bounds if st is None else _check("kv_page_bounds", st)


def paged_page_scores(q, bounds, block_table, seq_lens, scale=None, k_scale=1.0,
                      scores=None, stream=None):
    """scores [B, Hkv, max_blocks] fp32: what scale * k_scale * <q, K> can be at
    most for a key of the page, the largest over the kv head's query rows
    (include/svp.h: paged_page_scores); -inf past a sequence's pages."""
    r = (_calls or _load_calls()).page_scores(
        q, bounds, block_table, seq_lens, scale, k_scale, scores, _raw(stream))
    return r if type(r) is not int else _check("paged_page_scores", r)


def paged_select_pages(scores, seq_lens, n_select, n_sink=0, n_recent=1,
                       pages=None, stream=None):
    """pages [B, Hkv, n_select] int32: per sequence and kv head the first n_sink
    pages, the newest n_recent and the best-scored others, in increasing order,
    -1 padded (include/svp.h: paged_select_pages).  For a query to see its own
    key (and the drafts before it) n_recent covers the pages of the newest
    q_len positions: (q_len + 30) // 16."""
    r = (_calls or _load_calls()).select_pages(
        scores, seq_lens, n_select, n_sink, n_recent, pages, _raw(stream))
    return r if type(r) is not int else _check("paged_select_pages", r)


def paged_sparse_attention(q, k_cache, v_cache, block_table, seq_lens, pages,
                           tree_mask=None, scale=None, out=None, lse=None,
                           split_pages=0, stream=None, k_scale=1.0, v_scale=1.0):
    """out [B, q_len, Hq, D] and lse [B, q_len, Hq] of attention over the pages
    listed in pages [B, Hkv, n_select] int32 only (include/svp.h:
    paged_sparse_attention), causal within the newest q_len positions or, with
    tree_mask, along the draft tree.  Negative entries are holes.  A row that
    sees no listed key gets zeros and -inf."""
    r = (_calls or _load_calls()).sparse_attention(
        q, k_cache, v_cache, block_table, seq_lens, pages, tree_mask, scale, out,
        lse, split_pages, _raw(stream), k_scale, v_scale)
    return r if type(r) is tuple else _check("paged_sparse_attention", r)


def kv_assign_pages(block_table, seq_lens, new_lens, free_pages, free_count,
                    n_slots=None, slots=None, offsets=None, num_blocks=None,
                    stream=None):
    """Takes the sequences from seq_lens to new_lens (int32 [B]), in place:
    pages past the new lengths go back onto the stack free_pages (int32
    [capacity], free_count int32 [1] entries), missing ones are taken from it
    (include/svp.h: kv_assign_pages).  Returns (slots, offsets): with n_slots
    (or slots, int64 [n_slots]) the slots of the new positions, packed in the
    order of the sequences and -1 padded, for kv_append(slots=...), else None;
    offsets int32 [B + 1] say where each sequence's begin.  Ids outside
    [0, num_blocks) get no slot.

    Where pages run out, no sequence from the first that does not fit on that
    needs a new page is served, where slots do, none that has new positions:
    seq_lens (!= new_lens) and table stay as they were, slots are -1, and
    read_device_status() has DEV_NO_PAGES.  Sequences that shrink or, while
    slots suffice, grow within their last page are served all the same."""
    r = (_calls or _load_calls()).assign_pages(
        block_table, seq_lens, new_lens, free_pages, free_count, n_slots, slots,
        offsets, num_blocks, _raw(stream))
    return r if type(r) is tuple else _check("kv_assign_pages", r)


def token_logprobs(logits, tokens, n_top=0, temperature=1.0, allowed=None,
                   logprobs=None, entropy=None, ranks=None, top_logprobs=None,
                   top_tokens=None, stream=None):
    """(logprobs, entropy, ranks, top_logprobs, top_tokens) of int32 tokens
    [...] under softmax(logits / temperature), logits [..., V] fp32 or bf16,
    over the tokens that the mask `allowed` (int32/uint32 [..., ceil(V/32)], as
    spec_accept takes it) lets take part; top_* [..., n_top] are the most likely
    tokens (include/svp.h: token_logprobs).  Negative tokens are padding, so
    spec_accept's out_tokens go with its target_logits as they are."""
    r = (_calls or _load_calls()).logprobs(
        logits, tokens, n_top, temperature, allowed, logprobs, entropy, ranks,
        top_logprobs, top_tokens, _raw(stream))
    return r if type(r) is tuple else _check("token_logprobs", r)


def spec_accept(target_logits, draft_logits, draft_tokens, uniforms,
                out_tokens=None, n_accepted=None, stream=None,
                temperature=1.0, allowed=None, greedy=False):
    """Speculative acceptance (include/svp.h: spec_accept; with a
    temperature other than 1, an `allowed` token mask (int32/uint32
    [B, K+1, ceil(V/32)] on the GPU) or greedy=True: spec_accept_ex).
    Returns (out_tokens [B, K+1] int32, n_accepted [B] int32)."""
    lib = load_library()
    for t, n in ((target_logits, "target_logits"),
                 (draft_logits, "draft_logits"), (draft_tokens, "draft_tokens"),
                 (uniforms, "uniforms")):
        _cuda_contig(t, n)
    _need(target_logits.dtype == torch.float32 and
          draft_logits.dtype == torch.float32 and
          uniforms.dtype == torch.float32, "logits/uniforms must be float32")
    _need(draft_tokens.dtype == torch.int32, "draft_tokens must be int32")
    B, K1, V = target_logits.shape
    K = K1 - 1
    _need(tuple(draft_logits.shape) == (B, K, V), "draft_logits must be [B, K, V]")
    _need(tuple(draft_tokens.shape) == (B, K), "draft_tokens must be [B, K]")
    _need(tuple(uniforms.shape) == (B, K + 1), "uniforms must be [B, K+1]")
    dev = target_logits.device
    if out_tokens is None:
        out_tokens = torch.empty((B, K + 1), dtype=torch.int32, device=dev)
    if n_accepted is None:
        n_accepted = torch.empty((B,), dtype=torch.int32, device=dev)
    if temperature == 1.0 and allowed is None and not greedy:
        st = lib.spec_accept(B, K, V, target_logits.data_ptr(),
                             draft_logits.data_ptr(), draft_tokens.data_ptr(),
                             uniforms.data_ptr(), out_tokens.data_ptr(),
                             n_accepted.data_ptr(), _stream_handle(stream, dev))
        _check("spec_accept", st)
        return out_tokens, n_accepted
    if allowed is not None:
        _cuda_contig(allowed, "allowed")
        _need(tuple(allowed.shape) == (B, K + 1, (V + 31) // 32) and
              allowed.element_size() == 4,
              "allowed must be 32-bit [B, K+1, ceil(V/32)]")
    opts = SvpAcceptOpts(float(temperature),
                         None if allowed is None else allowed.data_ptr(),
                         int(bool(greedy)))
    st = lib.spec_accept_ex(B, K, V, target_logits.data_ptr(),
                            draft_logits.data_ptr(), draft_tokens.data_ptr(),
                            uniforms.data_ptr(), ctypes.byref(opts),
                            out_tokens.data_ptr(), n_accepted.data_ptr(),
                            _stream_handle(stream, dev))
    _check("spec_accept_ex", st)
    return out_tokens, n_accepted


def spec_accept_tree(target_logits, draft_logits, parents, node_tokens,
                     uniforms, out_tokens=None, out_nodes=None,
                     n_accepted=None, stream=None):
    """Tree acceptance (include/svp.h: spec_accept_tree).  Returns
    (out_tokens [B, N] int32, out_nodes [B, N] int32, n_accepted [B] int32)."""
    lib = load_library()
    for t, n in ((target_logits, "target_logits"),
                 (draft_logits, "draft_logits"), (parents, "parents"),
                 (node_tokens, "node_tokens"), (uniforms, "uniforms")):
        _cuda_contig(t, n)
    _need(target_logits.dtype == torch.float32 and
          draft_logits.dtype == torch.float32 and
          uniforms.dtype == torch.float32, "logits/uniforms must be float32")
    _need(parents.dtype == torch.int32 and node_tokens.dtype == torch.int32,
          "parents/node_tokens must be int32")
    B, N, V = target_logits.shape
    _need(tuple(draft_logits.shape) == (B, N, V), "draft_logits must be [B, N, V]")
    for t, n in ((parents, "parents"), (node_tokens, "node_tokens"),
                 (uniforms, "uniforms")):
        _need(tuple(t.shape) == (B, N), f"{n} must be [B, N]")
    dev = target_logits.device
    if out_tokens is None:
        out_tokens = torch.empty((B, N), dtype=torch.int32, device=dev)
    if out_nodes is None:
        out_nodes = torch.empty((B, N), dtype=torch.int32, device=dev)
    if n_accepted is None:
        n_accepted = torch.empty((B,), dtype=torch.int32, device=dev)
    st = lib.spec_accept_tree(B, N, V, target_logits.data_ptr(),
                              draft_logits.data_ptr(), parents.data_ptr(),
                              node_tokens.data_ptr(), uniforms.data_ptr(),
                              out_tokens.data_ptr(), out_nodes.data_ptr(),
                              n_accepted.data_ptr(), _stream_handle(stream, dev))
    _check("spec_accept_tree", st)
    return out_tokens, out_nodes, n_accepted


def read_device_status(stream=None, device=None) -> int:
    """Synchronise and return (and clear) the device-side SVP_DEV_* flags."""
    lib = load_library()
    flags = ctypes.c_int(0)
    st = lib.svp_read_device_status(_stream_handle(stream, device),
                                    ctypes.byref(flags))
    _check("svp_read_device_status", st)
    return flags.value


def last_launch_count() -> int:
    """Kernels launched by the last successful library call on this thread."""
    return int(load_library().svp_last_launch_count())


class StepRunner:
    """The graph-captured decode step (include/svp.h: svp_step_*): two
    ping-pong slots of pinned host buffers, each replayed as one CUDA graph
    (input copy, kv_append, attention, acceptance) with its result copied
    back on a separate stream.  host(slot, name) returns a numpy view of a
    slot's pinned buffer (bf16 as uint16 bits).  Draft chains take the
    verify epilogue options (temperature, greedy, use_mask: the token mask
    in field "allowed"); tree_nodes > 0 makes the step a draft-tree verify
    (fields "tree_mask", "parents", "node_tokens"; result "out_nodes")."""

    def __init__(self, k_cache, v_cache, batch, num_q_heads, q_len,
                 max_blocks_per_seq, n_sink=0, window=0, scale=None,
                 num_draft=0, vocab=0, split_pages=0, kernel_path=PATH_AUTO,
                 k_scale=1.0, v_scale=1.0, temperature=1.0, greedy=False,
                 use_mask=False, tree_nodes=0):
        lib = load_library()
        _cuda_contig(k_cache, "k_cache")
        _cuda_contig(v_cache, "v_cache")
        nb, Hkv, bs, _ = k_cache.shape
        D = _head_dim(k_cache)
        code = _any_cache_code(k_cache)
        dims = SvpDims(batch, num_q_heads, Hkv, D, bs, max_blocks_per_seq, nb,
                       code, None, 0, split_pages, kernel_path, k_scale,
                       v_scale)
        if scale is None:
            scale = 1.0 / math.sqrt(D)
        desc = SvpStepDesc(dims, q_len, n_sink, window, float(scale),
                           k_cache.data_ptr(), v_cache.data_ptr(), num_draft,
                           vocab, float(temperature), int(bool(greedy)),
                           int(bool(use_mask)), int(tree_nodes))
        h = ctypes.c_void_p()
        _check("svp_step_create", lib.svp_step_create(ctypes.byref(desc),
                                                      ctypes.byref(h)))
        self._lib, self._h = lib, h
        self._keep = (k_cache, v_cache)
        ed = np.float32 if code == SVP_F32 else np.uint16
        B, Q, K, V, N = batch, q_len, num_draft, vocab, tree_nodes
        rt = N if N else K + 1   # target rows, uniforms, output tokens
        rd = N if N else K       # draft rows
        self._spec = {
            "q": (ed, (B, Q, num_q_heads, D)), "k_new": (ed, (B, Q, Hkv, D)),
            "v_new": (ed, (B, Q, Hkv, D)),
            "block_table": (np.int32, (B, max_blocks_per_seq)),
            "seq_lens": (np.int32, (B,)),
            "target_logits": (np.float32, (B, rt, V)),
            "draft_logits": (np.float32, (B, rd, V)),
            "draft_tokens": (np.int32, (B, K)),
            "uniforms": (np.float32, (B, rt)),
            "out": (ed, (B, Q, num_q_heads, D)),
            "lse": (np.float32, (B, Q, num_q_heads)),
            "out_tokens": (np.int32, (B, rt)),
            "n_accepted": (np.int32, (B,)),
            "allowed": (np.uint32, (B, K + 1, (V + 31) // 32)),
            "tree_mask": (np.uint32, (B, N)),
            "parents": (np.int32, (B, N)),
            "node_tokens": (np.int32, (B, N)),
            "out_nodes": (np.int32, (B, N)),
        }
        self._views = {}

    def host(self, slot, name):
        key = (slot, name)
        if key not in self._views:
            n = ctypes.c_size_t()
            ptr = self._lib.svp_step_host_buffer(self._h, slot,
                                                 STEP_FIELDS.index(name),
                                                 ctypes.byref(n))
            _need(ptr is not None, f"slot {slot} has no field {name}")
            raw = (ctypes.c_uint8 * n.value).from_address(ptr)
            dt, shape = self._spec[name]
            self._views[key] = np.frombuffer(raw, dtype=dt).reshape(shape)
        return self._views[key]

    def launch(self, slot):
        _check("svp_step_launch", self._lib.svp_step_launch(self._h, slot))

    def wait(self, slot):
        _check("svp_step_wait", self._lib.svp_step_wait(self._h, slot))

    def close(self):
        if self._h:
            self._views.clear()
            _check("svp_step_destroy", self._lib.svp_step_destroy(self._h))
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
