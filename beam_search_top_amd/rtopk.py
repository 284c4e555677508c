"""Thin ctypes binding of librtopk.so (declared in include/rtopk.h).

The ``rtopk_*`` functions take integer device addresses and sizes, exactly like
the C ABI, and return its status codes. ``beam_step`` marshals torch tensors
(torch is used only for device memory and the current stream) and raises on a
non-OK status. Every step of the selection runs in the HIP kernels; there is no
fallback: without a built librtopk.so the import of this module's functions
fails loudly.
"""
from __future__ import annotations

import ctypes
import os
import re

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "librtopk.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "rtopk.h")

RTOPK_F32, RTOPK_F16, RTOPK_BF16 = 0, 1, 2
RTOPK_OK, RTOPK_EINVAL, RTOPK_ENOTSUP, RTOPK_ENOMEM, RTOPK_EHIP, RTOPK_ETIMEOUT = 0, -1, -2, -3, -4, -5
RTOPK_MAX_K, RTOPK_MAX_BEAM = 64, 512
RTOPK_WS_FIXED_BYTES = 1310976
RTOPK_NOALLOC_SCRATCH_BYTES = 8388608
RTOPK_DEFAULT_SPIN_LIMIT = 1 << 22
STATUS_NAMES = {0: "RTOPK_OK", -1: "RTOPK_EINVAL", -2: "RTOPK_ENOTSUP", -3: "RTOPK_ENOMEM", -4: "RTOPK_EHIP",
                -5: "RTOPK_ETIMEOUT"}


class RtopkError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class rtopk_plan_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "chunks", "threads", "vecs_per_thread", "vecs_per_chunk", "elems_per_vec", "ngroups",
        "chunk_limit", "queue_cap", "align_elems", "grid", "sort_keys", "lds_bytes", "pieces_per_group",
        "row_local")]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


_lib = None


def load():
    """Load librtopk.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m beam_search_top_amd._build` "
                          "(or __graft_entry__.build()); there is no fallback path")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    step_args = [vp, i32, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp]
    L.rtopk_beam_step.argtypes = step_args + [vp]
    L.rtopk_beam_step.restype = i32
    L.rtopk_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    L.rtopk_workspace_bytes.restype = sz
    L.rtopk_beam_step_ws.argtypes = step_args + [vp, sz, vp]
    L.rtopk_beam_step_ws.restype = i32
    L.rtopk_beam_step_noalloc.argtypes = step_args + [vp]
    L.rtopk_beam_step_noalloc.restype = i32
    L.rtopk_debug_step.argtypes = step_args + [vp, sz, vp, vp, vp, vp, vp, vp]
    L.rtopk_debug_step.restype = i32
    L.rtopk_plan.argtypes = [vp, i32, i32, i32, i32, i32, ctypes.POINTER(rtopk_plan_t)]
    L.rtopk_plan.restype = i32
    L.rtopk_set_override.argtypes = [i32, i32]
    L.rtopk_set_override.restype = i32
    L.rtopk_set_row_local.argtypes = [i32]
    L.rtopk_set_row_local.restype = i32
    L.rtopk_set_split.argtypes = [i32]
    L.rtopk_set_split.restype = i32
    L.rtopk_set_waves.argtypes = [i32]
    L.rtopk_set_waves.restype = i32
    L.rtopk_set_spin_limit.argtypes = [ctypes.c_uint]
    L.rtopk_set_spin_limit.restype = i32
    L.rtopk_check.argtypes = [vp, vp]
    L.rtopk_check.restype = i32
    L.rtopk_beam_step_sharded.argtypes = [ctypes.POINTER(vp), i32, i32, vp, vp, i32, i32, i32, i32, i32,
                                          vp, vp, vp, vp]
    L.rtopk_beam_step_sharded.restype = i32
    L.rtopk_sample_step.argtypes = [vp, i32, i32, i32, i32, ctypes.c_float, ctypes.c_uint64, ctypes.c_uint64,
                                    vp, vp, vp]
    L.rtopk_sample_step.restype = i32
    L.rtopk_lmhead_step.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp]
    L.rtopk_lmhead_step.restype = i32
    L.rtopk_beam_reorder.argtypes = [vp, vp, ctypes.c_longlong, i32, i32, ctypes.c_longlong, vp, i32, vp]
    L.rtopk_beam_reorder.restype = i32
    L.rtopk_page_tables.argtypes = [vp, vp, i32, i32, vp, i32, vp, i32, vp, i32, vp, vp, i32, i32, vp, vp, vp]
    L.rtopk_page_tables.restype = i32
    L.rtopk_cache_store.argtypes = [vp, vp, vp, vp, i32, vp, i32, i32, i32, vp, vp, vp, i32, i32, vp]
    L.rtopk_cache_store.restype = i32
    L.rtopk_tree_attention.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, vp, vp, vp, i32, i32, i32, i32, i32,
                                       ctypes.c_float, vp, vp, vp, sz, vp]
    L.rtopk_tree_attention.restype = i32
    L.rtopk_tree_attention_workspace_bytes.argtypes = [i32] * 7
    L.rtopk_tree_attention_workspace_bytes.restype = sz
    L.rtopk_cross_attention.argtypes = [vp, vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, i32,
                                        ctypes.c_float, vp, vp, vp, sz, vp]
    L.rtopk_cross_attention.restype = i32
    L.rtopk_cross_attention_workspace_bytes.argtypes = [i32] * 6
    L.rtopk_cross_attention_workspace_bytes.restype = sz
    L.rtopk_qk_norm_rope.argtypes = [vp, vp, vp, vp, i32, vp, vp, i32, i32, vp, vp, ctypes.c_float, i32, i32, i32, i32,
                                     vp, vp, vp, vp, vp]
    L.rtopk_qk_norm_rope.restype = i32
    L.rtopk_cache_store_fp8.argtypes = [vp, vp, vp, vp, i32, vp, i32, i32, i32, vp, vp, vp, vp, vp, i32, i32, vp]
    L.rtopk_cache_store_fp8.restype = i32
    L.rtopk_cache_load_fp8.argtypes = [vp, vp, vp, vp, vp, i32, i32, vp, i32, i32, i32, vp, vp, i32, vp]
    L.rtopk_cache_load_fp8.restype = i32
    L.rtopk_tree_attention_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, vp, vp, vp, i32, i32, i32,
                                           i32, i32, ctypes.c_float, vp, vp, vp, sz, vp]
    L.rtopk_tree_attention_fp8.restype = i32
    L.rtopk_tree_attention_fp8_workspace_bytes.argtypes = [i32] * 7
    L.rtopk_tree_attention_fp8_workspace_bytes.restype = sz
    L.rtopk_sample_filtered.argtypes = [vp, i32, i32, i32, ctypes.c_int64, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.rtopk_sample_filtered.restype = i32
    L.rtopk_sample_filtered_workspace_bytes.argtypes = [i32] * 2
    L.rtopk_sample_filtered_workspace_bytes.restype = sz
    L.rtopk_read_probe.argtypes = [vp, sz, ctypes.c_uint32, vp, vp]
    L.rtopk_read_probe.restype = i32
    L.rtopk_read_probe_shape.argtypes = [vp, sz, i32, i32, ctypes.c_uint32, vp, vp]
    L.rtopk_read_probe_shape.restype = i32
    L.rtopk_last_error.argtypes = []
    L.rtopk_last_error.restype = ctypes.c_char_p
    L.rtopk_release.argtypes = []
    L.rtopk_release.restype = None
    _lib = L
    return L


def declared_functions(header=HEADER):
    """Names of the functions include/rtopk.h declares."""
    text = open(header).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(rtopk_[a-z0-9_]+)\s*\(", text)))


# ------------------------------------------------------------------ C-ABI mirror
def rtopk_beam_step(logits, dtype, alive_scores, finished_mask, B, beam, V, k, eos_id,
                    out_beam_ids, out_token_ids, out_scores, stream):
    return load().rtopk_beam_step(logits, dtype, alive_scores, finished_mask, B, beam, V, k, eos_id,
                                  out_beam_ids, out_token_ids, out_scores, stream)


def rtopk_workspace_bytes(B, beam, V, k, dtype):
    return load().rtopk_workspace_bytes(B, beam, V, k, dtype)


def rtopk_beam_step_ws(logits, dtype, alive_scores, finished_mask, B, beam, V, k, eos_id,
                       out_beam_ids, out_token_ids, out_scores, workspace, ws_bytes, stream):
    return load().rtopk_beam_step_ws(logits, dtype, alive_scores, finished_mask, B, beam, V, k, eos_id,
                                     out_beam_ids, out_token_ids, out_scores, workspace, ws_bytes, stream)


def rtopk_beam_step_noalloc(logits, dtype, alive_scores, finished_mask, B, beam, V, k, eos_id,
                            out_beam_ids, out_token_ids, out_scores, stream):
    return load().rtopk_beam_step_noalloc(logits, dtype, alive_scores, finished_mask, B, beam, V, k, eos_id,
                                          out_beam_ids, out_token_ids, out_scores, stream)


def rtopk_debug_step(logits, dtype, alive_scores, finished_mask, B, beam, V, k, eos_id,
                     out_beam_ids, out_token_ids, out_scores, workspace, ws_bytes,
                     dbg_T, dbg_hits, dbg_lse, dbg_count, dbg_queue, stream):
    return load().rtopk_debug_step(logits, dtype, alive_scores, finished_mask, B, beam, V, k, eos_id,
                                   out_beam_ids, out_token_ids, out_scores, workspace, ws_bytes,
                                   dbg_T, dbg_hits, dbg_lse, dbg_count, dbg_queue, stream)


def rtopk_plan(logits, B, beam, V, k, dtype):
    """Returns (status, rtopk_plan_t)."""
    p = rtopk_plan_t()
    st = load().rtopk_plan(logits, B, beam, V, k, dtype, ctypes.byref(p))
    return st, p


def rtopk_set_override(vecs_per_thread, chunk_limit):
    return load().rtopk_set_override(vecs_per_thread, chunk_limit)


def rtopk_set_row_local(enable):
    return load().rtopk_set_row_local(enable)


def rtopk_set_split(enable):
    return load().rtopk_set_split(enable)


def rtopk_set_waves(waves):
    return load().rtopk_set_waves(waves)


def rtopk_set_spin_limit(polls):
    return load().rtopk_set_spin_limit(polls)


def rtopk_check(workspace, stream):
    return load().rtopk_check(workspace, stream)


def rtopk_beam_step_sharded(shards, dtype, alive_scores, finished_mask, B, beam, V_shard, k, eos_id,
                            out_beam_ids, out_token_ids, out_scores, stream):
    """`shards` is a Python sequence of device addresses (marshalled into the host array)."""
    arr = (ctypes.c_void_p * len(shards))(*shards) if shards is not None else None
    return load().rtopk_beam_step_sharded(arr, len(shards) if shards is not None else 0, dtype, alive_scores,
                                          finished_mask, B, beam, V_shard, k, eos_id, out_beam_ids,
                                          out_token_ids, out_scores, stream)


def beam_step_sharded(shards, alive, finished=None, k=None, eos_id=2):
    """One selection step over vocabulary shards (torch device tensors
    [B, beam, V_shard] of one dtype, shard g holding vocabulary indices
    g*V_shard ...), on the current stream. Returns (beam_ids, token_ids, scores)."""
    import torch
    s0 = shards[0]
    if any(t.shape != s0.shape or t.dtype != s0.dtype or not t.is_contiguous() for t in shards):
        raise ValueError("shards must be contiguous tensors of one shape and dtype")
    if not s0.is_cuda:
        raise ValueError("shards must be device tensors")
    for g, t in enumerate(shards):
        _on_device(t, s0.device, f"shard {g}")
    if k is None:
        k = s0.shape[1]
    B, beam, Vs = s0.shape
    _, _, _, finished, outs = _prepare(s0, alive, finished, k)
    stream = torch.cuda.current_stream(s0.device).cuda_stream
    _check(rtopk_beam_step_sharded([_ptr(t) for t in shards], dtype_code(s0), _ptr(alive), _ptr(finished),
                                   B, beam, Vs, k, eos_id, _ptr(outs[0]), _ptr(outs[1]), _ptr(outs[2]), stream))
    return outs


def rtopk_sample_step(logits, dtype, R, V, k, temperature, seed, step, out_token, out_logprob, stream):
    return load().rtopk_sample_step(logits, dtype, R, V, k, temperature, seed, step, out_token, out_logprob,
                                    stream)


def sample_step(logits, k, temperature=1.0, seed=0, step=0):
    """Top-k sampling of every row of logits [R, V] (torch device tensor) on
    the current stream. Returns (tokens [R] int32, logprobs [R] float32)."""
    import torch
    if logits.dim() != 2 or not logits.is_contiguous() or not logits.is_cuda:
        raise ValueError("logits must be a contiguous [R, V] device tensor")
    R, V = logits.shape
    tok = torch.empty(R, dtype=torch.int32, device=logits.device)
    lp = torch.empty(R, dtype=torch.float32, device=logits.device)
    stream = torch.cuda.current_stream(logits.device).cuda_stream
    _check(rtopk_sample_step(_ptr(logits), dtype_code(logits), R, V, k, float(temperature), int(seed), int(step),
                             _ptr(tok), _ptr(lp), stream))
    return tok, lp


def rtopk_lmhead_step(hidden, weight, alive_scores, finished_mask, B, beam, H, V, k, eos_id,
                      out_beam_ids, out_token_ids, out_scores, stream):
    return load().rtopk_lmhead_step(hidden, weight, alive_scores, finished_mask, B, beam, H, V, k, eos_id,
                                    out_beam_ids, out_token_ids, out_scores, stream)


def lmhead_step(hidden, weight, alive, finished=None, k=None, eos_id=2):
    """The step fused into the LM head, on torch device tensors (current
    stream): hidden [B*beam, H] and weight [V, H] bfloat16, alive [B, beam]
    float32, finished [B, beam] bool/uint8 or None. Returns (beam_ids,
    token_ids, scores), each [B, k]."""
    import torch
    if hidden.dtype != torch.bfloat16 or weight.dtype != torch.bfloat16:
        raise ValueError("hidden and weight must be bfloat16")
    if hidden.dim() != 2 or weight.dim() != 2 or hidden.shape[1] != weight.shape[1]:
        raise ValueError("hidden must be [B*beam, H] and weight [V, H]")
    if not (hidden.is_contiguous() and weight.is_contiguous()) or not hidden.is_cuda:
        raise ValueError("hidden and weight must be contiguous device tensors")
    dev = hidden.device
    _on_device(weight, dev, "weight")
    _on_device(alive, dev, "alive")
    if alive.dim() != 2 or alive.dtype != torch.float32 or not alive.is_contiguous():
        raise ValueError("alive must be a contiguous float32 [B, beam] tensor")
    B, beam = alive.shape
    if hidden.shape[0] != B * beam:
        raise ValueError("hidden must have B*beam rows")
    if finished is not None:
        _on_device(finished, dev, "finished")
        if finished.shape != (B, beam) or finished.dtype not in (torch.uint8, torch.bool):
            raise ValueError("finished must be a [B, beam] uint8/bool tensor")
        finished = finished.contiguous()
        if finished.dtype == torch.bool:
            finished = finished.view(torch.uint8)
    if k is None:
        k = beam
    V, H = weight.shape
    outs = (torch.empty((B, k), dtype=torch.int32, device=dev), torch.empty((B, k), dtype=torch.int32, device=dev),
            torch.empty((B, k), dtype=torch.float32, device=dev))
    stream = torch.cuda.current_stream(dev).cuda_stream
    _check(rtopk_lmhead_step(_ptr(hidden), _ptr(weight), _ptr(alive), _ptr(finished), B, beam, H, V, k, eos_id,
                             _ptr(outs[0]), _ptr(outs[1]), _ptr(outs[2]), stream))
    return outs


def rtopk_beam_reorder(src, dst, nslabs, B, beam, row_bytes, beam_ids, ld, stream):
    return load().rtopk_beam_reorder(src, dst, nslabs, B, beam, row_bytes, beam_ids, ld, stream)


def rtopk_page_tables(cache_lens, new_lens, B, page, free_pages, nfree, free_head, num_pages, table, table_ld, slots,
                      positions, T, rows, cu_new, free_next, stream):
    return load().rtopk_page_tables(cache_lens, new_lens, B, page, free_pages, nfree, free_head, num_pages, table,
                                    table_ld, slots, positions, T, rows, cu_new, free_next, stream)


def rtopk_cache_store(k, k_strides, v, v_strides, dtype, slots, T, Hkv, D, k_cache, v_cache, cache_strides, num_pages,
                      page, stream):
    """The stride arguments here and below are addresses of host int64 arrays (a ctypes array will do) or None."""
    return load().rtopk_cache_store(k, k_strides, v, v_strides, dtype, slots, T, Hkv, D, k_cache, v_cache,
                                    cache_strides, num_pages, page, stream)


def rtopk_tree_attention(q, q_strides, k_cache, v_cache, cache_strides, dtype, table, table_ld, num_pages, page,
                         cache_lens, parents, sizes, B, N, Hq, Hkv, D, scale, out, lse, workspace, ws_bytes, stream):
    return load().rtopk_tree_attention(q, q_strides, k_cache, v_cache, cache_strides, dtype, table, table_ld, num_pages,
                                       page, cache_lens, parents, sizes, B, N, Hq, Hkv, D, scale, out, lse, workspace,
                                       ws_bytes, stream)


def rtopk_tree_attention_workspace_bytes(B, N, Hq, Hkv, D, table_ld, page):
    return load().rtopk_tree_attention_workspace_bytes(B, N, Hq, Hkv, D, table_ld, page)


def rtopk_cross_attention(q, q_strides, k, k_strides, v, v_strides, dtype, lens, key_mask, B, N, S, Hq, Hkv, D, scale,
                          out, lse, workspace, ws_bytes, stream):
    return load().rtopk_cross_attention(q, q_strides, k, k_strides, v, v_strides, dtype, lens, key_mask, B, N, S, Hq,
                                        Hkv, D, scale, out, lse, workspace, ws_bytes, stream)


def rtopk_cross_attention_workspace_bytes(B, N, S, Hq, Hkv, D):
    return load().rtopk_cross_attention_workspace_bytes(B, N, S, Hq, Hkv, D)


def rtopk_qk_norm_rope(q, q_strides, k, k_strides, dtype, positions, freqs, rot, interleaved, q_weight, k_weight, eps, T,
                       Hq, Hkv, D, q_out, q_out_strides, k_out, k_out_strides, stream):
    return load().rtopk_qk_norm_rope(q, q_strides, k, k_strides, dtype, positions, freqs, rot, interleaved, q_weight,
                                     k_weight, eps, T, Hq, Hkv, D, q_out, q_out_strides, k_out, k_out_strides, stream)


def rtopk_cache_store_fp8(k, k_strides, v, v_strides, dtype, slots, T, Hkv, D, k_cache, v_cache, cache_strides, k_scales,
                          v_scales, num_pages, page, stream):
    return load().rtopk_cache_store_fp8(k, k_strides, v, v_strides, dtype, slots, T, Hkv, D, k_cache, v_cache,
                                        cache_strides, k_scales, v_scales, num_pages, page, stream)


def rtopk_cache_load_fp8(k_cache, v_cache, cache_strides, k_scales, v_scales, num_pages, page, slots, T, Hkv, D, k_out,
                         v_out, dtype, stream):
    return load().rtopk_cache_load_fp8(k_cache, v_cache, cache_strides, k_scales, v_scales, num_pages, page, slots, T, Hkv,
                                       D, k_out, v_out, dtype, stream)


def rtopk_tree_attention_fp8(q, q_strides, k_cache, v_cache, cache_strides, k_scales, v_scales, dtype, table, table_ld,
                             num_pages, page, cache_lens, parents, sizes, B, N, Hq, Hkv, D, scale, out, lse, workspace,
                             ws_bytes, stream):
    return load().rtopk_tree_attention_fp8(q, q_strides, k_cache, v_cache, cache_strides, k_scales, v_scales, dtype, table,
                                           table_ld, num_pages, page, cache_lens, parents, sizes, B, N, Hq, Hkv, D, scale,
                                           out, lse, workspace, ws_bytes, stream)


def rtopk_tree_attention_fp8_workspace_bytes(B, N, Hq, Hkv, D, table_ld, page):
    return load().rtopk_tree_attention_fp8_workspace_bytes(B, N, Hq, Hkv, D, table_ld, page)


def rtopk_sample_filtered(logits, dtype, R, V, ld, temperature, top_k, top_p, min_p, u, out_token, out_logprob, workspace,
                          ws_bytes, stream):
    return load().rtopk_sample_filtered(logits, dtype, R, V, ld, temperature, top_k, top_p, min_p, u, out_token,
                                        out_logprob, workspace, ws_bytes, stream)


def rtopk_sample_filtered_workspace_bytes(R, V):
    return load().rtopk_sample_filtered_workspace_bytes(R, V)


def rtopk_read_probe(src, nbytes, marker, out, stream):
    return load().rtopk_read_probe(src, nbytes, marker, out, stream)


def rtopk_read_probe_shape(src, nbytes, vecs_per_lane, threads, marker, out, stream):
    return load().rtopk_read_probe_shape(src, nbytes, vecs_per_lane, threads, marker, out, stream)


def rtopk_last_error():
    return load().rtopk_last_error().decode()


def rtopk_release():
    load().rtopk_release()


# ------------------------------------------------------------------ torch marshalling
def _check(status):
    if status != RTOPK_OK:
        raise RtopkError(status, rtopk_last_error())


def dtype_code(t):
    import torch
    codes = {torch.float32: RTOPK_F32, torch.float16: RTOPK_F16, torch.bfloat16: RTOPK_BF16}
    if t.dtype not in codes:
        raise TypeError(f"logits dtype {t.dtype} is not float32/float16/bfloat16")
    return codes[t.dtype]


def _ptr(t):
    return None if t is None else t.data_ptr()


def _on_device(t, dev, name):
    """Every tensor handed to the library must live on the logits' GPU: a host
    pointer in a kernel argument is a GPU memory fault, not an error code."""
    if not t.is_cuda or t.device != dev:
        raise ValueError(f"{name} must be a device tensor on {dev} (got {t.device})")


def _prepare(logits, alive, finished, k):
    import torch
    if logits.dim() != 3:
        raise ValueError("logits must be [B, beam, V]")
    if not logits.is_cuda:
        raise ValueError("logits must be a device tensor")
    B, beam, V = logits.shape
    if not logits.is_contiguous():
        raise ValueError("logits must be contiguous")
    dev = logits.device
    _on_device(alive, dev, "alive")
    if alive.shape != (B, beam) or alive.dtype != torch.float32 or not alive.is_contiguous():
        raise ValueError("alive must be a contiguous float32 [B, beam] tensor")
    if finished is not None:
        _on_device(finished, dev, "finished")
        if finished.shape != (B, beam) or finished.dtype not in (torch.uint8, torch.bool):
            raise ValueError("finished must be a [B, beam] uint8/bool tensor")
        finished = finished.contiguous()
        if finished.dtype == torch.bool:
            finished = finished.view(torch.uint8)
    outs = (torch.empty((B, k), dtype=torch.int32, device=dev),
            torch.empty((B, k), dtype=torch.int32, device=dev),
            torch.empty((B, k), dtype=torch.float32, device=dev))
    return B, beam, V, finished, outs


def _check_out(out, dev, B, k):
    """Caller-supplied outputs: (beam_ids int32, token_ids int32, scores float32), each [B, k]."""
    import torch
    if len(out) != 3:
        raise ValueError("out must hold three tensors (beam_ids, token_ids, scores)")
    for t, dt, name in zip(out, (torch.int32, torch.int32, torch.float32), ("beam_ids", "token_ids", "scores")):
        _on_device(t, dev, f"out {name}")
        if t.shape != (B, k) or t.dtype != dt or not t.is_contiguous():
            raise ValueError(f"out {name} must be a contiguous {dt} [{B}, {k}] tensor")
    return tuple(out)


def _check_workspace(ws, dev, need):
    import torch
    _on_device(ws, dev, "workspace")
    if ws.dtype != torch.uint8 or ws.dim() != 1 or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous 1-D uint8 tensor")
    if ws.numel() < need:
        raise ValueError(f"workspace holds {ws.numel()} bytes, {need} needed")


def beam_step(logits, alive, finished=None, k=None, eos_id=2, workspace=None, out=None):
    """One selection step on torch device tensors, on the current stream.

    logits [B, beam, V] float32/float16/bfloat16, alive [B, beam] float32,
    finished [B, beam] bool/uint8 or None. Returns (beam_ids, token_ids,
    scores), each [B, k]. ``workspace`` (a zero-filled uint8 device tensor of
    rtopk_workspace_bytes(...) bytes) selects rtopk_beam_step_ws; ``out`` may
    supply the three output tensors.
    """
    import torch
    if k is None:
        k = logits.shape[1]
    B, beam, V, finished, outs = _prepare(logits, alive, finished, k)
    if out is not None:
        outs = _check_out(out, logits.device, B, k)
    stream = torch.cuda.current_stream(logits.device).cuda_stream
    args = (_ptr(logits), dtype_code(logits), _ptr(alive), _ptr(finished), B, beam, V, k, eos_id,
            _ptr(outs[0]), _ptr(outs[1]), _ptr(outs[2]))
    if workspace is not None:
        _check_workspace(workspace, logits.device, rtopk_workspace_bytes(B, beam, V, k, dtype_code(logits)))
    if workspace is None:
        _check(rtopk_beam_step(*args, stream))
    else:
        _check(rtopk_beam_step_ws(*args, _ptr(workspace), workspace.numel() * workspace.element_size(), stream))
    return outs


def beam_reorder(src, dst, beam_ids):
    """Cache refresh on torch device tensors, on the current stream.

    src, dst: contiguous [nslabs, B*beam, ...] tensors of one dtype (e.g. the
    keys and values of every layer stacked along dim 0); beam_ids: [B, ld]
    int32 with ld >= beam (rtopk_beam_step's beam ids with k = beam). New beam
    j of batch element b takes the row of old beam beam_ids[b, j]; an id
    outside [0, beam) leaves that row of dst as it was. Returns dst.
    """
    import torch
    if src.shape != dst.shape or src.dtype != dst.dtype or src.device != dst.device:
        raise ValueError("src and dst must have the same shape, dtype and device")
    if not src.is_cuda:
        raise ValueError("src and dst must be device tensors")
    _on_device(beam_ids, src.device, "beam_ids")
    if not (src.is_contiguous() and dst.is_contiguous() and beam_ids.is_contiguous()):
        raise ValueError("src, dst and beam_ids must be contiguous")
    if beam_ids.dtype != torch.int32 or beam_ids.dim() != 2 or src.dim() < 2:
        raise ValueError("beam_ids must be a [B, ld] int32 tensor and src at least 2-D")
    B, ld = beam_ids.shape
    if src.shape[1] % B != 0:
        raise ValueError("src.shape[1] must be B * beam")
    beam = src.shape[1] // B
    row_bytes = (src[0, 0].numel() if src.dim() > 2 else 1) * src.element_size()
    stream = torch.cuda.current_stream(src.device).cuda_stream
    _check(rtopk_beam_reorder(_ptr(src), _ptr(dst), src.shape[0], B, beam, row_bytes, _ptr(beam_ids), ld, stream))
    return dst


# ------------------------------------------------------------------ paged cache and attention
_stride_arrays = {}


def _host_strides(st):
    """A host int64 array of these strides for the C ABI (which reads it during the call)."""
    arr = _stride_arrays.get(st)
    if arr is None:
        if len(_stride_arrays) > 4096:
            _stride_arrays.clear()
        arr = _stride_arrays[st] = (ctypes.c_int64 * len(st))(*st)
    return arr


def _strides(t, name):
    """The strides of all but the last dimension, which has to be contiguous; None where all are."""
    if t.is_contiguous():
        return None
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return _host_strides(st[:-1])


_torch = None  # the module, once one of the functions below has run (an import per call costs a launch's time)


def _get_torch():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
        _DTYPES.update({torch.float32: RTOPK_F32, torch.float16: RTOPK_F16, torch.bfloat16: RTOPK_BF16})
    return _torch


_DTYPES = {}


def _ints(t, shape, dev, name):
    """The address of a contiguous int32 tensor of this shape on device number `dev`."""
    if t.dtype is not _torch.int32 or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        _on_device(t, _torch.device("cuda", dev), name)
        raise ValueError(f"{name} must be a contiguous int32 {list(shape)} tensor")
    return t.data_ptr()


def _enqueue(dev, fn, *args):
    """fn(*args, stream) on the current stream of device number `dev`, with it the current device."""
    cuda = _torch._C
    if dev != cuda._cuda_getDevice():
        with _torch.cuda.device(dev):
            st = fn(*args, cuda._cuda_getCurrentRawStream(dev))
    else:
        st = fn(*args, cuda._cuda_getCurrentRawStream(dev))
    if st != RTOPK_OK:
        raise RtopkError(st, rtopk_last_error())


def _code(t):
    return _DTYPES[t.dtype] if t.dtype in _DTYPES else dtype_code(t)


def page_tables(cache_lens, new_lens, page, free_pages, table, num_pages, free_head=None, tokens=None, rows=None,
                out=None):
    """Page tables and slot maps from request lengths, on the current stream.

    cache_lens, new_lens [B] int32; free_pages [F] int32; table [B, ld] int32,
    updated in place; free_head [1] int32 or None. The slots are packed into
    [tokens], or laid out as [B, rows]; ``out`` may supply the four results.
    Returns (slots, positions, cu_new [B + 1], free_next [1]), all int32.
    """
    torch = _get_torch()
    if not table.is_cuda or table.dim() != 2:
        raise ValueError("table must be a [B, ld] device tensor")
    dev = table.get_device()
    B, ld = table.shape
    if out is not None:
        if len(out) != 4:
            raise ValueError("out must hold four tensors (slots, positions, cu_new, free_next)")
        slots, positions, cu, nxt = out
        shape = slots.shape
        if slots.dim() not in (1, 2) or (slots.dim() == 2 and shape[0] != B):
            raise ValueError("out slots must be a [tokens] or [B, rows] tensor")
        if tokens is not None and shape != (tokens,) or rows is not None and shape != (B, rows):
            raise ValueError("out slots must have the shape that tokens or rows asks for")
    else:
        if (tokens is None) == (rows is None):
            raise ValueError("give one of tokens (packed slots) and rows (slots per request)")
        shape = torch.Size((tokens,) if rows is None else (B, rows))
        slots = torch.empty(shape, dtype=torch.int32, device=table.device)
        positions = torch.empty_like(slots)
        cu = torch.empty(B + 1, dtype=torch.int32, device=table.device)
        nxt = torch.empty(1, dtype=torch.int32, device=table.device)
    n = slots.numel()
    if n == 0 or len(shape) == 2 and shape[1] == 0:
        raise ValueError("at least one slot is needed")
    if free_pages.dim() != 1:
        raise ValueError("free_pages must be a [F] tensor")
    _enqueue(dev, load().rtopk_page_tables, _ints(cache_lens, (B,), dev, "cache_lens"),
             _ints(new_lens, (B,), dev, "new_lens"), B, page, _ints(free_pages, free_pages.shape, dev, "free_pages"),
             free_pages.numel(), None if free_head is None else _ints(free_head, (1,), dev, "free_head"), num_pages,
             _ints(table, (B, ld), dev, "table"), ld, _ints(slots, shape, dev, "slots"),
             _ints(positions, shape, dev, "positions"), n, shape[1] if len(shape) == 2 else 0,
             _ints(cu, (B + 1,), dev, "cu_new"), _ints(nxt, (1,), dev, "free_next"))
    return slots, positions, cu, nxt


def _cache(k_cache, v_cache, dtype, dev):
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or k_cache.stride() != v_cache.stride():
        raise ValueError("k_cache and v_cache must be [pages, page, Hkv, D] tensors of the same strides")
    if k_cache.dtype is not dtype or v_cache.dtype is not dtype:
        raise ValueError(f"k_cache and v_cache must be {dtype}")
    if k_cache.get_device() != dev or v_cache.get_device() != dev:
        _on_device(k_cache, _torch.device("cuda", dev), "k_cache")
        _on_device(v_cache, _torch.device("cuda", dev), "v_cache")
    return k_cache.shape


def cache_store(k, v, slots, k_cache, v_cache):
    """Stores tokens' keys and values into a paged cache, on the current stream.

    k, v [..., Hkv, D] (the leading dimensions, which must be evenly strided,
    are the tokens), slots int32 of the leading shape (a slot outside the cache
    skips its token), k_cache, v_cache [pages, page, Hkv, D]. Returns (k_cache, v_cache).
    """
    _get_torch()
    if not k.is_cuda:
        raise ValueError("k must be a device tensor")
    dev = k.get_device()
    if v.get_device() != dev:
        _on_device(v, k.device, "v")
    if k.dim() < 3 or k.shape != v.shape or k.dtype is not v.dtype:
        raise ValueError("k and v must be [..., Hkv, D] tensors of one shape and type")
    if slots.shape != k.shape[:-2]:
        raise ValueError("slots must have the leading shape of k")
    if k.dim() > 3:
        k, v = (t.view(-1, *t.shape[-2:]) for t in (k, v))  # raises where the tokens are not evenly strided
    pages, page, Hkv, D = _cache(k_cache, v_cache, k.dtype, dev)
    if k.shape[1:] != (Hkv, D):
        raise ValueError("k and v must have the cache's heads")
    _enqueue(dev, load().rtopk_cache_store, k.data_ptr(), _strides(k, "k"), v.data_ptr(), _strides(v, "v"), _code(k),
             _ints(slots, slots.shape, dev, "slots"), k.shape[0], Hkv, D, k_cache.data_ptr(), v_cache.data_ptr(),
             _strides(k_cache, "k_cache"), pages, page)
    return k_cache, v_cache


def _cache8(k_cache, v_cache, k_scales, v_scales, dev):
    """The checks of an 8-bit cache: codes [pages, page, Hkv, D] and scales [pages, page, Hkv]."""
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape or k_cache.stride() != v_cache.stride():
        raise ValueError("k_cache and v_cache must be [pages, page, Hkv, D] tensors of the same strides")
    dt = k_cache.dtype
    if (dt is not _torch.float8_e4m3fn and dt is not _torch.uint8) or v_cache.dtype is not dt:
        raise ValueError("k_cache and v_cache must be float8_e4m3fn or uint8")
    rows = shape[:3]
    for t, name in ((k_scales, "k_scales"), (v_scales, "v_scales")):
        if t.dtype is not _torch.uint8 or t.shape != rows or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous uint8 [pages, page, Hkv] tensor")
    if not k_cache.get_device() == v_cache.get_device() == k_scales.get_device() == v_scales.get_device() == dev:
        for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache"), (k_scales, "k_scales"), (v_scales, "v_scales")):
            _on_device(t, _torch.device("cuda", dev), name)
    return shape


def cache_store_fp8(k, v, slots, k_cache, v_cache, k_scales, v_scales):
    """cache_store into a cache in 8 bits, quantising on the way.

    k, v, slots as cache_store; k_cache, v_cache [pages, page, Hkv, D]
    float8_e4m3fn (or uint8), k_scales, v_scales [pages, page, Hkv] uint8: the byte s
    of a token's head stands for 2 ** (s - 127). Returns (k_cache, v_cache, k_scales, v_scales).
    """
    _get_torch()
    if not k.is_cuda:
        raise ValueError("k must be a device tensor")
    dev = k.get_device()
    if v.get_device() != dev:
        _on_device(v, k.device, "v")
    shape = k.shape
    if len(shape) < 3 or v.shape != shape or k.dtype is not v.dtype:
        raise ValueError("k and v must be [..., Hkv, D] tensors of one shape and type")
    pages, page, Hkv, D = _cache8(k_cache, v_cache, k_scales, v_scales, dev)
    if shape[-2] != Hkv or shape[-1] != D:
        raise ValueError("k and v must have the cache's heads")
    at = _ints(slots, shape[:-2], dev, "slots")
    if len(shape) > 3:
        k, v = (t.view(-1, Hkv, D) for t in (k, v))  # raises where the tokens are not evenly strided
    _enqueue(dev, load().rtopk_cache_store_fp8, k.data_ptr(), _strides(k, "k"), v.data_ptr(), _strides(v, "v"), _code(k),
             at, k.size(0), Hkv, D, k_cache.data_ptr(), v_cache.data_ptr(), _strides(k_cache, "k_cache"), k_scales.data_ptr(), v_scales.data_ptr(), pages, page)
    return k_cache, v_cache, k_scales, v_scales


def cache_load_fp8(k_cache, v_cache, k_scales, v_scales, slots, dtype=None, out=None):
    """Reads tokens back out of a cache in 8 bits, on the current stream.

    slots int32 of any shape (one outside the cache gives zeros; they may repeat).
    Returns (k, v), each slots.shape + [Hkv, D] of `dtype` (None: bfloat16) or ``out``, which
    may supply them.
    """
    torch = _get_torch()
    if not k_cache.is_cuda:
        raise ValueError("k_cache must be a device tensor")
    dev = k_cache.get_device()
    pages, page, Hkv, D = _cache8(k_cache, v_cache, k_scales, v_scales, dev)
    lead = slots.shape
    shape = lead + (Hkv, D)
    if out is None:
        dtype = dtype or torch.bfloat16
        k, v = (torch.empty(shape, dtype=dtype, device=k_cache.device) for _ in range(2))
    else:
        if len(out) != 2:
            raise ValueError("out must hold two tensors (k, v)")
        k, v = out
        if k.shape != shape or v.shape != shape or k.dtype is not v.dtype or (dtype is not None and dtype is not k.dtype) or \
                not (k.is_contiguous() and v.is_contiguous()):
            raise ValueError(f"out must be two contiguous {list(shape)} tensors of one type")
        if not k.get_device() == v.get_device() == dev:
            _on_device(k, k_cache.device, "out k")
            _on_device(v, k_cache.device, "out v")
    _enqueue(dev, load().rtopk_cache_load_fp8, k_cache.data_ptr(), v_cache.data_ptr(), _strides(k_cache, "k_cache"),
             k_scales.data_ptr(), v_scales.data_ptr(), pages, page, _ints(slots, lead, dev, "slots"), slots.numel(),
             Hkv, D, k.data_ptr(), v.data_ptr(), _code(k))
    return k, v


def _rows3(t, name):
    """t as [tokens, heads, D]; a view, so that writing to it writes to t."""
    if t.dim() < 3:
        raise ValueError(f"{name} must be a [..., H, D] tensor")
    return t if t.dim() == 3 else t.view(-1, *t.shape[-2:])  # raises where the tokens are not evenly strided


def qk_norm_rope(q, k, positions, freqs, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, q_out=None,
                 k_out=None):
    """Norms of queries and keys and their rotation by position, on the current stream.

    q [..., Hq, D], k [..., Hkv, D] of one type (the leading dimensions, which must
    be evenly strided, are the tokens), positions int32 of the leading shape (where negative, the
    token's rows of the outputs stay as they were), freqs [rot / 2] float32 (radians per
    position; rot <= D elements are rotated), q_weight, k_weight [D] (None: no norm). The outputs
    may be supplied, q and k themselves among them; else they are new. Returns (q_out, k_out).
    """
    torch = _get_torch()
    if not q.is_cuda:
        raise ValueError("q must be a device tensor")
    dev = q.get_device()
    qs, ks, dt = q.shape, k.shape, q.dtype
    lead = qs[:-2]
    if len(qs) < 3 or ks[:-2] != lead or ks[-1] != qs[-1] or k.dtype is not dt:
        raise ValueError("q and k must be [..., Hq, D] and [..., Hkv, D] tensors of one type")
    D = qs[-1]
    if freqs.dtype is not torch.float32 or freqs.dim() != 1 or not freqs.is_contiguous():
        raise ValueError("freqs must be a contiguous float32 [rot / 2] tensor")
    if q_out is None:
        # rows of skipped tokens have to hold something: zeros
        q_out = torch.zeros(qs, dtype=dt, device=q.device)
    elif q_out.dtype is not dt or q_out.shape != qs:
        raise ValueError("q_out must have the shape and type of its input")
    if k_out is None:
        k_out = torch.zeros(ks, dtype=dt, device=q.device)
    elif k_out.dtype is not dt or k_out.shape != ks:
        raise ValueError("k_out must have the shape and type of its input")
    weights = [None, None]
    for i, (t, name) in enumerate(((q_weight, "q_weight"), (k_weight, "k_weight"))):
        if t is not None:
            if t.dtype is not dt or t.dim() != 1 or t.numel() != D or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous [D] tensor of q's type")
            if t.get_device() != dev:
                _on_device(t, q.device, name)
            weights[i] = t.data_ptr()
    if not k.get_device() == freqs.get_device() == q_out.get_device() == k_out.get_device() == dev:
        for t, name in ((k, "k"), (freqs, "freqs"), (q_out, "q_out"), (k_out, "k_out")):
            _on_device(t, q.device, name)
    q3, k3, qo, ko = (q, k, q_out, k_out) if len(qs) == 3 else \
        (_rows3(q, "q"), _rows3(k, "k"), _rows3(q_out, "q_out"), _rows3(k_out, "k_out"))
    _enqueue(dev, load().rtopk_qk_norm_rope, q3.data_ptr(), _strides(q3, "q"), k3.data_ptr(), _strides(k3, "k"), _code(q),
             _ints(positions, lead, dev, "positions"), freqs.data_ptr(), 2 * freqs.numel(), int(interleaved), weights[0],
             weights[1], eps, q3.size(0), qs[-2], ks[-2], D, qo.data_ptr(), _strides(qo, "q_out"), ko.data_ptr(),
             _strides(ko, "k_out"))
    return q_out, k_out


def _row_values(t, R, dtype, dev, name):
    """The address of a contiguous [R] tensor of this type on device number `dev`; None for None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != (R,) or not t.is_contiguous() or t.get_device() != dev:
        _on_device(t, _torch.device("cuda", dev), name)
        raise ValueError(f"{name} must be a contiguous {dtype} [{R}] tensor")
    return t.data_ptr()


def sample_filtered(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, out=None, workspace=None):
    """Sampling of every row of logits [R, V] with filters, from given random numbers, on the current stream.

    logits float32/float16/bfloat16, rows any distance apart; u [R] float32 in
    [0, 1); temperature, top_p, min_p [R] float32 and top_k [R] int32, each None for none:
    a row's k best, of those the shortest beginning with top_p of their weight, of those the ones with
    min_p of the largest weight. ``out`` may supply the two results. ``workspace`` (uint8, of
    rtopk_sample_filtered_workspace_bytes(R, V) bytes) lets few long rows be cut over workgroups under
    graph capture too; calls that share one must be ordered. Returns
    (tokens [R] int32, logprobs [R] float32 under what is kept).
    """
    torch = _get_torch()
    if not logits.is_cuda or logits.dim() != 2:
        raise ValueError("logits must be a [R, V] device tensor")
    dev = logits.get_device()
    R, V = logits.shape
    st = logits.stride()
    if st[1] != 1 and V > 1:
        raise ValueError("logits: the last dimension must be contiguous")
    if out is None:
        tok = torch.empty(R, dtype=torch.int32, device=logits.device)
        lp = torch.empty(R, dtype=torch.float32, device=logits.device)
    else:
        if len(out) != 2:
            raise ValueError("out must hold two tensors (tokens, logprobs)")
        tok, lp = out
    f32 = torch.float32
    wp, wn = None, 0
    if workspace is not None:
        _check_workspace(workspace, logits.device, 0)
        wp, wn = workspace.data_ptr(), workspace.numel()
    _enqueue(dev, load().rtopk_sample_filtered, logits.data_ptr(), _code(logits), R, V, st[0],
             _row_values(temperature, R, f32, dev, "temperature"), _row_values(top_k, R, torch.int32, dev, "top_k"),
             _row_values(top_p, R, f32, dev, "top_p"), _row_values(min_p, R, f32, dev, "min_p"),
             _row_values(u, R, f32, dev, "u"), _row_values(tok, R, torch.int32, dev, "out tokens"),
             _row_values(lp, R, f32, dev, "out logprobs"), wp, wn)
    return tok, lp


def _attention_args(q, Hkv, scale, out, lse, workspace, dev):
    """Checks what both attentions share; returns the scale, out and the addresses of lse and the workspace."""
    B, N, Hq, D = shape = q.shape
    if scale is None:
        scale = D ** -0.5
    if out is None:
        out = _torch.empty(shape, dtype=q.dtype, device=q.device)
    elif out.shape != shape or out.dtype is not q.dtype or not out.is_contiguous() or out.get_device() != dev:
        _on_device(out, q.device, "out")
        raise ValueError("out must be a contiguous tensor of q's shape and type")
    lp = None
    if lse is not None:
        if lse.shape != shape[:3] or lse.dtype is not _torch.float32 or not lse.is_contiguous() or lse.get_device() != dev:
            _on_device(lse, q.device, "lse")
            raise ValueError("lse must be a contiguous float32 [B, N, Hq] tensor")
        lp = lse.data_ptr()
    wp, wn = None, 0
    if workspace is not None:
        _check_workspace(workspace, q.device, 0)
        wp, wn = workspace.data_ptr(), workspace.numel()
    return scale, out, lp, wp, wn


def tree_attention(q, k_cache, v_cache, table, cache_lens, parents=None, sizes=None, scale=None, out=None, lse=None,
                   workspace=None):
    """Attention of a tree of drafted tokens over a paged cache, on the current stream.

    q [B, N, Hq, D] float16/bfloat16; k_cache, v_cache [pages, page, Hkv, D];
    table [B, ld], cache_lens [B], parents [B, N] (None: a chain), sizes [B]
    (None: N), all int32; scale None = D ** -0.5. ``out`` [B, N, Hq, D] and
    ``lse`` [B, N, Hq] float32 may be supplied; rows behind a tree's last node
    keep what they hold. ``workspace`` (zero-filled uint8, of
    rtopk_tree_attention_workspace_bytes(...) bytes) is needed under graph
    capture. Returns (out, lse); lse None unless supplied.
    """
    _get_torch()
    if not q.is_cuda or q.dim() != 4 or table.dim() != 2:
        raise ValueError("q must be a [B, N, Hq, D] device tensor and table [B, ld]")
    dev = q.get_device()
    B, N, Hq, D = q.shape
    pages, page, Hkv, Dk = _cache(k_cache, v_cache, q.dtype, dev)
    if Dk != D:
        raise ValueError("the cache must have q's head size")
    ld = table.shape[1]
    scale, out, lp, wp, wn = _attention_args(q, Hkv, scale, out, lse, workspace, dev)
    _enqueue(dev, load().rtopk_tree_attention, q.data_ptr(), _strides(q, "q"), k_cache.data_ptr(), v_cache.data_ptr(),
             _strides(k_cache, "k_cache"), _code(q), _ints(table, (B, ld), dev, "table"), ld, pages, page,
             _ints(cache_lens, (B,), dev, "cache_lens"), None if parents is None else _ints(parents, (B, N), dev, "parents"),
             None if sizes is None else _ints(sizes, (B,), dev, "sizes"), B, N, Hq, Hkv, D, scale, out.data_ptr(), lp, wp, wn)
    return out, lse


def tree_attention_fp8(q, k_cache, v_cache, k_scales, v_scales, table, cache_lens, parents=None, sizes=None, scale=None,
                       out=None, lse=None, workspace=None):
    """tree_attention over a cache in 8 bits, as cache_store_fp8 fills it: k_cache, v_cache
    [pages, page, Hkv, D] float8_e4m3fn (or uint8), D a multiple of 16, and k_scales, v_scales
    [pages, page, Hkv] uint8; everything else as tree_attention (a workspace has
    rtopk_tree_attention_fp8_workspace_bytes(...) bytes). Returns (out, lse)."""
    _get_torch()
    shape, rows = q.shape, table.shape
    if not q.is_cuda or len(shape) != 4 or len(rows) != 2:
        raise ValueError("q must be a [B, N, Hq, D] device tensor and table [B, ld]")
    dev = q.get_device()
    B, N, Hq, D = shape
    pages, page, Hkv, Dk = _cache8(k_cache, v_cache, k_scales, v_scales, dev)
    if Dk != D:
        raise ValueError("the cache must have q's head size")
    ld = rows[1]
    scale, out, lp, wp, wn = _attention_args(q, Hkv, scale, out, lse, workspace, dev)
    _enqueue(dev, load().rtopk_tree_attention_fp8, q.data_ptr(), _strides(q, "q"), k_cache.data_ptr(), v_cache.data_ptr(),
             _strides(k_cache, "k_cache"), k_scales.data_ptr(), v_scales.data_ptr(), _code(q),
             _ints(table, (B, ld), dev, "table"), ld, pages, page, _ints(cache_lens, (B,), dev, "cache_lens"),
             None if parents is None else _ints(parents, (B, N), dev, "parents"),
             None if sizes is None else _ints(sizes, (B,), dev, "sizes"), B, N, Hq, Hkv, D, scale, out.data_ptr(), lp, wp, wn)
    return out, lse


def cross_attention(q, k, v, lens=None, key_mask=None, scale=None, out=None, lse=None, workspace=None):
    """Attention of every beam's rows to its encoder's states, on the current stream.

    q [B, N, Hq, D] (N = beams x tokens) and k, v [B, S, Hkv, D] float16/bfloat16,
    any strides with a contiguous last dimension; lens [B] int32 (None: S);
    key_mask [B, S] uint8/bool, nonzero = left out; the rest as
    tree_attention. Returns (out, lse).
    """
    torch = _get_torch()
    if not q.is_cuda or q.dim() != 4 or k.dim() != 4 or k.shape != v.shape:
        raise ValueError("q must be a [B, N, Hq, D] device tensor and k, v [B, S, Hkv, D]")
    dev = q.get_device()
    if k.dtype is not q.dtype or v.dtype is not q.dtype:
        raise ValueError("q, k and v must have one type")
    if k.get_device() != dev or v.get_device() != dev:
        _on_device(k, q.device, "k")
        _on_device(v, q.device, "v")
    B, N, Hq, D = q.shape
    _, S, Hkv, _ = k.shape
    if k.shape[0] != B or k.shape[3] != D:
        raise ValueError("k and v must have q's batch and head size")
    mp = None
    if key_mask is not None:
        _on_device(key_mask, q.device, "key_mask")
        if key_mask.shape != (B, S) or key_mask.dtype not in (torch.uint8, torch.bool) or not key_mask.is_contiguous():
            raise ValueError("key_mask must be a contiguous [B, S] uint8/bool tensor")
        mp = key_mask.data_ptr()
    scale, out, lp, wp, wn = _attention_args(q, Hkv, scale, out, lse, workspace, dev)
    _enqueue(dev, load().rtopk_cross_attention, q.data_ptr(), _strides(q, "q"), k.data_ptr(), _strides(k, "k"),
             v.data_ptr(), _strides(v, "v"), _code(q), None if lens is None else _ints(lens, (B,), dev, "lens"), mp,
             B, N, S, Hq, Hkv, D, scale, out.data_ptr(), lp, wp, wn)
    return out, lse


def debug_step(logits, alive, finished=None, k=None, eos_id=2):
    """beam_step plus the kernel's intermediate values (for tests).

    Returns a dict with the outputs and the plan, the per-piece thresholds
    T [B*beam*chunks], hit counts, merged lse [B*beam], per-batch queue
    counts and the raw queue [B, queue_cap] (uint64 entries).
    """
    import torch
    if k is None:
        k = logits.shape[1]
    B, beam, V, finished, outs = _prepare(logits, alive, finished, k)
    code = dtype_code(logits)
    st, plan = rtopk_plan(_ptr(logits), B, beam, V, k, code)
    _check(st)
    dev = logits.device
    nbytes = rtopk_workspace_bytes(B, beam, V, k, code)
    ws = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
    npieces = B * beam * plan.chunks
    dT = torch.full((npieces,), float("nan"), dtype=torch.float32, device=dev)
    dh = torch.zeros(npieces, dtype=torch.int32, device=dev)
    dl = torch.zeros(B * beam, dtype=torch.float32, device=dev)
    dc = torch.zeros(B, dtype=torch.int32, device=dev)
    dq = torch.zeros((B, plan.queue_cap), dtype=torch.int64, device=dev)
    stream = torch.cuda.current_stream(dev).cuda_stream
    _check(rtopk_debug_step(_ptr(logits), code, _ptr(alive), _ptr(finished), B, beam, V, k, eos_id,
                            _ptr(outs[0]), _ptr(outs[1]), _ptr(outs[2]), _ptr(ws), nbytes,
                            _ptr(dT), _ptr(dh), _ptr(dl), _ptr(dc), _ptr(dq), stream))
    return dict(beam_ids=outs[0], token_ids=outs[1], scores=outs[2], plan=plan.as_dict(), T=dT, hits=dh,
                lse=dl, count=dc, queue=dq, workspace=ws)
