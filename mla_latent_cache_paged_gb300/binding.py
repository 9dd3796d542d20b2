"""Thin ctypes binding of libmla_decode (include/mla_decode.h).

Only argument marshalling lives here: torch tensors become device pointers,
the current torch stream becomes the ``stream`` argument, and non-zero
status codes become ``MlaError``. Every arithmetic step runs in the CUDA
library; if the library is missing the calls raise instead of falling back.
"""

from __future__ import annotations

import ctypes
import os

from .build import LIB_PATH

MLA_OK = 0
MLA_ERR_INVALID_ARG = -1
MLA_ERR_UNSUPPORTED = -2
MLA_ERR_WORKSPACE = -3
MLA_ERR_CUDA = -4
MLA_ERR_BAD_BLOCK_ID = -5
MLA_ERR_BAD_SEQ_LEN = -6
MLA_ERR_TIMEOUT = -7
MLA_ERR_SCRATCH_LIMIT = -8
MLA_ERR_RANGE = -9
MLA_ERR_NO_PAGES = -10
MLA_ERR_PAGE_STATE = -11
MLA_ERR_BAD_ROW = -12

MLA_KERNEL_SIMT = 1
MLA_KERNEL_TC = 2
MLA_PLAN_FORCE_SIMT = 0x1
MLA_PLAN_SPLIT_ONLY = 0x2
MLA_PLAN_FORCE_BALANCED = 0x4
MLA_PLAN_FP32_PARTIALS = 0x8
MLA_PLAN_DEBUG_WITHHOLD_LOAD = 0x100

KV_LORA_RANK = 512
ROPE_DIM = 64
HEAD_DIM = KV_LORA_RANK + ROPE_DIM
PAGE_SIZE = 64
STATUS_BYTES = 8192

EXPORTED_SYMBOLS = (
    "mla_decode_plan", "mla_workspace_init", "mla_decode", "mla_merge_splits",
    "mla_read_error", "mla_status_string", "mla_abi_version", "mla_debug_gather_pages",
    "mla_decode_noalloc", "mla_dcp_local_seq_lens", "mla_dcp_combine",
    "mla_q_absorb_concat_cache", "mla_v_up_proj", "mla_multi_token_scratch_bytes",
    "mla_decode_multi_token", "mla_debug_loader_pages", "mla_multi_token_row_lens",
    "mla_decode_fp8", "mla_merge_splits_v_up_proj", "mla_decode_v_up_proj",
    "mla_expand_kv", "mla_expand_kv_fp8", "mla_cache_workspace_bytes", "mla_cache_fork",
    "mla_cache_free", "mla_cache_compact", "mla_prefill_plan", "mla_prefill",
    "mla_cache_write", "mla_cache_write_fp8", "mla_cache_gather", "mla_cache_gather_fp8",
    "mla_span_plan", "mla_decode_shared", "mla_decode_shared_fp8", "mla_decode_window",
    "mla_decode_window_fp8",
)


class MlaError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


class MlaDecodePlan(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("num_heads", ctypes.c_int32),
        ("kv_lora_rank", ctypes.c_int32),
        ("rope_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32),
        ("max_seq_len", ctypes.c_int32),
        ("num_kv_splits", ctypes.c_int32),
        ("kernel", ctypes.c_int32),
        ("num_sms", ctypes.c_int32),
        ("grid_ctas", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
        ("workspace_bytes", ctypes.c_uint64),
        ("partial_offset", ctypes.c_uint64),
        ("lse_partial_offset", ctypes.c_uint64),
        ("sched_pairs", ctypes.c_int32),
        ("reserved", ctypes.c_uint32 * 7),
    ]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_ if name != "reserved"}


class MlaPrefillPlan(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("num_heads", ctypes.c_int32),
        ("total_q", ctypes.c_int32),
        ("num_kv_splits", ctypes.c_int32),
        ("num_sms", ctypes.c_int32),
        ("single_rows", ctypes.c_int32),
        ("workspace_bytes", ctypes.c_uint64),
        ("partial_offset", ctypes.c_uint64),
        ("lse_partial_offset", ctypes.c_uint64),
        ("split_rest", ctypes.c_int32),
        ("reserved", ctypes.c_uint32 * 5),
    ]


class MlaSpanPlan(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("num_heads", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32),
        ("max_groups", ctypes.c_int32),
        ("num_sms", ctypes.c_int32),
        ("pairs", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
        ("reserved0", ctypes.c_uint32),
        ("workspace_bytes", ctypes.c_uint64),
        ("reserved", ctypes.c_uint32 * 6),
    ]


_LIB = None


def load_library(path=None):
    """Load libmla_decode.so (raises if it has not been built)."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it first (mla_latent_cache_paged_gb300.build)")
    lib = ctypes.CDLL(path)
    vp, i32, i64, sz, f32 = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t,
                             ctypes.c_float)
    lib.mla_decode_plan.argtypes = [i32, i32, i32, i32, i32, i32, i32, vp, i32, i32,
                                    ctypes.c_uint32, ctypes.POINTER(MlaDecodePlan)]
    lib.mla_workspace_init.argtypes = [vp, sz, vp]
    lib.mla_decode.argtypes = [ctypes.POINTER(MlaDecodePlan), vp, vp, i64, vp, vp, f32, vp, vp,
                               vp, sz, vp]
    lib.mla_decode_fp8.argtypes = [ctypes.POINTER(MlaDecodePlan), vp, vp, i64, vp, vp, f32, f32,
                                   vp, vp, vp, sz, vp]
    lib.mla_merge_splits.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp]
    lib.mla_merge_splits_v_up_proj.argtypes = [vp, vp, i32, i32, i32, vp, vp, vp, vp, vp, sz,
                                               vp]
    lib.mla_decode_v_up_proj.argtypes = [ctypes.POINTER(MlaDecodePlan), vp, vp, i64, vp, vp, f32,
                                         vp, vp, vp, vp, vp, sz, vp]
    lib.mla_read_error.argtypes = [vp, ctypes.POINTER(ctypes.c_int), vp]
    lib.mla_status_string.argtypes = [i32]
    lib.mla_status_string.restype = ctypes.c_char_p
    lib.mla_abi_version.argtypes = []
    lib.mla_debug_gather_pages.argtypes = [vp, i64, vp, vp, i32, i32, i32, vp, vp, sz, vp]
    lib.mla_decode_noalloc.argtypes = [ctypes.POINTER(MlaDecodePlan), vp, vp, i64, vp, vp, f32, vp,
                                       vp, vp, vp]
    lib.mla_dcp_local_seq_lens.argtypes = [vp, i32, i32, i32, i32, vp]
    lib.mla_dcp_combine.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp]
    lib.mla_q_absorb_concat_cache.argtypes = [vp, vp, vp, vp, vp, vp, i64, i32, i32, vp, vp, sz,
                                              vp]
    lib.mla_v_up_proj.argtypes = [vp, vp, i32, i32, vp, vp, sz, vp]
    lib.mla_debug_loader_pages.argtypes = [ctypes.POINTER(MlaDecodePlan), vp, i64, vp, vp, i32,
                                           vp, vp, sz, vp]
    lib.mla_multi_token_scratch_bytes.argtypes = [i32, i32, i32]
    lib.mla_multi_token_row_lens.argtypes = [vp, i32, i32, i32, vp]
    lib.mla_decode_multi_token.argtypes = [ctypes.POINTER(MlaDecodePlan), i32, i32, i32, vp, vp,
                                           i64, vp, vp, f32, vp, vp, vp, sz, vp, sz, vp]
    lib.mla_expand_kv.argtypes = [vp, i64, vp, i32, vp, vp, i32, i32, i32, vp, vp, vp, vp, vp, sz,
                                  vp]
    lib.mla_expand_kv_fp8.argtypes = [vp, f32, i64, vp, i32, vp, vp, i32, i32, i32, vp, vp, vp, vp,
                                      vp, sz, vp]
    lib.mla_cache_workspace_bytes.argtypes = [i64, i32]
    lib.mla_cache_fork.argtypes = [vp, i32, i64, i64, i32, vp, vp, vp, i32, i32, vp, vp, vp, i32,
                                   vp, vp, sz, vp]
    lib.mla_cache_free.argtypes = [vp, vp, i64, vp, i32, i32, vp, vp, i32, vp, vp, sz, vp]
    lib.mla_cache_compact.argtypes = [vp, i32, i64, i64, i32, vp, vp, vp, vp, i32, i32, vp, vp, vp,
                                      vp, sz, vp]
    lib.mla_prefill_plan.argtypes = [i32, i32, i32, i32, i32, i32, i32,
                                     ctypes.POINTER(MlaPrefillPlan)]
    lib.mla_prefill.argtypes = [ctypes.POINTER(MlaPrefillPlan), vp, vp, vp, i32, vp, vp, i32, f32,
                                vp, vp, vp, sz, vp]
    lib.mla_cache_write.argtypes = [vp, i64, vp, i64, vp, i32, vp, i64, vp, sz, vp]
    lib.mla_cache_write_fp8.argtypes = [vp, i64, vp, i64, vp, i32, f32, vp, i64, vp, sz, vp]
    lib.mla_cache_gather.argtypes = [vp, i64, vp, i32, vp, vp, i32, i32, vp, vp, sz, vp]
    lib.mla_cache_gather_fp8.argtypes = [vp, f32, i64, vp, i32, vp, vp, i32, i32, vp, vp, sz, vp]
    lib.mla_span_plan.argtypes = [i32, i32, i32, i32, i32, ctypes.c_uint32,
                                  ctypes.POINTER(MlaSpanPlan)]
    span = [ctypes.POINTER(MlaSpanPlan), vp, vp, i64, vp, vp]
    lib.mla_decode_shared.argtypes = span + [vp, vp, i32, f32, vp, vp, vp, sz, vp]
    lib.mla_decode_shared_fp8.argtypes = span + [vp, vp, i32, f32, f32, vp, vp, vp, sz, vp]
    lib.mla_decode_window.argtypes = span + [i32, i32, f32, vp, vp, vp, sz, vp]
    lib.mla_decode_window_fp8.argtypes = span + [i32, i32, f32, f32, vp, vp, vp, sz, vp]
    for name in EXPORTED_SYMBOLS:
        if name != "mla_status_string":
            getattr(lib, name).restype = ctypes.c_int
    lib.mla_multi_token_scratch_bytes.restype = ctypes.c_size_t
    lib.mla_cache_workspace_bytes.restype = ctypes.c_size_t
    if path == LIB_PATH:
        _LIB = lib
    return lib


def status_string(status):
    try:
        return load_library().mla_status_string(int(status)).decode()
    except RuntimeError:
        return "library not loaded"


def _check(status, what):
    if status != MLA_OK:
        raise MlaError(status, what)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream_ptr(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def make_plan(batch, num_heads, max_blocks_per_seq, max_seq_len=None, *, seq_lens_host=None,
              num_kv_splits=0, num_sms=None, force_simt=False, schedule="auto", extra_flags=0):
    """Call mla_decode_plan (host only; no device work).

    ``schedule``: "auto" (the planner's estimate), "split" (never the
    page-balanced schedule) or "balanced" (the page-balanced schedule wherever
    it applies; needs num_kv_splits = 0). ``extra_flags``: further MLA_PLAN_*
    bits (tests use MLA_PLAN_DEBUG_WITHHOLD_LOAD).
    """
    if schedule not in ("auto", "split", "balanced"):
        raise ValueError(f"schedule must be auto, split or balanced, not {schedule!r}")
    lib = load_library()
    if max_seq_len is None:
        max_seq_len = max_blocks_per_seq * PAGE_SIZE
    if num_sms is None:
        import torch
        num_sms = (torch.cuda.get_device_properties(0).multi_processor_count
                   if torch.cuda.is_available() else 152)
    lens_ptr = ctypes.c_void_p(0)
    keep = None
    if seq_lens_host is not None:
        import numpy as np
        keep = np.ascontiguousarray(np.asarray(seq_lens_host, dtype=np.int32))
        lens_ptr = ctypes.c_void_p(keep.ctypes.data)
    plan = MlaDecodePlan()
    rc = lib.mla_decode_plan(int(batch), int(num_heads), KV_LORA_RANK, ROPE_DIM, PAGE_SIZE,
                             int(max_blocks_per_seq), int(max_seq_len), lens_ptr,
                             int(num_kv_splits), int(num_sms),
                             (MLA_PLAN_FORCE_SIMT if force_simt else 0) |
                             (MLA_PLAN_SPLIT_ONLY if schedule == "split" else 0) |
                             (MLA_PLAN_FORCE_BALANCED if schedule == "balanced" else 0) |
                             int(extra_flags),
                             ctypes.byref(plan))
    del keep
    _check(rc, "mla_decode_plan")
    return plan


def new_workspace(plan, device=None, stream=None):
    """Allocate (through torch) and initialise a workspace for `plan`."""
    import torch
    nbytes = max(int(plan.workspace_bytes), STATUS_BYTES)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")
    _check(load_library().mla_workspace_init(_ptr(ws), nbytes, _stream_ptr(stream)),
           "mla_workspace_init")
    return ws


def _check_tensor(t, name, dtype, shape=None):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def mla_decode(q, latent_cache, block_table, seq_lens, softmax_scale, *, plan=None,
               num_kv_splits=0, out=None, lse=None, return_lse=True, workspace=None,
               stream=None, force_simt=False):
    """Absorbed MLA decode. Returns ``(out bf16 [B,N,512], lse fp32 [B,N] | None)``.

    Mirrors the argument list of ModelOpt's ``mla_attention_decode``; the work
    is one ``mla_decode`` call of the C library on the current stream.
    """
    import torch
    B, N, D = q.shape
    if D != HEAD_DIM:
        raise ValueError(f"q last dim must be {HEAD_DIM}")
    _check_tensor(q, "q", torch.bfloat16)
    _check_tensor(latent_cache, "latent_cache", torch.bfloat16)
    if latent_cache.dim() != 3 or latent_cache.shape[1:] != (PAGE_SIZE, HEAD_DIM):
        raise ValueError("latent_cache must be [num_blocks, 64, 576]")
    _check_tensor(block_table, "block_table", torch.int32)
    _check_tensor(seq_lens, "seq_lens", torch.int32, (B,))
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_blocks_per_seq]")
    if plan is None:
        plan = make_plan(B, N, block_table.shape[1], num_kv_splits=num_kv_splits,
                         force_simt=force_simt)
    if out is None:
        out = torch.empty((B, N, KV_LORA_RANK), dtype=torch.bfloat16, device=q.device)
    _check_tensor(out, "out", torch.bfloat16, (B, N, KV_LORA_RANK))
    if lse is None and return_lse:
        lse = torch.empty((B, N), dtype=torch.float32, device=q.device)
    if lse is not None:
        _check_tensor(lse, "lse", torch.float32, (B, N))
    if workspace is None:
        workspace = new_workspace(plan, q.device, stream)
    rc = load_library().mla_decode(
        ctypes.byref(plan), _ptr(q), _ptr(latent_cache), int(latent_cache.shape[0]),
        _ptr(block_table), _ptr(seq_lens), float(softmax_scale), _ptr(out), _ptr(lse),
        _ptr(workspace), int(workspace.numel()), _stream_ptr(stream))
    _check(rc, "mla_decode")
    return out, lse


def mla_decode_fp8(q, latent_cache_fp8, block_table, seq_lens, softmax_scale, k_scale, *,
                   plan=None, num_kv_splits=0, out=None, lse=None, return_lse=True,
                   workspace=None, stream=None):
    """Absorbed MLA decode over an fp8 cache (uint8 E4M3 codes ``[num_blocks,
    64, 576]`` with a per-tensor ``k_scale``). Returns ``(out bf16 [B,N,512],
    lse fp32 [B,N] | None)``; one ``mla_decode_fp8`` call."""
    import torch
    B, N, D = q.shape
    if D != HEAD_DIM:
        raise ValueError(f"q last dim must be {HEAD_DIM}")
    _check_tensor(q, "q", torch.bfloat16)
    _check_tensor(latent_cache_fp8, "latent_cache_fp8", torch.uint8)
    if latent_cache_fp8.dim() != 3 or latent_cache_fp8.shape[1:] != (PAGE_SIZE, HEAD_DIM):
        raise ValueError("latent_cache_fp8 must be [num_blocks, 64, 576]")
    _check_tensor(block_table, "block_table", torch.int32)
    _check_tensor(seq_lens, "seq_lens", torch.int32, (B,))
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_blocks_per_seq]")
    if plan is None:
        plan = make_plan(B, N, block_table.shape[1], num_kv_splits=num_kv_splits)
    if out is None:
        out = torch.empty((B, N, KV_LORA_RANK), dtype=torch.bfloat16, device=q.device)
    _check_tensor(out, "out", torch.bfloat16, (B, N, KV_LORA_RANK))
    if lse is None and return_lse:
        lse = torch.empty((B, N), dtype=torch.float32, device=q.device)
    if lse is not None:
        _check_tensor(lse, "lse", torch.float32, (B, N))
    if workspace is None:
        workspace = new_workspace(plan, q.device, stream)
    rc = load_library().mla_decode_fp8(
        ctypes.byref(plan), _ptr(q), _ptr(latent_cache_fp8), int(latent_cache_fp8.shape[0]),
        _ptr(block_table), _ptr(seq_lens), float(softmax_scale), float(k_scale), _ptr(out),
        _ptr(lse), _ptr(workspace), int(workspace.numel()), _stream_ptr(stream))
    _check(rc, "mla_decode_fp8")
    return out, lse


def multi_token_row_lens(seq_lens_host, q_len, causal=True):
    """Tokens each (request, query token) row sees, row r = b * T + i, from
    ``mla_multi_token_row_lens`` (host C; numpy int32 ``[B * T]``)."""
    import numpy as np
    lens = np.ascontiguousarray(np.asarray(seq_lens_host, dtype=np.int32).reshape(-1))
    rows = np.empty(lens.size * int(q_len), dtype=np.int32)
    rc = load_library().mla_multi_token_row_lens(
        ctypes.c_void_p(lens.ctypes.data), int(lens.size), int(q_len), 1 if causal else 0,
        ctypes.c_void_p(rows.ctypes.data))
    _check(rc, "mla_multi_token_row_lens")
    return rows


def make_plan_multi_token(batch, q_len, num_heads, max_blocks_per_seq, *, seq_lens_host=None,
                          causal=True, expand=None, **kw):
    """A plan for a uniform multi-token decode: the T query tokens' heads as
    the rows of one decode when T * N <= 128 (each page read once), else
    B * T rows of N heads. ``expand=True`` forces the second form."""
    if expand is None:
        expand = int(q_len) * int(num_heads) > 128
    if not expand:
        if seq_lens_host is not None:
            kw["seq_lens_host"] = seq_lens_host
        return make_plan(batch, int(q_len) * int(num_heads), max_blocks_per_seq, **kw)
    if seq_lens_host is not None:
        rows = multi_token_row_lens(seq_lens_host, q_len, causal)
        kw.setdefault("max_seq_len", int(rows.max()) if rows.size else 0)
        kw["seq_lens_host"] = rows
    return make_plan(int(batch) * int(q_len), num_heads, max_blocks_per_seq, **kw)


def mla_decode_multi_token(q, latent_cache, block_table, seq_lens, softmax_scale, *,
                           causal=True, plan=None, num_kv_splits=0, out=None, lse=None,
                           return_lse=True, workspace=None, scratch=None, stream=None):
    """Uniform multi-token decode: ``q [B, T, N, 576]`` -> ``(out [B, T, N, 512],
    lse [B, T, N] | None)``; one ``mla_decode_multi_token`` call."""
    import torch
    B, T, N, D = q.shape
    if D != HEAD_DIM:
        raise ValueError(f"q last dim must be {HEAD_DIM}")
    _check_tensor(q, "q", torch.bfloat16)
    _check_tensor(latent_cache, "latent_cache", torch.bfloat16)
    _check_tensor(block_table, "block_table", torch.int32)
    _check_tensor(seq_lens, "seq_lens", torch.int32, (B,))
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_blocks_per_seq]")
    if plan is None:
        plan = make_plan_multi_token(B, T, N, block_table.shape[1], causal=causal,
                                     num_kv_splits=num_kv_splits)
    if out is None:
        out = torch.empty((B, T, N, KV_LORA_RANK), dtype=torch.bfloat16, device=q.device)
    _check_tensor(out, "out", torch.bfloat16, (B, T, N, KV_LORA_RANK))
    if lse is None and return_lse:
        lse = torch.empty((B, T, N), dtype=torch.float32, device=q.device)
    if lse is not None:
        _check_tensor(lse, "lse", torch.float32, (B, T, N))
    if workspace is None:
        workspace = new_workspace(plan, q.device, stream)
    lib = load_library()
    if scratch is None and plan.num_heads != T * N:
        nbytes = int(lib.mla_multi_token_scratch_bytes(B, T, block_table.shape[1]))
        scratch = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=q.device)
    rc = lib.mla_decode_multi_token(
        ctypes.byref(plan), int(T), int(N), 1 if causal else 0, _ptr(q), _ptr(latent_cache),
        int(latent_cache.shape[0]), _ptr(block_table), _ptr(seq_lens), float(softmax_scale),
        _ptr(out), _ptr(lse), _ptr(workspace), int(workspace.numel()), _ptr(scratch),
        int(scratch.numel()) if scratch is not None else 0, _stream_ptr(stream))
    _check(rc, "mla_decode_multi_token")
    return out, lse


def mla_merge_splits(o_part, lse_part, *, out=None, lse=None, return_lse=True, stream=None):
    """LSE merge of fp32 partials ``[B,N,S,V]`` / ``[B,N,S]`` -> bf16 ``[B,N,V]``, fp32 ``[B,N]``."""
    import torch
    B, N, S, V = o_part.shape
    _check_tensor(o_part, "o_part", torch.float32)
    _check_tensor(lse_part, "lse_part", torch.float32, (B, N, S))
    if out is None:
        out = torch.empty((B, N, V), dtype=torch.bfloat16, device=o_part.device)
    _check_tensor(out, "out", torch.bfloat16, (B, N, V))
    if lse is None and return_lse:
        lse = torch.empty((B, N), dtype=torch.float32, device=o_part.device)
    rc = load_library().mla_merge_splits(_ptr(o_part), _ptr(lse_part), B, N, S, V, _ptr(out),
                                         _ptr(lse), _stream_ptr(stream))
    _check(rc, "mla_merge_splits")
    return out, lse


def mla_merge_splits_v_up_proj(o_part, lse_part, w_uv, *, workspace, out=None, lse=None,
                               latent_out=None, stream=None):
    """Split merge and up-projection in one launch: fp32 ``[B,N,S,512]`` /
    ``[B,N,S]`` partials and ``W_UV [N,512,128]`` -> bf16 ``out [B,N,128]``
    (``lse`` and the merged ``latent_out`` rows only if given)."""
    import torch
    B, N, S, V = o_part.shape
    _check_tensor(o_part, "o_part", torch.float32)
    _check_tensor(lse_part, "lse_part", torch.float32, (B, N, S))
    _check_tensor(w_uv, "w_uv", torch.bfloat16, (N, 512, 128))
    if V != KV_LORA_RANK:
        raise ValueError("partials must be 512 wide")
    if out is None:
        out = torch.empty((B, N, 128), dtype=torch.bfloat16, device=o_part.device)
    _check_tensor(out, "out", torch.bfloat16, (B, N, 128))
    rc = load_library().mla_merge_splits_v_up_proj(
        _ptr(o_part), _ptr(lse_part), B, N, S, _ptr(w_uv), _ptr(out), _ptr(lse),
        _ptr(latent_out), _ptr(workspace), int(workspace.numel()), _stream_ptr(stream))
    _check(rc, "mla_merge_splits_v_up_proj")
    return out


def mla_decode_v_up_proj(q, latent_cache, block_table, seq_lens, softmax_scale, w_uv, *, plan,
                         workspace, out=None, lse=None, latent_out=None, stream=None):
    """Decode then up-projection (fused with the split merge for split plans):
    returns bf16 ``out [B, N, 128]``."""
    import torch
    B, N, _ = q.shape
    _check_tensor(w_uv, "w_uv", torch.bfloat16, (N, 512, 128))
    if out is None:
        out = torch.empty((B, N, 128), dtype=torch.bfloat16, device=q.device)
    _check_tensor(out, "out", torch.bfloat16, (B, N, 128))
    rc = load_library().mla_decode_v_up_proj(
        ctypes.byref(plan), _ptr(q), _ptr(latent_cache), int(latent_cache.shape[0]),
        _ptr(block_table), _ptr(seq_lens), float(softmax_scale), _ptr(w_uv), _ptr(out), _ptr(lse),
        _ptr(latent_out), _ptr(workspace), int(workspace.numel()), _stream_ptr(stream))
    _check(rc, "mla_decode_v_up_proj")
    return out


def dcp_local_seq_lens(seq_lens_host, world, rank, interleave):
    """Tokens of each request on ``rank`` of ``world`` (runs of ``interleave``
    tokens dealt round-robin): int32 numpy ``[B]``, computed on the host."""
    import numpy as np
    lens = np.ascontiguousarray(np.asarray(seq_lens_host, dtype=np.int32))
    local = np.empty_like(lens)
    rc = load_library().mla_dcp_local_seq_lens(
        ctypes.c_void_p(lens.ctypes.data), int(lens.size), int(world), int(rank),
        int(interleave), ctypes.c_void_p(local.ctypes.data))
    _check(rc, "mla_dcp_local_seq_lens")
    return local


def mla_dcp_combine(out_parts, lse_parts, *, out=None, lse=None, return_lse=True, stream=None):
    """Combine the ranks' results, bf16 ``[R,B,N,V]`` / fp32 ``[R,B,N]`` ->
    bf16 ``[B,N,V]``, fp32 ``[B,N]``."""
    import torch
    R, B, N, V = out_parts.shape
    _check_tensor(out_parts, "out_parts", torch.bfloat16)
    _check_tensor(lse_parts, "lse_parts", torch.float32, (R, B, N))
    if out is None:
        out = torch.empty((B, N, V), dtype=torch.bfloat16, device=out_parts.device)
    _check_tensor(out, "out", torch.bfloat16, (B, N, V))
    if lse is None and return_lse:
        lse = torch.empty((B, N), dtype=torch.float32, device=out_parts.device)
    rc = load_library().mla_dcp_combine(_ptr(out_parts), _ptr(lse_parts), R, B, N, V, _ptr(out),
                                        _ptr(lse), _stream_ptr(stream))
    _check(rc, "mla_dcp_combine")
    return out, lse


def new_status_workspace(device=None, stream=None):
    """A bare status header (for the calls that need no other workspace)."""
    import torch
    ws = torch.empty(STATUS_BYTES, dtype=torch.uint8, device=device or "cuda")
    _check(load_library().mla_workspace_init(_ptr(ws), STATUS_BYTES, _stream_ptr(stream)),
           "mla_workspace_init")
    return ws


def mla_q_absorb_concat_cache(q, w_uk_t, kv_c=None, k_pe=None, slot_mapping=None,
                              latent_cache=None, *, workspace, out=None, stream=None):
    """Decode front end: ``mqa_q [B, N, 576]`` from ``q [B, N, 192]`` and
    ``W_UK_T [N, 128, 512]``; with ``slot_mapping`` (int64 ``[B]``) the new
    tokens' ``[kv_c | k_pe]`` go into ``latent_cache`` in the same launch."""
    import torch
    B, N, _ = q.shape
    _check_tensor(q, "q", torch.bfloat16, (B, N, 192))
    _check_tensor(w_uk_t, "w_uk_t", torch.bfloat16, (N, 128, 512))
    num_blocks = 0
    if slot_mapping is not None:
        _check_tensor(slot_mapping, "slot_mapping", torch.int64, (B,))
        _check_tensor(kv_c, "kv_c", torch.bfloat16, (B, 512))
        _check_tensor(k_pe, "k_pe", torch.bfloat16, (B, 64))
        _check_tensor(latent_cache, "latent_cache", torch.bfloat16)
        num_blocks = latent_cache.shape[0]
    if out is None:
        out = torch.empty((B, N, 576), dtype=torch.bfloat16, device=q.device)
    _check_tensor(out, "out", torch.bfloat16, (B, N, 576))
    rc = load_library().mla_q_absorb_concat_cache(
        _ptr(q), _ptr(w_uk_t), _ptr(kv_c), _ptr(k_pe), _ptr(slot_mapping), _ptr(latent_cache),
        num_blocks, B, N, _ptr(out), _ptr(workspace), workspace.numel(), _stream_ptr(stream))
    _check(rc, "mla_q_absorb_concat_cache")
    return out


def mla_v_up_proj(x, w_uv, *, workspace, out=None, stream=None):
    """Up-projection: ``out [B, N, 128]`` from ``x [B, N, 512]`` and ``W_UV [N, 512, 128]``."""
    import torch
    B, N, _ = x.shape
    _check_tensor(x, "x", torch.bfloat16, (B, N, 512))
    _check_tensor(w_uv, "w_uv", torch.bfloat16, (N, 512, 128))
    if out is None:
        out = torch.empty((B, N, 128), dtype=torch.bfloat16, device=x.device)
    _check_tensor(out, "out", torch.bfloat16, (B, N, 128))
    rc = load_library().mla_v_up_proj(_ptr(x), _ptr(w_uv), B, N, _ptr(out), _ptr(workspace),
                                      workspace.numel(), _stream_ptr(stream))
    _check(rc, "mla_v_up_proj")
    return out


def _empty(shape, dtype, device, stream, fill=None):
    """A new tensor that belongs to the stream the call runs on."""
    import torch
    if stream is not None:
        with torch.cuda.stream(stream):
            return _empty(shape, dtype, device, None, fill)
    if fill is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return torch.full(shape, fill, dtype=dtype, device=device)


def _arg(name, t, dtype, device, shape=None):
    """The address of `t`, a contiguous tensor of that type (and shape) on
    `device`. The small calls take a few microseconds on the GPU, so the
    checks of what is right come first and cost least."""
    try:
        if (t.dtype is dtype and t.device == device and (shape is None or t.shape == shape)
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _check_tensor(t, name, dtype, shape)
    raise ValueError(f"{name} must be on {device}, got {t.device}")


_empty_strided = None    # torch.empty_strided, once a call has needed it


def _result(name, t, shape, dtype, device, stream):
    """The result tensor `t` of one to three dimensions, or a new one, and its address."""
    global _empty_strided
    if t is not None:
        return t, _arg(name, t, dtype, device, shape)
    if stream is not None:
        t = _empty(shape, dtype, device, stream)
    else:
        if _empty_strided is None:
            import torch
            _empty_strided = torch.empty_strided
        n = len(shape)
        strides = ((1,) if n == 1 else (shape[1], 1) if n == 2
                   else (shape[1] * shape[2], shape[2], 1))
        t = _empty_strided(shape, strides, dtype=dtype, device=device)
    return t, t.data_ptr()


def _ndim(name, t, ndim, what):
    """The shape of a tensor of `ndim` dimensions."""
    shape = getattr(t, "shape", None)
    if shape is None:
        raise TypeError(f"{name} must be a CUDA tensor")
    if len(shape) != ndim:
        raise ValueError(f"{name} must be {what}")
    return shape


def _device_of(name, t):
    """The CUDA device that a call's other tensors have to be on."""
    if not getattr(t, "is_cuda", False):
        raise TypeError(f"{name} must be a CUDA tensor")
    return t.device


def _call(device, stream, fn, *args):
    """Call a library function with `device` current, on `stream` or the
    device's current one; raises on a status."""
    import torch
    if torch._C._cuda_getDevice() != device.index:   # (CUDA is up: there is a tensor on it)
        with torch.cuda.device(device):
            return _call(device, stream, fn, *args)
    raw = (torch._C._cuda_getCurrentRawStream(device.index) if stream is None
           else stream.cuda_stream)
    rc = fn(*args, raw)
    if rc != MLA_OK:
        raise MlaError(rc, fn.__name__)


def _expand_kv(fn, cache_dtype, latent_cache, block_table, cu_seqlens_k, w_uk_t, w_uv, k_scale,
               total_k, first_token, kv, k_pe, workspace, stream):
    import torch
    bf16, i32 = torch.bfloat16, torch.int32
    dev = _device_of("latent_cache", latent_cache)
    blocks = _ndim("latent_cache", latent_cache, 3, "[num_blocks, 64, 576]")[0]
    B = _ndim("cu_seqlens_k", cu_seqlens_k, 1, "[B + 1]")[0] - 1
    rows, mb = _ndim("block_table", block_table, 2, "[B, max_blocks_per_seq]")
    N = _ndim("w_uk_t", w_uk_t, 3, "[N, 128, 512]")[0]
    T = int(total_k)
    if B < 0:
        raise ValueError("cu_seqlens_k must be [B + 1]")
    if T < 0:
        raise ValueError("total_k must not be negative")
    kv, kv_ptr = _result("kv", kv, (T, N, 256), bf16, dev, stream)
    k_pe, pe_ptr = _result("k_pe", k_pe, (T, ROPE_DIM), bf16, dev, stream)
    _call(dev, stream, fn,
          _arg("latent_cache", latent_cache, cache_dtype, dev, (blocks, PAGE_SIZE, HEAD_DIM)),
          *(() if k_scale is None else (float(k_scale),)), blocks,
          _arg("block_table", block_table, i32, dev, (B, mb)), mb,
          None if first_token is None else _arg("first_token", first_token, i32, dev, (B,)),
          _arg("cu_seqlens_k", cu_seqlens_k, i32, dev), B, T, N,
          _arg("w_uk_t", w_uk_t, bf16, dev, (N, 128, 512)),
          _arg("w_uv", w_uv, bf16, dev, (N, 512, 128)), kv_ptr, pe_ptr,
          _arg("workspace", workspace, torch.uint8, dev), workspace.numel())
    return kv, k_pe


def mla_expand_kv(latent_cache, block_table, cu_seqlens_k, w_uk_t, w_uv, *, total_k, workspace,
                  first_token=None, kv=None, k_pe=None, stream=None):
    """Per-head keys and values of cached tokens: packed row t of request b is
    its token ``first_token[b] + t - cu_seqlens_k[b]``. Returns ``(kv bf16
    [total_k, N, 256] = [k_nope | v], k_pe bf16 [total_k, 64])``; rows from
    ``cu_seqlens_k[B]`` on are not written."""
    import torch
    return _expand_kv(load_library().mla_expand_kv, torch.bfloat16, latent_cache, block_table,
                      cu_seqlens_k, w_uk_t, w_uv, None, total_k, first_token, kv, k_pe, workspace,
                      stream)


def mla_expand_kv_fp8(latent_cache_fp8, block_table, cu_seqlens_k, w_uk_t, w_uv, k_scale, *,
                      total_k, workspace, first_token=None, kv=None, k_pe=None, stream=None):
    """``mla_expand_kv`` over an fp8 cache (uint8 E4M3 codes, per-tensor ``k_scale``)."""
    import torch
    return _expand_kv(load_library().mla_expand_kv_fp8, torch.uint8, latent_cache_fp8, block_table,
                      cu_seqlens_k, w_uk_t, w_uv, k_scale, total_k, first_token, kv, k_pe,
                      workspace, stream)


def make_prefill_plan(batch, num_heads, total_q, max_q_len, max_k_len, *, num_kv_splits=0,
                      num_sms=None):
    """Call mla_prefill_plan (host only; no device work)."""
    if num_sms is None:
        import torch
        num_sms = (torch.cuda.get_device_properties(0).multi_processor_count
                   if torch.cuda.is_available() else 152)
    plan = MlaPrefillPlan()
    _check(load_library().mla_prefill_plan(int(batch), int(num_heads), int(total_q),
                                           int(max_q_len), int(max_k_len), int(num_kv_splits),
                                           int(num_sms), ctypes.byref(plan)), "mla_prefill_plan")
    return plan


def mla_prefill(q, kv, k_pe, cu_seqlens_q, cu_seqlens_k, softmax_scale, *, causal=True, plan=None,
                max_q_len=None, max_k_len=None, num_kv_splits=0, out=None, lse=None,
                return_lse=True, workspace=None, stream=None):
    """Expanded-form attention of packed sequences: ``q [Tq, N, 192]`` over
    ``kv [Tk, N, 256] = [k_nope | v]`` and ``k_pe [Tk, 64]``; query i of a
    sequence sees its keys up to ``Lk - Lq + i`` (``causal``) or all of them.
    Returns ``(out bf16 [Tq, N, 128], lse fp32 [Tq, N] | None)``; rows past
    ``cu_seqlens_q[B]`` are not written.

    Without a ``plan`` the call makes one for sequences of up to ``max_q_len``
    queries and ``max_k_len`` keys; a length that is not given (the starts lie
    on the device) is taken to be the same for all: ``Tq / B``, ``Tk / B``. The
    lengths pick the kernel and the splits alone; longer sequences are computed
    too, more slowly."""
    import torch
    bf16, i32 = torch.bfloat16, torch.int32
    dev = _device_of("q", q)
    T, N, _ = _ndim("q", q, 3, "[total_q, N, 192]")
    Tk = _ndim("kv", kv, 3, "[total_k, N, 256]")[0]
    B = _ndim("cu_seqlens_q", cu_seqlens_q, 1, "[B + 1]")[0] - 1
    if B < 0:
        raise ValueError("cu_seqlens_q must be [B + 1]")
    if plan is None:
        seqs = max(B, 1)
        plan = make_prefill_plan(
            B, N, T, -(-T // seqs) if max_q_len is None else max_q_len,
            -(-Tk // seqs) if max_k_len is None else max_k_len, num_kv_splits=num_kv_splits,
            num_sms=torch.cuda.get_device_properties(dev).multi_processor_count)
    elif plan.batch != B or plan.num_heads != N or plan.total_q != T:
        raise ValueError(f"the plan is for (B, N, total_q) = "
                         f"{plan.batch, plan.num_heads, plan.total_q}, not {B, N, T}")
    out, out_ptr = _result("out", out, (T, N, 128), bf16, dev, stream)
    lse_ptr = None
    if lse is not None or return_lse:
        lse, lse_ptr = _result("lse", lse, (T, N), torch.float32, dev, stream)
    if workspace is None:
        workspace = _empty((int(plan.workspace_bytes),), torch.uint8, dev, stream)
        _call(dev, stream, load_library().mla_workspace_init, workspace.data_ptr(),
              workspace.numel())
    _call(dev, stream, load_library().mla_prefill, ctypes.byref(plan),
          _arg("q", q, bf16, dev, (T, N, 192)), _arg("kv", kv, bf16, dev, (Tk, N, 256)),
          _arg("k_pe", k_pe, bf16, dev, (Tk, ROPE_DIM)), Tk,
          _arg("cu_seqlens_q", cu_seqlens_q, i32, dev),
          _arg("cu_seqlens_k", cu_seqlens_k, i32, dev, (B + 1,)), 1 if causal else 0,
          float(softmax_scale), out_ptr, lse_ptr,
          _arg("workspace", workspace, torch.uint8, dev), workspace.numel())
    return out, lse


def new_cache_workspace(num_blocks, children=0, device=None, stream=None):
    """A workspace for mla_cache_fork (of up to `children`), _free and _compact."""
    nbytes = int(load_library().mla_cache_workspace_bytes(int(num_blocks), int(children)))
    if nbytes == 0:
        raise MlaError(MLA_ERR_UNSUPPORTED, "mla_cache_workspace_bytes")
    import torch
    dev = torch.device(device or "cuda")
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    ws = _empty((nbytes,), torch.uint8, dev, stream)
    _call(dev, stream, load_library().mla_workspace_init, ws.data_ptr(), nbytes)
    return ws


def _cache_view(latent_cache, device):
    """(pointer, layers, layer stride in bytes, blocks, bytes per entry) of a
    cache [num_blocks, 64, 576] or [layers, num_blocks, 64, 576], bf16 or
    uint8; each layer contiguous, the layers any distance apart."""
    import torch
    t = latent_cache
    if _device_of("latent_cache", t) != device:
        raise ValueError(f"latent_cache must be on {device}, got {t.device}")
    if t.dtype is not torch.bfloat16 and t.dtype is not torch.uint8:
        raise TypeError(f"latent_cache must be bfloat16 or uint8, got {t.dtype}")
    shape, size = t.shape, t.element_size()
    if len(shape) not in (3, 4) or shape[-2:] != (PAGE_SIZE, HEAD_DIM):
        raise ValueError("latent_cache must be [num_blocks, 64, 576] or "
                         "[layers, num_blocks, 64, 576]")
    if not t.is_contiguous() and (len(shape) == 3 or not t[0].is_contiguous()):
        raise ValueError("each layer of latent_cache must be contiguous")
    if len(shape) == 3:
        return t.data_ptr(), 1, 0, shape[0], size
    return t.data_ptr(), shape[0], t.stride(0) * size, shape[1], size


def mla_cache_fork(latent_cache, ref_counts, block_table, parents, shared_lens, child_lens, *,
                   workspace, child_table=None, ref_counts_out=None, stream=None):
    """Requests that start from cached ones: child c shares the whole pages of
    the first ``shared_lens[c]`` tokens of row ``parents[c]``, gets a copy of
    the rest of them and fresh pages up to ``child_lens[c]`` tokens. Returns
    ``(child_table int32 [C, max_blocks], counts)``; the counts are
    ``ref_counts`` itself unless ``ref_counts_out`` is given, and a new child
    table's unused entries are -1. All or nothing: see the header."""
    import torch
    i32 = torch.int32
    dev = _device_of("ref_counts", ref_counts)
    view = _cache_view(latent_cache, dev)
    blocks = view[3]
    rows, mb = _ndim("block_table", block_table, 2, "[rows, max_blocks_per_seq]")
    C = _ndim("parents", parents, 1, "[children]")[0]
    if child_table is None:
        child_table = _empty((C, mb), i32, dev, stream, fill=-1)
    out = ref_counts if ref_counts_out is None else ref_counts_out
    _call(dev, stream, load_library().mla_cache_fork, *view,
          _arg("ref_counts", ref_counts, i32, dev, (blocks,)),
          _arg("ref_counts_out", out, i32, dev, (blocks,)),
          _arg("block_table", block_table, i32, dev), rows, mb,
          _arg("parents", parents, i32, dev), _arg("shared_lens", shared_lens, i32, dev, (C,)),
          _arg("child_lens", child_lens, i32, dev, (C,)), C,
          _arg("child_table", child_table, i32, dev, (C, mb)),
          _arg("workspace", workspace, torch.uint8, dev), workspace.numel())
    return child_table, out


def mla_cache_free(ref_counts, block_table, seq_lens, free_rows, *, workspace, ref_counts_out=None,
                   num_freed=None, stream=None):
    """Take the rows ``free_rows`` (int32 [count]) off their pages' counts.
    Returns ``(counts, num_freed int32 [1])``; the counts are ``ref_counts``
    itself unless ``ref_counts_out`` is given."""
    import torch
    i32 = torch.int32
    dev = _device_of("ref_counts", ref_counts)
    blocks = _ndim("ref_counts", ref_counts, 1, "[num_blocks]")[0]
    rows, mb = _ndim("block_table", block_table, 2, "[rows, max_blocks_per_seq]")
    count = _ndim("free_rows", free_rows, 1, "[count]")[0]
    out = ref_counts if ref_counts_out is None else ref_counts_out
    num_freed, freed_ptr = _result("num_freed", num_freed, (1,), i32, dev, stream)
    _call(dev, stream, load_library().mla_cache_free, _arg("ref_counts", ref_counts, i32, dev),
          _arg("ref_counts_out", out, i32, dev, (blocks,)), blocks,
          _arg("block_table", block_table, i32, dev), rows, mb,
          _arg("seq_lens", seq_lens, i32, dev, (rows,)), _arg("free_rows", free_rows, i32, dev),
          count, freed_ptr, _arg("workspace", workspace, torch.uint8, dev), workspace.numel())
    return out, num_freed


def mla_cache_compact(latent_cache, ref_counts, block_table, seq_lens, *, workspace,
                      block_table_out=None, ref_counts_out=None, page_map=None, num_live=None,
                      stream=None):
    """Move the M live pages into ids 0..M-1 with the fewest copies. Returns
    ``(block table, counts, page_map int32 [num_blocks], num_live int32 [1])``;
    table and counts are changed in place unless ``*_out`` are given."""
    import torch
    i32 = torch.int32
    dev = _device_of("ref_counts", ref_counts)
    view = _cache_view(latent_cache, dev)
    blocks = view[3]
    rows, mb = _ndim("block_table", block_table, 2, "[rows, max_blocks_per_seq]")
    out = ref_counts if ref_counts_out is None else ref_counts_out
    table = block_table if block_table_out is None else block_table_out
    page_map, map_ptr = _result("page_map", page_map, (blocks,), i32, dev, stream)
    num_live, live_ptr = _result("num_live", num_live, (1,), i32, dev, stream)
    _call(dev, stream, load_library().mla_cache_compact, *view,
          _arg("ref_counts", ref_counts, i32, dev, (blocks,)),
          _arg("ref_counts_out", out, i32, dev, (blocks,)),
          _arg("block_table", block_table, i32, dev),
          _arg("block_table_out", table, i32, dev, (rows, mb)), rows, mb,
          _arg("seq_lens", seq_lens, i32, dev, (rows,)),
          map_ptr, live_ptr, _arg("workspace", workspace, torch.uint8, dev), workspace.numel())
    return table, out, page_map, num_live


# The GPU is done with the smallest of the calls below in a few microseconds, so
# what they cost is what the host takes. Each has its checks in one expression
# (a decode over a shared prefix: 20.3 -> 17.4 us of the host's time a call); only
# a call that fails it goes through them one by one, to the error.

_NOT_FINE = (AttributeError, IndexError, TypeError, ValueError)


def _check_rows(name, t, rows, width, device):
    """`t` is bf16 [rows, width], columns contiguous, rows a multiple of 8 elements apart."""
    import torch
    if _device_of(name, t) != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.shape != (rows, width) or t.stride(1) != 1:
        raise ValueError(f"{name} must be [{rows}, {width}], a row for each slot, with "
                         "contiguous columns")
    if rows > 1 and t.stride(0) % 8:
        raise ValueError(f"{name}'s rows must lie a multiple of 8 elements apart, not {t.stride(0)}")


def _check_write(cache_dtype, kv_c, k_pe, slot_mapping, latent_cache, workspace):
    import torch
    dev = _device_of("latent_cache", latent_cache)
    blocks = _ndim("latent_cache", latent_cache, 3, "[num_blocks, 64, 576]")[0]
    T = _ndim("slot_mapping", slot_mapping, 1, "[T]")[0]
    _check_rows("kv_c", kv_c, T, KV_LORA_RANK, dev)
    _check_rows("k_pe", k_pe, T, ROPE_DIM, dev)
    _arg("latent_cache", latent_cache, cache_dtype, dev, (blocks, PAGE_SIZE, HEAD_DIM))
    _arg("slot_mapping", slot_mapping, torch.int64, dev)
    _arg("workspace", workspace, torch.uint8, dev)


def _cache_write(fn, cache_dtype, kv_c, k_pe, slot_mapping, latent_cache, scales, workspace, stream):
    import torch
    bf16 = torch.bfloat16
    try:
        dev, shape, T = latent_cache.device, latent_cache.shape, slot_mapping.shape[0]
        fine = (latent_cache.is_cuda and latent_cache.dtype is cache_dtype
                and shape == (shape[0], PAGE_SIZE, HEAD_DIM) and latent_cache.is_contiguous()
                and slot_mapping.dtype is torch.int64 and slot_mapping.device == dev
                and slot_mapping.shape == (T,) and slot_mapping.is_contiguous()
                and kv_c.dtype is bf16 and kv_c.device == dev and kv_c.shape == (T, KV_LORA_RANK)
                and k_pe.dtype is bf16 and k_pe.device == dev and k_pe.shape == (T, ROPE_DIM)
                and workspace.dtype is torch.uint8 and workspace.device == dev
                and workspace.is_contiguous())
        if fine:
            (kv_stride, kv_inner), (pe_stride, pe_inner) = kv_c.stride(), k_pe.stride()
            fine = kv_inner == 1 and pe_inner == 1 and (T == 1 or not (kv_stride | pe_stride) & 7)
    except _NOT_FINE:
        fine = False
    if not fine:
        _check_write(cache_dtype, kv_c, k_pe, slot_mapping, latent_cache, workspace)
    if T <= 1:                          # (the distance of rows means nothing)
        kv_stride, pe_stride = KV_LORA_RANK, ROPE_DIM
    _call(dev, stream, fn, kv_c.data_ptr(), kv_stride, k_pe.data_ptr(), pe_stride,
          slot_mapping.data_ptr(), T, *scales, latent_cache.data_ptr(), shape[0],
          workspace.data_ptr(), workspace.numel())
    return latent_cache


def mla_cache_write(kv_c, k_pe, slot_mapping, latent_cache, *, workspace, stream=None):
    """New tokens' entries ``[kv_c | k_pe]`` (bf16 ``[T, 512]`` and ``[T, 64]``,
    their rows any multiple of 8 elements apart) into the rows ``slot_mapping``
    (int64 ``[T]``; negative: none) of ``latent_cache``, which is returned."""
    import torch
    return _cache_write(load_library().mla_cache_write, torch.bfloat16, kv_c, k_pe, slot_mapping,
                        latent_cache, (), workspace, stream)


def mla_cache_write_fp8(kv_c, k_pe, slot_mapping, latent_cache_fp8, k_scale, *, workspace,
                        stream=None):
    """``mla_cache_write`` into an fp8 cache: the E4M3 codes (uint8) nearest to
    the entries divided by ``k_scale``, saturating at +-448."""
    import torch
    return _cache_write(load_library().mla_cache_write_fp8, torch.uint8, kv_c, k_pe, slot_mapping,
                        latent_cache_fp8, (float(k_scale),), workspace, stream)


def _check_gather(cache_dtype, latent_cache, block_table, cu_seqlens_k, total_k, first_token,
                  workspace):
    import torch
    i32 = torch.int32
    dev = _device_of("latent_cache", latent_cache)
    blocks = _ndim("latent_cache", latent_cache, 3, "[num_blocks, 64, 576]")[0]
    B = _ndim("cu_seqlens_k", cu_seqlens_k, 1, "[B + 1]")[0] - 1
    _, mb = _ndim("block_table", block_table, 2, "[B, max_blocks_per_seq]")
    if B < 0:
        raise ValueError("cu_seqlens_k must be [B + 1]")
    if total_k < 0:
        raise ValueError("total_k must not be negative")
    _arg("latent_cache", latent_cache, cache_dtype, dev, (blocks, PAGE_SIZE, HEAD_DIM))
    _arg("block_table", block_table, i32, dev, (B, mb))
    if first_token is not None:
        _arg("first_token", first_token, i32, dev, (B,))
    _arg("cu_seqlens_k", cu_seqlens_k, i32, dev)
    _arg("workspace", workspace, torch.uint8, dev)


def _cache_gather(fn, cache_dtype, latent_cache, block_table, cu_seqlens_k, scales, total_k,
                  first_token, rows, workspace, stream):
    import torch
    i32, T = torch.int32, int(total_k)
    try:
        dev, shape, (B, mb) = latent_cache.device, latent_cache.shape, block_table.shape
        fine = (latent_cache.is_cuda and latent_cache.dtype is cache_dtype
                and shape == (shape[0], PAGE_SIZE, HEAD_DIM) and latent_cache.is_contiguous()
                and block_table.dtype is i32 and block_table.device == dev
                and block_table.is_contiguous() and cu_seqlens_k.dtype is i32
                and cu_seqlens_k.device == dev and cu_seqlens_k.shape == (B + 1,)
                and cu_seqlens_k.is_contiguous()
                and (first_token is None or first_token.dtype is i32
                     and first_token.device == dev and first_token.shape == (B,)
                     and first_token.is_contiguous())
                and workspace.dtype is torch.uint8 and workspace.device == dev
                and workspace.is_contiguous() and T >= 0)
    except _NOT_FINE:
        fine = False
    if not fine:
        _check_gather(cache_dtype, latent_cache, block_table, cu_seqlens_k, T, first_token,
                      workspace)
    rows, rows_ptr = _result("rows", rows, (T, HEAD_DIM), torch.bfloat16, dev, stream)
    _call(dev, stream, fn, latent_cache.data_ptr(), *scales, shape[0], block_table.data_ptr(), mb,
          None if first_token is None else first_token.data_ptr(), cu_seqlens_k.data_ptr(), B, T,
          rows_ptr, workspace.data_ptr(), workspace.numel())
    return rows


def mla_cache_gather(latent_cache, block_table, cu_seqlens_k, *, total_k, workspace,
                     first_token=None, rows=None, stream=None):
    """Cached entries side by side: packed row t of request b is its token
    ``first_token[b] + t - cu_seqlens_k[b]``. Returns ``rows`` bf16 ``[total_k,
    576]``; rows from ``cu_seqlens_k[B]`` on are not written."""
    import torch
    return _cache_gather(load_library().mla_cache_gather, torch.bfloat16, latent_cache, block_table,
                         cu_seqlens_k, (), total_k, first_token, rows, workspace, stream)


def mla_cache_gather_fp8(latent_cache_fp8, block_table, cu_seqlens_k, k_scale, *, total_k,
                         workspace, first_token=None, rows=None, stream=None):
    """``mla_cache_gather`` over an fp8 cache (uint8 E4M3 codes, per-tensor ``k_scale``)."""
    import torch
    return _cache_gather(load_library().mla_cache_gather_fp8, torch.uint8, latent_cache_fp8,
                         block_table, cu_seqlens_k, (float(k_scale),), total_k, first_token, rows,
                         workspace, stream)


def make_span_plan(batch, num_heads, max_blocks_per_seq, *, max_groups=0, num_sms=None,
                   extra_flags=0):
    """Call mla_span_plan (host only; no device work): a plan for
    ``mla_decode_shared`` of up to `max_groups` groups, or ``mla_decode_window``."""
    if num_sms is None:
        import torch
        num_sms = (torch.cuda.get_device_properties(0).multi_processor_count
                   if torch.cuda.is_available() else 152)
    plan = MlaSpanPlan()
    _check(load_library().mla_span_plan(int(batch), int(num_heads), int(max_blocks_per_seq),
                                        int(max_groups), int(num_sms), int(extra_flags),
                                        ctypes.byref(plan)), "mla_span_plan")
    return plan


def _check_span(cache_dtype, q, latent_cache, block_table, seq_lens, groups, plan):
    import torch
    i32 = torch.int32
    dev = _device_of("q", q)
    B, N, _ = _ndim("q", q, 3, "[B, N, 576]")
    blocks = _ndim("latent_cache", latent_cache, 3, "[num_blocks, 64, 576]")[0]
    mb = _ndim("block_table", block_table, 2, "[B, max_blocks_per_seq]")[1]
    if plan is not None and (plan.batch, plan.num_heads, plan.max_blocks_per_seq) != (B, N, mb):
        raise ValueError(f"the plan is for (B, N, max_blocks_per_seq) = "
                         f"{plan.batch, plan.num_heads, plan.max_blocks_per_seq}, not {B, N, mb}")
    _arg("q", q, torch.bfloat16, dev, (B, N, HEAD_DIM))
    _arg("latent_cache", latent_cache, cache_dtype, dev, (blocks, PAGE_SIZE, HEAD_DIM))
    _arg("block_table", block_table, i32, dev, (B, mb))
    _arg("seq_lens", seq_lens, i32, dev, (B,))
    if groups is not None:
        group_starts, shared_lens = groups
        G = _ndim("shared_lens", shared_lens, 1, "[groups]")[0]
        if plan is not None and G > plan.max_groups:
            raise ValueError(f"the plan is for up to {plan.max_groups} groups, not {G}")
        _arg("group_starts", group_starts, i32, dev, (G + 1,))
        _arg("shared_lens", shared_lens, i32, dev, (G,))


def _decode_span(fn, cache_dtype, q, latent_cache, block_table, seq_lens, groups, window, scales,
                 plan, out, lse, return_lse, workspace, stream):
    """One of the decodes over parts of the tokens: `groups` (their starts and
    shared lengths) or None, and else the window and the sinks."""
    import torch
    i32, G, middle = torch.int32, 0, window
    try:
        dev, (B, N, width), shape = q.device, q.shape, latent_cache.shape
        mb = block_table.shape[1]
        fine = (q.is_cuda and q.dtype is torch.bfloat16 and width == HEAD_DIM and q.is_contiguous()
                and latent_cache.dtype is cache_dtype and latent_cache.device == dev
                and shape == (shape[0], PAGE_SIZE, HEAD_DIM) and latent_cache.is_contiguous()
                and block_table.dtype is i32 and block_table.device == dev
                and block_table.shape == (B, mb) and block_table.is_contiguous()
                and seq_lens.dtype is i32 and seq_lens.device == dev and seq_lens.shape == (B,)
                and seq_lens.is_contiguous()
                and (plan is None or plan.batch == B and plan.num_heads == N
                     and plan.max_blocks_per_seq == mb))
        if fine and groups is not None:
            group_starts, shared_lens = groups
            G = shared_lens.shape[0]
            fine = (shared_lens.dtype is i32 and shared_lens.device == dev
                    and shared_lens.shape == (G,) and shared_lens.is_contiguous()
                    and group_starts.dtype is i32 and group_starts.device == dev
                    and group_starts.shape == (G + 1,) and group_starts.is_contiguous()
                    and (plan is None or G <= plan.max_groups))
            middle = (group_starts.data_ptr(), shared_lens.data_ptr(), G)
    except _NOT_FINE:
        fine = False
    if not fine:
        _check_span(cache_dtype, q, latent_cache, block_table, seq_lens, groups, plan)
    if plan is None:
        plan = make_span_plan(B, N, mb, max_groups=G, num_sms=torch.cuda.get_device_properties(
            dev).multi_processor_count)
    out, out_ptr = _result("out", out, (B, N, KV_LORA_RANK), torch.bfloat16, dev, stream)
    lse_ptr = None
    if lse is not None or return_lse:
        lse, lse_ptr = _result("lse", lse, (B, N), torch.float32, dev, stream)
    if workspace is None:
        workspace = _empty((int(plan.workspace_bytes),), torch.uint8, dev, stream)
        _call(dev, stream, load_library().mla_workspace_init, workspace.data_ptr(),
              workspace.numel())
    _call(dev, stream, fn, ctypes.byref(plan), q.data_ptr(), latent_cache.data_ptr(), shape[0],
          block_table.data_ptr(), seq_lens.data_ptr(), *middle, *scales, out_ptr, lse_ptr,
          _arg("workspace", workspace, torch.uint8, dev), workspace.numel())
    return out, lse


def mla_decode_shared(q, latent_cache, block_table, seq_lens, group_starts, shared_lens,
                      softmax_scale, *, plan=None, out=None, lse=None, return_lse=True,
                      workspace=None, stream=None):
    """``mla_decode`` of a batch whose requests ``group_starts[g]`` ..
    ``group_starts[g + 1] - 1`` (int32 ``[G + 1]``) share their first
    ``shared_lens[g]`` tokens (int32 ``[G]``). Where that saves time, their whole
    pages are attended to once for the group's rows together; a batch that
    would gain little, and any of 128 heads, is decoded request by request.
    Returns ``(out bf16 [B, N, 512], lse fp32 [B, N] | None)``, as ``mla_decode``
    would."""
    import torch
    return _decode_span(load_library().mla_decode_shared, torch.bfloat16, q, latent_cache,
                        block_table, seq_lens, (group_starts, shared_lens), None,
                        (float(softmax_scale),), plan, out, lse, return_lse, workspace, stream)


def mla_decode_shared_fp8(q, latent_cache_fp8, block_table, seq_lens, group_starts, shared_lens,
                          softmax_scale, k_scale, *, plan=None, out=None, lse=None,
                          return_lse=True, workspace=None, stream=None):
    """``mla_decode_shared`` over an fp8 cache (uint8 E4M3 codes, per-tensor ``k_scale``)."""
    import torch
    return _decode_span(load_library().mla_decode_shared_fp8, torch.uint8, q, latent_cache_fp8,
                        block_table, seq_lens, (group_starts, shared_lens), None,
                        (float(softmax_scale), float(k_scale)), plan, out, lse, return_lse,
                        workspace, stream)


def _window(window, sinks):
    """(a window or sinks past every length see what the longest lengths would)"""
    most = 2 ** 31 - 1
    window, sinks = min(int(window), most), min(int(sinks), most)
    if window < 1 or sinks < 0:
        raise ValueError("window must be at least 1, sinks at least 0")
    return window, sinks


def mla_decode_window(q, latent_cache, block_table, seq_lens, softmax_scale, *, window, sinks=0,
                      plan=None, out=None, lse=None, return_lse=True, workspace=None, stream=None):
    """``mla_decode`` in which a request of L tokens sees its last ``window``
    ones and its first ``sinks`` ones; pages in between are not read. Returns
    ``(out bf16 [B, N, 512], lse fp32 [B, N] | None)``."""
    import torch
    return _decode_span(load_library().mla_decode_window, torch.bfloat16, q, latent_cache,
                        block_table, seq_lens, None, _window(window, sinks),
                        (float(softmax_scale),), plan, out, lse, return_lse, workspace, stream)


def mla_decode_window_fp8(q, latent_cache_fp8, block_table, seq_lens, softmax_scale, k_scale, *,
                          window, sinks=0, plan=None, out=None, lse=None, return_lse=True,
                          workspace=None, stream=None):
    """``mla_decode_window`` over an fp8 cache (uint8 E4M3 codes, per-tensor ``k_scale``)."""
    import torch
    return _decode_span(load_library().mla_decode_window_fp8, torch.uint8, q, latent_cache_fp8,
                        block_table, seq_lens, None, _window(window, sinks),
                        (float(softmax_scale), float(k_scale)), plan, out, lse, return_lse,
                        workspace, stream)


def read_error(workspace, stream=None):
    """Synchronise and return (and clear) the device status word of `workspace`."""
    st = ctypes.c_int(0)
    _check(load_library().mla_read_error(_ptr(workspace), ctypes.byref(st), _stream_ptr(stream)),
           "mla_read_error")
    return st.value


def debug_gather_pages(latent_cache, block_table, seq_lens, dst, workspace, stream=None):
    """Test hook: dense gather of every request's rows into ``dst [B, T, 576]``."""
    import torch
    _check_tensor(latent_cache, "latent_cache", torch.bfloat16)
    _check_tensor(dst, "dst", torch.bfloat16)
    B = block_table.shape[0]
    rc = load_library().mla_debug_gather_pages(
        _ptr(latent_cache), int(latent_cache.shape[0]), _ptr(block_table), _ptr(seq_lens), B,
        int(block_table.shape[1]), int(dst.shape[1]), _ptr(dst), _ptr(workspace),
        int(workspace.numel()), _stream_ptr(stream))
    _check(rc, "mla_debug_gather_pages")
    return dst


def debug_loader_pages(plan, latent_cache, block_table, seq_lens, dst, workspace, stream=None):
    """Test hook: the tensor-core kernel's page loaders alone under ``plan``;
    ``dst`` bf16 ``[2, B, T, 576]`` receives, per CTA rank, the rows it loaded."""
    import torch
    _check_tensor(latent_cache, "latent_cache", torch.bfloat16)
    _check_tensor(dst, "dst", torch.bfloat16)
    if dst.dim() != 4 or dst.shape[0] != 2 or dst.shape[1] != plan.batch or dst.shape[3] != 576:
        raise ValueError("dst must be [2, B, T, 576]")
    rc = load_library().mla_debug_loader_pages(
        ctypes.byref(plan), _ptr(latent_cache), int(latent_cache.shape[0]), _ptr(block_table),
        _ptr(seq_lens), int(dst.shape[2]), _ptr(dst), _ptr(workspace), int(workspace.numel()),
        _stream_ptr(stream))
    _check(rc, "mla_debug_loader_pages")
    return dst


def mla_decode_noalloc(q, latent_cache, block_table, seq_lens, softmax_scale, *, plan,
                       out=None, lse=None, device_status=None, stream=None):
    """The decode without a workspace, for callers that cannot allocate device
    memory (see ``mla_decode_noalloc`` in include/mla_decode.h): scratch comes
    from a fixed array inside the library. ``out``/``lse``/``device_status``
    may be given preallocated; nothing here allocates when all three are."""
    import torch
    B, N, _ = q.shape
    if out is None:
        out = torch.empty((B, N, KV_LORA_RANK), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, N), dtype=torch.float32, device=q.device)
    rc = load_library().mla_decode_noalloc(
        ctypes.byref(plan), _ptr(q), _ptr(latent_cache), int(latent_cache.shape[0]),
        _ptr(block_table), _ptr(seq_lens), float(softmax_scale), _ptr(out), _ptr(lse),
        _ptr(device_status), _stream_ptr(stream))
    _check(rc, "mla_decode_noalloc")
    return out, lse
