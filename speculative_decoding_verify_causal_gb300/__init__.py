"""GB300-native speculative-decoding verify attention.

Thin ctypes binding over ``libverify_attn.so`` (built in-tree by
``speculative_decoding_verify_causal_gb300.build``).  The functions carry the
C ABI's names and do argument marshalling only: every step of the attention
runs in the library's CUDA kernels.  PyTorch supplies device memory and
streams.  There is no CPU fallback: importing this package without the built
library raises.

Layouts (see ``include/verify_attn.h``):
  q bf16 [B, T, Hq, D]; k_pages / v_pages [num_pages, 16, Hkv, D] of
  bf16 / fp8-e4m3 (uint8 storage) / int8; k_scale / v_scale fp32
  [num_pages, 16, Hkv]; block_table int32 [B, stride]; seq_lens int32 [B];
  out bf16 [B, T, Hq, D]; lse fp32 [B, T, Hq].

Around the verify step: ``verify_attn_rope`` and ``verify_attn_rope_append``
(rotary positions with several axes, alone and with the KV append),
``verify_attn_accept_probs`` (acceptance from given probabilities and random
numbers) and ``PagePool`` with ``verify_attn_pages_resize`` / ``_fork`` /
``_compact`` (the pages behind the block table).

A prompt in chunks: ``verify_attn_chunk`` over a ``verify_attn_chunk_plan``
(attention of ragged chunks of new tokens), ``verify_attn_chunk_weights`` (the
attention weight that cached tokens gather), ``verify_attn_evict`` (cutting
sequences back to their heaviest tokens) and ``verify_attn_logprobs`` (log
probabilities, places, entropy and top alternatives).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libverify_attn.so")

VA_BF16, VA_FP8_E4M3, VA_INT8, VA_INT4, VA_INT2 = 0, 1, 2, 3, 4
KV_DTYPE_CODES = {"bf16": VA_BF16, "fp8_e4m3": VA_FP8_E4M3, "int8": VA_INT8, "int4": VA_INT4, "int2": VA_INT2}
VA_PATH_AUTO, VA_PATH_WARP, VA_PATH_MMA = 0, 1, 2
PATH_CODES = {"auto": VA_PATH_AUTO, "warp": VA_PATH_WARP, "mma": VA_PATH_MMA}
PAGE_SIZE = 16
VA_FLOAT_BF16, VA_FLOAT_FP16, VA_FLOAT_FP32 = 0, 1, 2
ROPE_MAX_PAIRS, ROPE_MAX_AXES = 128, 4
LOGPROBS_MAX_TOP = 32
# bits of a page pool's flag word
VA_PAGES_BAD_ENTRY, VA_PAGES_EXHAUSTED, VA_PAGES_BAD_REQUEST, VA_PAGES_BAD_COUNT = 1, 8, 16, 32

STATUS_NAMES = {
    0: "VA_OK", -1: "VA_ERR_INVALID_ARGUMENT", -2: "VA_ERR_UNSUPPORTED",
    -3: "VA_ERR_PLAN_MISMATCH", -4: "VA_ERR_NO_PLAN", -5: "VA_ERR_CUDA",
    -6: "VA_ERR_OUT_OF_MEMORY", -7: "VA_ERR_NO_DEVICE", -8: "VA_ERR_SCRATCH_TOO_SMALL",
}


class VerifyAttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = f"{what}: {STATUS_NAMES.get(status, status)} ({verify_attn_status_string(status)})"
        if status == -5:
            lib = _load()
            msg += f" [cuda error {lib.verify_attn_last_cuda_error()}: " \
                   f"{lib.verify_attn_last_cuda_error_string().decode()}]"
        super().__init__(msg)


class _Options(ctypes.Structure):
    _fields_ = [("block_table_stride", ctypes.c_int), ("tokens_per_split", ctypes.c_int),
                ("path", ctypes.c_int), ("num_pages", ctypes.c_int)]


class PlanInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "num_seqs", "T", "num_q_heads", "num_kv_heads", "head_dim", "kv_dtype", "path",
        "rows_per_group", "num_row_groups", "tokens_per_split", "num_items",
        "num_split_groups", "max_splits", "num_sms")] + [("workspace_bytes", ctypes.c_longlong)]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class ChunkPlanInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "num_seqs", "num_q_heads", "num_kv_heads", "head_dim", "kv_dtype", "num_tokens", "max_blocks", "num_items",
        "num_split_groups", "max_item_keys", "num_sms")] + [("workspace_bytes", ctypes.c_longlong)]

    as_dict = PlanInfo.as_dict


class _Rope(ctypes.Structure):
    _fields_ = [("turn", ctypes.c_uint64 * ROPE_MAX_PAIRS), ("axis", ctypes.c_uint8 * ROPE_MAX_PAIRS),
                ("num_pairs", ctypes.c_int32), ("num_axes", ctypes.c_int32), ("adjacent", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class _Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride_seq", ctypes.c_int64), ("stride_token", ctypes.c_int64),
                ("stride_head", ctypes.c_int64), ("num_heads", ctypes.c_int)]


class _Positions(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride_axis", ctypes.c_int64), ("stride_seq", ctypes.c_int64),
                ("stride_token", ctypes.c_int64)]


class _Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride_seq", ctypes.c_int64), ("stride_pos", ctypes.c_int64)]


class _PageBuffer(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("page_bytes", ctypes.c_size_t)]


class _PagePool(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("block_table", "seq_lens", "ref_count", "free_list", "num_free", "flags")
                ] + [(n, ctypes.c_int) for n in ("block_table_stride", "num_seqs", "num_pages", "num_buffers")
                     ] + [("buffers", ctypes.POINTER(_PageBuffer)), ("workspace", ctypes.c_void_p)]


_lib = None
_lib_lock = threading.Lock()


def _load():
    global _lib
    with _lib_lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is not built: run `python -m speculative_decoding_verify_causal_gb300.build` "
                "(the package has no CPU fallback)")
        lib = ctypes.CDLL(LIB_PATH)
        P, I = ctypes.c_void_p, ctypes.c_int
        lib.verify_attn_plan.argtypes = [P, I, I, I, I, I, I, I, ctypes.POINTER(P)]
        lib.verify_attn_plan_ex.argtypes = [P, I, I, I, I, I, I, I, ctypes.POINTER(_Options), ctypes.POINTER(P)]
        lib.verify_attn.argtypes = [P] * 7 + [I, P, P, P]
        lib.verify_attn_with_plan.argtypes = [P] + [P] * 7 + [I, P, P, P]
        lib.verify_attn_plan_destroy.argtypes = [P]
        lib.verify_attn_plan_destroy.restype = None
        lib.verify_attn_status_string.argtypes = [I]
        lib.verify_attn_status_string.restype = ctypes.c_char_p
        lib.verify_attn_plan_get_info.argtypes = [P, ctypes.POINTER(PlanInfo)]
        lib.verify_attn_plan_describe.argtypes = [P, I, I, I, I, I, I, I, ctypes.POINTER(_Options),
                                                  ctypes.POINTER(PlanInfo), P, I]
        lib.verify_attn_plan_device_flags.argtypes = [P, I, ctypes.POINTER(I), P]
        lib.verify_attn_plan_set_events.argtypes = [P, P, P]
        lib.verify_attn_plan_set_events.restype = I
        lib.verify_attn_last_cuda_error.argtypes = []
        lib.verify_attn_last_cuda_error.restype = I
        lib.verify_attn_last_cuda_error_string.argtypes = []
        lib.verify_attn_last_cuda_error_string.restype = ctypes.c_char_p
        lib.verify_attn_noalloc.argtypes = [P, I, I, I, I, I, I] + [P] * 6 + [I, I, P, P, P, P]
        lib.verify_attn_noalloc_flags.argtypes = [I, ctypes.POINTER(I), P]
        lib.verify_attn_noalloc_flags.restype = I
        lib.verify_attn_noalloc.restype = I
        lib.verify_attn_kv_append.argtypes = [P, P, I, I, I, I, I, P, P, P, P, P, I, P, I, P, P]
        lib.verify_attn_kv_append.restype = I
        lib.verify_attn_lookup_draft.argtypes = [P, I, P, I, I, I, I, P, P, P, P, P]
        lib.verify_attn_lookup_draft.restype = I
        lib.verify_attn_accept_workspace_bytes.argtypes = [I, I]
        lib.verify_attn_accept_workspace_bytes.restype = ctypes.c_size_t
        lib.verify_attn_accept.argtypes = [P, P, P, P, I, I, I, ctypes.c_uint64, P, P, P, P]
        lib.verify_attn_accept.restype = I
        lib.verify_attn_validate_host.argtypes = [P, I, I, P, I, I, ctypes.POINTER(I), ctypes.POINTER(I)]
        lib.verify_attn_validate_host.restype = I
        lib.verify_attn_rope_init.argtypes = [P, P, P, I, I, I, ctypes.c_float]
        H, S, R = ctypes.POINTER(_Heads), ctypes.POINTER(_Positions), ctypes.POINTER(_Rows)
        lib.verify_attn_rope.argtypes = [P, S, I, I, I, I, H, H, H, H, I, P]
        lib.verify_attn_rope_append.argtypes = [P, S, I, I, I, H, P, H, H, I, P, P, P, P, P, I, P, I, P, P]
        lib.verify_attn_accept_probs.argtypes = [R, R, I, P, P, P, P, I, I, I, P, P, P]
        lib.verify_attn_pages_workspace_bytes.argtypes = [I, I]
        lib.verify_attn_pages_workspace_bytes.restype = ctypes.c_size_t
        lib.verify_attn_pages_resize.argtypes = [P, P, P]
        lib.verify_attn_pages_resize_ex.argtypes = [P, P, P, P]
        lib.verify_attn_pages_fork.argtypes = [P, P, P, P, I, I, P]
        lib.verify_attn_pages_compact.argtypes = [P, P]
        lib.verify_attn_chunk_plan.argtypes = [P, P, I, I, I, I, I, I, ctypes.POINTER(P)]
        lib.verify_attn_chunk_plan_describe.argtypes = [P, P, I, I, I, I, I, I, ctypes.POINTER(ChunkPlanInfo), P, I]
        lib.verify_attn_chunk_plan_describe.restype = I
        lib.verify_attn_chunk_plan_destroy.argtypes = [P]
        lib.verify_attn_chunk_plan_destroy.restype = None
        lib.verify_attn_chunk_plan_get_info.argtypes = [P, ctypes.POINTER(ChunkPlanInfo)]
        lib.verify_attn_chunk_plan_device_flags.argtypes = [P, I, ctypes.POINTER(I), P]
        lib.verify_attn_chunk.argtypes = [P, H, P, P, P, P, P, I, I, P, P, P]
        lib.verify_attn_chunk_weights.argtypes = [P, H, P, P, P, I, I, P, P, ctypes.c_int64, ctypes.c_int64, I, P, P, P]
        lib.verify_attn_logprobs.argtypes = [P, ctypes.c_int64, I, P, I, I, I, P, P, P, P, P, P]
        lib.verify_attn_evict_workspace_bytes.argtypes = [I, I, I]
        lib.verify_attn_evict_workspace_bytes.restype = ctypes.c_size_t
        lib.verify_attn_evict.argtypes = [P, P, P, P, I, P, I, P, I, I, I, I, P, P, ctypes.c_int64, ctypes.c_int64, I, P, I,
                                          P, P, P, P, P, P]
        for f in ("verify_attn_chunk_plan", "verify_attn_chunk_plan_get_info", "verify_attn_chunk_plan_device_flags",
                  "verify_attn_chunk", "verify_attn_chunk_weights", "verify_attn_logprobs", "verify_attn_evict"):
            getattr(lib, f).restype = I
        for f in ("verify_attn_rope_init", "verify_attn_rope", "verify_attn_rope_append", "verify_attn_accept_probs",
                  "verify_attn_pages_resize", "verify_attn_pages_resize_ex", "verify_attn_pages_fork",
                  "verify_attn_pages_compact"):
            getattr(lib, f).restype = I
        for f in ("verify_attn_plan", "verify_attn_plan_ex", "verify_attn", "verify_attn_with_plan",
                  "verify_attn_plan_get_info", "verify_attn_plan_describe", "verify_attn_plan_device_flags"):
            getattr(lib, f).restype = I
        _lib = lib
        return lib


def library():
    """The loaded ctypes library (raises if it is not built)."""
    return _load()


def verify_attn_status_string(status: int) -> str:
    return _load().verify_attn_status_string(int(status)).decode()


def _check(rc, what):
    if rc != 0:
        raise VerifyAttnError(rc, what)


def _dtype_code(kv_dtype):
    return KV_DTYPE_CODES[kv_dtype] if isinstance(kv_dtype, str) else int(kv_dtype)


def _options(block_table_stride=0, tokens_per_split=0, path="auto", num_pages=0):
    return _Options(int(block_table_stride), int(tokens_per_split),
                    PATH_CODES[path] if isinstance(path, str) else int(path), int(num_pages))


_current = threading.local()  # .table: rows and stride of the table of this thread's current plan


def _host_lens(seq_lens):
    try:
        import torch
        if isinstance(seq_lens, torch.Tensor):
            seq_lens = seq_lens.detach().cpu().numpy()
    except ImportError:  # pragma: no cover
        pass
    lens = np.asarray(seq_lens)
    if lens.size and not (-2 ** 31 <= lens.min() and lens.max() < 2 ** 31):
        raise ValueError(f"lengths between {lens.min()} and {lens.max()} are past 32 bits")
    return np.ascontiguousarray(lens.astype(np.int32, copy=False).reshape(-1))


def _table_stride(lens, stride):
    """Entries between a block table's rows: as given, or the longest sequence's pages."""
    return int(stride) if stride > 0 else (int(lens.max(initial=0)) + PAGE_SIZE - 1) // PAGE_SIZE


def _check_table(block_table, num_seqs, stride):
    """The kernels step through the table by ``stride``; of one sequence a wider row will do.  (A table that is not
    [num_seqs, stride] is taken as it lies.)"""
    n = getattr(block_table, "shape", ())
    if len(n) == 2 and (n[0] < num_seqs or n[1] < stride or (n[1] != stride and num_seqs > 1)):
        raise ValueError(f"block_table is {list(n)}, the call goes by [{num_seqs}, {stride}]: give its width as block_table_stride")


class Plan:
    """Owning handle of a ``va_plan`` (freed on ``destroy()`` or collection)."""

    def __init__(self, handle, seq_lens, T, kv_dtype, block_table_stride=0):
        self._h = ctypes.c_void_p(handle)
        self.seq_lens = seq_lens
        self.T = T
        self.kv_dtype = kv_dtype
        self.block_table_stride = _table_stride(seq_lens, block_table_stride)

    @property
    def handle(self):
        return self._h

    def info(self) -> dict:
        return verify_attn_plan_get_info(self)

    def destroy(self):
        if self._h and self._h.value:
            _load().verify_attn_plan_destroy(self._h)
            self._h = ctypes.c_void_p(0)

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def verify_attn_plan(seq_lens, T, num_q_heads, num_kv_heads, head_dim, kv_dtype, num_sms=0,
                     **options) -> Plan:
    """Plan one batch shape from the host ``seq_lens`` (lengths include the T
    verify tokens).  Keyword options: block_table_stride, tokens_per_split,
    path ("auto" | "warp" | "mma"), num_pages (enables device bound checks).
    The new plan also becomes this thread's current plan for ``verify_attn``."""
    lib = _load()
    lens = _host_lens(seq_lens)
    out = ctypes.c_void_p()
    opts = _options(**options)
    rc = lib.verify_attn_plan_ex(lens.ctypes.data_as(ctypes.c_void_p), len(lens), int(T), int(num_q_heads),
                                 int(num_kv_heads), int(head_dim), _dtype_code(kv_dtype), int(num_sms),
                                 ctypes.byref(opts), ctypes.byref(out))
    _check(rc, "verify_attn_plan")
    plan = Plan(out.value, lens, int(T), _dtype_code(kv_dtype), opts.block_table_stride)
    _current.table = len(lens), plan.block_table_stride
    return plan


def verify_attn_plan_destroy(plan: Plan):
    plan.destroy()


def verify_attn_validate_host(seq_lens, T, block_table, num_pages):
    """Host check of the paging inputs (no GPU needed).  Returns None when
    they are valid, else (sequence, block index or -1) of the first fault."""
    lens = _host_lens(seq_lens)
    try:
        import torch
        if isinstance(block_table, torch.Tensor):
            block_table = block_table.detach().cpu().numpy()
    except ImportError:  # pragma: no cover
        pass
    bt = np.ascontiguousarray(np.asarray(block_table, dtype=np.int32))
    if bt.ndim != 2 or bt.shape[0] != len(lens):
        raise ValueError("block_table must be [num_seqs, stride]")
    bad_seq, bad_block = ctypes.c_int(-1), ctypes.c_int(-1)
    rc = _load().verify_attn_validate_host(lens.ctypes.data_as(ctypes.c_void_p), len(lens), int(T),
                                           bt.ctypes.data_as(ctypes.c_void_p), bt.shape[1], int(num_pages),
                                           ctypes.byref(bad_seq), ctypes.byref(bad_block))
    if rc == 0:
        return None
    if bad_seq.value < 0:
        _check(rc, "verify_attn_validate_host")
    return bad_seq.value, bad_block.value


def verify_attn_plan_get_info(plan: Plan) -> dict:
    info = PlanInfo()
    _check(_load().verify_attn_plan_get_info(plan.handle, ctypes.byref(info)), "verify_attn_plan_get_info")
    return info.as_dict()


def verify_attn_plan_describe(seq_lens, T, num_q_heads, num_kv_heads, head_dim, kv_dtype, num_sms,
                              max_items=None, **options):
    """Host-only planning (no GPU needed): (info dict, items int32 [n, 5])
    with items = (seq, kv_head, row_group, key_begin, key_end)."""
    lib = _load()
    lens = _host_lens(seq_lens)
    opts = _options(**options)
    info = PlanInfo()
    rc = lib.verify_attn_plan_describe(lens.ctypes.data_as(ctypes.c_void_p), len(lens), int(T),
                                       int(num_q_heads), int(num_kv_heads), int(head_dim),
                                       _dtype_code(kv_dtype), int(num_sms), ctypes.byref(opts),
                                       ctypes.byref(info), None, 0)
    _check(rc, "verify_attn_plan_describe")
    n = info.num_items if max_items is None else min(int(max_items), info.num_items)
    items = np.zeros((max(n, 1), 5), np.int32)
    rc = lib.verify_attn_plan_describe(lens.ctypes.data_as(ctypes.c_void_p), len(lens), int(T),
                                       int(num_q_heads), int(num_kv_heads), int(head_dim),
                                       _dtype_code(kv_dtype), int(num_sms), ctypes.byref(opts),
                                       ctypes.byref(info), items.ctypes.data_as(ctypes.c_void_p), n)
    _check(rc, "verify_attn_plan_describe")
    return info.as_dict(), items[:n]


_INT_MAX = 0x7FFFFFFF  # ctypes cuts a larger size to its low 32 bits


def _too_large(what, shape):
    return ValueError(f"{what}: {list(shape)} has a size past 32 bits")


def _dev_ptr(t, name, dtypes, allow_none=False):
    import torch
    if t is None:
        if allow_none:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _kv_dtypes(code):
    import torch
    if code == VA_BF16:
        return (torch.bfloat16, torch.int16, torch.uint16) if hasattr(torch, "uint16") else (torch.bfloat16, torch.int16)
    if code == VA_FP8_E4M3:
        return (torch.uint8, torch.float8_e4m3fn)
    if code in (VA_INT4, VA_INT2):  # packed bytes
        return (torch.uint8, torch.int8)
    return (torch.int8,)


def _marshal(kv_code, q, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, out, lse, stream):
    import torch
    q16 = (torch.bfloat16, torch.int16)
    kvd = _kv_dtypes(kv_code)
    args = [
        _dev_ptr(q, "q", q16),
        _dev_ptr(k_pages, "k_pages", kvd),
        _dev_ptr(v_pages, "v_pages", kvd),
        _dev_ptr(k_scale, "k_scale", (torch.float32,), allow_none=kv_code == VA_BF16),
        _dev_ptr(v_scale, "v_scale", (torch.float32,), allow_none=kv_code == VA_BF16),
        _dev_ptr(block_table, "block_table", (torch.int32,)),
        _dev_ptr(seq_lens, "seq_lens", (torch.int32,)),
    ]
    tail = [_dev_ptr(out, "out", q16), _dev_ptr(lse, "lse", (torch.float32,), allow_none=True)]
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    s = ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))
    return args, tail, s


def verify_attn_with_plan(plan: Plan, q, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, T,
                          out, lse=None, stream=None):
    """Enqueue verify attention with an explicit plan on ``stream`` (default:
    torch's current stream).  Writes ``out`` (and ``lse`` if given)."""
    _check_table(block_table, len(plan.seq_lens), plan.block_table_stride)
    args, tail, s = _marshal(plan.kv_dtype, q, k_pages, v_pages, k_scale, v_scale, block_table,
                             seq_lens, out, lse, stream)
    _check(_load().verify_attn_with_plan(plan.handle, *args, int(T), *tail, s), "verify_attn_with_plan")


def verify_attn(q, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, T, out, lse=None,
                stream=None, kv_dtype=None):
    """Enqueue verify attention with this thread's current plan.  ``kv_dtype``
    only selects the accepted tensor dtypes for marshalling (inferred from
    ``k_pages`` when omitted: a byte cache whose rows are D / 2 or D / 4 bytes
    long is the 4-bit or 2-bit one)."""
    import torch
    if kv_dtype is None:
        kv_code = {torch.int8: VA_INT8, torch.uint8: VA_FP8_E4M3,
                   torch.float8_e4m3fn: VA_FP8_E4M3}.get(k_pages.dtype, VA_BF16)
        if kv_code != VA_BF16 and k_pages.dim() == 4:
            D = q.shape[-1]
            kv_code = {D // 2: VA_INT4, D // 4: VA_INT2}.get(k_pages.shape[-1], kv_code)
    else:
        kv_code = _dtype_code(kv_dtype)
    table = getattr(_current, "table", None)
    if table is not None:
        _check_table(block_table, *table)
    args, tail, s = _marshal(kv_code, q, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens,
                             out, lse, stream)
    _check(_load().verify_attn(*args, int(T), *tail, s), "verify_attn")


def verify_attn_plan_device_flags(plan: Plan, clear=True, stream=None) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    flags = ctypes.c_int(0)
    _check(_load().verify_attn_plan_device_flags(plan.handle, int(bool(clear)), ctypes.byref(flags),
                                                 ctypes.c_void_p(stream.cuda_stream)),
           "verify_attn_plan_device_flags")
    return flags.value


def verify_attn_plan_set_events(plan: Plan, ev_before=None, ev_after=None):
    """Record two torch.cuda.Event objects around the partial-attention
    kernel of every later call with ``plan`` (None, None stops)."""
    b = ctypes.c_void_p(ev_before.cuda_event) if ev_before is not None else None
    a = ctypes.c_void_p(ev_after.cuda_event) if ev_after is not None else None
    _check(_load().verify_attn_plan_set_events(plan.handle, b, a), "verify_attn_plan_set_events")


def verify_attn_noalloc(seq_lens_host, T, num_q_heads, num_kv_heads, head_dim, kv_dtype, q, k_pages,
                        v_pages, k_scale, v_scale, block_table, seq_lens, out, lse=None,
                        block_table_stride=0, num_pages=0, stream=None):
    """Verify attention that allocates no device memory: plans from the host
    ``seq_lens_host`` on every call and keeps its scratch in the library's
    static device array (see ``include/verify_attn.h``).  For callers that
    cannot call cudaMalloc.  Calls share that array, so order them on one
    stream; not for CUDA-graph capture.  ``num_pages`` > 0 checks every
    block-table entry (bad ones are skipped and flagged, see
    ``verify_attn_noalloc_flags``)."""
    lens = _host_lens(seq_lens_host)
    code = _dtype_code(kv_dtype)
    _check_table(block_table, len(lens), _table_stride(lens, block_table_stride))
    args, tail, s = _marshal(code, q, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, out, lse,
                             stream)
    rc = _load().verify_attn_noalloc(lens.ctypes.data_as(ctypes.c_void_p), len(lens), int(T), int(num_q_heads),
                                     int(num_kv_heads), int(head_dim), code, *args[:6],
                                     int(block_table_stride), int(num_pages), args[6], *tail, s)
    _check(rc, "verify_attn_noalloc")


def verify_attn_noalloc_flags(clear=True, stream=None):
    """Flag word of the last verify_attn_noalloc call on the current device
    (same bits as verify_attn_plan_device_flags); clears it by default."""
    import torch
    stream = stream or torch.cuda.current_stream()
    flags = ctypes.c_int(0)
    _check(_load().verify_attn_noalloc_flags(int(bool(clear)), ctypes.byref(flags),
                                             ctypes.c_void_p(stream.cuda_stream)), "verify_attn_noalloc_flags")
    return flags.value


def verify_attn_kv_append(k_new, v_new, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, T,
                          kv_dtype, num_pages=0, flags=None, stream=None):
    """KV append with quantise-on-write: store the T new tokens' K and V rows
    (bf16 ``[B, T, Hkv, D]``) at positions ``seq_lens[b] - T + t`` of the paged
    cache, quantised per (token, kv head) for fp8 / int8 caches (definition in
    ``include/verify_attn.h``).  ``flags`` is an optional int32 device tensor
    into which bit 0 is ORed for a skipped row."""
    import torch
    code = _dtype_code(kv_dtype)
    B, T_, Hkv, D = k_new.shape
    if int(T) != T_ or tuple(v_new.shape) != tuple(k_new.shape):
        raise ValueError("k_new and v_new must both be [B, T, Hkv, D] with the given T")
    if B | T_ | Hkv | D | block_table.shape[1] > _INT_MAX:
        raise _too_large("k_new or block_table", (*k_new.shape, block_table.shape[1]))
    q16 = (torch.bfloat16, torch.int16)
    kvd = _kv_dtypes(code)
    ptrs = [_dev_ptr(k_new, "k_new", q16), _dev_ptr(v_new, "v_new", q16)]
    cache = [_dev_ptr(k_pages, "k_pages", kvd), _dev_ptr(v_pages, "v_pages", kvd),
             _dev_ptr(k_scale, "k_scale", (torch.float32,), allow_none=code == VA_BF16),
             _dev_ptr(v_scale, "v_scale", (torch.float32,), allow_none=code == VA_BF16)]
    bt = _dev_ptr(block_table, "block_table", (torch.int32,))
    sl = _dev_ptr(seq_lens, "seq_lens", (torch.int32,))
    fl = _dev_ptr(flags, "flags", (torch.int32,), allow_none=True)
    if stream is None:
        stream = torch.cuda.current_stream(k_new.device)
    st = ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))
    rc = _load().verify_attn_kv_append(*ptrs, int(B), int(T), int(Hkv), int(D), code, *cache, bt,
                                       int(block_table.shape[1]), sl, int(num_pages), fl, st)
    _check(rc, "verify_attn_kv_append")


def verify_attn_lookup_draft(tokens, lens, num_draft, min_match=6, max_match=12, match_end=None,
                            match_len=None, stream=None):
    """Lookup-augmented drafting over token histories ``tokens`` (int32 CUDA
    tensor ``[num_seqs, stride]``, the first ``lens[b]`` entries valid): the
    most recent earlier occurrence of each history's last tokens (longest
    match first, ``min_match``..``max_match``) and up to ``num_draft`` tokens
    that followed it.  Returns (draft int32 ``[num_seqs, num_draft]``, -1 past
    the proposal, draft_len int32 ``[num_seqs]``); ``match_end`` /
    ``match_len`` (int32 ``[num_seqs]``) are filled when given."""
    import torch
    if tokens.dim() != 2:
        raise ValueError("tokens must be [num_seqs, stride]")
    B, stride = tokens.shape
    if B | stride > _INT_MAX:
        raise _too_large("tokens", tokens.shape)
    i32 = (torch.int32,)
    tp = _dev_ptr(tokens, "tokens", i32)
    lp = _dev_ptr(lens, "lens", i32)
    me = _dev_ptr(match_end, "match_end", i32, allow_none=True)
    ml = _dev_ptr(match_len, "match_len", i32, allow_none=True)
    st, guard = _launch_on(tokens.device, stream)
    with guard:
        draft = torch.empty((B, int(num_draft)), dtype=torch.int32, device=tokens.device)
        dlen = torch.empty((B,), dtype=torch.int32, device=tokens.device)
        rc = _load().verify_attn_lookup_draft(tp, int(stride), lp, int(B), int(min_match), int(max_match),
                                              int(num_draft), ctypes.c_void_p(draft.data_ptr()),
                                              ctypes.c_void_p(dlen.data_ptr()), me, ml, st)
    _check(rc, "verify_attn_lookup_draft")
    return draft, dlen


def verify_attn_accept(target_logits, draft_tokens, temperature, seed, draft_logits=None, stream=None):
    """Speculative acceptance (rejection sampler) after the verify pass:
    ``target_logits`` fp32 ``[B, T+1, V]``, ``draft_tokens`` int32 ``[B, T]``,
    ``temperature`` fp32 ``[B]`` (<= 0: greedy), ``draft_logits`` fp32
    ``[B, T, V]`` or None (a point-mass proposal, as for lookup drafts), all
    CUDA tensors; ``seed`` picks the Philox stream.  Returns (out_tokens int32
    ``[B, T+1]`` with -1 after the emitted token, num_accepted int32 ``[B]``)."""
    import torch
    if target_logits.dim() != 3 or draft_tokens.dim() != 2:
        raise ValueError("target_logits must be [B, T+1, V] and draft_tokens [B, T]")
    B, T1, V = target_logits.shape
    if B | T1 | V > _INT_MAX:
        raise _too_large("target_logits", target_logits.shape)
    T = T1 - 1
    if tuple(draft_tokens.shape) != (B, T):
        raise ValueError("draft_tokens must be [B, T]")
    if draft_logits is not None and tuple(draft_logits.shape) != (B, T, V):
        raise ValueError("draft_logits must be [B, T, V]")
    f32, i32 = (torch.float32,), (torch.int32,)
    zp = _dev_ptr(target_logits, "target_logits", f32)
    wp = _dev_ptr(draft_logits, "draft_logits", f32, allow_none=True)
    dp = _dev_ptr(draft_tokens, "draft_tokens", i32)
    tp = _dev_ptr(temperature, "temperature", f32)
    lib = _load()
    st, guard = _launch_on(target_logits.device, stream)
    with guard:
        ws = torch.empty(max(16, int(lib.verify_attn_accept_workspace_bytes(int(B), int(T)))), dtype=torch.uint8,
                         device=target_logits.device)
        out = torch.empty((B, T1), dtype=torch.int32, device=target_logits.device)
        nacc = torch.empty((B,), dtype=torch.int32, device=target_logits.device)
        rc = lib.verify_attn_accept(zp, wp, dp, tp, int(B), int(T), int(V), int(seed) & 0xFFFFFFFFFFFFFFFF,
                                    ctypes.c_void_p(ws.data_ptr()), ctypes.c_void_p(out.data_ptr()),
                                    ctypes.c_void_p(nacc.data_ptr()), st)
    _check(rc, "verify_attn_accept")
    return out, nacc


_here = contextlib.nullcontext()
_torch = None


def _bind_torch():
    """What the calls below need of torch, looked up once: a call's checks and marshalling are most of
    its cost on small batches."""
    global _torch, _FLOAT_CODES, _CACHE_TYPES, _raw_stream, _current_device, _grad_mode
    import torch
    _FLOAT_CODES = {torch.bfloat16: VA_FLOAT_BF16, torch.float16: VA_FLOAT_FP16, torch.float32: VA_FLOAT_FP32}
    _CACHE_TYPES = {code: _kv_dtypes(code) for code in KV_DTYPE_CODES.values()}
    # the current stream's handle without a Stream object around it, where torch offers that
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)
    _current_device = torch.cuda.current_device
    _grad_mode = torch.is_grad_enabled
    _torch = torch
    return torch


def _float_code(t, name):
    code = _FLOAT_CODES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} has dtype {t.dtype}, expected bfloat16, float16 or float32")
    return code


def _launch_on(device, stream):
    """(stream handle, guard): a call runs on the tensors' device and on ``stream`` there (a
    torch stream or a raw handle; default: torch's current stream of that device).  What the
    call allocates is allocated inside the guard, so it belongs to that stream."""
    torch = _torch or _bind_torch()
    if stream is None:
        index = device.index
        return _raw_stream(index), _here if _current_device() == index else torch.cuda.device(device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    elif stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
    return stream.cuda_stream, torch.cuda.stream(stream)


def _device_of(t, name):
    """The device of a CUDA tensor and its index."""
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"{name} must be a CUDA tensor")
    device = t.device
    return device, device.index


def _ptr(t, name, dtype, index, shape=None):
    """Address of a contiguous tensor of that type (and shape) on CUDA device ``index``."""
    try:
        if (t.dtype is dtype and t.get_device() == index and t.is_contiguous()
                and (shape is None or t.shape == shape)):
            return t.data_ptr()
    except AttributeError:
        raise ValueError(f"{name} must be a CUDA tensor") from None
    want = "" if shape is None else f" of shape {list(shape)}"
    raise ValueError(f"{name} must be a contiguous {dtype} tensor{want} on cuda:{index}, "
                     f"got {t.dtype} {list(t.shape)} on {t.device}")


def _ptr_of(t, name, dtypes, index):
    """``_ptr`` of a tensor that may have one of several types."""
    dtype = getattr(t, "dtype", None)
    if dtype not in dtypes:
        raise ValueError(f"{name} has dtype {dtype}, expected one of {dtypes}")
    return _ptr(t, name, dtype, index)


def _heads(t, name, dtype, index, shape=None):
    """A [B, T, H, D] tensor, any strides but a contiguous last dimension, as a ``va_heads``."""
    try:
        n, s = t.shape, t.stride()
        if (t.dtype is dtype and t.get_device() == index and len(n) == 4 and (s[3] == 1 or n[3] <= 1)
                and (shape is None or n == shape)):
            if n[0] | n[1] | n[2] | n[3] > _INT_MAX:
                raise _too_large(name, n)
            return _Heads(t.data_ptr(), s[0], s[1], s[2], n[2])
    except AttributeError:
        raise ValueError(f"{name} must be a CUDA tensor") from None
    want = "[B, T, H, D]" if shape is None else list(shape)
    raise ValueError(f"{name} must be a {dtype} tensor {want} on cuda:{index}, contiguous in its last dimension, "
                     f"got {t.dtype} {list(n)} with strides {list(s)} on {t.device}")


def _positions(t, rope, B, T, index):
    shape = (rope._struct.num_axes, B, T)
    try:
        if t.dtype is _torch.int32 and t.get_device() == index and t.shape == shape:
            s = t.stride()
            return _Positions(t.data_ptr(), s[0], s[1], s[2])
    except AttributeError:
        pass
    raise ValueError(f"positions must be an int32 tensor {list(shape)} on cuda:{index}")


def _wants_gradient(t):
    return getattr(t, "requires_grad", False)


def _gradient_lost(what):
    """The error in place of a result without its gradient."""
    return ValueError(f"{what} is not recorded by autograd and would lose its inputs' gradient: call it under "
                      "torch.no_grad(), on detached tensors, or in a torch.autograd.Function whose backward rotates "
                      "with inverse=True")


def _gradient_refused(what):
    return ValueError(f"{what} is not recorded by autograd and would lose its inputs' gradient: call it under "
                      "torch.no_grad() or on detached tensors")


class Rope:
    """A rotation (``va_rope``): host data, made by ``verify_attn_rope_spec``."""

    def __init__(self, struct):
        self._struct = struct
        self._ref = ctypes.byref(struct)

    num_pairs = property(lambda self: self._struct.num_pairs)
    num_axes = property(lambda self: self._struct.num_axes)
    axis = property(lambda self: list(self._struct.axis[:self._struct.num_pairs]))


def verify_attn_rope_spec(rotary_dim, base=1.0e6, inv_freq=None, sections=None, layout="blocked", pairing="half",
                          scale=1.0) -> Rope:
    """Describe a rotation of the first ``rotary_dim`` elements of each head.
    ``inv_freq``: the ``rotary_dim / 2`` frequencies (default ``base ** (-i /
    pairs)``).  ``sections``: how many pairs turn by each axis's position
    (default: all by one axis); ``layout`` "blocked" puts the axes' pairs one
    after the other, "dealt" deals pairs round to the axes that have some
    left.  ``pairing`` "half" pairs element i with i + rotary_dim / 2,
    "adjacent" 2 i with 2 i + 1.  ``scale`` multiplies the rotated elements."""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and at least 2")
    pairs = int(rotary_dim) // 2
    if pairs > ROPE_MAX_PAIRS:
        raise ValueError(f"rotary_dim must be at most {2 * ROPE_MAX_PAIRS}")
    if inv_freq is None:
        inv_freq = float(base) ** (-np.arange(pairs, dtype=np.float64) / pairs)
    freq = np.ascontiguousarray(np.asarray(inv_freq, np.float64).reshape(-1))
    if freq.size != pairs:
        raise ValueError(f"inv_freq must have {pairs} entries")
    sections = [pairs] if sections is None else [int(n) for n in sections]
    if not 1 <= len(sections) <= ROPE_MAX_AXES or min(sections) < 0 or sum(sections) != pairs:
        raise ValueError(f"sections must be 1 to {ROPE_MAX_AXES} counts that sum to {pairs}")
    if layout not in ("blocked", "dealt") or pairing not in ("half", "adjacent"):
        raise ValueError("layout is 'blocked' or 'dealt', pairing 'half' or 'adjacent'")
    if layout == "blocked":
        axis = [a for a, n in enumerate(sections) for _ in range(n)]
    else:
        left, axis = list(sections), []
        while any(left):
            for a, n in enumerate(left):
                if n:
                    left[a] -= 1
                    axis.append(a)
    axis = np.asarray(axis, np.int32)
    r = _Rope()
    _check(_load().verify_attn_rope_init(ctypes.byref(r), freq.ctypes.data, axis.ctypes.data, pairs, len(sections),
                                         int(pairing == "adjacent"), float(scale)), "verify_attn_rope_spec")
    return Rope(r)


def verify_attn_rope(rope: Rope, positions, q, k=None, q_out=None, k_out=None, inverse=False, stream=None):
    """Rotate ``q`` and ``k`` (``[B, T, H, D]`` bf16, fp16 or fp32, any strides
    with a contiguous last dimension) by ``positions`` (int32 ``[axes, B, T]``,
    any strides).  ``q_out`` / ``k_out`` default to new contiguous tensors; pass
    ``q`` / ``k`` themselves to work in place, otherwise outputs must not overlap
    inputs.  ``inverse=True`` rotates back, which is also the way of the gradient:
    a ``torch.autograd.Function`` calls this in its forward and, with
    ``inverse=True`` on the outputs' gradients, in its backward.  The call itself
    is not recorded by autograd, and in grad mode tensors that require a gradient
    are refused.  Returns (q_out, k_out), k_out None without ``k``."""
    torch = _torch or _bind_torch()
    if _grad_mode() and (_wants_gradient(q) or _wants_gradient(k) or _wants_gradient(q_out) or _wants_gradient(k_out)):
        raise _gradient_lost("verify_attn_rope")
    device, index = _device_of(q, "q")
    code = _float_code(q, "q")
    dtype = q.dtype
    hq = _heads(q, "q", dtype, index)
    B, T, _, D = n = q.shape
    hk = None
    if k is not None:
        hk = _heads(k, "k", dtype, index)
        nk = k.shape
        if nk[0] != B or nk[1] != T or nk[3] != D:
            raise ValueError(f"k must be [{B}, {T}, heads, {D}], got {list(nk)}")
    elif k_out is not None:
        raise ValueError("k_out without k")
    pos = _positions(positions, rope, B, T, index)
    st, guard = _launch_on(device, stream)
    with guard:
        if q_out is None:
            q_out = torch.empty(n, dtype=dtype, device=device)
        oq, ok = _heads(q_out, "q_out", dtype, index, n), None
        if k is not None:
            if k_out is None:
                k_out = torch.empty(nk, dtype=dtype, device=device)
            ok = _heads(k_out, "k_out", dtype, index, nk)
        rc = (_lib or _load()).verify_attn_rope(rope._ref, pos, code, B, T, D, hq, oq, hk, ok, 1 if inverse else 0, st)
    if rc:
        _check(rc, "verify_attn_rope")
    return q_out, k_out


def verify_attn_rope_append(rope: Rope, positions, q, k_new, v_new, k_pages, v_pages, k_scale, v_scale, block_table,
                            seq_lens, kv_dtype, q_out=None, num_pages=0, flags=None, stream=None):
    """Rotate ``q`` and ``k_new`` and append ``k_new`` / ``v_new`` to the paged
    cache in one launch (``[B, T, heads, D]`` bf16, any strides with a
    contiguous last dimension, for instance slices of a fused projection).
    Cache arguments, ``num_pages`` and ``flags`` as for
    ``verify_attn_kv_append``; the cache gets the rotated keys, quantised from
    their unrounded values.  ``positions`` None: every axis is the token's
    place in its sequence, ``seq_lens[b] - T + t``.  ``q`` may be None.  Not
    recorded by autograd: in grad mode tensors that require a gradient are
    refused.  Returns the rotated q, contiguous bf16."""
    torch = _torch or _bind_torch()
    if _grad_mode() and (_wants_gradient(q) or _wants_gradient(k_new) or _wants_gradient(v_new) or _wants_gradient(q_out)):
        raise _gradient_lost("verify_attn_rope_append")
    code = _dtype_code(kv_dtype)
    device, index = _device_of(k_new, "k_new")
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    hk = _heads(k_new, "k_new", bf16, index)
    B, T, Hkv, D = n = k_new.shape
    hv = _heads(v_new, "v_new", bf16, index, n)
    hq = None
    if q is not None:
        hq = _heads(q, "q", bf16, index)
        nq = q.shape
        if nq[0] != B or nq[1] != T or nq[3] != D:
            raise ValueError(f"q must be [{B}, {T}, heads, {D}], got {list(nq)}")
    elif q_out is not None:
        raise ValueError("q_out without q")
    pos = None if positions is None else _positions(positions, rope, B, T, index)
    kvd = _CACHE_TYPES.get(code, ())
    kp, vp = _ptr_of(k_pages, "k_pages", kvd, index), _ptr_of(v_pages, "v_pages", kvd, index)
    pages = k_pages.shape[0] if k_pages.dim() else 0
    cache = (pages, PAGE_SIZE, Hkv, D // 2 if code == VA_INT4 else D // 4 if code == VA_INT2 else D)
    if k_pages.shape != cache or v_pages.shape != cache:
        raise ValueError(f"k_pages and v_pages must be [num_pages, {PAGE_SIZE}, {Hkv}, {cache[3]}], got "
                         f"{list(k_pages.shape)} and {list(v_pages.shape)}")
    if num_pages > pages:
        raise ValueError(f"num_pages is {num_pages}, the cache has {pages}")
    ks = vs = None
    if code != VA_BF16:
        ks, vs = _ptr(k_scale, "k_scale", f32, index, cache[:3]), _ptr(v_scale, "v_scale", f32, index, cache[:3])
    bt, sl = _ptr(block_table, "block_table", i32, index), _ptr(seq_lens, "seq_lens", i32, index, (B,))
    nt = block_table.shape
    if len(nt) != 2 or nt[0] != B:
        raise ValueError(f"block_table must be [{B}, stride], got {list(nt)}")
    if nt[1] | pages > _INT_MAX:
        raise _too_large("block_table or k_pages", (nt[1], pages))
    fl = None if flags is None else _ptr(flags, "flags", i32, index)
    st, guard = _launch_on(device, stream)
    with guard:
        oq = None
        if q is not None:
            if q_out is None:
                q_out = torch.empty(nq, dtype=bf16, device=device)
            oq = _ptr(q_out, "q_out", bf16, index, nq)
        rc = (_lib or _load()).verify_attn_rope_append(
            rope._ref, pos, B, T, D, hq, oq, hk, hv, code, kp, vp, ks, vs, bt, nt[1], sl,
            num_pages or pages, fl, st)
    if rc:
        _check(rc, "verify_attn_rope_append")
    return q_out


def verify_attn_accept_probs(target_probs, draft_tokens, u_accept, u_emit, draft_probs=None, draft_lens=None,
                             out_tokens=None, num_accepted=None, stream=None):
    """Speculative acceptance from given probabilities and random numbers:
    ``target_probs`` ``[B, T+1, V]`` and ``draft_probs`` ``[B, T, V]`` (None: point-mass
    proposals) of one type (fp32, bf16 or fp16; any strides with a contiguous
    last dimension, for instance padded vocabularies), ``draft_tokens`` int32 ``[B,
    T]``, ``draft_lens`` int32 ``[B]`` (None: T each), uniforms ``u_accept`` fp32
    ``[B, T]`` (one per draft) and ``u_emit`` fp32 ``[B]`` (for the emitted
    token).  Definition in ``include/verify_attn.h``.  Returns (out_tokens int32
    ``[B, T+1]`` with -1 after the emitted token, num_accepted int32 ``[B]``)."""
    torch = _torch or _bind_torch()
    f32, i32 = torch.float32, torch.int32
    device, index = _device_of(target_probs, "target_probs")
    code = _float_code(target_probs, "target_probs")
    dtype, n = target_probs.dtype, target_probs.shape
    if len(n) != 3 or n[1] < 1:
        raise ValueError("target_probs must be [B, T+1, V]")
    B, T1, V = n
    if B | T1 | V > _INT_MAX:
        raise _too_large("target_probs", n)
    T = T1 - 1
    p = _prob_rows(target_probs, "target_probs", dtype, index, n)
    q = d = ua = None
    if T:
        if draft_probs is not None:
            q = _prob_rows(draft_probs, "draft_probs", dtype, index, (B, T, V))
        d, ua = _ptr(draft_tokens, "draft_tokens", i32, index, (B, T)), _ptr(u_accept, "u_accept", f32, index, (B, T))
    ue = _ptr(u_emit, "u_emit", f32, index, (B,))
    dl = None if draft_lens is None else _ptr(draft_lens, "draft_lens", i32, index, (B,))
    st, guard = _launch_on(device, stream)
    with guard:
        if out_tokens is None:
            out_tokens = torch.empty((B, T1), dtype=i32, device=device)
        if num_accepted is None:
            num_accepted = torch.empty((B,), dtype=i32, device=device)
        ot, na = _ptr(out_tokens, "out_tokens", i32, index, (B, T1)), _ptr(num_accepted, "num_accepted", i32, index, (B,))
        rc = (_lib or _load()).verify_attn_accept_probs(p, q, code, d, dl, ua, ue, B, T, V, ot, na, st)
    if rc:
        _check(rc, "verify_attn_accept_probs")
    return out_tokens, num_accepted


def _prob_rows(t, name, dtype, index, shape):
    """A [B, positions, V] tensor, any strides but a contiguous last dimension, as a ``va_rows``."""
    try:
        s = t.stride()
        if t.dtype is dtype and t.get_device() == index and t.shape == shape and (s[2] == 1 or shape[2] <= 1):
            return _Rows(t.data_ptr(), s[0], s[1])
    except AttributeError:
        raise ValueError(f"{name} must be a CUDA tensor") from None
    raise ValueError(f"{name} must be a {dtype} tensor {list(shape)} on cuda:{index}, contiguous in its last dimension, "
                     f"got {t.dtype} {list(t.shape)} with strides {list(s)} on {t.device}")


class PagePool:
    """The pages of a paged cache (``va_page_pool``): the tensors of the block
    table and the free list, the pools that the pages lie in, and the
    workspace.  ``PagePool.create`` makes an empty one; the constructor takes
    tensors that exist (int32, contiguous, on one device): ``block_table``
    ``[num_seqs, stride]``, ``seq_lens`` ``[num_seqs]``, ``ref_count`` and
    ``free_list`` ``[num_pages]``, ``num_free`` ``[1]``, ``flags`` ``[1]`` or None
    (made).  ``buffers``: tensors whose first dimension is the pages (K and V
    pages and scales of every layer), contiguous.  Give ``block_table`` and
    ``seq_lens`` to ``verify_attn_rope_append`` and ``verify_attn_with_plan``
    (with ``block_table_stride`` and ``num_pages`` as plan options).

    The pool's tensors, the workspace among them, are recorded on the torch
    streams that its calls run on, so a pool may be dropped while calls are
    queued there.  It has to outlive the work on a raw stream handle (or an
    ``ExternalStream``) and the replays of a captured graph."""

    def __init__(self, block_table, seq_lens, ref_count, free_list, num_free, buffers, flags=None):
        torch = _torch or _bind_torch()
        i32 = torch.int32
        device, index = _device_of(block_table, "block_table")
        if block_table.dim() != 2 or ref_count.dim() != 1:
            raise ValueError("block_table must be [num_seqs, stride] and ref_count [num_pages]")
        if flags is None:
            flags = torch.zeros(1, dtype=i32, device=device)
        B, stride = block_table.shape
        P = ref_count.shape[0]
        if B | stride | P > _INT_MAX:
            raise _too_large("block_table or ref_count", (B, stride, P))
        self.block_table, self.seq_lens, self.ref_count = block_table, seq_lens, ref_count
        self.free_list, self.num_free, self.flags = free_list, num_free, flags
        self.buffers = list(buffers)
        self.num_seqs, self.num_pages, self.device, self._index = B, P, device, index
        size = int(_load().verify_attn_pages_workspace_bytes(B, P))
        if not size:
            raise ValueError(f"{B} sequences or {P} pages are out of range")
        array = (_PageBuffer * max(1, len(self.buffers)))()
        for i, t in enumerate(self.buffers):
            if not t.is_contiguous() or t.device != device or t.dim() < 1 or t.shape[0] != P:
                raise ValueError(f"buffer {i} must be a contiguous tensor on {device} with {P} pages in its first dimension")
            array[i].data, array[i].page_bytes = t.data_ptr(), t.numel() // P * t.element_size()
        self.workspace = torch.empty(size, dtype=torch.uint8, device=device)
        self._array = array
        self._struct = _PagePool(
            _ptr(block_table, "block_table", i32, index), _ptr(seq_lens, "seq_lens", i32, index, (B,)),
            _ptr(ref_count, "ref_count", i32, index), _ptr(free_list, "free_list", i32, index, (P,)),
            _ptr(num_free, "num_free", i32, index, (1,)), _ptr(flags, "flags", i32, index, (1,)), stride, B, P,
            len(self.buffers), array, self.workspace.data_ptr())
        self._ref = ctypes.byref(self._struct)
        self._tensors = [block_table, seq_lens, ref_count, free_list, num_free, flags, self.workspace, *self.buffers]
        self._recorded = set()  # handles of the streams that the tensors are recorded on

    def _launch_on(self, stream):
        """``_launch_on`` of the pool's device, with the pool's tensors recorded on a torch stream the first time."""
        st, guard = _launch_on(self.device, stream)
        if st not in self._recorded:
            torch = _torch
            if stream is None:
                stream = torch.cuda.current_stream(self.device)
            if isinstance(stream, torch.cuda.Stream) and not isinstance(stream, torch.cuda.ExternalStream):
                for t in self._tensors:  # no more than a look where a tensor was made on that stream
                    t.record_stream(stream)
                self._recorded.add(st)
        return st, guard

    @classmethod
    def create(cls, num_pages, num_seqs, max_blocks, buffers, device="cuda"):
        """An empty pool: no sequence holds anything, the lowest page is taken first."""
        import torch
        device = torch.device(device)
        if device.index is None:
            device = torch.device(device.type, torch.cuda.current_device())
        kw = dict(dtype=torch.int32, device=device)
        return cls(torch.full((num_seqs, max_blocks), -1, **kw), torch.zeros(num_seqs, **kw),
                   torch.zeros(num_pages, **kw), torch.arange(num_pages - 1, -1, -1, **kw),
                   torch.full((1,), num_pages, **kw), buffers)


def verify_attn_pages_resize(pool: PagePool, new_lens, stream=None, kept_lens=None):
    """Change the sequences' lengths to ``new_lens`` (int32 ``[num_seqs]`` on the
    device, negative: left alone): pages past a shorter length go back to the
    pool, a longer one takes pages, and a growing sequence whose partly filled
    last page is shared gets a copy of its own.  ``kept_lens`` (int32
    ``[num_seqs]``): the sequences are first cut back to these, so that the tokens
    behind them (rejected drafts) are written anew in pages of their own; after a
    verify step give the accepted lengths, and in ``new_lens`` those plus the
    next block."""
    i32, shape = _torch.int32, (pool.num_seqs,)
    n = _ptr(new_lens, "new_lens", i32, pool._index, shape)
    kept = None if kept_lens is None else _ptr(kept_lens, "kept_lens", i32, pool._index, shape)
    st, guard = pool._launch_on(stream)
    with guard:
        rc = (_lib or _load()).verify_attn_pages_resize_ex(pool._ref, kept, n, st)
    if rc:
        _check(rc, "verify_attn_pages_resize")


def verify_attn_pages_fork(pool: PagePool, parents, children, lens=None, share=True, stream=None):
    """Make the empty slots ``children`` copies of ``parents`` (int32 ``[F]`` on
    the device), of their first ``lens`` tokens where given.  ``share``: full
    pages are held in common and a partly filled last page is copied; otherwise
    every page is copied.  Where a parent's length counts tokens that are still to
    be written, give ``lens`` without them, or cut both back (``kept_lens`` of
    ``verify_attn_pages_resize``) before either is written."""
    i32, index = _torch.int32, pool._index
    pa = _ptr(parents, "parents", i32, index)
    shape = parents.shape
    if len(shape) != 1:
        raise ValueError("parents must be [F]")
    if shape[0] > _INT_MAX:
        raise _too_large("parents", shape)
    ch = _ptr(children, "children", i32, index, shape)
    ln = None if lens is None else _ptr(lens, "lens", i32, index, shape)
    st, guard = pool._launch_on(stream)
    with guard:
        rc = (_lib or _load()).verify_attn_pages_fork(pool._ref, pa, ch, ln, shape[0], 1 if share else 0, st)
    if rc:
        _check(rc, "verify_attn_pages_fork")


def verify_attn_pages_compact(pool: PagePool, stream=None):
    """Move the held pages to the front of the pool (block tables and counts
    follow); the free list then holds the pages behind them, lowest first."""
    st, guard = pool._launch_on(stream)
    with guard:
        rc = (_lib or _load()).verify_attn_pages_compact(pool._ref, st)
    if rc:
        _check(rc, "verify_attn_pages_compact")


def verify_attn_pages_flags(pool: PagePool, clear=True) -> int:
    """The pool's flag word (``VA_PAGES_*`` bits), cleared by default.  Waits for
    torch's current stream."""
    flags = int(pool.flags.item())
    if clear and flags:
        pool.flags.zero_()
    return flags


class ChunkPlan:
    """Owning handle of a ``va_chunk_plan`` (freed on ``destroy()`` or collection)."""

    def __init__(self, handle, shape, index):
        self._h = ctypes.c_void_p(handle)
        self._index = index  # CUDA device that the plan's memory is on
        (self.num_seqs, self.num_q_heads, self.num_kv_heads, self.head_dim, self.kv_dtype, self.num_tokens,
         self.max_len) = shape  # max_len: the longest sequence that takes part

    @property
    def handle(self):
        return self._h

    def info(self) -> dict:
        info = ChunkPlanInfo()
        _check(_load().verify_attn_chunk_plan_get_info(self._h, ctypes.byref(info)), "verify_attn_chunk_plan_get_info")
        return info.as_dict()

    def destroy(self):
        if self._h and self._h.value:
            _load().verify_attn_chunk_plan_destroy(self._h)
            self._h = ctypes.c_void_p(0)

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def verify_attn_chunk_plan(chunk_lens, seq_lens, num_q_heads, num_kv_heads, head_dim, kv_dtype, num_sms=0) -> ChunkPlan:
    """Plan a batch in which sequence b ends with ``chunk_lens[b]`` new tokens (0: it
    takes no part) of its ``seq_lens[b]`` cached ones, both on the host.  The plan
    owns its workspace on the current CUDA device; calls on it must be ordered on
    one stream."""
    lib = _load()
    torch = _torch or _bind_torch()
    new, lens = _host_lens(chunk_lens), _host_lens(seq_lens)
    if len(new) != len(lens):
        raise ValueError(f"{len(new)} chunk_lens and {len(lens)} seq_lens")
    code = _dtype_code(kv_dtype)
    out = ctypes.c_void_p()
    _check(lib.verify_attn_chunk_plan(new.ctypes.data, lens.ctypes.data, len(new), int(num_q_heads), int(num_kv_heads),
                                      int(head_dim), code, int(num_sms), ctypes.byref(out)), "verify_attn_chunk_plan")
    return ChunkPlan(out.value, (len(new), int(num_q_heads), int(num_kv_heads), int(head_dim), code, int(new.sum()),
                                 int(lens[new > 0].max(initial=0))),
                     torch.cuda.current_device())


def verify_attn_chunk_plan_describe(chunk_lens, seq_lens, num_q_heads, num_kv_heads, head_dim, kv_dtype, num_sms):
    """Host-only planning (no GPU needed): (info dict, items int32 [n, 6]) with
    items = (seq, kv_head, first row of q, tokens, key_begin, key_end)."""
    lib = _load()
    new, lens = _host_lens(chunk_lens), _host_lens(seq_lens)
    if len(new) != len(lens):
        raise ValueError(f"{len(new)} chunk_lens and {len(lens)} seq_lens")
    args = (new.ctypes.data, lens.ctypes.data, len(new), int(num_q_heads), int(num_kv_heads), int(head_dim),
            _dtype_code(kv_dtype), int(num_sms))
    info = ChunkPlanInfo()
    _check(lib.verify_attn_chunk_plan_describe(*args, ctypes.byref(info), None, 0), "verify_attn_chunk_plan_describe")
    items = np.zeros((max(info.num_items, 1), 6), np.int32)
    _check(lib.verify_attn_chunk_plan_describe(*args, ctypes.byref(info), items.ctypes.data, info.num_items),
           "verify_attn_chunk_plan_describe")
    return info.as_dict(), items[:info.num_items]


def verify_attn_chunk_plan_destroy(plan: ChunkPlan):
    plan.destroy()


def verify_attn_chunk_plan_device_flags(plan: ChunkPlan, clear=True, stream=None) -> int:
    """The plan's flag word (bit 0: a block-table entry outside the pool was
    skipped, bit 2: a wait gave up), cleared by default.  Waits for the stream."""
    st, guard = _launch_on(_torch.device("cuda", plan._index), stream)
    flags = ctypes.c_int(0)
    with guard:
        rc = _load().verify_attn_chunk_plan_device_flags(plan._h, int(bool(clear)), ctypes.byref(flags), st)
    _check(rc, "verify_attn_chunk_plan_device_flags")
    return flags.value


def _chunk_q(plan, q):
    """q [tokens or more, Hq, D] as a ``va_heads``, its device and the device's index."""
    device, index = _device_of(q, "q")
    n, s = q.shape, q.stride()
    if (q.dtype is not _torch.bfloat16 or len(n) != 3 or n[0] < plan.num_tokens or n[1] != plan.num_q_heads
            or n[2] != plan.head_dim or s[2] != 1):
        raise ValueError(f"q must be a bfloat16 tensor [{plan.num_tokens}, {plan.num_q_heads}, {plan.head_dim}], contiguous "
                         f"in its last dimension, got {q.dtype} {list(n)} with strides {list(s)}")
    if index != plan._index:
        raise ValueError(f"q is on cuda:{index}, the plan on cuda:{plan._index}")
    return _Heads(q.data_ptr(), 0, s[0], s[1], n[1]), device, index


def _chunk_cache(plan, pages, scale, what, index):
    """Addresses of one of the cache's pools and its scales, and the number of pages."""
    code = plan.kv_dtype
    ptr = _ptr_of(pages, f"{what}_pages", _CACHE_TYPES[code], index)
    row = plan.head_dim * (16 if code == VA_BF16 else 4 if code == VA_INT4 else 2 if code == VA_INT2 else 8) // 8
    n = pages.shape
    cache = (n[0] if len(n) else 0, PAGE_SIZE, plan.num_kv_heads, row // 2 if code == VA_BF16 else row)
    if n != cache:
        raise ValueError(f"{what}_pages must be [num_pages, {PAGE_SIZE}, {plan.num_kv_heads}, {cache[3]}], got {list(n)}")
    if cache[0] > _INT_MAX:
        raise _too_large(f"{what}_pages", n)
    return ptr, None if code == VA_BF16 else _ptr(scale, f"{what}_scale", _torch.float32, index, cache[:3]), cache[0]


def _chunk_table(plan, block_table, index):
    ptr = _ptr(block_table, "block_table", _torch.int32, index)
    n = block_table.shape
    if len(n) != 2 or n[0] != plan.num_seqs:
        raise ValueError(f"block_table must be [{plan.num_seqs}, stride], got {list(n)}")
    if n[1] > _INT_MAX:
        raise _too_large("block_table", n)
    return ptr, n[1]


def verify_attn_chunk(plan: ChunkPlan, q, k_pages, v_pages, k_scale, v_scale, block_table, out=None, lse=None,
                      num_pages=0, stream=None):
    """Attention of chunks of new tokens over the paged cache: ``q`` bf16 ``[tokens,
    Hq, D]``, the new tokens of all sequences one after the other (any strides that
    are multiples of 8 elements with a contiguous last dimension, for instance a
    slice of a fused projection; rows behind the plan's tokens are not read).  The
    new keys and values are in the cache already.  ``num_pages``: pages that the
    block table may name (default: all of the pool's); others are skipped and
    flagged.  ``out`` (bf16) and ``lse`` (fp32 ``[tokens, Hq]``) default to new tensors
    with as many rows as ``q``; rows behind the plan's tokens are left as they are.
    Not recorded by autograd: in grad mode tensors that require a gradient are
    refused.  Returns (out, lse)."""
    torch = _torch or _bind_torch()
    if _grad_mode() and (_wants_gradient(q) or _wants_gradient(k_pages) or _wants_gradient(v_pages)
                         or _wants_gradient(k_scale) or _wants_gradient(v_scale) or _wants_gradient(out)
                         or _wants_gradient(lse)):
        raise _gradient_refused("verify_attn_chunk")
    heads, device, index = _chunk_q(plan, q)
    kp, ks, pages = _chunk_cache(plan, k_pages, k_scale, "k", index)
    vp, vs, pages_v = _chunk_cache(plan, v_pages, v_scale, "v", index)
    if pages_v != pages or num_pages > pages:
        raise ValueError(f"k_pages has {pages} pages, v_pages {pages_v}, num_pages is {num_pages}")
    bt, stride = _chunk_table(plan, block_table, index)
    n = q.shape
    st, guard = _launch_on(device, stream)
    with guard:
        if out is None:
            out = torch.empty(n, dtype=torch.bfloat16, device=device)
        if lse is None:
            lse = torch.empty(n[:2], dtype=torch.float32, device=device)
        rc = (_lib or _load()).verify_attn_chunk(
            plan._h, heads, kp, vp, ks, vs, bt, stride, num_pages or pages, _ptr(out, "out", torch.bfloat16, index, n),
            _ptr(lse, "lse", torch.float32, index, n[:2]), st)
    if rc:
        _check(rc, "verify_attn_chunk")
    return out, lse


def _per_slot(t, name, dtype, index, shape):
    """Address and the strides of a [B, Hkv, slots] tensor, contiguous in its last dimension."""
    try:
        n, s = t.shape, t.stride()
        if (t.dtype is dtype and t.get_device() == index and len(n) == 3 and n[:2] == shape[:2] and n[2] >= shape[2]
                and (s[2] == 1 or n[2] <= 1)):
            return t.data_ptr(), s[0], s[1]
    except AttributeError:
        raise ValueError(f"{name} must be a CUDA tensor") from None
    raise ValueError(f"{name} must be a {dtype} tensor {list(shape)} (or more slots) on cuda:{index}, contiguous in its "
                     f"last dimension, got {t.dtype} {list(n)} with strides {list(s)} on {t.device}")


def verify_attn_chunk_weights(plan: ChunkPlan, q, k_pages, k_scale, block_table, lse, weights, accumulate=True,
                              slot_pos=None, positions=None, num_pages=0, stream=None):
    """The attention weight that each cached token gathers from the chunks: ``weights``
    (fp32 ``[num_seqs, Hkv, slots]``, any strides with a contiguous last dimension)
    is added to at the tokens that were cached before (``accumulate=False``: set) and
    set at the new ones; slots past a sequence's length are left as they are.
    ``lse``: what ``verify_attn_chunk`` returned for the same queries.  ``slot_pos``
    (int32, shape and strides as ``weights``) with ``positions`` (int32 ``[tokens]``): also
    keeps the new tokens' positions, for ``verify_attn_evict``.  Other arguments as
    for ``verify_attn_chunk``; in grad mode tensors that require a gradient are
    refused.  Returns ``weights``."""
    torch = _torch or _bind_torch()
    if _grad_mode() and (_wants_gradient(q) or _wants_gradient(k_pages) or _wants_gradient(k_scale)
                         or _wants_gradient(lse) or _wants_gradient(weights)):
        raise _gradient_refused("verify_attn_chunk_weights")
    heads, device, index = _chunk_q(plan, q)
    kp, ks, pages = _chunk_cache(plan, k_pages, k_scale, "k", index)
    if num_pages > pages:
        raise ValueError(f"num_pages is {num_pages}, the cache has {pages}")
    bt, stride = _chunk_table(plan, block_table, index)
    lp = _ptr(lse, "lse", torch.float32, index)
    n = lse.shape
    if len(n) != 2 or n[0] < plan.num_tokens or n[1] != plan.num_q_heads:
        raise ValueError(f"lse must be [{plan.num_tokens}, {plan.num_q_heads}], got {list(n)}")
    shape = (plan.num_seqs, plan.num_kv_heads, plan.max_len)
    wp, seq, head = _per_slot(weights, "weights", torch.float32, index, shape)
    sp = pos = None
    if slot_pos is not None:
        sp, *strides = _per_slot(slot_pos, "slot_pos", torch.int32, index, shape)
        if strides != [seq, head]:
            raise ValueError("slot_pos must have the strides of weights")
        pos = _ptr(positions, "positions", torch.int32, index)
        if positions.dim() != 1 or positions.shape[0] < plan.num_tokens:
            raise ValueError(f"slot_pos needs positions [{plan.num_tokens}], got {list(positions.shape)}")
    st, guard = _launch_on(device, stream)
    with guard:
        rc = (_lib or _load()).verify_attn_chunk_weights(plan._h, heads, kp, ks, bt, stride, num_pages or pages, lp, wp,
                                                         seq, head, 1 if accumulate else 0, sp, pos, st)
    if rc:
        _check(rc, "verify_attn_chunk_weights")
    return weights


def verify_attn_logprobs(logits, tokens, num_top=0, stream=None):
    """Log probabilities of ``tokens`` (int32 ``[N]``) under ``softmax(logits)`` (``[N,
    V]`` fp32, bf16 or fp16, any row stride), their place in the descending order,
    the rows' entropy and the ``num_top`` (at most ``LOGPROBS_MAX_TOP``) likeliest
    tokens.  Definition in ``include/verify_attn.h``.  Not recorded by autograd: in
    grad mode logits that require a gradient are refused.  Returns (logprobs fp32
    ``[N]``, ranks int32 ``[N]``, entropy fp32 ``[N]``, top_tokens int32 ``[N, num_top]``,
    top_logprobs fp32 ``[N, num_top]``)."""
    torch = _torch or _bind_torch()
    if _grad_mode() and _wants_gradient(logits):
        raise _gradient_refused("verify_attn_logprobs")
    f32, i32 = torch.float32, torch.int32
    device, index = _device_of(logits, "logits")
    code = _float_code(logits, "logits")
    n = logits.shape
    if len(n) != 2 or (n[1] > 1 and logits.stride(1) != 1):
        raise ValueError(f"logits must be [N, V], contiguous in its last dimension, got {list(n)} with strides "
                         f"{list(logits.stride())}")
    N, V = n
    if N | V > _INT_MAX:
        raise _too_large("logits", n)
    K = int(num_top)
    if not 0 <= K <= min(LOGPROBS_MAX_TOP, V):
        raise ValueError(f"num_top must be between 0 and {min(LOGPROBS_MAX_TOP, V)}")
    tp = _ptr(tokens, "tokens", i32, index, (N,))
    st, guard = _launch_on(device, stream)
    with guard:
        logprobs, entropy = torch.empty((N,), dtype=f32, device=device), torch.empty((N,), dtype=f32, device=device)
        ranks = torch.empty((N,), dtype=i32, device=device)
        top_tokens = torch.empty((N, K), dtype=i32, device=device)
        top_logprobs = torch.empty((N, K), dtype=f32, device=device)
        rc = 0
        if N:
            rc = (_lib or _load()).verify_attn_logprobs(
                logits.data_ptr(), logits.stride(0), code, tp, N, V, K, logprobs.data_ptr(), ranks.data_ptr(),
                entropy.data_ptr(), top_tokens.data_ptr(), top_logprobs.data_ptr(), st)
    if rc:
        _check(rc, "verify_attn_logprobs")
    return logprobs, ranks, entropy, top_tokens, top_logprobs


def verify_attn_evict(k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, weights, keep_lens, kv_dtype, slot_pos=None,
                      num_sinks=0, recent_from=None, ref_count=None, new_lens=None, flags=None, num_pages=0, stream=None):
    """Cut sequences back to ``keep_lens`` (int32 ``[num_seqs]`` on the device; negative
    or not below the length: left alone) cached tokens: every kv head keeps the
    protected tokens (positions below ``num_sinks`` or from ``recent_from``, int32
    ``[num_seqs]``, on) and then those with the largest ``weights`` (fp32 ``[num_seqs,
    Hkv, slots]``, as ``verify_attn_chunk_weights`` gathers them).  Rows of K and V,
    scales, ``weights`` and ``slot_pos`` (int32 like ``weights``: the position of each
    slot's token; None: the slot) move into the first slots, in place.  Pass
    ``ref_count`` of a page pool whose sequences may share pages: sequences that do
    are left alone and flagged.  Call it for every layer, then give the result to
    ``verify_attn_pages_resize``.  Definition in ``include/verify_attn.h``.  In grad mode
    tensors that require a gradient are refused.  Returns the new lengths, int32
    ``[num_seqs]``."""
    torch = _torch or _bind_torch()
    if _grad_mode() and (_wants_gradient(weights) or _wants_gradient(k_pages) or _wants_gradient(v_pages)
                         or _wants_gradient(k_scale) or _wants_gradient(v_scale)):
        raise _gradient_refused("verify_attn_evict")
    code = _dtype_code(kv_dtype)
    device, index = _device_of(k_pages, "k_pages")
    f32, i32 = torch.float32, torch.int32
    kvd = _CACHE_TYPES.get(code, ())
    kp, vp = _ptr_of(k_pages, "k_pages", kvd, index), _ptr_of(v_pages, "v_pages", kvd, index)
    n = k_pages.shape
    if len(n) != 4 or n[1] != PAGE_SIZE or v_pages.shape != n:
        raise ValueError(f"k_pages and v_pages must be [num_pages, {PAGE_SIZE}, Hkv, row], got {list(n)} and "
                         f"{list(v_pages.shape)}")
    pages, _, Hkv, D = n
    D = D * 2 if code == VA_INT4 else D * 4 if code == VA_INT2 else D
    bt, sl = _ptr(block_table, "block_table", i32, index), _ptr(seq_lens, "seq_lens", i32, index)
    nt = block_table.shape
    if len(nt) != 2 or seq_lens.shape != nt[:1]:
        raise ValueError(f"block_table must be [num_seqs, stride] and seq_lens [num_seqs], got {list(nt)} and "
                         f"{list(seq_lens.shape)}")
    B, stride = nt
    wp, seq, head = _per_slot(weights, "weights", f32, index, (B, Hkv, 0))
    slots = weights.shape[2]
    if pages | B | Hkv | stride | slots > _INT_MAX:
        raise _too_large("k_pages, block_table or weights", (*n, *nt, *weights.shape))
    if num_pages > pages:
        raise ValueError(f"num_pages is {num_pages}, the cache has {pages}")
    if num_sinks > _INT_MAX:
        raise ValueError(f"num_sinks is {num_sinks}, past 32 bits")
    ks = vs = None
    if code != VA_BF16:
        ks, vs = _ptr(k_scale, "k_scale", f32, index, n[:3]), _ptr(v_scale, "v_scale", f32, index, n[:3])
    sp = None
    if slot_pos is not None:
        sp, *strides = _per_slot(slot_pos, "slot_pos", i32, index, (B, Hkv, slots))
        if strides != [seq, head]:
            raise ValueError("slot_pos must have the strides of weights")
    kl = _ptr(keep_lens, "keep_lens", i32, index, (B,))
    rf = None if recent_from is None else _ptr(recent_from, "recent_from", i32, index, (B,))
    rc_ = None if ref_count is None else _ptr(ref_count, "ref_count", i32, index, (pages,))
    fl = None if flags is None else _ptr(flags, "flags", i32, index)
    lib = _lib or _load()
    size = lib.verify_attn_evict_workspace_bytes(B, Hkv, slots)
    st, guard = _launch_on(device, stream)
    with guard:
        workspace = torch.empty(max(1, size), dtype=torch.uint8, device=device)
        if new_lens is None:
            new_lens = torch.empty((B,), dtype=i32, device=device)
        rc = lib.verify_attn_evict(kp, vp, ks, vs, code, bt, stride, sl, B, Hkv, D, num_pages or pages, wp, sp, seq, head,
                                   slots, kl, int(num_sinks), rf, rc_, _ptr(new_lens, "new_lens", i32, index, (B,)),
                                   workspace.data_ptr(), fl, st)
    if rc:
        _check(rc, "verify_attn_evict")
    return new_lens


__all__ = [
    "verify_attn_evict",
    "verify_attn_logprobs", "LOGPROBS_MAX_TOP",
    "verify_attn_chunk_weights",
    "ChunkPlan", "verify_attn_chunk_plan", "verify_attn_chunk_plan_describe", "verify_attn_chunk_plan_destroy", "verify_attn_chunk_plan_device_flags",
    "verify_attn_chunk",
    "Rope", "verify_attn_rope_spec", "verify_attn_rope", "verify_attn_rope_append", "verify_attn_accept_probs",
    "PagePool", "verify_attn_pages_resize", "verify_attn_pages_fork", "verify_attn_pages_compact",
    "verify_attn_pages_flags",
    "verify_attn_accept",
    "verify_attn_lookup_draft",
    "verify_attn_kv_append",
    "verify_attn_noalloc",
    "verify_attn_noalloc_flags",
    "verify_attn_plan_set_events",
    "verify_attn_plan", "verify_attn", "verify_attn_with_plan", "verify_attn_plan_destroy",
    "verify_attn_status_string", "verify_attn_plan_get_info", "verify_attn_plan_describe",
    "verify_attn_plan_device_flags", "verify_attn_validate_host", "Plan", "VerifyAttnError", "library",
    "LIB_PATH",
]
