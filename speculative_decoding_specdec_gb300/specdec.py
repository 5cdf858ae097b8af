"""ctypes binding of libspecdec.so (see include/specdec.h for the full contract).

Argument marshalling only: tensors become device pointers, strides and sizes; every step runs in
the library's CUDA kernels.  Importing this module raises ImportError when the library has not
been built -- there is no fallback.  Host-detected errors raise SpecdecError; device-detected
errors land in the caller's ``status`` tensor (zero it before the call, read it when convenient).
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libspecdec.so")
if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                      "(or python -m speculative_decoding_specdec_gb300._build)")
lib = ctypes.CDLL(LIB_PATH)

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_CAPACITY, ERR_INPUT_RANGE, ERR_TIMEOUT = range(7)
F32, BF16 = 0, 1
MAX_DRAFT = 31
GREEDY_SCRATCH_BYTES = 73728   # SPECDEC_GREEDY_SCRATCH_BYTES
REALIGN_PDL = 1                # SPECDEC_REALIGN_PDL
MAX_TREE = 64                  # SPECDEC_MAX_TREE

c_i32p = ctypes.POINTER(ctypes.c_int32)


class KvView(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p),
                ("stride_layer", ctypes.c_longlong), ("stride_kv", ctypes.c_longlong),
                ("stride_row", ctypes.c_longlong), ("stride_head", ctypes.c_longlong),
                ("dtype", ctypes.c_int), ("layers", ctypes.c_int), ("rows", ctypes.c_int),
                ("heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("cap_cols", ctypes.c_int)]


class RealignArgs(ctypes.Structure):
    _fields_ = [("src", KvView), ("dst", KvView), ("B", ctypes.c_int), ("D", ctypes.c_int),
                ("pad_id", ctypes.c_int32), ("copy_engine", ctypes.c_int),
                ("n_committed", ctypes.c_void_p), ("width", ctypes.c_void_p),
                ("accept_len", ctypes.c_void_p), ("out_token", ctypes.c_void_p),
                ("draft", ctypes.c_void_p), ("ids_src", ctypes.c_void_p),
                ("ids_dst", ctypes.c_void_p), ("mask_dst", ctypes.c_void_p),
                ("pos_dst", ctypes.c_void_p), ("n_committed_dst", ctypes.c_void_p),
                ("width_dst", ctypes.c_void_p), ("dev_status", ctypes.c_void_p),
                ("flags", ctypes.c_int), ("schedule", ctypes.c_void_p)]


class PoolArgs(ctypes.Structure):
    _fields_ = [("arena", KvView), ("scratch", KvView), ("n_rows", ctypes.c_int),
                ("D", ctypes.c_int), ("pad_id", ctypes.c_int32), ("in_place", ctypes.c_int),
                ("rows", ctypes.c_void_p), ("slot_col", ctypes.c_void_p),
                ("slot_cap", ctypes.c_void_p), ("slot_len", ctypes.c_void_p),
                ("pool_ids", ctypes.c_void_p), ("ids_cap", ctypes.c_int),
                ("batch_len", ctypes.c_void_p), ("width", ctypes.c_void_p),
                ("scratch_ids", ctypes.c_void_p), ("scratch_mask", ctypes.c_void_p),
                ("scratch_pos", ctypes.c_void_p), ("accept_len", ctypes.c_void_p),
                ("out_token", ctypes.c_void_p), ("draft", ctypes.c_void_p),
                ("by_slot", ctypes.c_int), ("dev_status", ctypes.c_void_p),
                ("slot_state", ctypes.c_void_p), ("slot_limit", ctypes.c_void_p),
                ("eos_id", ctypes.c_int32), ("schedule", ctypes.c_void_p)]


class ScheduleArgs(ctypes.Structure):
    _fields_ = [("S", ctypes.c_int), ("batch_size", ctypes.c_int), ("window", ctypes.c_int),
                ("slot_state", ctypes.c_void_p), ("slot_len", ctypes.c_void_p),
                ("perm", ctypes.c_void_p), ("batch_offsets", ctypes.c_void_p),
                ("batch_uniform", ctypes.c_void_p), ("finished", ctypes.c_void_p),
                ("finished_reason", ctypes.c_void_p), ("counts", ctypes.c_void_p),
                ("dev_status", ctypes.c_void_p)]


class AdmitArgs(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int), ("S", ctypes.c_int), ("D", ctypes.c_int),
                ("ids_cap", ctypes.c_int), ("arena_cols", ctypes.c_int64),
                ("slots", ctypes.c_void_p), ("cols", ctypes.c_void_p), ("caps", ctypes.c_void_p),
                ("limits", ctypes.c_void_p), ("prompt_ids", ctypes.c_void_p),
                ("prompt_off", ctypes.c_void_p), ("slot_state", ctypes.c_void_p),
                ("slot_col", ctypes.c_void_p), ("slot_cap", ctypes.c_void_p),
                ("slot_len", ctypes.c_void_p), ("slot_limit", ctypes.c_void_p),
                ("pool_ids", ctypes.c_void_p), ("dev_status", ctypes.c_void_p)]


class RotaryArgs(ctypes.Structure):
    _fields_ = [("cache", KvView), ("layer", ctypes.c_int), ("B", ctypes.c_int),
                ("T", ctypes.c_int), ("heads_q", ctypes.c_int), ("rot_dim", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("table_len", ctypes.c_int),
                ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q_out", ctypes.c_void_p),
                ("q_stride_row", ctypes.c_longlong), ("q_stride_token", ctypes.c_longlong),
                ("k_stride_row", ctypes.c_longlong), ("k_stride_token", ctypes.c_longlong),
                ("v_stride_row", ctypes.c_longlong), ("v_stride_token", ctypes.c_longlong),
                ("q_out_stride_row", ctypes.c_longlong),
                ("q_out_stride_token", ctypes.c_longlong), ("table", ctypes.c_void_p),
                ("n_committed", ctypes.c_void_p), ("width", ctypes.c_void_p),
                ("parents", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("columns", ctypes.c_void_p), ("dev_status", ctypes.c_void_p)]


class SampleArgs(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("dtype", ctypes.c_int), ("R", ctypes.c_int),
                ("V", ctypes.c_int), ("row_stride", ctypes.c_longlong),
                ("temperature", ctypes.c_void_p), ("top_k", ctypes.c_void_p),
                ("top_p", ctypes.c_void_p), ("min_p", ctypes.c_void_p),
                ("uniforms", ctypes.c_void_p), ("token", ctypes.c_void_p),
                ("logprob", ctypes.c_void_p), ("keep_bounds", ctypes.c_void_p),
                ("bounds_stride", ctypes.c_longlong), ("dev_status", ctypes.c_void_p)]


class NormRotaryArgs(ctypes.Structure):
    _fields_ = [("rotary", RotaryArgs), ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("weight_dtype", ctypes.c_int), ("eps", ctypes.c_float),
                ("weight_offset", ctypes.c_float), ("start", ctypes.c_void_p)]


class TreeAttentionArgs(ctypes.Structure):
    _fields_ = [("cache", KvView), ("layer", ctypes.c_int), ("B", ctypes.c_int),
                ("T", ctypes.c_int), ("heads_q", ctypes.c_int), ("scale", ctypes.c_float),
                ("q", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("q_stride_row", ctypes.c_longlong), ("q_stride_token", ctypes.c_longlong),
                ("out_stride_row", ctypes.c_longlong), ("out_stride_token", ctypes.c_longlong),
                ("n_committed", ctypes.c_void_p), ("width", ctypes.c_void_p),
                ("parents", ctypes.c_void_p), ("rows", ctypes.c_void_p),
                ("first_col", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("dev_status", ctypes.c_void_p)]


class PrefixAttentionArgs(ctypes.Structure):
    _fields_ = [("own", TreeAttentionArgs), ("prefix", KvView), ("P", ctypes.c_int),
                ("prefix_len", ctypes.c_void_p), ("prefix_first", ctypes.c_void_p),
                ("group_start", ctypes.c_void_p)]


class TreeCommitArgs(ctypes.Structure):
    _fields_ = [("src", KvView), ("dst", KvView), ("B", ctypes.c_int), ("T", ctypes.c_int),
                ("D", ctypes.c_int), ("width", ctypes.c_void_p), ("width_dst", ctypes.c_void_p),
                ("accept_len", ctypes.c_void_p), ("path", ctypes.c_void_p),
                ("n_committed", ctypes.c_void_p), ("rows", ctypes.c_void_p),
                ("first_col", ctypes.c_void_p), ("dev_status", ctypes.c_void_p)]


SLOT_FREE, SLOT_ACTIVE, SLOT_FINISHED_EOS, SLOT_FINISHED_LENGTH = range(4)


_vp, _ll, _i, _f = ctypes.c_void_p, ctypes.c_longlong, ctypes.c_int, ctypes.c_float
lib.specdec_version.restype = _i
lib.specdec_version.argtypes = []
lib.specdec_status_string.restype = ctypes.c_char_p
lib.specdec_status_string.argtypes = [_i]
lib.specdec_wait_selftest.restype = _i
lib.specdec_wait_selftest.argtypes = [ctypes.c_uint32, ctypes.c_uint32, _vp, _vp]
_sz = ctypes.c_size_t
lib.specdec_verify_greedy.restype = _i
lib.specdec_verify_greedy.argtypes = [_vp, _i, _i, _i, _i, _ll, _vp, _vp, _vp, _vp, _sz, _vp, _vp]
lib.specdec_verify_greedy_workspace.restype = _sz
lib.specdec_verify_greedy_workspace.argtypes = [_i, _i]
lib.specdec_verify_greedy_noalloc.restype = _i
lib.specdec_verify_greedy_noalloc.argtypes = [_vp, _i, _i, _i, _i, _ll, _vp, _vp, _vp, _vp, _vp]
lib.specdec_realign.restype = _i
lib.specdec_realign.argtypes = [ctypes.POINTER(RealignArgs), _vp]
lib.specdec_realign_inplace.restype = _i
lib.specdec_realign_inplace.argtypes = [ctypes.POINTER(RealignArgs), _vp]
lib.specdec_group_by_length.restype = _i
lib.specdec_group_by_length.argtypes = [_vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
lib.specdec_pool_gather.restype = _i
lib.specdec_pool_gather.argtypes = [ctypes.POINTER(PoolArgs), _vp]
lib.specdec_pool_append.restype = _i
lib.specdec_pool_append.argtypes = [ctypes.POINTER(PoolArgs), _vp]
if hasattr(lib, "specdec_verify_sample"):
    lib.specdec_verify_sample.restype = _i
    lib.specdec_verify_sample.argtypes = [_vp, _vp, _i, _i, _i, _i, _ll, _f, _vp, _vp, _vp, _vp,
                                          _vp, _vp, _vp, _vp]
lib.specdec_philox_uniforms.restype = _i
lib.specdec_philox_uniforms.argtypes = [ctypes.c_uint64, ctypes.c_uint64, _i, _i, _vp, _vp]
lib.specdec_verify_sample_philox.restype = _i
lib.specdec_verify_sample_philox.argtypes = [_vp, _vp, _i, _i, _i, _i, _ll, _f, _vp,
                                             ctypes.c_uint64, ctypes.c_uint64, _vp, _vp, _vp,
                                             _vp, _vp, _vp]
lib.specdec_sampling_filter.restype = _i
lib.specdec_sampling_filter.argtypes = [_vp, _vp, _i, _i, _i, _i, _ll, _f, _i, _f, _vp, _vp, _vp]
lib.specdec_pool_schedule.restype = _i
lib.specdec_pool_schedule.argtypes = [ctypes.POINTER(ScheduleArgs), _vp]
lib.specdec_pool_admit.restype = _i
lib.specdec_pool_admit.argtypes = [ctypes.POINTER(AdmitArgs), _vp]
lib.specdec_rotary_append.restype = _i
lib.specdec_rotary_append.argtypes = [_vp, _vp]  # specdec_rotary_args
lib.specdec_norm_rotary_append.restype = _i
lib.specdec_norm_rotary_append.argtypes = [_vp, _vp]  # specdec_norm_rotary_args
lib.specdec_sample.restype = _i
lib.specdec_sample.argtypes = [_vp, _vp]  # specdec_sample_args
lib.specdec_tree_attention.restype = _i
lib.specdec_tree_attention.argtypes = [_vp, _vp]  # specdec_tree_attention_args
lib.specdec_tree_attention_workspace.restype = _sz
lib.specdec_tree_attention_workspace.argtypes = [_i, _i, _i, _i, _i, _i]
lib.specdec_prefix_attention.restype = _i
lib.specdec_prefix_attention.argtypes = [_vp, _vp]  # specdec_prefix_attention_args
lib.specdec_prefix_attention_workspace.restype = _sz
lib.specdec_prefix_attention_workspace.argtypes = [_i, _i, _i, _i, _i, _i, _i]
lib.specdec_verify_tree_greedy.restype = _i
lib.specdec_verify_tree_greedy.argtypes = [_vp, _i, _i, _i, _i, _ll, _vp, _vp, _i, _vp, _vp, _vp,
                                           _vp, _vp, _vp]
lib.specdec_verify_tree_sample.restype = _i
lib.specdec_verify_tree_sample.argtypes = [_vp, _vp, _i, _i, _i, _i, _ll, _f, _vp, _vp, _vp, _i,
                                           _i, _vp, _vp, _vp, _vp, _vp, _vp]
lib.specdec_tree_commit.restype = _i
lib.specdec_tree_commit.argtypes = [_vp, _vp]  # specdec_tree_commit_args
_i64, _i64p = ctypes.c_int64, ctypes.POINTER(ctypes.c_int64)
lib.specdec_arena_create.restype = _i
lib.specdec_arena_create.argtypes = [_i64, ctypes.POINTER(_vp)]
lib.specdec_arena_destroy.restype = None
lib.specdec_arena_destroy.argtypes = [_vp]
lib.specdec_arena_alloc.restype = _i
lib.specdec_arena_alloc.argtypes = [_vp, _i64, _i64p]
lib.specdec_arena_free.restype = _i
lib.specdec_arena_free.argtypes = [_vp, _i64]
lib.specdec_arena_stats.restype = _i
lib.specdec_arena_stats.argtypes = [_vp, _i64p, _i64p, _i64p]


class KeepBound(ctypes.Structure):
    """specdec_keep_bound: the last kept token of a row under the sampling settings."""
    _fields_ = [("key", ctypes.c_uint32), ("index", ctypes.c_int32)]


class SpecdecError(RuntimeError):
    def __init__(self, code, what):
        super().__init__(f"{what}: {status_string(code)} (status {code})")
        self.code = code


def version() -> int:
    return lib.specdec_version()


def status_string(code: int) -> str:
    return lib.specdec_status_string(int(code)).decode()


def wait_selftest(polls, sleep_ns, status, stream=None):
    """Run the library's bounded wait on a barrier nothing completes (at most ``polls`` polls of
    about ``sleep_ns`` ns); it records ERR_TIMEOUT in ``status`` (int32 CUDA tensor)."""
    _need(status, torch.int32, "status")
    _check(lib.specdec_wait_selftest(int(polls), int(sleep_ns), _ptr(status), _stream(stream)),
           "specdec_wait_selftest")


def _check(rc, what):
    if rc != OK:
        raise SpecdecError(rc, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return F32
    if dt == torch.bfloat16:
        return BF16
    raise ValueError(f"unsupported dtype {dt}")


def _need(t, dtype, name):
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")


def kv_view(t: torch.Tensor) -> KvView:
    """View of a cache tensor shaped [L, 2, rows, H, cap, head_dim] whose last two dims are
    contiguous (a column of a head is contiguous and columns follow each other)."""
    if t.dim() != 6 or t.shape[1] != 2:
        raise ValueError("cache must be [L, 2, rows, H, cap, head_dim]")
    L, _, R, H, S, hd = t.shape
    if t.stride(5) != 1 or t.stride(4) != hd:
        raise ValueError("cache columns must be contiguous")
    return KvView(t.data_ptr(), t.stride(0), t.stride(1), t.stride(2), t.stride(3),
                  dtype_code(t.dtype), L, R, H, hd, S)


def _score_rows(x, B, rows, name):
    """(row_stride) of a [B, rows, V] score tensor whose rows are evenly spaced."""
    if x.dim() != 3 or x.shape[0] != B or x.shape[1] != rows:
        raise ValueError(f"{name}: expected [B, {rows}, V], got {tuple(x.shape)}")
    if x.stride(2) != 1 or (B > 1 and x.stride(0) != rows * x.stride(1)):
        raise ValueError(f"{name}: rows must be evenly spaced with unit element stride")
    return x.stride(1)


def greedy_workspace_bytes(B, D) -> int:
    """Workspace bytes greedy verification needs for B rows of D drafts."""
    return int(lib.specdec_verify_greedy_workspace(int(B), int(D)))


def _workspace(ws, need, name):
    if ws is None or ws.dtype != torch.uint8 or not ws.is_cuda or not ws.is_contiguous():
        raise ValueError(f"{name}: workspace must be a contiguous CUDA uint8 tensor")
    if ws.numel() < need:
        raise ValueError(f"{name}: workspace of {ws.numel()} bytes, {need} needed")
    return ctypes.c_void_p(ws.data_ptr()), ws.numel()


def verify_greedy(logits, draft, accept_len, out_token, status, workspace, stream=None):
    """Greedy verification: logits [B, D+1, V] (fp32/bf16), draft [B, D] int32 ->
    accept_len[B], out_token[B] int32 (written asynchronously on ``stream``).  ``workspace``: a
    zero-filled uint8 CUDA tensor of at least greedy_workspace_bytes(B, D) bytes; every call leaves
    it zero-filled again, so it is reused as is."""
    B, D = draft.shape
    V = logits.shape[-1]
    rs = _score_rows(logits, B, D + 1, "logits")
    for t, n in ((draft, "draft"), (accept_len, "accept_len"), (out_token, "out_token"),
                 (status, "status")):
        _need(t, torch.int32, n)
    wp, wn = _workspace(workspace, greedy_workspace_bytes(B, D) if B else 0,
                        "verify_greedy")
    _check(lib.specdec_verify_greedy(_ptr(logits), dtype_code(logits.dtype), B, D, V, rs,
                                     _ptr(draft), _ptr(accept_len), _ptr(out_token), wp, wn,
                                     _ptr(status), _stream(stream)), "specdec_verify_greedy")


def verify_greedy_noalloc(logits, draft, accept_len, out_token, status, stream=None):
    """Greedy verification on the library's static per-device scratch instead of a workspace
    (for callers that cannot allocate or keep a device buffer).  Calls that may overlap on one
    device share that scratch: keep them on one stream."""
    B, D = draft.shape
    V = logits.shape[-1]
    rs = _score_rows(logits, B, D + 1, "logits")
    for t, n in ((draft, "draft"), (accept_len, "accept_len"), (out_token, "out_token"),
                 (status, "status")):
        _need(t, torch.int32, n)
    _check(lib.specdec_verify_greedy_noalloc(_ptr(logits), dtype_code(logits.dtype), B, D, V, rs,
                                             _ptr(draft), _ptr(accept_len), _ptr(out_token),
                                             _ptr(status), _stream(stream)),
           "specdec_verify_greedy_noalloc")


def sampling_filter(target_logits, draft_logits, temperature, top_k, top_p, keep_bounds, status,
                    stream=None):
    """Top-k / top-p keep bounds of every score row into ``keep_bounds``, an int32 CUDA tensor
    [B, 2D+1, 2] holding specdec_keep_bound (key bits, index) per row."""
    B, Dp1 = target_logits.shape[0], target_logits.shape[1]
    D = Dp1 - 1
    V = target_logits.shape[-1]
    rs = _score_rows(target_logits, B, D + 1, "target_logits")
    rs2 = _score_rows(draft_logits, B, D, "draft_logits")
    if rs != rs2 or draft_logits.dtype != target_logits.dtype or draft_logits.shape[-1] != V:
        raise ValueError("target and draft scores must share dtype, V and row stride")
    _need(keep_bounds, torch.int32, "keep_bounds")
    _need(status, torch.int32, "status")
    if tuple(keep_bounds.shape) != (B, 2 * D + 1, 2) or not keep_bounds.is_contiguous():
        raise ValueError("keep_bounds must be a contiguous [B, 2D+1, 2] int32 tensor")
    _check(lib.specdec_sampling_filter(_ptr(target_logits), _ptr(draft_logits),
                                       dtype_code(target_logits.dtype), B, D, V, rs,
                                       float(temperature), int(top_k), float(top_p),
                                       _ptr(keep_bounds), _ptr(status), _stream(stream)),
           "specdec_sampling_filter")


def verify_sample(target_logits, draft_logits, draft, uniforms, temperature, accept_len,
                  out_token, status, residual=None, stream=None, keep_bounds=None):
    """Sampled verification (min(1, p/q) acceptance, normalised max(0, p - q) residual draw);
    ``keep_bounds`` from sampling_filter applies top-k / top-p."""
    B, D = draft.shape
    V = target_logits.shape[-1]
    rs = _score_rows(target_logits, B, D + 1, "target_logits")
    rs2 = _score_rows(draft_logits, B, D, "draft_logits")
    if rs != rs2 or draft_logits.dtype != target_logits.dtype or draft_logits.shape[-1] != V:
        raise ValueError("target and draft scores must share dtype, V and row stride")
    _need(uniforms, torch.float32, "uniforms")
    if tuple(uniforms.shape) != (B, D + 1) or not uniforms.is_contiguous():
        raise ValueError("uniforms must be a contiguous [B, D+1] float32 tensor")
    if residual is not None:
        _need(residual, torch.float32, "residual")
        if tuple(residual.shape) != (B, V) or not residual.is_contiguous():
            raise ValueError("residual must be a contiguous [B, V] float32 tensor")
    _check(lib.specdec_verify_sample(_ptr(target_logits), _ptr(draft_logits),
                                     dtype_code(target_logits.dtype), B, D, V, rs,
                                     float(temperature), _ptr(draft), _ptr(uniforms),
                                     _ptr(accept_len), _ptr(out_token), _ptr(residual),
                                     _ptr(keep_bounds), _ptr(status), _stream(stream)),
           "specdec_verify_sample")


def philox_uniforms(seed, offset, out, stream=None):
    """The uniforms [B, D+1] that verify_sample_philox draws for (seed, offset), into ``out``."""
    _need(out, torch.float32, "out")
    if out.dim() != 2 or not out.is_contiguous():
        raise ValueError("out must be a contiguous [B, D+1] float32 tensor")
    B, Dp1 = out.shape
    _check(lib.specdec_philox_uniforms(int(seed) & (2 ** 64 - 1), int(offset) & (2 ** 64 - 1),
                                       B, Dp1 - 1, _ptr(out), _stream(stream)),
           "specdec_philox_uniforms")


def verify_sample_philox(target_logits, draft_logits, draft, seed, offset, temperature,
                         accept_len, out_token, status, residual=None, stream=None,
                         keep_bounds=None):
    """Sampled verification with the uniforms drawn in-kernel from (seed, offset) by
    Philox4x32-10 (see specdec.h); advance ``offset`` every round."""
    B, D = draft.shape
    V = target_logits.shape[-1]
    rs = _score_rows(target_logits, B, D + 1, "target_logits")
    rs2 = _score_rows(draft_logits, B, D, "draft_logits")
    if rs != rs2 or draft_logits.dtype != target_logits.dtype or draft_logits.shape[-1] != V:
        raise ValueError("target and draft scores must share dtype, V and row stride")
    if residual is not None:
        _need(residual, torch.float32, "residual")
        if tuple(residual.shape) != (B, V) or not residual.is_contiguous():
            raise ValueError("residual must be a contiguous [B, V] float32 tensor")
    _check(lib.specdec_verify_sample_philox(
        _ptr(target_logits), _ptr(draft_logits), dtype_code(target_logits.dtype), B, D, V, rs,
        float(temperature), _ptr(draft), int(seed) & (2 ** 64 - 1), int(offset) & (2 ** 64 - 1),
        _ptr(accept_len), _ptr(out_token), _ptr(residual), _ptr(keep_bounds), _ptr(status),
        _stream(stream)), "specdec_verify_sample_philox")


def _schedule(t):
    """Device address of a pair of scheduling words (None: fixed shares)."""
    if t is None:
        return None
    _need(t, torch.int32, "schedule")
    if t.numel() < 2 or not t.is_contiguous():
        raise ValueError("schedule needs 2 contiguous int32 elements")
    return t.data_ptr()


def realign(src, dst, n_committed, width, accept_len, out_token, draft, ids_src, ids_dst,
            mask_dst, pos_dst, n_committed_dst, width_dst, status, pad_id=0, copy_engine=0,
            pdl=False, stream=None, schedule=None):
    """EQSPEC realignment from cache ``src`` into cache ``dst`` (both [L, 2, B, H, cap, hd]).
    Passing the same tensor as ``src`` and ``dst`` moves the K/V in place
    (specdec_realign_inplace); the metadata outputs stay separate.  ``pdl`` launches it as a
    programmatic dependent of the kernel ahead of it (SPECDEC_REALIGN_PDL).  ``schedule``: None
    (fixed equal shares per CTA) or a zero-filled int32 CUDA tensor of 2 elements that the call
    leaves zero (work items taken from a counter; calls on other streams need their own)."""
    B, D = draft.shape
    in_place = src.data_ptr() == dst.data_ptr()
    a = RealignArgs()
    a.src = kv_view(src)
    a.dst = kv_view(dst)
    a.B, a.D, a.pad_id, a.copy_engine = B, D, int(pad_id), int(copy_engine)
    a.flags = REALIGN_PDL if pdl else 0
    a.schedule = _schedule(schedule)
    for name, t in (("n_committed", n_committed), ("width", width), ("accept_len", accept_len),
                    ("out_token", out_token), ("draft", draft), ("ids_src", ids_src),
                    ("ids_dst", ids_dst), ("pos_dst", pos_dst),
                    ("n_committed_dst", n_committed_dst), ("width_dst", width_dst),
                    ("dev_status", status)):
        _need(t, torch.int32, name)
        setattr(a, name, t.data_ptr())
    _need(mask_dst, torch.uint8, "mask_dst")
    a.mask_dst = mask_dst.data_ptr()
    if ids_src.shape != (B, src.shape[4]) or not ids_src.is_contiguous():
        raise ValueError("ids_src must be a contiguous [B, src cap] int32 tensor")
    for t, n in ((ids_dst, "ids_dst"), (mask_dst, "mask_dst"), (pos_dst, "pos_dst")):
        if t.shape != (B, dst.shape[4]) or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous [B, dst cap] tensor")
    if in_place:
        _check(lib.specdec_realign_inplace(ctypes.byref(a), _stream(stream)),
               "specdec_realign_inplace")
    else:
        _check(lib.specdec_realign(ctypes.byref(a), _stream(stream)), "specdec_realign")


def group_by_length(lengths, batch_size, max_len, perm, batch_offsets, batch_uniform,
                    num_batches, num_uniform, status, stream=None):
    """EXSPEC grouping of pool rows by length (stable counting sort, uniform batches first)."""
    N = lengths.numel()
    for t, n in ((lengths, "lengths"), (perm, "perm"), (batch_offsets, "batch_offsets"),
                 (num_batches, "num_batches"), (num_uniform, "num_uniform"), (status, "status")):
        _need(t, torch.int32, n)
    _need(batch_uniform, torch.uint8, "batch_uniform")
    if perm.numel() < N or batch_offsets.numel() < N + 1 or batch_uniform.numel() < N:
        raise ValueError("output buffers too small")
    _check(lib.specdec_group_by_length(_ptr(lengths), N, int(batch_size), int(max_len),
                                       _ptr(perm), _ptr(batch_offsets), _ptr(batch_uniform),
                                       _ptr(num_batches), _ptr(num_uniform), _ptr(status),
                                       _stream(stream)), "specdec_group_by_length")


def _pool_args(arena, scratch, rows, D, slot_col, slot_cap, slot_len, pool_ids, batch_len, width,
               status, pad_id, in_place):
    a = PoolArgs()
    a.arena = kv_view(arena)
    a.scratch = kv_view(scratch)
    a.n_rows, a.D, a.pad_id, a.in_place = rows.numel(), int(D), int(pad_id), int(bool(in_place))
    for name, t in (("rows", rows), ("slot_col", slot_col), ("slot_cap", slot_cap),
                    ("slot_len", slot_len), ("pool_ids", pool_ids), ("batch_len", batch_len),
                    ("width", width), ("dev_status", status)):
        _need(t, torch.int32, name)
        setattr(a, name, t.data_ptr())
    if pool_ids.dim() != 2 or not pool_ids.is_contiguous():
        raise ValueError("pool_ids must be a contiguous [slots, ids_cap] int32 tensor")
    a.ids_cap = pool_ids.shape[1]
    return a


def pool_gather(arena, scratch, rows, D, slot_col, slot_cap, slot_len, pool_ids, batch_len, width,
                status, scratch_ids=None, scratch_mask=None, scratch_pos=None, pad_id=0,
                in_place=False, stream=None, schedule=None):
    """Gather pool slots ``rows`` into the padded batch buffer ``scratch`` (see specdec.h).
    ``schedule``: as in ``realign``."""
    a = _pool_args(arena, scratch, rows, D, slot_col, slot_cap, slot_len, pool_ids, batch_len,
                   width, status, pad_id, in_place)
    a.schedule = _schedule(schedule)
    if not in_place:
        for t, n, dt in ((scratch_ids, "scratch_ids", torch.int32),
                         (scratch_mask, "scratch_mask", torch.uint8),
                         (scratch_pos, "scratch_pos", torch.int32)):
            _need(t, dt, n)
            if t.shape != (scratch.shape[2], scratch.shape[4]) or not t.is_contiguous():
                raise ValueError(f"{n} must be a contiguous [rows, scratch cap] tensor")
        a.scratch_ids, a.scratch_mask, a.scratch_pos = (scratch_ids.data_ptr(),
                                                        scratch_mask.data_ptr(),
                                                        scratch_pos.data_ptr())
    _check(lib.specdec_pool_gather(ctypes.byref(a), _stream(stream)), "specdec_pool_gather")


def pool_append(arena, scratch, rows, D, slot_col, slot_cap, slot_len, pool_ids, batch_len, width,
                accept_len, out_token, draft, status, in_place=False, by_slot=False,
                slot_state=None, slot_limit=None, eos_id=-1, stream=None, schedule=None):
    """Append a verified batch back to its pool slots (see specdec.h).  With ``by_slot`` the
    accept lengths, tokens and drafts are pool-wide arrays indexed by slot.  With ``slot_state``
    (and ``slot_limit``) finished sequences are retired: end-of-sequence token ``eos_id`` or the
    length limit.  ``schedule``: as in ``realign``."""
    a = _pool_args(arena, scratch, rows, D, slot_col, slot_cap, slot_len, pool_ids, batch_len,
                   width, status, 0, in_place)
    a.schedule = _schedule(schedule)
    a.by_slot = int(bool(by_slot))
    for name, t in (("accept_len", accept_len), ("out_token", out_token), ("draft", draft)):
        _need(t, torch.int32, name)
        setattr(a, name, t.data_ptr())
    if slot_state is not None:
        _need(slot_state, torch.uint8, "slot_state")
        _need(slot_limit, torch.int32, "slot_limit")
        a.slot_state, a.slot_limit, a.eos_id = (slot_state.data_ptr(), slot_limit.data_ptr(),
                                                int(eos_id))
    _check(lib.specdec_pool_append(ctypes.byref(a), _stream(stream)), "specdec_pool_append")


# ------------------------------------------------------------------------ SequencePool lifecycle

def pool_schedule(slot_state, slot_len, batch_size, window, perm, batch_offsets, batch_uniform,
                  finished, finished_reason, counts, status, stream=None):
    """Group the ACTIVE slots by length window, list (and free) the finished ones; counts =
    {num_batches, num_windowed, num_active, num_finished} (see specdec.h)."""
    S = slot_state.numel()
    _need(slot_state, torch.uint8, "slot_state")
    _need(batch_uniform, torch.uint8, "batch_uniform")
    _need(finished_reason, torch.uint8, "finished_reason")
    for t, n in ((slot_len, "slot_len"), (perm, "perm"), (batch_offsets, "batch_offsets"),
                 (finished, "finished"), (counts, "counts"), (status, "status")):
        _need(t, torch.int32, n)
    if (slot_len.numel() < S or perm.numel() < S or batch_offsets.numel() < S + 1 or
            batch_uniform.numel() < S or finished.numel() < S or finished_reason.numel() < S or
            counts.numel() < 4):
        raise ValueError("buffers too small")
    a = ScheduleArgs()
    a.S, a.batch_size, a.window = S, int(batch_size), int(window)
    for name, t in (("slot_state", slot_state), ("slot_len", slot_len), ("perm", perm),
                    ("batch_offsets", batch_offsets), ("batch_uniform", batch_uniform),
                    ("finished", finished), ("finished_reason", finished_reason),
                    ("counts", counts), ("dev_status", status)):
        setattr(a, name, t.data_ptr())
    _check(lib.specdec_pool_schedule(ctypes.byref(a), _stream(stream)), "specdec_pool_schedule")


def pool_admit(slots, cols, caps, limits, prompt_ids, prompt_off, D, arena_cols, slot_state,
               slot_col, slot_cap, slot_len, slot_limit, pool_ids, status, stream=None):
    """Admit prompts (concatenated in ``prompt_ids``, bounds in ``prompt_off``) into FREE slots
    (see specdec.h)."""
    n = slots.numel()
    _need(slot_state, torch.uint8, "slot_state")
    for t, nm in ((slots, "slots"), (cols, "cols"), (caps, "caps"), (limits, "limits"),
                  (prompt_ids, "prompt_ids"), (prompt_off, "prompt_off"), (slot_col, "slot_col"),
                  (slot_cap, "slot_cap"), (slot_len, "slot_len"), (slot_limit, "slot_limit"),
                  (pool_ids, "pool_ids"), (status, "status")):
        _need(t, torch.int32, nm)
    if cols.numel() < n or caps.numel() < n or limits.numel() < n or prompt_off.numel() < n + 1:
        raise ValueError("per-entry arrays too small")
    if pool_ids.dim() != 2 or not pool_ids.is_contiguous():
        raise ValueError("pool_ids must be a contiguous [slots, ids_cap] int32 tensor")
    a = AdmitArgs()
    a.n, a.S, a.D, a.ids_cap = n, slot_state.numel(), int(D), pool_ids.shape[1]
    a.arena_cols = int(arena_cols)
    for name, t in (("slots", slots), ("cols", cols), ("caps", caps), ("limits", limits),
                    ("prompt_ids", prompt_ids), ("prompt_off", prompt_off),
                    ("slot_state", slot_state), ("slot_col", slot_col), ("slot_cap", slot_cap),
                    ("slot_len", slot_len), ("slot_limit", slot_limit), ("pool_ids", pool_ids),
                    ("dev_status", status)):
        setattr(a, name, t.data_ptr())
    _check(lib.specdec_pool_admit(ctypes.byref(a), _stream(stream)), "specdec_pool_admit")


# ------------------------------------------------------------------------ tree speculation
#
# One of these calls is made per layer and round, and the smallest take a few microseconds on the
# GPU, so the marshalling is kept short: each argument struct is packed by one call (the formats
# lay out the ctypes structures above), and a tensor's layout is read once.

_KV = "Pqqqqiiiiii"
_ROTARY = _KV + "iiiiiii" + "PPPP" + "qqqqqqqq" + "PPPPPPP"
_PACK_ROTARY = struct.Struct("@" + _ROTARY)
_PACK_NORM_ROTARY = struct.Struct("@" + _ROTARY + "PPiffP")
_ATTENTION = _KV + "iiiif" + "PPP" + "qqqq" + "PPPPPPnP"
_PACK_ATTENTION = struct.Struct("@" + _ATTENTION)
_PACK_PREFIX = struct.Struct("@" + _ATTENTION + _KV + "iPPP")
_PACK_SAMPLE = struct.Struct("@Piiiq" + "PPPPPPPP" + "qP")
_PACK_COMMIT = struct.Struct("@" + _KV + _KV + "iii" + "PPPPPPPP")
_DTYPES = {torch.float32: F32, torch.bfloat16: BF16}
_cuda_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _raw(stream):
    return _raw_stream(_cuda_device()) if stream is None else stream.cuda_stream


def _kv(t):
    """The fields of specdec_kv_view for a cache [L, 2, rows, H, cap, head_dim]."""
    shape, s, code = t.shape, t.stride(), _DTYPES.get(t.dtype)
    if len(shape) != 6 or shape[1] != 2:
        raise ValueError("cache must be [L, 2, rows, H, cap, head_dim]")
    hd = shape[5]
    if s[5] != 1 or s[4] != hd or code is None or not t.is_cuda:
        raise ValueError("cache must be a float32 or bfloat16 CUDA tensor with contiguous columns")
    return t.data_ptr(), s[0], s[1], s[2], s[3], code, shape[0], shape[2], shape[3], hd, shape[4]


def _ints(t, shape, name):
    """Device address of a contiguous int32 CUDA tensor of that shape; of None, 0."""
    if t is None:
        return 0
    if (t.dtype is not torch.int32 or not t.is_cuda or t.shape != shape
            or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {list(shape)} int32 CUDA tensor")
    return t.data_ptr()


def _ints_of_any(t, name):
    """Device address of a contiguous int32 CUDA tensor (one value, or one per slot); of None, 0."""
    if t is None:
        return 0
    if t.dtype is not torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 CUDA tensor")
    return t.data_ptr()


def _at_least(t, count, name):
    """As _ints_of_any, of a tensor of which ``count`` values are read."""
    if t is not None and t.numel() < count:
        raise ValueError(f"{name} must have {count} values")
    return _ints_of_any(t, name)


def _given(t, name):
    if t is None:
        raise ValueError(f"{name} is needed")
    return t


def _tokens(t, shape, dtype, name):
    """(address, row stride, token stride) of [B, T, heads, head_dim] whose heads are contiguous."""
    s = t.stride()
    if t.shape != shape or t.dtype is not dtype or not t.is_cuda:
        raise ValueError(f"{name} must be a {list(shape)} {dtype} CUDA tensor")
    if s[3] != 1 or (s[2] != shape[3] and shape[2] > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), s[0], s[1]


def _rotary_fields(q, k, v, cache, layer, table, q_out, status, n_committed, width, parents,
                   positions, columns, interleaved):
    """The fields of specdec_rotary_args."""
    view = _kv(cache)
    dtype = cache.dtype
    shape = q.shape
    B, T, Hq, hd = shape
    new = (B, T, view[8], view[9])
    tab = table.shape
    if (len(tab) != 3 or tab[2] != 2 or table.dtype is not torch.float32 or not table.is_cuda
            or not table.is_contiguous()):
        raise ValueError("table must be a contiguous [positions, rot_dim / 2, 2] float32 CUDA tensor")
    if hd != view[9]:
        raise ValueError("q and the cache must have one head_dim")
    qp, qr, qt = _tokens(q, shape, dtype, "q")
    kp, kr, kt = _tokens(k, new, dtype, "k")
    vp, vr, vt = _tokens(v, new, dtype, "v")
    op, outr, outt = _tokens(q_out, shape, dtype, "q_out")
    if positions is None and columns is None:
        where = (_ints(_given(n_committed, "n_committed"), (B,), "n_committed"),
                 _ints_of_any(_given(width, "width"), "width"), _ints(parents, (B, T), "parents"),
                 0, 0)
    else:
        if n_committed is not None or width is not None or parents is not None:
            raise ValueError("positions and columns exclude n_committed, width and parents")
        where = (0, 0, 0, _ints(_given(positions, "positions"), (B, T), "positions"),
                 _ints(_given(columns, "columns"), (B, T), "columns"))
    return (*view, layer, B, T, Hq, 2 * tab[1], 1 if interleaved else 0, tab[0], qp, kp, vp, op,
            qr, qt, kr, kt, vr, vt, outr, outt, table.data_ptr(), *where,
            _ints_of_any(_given(status, "status"), "status"))


def rotary_append(q, k, v, cache, layer, table, q_out, status, n_committed=None, width=None,
                  parents=None, positions=None, columns=None, interleaved=False, stream=None):
    """Rotary positions of the new tokens' q [B, T, Hq, hd] (into ``q_out``) and k [B, T, H, hd],
    and the append of k and v to their columns of ``cache`` [L, 2, rows, H, cap, hd], layer
    ``layer``.  ``table`` [positions, rot_dim / 2, 2] float32 holds cosines and sines.  Columns and
    positions come from a verification pass (``n_committed``, ``width`` and ``parents``, None for a
    chain) or are given (``positions``, ``columns`` [B, T], negative columns: padding)."""
    rc = lib.specdec_rotary_append(
        _PACK_ROTARY.pack(*_rotary_fields(q, k, v, cache, layer, table, q_out, status, n_committed,
                                          width, parents, positions, columns, interleaved)),
        _raw(stream))
    if rc:
        _check(rc, "specdec_rotary_append")


def norm_rotary_append(q, k, v, cache, layer, table, q_out, status, q_weight, k_weight, eps=1e-6,
                       weight_offset=0.0, start=None, n_committed=None, width=None, parents=None,
                       positions=None, columns=None, interleaved=False, stream=None):
    """As rotary_append, with the heads of q and k normed before they are rotated:
    x / sqrt(mean(x^2) + eps) * (weight_offset + weight).  ``q_weight``, ``k_weight`` [hd]: float32 or
    bfloat16, both of one type, None for a side without a norm.  ``start`` [B]: added to the rows'
    positions (the length of a prefix that they share)."""
    fields = _rotary_fields(q, k, v, cache, layer, table, q_out, status, n_committed, width, parents,
                            positions, columns, interleaved)
    one, at, code = (q.shape[3],), [0, 0], F32
    for i, t in enumerate((q_weight, k_weight)):
        if t is None:
            continue
        code = _DTYPES.get(t.dtype)
        if code is None or t.shape != one or not t.is_cuda or not t.is_contiguous():
            raise ValueError("weights must be contiguous [head_dim] float32 or bfloat16 CUDA tensors")
        at[i] = t.data_ptr()
    if q_weight is not None and k_weight is not None and q_weight.dtype is not k_weight.dtype:
        raise ValueError("q_weight and k_weight must have one dtype")
    rc = lib.specdec_norm_rotary_append(
        _PACK_NORM_ROTARY.pack(*fields, *at, code, eps, weight_offset,
                               _ints(start, (q.shape[0],), "start")), _raw(stream))
    if rc:
        _check(rc, "specdec_norm_rotary_append")


def tree_attention_workspace_bytes(q, cache) -> int:
    """Workspace bytes tree_attention needs for this q [B, T, Hq, hd] over this cache, whatever
    the lengths."""
    B, T, Hq, hd = q.shape
    return int(lib.specdec_tree_attention_workspace(dtype_code(q.dtype), B, T, Hq, cache.shape[3],
                                                    hd))


def _attention_fields(q, cache, layer, out, n_committed, width, parents, status, workspace, scale, lse,
                      rows, first_col):
    """The fields of specdec_tree_attention_args."""
    view = _kv(cache)
    dtype = cache.dtype
    shape = q.shape
    B, T, Hq, hd = shape
    if hd != view[9]:
        raise ValueError("q and the cache must have one head_dim")
    qp, qr, qt = _tokens(q, shape, dtype, "q")
    op, outr, outt = _tokens(out, shape, dtype, "out")
    lp = 0
    if lse is not None:
        if (lse.dtype is not torch.float32 or lse.shape != (B, T, Hq) or not lse.is_cuda
                or not lse.is_contiguous()):
            raise ValueError("lse must be a contiguous [B, T, Hq] float32 CUDA tensor")
        lp = lse.data_ptr()
    np_ = (_ints(_given(n_committed, "n_committed"), (B,), "n_committed") if rows is None
           else _ints_of_any(_given(n_committed, "n_committed"), "n_committed"))
    if (workspace.dtype is not torch.uint8 or not workspace.is_cuda
            or not workspace.is_contiguous()):
        raise ValueError("tree_attention: workspace must be a contiguous CUDA uint8 tensor")
    return (
        *view, layer, B, T, Hq, hd ** -0.5 if scale is None else scale, qp, op, lp, qr, qt, outr,
        outt, np_, _ints_of_any(width, "width"), _ints(parents, (B, T), "parents"),
        _ints(rows, (B,), "rows"),
        _at_least(first_col, B if rows is None else n_committed.numel(), "first_col"),
        workspace.data_ptr(), workspace.numel(),
        _ints_of_any(_given(status, "status"), "status"))


def tree_attention(q, cache, layer, out, n_committed, width, parents, status, workspace,
                   scale=None, lse=None, rows=None, first_col=None, stream=None):
    """Attention of a verification pass: q [B, T, Hq, hd] (node 0 the pending token, the others the
    drafted tree of ``parents`` [B, T], None for a chain) against every row's committed columns of
    ``cache`` [L, 2, rows, H, cap, hd], layer ``layer``, and the nodes' own ancestors, into
    ``out`` (and ``lse`` [B, T, Hq] float32).  ``scale`` defaults to hd ** -0.5.  ``workspace``: a
    zero-filled uint8 CUDA tensor of tree_attention_workspace_bytes(q, cache), reused as is.
    ``first_col`` (and ``rows``): tokens elsewhere than right-aligned at ``width``, as in a pool's
    arena."""
    rc = lib.specdec_tree_attention(
        _PACK_ATTENTION.pack(*_attention_fields(q, cache, layer, out, n_committed, width, parents, status,
                                                workspace, scale, lse, rows, first_col)), _raw(stream))
    if rc:
        _check(rc, "specdec_tree_attention")


def prefix_attention_workspace_bytes(q, cache, prefixes) -> int:
    """Workspace bytes prefix_attention needs for this q [B, T, Hq, hd] over this cache and
    ``prefixes`` prefixes, whatever the lengths (enough for tree_attention too)."""
    B, T, Hq, hd = q.shape
    return int(lib.specdec_prefix_attention_workspace(dtype_code(q.dtype), B, T, Hq, cache.shape[3],
                                                      hd, int(prefixes)))


def prefix_attention(q, cache, layer, out, n_committed, width, parents, status, workspace, prefix,
                     prefix_len, group_start, prefix_first=None, scale=None, lse=None, rows=None,
                     first_col=None, stream=None):
    """As tree_attention, over a prefix that rows share as well: batch rows ``group_start[p]`` ..
    ``group_start[p + 1]`` see ``prefix_len[p]`` columns of row p of ``prefix`` [L, 2, P, H, cap, hd]
    (from ``prefix_first[p]`` on; with one row, all in it) before their own.  ``workspace``:
    prefix_attention_workspace_bytes(q, cache, P)."""
    fields = _attention_fields(q, cache, layer, out, n_committed, width, parents, status, workspace,
                               scale, lse, rows, first_col)
    P = prefix_len.shape[0]
    one = (P,)
    rc = lib.specdec_prefix_attention(
        _PACK_PREFIX.pack(*fields, *_kv(prefix), P, _ints(prefix_len, one, "prefix_len"),
                          _ints(prefix_first, one, "prefix_first"),
                          _ints(_given(group_start, "group_start"), (P + 1,), "group_start")),
        _raw(stream))
    if rc:
        _check(rc, "specdec_prefix_attention")


def _scores(t, name):
    """(address, dtype code, B, T, V, row stride) of evenly spaced score rows [B, T, V]."""
    shape, s, code = t.shape, t.stride(), _DTYPES.get(t.dtype)
    if len(shape) != 3 or s[2] != 1 or (shape[0] > 1 and shape[1] > 1 and s[0] != shape[1] * s[1]):
        raise ValueError(f"{name}: expected [B, T, V] with evenly spaced rows of unit stride")
    if code is None or not t.is_cuda:
        raise ValueError(f"{name}: expected a float32 or bfloat16 CUDA tensor")
    # (a row stride below V, as an expanded tensor has, is refused by the library)
    return (t.data_ptr(), code, shape[0], shape[1], shape[2],
            s[0] if shape[1] == 1 and shape[0] > 1 else s[1])


def verify_tree_greedy(logits, tokens, parents, accept_len, out_token, path, draft, status,
                       stream=None):
    """Greedy verification of the trees (``tokens``, ``parents`` [B, T]; parents None: chains)
    against the target's scores ``logits`` [B, T, V]: accept_len [B], out_token [B], the accepted
    nodes ``path`` [B, D] (-1 behind them; the walk goes at most D deep) and their tokens ``draft``
    [B, D] (0 behind them), ready for a realignment."""
    zp, code, B, T, V, rs = _scores(logits, "logits")
    D = path.shape[-1]
    one, two, tree = (B,), (B, D), (B, T)
    rc = lib.specdec_verify_tree_greedy(
        zp, code, B, T, V, rs, _ints(_given(tokens, "tokens"), tree, "tokens"),
        _ints(parents, tree, "parents"), D,
        _ints(_given(accept_len, "accept_len"), one, "accept_len"),
        _ints(_given(out_token, "out_token"), one, "out_token"), _ints(path, two, "path"),
        _ints(_given(draft, "draft"), two, "draft"),
        _ints_of_any(_given(status, "status"), "status"), _raw(stream))
    if rc:
        _check(rc, "specdec_verify_tree_greedy")


def verify_tree_sample(target_logits, draft_logits, tokens, parents, uniforms, temperature,
                       accept_len, out_token, path, draft, status, replacement=False,
                       stream=None):
    """Sampled verification of the trees against the target's [B, T, V] and the draft model's
    [B, T, V] scores: uniforms [B, T] (column 0 for the final draw, column i for node i);
    ``replacement`` if the draft model drew siblings independently, else without replacement.
    Outputs as for verify_tree_greedy."""
    zp, *like = _scores(target_logits, "target_logits")
    wp, *same = _scores(draft_logits, "draft_logits")
    if like != same:
        raise ValueError("target and draft scores must share shape, dtype and row stride")
    code, B, T, V, rs = like
    D = path.shape[-1]
    one, two, tree = (B,), (B, D), (B, T)
    if (uniforms.dtype is not torch.float32 or uniforms.shape != tree or not uniforms.is_cuda
            or not uniforms.is_contiguous()):
        raise ValueError("uniforms must be a contiguous [B, T] float32 CUDA tensor")
    rc = lib.specdec_verify_tree_sample(
        zp, wp, code, B, T, V, rs, temperature, _ints(_given(tokens, "tokens"), tree, "tokens"),
        _ints(parents, tree, "parents"), uniforms.data_ptr(), 1 if replacement else 0, D,
        _ints(_given(accept_len, "accept_len"), one, "accept_len"),
        _ints(_given(out_token, "out_token"), one, "out_token"), _ints(path, two, "path"),
        _ints(_given(draft, "draft"), two, "draft"),
        _ints_of_any(_given(status, "status"), "status"), _raw(stream))
    if rc:
        _check(rc, "specdec_verify_tree_sample")


def _per_row(t, shape, dtype, name):
    """Device address of a contiguous CUDA tensor of that shape and dtype; of None, 0."""
    if t is None:
        return 0
    if t.dtype is not dtype or not t.is_cuda or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {list(shape)} {dtype} CUDA tensor")
    return t.data_ptr()


def sample(logits, uniforms, token, status, temperature=None, top_k=None, top_p=None, min_p=None,
           logprob=None, keep_bounds=None, stream=None):
    """Tokens from scores ``logits`` [R, V] with each row's settings: ``temperature`` (0: the highest
    score), ``top_p``, ``min_p`` [R] float32 and ``top_k`` [R] int32, None for none, and ``uniforms``
    [R] float32 in [0, 1); ``token`` [R] int32 out, ``logprob`` [R] float32 out.  ``keep_bounds``
    [R, 2] int32 (rows may be strided): the kept sets, as verify_sample takes them, so that
    ``bounds[:, D + 1 + j]`` of a verification's [B, 2 D + 1, 2] is filled as draft j is drawn."""
    shape, s, code = logits.shape, logits.stride(), _DTYPES.get(logits.dtype)
    if len(shape) != 2 or code is None or not logits.is_cuda or (s[1] != 1 and shape[1] > 1):
        raise ValueError("logits must be a [R, V] float32 or bfloat16 CUDA tensor with rows of unit stride")
    R, V = shape
    one, f32 = (R,), torch.float32
    kp = ks = 0
    if keep_bounds is not None:
        b = keep_bounds.stride()
        if (keep_bounds.dtype is not torch.int32 or keep_bounds.shape != (R, 2) or not keep_bounds.is_cuda
                or b[1] != 1 or b[0] % 2):
            raise ValueError("keep_bounds must be a [R, 2] int32 CUDA tensor of whole bounds")
        kp, ks = keep_bounds.data_ptr(), b[0] // 2
    args = _PACK_SAMPLE.pack(
        logits.data_ptr(), code, R, V, s[0] if R > 1 else V, _per_row(temperature, one, f32, "temperature"),
        _ints(top_k, one, "top_k"), _per_row(top_p, one, f32, "top_p"), _per_row(min_p, one, f32, "min_p"),
        _per_row(_given(uniforms, "uniforms"), one, f32, "uniforms"),
        _ints(_given(token, "token"), one, "token"), _per_row(logprob, one, f32, "logprob"), kp, ks,
        _ints_of_any(_given(status, "status"), "status"))
    rc = lib.specdec_sample(args, _raw(stream))
    if rc:
        _check(rc, "specdec_sample")


def tree_commit(src, dst, width, accept_len, path, status, width_dst=None, nodes=MAX_TREE,
                n_committed=None, rows=None, first_col=None, stream=None):
    """Make the accepted paths' K/V columns contiguous (see specdec.h): in place (``dst`` is
    ``src``) before a realignment, or into the realigned cache ``dst`` of width ``width_dst``
    after it.  ``first_col`` (with ``n_committed`` and ``rows``): in a pool's arena."""
    B, D = path.shape
    one = (B,)
    sv = _kv(src)
    args = _PACK_COMMIT.pack(
        *sv, *(sv if dst is src else _kv(dst)), B, nodes, D, _ints_of_any(width, "width"),
        _ints_of_any(width_dst, "width_dst"),
        _ints(_given(accept_len, "accept_len"), one, "accept_len"), _ints(path, (B, D), "path"),
        _at_least(n_committed, B if rows is None else 1, "n_committed"), _ints(rows, one, "rows"),
        _at_least(first_col, B if rows is None or n_committed is None else n_committed.numel(),
                  "first_col"),
        _ints_of_any(_given(status, "status"), "status"))
    rc = lib.specdec_tree_commit(args, _raw(stream))
    if rc:
        _check(rc, "specdec_tree_commit")


class Arena:
    """Host first-fit allocator of arena columns (specdec_arena_*; no GPU involved)."""

    def __init__(self, cols: int):
        h = ctypes.c_void_p()
        _check(lib.specdec_arena_create(int(cols), ctypes.byref(h)), "specdec_arena_create")
        self._h = h
        self.cols = int(cols)

    def alloc(self, ncols: int):
        """Lowest free run of ``ncols`` columns, or None when none is free."""
        c = ctypes.c_int64()
        rc = lib.specdec_arena_alloc(self._h, int(ncols), ctypes.byref(c))
        if rc == ERR_CAPACITY:
            return None
        _check(rc, "specdec_arena_alloc")
        return c.value

    def free(self, col: int) -> None:
        _check(lib.specdec_arena_free(self._h, int(col)), "specdec_arena_free")

    def stats(self):
        """(free columns, largest free run, allocations)."""
        v = [ctypes.c_int64() for _ in range(3)]
        _check(lib.specdec_arena_stats(self._h, *[ctypes.byref(x) for x in v]),
               "specdec_arena_stats")
        return tuple(x.value for x in v)

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            lib.specdec_arena_destroy(h)
            self._h = None
