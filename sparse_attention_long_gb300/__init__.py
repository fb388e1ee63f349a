"""Python binding of the GB300 DSA library (libdsa_gb300.so): argument
marshalling only.  Every step of the path runs in the library's CUDA kernels;
torch tensors are used for device memory and streams.

The library must be built first (``python -m sparse_attention_long_gb300._build``
or ``__graft_entry__.build()``); importing this module without it raises.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdsa_gb300.so")

DSA_OK, DSA_ERR_INVALID_ARG, DSA_ERR_UNSUPPORTED, DSA_ERR_WORKSPACE = 0, -1, -2, -3
DSA_ERR_CUDA, DSA_ERR_TIMEOUT, DSA_ERR_INDEX, DSA_ERR_PAGES = -4, -5, -6, -7
DSA_BSND, DSA_TND = 0, 1
DSA_BF16, DSA_FP32 = 0, 1
DSA_CP_COLOSSAL, DSA_CP_ULYSSES = 0, 1
DSA_CALL_FORWARD, DSA_CALL_ATTN_FWD, DSA_CALL_ATTN_BWD, DSA_CALL_KL_BWD, DSA_CALL_BACKWARD = 0, 1, 2, 3, 4
DSA_CALL_INDEXER_TOPK = 5
DSA_FLAG_CAUSAL_ONLY, DSA_FLAG_FP8_INDEXER, DSA_FLAG_FUSED_TOPK = 1, 2, 4
DSA_ROPE_INTERLEAVED, DSA_ROPE_HALF = 0, 1
DSA_ROPE_PLAIN, DSA_ROPE_LINEAR, DSA_ROPE_NTK, DSA_ROPE_YARN = 0, 1, 2, 3
DSA_ROPE_PARTS, DSA_ROPE_MAX_DIM = 4, 256

_ERRNAMES = {0: "DSA_OK", -1: "DSA_ERR_INVALID_ARG", -2: "DSA_ERR_UNSUPPORTED",
             -3: "DSA_ERR_WORKSPACE", -4: "DSA_ERR_CUDA", -5: "DSA_ERR_TIMEOUT", -6: "DSA_ERR_INDEX",
             -7: "DSA_ERR_PAGES"}


class DSAError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {_ERRNAMES.get(code, code)}")
        self.code = code


class dsa_params(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int32), ("dtype", ctypes.c_int32), ("cp_mode", ctypes.c_int32),
                ("flags", ctypes.c_int32),
                ("B", ctypes.c_int64), ("S_q", ctypes.c_int64), ("S_k", ctypes.c_int64),
                ("H", ctypes.c_int64), ("d_qk", ctypes.c_int64), ("d_v", ctypes.c_int64),
                ("H_I", ctypes.c_int64), ("d_I", ctypes.c_int64), ("topk", ctypes.c_int64),
                ("scale", ctypes.c_float), ("reserved1", ctypes.c_int32),
                ("q_row_offset", ctypes.c_int64), ("q_row_index", ctypes.c_void_p),
                ("wave_rows", ctypes.c_int64)]


class dsa_cache(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int64), ("n_pages", ctypes.c_int64), ("page_rows", ctypes.c_int64),
                ("max_pages", ctypes.c_int64)]


class dsa_pool(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("n_layers", ctypes.c_int64), ("layer_stride", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("row_bytes", ctypes.c_int64)]


class dsa_tree(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("scale", ctypes.c_float), ("n_tok", ctypes.c_int64),
                ("H", ctypes.c_int64), ("d_qk", ctypes.c_int64), ("d_v", ctypes.c_int64),
                ("mask_words", ctypes.c_int64)]


class dsa_beam(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("reserved0", ctypes.c_int32), ("n_batch", ctypes.c_int64),
                ("beams_in", ctypes.c_int64), ("beams_out", ctypes.c_int64), ("vocab", ctypes.c_int64),
                ("ld", ctypes.c_int64), ("eos", ctypes.c_int64)]


class dsa_rope_part(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("layout", ctypes.c_int32), ("heads", ctypes.c_int64),
                ("dim", ctypes.c_int64), ("offset", ctypes.c_int64)]


class dsa_rope(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("n_parts", ctypes.c_int32), ("mscale", ctypes.c_float),
                ("reserved0", ctypes.c_int32), ("part", dsa_rope_part * DSA_ROPE_PARTS),
                ("step", ctypes.c_uint64 * (DSA_ROPE_MAX_DIM // 2))]


class dsa_rope_rows(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("tok_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class dsa_sampler(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("reserved0", ctypes.c_int32), ("rows", ctypes.c_int64),
                ("vocab", ctypes.c_int64), ("ld", ctypes.c_int64), ("requests", ctypes.c_int64)]


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                      "(nvcc, sm_103a); there is no fallback implementation")
lib = ctypes.CDLL(LIB_PATH)

_vp, _i64, _i32p = ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p
_P = ctypes.POINTER(dsa_params)
_C, _L, _T = ctypes.POINTER(dsa_cache), ctypes.POINTER(dsa_pool), ctypes.POINTER(dsa_tree)
_B = ctypes.POINTER(dsa_beam)
_R, _RR, _S = ctypes.POINTER(dsa_rope), ctypes.POINTER(dsa_rope_rows), ctypes.POINTER(dsa_sampler)
_f64 = ctypes.c_double
_sigs = {
    "dsa_version": ([], ctypes.c_int),
    "dsa_workspace_size": ([_P, ctypes.c_int], ctypes.c_size_t),
    "dsa_indexer_scores": ([_P, _vp, _vp, _vp, _i64, _i64, _vp, _vp], ctypes.c_int),
    "dsa_indexer_quantize_fp8": ([_P] + [_vp] * 7, ctypes.c_int),
    "dsa_indexer_scores_fp8": ([_P, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _vp, _vp], ctypes.c_int),
    "dsa_topk": ([_P, _vp, _i64, _i64, _vp, _vp], ctypes.c_int),
    "dsa_indexer_topk": ([_P, _vp, _vp, _vp, _i64, _i64, _vp, _vp, _vp], ctypes.c_int),
    "dsa_sparse_attn_fwd": ([_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp], ctypes.c_int),
    "dsa_sparse_attn_bwd": ([_P] + [_vp] * 11, ctypes.c_int),
    "dsa_indexer_kl_loss_bwd": ([_P] + [_vp] * 14, ctypes.c_int),
    "dsa_backward": ([_P] + [_vp] * 18, ctypes.c_int),
    "dsa_forward": ([_P] + [_vp] * 11, ctypes.c_int),
    "dsa_forward_static_ws": ([_P] + [_vp] * 10, ctypes.c_int),
    "dsa_cache_fork": ([_C] + [_vp] * 10, ctypes.c_int),
    "dsa_cache_extend": ([_C] + [_vp] * 7 + [_i64, _vp], ctypes.c_int),
    "dsa_cache_compact": ([_C] + [_vp] * 9, ctypes.c_int),
    "dsa_cache_copy_pages": ([_C, _L, _vp, _vp, _i64, _vp], ctypes.c_int),
    "dsa_cache_write": ([_C, _L, _vp, _i64, _i64, _vp, _vp, _i64, _vp], ctypes.c_int),
    "dsa_tree_workspace_size": ([_C, _T], ctypes.c_size_t),
    "dsa_tree_attn_fwd": ([_C, _T, _vp, _L] + [_vp] * 10, ctypes.c_int),
    "dsa_beam_workspace_size": ([_B], ctypes.c_size_t),
    "dsa_beam_select": ([_B] + [_vp] * 9, ctypes.c_int),
    "dsa_rope_steps": ([_R, _f64, ctypes.c_int, _f64, _f64, _f64, _f64], ctypes.c_int),
    "dsa_rope_apply": ([_R, _i64, _vp, _RR, _RR, ctypes.c_int, _vp], ctypes.c_int),
    "dsa_sample": ([_S] + [_vp] * 10, ctypes.c_int),
    "dsa_tree_accept": ([_C, _T] + [_vp] * 4 + [_i64] + [_vp] * 5, ctypes.c_int),
    "dsa_get_status": ([_vp, ctypes.POINTER(ctypes.c_int)], ctypes.c_int),
    "dsa_set_wait_budget_ns": ([ctypes.c_uint64], ctypes.c_int),
    "dsa_selftest_wait_timeout": ([ctypes.c_uint64, _vp], ctypes.c_int),
}
for _n, (_a, _r) in _sigs.items():
    _f = getattr(lib, _n)
    _f.argtypes, _f.restype = _a, _r


def _chk(rc: int, where: str):
    if rc != DSA_OK:
        raise DSAError(rc, where)


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def make_params(*, B, S_q, S_k, H, d_qk, d_v, H_I, d_I, topk, scale, dtype="bf16",
                layout="BSND", q_row_offset=0, q_row_index=None, wave_rows=0,
                cp_mode="colossal", flags=0) -> dsa_params:
    """Builds the C parameter block.  ``q_row_index`` is a device int32 tensor
    (kept alive by the caller) or None."""
    p = dsa_params()
    p.layout = {"BSND": DSA_BSND, "TND": DSA_TND}[layout]
    p.dtype = {"bf16": DSA_BF16, "fp32": DSA_FP32}[dtype]
    p.cp_mode = {"colossal": DSA_CP_COLOSSAL, "ulysses": DSA_CP_ULYSSES}[cp_mode]
    p.B, p.S_q, p.S_k, p.H, p.d_qk, p.d_v = B, S_q, S_k, H, d_qk, d_v
    p.H_I, p.d_I, p.topk, p.scale = H_I, d_I, topk, float(scale)
    p.q_row_offset = q_row_offset
    p.q_row_index = None if q_row_index is None else _ptr(q_row_index)
    p.wave_rows = wave_rows
    p.flags = flags
    return p


def wave_rows(p: dsa_params) -> int:
    """Rows per indexer/top-k wave dsa_forward uses: its plain score ring holds
    one wave of S_k fp32 scores per row, so the library's workspace size for
    the same shape without the indexer flags gives it."""
    q = dsa_params.from_buffer_copy(p)
    q.flags &= ~(DSA_FLAG_FP8_INDEXER | DSA_FLAG_FUSED_TOPK)
    return workspace_size(q, DSA_CALL_FORWARD) // (4 * q.S_k)


def version() -> int:
    return lib.dsa_version()


def workspace_size(p: dsa_params, which: int) -> int:
    return lib.dsa_workspace_size(ctypes.byref(p), which)


def indexer_scores(p, q_I, k_I, w, row_begin, rows, scores, stream=None):
    _chk(lib.dsa_indexer_scores(ctypes.byref(p), _ptr(q_I), _ptr(k_I), _ptr(w), row_begin, rows,
                                _ptr(scores), _stream(stream)), "dsa_indexer_scores")


def indexer_quantize_fp8(p, q_I, k_I, q8, q_scale, k8, k_scale, stream=None):
    _chk(lib.dsa_indexer_quantize_fp8(ctypes.byref(p), _ptr(q_I), _ptr(k_I), _ptr(q8), _ptr(q_scale),
                                      _ptr(k8), _ptr(k_scale), _stream(stream)),
         "dsa_indexer_quantize_fp8")


def indexer_scores_fp8(p, q8, q_scale, k8, k_scale, w, row_begin, rows, scores, stream=None):
    _chk(lib.dsa_indexer_scores_fp8(ctypes.byref(p), _ptr(q8), _ptr(q_scale), _ptr(k8), _ptr(k_scale),
                                    _ptr(w), row_begin, rows, _ptr(scores), _stream(stream)),
         "dsa_indexer_scores_fp8")


def topk(p, scores, row_begin, rows, idx, stream=None):
    _chk(lib.dsa_topk(ctypes.byref(p), _ptr(scores), row_begin, rows, _ptr(idx), _stream(stream)),
         "dsa_topk")


def indexer_topk(p, q_I, k_I, w, row_begin, rows, idx, workspace, stream=None):
    """Fused indexer + streaming top-k: the indices dsa_indexer_scores +
    dsa_topk give, without a score matrix (workspace: DSA_CALL_INDEXER_TOPK)."""
    _chk(lib.dsa_indexer_topk(ctypes.byref(p), _ptr(q_I), _ptr(k_I), _ptr(w), row_begin, rows,
                              _ptr(idx), _ptr(workspace), _stream(stream)), "dsa_indexer_topk")


def sparse_attn_fwd(p, q, kv, idx, out, softmax_max, softmax_sum, workspace=None, stream=None):
    _chk(lib.dsa_sparse_attn_fwd(ctypes.byref(p), _ptr(q), _ptr(kv), _ptr(idx), _ptr(out),
                                 _ptr(softmax_max), _ptr(softmax_sum), _ptr(workspace),
                                 _stream(stream)), "dsa_sparse_attn_fwd")


def sparse_attn_bwd(p, q, kv, idx, out, dout, softmax_max, softmax_sum, dq, dkv, workspace=None,
                    stream=None):
    _chk(lib.dsa_sparse_attn_bwd(ctypes.byref(p), _ptr(q), _ptr(kv), _ptr(idx), _ptr(out),
                                 _ptr(dout), _ptr(softmax_max), _ptr(softmax_sum), _ptr(dq),
                                 _ptr(dkv), _ptr(workspace), _stream(stream)), "dsa_sparse_attn_bwd")


def indexer_kl_loss_bwd(p, q, kv, q_I, k_I, w, idx, softmax_max, softmax_sum, loss, dq_I, dk_I, dw,
                        workspace=None, stream=None):
    _chk(lib.dsa_indexer_kl_loss_bwd(ctypes.byref(p), _ptr(q), _ptr(kv), _ptr(q_I), _ptr(k_I),
                                     _ptr(w), _ptr(idx), _ptr(softmax_max), _ptr(softmax_sum),
                                     _ptr(loss), _ptr(dq_I), _ptr(dk_I), _ptr(dw),
                                     _ptr(workspace), _stream(stream)), "dsa_indexer_kl_loss_bwd")


def backward(p, q, kv, idx, out, dout, softmax_max, softmax_sum, q_I, k_I, w, dq, dkv, loss, dq_I,
             dk_I, dw, workspace=None, stream=None):
    """sparse_attn_bwd and indexer_kl_loss_bwd in one call sharing the recompute of P."""
    _chk(lib.dsa_backward(ctypes.byref(p), _ptr(q), _ptr(kv), _ptr(idx), _ptr(out), _ptr(dout),
                          _ptr(softmax_max), _ptr(softmax_sum), _ptr(q_I), _ptr(k_I), _ptr(w),
                          _ptr(dq), _ptr(dkv), _ptr(loss), _ptr(dq_I), _ptr(dk_I), _ptr(dw),
                          _ptr(workspace), _stream(stream)), "dsa_backward")


def forward(p, q_I, k_I, w, q, kv, idx_out, out, softmax_max, softmax_sum, workspace, stream=None):
    _chk(lib.dsa_forward(ctypes.byref(p), _ptr(q_I), _ptr(k_I), _ptr(w), _ptr(q), _ptr(kv),
                         _ptr(idx_out), _ptr(out), _ptr(softmax_max), _ptr(softmax_sum),
                         _ptr(workspace), _stream(stream)), "dsa_forward")


def forward_static_ws(p, q_I, k_I, w, q, kv, idx_out, out, softmax_max, softmax_sum, stream=None):
    """dsa_forward without a workspace argument: the score ring is the
    library's own fixed device array (for callers that cannot allocate)."""
    _chk(lib.dsa_forward_static_ws(ctypes.byref(p), _ptr(q_I), _ptr(k_I), _ptr(w), _ptr(q),
                                   _ptr(kv), _ptr(idx_out), _ptr(out), _ptr(softmax_max),
                                   _ptr(softmax_sum), _stream(stream)), "dsa_forward_static_ws")


# ------------------------------- paged cache -------------------------------
# These calls are made once or several times per generated token.  _native makes
# them in a few hundred nanoseconds on top of the launch; it answers 1, having
# done nothing, when an argument is not exactly what the call needs or a stream
# is given.  The Python code below it then makes the call or says what is wrong.
class _Absent:
    def __getattr__(self, name):
        return lambda *args: 1


def _present_stamp():
    # (by its path: `python -m` runs the same file as a module of this package)
    spec = importlib.util.spec_from_file_location("_dsa_build", os.path.join(_HERE, "_build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    return build.binding_stamp(torch.__version__)


def _load_native():
    try:
        from . import _binding
        present = _present_stamp()
    except (ImportError, OSError):                 # built without PyTorch's or Python's headers; no sources here
        return _Absent()
    if getattr(_binding, "stamp", None) != present:  # made of another dsa.h, PyTorch or Python
        return _Absent()
    names = ("dsa_cache_fork", "dsa_cache_extend", "dsa_cache_compact", "dsa_cache_copy_pages", "dsa_cache_write",
             "dsa_tree_attn_fwd", "dsa_tree_workspace_size", "dsa_beam_select", "dsa_beam_workspace_size",
             "dsa_rope_apply", "dsa_sample", "dsa_tree_accept")
    _binding.bind(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names), dsa_cache, dsa_tree, dsa_beam,
                  dsa_rope, dsa_sampler)
    return _binding


_native = _load_native()


def _made(rc, where):
    if rc < 0:
        raise DSAError(rc, where)
    return rc == 0


def _refuse(where, name, t, dtype, numel, device, at_least=False):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{where}: {name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{where}: {name} is not a CUDA tensor")
    if t.get_device() != device:
        raise ValueError(f"{where}: {name} is on {t.device}, other tensors on cuda:{device}")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{where}: {name} is {t.dtype}, needs {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be contiguous")
    if not (t.numel() >= numel if at_least else t.numel() == numel):
        raise ValueError(f"{where}: {name} has {t.numel()} elements, needs {numel}")


def _device(t, where, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _refuse(where, name, t, None, 0, -1)
    return t.get_device()


def _arg(t, name, dtype, numel, device, where):
    """Address of a contiguous CUDA tensor of this type and size on this device."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.numel() == numel and t.get_device() == device \
            and t.is_contiguous():
        return t.data_ptr()
    _refuse(where, name, t, dtype, numel, device)


def _list(t, name, numel, device, where):
    """The same for an int32 list that may be longer."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or t.numel() < numel or \
            t.get_device() != device or not t.is_contiguous():
        _refuse(where, name, t, torch.int32, numel, device, at_least=True)
    return t.data_ptr()


def _pool(c, t, where):
    """(dsa_pool, layers, D) of a tensor [n_pages, page_rows, D] or [layers, n_pages, page_rows, D] whose
    rows are contiguous within a page (layers and pages may have any stride)."""
    sh, st = t.shape, t.stride()
    if len(sh) == 3:
        sh, st = (1, *sh), (0, *st)
    if len(sh) != 4 or sh[1] != c.n_pages or sh[2] != c.page_rows:
        raise ValueError(f"{where}: pool must be [(layers,) n_pages, page_rows, D]")
    D = sh[3]
    if (D > 1 and st[3] != 1) or (sh[2] > 1 and st[2] != D):
        raise ValueError(f"{where}: the rows of a pool's page must be contiguous")
    e = t.element_size()
    page = sh[2] * D * e
    return dsa_pool(t.data_ptr(), sh[0], st[0] * e if sh[0] > 1 else page, st[1] * e if sh[1] > 1 else page,
                    D * e), sh[0], D


def _workspace(t, need, device, where):
    """Address of a workspace tensor of any type with at least `need` bytes (None if 0)."""
    if t is None and need == 0:
        return None
    if t is None or t.numel() * t.element_size() < need:
        raise DSAError(DSA_ERR_WORKSPACE, where)
    if t.get_device() != device or not t.is_contiguous():
        _refuse(where, "workspace", t, t.dtype, t.numel(), device)
    return t.data_ptr()


def _call(fn, where, device, stream, *args):
    """fn(*args, stream) with `device` current."""
    if device == torch._C._cuda_getDevice():
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, _stream(stream))
    if rc != DSA_OK:
        raise DSAError(rc, where)


_I32 = torch.int32


def make_cache(*, n_seqs, n_pages, page_rows, max_pages) -> dsa_cache:
    """Sizes of a paged cache: table [n_seqs, max_pages], lens [n_seqs] and refs [n_pages]
    are int32 tensors of the caller; a new cache has lens and refs all zero."""
    return dsa_cache(n_seqs, n_pages, page_rows, max_pages)


def cache_fork(c, parent, table, lens, refs, table_out, lens_out, refs_out, copies, n_copies, stream=None):
    """Sequence i becomes a copy of old sequence parent[i] (-1: emptied); full pages are shared.
    Follow with cache_copy_pages(copies, n_copies) on every pool."""
    w = "dsa_cache_fork"
    if stream is None and _made(_native.cache_fork(c, parent, table, lens, refs, table_out, lens_out, refs_out, copies,
                                                   n_copies), w):
        return
    d, n, t, p = _device(parent, w, "parent"), c.n_seqs, c.n_seqs * c.max_pages, c.n_pages
    _call(lib.dsa_cache_fork, w, d, stream, ctypes.byref(c), _arg(parent, "parent", _I32, n, d, w),
          _arg(table, "table", _I32, t, d, w), _arg(lens, "lens", _I32, n, d, w), _arg(refs, "refs", _I32, p, d, w),
          _arg(table_out, "table_out", _I32, t, d, w), _arg(lens_out, "lens_out", _I32, n, d, w),
          _arg(refs_out, "refs_out", _I32, p, d, w), _list(copies, "copies", 3 * n, d, w),
          _arg(n_copies, "n_copies", _I32, 1, d, w))


def cache_extend(c, n_new, table, lens, refs, lens_out, refs_out, slots, stream=None):
    """Takes pages for n_new[i] further rows of each sequence (table in place; lens_out and
    refs_out may be lens and refs) and writes the slots of the new rows, -1 behind the last."""
    w = "dsa_cache_extend"
    if stream is None and _made(_native.cache_extend(c, n_new, table, lens, refs, lens_out, refs_out, slots), w):
        return
    d, n, p = _device(n_new, w, "n_new"), c.n_seqs, c.n_pages
    _call(lib.dsa_cache_extend, w, d, stream, ctypes.byref(c), _arg(n_new, "n_new", _I32, n, d, w),
          _arg(table, "table", _I32, n * c.max_pages, d, w), _arg(lens, "lens", _I32, n, d, w),
          _arg(refs, "refs", _I32, p, d, w), _arg(lens_out, "lens_out", _I32, n, d, w),
          _arg(refs_out, "refs_out", _I32, p, d, w), _list(slots, "slots", 1, d, w), slots.numel())


def cache_compact(c, table, lens, refs, table_out, refs_out, page_map, copies, n_copies, stream=None):
    """Moves the used pages to the lowest ids; page_map gives each its new id. Follow with
    cache_copy_pages(copies, n_copies) on every pool (copies: [n_pages // 2 + 1, 3])."""
    w = "dsa_cache_compact"
    if stream is None and _made(_native.cache_compact(c, table, lens, refs, table_out, refs_out, page_map, copies,
                                                      n_copies), w):
        return
    d, n, t, p = _device(table, w, "table"), c.n_seqs, c.n_seqs * c.max_pages, c.n_pages
    _call(lib.dsa_cache_compact, w, d, stream, ctypes.byref(c), _arg(table, "table", _I32, t, d, w),
          _arg(lens, "lens", _I32, n, d, w), _arg(refs, "refs", _I32, p, d, w),
          _arg(table_out, "table_out", _I32, t, d, w), _arg(refs_out, "refs_out", _I32, p, d, w),
          _arg(page_map, "page_map", _I32, p, d, w), _list(copies, "copies", 3 * (p // 2 + 1), d, w),
          _arg(n_copies, "n_copies", _I32, 1, d, w))


def cache_copy_pages(c, pool, copies, n_copies, stream=None):
    """Carries out a copy list on a pool tensor [(layers,) n_pages, page_rows, D] of any type."""
    w = "dsa_cache_copy_pages"
    if stream is None and _made(_native.cache_copy_pages(c, pool, copies, n_copies), w):
        return
    d = _device(pool, w, "pool")
    pl, _, _ = _pool(c, pool, w)
    _call(lib.dsa_cache_copy_pages, w, d, stream, ctypes.byref(c), ctypes.byref(pl), _list(copies, "copies", 3, d, w),
          _arg(n_copies, "n_copies", _I32, 1, d, w), copies.numel() // 3)


def cache_write(c, pool, rows, slots, row_index=None, stream=None):
    """rows [(layers,) n, D] (of the pool's type) to slots [n] of cache_extend; with row_index
    [len(slots)] the row written to slots[i] is rows[row_index[i]]."""
    w = "dsa_cache_write"
    if stream is None and _made(_native.cache_write(c, pool, rows, slots, row_index), w):
        return
    d = _device(pool, w, "pool")
    pl, layers, D = _pool(c, pool, w)
    if _device(rows, w, "rows") != d:
        raise ValueError(f"{w}: rows is on {rows.device}, other tensors on cuda:{d}")
    sh, st = rows.shape, rows.stride()
    if len(sh) == 2:
        sh, st = (1, *sh), (0, *st)
    if len(sh) != 3 or sh[0] != layers or sh[2] != D or rows.dtype is not pool.dtype:
        raise ValueError(f"{w}: rows must be [(layers,) n, D] of the pool's type")
    if (D > 1 and st[2] != 1) or (sh[1] > 1 and st[1] != D):
        raise ValueError(f"{w}: the rows of a layer must be contiguous")
    sp = _list(slots, "slots", 1, d, w)
    n = slots.numel()
    if row_index is None and sh[1] < n:
        raise ValueError(f"{w}: fewer rows than slots")
    _call(lib.dsa_cache_write, w, d, stream, ctypes.byref(c), ctypes.byref(pl), rows.data_ptr(), sh[1],
          st[0] * rows.element_size() if layers > 1 else 0, sp,
          None if row_index is None else _arg(row_index, "row_index", _I32, n, d, w), n)


# ------------------- attention of drafted tokens over the cache -------------------
def make_tree(*, n_tok, H, d_qk, d_v, scale, dtype="bf16", mask_words=0) -> dsa_tree:
    """Sizes of tree_attn_fwd: n_tok drafted tokens of all sequences together."""
    return dsa_tree({"bf16": DSA_BF16, "fp32": DSA_FP32}[dtype], float(scale), n_tok, H, d_qk, d_v, mask_words)


def tree_workspace_size(c, t) -> int:
    return lib.dsa_tree_workspace_size(ctypes.byref(c), ctypes.byref(t))


def tree_attn_fwd(c, t, q, pool, table, lens, kv_new, tok_start, mask, out, softmax_max, softmax_sum, workspace=None,
                  stream=None):
    """Attention of each sequence's drafted tokens (rows tok_start[b] .. tok_start[b+1] of q and
    kv_new) over its cached rows and the drafted ones that mask [n_tok, mask_words] (int64 bits)
    names; mask None: token t sees drafted tokens 0 .. t."""
    w = "dsa_tree_attn_fwd"
    if stream is None and _made(_native.tree_attn_fwd(c, t, q, pool, table, lens, kv_new, tok_start, mask, out,
                                                      softmax_max, softmax_sum, workspace), w):
        return
    dt, f32 = torch.bfloat16 if t.dtype == DSA_BF16 else torch.float32, torch.float32
    d = _device(q, w, "q")
    if _device(pool, w, "pool") != d:
        raise ValueError(f"{w}: pool is on {pool.device}, other tensors on cuda:{d}")
    pl, layers, D = _pool(c, pool, w)
    if pool.dtype is not dt or layers != 1 or D != t.d_qk:
        raise ValueError(f"{w}: pool must be [n_pages, page_rows, d_qk] of the call's type")
    n, rows, n_tok = c.n_seqs, t.n_tok * t.H, t.n_tok
    _call(lib.dsa_tree_attn_fwd, w, d, stream, ctypes.byref(c), ctypes.byref(t),
          _arg(q, "q", dt, rows * D, d, w), ctypes.byref(pl), _arg(table, "table", _I32, n * c.max_pages, d, w),
          _arg(lens, "lens", _I32, n, d, w), _arg(kv_new, "kv_new", dt, n_tok * D, d, w),
          _arg(tok_start, "tok_start", _I32, n + 1, d, w),
          None if mask is None else _arg(mask, "mask", torch.int64, n_tok * t.mask_words, d, w),
          _arg(out, "out", dt, rows * t.d_v, d, w), _arg(softmax_max, "softmax_max", f32, rows, d, w),
          _arg(softmax_sum, "softmax_sum", f32, rows, d, w),
          _workspace(workspace, tree_workspace_size(c, t), d, w))


# ------------------------------ beam selection ------------------------------
def make_beam(*, n_batch, beams_in, beams_out, vocab, ld=None, dtype="bf16", eos=-1) -> dsa_beam:
    """Sizes of beam_select; logits rows are ld >= vocab elements apart (vocab if None)."""
    return dsa_beam({"bf16": DSA_BF16, "fp32": DSA_FP32}[dtype], 0, n_batch, beams_in, beams_out, vocab,
                    vocab if ld is None else ld, eos)


def beam_workspace_size(b) -> int:
    return lib.dsa_beam_workspace_size(ctypes.byref(b))


def beam_select(b, logits, scores, finished, parent, token, scores_out, finished_out, workspace, stream=None):
    """The beams_out best continuations of each request: parent (row of the input, for
    cache_fork), token, score, finished; finished / finished_out (uint8) may be None."""
    w, u8, f32 = "dsa_beam_select", torch.uint8, torch.float32
    if stream is None and _made(_native.beam_select(b, logits, scores, finished, parent, token, scores_out,
                                                    finished_out, workspace), w):
        return
    d, rows, outs = _device(logits, w, "logits"), b.n_batch * b.beams_in, b.n_batch * b.beams_out
    _call(lib.dsa_beam_select, w, d, stream, ctypes.byref(b),
          _arg(logits, "logits", torch.bfloat16 if b.dtype == DSA_BF16 else f32, rows * b.ld, d, w),
          _arg(scores, "scores", f32, rows, d, w),
          None if finished is None else _arg(finished, "finished", u8, rows, d, w),
          _arg(parent, "parent", _I32, outs, d, w), _arg(token, "token", _I32, outs, d, w),
          _arg(scores_out, "scores_out", f32, outs, d, w),
          None if finished_out is None else _arg(finished_out, "finished_out", u8, outs, d, w),
          _workspace(workspace, beam_workspace_size(b), d, w))


# ------------------------------ rotary positions ------------------------------
def rope_part(*, heads, dim, offset=0, layout="interleaved", dtype="bf16") -> dsa_rope_part:
    """One tensor of rope_apply: rows of `heads` heads of `dim` columns, of which rot_dim from `offset` on are rotated;
    layout "interleaved" pairs columns 2i and 2i + 1, "half" i and i + rot_dim / 2."""
    return dsa_rope_part({"bf16": DSA_BF16, "fp32": DSA_FP32}[dtype],
                         {"interleaved": DSA_ROPE_INTERLEAVED, "half": DSA_ROPE_HALF}[layout], heads, dim, offset)


def make_rope(*, rot_dim, parts, base=10000.0, scaling=None, factor=1.0, original=0, beta_fast=32.0, beta_slow=1.0,
              mscale=1.0) -> dsa_rope:
    """Frequencies base^(-2i / rot_dim) and up to four tensors (rope_part) that rope_apply rotates.  scaling, for a
    context `factor` times the trained one: None, "linear", "ntk" or "yarn" (`original`: the trained length)."""
    parts = list(parts)
    if not 1 <= len(parts) <= DSA_ROPE_PARTS:
        raise ValueError(f"make_rope: 1 to {DSA_ROPE_PARTS} parts")
    r = dsa_rope(rot_dim, len(parts), mscale, 0, tuple(parts))
    kind = {None: DSA_ROPE_PLAIN, "linear": DSA_ROPE_LINEAR, "ntk": DSA_ROPE_NTK, "yarn": DSA_ROPE_YARN}[scaling]
    _chk(lib.dsa_rope_steps(ctypes.byref(r), base, kind, factor, original, beta_fast, beta_slow), "dsa_rope_steps")
    return r


def _rope_rows(t, name, part, n_tok, device, where):
    """dsa_rope_rows of a tensor [..., heads, dim] ([..., dim] with one head) whose leading dimensions are n_tok rows at
    one stride."""
    dt = torch.bfloat16 if part.dtype == DSA_BF16 else torch.float32
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.get_device() != device or t.dtype is not dt:
        _refuse(where, name, t, dt, 0, device, at_least=True)
        raise TypeError(f"{where}: {name} is {t.dtype}, needs {dt}")
    sh, st = list(t.shape), list(t.stride())
    if not sh or sh[-1] != part.dim or (part.dim > 1 and st[-1] != 1):
        raise ValueError(f"{where}: {name} must have {part.dim} contiguous columns")
    sh, st, head = sh[:-1], st[:-1], 0
    if part.heads > 1:
        if not sh or sh[-1] != part.heads:
            raise ValueError(f"{where}: {name} must be [..., {part.heads}, {part.dim}]")
        head, sh, st = st[-1], sh[:-1], st[:-1]
    n, tok = 1, 0
    for size, stride in zip(reversed(sh), reversed(st)):
        if size == 1:
            continue
        if n == 1:
            tok = stride
        elif stride != tok * n:
            raise ValueError(f"{where}: the tokens of {name} must lie at one stride")
        n *= size
    if n != n_tok:
        raise ValueError(f"{where}: {name} has {n} tokens, pos {n_tok}")
    return dsa_rope_rows(t.data_ptr(), tok, head)


def rope_apply(r, pos, x, out=None, transposed=False, stream=None):
    """Rotates the tensors x (one per part of r, [..., heads, dim]) of the tokens at pos (int32) into out (None: in
    place); transposed: gradients of the results into gradients of the inputs."""
    w = "dsa_rope_apply"
    out = x if out is None else out
    if stream is None and _made(_native.rope_apply(r, pos, x, out, transposed), w):
        return
    d = _device(pos, w, "pos")
    n = pos.numel()
    if len(x) != r.n_parts or len(out) != r.n_parts:
        raise ValueError(f"{w}: x and out must have {r.n_parts} tensors")
    rows = [(dsa_rope_rows * r.n_parts)(*(_rope_rows(t, f"{name}[{i}]", r.part[i], n, d, w) for i, t in enumerate(ts)))
            for name, ts in (("x", x), ("out", out))]
    _call(lib.dsa_rope_apply, w, d, stream, ctypes.byref(r), n, _arg(pos, "pos", _I32, n, d, w), *rows,
          int(bool(transposed)))


# ---------------------------------- sampling ----------------------------------
def make_sampler(*, rows, vocab, ld=None, dtype="bf16", requests=None) -> dsa_sampler:
    """Sizes of sample; logits rows are ld >= vocab elements apart (vocab if None).  requests: how many settings there
    are, if not one per row."""
    return dsa_sampler({"bf16": DSA_BF16, "fp32": DSA_FP32}[dtype], 0, rows, vocab, vocab if ld is None else ld,
                       rows if requests is None else requests)


def sample(s, logits, u, temperature, top_k, top_p, min_p, index, token, prob=None, stream=None):
    """A token per row of logits by the uniform numbers u, and its probability.  Settings [requests] fp32 (top_k int32)
    or None; row r has those of index[r] (int32), of r without an index."""
    w, f32 = "dsa_sample", torch.float32
    if stream is None and _made(_native.sample(s, logits, u, temperature, top_k, top_p, min_p, index, token, prob), w):
        return
    d, n, m = _device(logits, w, "logits"), s.rows, s.requests
    setting = lambda t, name, dt: None if t is None else _arg(t, name, dt, m, d, w)
    _call(lib.dsa_sample, w, d, stream, ctypes.byref(s),
          _arg(logits, "logits", torch.bfloat16 if s.dtype == DSA_BF16 else f32, n * s.ld, d, w),
          _arg(u, "u", f32, n, d, w), setting(temperature, "temperature", f32), setting(top_k, "top_k", _I32),
          setting(top_p, "top_p", f32), setting(min_p, "min_p", f32),
          None if index is None else _arg(index, "index", _I32, n, d, w), _arg(token, "token", _I32, n, d, w),
          None if prob is None else _arg(prob, "prob", f32, n, d, w))


# ------------------------ acceptance of drafted tokens ------------------------
def tree_accept(c, t, tok_start, mask, drafted, sampled, n_new, row_index, tokens, next_token, eos=-1, stream=None):
    """Which drafted tokens of tree_attn_fwd each sequence keeps, given the tokens sampled at each: n_new (for
    cache_extend), row_index [n_tok] (for cache_write, -1 behind the last), tokens [n_tok] (what was gained) and
    next_token (each sequence's last)."""
    w = "dsa_tree_accept"
    if stream is None and _made(_native.tree_accept(c, t, tok_start, mask, drafted, sampled, n_new, row_index, tokens,
                                                    next_token, eos), w):
        return
    d, n, n_tok = _device(tok_start, w, "tok_start"), c.n_seqs, t.n_tok
    _call(lib.dsa_tree_accept, w, d, stream, ctypes.byref(c), ctypes.byref(t),
          _arg(tok_start, "tok_start", _I32, n + 1, d, w),
          None if mask is None else _arg(mask, "mask", torch.int64, n_tok * t.mask_words, d, w),
          _arg(drafted, "drafted", _I32, n_tok, d, w), _arg(sampled, "sampled", _I32, n_tok, d, w), eos,
          _arg(n_new, "n_new", _I32, n, d, w), _arg(row_index, "row_index", _I32, n_tok, d, w),
          _arg(tokens, "tokens", _I32, n_tok, d, w), _arg(next_token, "next_token", _I32, n, d, w))


def get_status(stream=None) -> int:
    v = ctypes.c_int(0)
    _chk(lib.dsa_get_status(_stream(stream), ctypes.byref(v)), "dsa_get_status")
    return v.value


def set_wait_budget_ns(ns: int):
    _chk(lib.dsa_set_wait_budget_ns(int(ns)), "dsa_set_wait_budget_ns")


def selftest_wait_timeout(ns: int, stream=None):
    _chk(lib.dsa_selftest_wait_timeout(int(ns), _stream(stream)), "dsa_selftest_wait_timeout")
