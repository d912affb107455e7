"""ctypes binding of ``include/dls.h`` (argument marshalling only).

Every step of the decode path runs in the CUDA library; this module only
passes pointers and sizes.  If the library is missing or fails to load it
raises: there is no fallback.  PyTorch supplies device memory (through the
allocator callbacks) and streams.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import numpy as np

from . import _build

_lock = threading.Lock()
_lib = None

DLS_OK, DLS_ERR_ARG, DLS_ERR_BUDGET, DLS_ERR_CAPACITY, DLS_ERR_CUDA, DLS_ERR_TIMEOUT, DLS_ERR_STATE = 0, -1, -2, -3, -4, -5, -6
DLS_Q4_0, DLS_Q8_0 = 4, 8
TENSOR_IDS = {"wq": 0, "wk": 1, "wv": 2, "wo": 3, "w_gate": 4, "w_up": 5, "w_down": 6, "tok_embd": 7, "output": 8}

i32, u64, vp, sz = ctypes.c_int32, ctypes.c_uint64, ctypes.c_void_p, ctypes.c_size_t


class DlsError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(msg)
        self.code = code


class dls_allocator(ctypes.Structure):
    _fields_ = [("alloc", ctypes.CFUNCTYPE(vp, vp, sz, vp)),
                ("free", ctypes.CFUNCTYPE(None, vp, vp, vp)),
                ("ctx", vp)]


class dls_layer_desc(ctypes.Structure):
    _fields_ = [(n, vp) for n in ("attn_norm", "ffn_norm", "wq", "wk", "wv", "wo", "w_gate", "w_up", "w_down")] + \
               [("types", i32 * 7)]


class dls_model_desc(ctypes.Structure):
    _fields_ = [("n_layers", i32), ("hidden", i32), ("n_heads", i32), ("n_kv_heads", i32), ("head_dim", i32),
                ("ffn", i32), ("vocab", i32), ("rope_theta", ctypes.c_float), ("rms_eps", ctypes.c_float),
                ("tied_embeddings", i32), ("wtype", i32), ("page_tokens", i32), ("max_seqs", i32),
                ("max_ctx", i32), ("max_batch", i32), ("device_budget_bytes", u64), ("tok_embd", vp),
                ("output", vp), ("output_norm", vp), ("layers", ctypes.POINTER(dls_layer_desc)),
                ("kv_pool_pages", i32), ("tok_embd_type", i32), ("output_type", i32)]


_SIGS = {
    "dls_abi_version": (ctypes.c_int, []),
    "dls_status_name": (ctypes.c_char_p, [ctypes.c_int]),
    "dls_last_error": (ctypes.c_char_p, [vp]),
    "dls_model_create": (ctypes.c_int, [ctypes.POINTER(dls_model_desc), ctypes.POINTER(dls_allocator), vp,
                                        ctypes.POINTER(vp)]),
    "dls_model_destroy": (None, [vp]),
    "dls_device_bytes": (u64, [vp]),
    "dls_device_budget": (u64, [vp]),
    "dls_seq_create": (ctypes.c_int, [vp, ctypes.POINTER(i32)]),
    "dls_seq_free": (ctypes.c_int, [vp, i32]),
    "dls_seq_length": (i32, [vp, i32]),
    "dls_prefill": (ctypes.c_int, [vp, i32, vp, i32, vp]),
    "dls_decode_step": (ctypes.c_int, [vp, i32, i32, i32, vp]),
    "dls_decode_batch": (ctypes.c_int, [vp, i32, vp, vp, vp, vp]),
    "dls_generate": (ctypes.c_int, [vp, i32, vp, vp, i32, vp, vp]),
    "dls_argmax": (ctypes.c_int, [vp, vp, i32, vp]),
    "dls_kv_fork": (ctypes.c_int, [vp, i32, vp, i32]),
    "dls_kv_fork_shared": (ctypes.c_int, [vp, i32, vp, i32]),
    "dls_kv_free_pages": (i32, [vp]),
    "dls_set_layer_skip": (ctypes.c_int, [vp, vp, i32]),
    "dls_layer_cosines": (ctypes.c_int, [vp, i32, i32, i32, vp]),
    "dls_seq_truncate": (ctypes.c_int, [vp, i32, i32]),
    "dls_verify": (ctypes.c_int, [vp, i32, vp, i32, vp, vp]),
    "dls_generate_speculative": (ctypes.c_int, [vp, i32, i32, i32, vp, i32, vp, vp]),
    "dls_check_context_budget": (ctypes.c_int, [i32, i32, i32, i32]),
    "dls_h2d_copy_sm": (ctypes.c_int, [vp, vp, sz, i32, vp]),
    "dls_set_resident_layers": (ctypes.c_int, [vp, i32]),
    "dls_resident_layers": (i32, [vp]),
    "dls_layer_bytes": (u64, [vp]),
    "dls_attention_decode": (ctypes.c_int, [vp, vp, vp, vp, vp, vp, vp, sz, i32, i32, i32, i32, i32, i32, i32, vp, vp]),
    "dls_attention_status": (ctypes.c_int, [vp, vp]),
    "dls_attention_workspace_bytes": (sz, [i32, i32, i32, i32, i32]),
    "dls_attention_decode_noalloc": (ctypes.c_int, [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, vp, vp]),
    "dls_qk_norm_rope": (ctypes.c_int, [vp, vp]),
    "dls_kv_append": (ctypes.c_int, [vp, vp]),
    "dls_attention_chunk": (ctypes.c_int, [vp, vp]),
    "dls_attention_chunk_workspace_bytes": (ctypes.c_uint64, [i32]),
    "dls_kv_reserve": (ctypes.c_int, [vp, vp]),
    "dls_kv_append8": (ctypes.c_int, [vp, vp]),
    "dls_attention_chunk8": (ctypes.c_int, [vp, vp]),
    "dls_verify_draft": (ctypes.c_int, [vp, vp]),
    "dls_kquant_packed_bytes": (ctypes.c_uint64, [i32, i32, i32]),
    "dls_kquant_pack": (ctypes.c_int, [i32, vp, i32, i32, vp, vp]),
    "dls_kquant_gemv": (ctypes.c_int, [i32, vp, i32, i32, vp, vp, vp, vp]),
    "dls_debug_capture": (ctypes.c_int, [vp, vp]),
    "dls_debug_read_kv": (ctypes.c_int, [vp, i32, i32, vp, vp]),
    "dls_debug_bounded_wait": (ctypes.c_int, [vp, ctypes.c_int64]),
    "dls_debug_dequant": (ctypes.c_int, [vp, i32, i32, vp]),
    "dls_debug_gemv": (ctypes.c_int, [vp, i32, i32, vp, vp]),
    "dls_debug_gemm": (ctypes.c_int, [vp, i32, i32, i32, vp, vp]),
    "dls_debug_launches_per_step": (i32, [vp]),
    "dls_debug_profile_step": (ctypes.c_int, [vp, i32, i32, i32, i32, vp, vp, vp]),
    "dls_debug_step_trace": (ctypes.c_int, [vp, vp, i32, vp]),
    "dls_step_kernel_in_use": (i32, [vp, vp]),
    "dls_debug_profile_batch": (ctypes.c_int, [vp, i32, vp, vp, vp, i32, vp, vp, vp]),
}


def exported_symbols():
    """Names the header declares (the binding's contract)."""
    return sorted(_SIGS)


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True):
    """Load the CUDA library (building it first if needed)."""
    global _lib
    with _lock:
        if _lib is None:
            if build_if_missing and not _build.up_to_date():
                _build.build()
            if not os.path.exists(_build.LIB):
                raise RuntimeError(f"decode-step CUDA library missing: {_build.LIB}")
            lib = ctypes.CDLL(_build.LIB)
            for name, (res, args) in _SIGS.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def _ptr(obj):
    """Device or host pointer of a torch tensor / numpy array / int / None."""
    if obj is None:
        return None
    if isinstance(obj, int):
        return obj
    if isinstance(obj, np.ndarray):
        if not obj.flags["C_CONTIGUOUS"]:
            raise ValueError("array must be C-contiguous")
        return obj.ctypes.data
    if hasattr(obj, "data_ptr"):
        if not obj.is_contiguous():
            raise ValueError("tensor must be contiguous")
        return obj.data_ptr()
    raise TypeError(f"cannot pass {type(obj)} as a pointer")


def _check(rc: int, model_handle=None):
    if rc != DLS_OK:
        lib = load(False)
        msg = lib.dls_last_error(model_handle).decode(errors="replace")
        raise DlsError(rc, msg or lib.dls_status_name(rc).decode())


def status_name(code: int) -> str:
    return load().dls_status_name(code).decode()


def h2d_copy_sm(dst, src_host, nbytes: int, ctas: int = 64, stream=None):
    """Copy pinned host memory to the device with an SM-driven kernel."""
    _check(load().dls_h2d_copy_sm(_ptr(dst), _ptr(src_host), int(nbytes), int(ctas), _stream_handle(stream)))


def check_context_budget(prefix_tokens: int, max_branch_tokens: int, headroom: int, n_ctx: int) -> None:
    _check(load().dls_check_context_budget(prefix_tokens, max_branch_tokens, headroom, n_ctx))


def attention_workspace_bytes(n_batch, n_heads, n_kv_heads, head_dim, n_splits) -> int:
    return int(load().dls_attention_workspace_bytes(n_batch, n_heads, n_kv_heads, head_dim, n_splits))


def attention_decode(q, k_pages, v_pages, page_table, lengths, o, workspace, workspace_bytes, n_batch, n_heads,
                     n_kv_heads, head_dim, page_tokens, max_pages, n_splits=0, status=None, stream=None):
    """Split-K GQA decode attention over a paged fp16 cache (device buffers).
    ``status``: optional device int32[1] the kernel reports into; read it
    with attention_status()."""
    _check(load().dls_attention_decode(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table), _ptr(lengths),
                                       _ptr(o), _ptr(workspace), workspace_bytes, n_batch, n_heads, n_kv_heads,
                                       head_dim, page_tokens, max_pages, n_splits, _ptr(status),
                                       _stream_handle(stream)))


def attention_status(status, stream=None):
    """Wait for the stream and raise DlsError (DLS_ERR_STATE or
    DLS_ERR_TIMEOUT) if the attention kernel flagged its status word."""
    _check(load().dls_attention_status(_ptr(status), _stream_handle(stream)))


NOALLOC_SCRATCH_BYTES = 4 << 20  # DLS_ATTENTION_NOALLOC_SCRATCH_BYTES


def attention_decode_noalloc(q, k_pages, v_pages, page_table, lengths, o, n_batch, n_heads, n_kv_heads, head_dim,
                             page_tokens, max_pages, n_splits=0, status=None, stream=None):
    """dls_attention_decode without a workspace: for callers that may not
    allocate device memory; the scratch is a fixed array in the library."""
    _check(load().dls_attention_decode_noalloc(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table),
                                               _ptr(lengths), _ptr(o), n_batch, n_heads, n_kv_heads, head_dim,
                                               page_tokens, max_pages, n_splits, _ptr(status),
                                               _stream_handle(stream)))


# --- the paged cache: filling it and attending over it
# (stream None is the default stream, as everywhere here: under torch.cuda.stream(s) or a capture pass that stream)

DLS_F32, DLS_F16, DLS_BF16 = 1, 2, 3
ROPE_PAIRINGS = {"adjacent": 0, "halves": 1}
# the header's descriptors, packed in one go (native sizes and alignment)
_QK_NORM_ROPE = struct.Struct("@4P4q4P8if")
_KV_APPEND = struct.Struct("@6P4q2P5P12if")
_ATTENTION_CHUNK = struct.Struct("@8PPQP2q11if")
_torch = None
_dtypes = {}


def _types():
    """torch's types by the header's numbers; torch is imported with the first call."""
    global _torch
    import torch

    _torch = torch
    _dtypes.update({torch.float32: DLS_F32, torch.float16: DLS_F16, torch.bfloat16: DLS_BF16})
    return _dtypes


def _dtype(t, name):
    typ = (_dtypes or _types()).get(t.dtype)
    if typ is None:
        raise ValueError(f"{name}: type {t.dtype} (float32, float16 or bfloat16)")
    return typ


def _rows(t, name, n, heads, hd, dtype, device):
    """(pointer, elements between tokens) of a [n, heads, hd] tensor whose rows are contiguous.  These checks run
    before every launch, which itself takes a few microseconds: few calls into torch, and no strings before an error."""
    shape, stride = t.shape, t.stride()
    if shape != (n, heads, hd):
        raise ValueError(f"{name}: shape {tuple(shape)}, wanted {(n, heads, hd)} ([tokens, heads, head_dim])")
    if t.dtype != dtype:
        raise ValueError(f"{name}: type {t.dtype}, wanted {dtype}")
    if (stride[2] != 1 and hd > 1) or (stride[1] != hd and heads > 1):
        raise ValueError(f"{name}: a token's heads must be contiguous (strides {stride})")
    if t.get_device() != device:
        raise ValueError(f"{name}: on {t.device}: all tensors must be on one CUDA device")
    return t.data_ptr(), (stride[0] if n > 1 else heads * hd)


def _array(t, name, dtype, shape, device):
    """Pointer of a contiguous tensor of the given type and shape; None -> 0."""
    if t is None:
        return 0
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)}, wanted contiguous {dtype} {shape}")
    if t.get_device() != device:
        raise ValueError(f"{name}: on {t.device}: all tensors must be on one CUDA device")
    return t.data_ptr()


def _dims(t, name):
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name}: shape {tuple(shape)} ([tokens, heads, head_dim])")
    return shape


def _call(fn, desc, stream, device):
    """One library call on the tensors' own device."""
    if device < 0:
        raise ValueError("all tensors must be on one CUDA device")
    if _torch.cuda.current_device() == device:
        _check(fn(desc, _stream_handle(stream)))
    else:
        with _torch.cuda.device(device):
            _check(fn(desc, _stream_handle(stream)))


def _pairing(name):
    number = ROPE_PAIRINGS.get(name)
    if number is None:
        raise ValueError(f"pairing: {name!r} ({' or '.join(ROPE_PAIRINGS)})")
    return number


def _inv_freq(inv_freq):
    """(array to keep, pointer, rot_dim) of host frequencies."""
    if inv_freq is None:
        return None, 0, 0
    a = np.ascontiguousarray(inv_freq, dtype=np.float64)
    if a.ndim != 1:
        raise ValueError(f"inv_freq: shape {a.shape} ([rot_dim / 2])")
    try:
        at = ctypes.addressof(ctypes.c_char.from_buffer(a))  # a third of what __array_interface__ takes
    except (TypeError, ValueError):                          # read-only, or empty
        at = a.__array_interface__["data"][0]
    return a, at, 2 * a.size


def _pools(k_pages, v_pages, page_table, cu_q, kv_len, device):
    """Shapes and pointers of the cache and the batch: (pages, KV heads, page tokens, head_dim, k and v pointers, table
    pointer, entries of a sequence, cu_q and kv_len pointers, sequences)."""
    shape = k_pages.shape
    if len(shape) != 4 or v_pages.shape != shape or k_pages.dtype != v_pages.dtype:
        raise ValueError(f"k_pages {tuple(k_pages.shape)} {k_pages.dtype}, v_pages {tuple(v_pages.shape)} {v_pages.dtype}: "
                         "one [pages, kv_heads, page_tokens, head_dim] and type wanted")
    if not k_pages.is_contiguous() or not v_pages.is_contiguous():
        raise ValueError("k_pages and v_pages must be contiguous")
    if k_pages.get_device() != device or v_pages.get_device() != device:
        raise ValueError(f"k_pages on {k_pages.device}, v_pages on {v_pages.device}: all tensors must be on one CUDA device")
    if page_table.dim() != 2:
        raise ValueError(f"page_table: shape {tuple(page_table.shape)} ([sequences, pages])")
    n, most = page_table.shape
    i32_ = _torch.int32
    return (*shape, k_pages.data_ptr(), v_pages.data_ptr(), _array(page_table, "page_table", i32_, (n, most), device), most,
            _array(cu_q, "cu_q", i32_, (n + 1,), device), _array(kv_len, "kv_len", i32_, (n,), device), n)


def rope_inv_freq(rot_dim: int, theta: float) -> np.ndarray:
    """theta^(-2 i / rot_dim), radians per position: the frequencies of the model's own decode path."""
    return float(theta) ** (-np.arange(0, rot_dim, 2, dtype=np.float64) / rot_dim)


def qk_norm_rope(q, k, positions, inv_freq, q_out, k_out, *, q_norm=None, k_norm=None, eps=1e-5, pairing="adjacent",
                 stream=None):
    """Per-head RMSNorm (where a norm is given) and rotation of q and k [tokens, heads, head_dim] into q_out and
    k_out, which may be q and k themselves.  Either pair may be None.  positions: device int32 [tokens]; inv_freq:
    host float64 [rot_dim / 2], or None for no rotation.  stream None is the default stream, whatever torch's current
    one is: under torch.cuda.stream(s) or a capture pass that stream."""
    one, one_out = (q, q_out) if q is not None else (k, k_out)
    if one is None or (q is None) != (q_out is None) or (k is None) != (k_out is None):
        raise ValueError("q with q_out, k with k_out, or both")
    n, _, hd = _dims(one, "q" if q is not None else "k")
    typ, out, device = _dtype(one, "q"), _dtype(one_out, "q_out"), one.get_device()
    tin, tout, f32 = one.dtype, one_out.dtype, _torch.float32
    qp = qs = qop = qos = qh = kp = ks = kop = kos = kh = 0
    if q is not None:
        qh = q.shape[1]
        qp, qs = _rows(q, "q", n, qh, hd, tin, device)
        qop, qos = _rows(q_out, "q_out", n, qh, hd, tout, device)
    if k is not None:
        kh = _dims(k, "k")[1]
        kp, ks = _rows(k, "k", n, kh, hd, tin, device)
        kop, kos = _rows(k_out, "k_out", n, kh, hd, tout, device)
    keep, fp, rot = _inv_freq(inv_freq)
    desc = _QK_NORM_ROPE.pack(qp, kp, qop, kop, qs, ks, qos, kos, _array(q_norm, "q_norm", f32, (hd,), device),
                              _array(k_norm, "k_norm", f32, (hd,), device),
                              _array(positions, "positions", _torch.int32, (n,), device), fp, n, qh, kh, hd, rot,
                              _pairing(pairing), typ, out, eps)
    _call((_lib or load()).dls_qk_norm_rope, desc, stream, device)


def kv_append(k, v, k_pages, v_pages, page_table, cu_q, kv_len, inv_freq, *, q=None, q_out=None, q_norm=None, k_norm=None,
              eps=1e-5, pairing="adjacent", status=None, stream=None):
    """Append a ragged chunk's keys (normed where k_norm is given, rotated by their cache position) and values
    [tokens, kv_heads, head_dim] to the pages; with q, q_out = q normed and rotated in the same pass, in the
    cache's type; q_out may be q where it has that type.  cu_q: device int32 [sequences + 1], kv_len: device int32
    [sequences], the new tokens counted.  stream None is the default stream, as in qk_norm_rope."""
    if (q is None) != (q_out is None):
        raise ValueError("q with q_out, or neither")
    typ, kv_type, device = _dtype(k, "k"), _dtype(k_pages, "k_pages"), k.get_device()
    pages, kvh, pt, hd, kpp, vpp, table, most, cu, kl, seqs = _pools(k_pages, v_pages, page_table, cu_q, kv_len, device)
    n, tin, f32 = _dims(k, "k")[0], k.dtype, _torch.float32
    kp, ks = _rows(k, "k", n, kvh, hd, tin, device)
    vptr, vs = _rows(v, "v", n, kvh, hd, tin, device)
    qp = qs = qop = qos = qh = 0
    if q is not None:
        qh = _dims(q, "q")[1]
        qp, qs = _rows(q, "q", n, qh, hd, tin, device)
        qop, qos = _rows(q_out, "q_out", n, qh, hd, k_pages.dtype, device)
    keep, fp, rot = _inv_freq(inv_freq)
    desc = _KV_APPEND.pack(kp, vptr, qp, kpp, vpp, qop, ks, vs, qs, qos, _array(k_norm, "k_norm", f32, (hd,), device),
                           _array(q_norm, "q_norm", f32, (hd,), device), table, cu, kl, fp,
                           _array(status, "status", _torch.int32, (1,), device), n, seqs, qh, kvh, hd, rot,
                           _pairing(pairing), typ, kv_type, pt, pages, most, eps)
    _call((_lib or load()).dls_kv_append, desc, stream, device)


def attention_chunk_workspace_bytes(head_dim: int) -> int:
    return int(load().dls_attention_chunk_workspace_bytes(head_dim))


def attention_chunk(q, k_pages, v_pages, page_table, cu_q, kv_len, o, workspace, *, lse=None, scale=0.0, causal=True,
                    window=0, status=None, stream=None):
    """Attention of ragged chunks of new tokens (q, o [tokens, heads, head_dim] in the cache's type) over the paged
    cache; o may be q.  workspace: a uint8 tensor of attention_chunk_workspace_bytes(head_dim) zeros, kept from call to
    call, one for each of the calls that may overlap.  lse: fp32 [tokens, heads] or None.  scale 0: 1 / sqrt(head_dim).
    stream None is the default stream, as in qk_norm_rope."""
    kv_type, device = _dtype(k_pages, "k_pages"), q.get_device()
    pages, kvh, pt, hd, kpp, vpp, table, most, cu, kl, seqs = _pools(k_pages, v_pages, page_table, cu_q, kv_len, device)
    n, heads, _ = _dims(q, "q")
    qp, qs = _rows(q, "q", n, heads, hd, k_pages.dtype, device)
    op, os_ = _rows(o, "o", n, heads, hd, k_pages.dtype, device)
    if not workspace.is_contiguous() or workspace.get_device() != device:
        raise ValueError(f"workspace: on {workspace.device}: contiguous, and all tensors on one CUDA device")
    desc = _ATTENTION_CHUNK.pack(qp, kpp, vpp, table, cu, kl, op, _array(lse, "lse", _torch.float32, (n, heads), device),
                                 workspace.data_ptr(), workspace.nbytes,
                                 _array(status, "status", _torch.int32, (1,), device), qs, os_, n, seqs, heads, kvh, hd, pt,
                                 pages, most, kv_type, 1 if causal else 0, window, scale)
    _call((_lib or load()).dls_attention_chunk, desc, stream, device)


# --- the paged cache in 8 bits, and a step whose lengths stay on the device

DLS_E4M3, DLS_I8 = 4, 5
_KV_RESERVE = struct.Struct("@14P5i")
_KV_APPEND8 = struct.Struct("@6P2q6P12if")
_ATTENTION_CHUNK8 = struct.Struct("@11PQP2q13if")
_VERIFY_DRAFT = struct.Struct("@11P2q4i")
_code_types = {}


def _codes(k_pages, v_pages, k_scales, v_scales, device):
    """(code type, block_tokens, scales' pointers) of pools of codes."""
    if not _code_types:
        _types()
        _code_types.update({_torch.float8_e4m3fn: DLS_E4M3, _torch.int8: DLS_I8})
    code, shape, grid = _code_types.get(k_pages.dtype), k_pages.shape, k_scales.shape
    if code is None:
        raise ValueError(f"k_pages: type {k_pages.dtype} (float8_e4m3fn or int8)")
    if len(shape) != 4 or len(grid) != 3 or grid[:2] != shape[:2] or not grid[2] or shape[2] % grid[2]:
        raise ValueError(f"k_scales: shape {tuple(grid)} ([pages, kv_heads, page_tokens / block_tokens] of pages {tuple(shape)})")
    f32 = _torch.float32
    return (code, shape[2] // grid[2], _array(k_scales, "k_scales", f32, grid, device),
            _array(v_scales, "v_scales", f32, grid, device))


def kv_reserve(new_len, kv_len, held, page_table, free_pages, free_count, kv_len_out, held_out, free_count_out, cu_q,
               page_tokens, *, positions=None, slots=None, seq_ids=None, max_rows=None, status=None, stream=None):
    """Pages and rows of a batch from its requests' lengths (device int32 [sequences]): new_len tokens join kv_len ones
    (negative: the request is over, its pages go back on the stack free_pages, whose free_count lowest entries are
    free; in place, one in a state that cannot be keeps it).  Fresh pages go into page_table [sequences, pages], rows into
    cu_q [sequences + 1] and, where given, positions, slots (page * page_tokens + offset) and seq_ids [rows].  kv_len_out,
    held_out and free_count_out may be their inputs.  max_rows: the arrays' length where one is given.  stream None is
    the default stream, as in qk_norm_rope."""
    _dtypes or _types()
    i32_, device = _torch.int32, new_len.get_device()
    if page_table.dim() != 2:
        raise ValueError(f"page_table: shape {tuple(page_table.shape)} ([sequences, pages])")
    n, most = page_table.shape
    one = positions if positions is not None else slots if slots is not None else seq_ids
    if one is not None:
        if max_rows is None:
            max_rows = one.shape[0]
        elif max_rows > one.shape[0]:
            raise ValueError(f"max_rows: {max_rows}, the arrays hold {one.shape[0]}")
        rows = tuple(one.shape)
    else:
        rows = ()
        if max_rows is None:
            raise ValueError("max_rows, or one of positions, slots and seq_ids")
    if free_pages.dim() != 1:
        raise ValueError(f"free_pages: shape {tuple(free_pages.shape)} ([pages])")
    pages = free_pages.shape[0]
    desc = _KV_RESERVE.pack(
        _array(new_len, "new_len", i32_, (n,), device), _array(kv_len, "kv_len", i32_, (n,), device),
        _array(held, "held", i32_, (n,), device), _array(page_table, "page_table", i32_, (n, most), device),
        _array(free_pages, "free_pages", i32_, (pages,), device), _array(free_count, "free_count", i32_, (1,), device),
        _array(kv_len_out, "kv_len_out", i32_, (n,), device), _array(held_out, "held_out", i32_, (n,), device),
        _array(free_count_out, "free_count_out", i32_, (1,), device), _array(cu_q, "cu_q", i32_, (n + 1,), device),
        _array(positions, "positions", i32_, rows, device), _array(slots, "slots", i32_, rows, device),
        _array(seq_ids, "seq_ids", i32_, rows, device), _array(status, "status", i32_, (1,), device), n, max_rows,
        page_tokens, pages, most)
    _call((_lib or load()).dls_kv_reserve, desc, stream, device)


def kv_append8(k, v, k_pages, v_pages, k_scales, v_scales, page_table, cu_q, kv_len, inv_freq, *, k_norm=None, eps=1e-5,
               pairing="adjacent", status=None, stream=None):
    """Append a ragged chunk's keys (normed where k_norm is given, rotated by their cache position) and values
    [tokens, kv_heads, head_dim] to pages of codes (float8_e4m3fn or int8), with a scale for each block of tokens and
    head: k_scales and v_scales, fp32 [pages, kv_heads, page_tokens / block_tokens].  cu_q: device int32
    [sequences + 1], kv_len: device int32 [sequences], the new tokens counted.  stream None is the default stream, as
    in qk_norm_rope."""
    typ, device = _dtype(k, "k"), k.get_device()
    code, block, ksp, vsp = _codes(k_pages, v_pages, k_scales, v_scales, device)
    pages, kvh, pt, hd, kpp, vpp, table, most, cu, kl, seqs = _pools(k_pages, v_pages, page_table, cu_q, kv_len, device)
    n, tin = _dims(k, "k")[0], k.dtype
    kp, ks = _rows(k, "k", n, kvh, hd, tin, device)
    vptr, vs = _rows(v, "v", n, kvh, hd, tin, device)
    keep, fp, rot = _inv_freq(inv_freq)
    desc = _KV_APPEND8.pack(kp, vptr, kpp, vpp, ksp, vsp, ks, vs, _array(k_norm, "k_norm", _torch.float32, (hd,), device),
                            table, cu, kl, fp, _array(status, "status", _torch.int32, (1,), device), n, seqs, kvh, hd, rot,
                            _pairing(pairing), typ, code, pt, block, pages, most, eps)
    _call((_lib or load()).dls_kv_append8, desc, stream, device)


def attention_chunk8(q, k_pages, v_pages, k_scales, v_scales, page_table, cu_q, kv_len, o, workspace, *, lse=None, scale=0.0,
                     causal=True, window=0, status=None, stream=None):
    """attention_chunk over pages of codes (float8_e4m3fn or int8) with a scale for each block of tokens and head; q and
    o [tokens, heads, head_dim] in float16 or bfloat16.  workspace: as attention_chunk's, which may be the same one.  A
    batch of single tokens and long chunks does better as a call for each kind of sequence (parts of page_table, cu_q and
    kv_len; q and o up to the kind's last row)."""
    typ, device = _dtype(q, "q"), q.get_device()
    code, block, ksp, vsp = _codes(k_pages, v_pages, k_scales, v_scales, device)
    pages, kvh, pt, hd, kpp, vpp, table, most, cu, kl, seqs = _pools(k_pages, v_pages, page_table, cu_q, kv_len, device)
    n, heads, _ = _dims(q, "q")
    qp, qs = _rows(q, "q", n, heads, hd, q.dtype, device)
    op, os_ = _rows(o, "o", n, heads, hd, q.dtype, device)
    if not workspace.is_contiguous() or workspace.get_device() != device:
        raise ValueError(f"workspace: on {workspace.device}: contiguous, and all tensors on one CUDA device")
    desc = _ATTENTION_CHUNK8.pack(qp, kpp, vpp, ksp, vsp, table, cu, kl, op,
                                  _array(lse, "lse", _torch.float32, (n, heads), device), workspace.data_ptr(),
                                  workspace.nbytes, _array(status, "status", _torch.int32, (1,), device), qs, os_, n, seqs,
                                  heads, kvh, hd, pt, block, pages, most, typ, code, 1 if causal else 0, window, scale)
    _call((_lib or load()).dls_attention_chunk8, desc, stream, device)


def _prob_rows(t, name, n, vocab, dtype, device):
    """(pointer, elements between rows) of probabilities [n, vocab] whose rows are contiguous; None -> (0, 0)."""
    if t is None:
        return 0, 0
    shape, stride = t.shape, t.stride()
    if shape != (n, vocab) or t.dtype != dtype:
        raise ValueError(f"{name}: {t.dtype} {tuple(shape)}, wanted {dtype} {(n, vocab)}")
    if stride[1] != 1 and vocab > 1:
        raise ValueError(f"{name}: a row's probabilities must be contiguous (strides {stride})")
    if t.get_device() != device:
        raise ValueError(f"{name}: on {t.device}: all tensors must be on one CUDA device")
    return t.data_ptr(), (stride[0] if n > 1 else vocab)


def verify_draft(tokens, target, cu_q, accept, pick, out_tokens, n_accepted, *, draft=None, kv_len=None, kv_len_out=None,
                 status=None, stream=None):
    """Drafted tokens against the target's probabilities [rows, vocab] (float32, float16 or bfloat16), from given random
    numbers: accept fp32 [rows], pick fp32 [sequences].  tokens, out_tokens: int32 [rows], a sequence's rows its current
    token and its drafts; draft: the probabilities that row r + 1's token was drawn from in row r, None for certain
    ones.  n_accepted: int32 [sequences]; kv_len_out (may be kv_len) = kv_len less the drafts that do not stand."""
    if len(target.shape) != 2:
        raise ValueError(f"target: shape {tuple(target.shape)} ([rows, vocab])")
    typ, device = _dtype(target, "target"), target.get_device()
    n, vocab = target.shape
    seqs = n_accepted.shape[0] if n_accepted.dim() == 1 else -1
    i32_, f32 = _torch.int32, _torch.float32
    tp, ts = _prob_rows(target, "target", n, vocab, target.dtype, device)
    dp, ds = _prob_rows(draft, "draft", n, vocab, target.dtype, device)
    desc = _VERIFY_DRAFT.pack(
        _array(tokens, "tokens", i32_, (n,), device), tp, dp, _array(cu_q, "cu_q", i32_, (seqs + 1,), device),
        _array(accept, "accept", f32, (n,), device), _array(pick, "pick", f32, (seqs,), device),
        _array(kv_len, "kv_len", i32_, (seqs,), device), _array(out_tokens, "out_tokens", i32_, (n,), device),
        _array(n_accepted, "n_accepted", i32_, (seqs,), device), _array(kv_len_out, "kv_len_out", i32_, (seqs,), device),
        _array(status, "status", i32_, (1,), device), ts, ds, n, seqs, vocab, typ)
    _call((_lib or load()).dls_verify_draft, desc, stream, device)


DLS_Q4_K = 12
DLS_Q5_K = 13
DLS_Q6_K = 14
KQUANT_TYPES = {"q4_k": DLS_Q4_K, "q5_k": DLS_Q5_K, "q6_k": DLS_Q6_K}


def kquant_packed_bytes(fmt: str, rows: int, cols: int) -> int:
    return int(load().dls_kquant_packed_bytes(KQUANT_TYPES[fmt], rows, cols))


def kquant_pack(fmt: str, blocks, rows: int, cols: int, packed, stream=None):
    """GGUF K-quant super-blocks (device) -> the GEMV's device layout."""
    _check(load().dls_kquant_pack(KQUANT_TYPES[fmt], _ptr(blocks), rows, cols, _ptr(packed), _stream_handle(stream)))


def kquant_gemv(fmt: str, packed, rows: int, cols: int, x, y, status=None, stream=None):
    """y = W x on a packed K-quant matrix (device buffers)."""
    _check(load().dls_kquant_gemv(KQUANT_TYPES[fmt], _ptr(packed), rows, cols, _ptr(x), _ptr(y), _ptr(status),
                                  _stream_handle(stream)))


def _stream_handle(stream):
    if stream is None:
        return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class TorchAllocator:
    """Device memory from PyTorch's caching allocator, through the library's
    allocator callbacks.  ``live`` maps the pointers it handed out to their
    sizes.  ``fail_at`` = k makes the k-th allocation call from now on return
    NULL (the library then reports DLS_ERR_CUDA and rolls the call back);
    ``calls`` counts allocation calls."""

    def __init__(self, device: int, fail_at=None):
        import torch

        self.torch = torch
        self.device = device
        self.live = {}
        self.calls = 0
        self.fail_at = fail_at

        def _alloc(ctx, nbytes, stream):
            self.calls += 1
            if self.fail_at is not None:
                self.fail_at -= 1
                if self.fail_at == 0:
                    self.fail_at = None
                    return None
            try:
                p = torch.cuda.caching_allocator_alloc(int(nbytes), self.device, int(stream or 0))
                self.live[p] = nbytes
                return p
            except Exception:  # out of memory -> NULL -> DLS_ERR_CUDA
                return None

        def _free(ctx, ptr, stream):
            try:
                if ptr in self.live:
                    del self.live[ptr]
                    torch.cuda.caching_allocator_delete(ptr)
            except Exception:
                pass

        self._alloc_cb = dls_allocator._fields_[0][1](_alloc)
        self._free_cb = dls_allocator._fields_[1][1](_free)
        self.struct = dls_allocator(self._alloc_cb, self._free_cb, None)


class Model:
    """A model on the GPU: weights, paged KV pool, decode step.

    ``weights`` is the dict the synthetic generator returns (GGUF-style
    block bytes, host numpy arrays).  ``cfg`` supplies the shapes.
    """

    def __init__(self, cfg, weights, *, max_seqs=1, max_ctx=1024, max_batch=1, page_tokens=64,
                 device_budget_bytes=0, stream=None, torch_allocator=True, allocator=None, kv_pool_pages=0):
        self.lib = load()
        self.cfg = cfg
        self.stream = stream
        L = cfg.n_layers
        keep = []

        def host(a, dtype):
            a = np.ascontiguousarray(a, dtype=dtype)
            keep.append(a)
            return a.ctypes.data

        # per-matrix weight types (weights["formats"]: (layer, name) -> "q4_k" / "q5_k" / "q6_k"; others
        # are the config's Q8_0 / Q4_0)
        fmts = weights.get("formats", {})
        names = ("wq", "wk", "wv", "wo", "w_gate", "w_up", "w_down")
        layers = (dls_layer_desc * L)()
        for l in range(L):
            lw = weights["layers"][l]
            if lw is None:
                raise ValueError(f"layer {l} weights missing")
            types = (i32 * 7)(*(KQUANT_TYPES.get(fmts.get((l, n)), 0) for n in names))
            layers[l] = dls_layer_desc(host(lw["attn_norm"], np.float32), host(lw["ffn_norm"], np.float32),
                                       *(host(lw[n], np.uint8) for n in names), types)
        out = weights.get("output")
        d = dls_model_desc(L, cfg.hidden, cfg.n_heads, cfg.n_kv_heads, cfg.head_dim, cfg.ffn, cfg.vocab,
                           float(cfg.rope_theta), float(cfg.rms_eps), int(bool(cfg.tied)), int(cfg.wtype),
                           page_tokens, max_seqs, max_ctx, max_batch, int(device_budget_bytes),
                           host(weights["tok_embd"], np.uint8), None if out is None else host(out, np.uint8),
                           host(weights["output_norm"], np.float32), layers)
        d.kv_pool_pages = int(kv_pool_pages)
        d.tok_embd_type = KQUANT_TYPES.get(fmts.get((None, "tok_embd")), 0)
        d.output_type = KQUANT_TYPES.get(fmts.get((None, "output")), 0)
        self._alloc = None
        alloc_ptr = None
        if allocator is not None:
            self._alloc = allocator
            alloc_ptr = ctypes.pointer(allocator.struct)
        elif torch_allocator:
            import torch

            self._alloc = TorchAllocator(torch.cuda.current_device())
            alloc_ptr = ctypes.pointer(self._alloc.struct)
        h = vp()
        _check(self.lib.dls_model_create(ctypes.byref(d), alloc_ptr, _stream_handle(stream), ctypes.byref(h)))
        self.handle = h.value
        self.max_ctx, self.max_seqs, self.max_batch = max_ctx, max_seqs, max_batch

    def close(self):
        if getattr(self, "handle", None):
            self.lib.dls_model_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _c(self, rc):
        _check(rc, self.handle)

    # --- sequences
    def seq_create(self) -> int:
        s = i32()
        self._c(self.lib.dls_seq_create(self.handle, ctypes.byref(s)))
        return s.value

    def seq_free(self, seq: int):
        self._c(self.lib.dls_seq_free(self.handle, seq))

    def seq_length(self, seq: int) -> int:
        return int(self.lib.dls_seq_length(self.handle, seq))

    # --- hot path
    def prefill(self, seq: int, tokens, logits_out=None):
        t = np.ascontiguousarray(tokens, dtype=np.int32)
        self._c(self.lib.dls_prefill(self.handle, seq, t.ctypes.data, t.size, _ptr(logits_out)))

    def decode_step(self, seq: int, token: int, pos: int, logits_out=None):
        self._c(self.lib.dls_decode_step(self.handle, seq, int(token), int(pos), _ptr(logits_out)))

    def decode_batch(self, seqs, tokens, pos, logits_out=None):
        s = np.ascontiguousarray(seqs, dtype=np.int32)
        t = np.ascontiguousarray(tokens, dtype=np.int32)
        p = np.ascontiguousarray(pos, dtype=np.int32)
        self._c(self.lib.dls_decode_batch(self.handle, s.size, s.ctypes.data, t.ctypes.data, p.ctypes.data,
                                          _ptr(logits_out)))

    def generate(self, seqs, tokens, n_steps: int, last_logits=None) -> np.ndarray:
        s = np.ascontiguousarray(seqs, dtype=np.int32)
        t = np.ascontiguousarray(tokens, dtype=np.int32)
        out = np.empty((n_steps, s.size), dtype=np.int32)
        self._c(self.lib.dls_generate(self.handle, s.size, s.ctypes.data, t.ctypes.data, n_steps, out.ctypes.data,
                                      _ptr(last_logits)))
        return out

    def argmax(self, logits, n_rows: int, out=None):
        res = np.empty(n_rows, dtype=np.int32) if out is None else out
        self._c(self.lib.dls_argmax(self.handle, _ptr(logits), n_rows, _ptr(res)))
        return res

    def kv_fork(self, src_seq: int, dst_seqs, shared: bool = False):
        """Fork src's KV into each destination: a page copy, or (shared=True)
        shared prefix pages plus a private copy of the partly filled page."""
        d = np.ascontiguousarray(dst_seqs, dtype=np.int32)
        fn = self.lib.dls_kv_fork_shared if shared else self.lib.dls_kv_fork
        self._c(fn(self.handle, src_seq, d.ctypes.data, d.size))

    def kv_free_pages(self) -> int:
        return int(self.lib.dls_kv_free_pages(self.handle))

    # --- layer skip
    def set_layer_skip(self, skip=None):
        """Layers decode steps skip (a boolean per layer), or None for none."""
        if skip is None:
            self._c(self.lib.dls_set_layer_skip(self.handle, None, 0))
            return
        a = np.ascontiguousarray(np.asarray(skip, dtype=bool).astype(np.uint8))
        self._c(self.lib.dls_set_layer_skip(self.handle, a.ctypes.data, a.size))

    def layer_cosines(self, seq: int, token: int, pos: int) -> np.ndarray:
        """One decode step; cosine of each layer's output with its input."""
        out = np.zeros(self.cfg.n_layers, dtype=np.float32)
        self._c(self.lib.dls_layer_cosines(self.handle, seq, int(token), int(pos), out.ctypes.data))
        return out

    def seq_truncate(self, seq: int, length: int):
        self._c(self.lib.dls_seq_truncate(self.handle, seq, int(length)))

    def verify(self, seq: int, tokens, logits_out=None) -> np.ndarray:
        """Score tokens at the sequence end in one pass; each position's greedy pick."""
        t = np.ascontiguousarray(tokens, dtype=np.int32)
        out = np.empty(t.size, dtype=np.int32)
        self._c(self.lib.dls_verify(self.handle, seq, t.ctypes.data, t.size, _ptr(logits_out), out.ctypes.data))
        return out

    def generate_speculative(self, seq: int, token: int, n_tokens: int, draft_skip, draft_k: int = 3):
        """Greedy self-speculative generation; (tokens [n_tokens], stats dict)."""
        mask = np.ascontiguousarray(np.asarray(draft_skip, dtype=bool).astype(np.uint8))
        if mask.size != self.cfg.n_layers:
            raise ValueError(f"draft_skip has {mask.size} entries, the model {self.cfg.n_layers} layers")
        out = np.empty(int(n_tokens), dtype=np.int32)
        st = np.zeros(3, dtype=np.int32)
        self._c(self.lib.dls_generate_speculative(self.handle, seq, int(token), int(n_tokens), mask.ctypes.data,
                                                  int(draft_k), out.ctypes.data, st.ctypes.data))
        return out, {"rounds": int(st[0]), "drafted": int(st[1]), "accepted": int(st[2])}

    # --- residency
    def set_resident_layers(self, n: int):
        self._c(self.lib.dls_set_resident_layers(self.handle, n))

    def resident_layers(self) -> int:
        return int(self.lib.dls_resident_layers(self.handle))

    def layer_bytes(self) -> int:
        return int(self.lib.dls_layer_bytes(self.handle))

    def device_bytes(self) -> int:
        return int(self.lib.dls_device_bytes(self.handle))

    def device_budget(self) -> int:
        return int(self.lib.dls_device_budget(self.handle))

    # --- hooks
    def debug_capture(self, per_layer_out):
        self._c(self.lib.dls_debug_capture(self.handle, _ptr(per_layer_out)))

    def debug_bounded_wait(self, limit_ns: int):
        """A bounded device wait that nothing satisfies (raises DLS_ERR_TIMEOUT)."""
        self._c(self.lib.dls_debug_bounded_wait(self.handle, int(limit_ns)))

    def debug_read_kv(self, seq: int, layer: int, k_out, v_out):
        self._c(self.lib.dls_debug_read_kv(self.handle, seq, layer, _ptr(k_out), _ptr(v_out)))

    def debug_dequant(self, layer: int, tensor: str, out):
        self._c(self.lib.dls_debug_dequant(self.handle, layer, TENSOR_IDS[tensor], _ptr(out)))

    def debug_gemv(self, layer: int, tensor: str, x, y):
        self._c(self.lib.dls_debug_gemv(self.handle, layer, TENSOR_IDS[tensor], _ptr(x), _ptr(y)))

    def debug_gemm(self, layer: int, tensor: str, x, y):
        """y[t] = W x[t] with the prefill GEMM; x device fp32 [T][cols], y [T][rows]."""
        self._c(self.lib.dls_debug_gemm(self.handle, layer, TENSOR_IDS[tensor], int(x.shape[0]), _ptr(x), _ptr(y)))

    def profile_step(self, seq: int, token: int, pos: int, max_kernels: int = 4096):
        """(durations_ms, kinds) of every kernel of one decode step."""
        ms = np.zeros(max_kernels, dtype=np.float32)
        kinds = np.zeros(max_kernels, dtype=np.int32)
        n = i32()
        self._c(self.lib.dls_debug_profile_step(self.handle, seq, int(token), int(pos), max_kernels, ms.ctypes.data,
                                                kinds.ctypes.data, ctypes.byref(n)))
        return ms[: n.value].copy(), kinds[: n.value].copy()

    def profile_batch(self, seqs, tokens, pos, max_kernels: int = 8192):
        """(durations_ms, kinds) of every kernel of one batched decode step."""
        n = len(seqs)
        sa = np.ascontiguousarray(seqs, dtype=np.int32)
        ta = np.ascontiguousarray(tokens, dtype=np.int32)
        pa = np.ascontiguousarray(pos, dtype=np.int32)
        ms = np.zeros(max_kernels, dtype=np.float32)
        kinds = np.zeros(max_kernels, dtype=np.int32)
        cnt = i32()
        self._c(self.lib.dls_debug_profile_batch(self.handle, n, sa.ctypes.data, ta.ctypes.data, pa.ctypes.data,
                                                 max_kernels, ms.ctypes.data, kinds.ctypes.data, ctypes.byref(cnt)))
        return ms[: cnt.value].copy(), kinds[: cnt.value].copy()

    def step_trace(self, max_entries: int = 1 << 22) -> np.ndarray:
        """Per-CTA phase timestamps of the last profiled persistent step: [phase, cta, 4] (ns)."""
        out = np.zeros(max_entries, dtype=np.uint64)
        n = ctypes.c_int32(0)
        self._c(self.lib.dls_debug_step_trace(self.handle, out.ctypes.data, max_entries, ctypes.byref(n)))
        return out[: n.value]

    def launches_per_step(self) -> int:
        return int(self.lib.dls_debug_launches_per_step(self.handle))

    def step_kernel_in_use(self):
        """(True, None) when batch-1 steps run as the persistent step kernel,
        else (False, reason)."""
        why = ctypes.c_char_p()
        used = bool(self.lib.dls_step_kernel_in_use(self.handle, ctypes.byref(why)))
        return used, (why.value.decode() if why.value else None)

    def last_error(self) -> str:
        return self.lib.dls_last_error(self.handle).decode(errors="replace")
