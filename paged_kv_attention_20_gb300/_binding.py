"""ctypes binding of libpagedattn.so: argument marshalling only.

Every computation happens in the library's CUDA kernels.  This module checks
what only the Python side can see (tensor device, dtype, contiguity, rank,
storage overlap of the output with the inputs -- ruDNN 0.1.7,
src/paged_attention/mod.rs, `attention_into`: "the PyTorch adapter enforces
storage-overlap checks"), passes raw pointers and the current CUDA stream, and
turns non-OK statuses into exceptions.  If the library is missing it raises;
there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

from . import buildlib as _build

_LIB = None

PA_OK = 0
STATUS_NAMES = {0: "PA_OK", 1: "PA_ERR_ARG", 2: "PA_ERR_SHAPE", 3: "PA_ERR_DTYPE", 4: "PA_ERR_RANGE",
                5: "PA_ERR_WRITE_CONFLICT", 6: "PA_ERR_WORKSPACE", 7: "PA_ERR_SPLITS", 8: "PA_ERR_LIMIT",
                9: "PA_ERR_CUDA", 10: "PA_ERR_STATE"}
_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
MAX_SPLITS = 64

EXPORTED = ["pa_last_error", "pa_status_string", "pa_abi_version", "paged_attn_plan",
            "pa_plan_device_bytes", "pa_plan_upload", "pa_plan_stage", "pa_plan_destroy", "pa_plan_describe",
            "pa_workspace_bytes", "paged_attn_split_heuristic", "paged_mla_split_heuristic",
            "paged_attn_decode_sms_beside_prefill", "paged_kv_store", "paged_attn_forward",
            "paged_attn_forward_split", "paged_mla_forward", "pa_plan_advance", "pa_time_next_kernel",
            "pa_device_status", "paged_qk_norm_rope_store", "pa_mass_workspace_bytes", "paged_attn_forward_mass",
            "paged_kv_evict"]


class PagedAttentionError(RuntimeError):
    """A library call returned a status other than PA_OK."""

    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def lib_path() -> str:
    return _build.LIB


def load() -> ctypes.CDLL:
    """Load libpagedattn.so (built by build.build()); raise if it is missing."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with paged_kv_attention_20_gb300.build() "
                           "(nvcc, sm_103a); there is no fallback path")
    lib = ctypes.CDLL(path)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.pa_last_error.restype = ctypes.c_char_p
    lib.pa_status_string.restype = ctypes.c_char_p
    lib.pa_status_string.argtypes = [ctypes.c_int]
    lib.pa_abi_version.restype = i32
    lib.paged_attn_plan.argtypes = [vp, i32, vp, i32, vp, vp, i32, i32, i32, ctypes.POINTER(vp)]
    lib.paged_attn_plan.restype = ctypes.c_int
    lib.pa_plan_device_bytes.argtypes = [vp]
    lib.pa_plan_device_bytes.restype = sz
    lib.pa_plan_upload.argtypes = [vp, vp, sz, vp]
    lib.pa_plan_upload.restype = ctypes.c_int
    lib.pa_plan_stage.argtypes = [vp, vp, sz, vp, sz]
    lib.pa_plan_stage.restype = ctypes.c_int
    lib.pa_plan_destroy.argtypes = [vp]
    lib.pa_plan_destroy.restype = None
    lib.pa_plan_describe.argtypes = [vp, ctypes.POINTER(i64)]
    lib.pa_plan_describe.restype = ctypes.c_int
    lib.pa_workspace_bytes.argtypes = [i32, i32, i32, i32]
    lib.pa_workspace_bytes.restype = sz
    lib.paged_attn_split_heuristic.argtypes = [vp, i32, i32, i32, i32]
    lib.paged_attn_split_heuristic.restype = i32
    lib.paged_mla_split_heuristic.argtypes = [vp, i32, i32, i32]
    lib.paged_mla_split_heuristic.restype = i32
    lib.paged_attn_decode_sms_beside_prefill.argtypes = [vp, i32, i32, i32, i32, i32, i32, i32, i32]
    lib.paged_attn_decode_sms_beside_prefill.restype = i32
    lib.paged_kv_store.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, ctypes.c_int, vp]
    lib.paged_kv_store.restype = ctypes.c_int
    lib.paged_attn_forward.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, ctypes.c_float, i32, i32,
                                       ctypes.c_int, vp]
    lib.paged_attn_forward.restype = ctypes.c_int
    lib.paged_attn_forward_split.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, ctypes.c_float, i32,
                                             i32, ctypes.c_int, vp, sz, i32, vp]
    lib.paged_attn_forward_split.restype = ctypes.c_int
    lib.paged_mla_forward.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, ctypes.c_float, i32, i32,
                                      ctypes.c_int, vp, sz, i32, vp]
    lib.paged_mla_forward.restype = ctypes.c_int
    lib.pa_plan_advance.argtypes = [vp, vp]
    lib.pa_plan_advance.restype = ctypes.c_int
    lib.paged_qk_norm_rope_store.argtypes = [vp, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, vp, i32, i32, i32, vp,
                                             vp, vp, ctypes.c_float, i32, i32, i32, i32, ctypes.c_int, vp]
    lib.paged_qk_norm_rope_store.restype = ctypes.c_int
    lib.pa_mass_workspace_bytes.argtypes = [vp, i32, i32, i32, i32, i32, i64]
    lib.pa_mass_workspace_bytes.restype = sz
    lib.paged_attn_forward_mass.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, ctypes.c_float, i32, i32,
                                            ctypes.c_int, vp, sz, i32, vp]
    lib.paged_attn_forward_mass.restype = ctypes.c_int
    lib.paged_kv_evict.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, ctypes.c_int, vp]
    lib.paged_kv_evict.restype = ctypes.c_int
    lib.pa_time_next_kernel.argtypes = [vp, vp]
    lib.pa_time_next_kernel.restype = ctypes.c_int
    lib.pa_device_status.argtypes = [ctypes.POINTER(i32), i32]
    lib.pa_device_status.restype = ctypes.c_int
    _LIB = lib
    return lib


def _check(status: int) -> None:
    if status != PA_OK:
        raise PagedAttentionError(status, load().pa_last_error().decode())


def _i32_array(a) -> np.ndarray:
    if isinstance(a, torch.Tensor):
        a = a.detach().cpu().numpy()
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


# the current stream's handle without building a torch.cuda.Stream (2 us of a small call's time)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current_stream(index: int) -> int:
    return _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream


def _stream(device) -> int:
    if device.index is not None:
        return _current_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


class Plan:
    """A validated schedule (`paged_attn_plan`) and, once uploaded, its device copy."""

    def __init__(self, handle: int, counts: np.ndarray):
        self._handle = ctypes.c_void_p(handle)
        self.queries, self.sequences, self.width, self.page_size, self.pages = (int(x) for x in counts[:5])
        self.n_decode, self.n_tiles, self.n_tile_queries = (int(x) for x in counts[5:8])
        self.longest = 0    # keys of the longest sequence the plan was built with
        self.words = None
        self.device = None
        self._index = -1    # CUDA index of the device copy, -1 before the upload

    @property
    def handle(self) -> ctypes.c_void_p:
        return self._handle

    def device_bytes(self) -> int:
        return int(load().pa_plan_device_bytes(self._handle))

    def upload(self, device=None) -> "Plan":
        """Allocate the metadata buffer on `device` and enqueue its upload on the current stream."""
        device = torch.device(device if device is not None else "cuda")
        n = self.device_bytes()
        self.words = torch.empty(max(16, n), dtype=torch.uint8, device=device)
        self.device = self.words.device
        self._index = self.words.get_device()
        _check(load().pa_plan_upload(self._handle, self.words.data_ptr(), self.words.numel(),
                                     _stream(self.device)))
        return self

    def upload_into(self, words: torch.Tensor) -> "Plan":
        """Upload into a caller-provided device byte buffer (reused across steps)."""
        self.words = words
        self.device = words.device
        self._index = words.get_device()
        _check(load().pa_plan_upload(self._handle, words.data_ptr(), words.numel(), _stream(words.device)))
        return self

    def stage(self, host_words: torch.Tensor, device_words: torch.Tensor) -> "Plan":
        """Write the device image into `host_words` (CPU uint8, e.g. pinned) and bind `device_words`.

        Nothing is copied to the device: the caller copies host_words into
        device_words on its stream (capturable in a CUDA graph) before the
        next call that uses this plan.
        """
        for t, name, on_cuda in ((host_words, "host_words", False), (device_words, "device_words", True)):
            if t.dtype != torch.uint8 or not t.is_contiguous() or t.is_cuda != on_cuda:
                raise ValueError(f"{name} must be a contiguous uint8 {'CUDA' if on_cuda else 'CPU'} tensor")
        _check(load().pa_plan_stage(self._handle, host_words.data_ptr(), host_words.numel(),
                                    device_words.data_ptr(), device_words.numel()))
        self.words = device_words
        self.device = device_words.device
        self._index = device_words.get_device()
        return self

    def __del__(self):
        h = getattr(self, "_handle", None)
        if h is not None and h.value and _LIB is not None:
            _LIB.pa_plan_destroy(h)
            self._handle = ctypes.c_void_p(0)


def paged_attn_plan(seq_lens, block_table, query_seq, query_pos, page_size: int, num_pages: int,
                    device=None, upload: bool = True) -> Plan:
    """Build (and by default upload) a schedule; see paged_attn_plan in paged_attn.h."""
    lib = load()
    seq_lens = _i32_array(seq_lens)
    bt = _i32_array(block_table)
    if bt.ndim == 1:
        bt = bt.reshape(len(seq_lens), -1) if len(seq_lens) else bt.reshape(0, 0)
    width = int(bt.shape[1]) if bt.ndim == 2 else 0
    qs, qp = _i32_array(query_seq), _i32_array(query_pos)
    if qs.shape != qp.shape:
        raise ValueError("query_seq and query_pos must have the same length")
    handle = ctypes.c_void_p()
    _check(lib.paged_attn_plan(seq_lens.ctypes.data, len(seq_lens), bt.ctypes.data, width, qs.ctypes.data,
                               qp.ctypes.data, len(qs), int(page_size), int(num_pages), ctypes.byref(handle)))
    counts = (ctypes.c_int64 * 8)()
    _check(lib.pa_plan_describe(handle, counts))
    plan = Plan(handle.value, np.array(counts[:], dtype=np.int64))
    plan.longest = int(seq_lens.max()) if len(seq_lens) else 0
    if upload:
        plan.upload(device)
    return plan


def _tensor(t: torch.Tensor, name: str, dtype, device, rank: int) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dim() != rank:
        raise ValueError(f"{name} must have rank {rank}")


def _storage_span(t: torch.Tensor):
    start = t.data_ptr()
    return start, start + t.numel() * t.element_size()


def _check_disjoint(out: torch.Tensor, *inputs) -> None:
    o0, o1 = _storage_span(out)
    for t in inputs:
        if t is None or t.numel() == 0:
            continue
        a0, a1 = _storage_span(t)
        if a0 < o1 and o0 < a1:
            raise ValueError("output overlaps an input tensor")


def _plan_ready(plan: Plan, device) -> None:
    if plan.words is None:
        raise ValueError("plan has not been uploaded")
    if plan.device != device:
        raise ValueError(f"plan metadata is on {plan.device}, tensors on {device}")


def workspace_bytes(queries: int, heads: int, value_dim: int, splits: int) -> int:
    return int(load().pa_workspace_bytes(int(queries), int(heads), int(value_dim), int(splits)))


def make_workspace(plan: Plan, heads: int, value_dim: int, splits: int, device=None) -> torch.Tensor:
    """Caller-owned fp32 workspace sized for `splits` partials."""
    n = workspace_bytes(plan.queries, heads, value_dim, splits)
    return torch.empty((n + 3) // 4, dtype=torch.float32, device=device or plan.device)


def paged_attn_split_heuristic(plan: Plan, num_heads: int, num_kv_heads: int, num_sms: int | None = None,
                               window: int = 0) -> int:
    if num_sms is None:
        num_sms = torch.cuda.get_device_properties(plan.device or 0).multi_processor_count
    return int(load().paged_attn_split_heuristic(plan.handle, int(num_heads), int(num_kv_heads), int(window),
                                                 int(num_sms)))


def paged_mla_split_heuristic(plan: Plan, num_heads: int, num_sms: int | None = None, window: int = 0) -> int:
    if num_sms is None:
        num_sms = torch.cuda.get_device_properties(plan.device or 0).multi_processor_count
    return int(load().paged_mla_split_heuristic(plan.handle, int(num_heads), int(window), int(num_sms)))


def paged_attn_decode_sms_beside_prefill(plan: Plan, num_heads: int, num_kv_heads: int, head_dim: int,
                                         value_dim: int, causal: bool = True, window: int = 0,
                                         dtype=torch.bfloat16, num_sms: int | None = None) -> int:
    """SMs an attention call on this plan leaves to its decode items beside the prefill tiles (0: serial)."""
    if num_sms is None:
        num_sms = torch.cuda.get_device_properties(plan.device or 0).multi_processor_count
    return int(load().paged_attn_decode_sms_beside_prefill(plan.handle, int(num_heads), int(num_kv_heads),
                                                           int(head_dim), int(value_dim), 1 if causal else 0,
                                                           int(window), _DTYPES[dtype], int(num_sms)))


def paged_kv_store(plan: Plan, new_k, new_v, k_cache, v_cache) -> None:
    """Append new_k [Q, H, d] / new_v [Q, H, dv] into the caches at the plan's slots."""
    dev = k_cache.device
    dt = k_cache.dtype
    for name, t, r in (("new_k", new_k, 3), ("new_v", new_v, 3), ("k_cache", k_cache, 4), ("v_cache", v_cache, 4)):
        _tensor(t, name, dt, dev, r)
    _plan_ready(plan, dev)
    heads, d, dv = k_cache.shape[2], k_cache.shape[3], v_cache.shape[3]
    if tuple(k_cache.shape[:3]) != tuple(v_cache.shape[:3]) or k_cache.shape[0] != plan.pages \
            or k_cache.shape[1] != plan.page_size:
        raise ValueError("cache shapes do not match the plan")
    if tuple(new_k.shape) != (plan.queries, heads, d) or tuple(new_v.shape) != (plan.queries, heads, dv):
        raise ValueError("new rows must be [queries, heads, d|dv]")
    _check(load().paged_kv_store(plan.handle, new_k.data_ptr(), new_v.data_ptr(), k_cache.data_ptr(),
                                 v_cache.data_ptr(), heads, d, dv, _DTYPES[dt], _stream(dev)))


def _attn_common(plan, q, k_cache, v_cache, out):
    dev, dt = q.device, q.dtype
    if dt not in _DTYPES:
        raise TypeError("dtype must be float32, float16 or bfloat16")
    _tensor(q, "q", dt, dev, 3)
    _tensor(k_cache, "k_cache", dt, dev, 4)
    _tensor(v_cache, "v_cache", dt, dev, 4)
    _plan_ready(plan, dev)
    if k_cache.shape[0] != plan.pages or k_cache.shape[1] != plan.page_size \
            or tuple(k_cache.shape[:3]) != tuple(v_cache.shape[:3]):
        raise ValueError("cache shapes do not match the plan")
    if q.shape[0] != plan.queries or q.shape[2] != k_cache.shape[3]:
        raise ValueError("q must be [queries, num_heads, head_dim] matching the plan and cache")
    shape = (q.shape[0], q.shape[1], v_cache.shape[3])
    if out is None:
        out = torch.empty(shape, dtype=dt, device=dev)
    else:
        _tensor(out, "out", dt, dev, 3)
        if tuple(out.shape) != shape:
            raise ValueError(f"out must have shape {shape}")
    _check_disjoint(out, q, k_cache, v_cache)
    return out


def paged_attn_forward(plan: Plan, q, k_cache, v_cache, scale: float, causal: bool = True, out=None,
                       window: int = 0):
    """Paged MHA/GQA attention; returns out [queries, num_heads, value_dim].
    window > 0: a query at position p sees keys p - window + 1 and later."""
    out = _attn_common(plan, q, k_cache, v_cache, out)
    _check(load().paged_attn_forward(plan.handle, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                     out.data_ptr(), q.shape[1], k_cache.shape[2], q.shape[2],
                                     v_cache.shape[3], float(scale), 1 if causal else 0, int(window),
                                     _DTYPES[q.dtype], _stream(q.device)))
    return out


def paged_attn_forward_split(plan: Plan, q, k_cache, v_cache, scale: float, splits: int, workspace=None,
                             causal: bool = True, out=None, window: int = 0):
    """Split-KV paged attention with an fp32 workspace (allocated here when not given)."""
    out = _attn_common(plan, q, k_cache, v_cache, out)
    if workspace is None:
        workspace = make_workspace(plan, q.shape[1], v_cache.shape[3], splits, q.device)
    _check_disjoint(out, workspace)
    _check(load().paged_attn_forward_split(plan.handle, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                           out.data_ptr(), q.shape[1], k_cache.shape[2], q.shape[2],
                                           v_cache.shape[3], float(scale), 1 if causal else 0, int(window),
                                           _DTYPES[q.dtype], workspace.data_ptr(),
                                           workspace.numel() * workspace.element_size(), int(splits),
                                           _stream(q.device)))
    return out


def paged_mla_forward(plan: Plan, q, qp, latent_cache, pos_cache, scale: float, causal: bool = True,
                      workspace=None, splits: int = 1, out=None, window: int = 0):
    """MLA attention over a shared latent head plus a rotated position cache."""
    dev, dt = q.device, q.dtype
    if dt not in _DTYPES:
        raise TypeError("dtype must be float32, float16 or bfloat16")
    _tensor(q, "q", dt, dev, 3)
    _tensor(qp, "qp", dt, dev, 3)
    _tensor(latent_cache, "latent_cache", dt, dev, 4)
    _tensor(pos_cache, "pos_cache", dt, dev, 4)
    _plan_ready(plan, dev)
    if latent_cache.shape[2] != 1 or pos_cache.shape[2] != 1:
        raise ValueError("MLA latent cache must have one shared head")
    if latent_cache.shape[0] != plan.pages or latent_cache.shape[1] != plan.page_size \
            or tuple(pos_cache.shape[:2]) != tuple(latent_cache.shape[:2]):
        raise ValueError("cache shapes do not match the plan")
    if q.shape[0] != plan.queries or q.shape[2] != latent_cache.shape[3] or tuple(qp.shape[:2]) != tuple(q.shape[:2]) \
            or qp.shape[2] != pos_cache.shape[3]:
        raise ValueError("incompatible MLA query / cache dimensions")
    shape = tuple(q.shape)
    if out is None:
        out = torch.empty(shape, dtype=dt, device=dev)
    else:
        _tensor(out, "out", dt, dev, 3)
        if tuple(out.shape) != shape:
            raise ValueError(f"out must have shape {shape}")
    if splits > 1 and workspace is None:
        workspace = make_workspace(plan, q.shape[1], q.shape[2], splits, dev)
    _check_disjoint(out, q, qp, latent_cache, pos_cache, workspace)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().paged_mla_forward(plan.handle, q.data_ptr(), qp.data_ptr(), latent_cache.data_ptr(),
                                    pos_cache.data_ptr(), out.data_ptr(), q.shape[1], q.shape[2], qp.shape[2],
                                    float(scale), 1 if causal else 0, int(window), _DTYPES[dt], ws_ptr, ws_bytes,
                                    int(splits), _stream(dev)))
    return out


def _dense(t, name: str, dtype, index: int, rank: int):
    """Shape of a dense operand on CUDA device `index` (-1: the host)."""
    try:
        if t.dtype is dtype and t.get_device() == index and t.is_contiguous():
            shape = t.shape
            if len(shape) == rank:
                return shape
    except AttributeError:
        pass
    _tensor(t, name, dtype, torch.device("cuda", index) if index >= 0 else torch.device("cpu"), rank)
    return t.shape


def _key_mass(t, pages: int, heads: int, page_size: int, index: int) -> None:
    if _dense(t, "key_mass", torch.float32, index, 3) != (pages, heads, page_size):
        raise ValueError("key_mass must be [pages, kv_heads, page_size]")


def _caches(plan: Plan, k_cache, v_cache):
    """Checks of a K/V cache pair against the plan; (dtype, its code, device index, K shape, value dim)."""
    if not isinstance(k_cache, torch.Tensor):
        raise TypeError("k_cache must be a torch.Tensor")
    dt, index = k_cache.dtype, k_cache.get_device()
    code = _DTYPES.get(dt)
    if code is None:
        raise TypeError("dtype must be float32, float16 or bfloat16")
    shape = _dense(k_cache, "k_cache", dt, index, 4)
    pages, ps, hkv, dv = _dense(v_cache, "v_cache", dt, index, 4)
    if plan._index != index or index < 0:
        _plan_ready(plan, k_cache.device)
    if shape[0] != pages or shape[1] != ps or shape[2] != hkv or pages != plan.pages or ps != plan.page_size:
        raise ValueError("cache shapes do not match the plan")
    return dt, code, index, shape, dv


def _rows(t, name: str, dtype, index: int, queries: int, dim: int):
    """A [queries, heads, dim] operand whose rows may lie apart; returns (heads, row stride in elements)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected CUDA device {index}")
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must have rank 3")
    n, heads, d = shape
    if n != queries or d != dim:
        raise ValueError(f"{name} must be [queries, heads, {dim}] matching the plan and cache")
    sq, sh, sd = t.stride()
    if (sd != 1 and dim > 1) or (sh != dim and heads > 1):
        raise ValueError(f"{name}: each row's heads must be contiguous")
    return heads, sq if queries > 1 else heads * dim


def paged_qk_norm_rope_store(plan: Plan, q, new_k, new_v, k_cache, v_cache, rope_table=None, q_weight=None,
                             k_weight=None, eps: float = 1e-6, interleaved: bool = False, positions=None,
                             key_mass=None, q_out=None):
    """RMS-norm and rotate q [Q, Hq, d] and new_k [Q, Hkv, d] per head, append new_k and new_v [Q, Hkv, dv].

    q, new_k and new_v may be views whose rows lie apart (slices of one projection output).  rope_table is
    fp32 [max_positions, rope_dim], cosines then sines; `positions` (int32 [Q]) replaces the plan's positions for
    the rotation; key_mass, when given, is zeroed at the written keys.  Returns the queries, dense (`q_out` may be
    a dense q itself)."""
    dt, code, index, (pages, ps, hkv, d), dv = _caches(plan, k_cache, v_cache)
    n = plan.queries
    hq, q_stride = _rows(q, "q", dt, index, n, d)
    hk, k_stride = _rows(new_k, "new_k", dt, index, n, d)
    hv, v_stride = _rows(new_v, "new_v", dt, index, n, dv)
    if hk != hkv or hv != hkv:
        raise ValueError("new rows must be [queries, kv_heads, d|dv]")
    table_ptr = pos_ptr = mass_ptr = qw_ptr = kw_ptr = None
    far = rot = 0
    if rope_table is not None:
        far, rot = _dense(rope_table, "rope_table", torch.float32, index, 2)
        if far == 0 or rot == 0:        # an empty tensor's null pointer would read as "no table"
            raise ValueError("the rope table is empty")
        table_ptr = rope_table.data_ptr()
    if positions is not None:
        if _dense(positions, "positions", torch.int32, index, 1)[0] != n:
            raise ValueError("positions must be [queries]")
        pos_ptr = positions.data_ptr()
    if q_weight is not None:
        if _dense(q_weight, "q_weight", dt, index, 1)[0] != d:
            raise ValueError("norm weights must be [head_dim]")
        qw_ptr = q_weight.data_ptr()
    if k_weight is not None:
        if _dense(k_weight, "k_weight", dt, index, 1)[0] != d:
            raise ValueError("norm weights must be [head_dim]")
        kw_ptr = k_weight.data_ptr()
    if key_mass is not None:
        _key_mass(key_mass, pages, hkv, ps, index)
        mass_ptr = key_mass.data_ptr()
    if q_out is None:
        q_out = torch.empty((n, hq, d), dtype=dt, device=k_cache.device)
    elif _dense(q_out, "q_out", dt, index, 3) != (n, hq, d):
        raise ValueError(f"q_out must have shape {(n, hq, d)}")
    lib = _LIB or load()
    status = lib.paged_qk_norm_rope_store(
        plan._handle, q.data_ptr(), q_stride, new_k.data_ptr(), k_stride, new_v.data_ptr(), v_stride, q_out.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), mass_ptr, table_ptr, far, rot, 1 if interleaved else 0, pos_ptr, qw_ptr,
        kw_ptr, eps, hq, hkv, d, dv, code, _current_stream(index))
    if status:
        _check(status)
    return q_out


def mass_workspace_bytes(plan: Plan, heads: int, kv_heads: int, value_dim: int, splits: int, window: int = 0,
                         max_keys: int = 0) -> int:
    return int(load().pa_mass_workspace_bytes(plan.handle, int(heads), int(kv_heads), int(value_dim), int(splits),
                                              int(window), int(max_keys)))


def make_mass_workspace(plan: Plan, heads: int, kv_heads: int, value_dim: int, splits: int, window: int = 0,
                        max_keys: int = 0, device=None) -> torch.Tensor:
    """Caller-owned workspace of paged_attn_forward_mass (window: 0 for calls that are not causal; max_keys: room
    for the histories a captured decode loop will reach)."""
    n = mass_workspace_bytes(plan, heads, kv_heads, value_dim, splits, window, max_keys)
    return torch.empty((n + 3) // 4, dtype=torch.float32, device=device or plan.device)


def paged_attn_forward_mass(plan: Plan, q, k_cache, v_cache, key_mass, scale: float, splits: int | None = None,
                            workspace=None, causal: bool = True, out=None, window: int = 0):
    """Paged attention that adds each key's softmax weights, over the plan's queries and a KV head's query heads, to
    key_mass [pages, kv_heads, page_size] (fp32).  splits defaults to the split heuristic; the workspace is allocated
    here when not given (make_mass_workspace)."""
    dt, code, index, (pages, ps, hkv, d), dv = _caches(plan, k_cache, v_cache)
    n, hq, dq = _dense(q, "q", dt, index, 3)
    if n != plan.queries or dq != d:
        raise ValueError("q must be [queries, num_heads, head_dim] matching the plan and cache")
    if out is None:
        out = torch.empty((n, hq, dv), dtype=dt, device=k_cache.device)
    elif _dense(out, "out", dt, index, 3) != (n, hq, dv):
        raise ValueError(f"out must have shape {(n, hq, dv)}")
    _key_mass(key_mass, pages, hkv, ps, index)
    if splits is None:
        splits = paged_attn_split_heuristic(plan, hq, hkv, window=window)
    if workspace is None:
        workspace = make_mass_workspace(plan, hq, hkv, dv, splits, window if causal else 0, device=k_cache.device)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    lib = _LIB or load()
    status = lib.paged_attn_forward_mass(
        plan._handle, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(), key_mass.data_ptr(), hq, hkv, d,
        dv, scale, 1 if causal else 0, window, code, workspace.data_ptr(), workspace.nbytes, splits, _current_stream(index))
    if status:
        _check(status)
    return out


def paged_kv_evict(plan: Plan, kept_plan: Plan, key_mass, k_cache, v_cache, sink: int = 0, recent: int = 0, kept=None):
    """Shrink every sequence of `plan` to its length in `kept_plan`: the first `sink`, the last `recent` and, between
    them, the keys with the largest key_mass stay and move to the kept schedule's rows.  Returns the kept keys' former
    indices, int32 [sequences, kv_heads, longest kept history], -1 past a sequence's kept length."""
    dt, code, index, (pages, ps, hkv, d), dv = _caches(plan, k_cache, v_cache)
    if kept_plan._index != index:
        _plan_ready(kept_plan, k_cache.device)
    _key_mass(key_mass, pages, hkv, ps, index)
    if kept is None:
        kept = torch.empty((plan.sequences, hkv, kept_plan.longest), dtype=torch.int32, device=k_cache.device)
        stride = kept_plan.longest
    else:
        sequences, heads, stride = _dense(kept, "kept", torch.int32, index, 3)
        if sequences != plan.sequences or heads != hkv:
            raise ValueError("kept must be [sequences, kv_heads, n]")
    lib = _LIB or load()
    status = lib.paged_kv_evict(plan._handle, kept_plan._handle, key_mass.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                kept.data_ptr(), stride, sink, recent, hkv, d, dv, code, _current_stream(index))
    if status:
        _check(status)
    return kept


def paged_attn_plan_advance(plan: Plan) -> None:
    """Move every query of a decode plan one position forward, on the device (graph-capturable)."""
    if plan.words is None:
        raise ValueError("plan has not been uploaded")
    _check(load().pa_plan_advance(plan.handle, _stream(plan.device)))


def time_next_kernel(start: torch.cuda.Event, stop: torch.cuda.Event) -> None:
    """Have the next attention call record `start`/`stop` around its main kernel."""
    for ev in (start, stop):
        if not ev.cuda_event:   # torch creates the CUDA event lazily
            ev.record()
    _check(load().pa_time_next_kernel(start.cuda_event, stop.cuda_event))


def device_status(clear: bool = True) -> int:
    """Synchronise and read (and clear) the device timeout word; 0 means no wait ran out."""
    code = ctypes.c_int32(0)
    _check(load().pa_device_status(ctypes.byref(code), 1 if clear else 0))
    return int(code.value)
