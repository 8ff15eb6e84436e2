"""Binding of ``libgqa_decode.so`` -- argument marshalling only, by ctypes, and by the extension module
``_calls`` for the calls of every layer.

Every function here has the name of the C entry point it calls (see
``include/gqa_decode.h``), takes torch tensors where the C call takes device
pointers, reads sizes off the tensors' shapes, and raises :class:`GQAError`
when the call returns a non-OK status.  All compute runs in the library's CUDA
kernels; there is no other code path.  If the library has not been built,
importing this module raises.
"""
from __future__ import annotations

import ctypes
import importlib
import math
import os
import threading
from typing import Optional, Sequence, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgqa_decode.so")

GQA_OK = 0
GQA_ERR_INVALID_ARG = 1
GQA_ERR_UNSUPPORTED = 2
GQA_ERR_WORKSPACE = 3
GQA_ERR_CUDA = 4
GQA_ERR_TIMEOUT = 5
GQA_ERR_BOUNDS = 6
GQA_BUILD_BOUNDS_CHECK = 1
GQA_CACHE_ROWS = 0
GQA_CACHE_VLLM = 1
GQA_CACHE_KV8 = 2
GQA_CACHE_KV4 = 4


class GQAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {gqa_status_string(status)} (status {status})")


class gqa_options(ctypes.Structure):
    _fields_ = [("n_splits", ctypes.c_int), ("merge_mode", ctypes.c_int),
                ("timeout_us", ctypes.c_uint32), ("test_stall_cta", ctypes.c_int),
                ("paged_head_group", ctypes.c_int), ("causal", ctypes.c_int), ("bf16", ctypes.c_int),
                ("mma_path", ctypes.c_int)]


class gqa_append_args(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q", "k", "v", "q_out")] +
                [(n, ctypes.c_int64) for n in ("q_stride", "k_stride", "v_stride", "q_out_stride")] +
                [(n, ctypes.c_void_p) for n in ("q_weight", "k_weight", "cos_sin", "positions", "slots", "k_cache",
                                                "v_cache")] +
                [(n, ctypes.c_int) for n in ("num_tokens", "h_q", "h_kv", "d_head", "max_position", "rot_dim",
                                             "interleaved", "num_blocks", "block_size", "cache_layout", "bf16")] +
                [("eps", ctypes.c_float)])


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build the CUDA library first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    return ctypes.CDLL(LIB_PATH)


lib = _load()

_p, _i, _i64, _sz, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
_opt = ctypes.POINTER(gqa_options)
_SIGS = {
    "gqa_default_options": ([], gqa_options),
    "gqa_status_string": ([_i], ctypes.c_char_p),
    "gqa_version": ([], _i),
    "gqa_build_flags": ([], _i),
    "gqa_decode_num_splits": ([_i, _i, _i64, _i, _i, _i], _i),
    "gqa_decode_plan": ([_i, _i, _i64, _i, _i, _i, _opt, _p, _p, _p], _i),
    "gqa_decode_plan_ex": ([_i, _i, _i64, _i, _i, _i, _opt, _p, _p, _p, _p, _p], _i),
    "gqa_paged_plan": ([_i, _i, _i, _i, _i, _i, _i, _i, _opt, _p, _p, _p], _i),
    "gqa_decode_workspace_size": ([_i, _i, _i64, _i, _i, _i, _i], _sz),
    "gqa_workspace_size": ([_i, _i, _i64, _i, _i, _i], _sz),
    "gqa_paged_workspace_size": ([_i, _i, _i, _i, _i, _i], _sz),
    "gqa_workspace_init": ([_p, _sz, _p], _i),
    "gqa_workspace_check": ([_p, _p], _i),
    "gqa_decode": ([_p, _p, _p, _p, _i, _i, _i64, _i, _i, _i, _f, _p, _sz, _p], _i),
    "gqa_decode_ex": ([_p, _p, _p, _p, _i, _i, _i64, _i, _i, _i, _f, _p, _sz, _p, _opt], _i),
    "gqa_decode_partial": ([_p, _p, _p, _p, _p, _p, _i, _i, _i64, _i64, _i64, _i, _i, _i, _f, _p, _sz, _p], _i),
    "gqa_decode_partial_ex": ([_p, _p, _p, _p, _p, _p, _i, _i, _i64, _i64, _i64, _i, _i, _i, _f, _p, _sz, _p,
                               _opt], _i),
    "gqa_merge": ([_p, _p, _p, _i, _i64, _i, _p, _p], _i),
    "gqa_merge_ex": ([_p, _p, _p, _i, _i64, _i, _p, _p, _opt], _i),
    "gqa_merge_partial": ([_p, _p, _p, _i, _i64, _i, _p, _p, _p, _p], _i),
    "gqa_decode_paged": ([_p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _f, _i, _p, _sz, _p], _i),
    "gqa_decode_paged_ex": ([_p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _f, _i, _p, _sz, _p, _opt],
                            _i),
    "gqa_decode_noalloc": ([_p, _p, _p, _p, _i, _i, _i64, _i, _i, _i, _f, _p], _i),
    "gqa_decode_noalloc_check": ([_p], _i),
    "gqa_decode_paged_vllm": ([_p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _f, _i, _p, _sz, _p], _i),
    "gqa_kv8_block_bytes": ([_i, _i], _sz),
    "gqa_append": ([ctypes.POINTER(gqa_append_args), _p, _sz, _p], _i),
    "gqa_decode_kv8_workspace_size": ([_i, _i, _i, _i, _i], _sz),
    "gqa_decode_kv8": ([_p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _f, _p, _sz, _p, _opt], _i),
    "gqa_decode_kv8_status": ([_p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _f, _p, _sz, _p, _p, _opt], _i),
    "gqa_device_status": ([], _p),
    "gqa_kv8_read": ([_p, _p, _p, _p, _p, _p, _i, _i64, _i, _i, _i, _i, _i, _p, _sz, _p, _opt], _i),
    "gqa_kv4_block_bytes": ([_i, _i], _sz),
    "gqa_append_axes": ([ctypes.POINTER(gqa_append_args), _p, _i, _p, _sz, _p], _i),
    "gqa_decode_window_workspace_size": ([_i, _i, _i, _i, _i, _i], _sz),
    "gqa_decode_kv4": ([_p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _f, _i, _i, _p, _sz, _p, _p, _opt], _i),
    "gqa_decode_window": ([_p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _f, _i, _i, _p, _sz, _p, _p, _opt], _i),
    "gqa_kv4_read": ([_p, _p, _p, _p, _p, _p, _i, _i64, _i, _i, _i, _i, _i, _p, _sz, _p, _opt], _i),
    "gqa_decode_paged_vllm_ex": ([_p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _f, _i, _p, _sz, _p,
                                  _opt], _i),
}
def _bind(cdll):
    for name, (args, res) in _SIGS.items():
        fn = getattr(cdll, name)
        fn.argtypes = args
        fn.restype = res
    return cdll


_bind(lib)


def open_library(path: str):
    """Another build of the library (e.g. the bounds-checked ``libgqa_decode_checked.so``) as a
    ctypes handle with every entry point's signature set; its functions are called directly."""
    return _bind(ctypes.CDLL(path))

EXPORTED = tuple(_SIGS)


def gqa_status_string(status: int) -> str:
    return lib.gqa_status_string(int(status)).decode()


def gqa_version() -> int:
    return lib.gqa_version()


def _check(status: int, where: str) -> None:
    if status != GQA_OK:
        raise GQAError(status, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _f16(t: torch.Tensor, name: str) -> None:
    if not (t.is_cuda and t.dtype == torch.float16 and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous float16 CUDA tensor")


def _h16(t: torch.Tensor, name: str, dtype=None) -> None:
    """float16 or bfloat16 (and equal to ``dtype`` when given)."""
    if not (t.is_cuda and t.dtype in (torch.float16, torch.bfloat16) and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous float16 or bfloat16 CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype}")


def _f32(t: torch.Tensor, name: str) -> None:
    if not (t.is_cuda and t.dtype == torch.float32 and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous float32 CUDA tensor")


def _opts(n_splits=0, merge_mode=0, timeout_us=0, test_stall_cta=-1, paged_head_group=0, causal=False,
          bf16=False, mma_path=0):
    o = gqa_options()
    o.n_splits, o.merge_mode, o.timeout_us, o.test_stall_cta = int(n_splits), int(merge_mode), int(timeout_us), \
        int(test_stall_cta)
    o.paged_head_group = int(paged_head_group)
    o.causal = 1 if causal else 0
    o.bf16 = 1 if bf16 else 0
    o.mma_path = int(mma_path)
    return o


# ---------------------------------------------------------------- workspaces
_ws_lock = threading.Lock()
_ws_cache = {}


def workspace(nbytes: int, device=None, stream=None, use: Optional[str] = None) -> torch.Tensor:
    """A zero-initialised workspace of at least ``nbytes``, cached per (device, stream), and per ``use`` for
    calls whose partials may lie where others expect zeroed counters.

    Calls that share a workspace must not overlap on the GPU: keep one per stream."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    sid = _stream(stream).value or 0
    key = (dev.index, sid) if use is None else (dev.index, sid, use)
    with _ws_lock:
        t = _ws_cache.get(key)
        if t is None or t.numel() < nbytes:
            # growing the cache (rare): the replaced workspace may still be in use on `stream`, and
            # the new one is zero-filled on the current stream, which need not be `stream`; a device
            # synchronisation orders both (not while a graph is being captured: there the fill is
            # captured on the capturing stream)
            capturing = torch.cuda.is_current_stream_capturing()
            if not capturing:
                torch.cuda.synchronize(dev)
            t = torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=dev)
            if not capturing:
                torch.cuda.synchronize(dev)
            _ws_cache[key] = t
        return t


def gqa_decode_num_splits(batch, T_q, S_kv, h_q, h_kv, d_head) -> int:
    return lib.gqa_decode_num_splits(batch, T_q, S_kv, h_q, h_kv, d_head)


def gqa_paged_plan(num_seqs, h_q, h_kv, d_head, max_seq_len, partition_size=0, *, block_size=16,
                   vllm_layout=False, head_group=0):
    """(partition_size, head_group, launches) a paged call with these shapes makes on the current device
    (partition_size 0 resolved to the automatic choice)."""
    opt = _opts(0, 0, paged_head_group=head_group)
    part, hg, launches = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    st = lib.gqa_paged_plan(num_seqs, h_q, h_kv, d_head, int(block_size), int(max_seq_len), int(partition_size),
                            1 if vllm_layout else 0, ctypes.byref(opt), ctypes.byref(part), ctypes.byref(hg),
                            ctypes.byref(launches))
    _check(st, "gqa_paged_plan")
    return part.value, hg.value, launches.value


KERNELS = {0: "split", 1: "split-cluster", 2: "split-deep-ring", 3: "tcgen05"}   # GQA_KERNEL_*
FOLDS = {0: "none", 1: "cluster", 2: "merge-kernel", 3: "last-cta"}                # GQA_FOLD_*


def gqa_decode_plan(batch, T_q, S_kv, h_q, h_kv, d_head, *, n_splits=0, merge_mode=0, mma_path=0, causal=False,
                    detail=False):
    """(n_splits, mma_path, launches) of a gqa_decode call with these shapes and options on the current
    device: mma_path 1 = mma.sync split kernel, 2 = tcgen05 kernel; launches 2 with the merge kernel.
    ``detail``: a dict with those and the kernel variant and fold (names from KERNELS and FOLDS)."""
    opt = _opts(n_splits, merge_mode, causal=causal, mma_path=mma_path)
    n, path, launches, kernel, fold = (ctypes.c_int(0) for _ in range(5))
    st = lib.gqa_decode_plan_ex(batch, T_q, S_kv, h_q, h_kv, d_head, ctypes.byref(opt), ctypes.byref(n),
                                ctypes.byref(path), ctypes.byref(launches), ctypes.byref(kernel), ctypes.byref(fold))
    _check(st, "gqa_decode_plan_ex")
    if detail:
        return {"n_splits": n.value, "mma_path": path.value, "launches": launches.value,
                "kernel": KERNELS[kernel.value], "fold": FOLDS[fold.value]}
    return n.value, path.value, launches.value


def gqa_decode_workspace_size(batch, T_q, S_kv, h_q, h_kv, d_head, n_splits=0) -> int:
    return lib.gqa_decode_workspace_size(batch, T_q, S_kv, h_q, h_kv, d_head, n_splits)


def gqa_workspace_size(batch, T_q, S_kv, h_q, h_kv, d_head) -> int:
    """Workspace bytes of a gqa_decode call with the automatic split count (0: invalid shape)."""
    return lib.gqa_workspace_size(batch, T_q, S_kv, h_q, h_kv, d_head)


def gqa_paged_workspace_size(num_seqs, h_q, h_kv, d_head, max_seq_len, partition_size=512) -> int:
    return lib.gqa_paged_workspace_size(num_seqs, h_q, h_kv, d_head, max_seq_len, partition_size)


def gqa_workspace_init(ws: torch.Tensor, stream=None) -> None:
    _check(lib.gqa_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)), "gqa_workspace_init")


def gqa_workspace_check(ws: torch.Tensor, stream=None) -> int:
    """Status word of the last calls on this workspace (synchronises ``stream``)."""
    return lib.gqa_workspace_check(_ptr(ws), _stream(stream))


# ---------------------------------------------------------------- calls
def _shape_qkv(q, k, v, h_q, h_kv):
    _h16(q, "q"), _h16(k, "k", q.dtype), _h16(v, "v", q.dtype)
    if q.dim() != 3 or k.dim() != 3 or k.shape != v.shape or k.shape[0] != q.shape[0]:
        raise ValueError("q must be (batch, T_q, h_q*d_head), k and v (batch, S_kv, h_kv*d_head)")
    B, T_q, qc = q.shape
    S = k.shape[1]
    if qc % h_q or k.shape[2] % h_kv or qc // h_q != k.shape[2] // h_kv:
        raise ValueError("inconsistent head sizes")
    return B, T_q, S, qc // h_q


def gqa_decode(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, h_q: int, h_kv: int,
               scale: Optional[float] = None, *, out: Optional[torch.Tensor] = None,
               workspace_tensor: Optional[torch.Tensor] = None, stream=None, n_splits: int = 0,
               merge_mode: int = 0, timeout_us: int = 0, test_stall_cta: int = -1,
               causal: bool = False, mma_path: int = 0) -> torch.Tensor:
    """O = softmax(scale Q K^T) V for GQA decode; q (B, T_q, h_q*D), k/v (B, S_kv, h_kv*D) float16 or
    bfloat16 (all the same; the output has that dtype too).
    ``causal``: query token t sees keys j <= S_kv - T_q + t only.
    ``mma_path``: 0 automatic, 1 the mma.sync split kernel (G*T_q <= 64), 2 the tcgen05 kernel
    (G*T_q <= 128).
    ``merge_mode``: 0 automatic, 1 separate merge kernel, 2 last-arriving CTA, 3 the splits of a
    (sequence, KV head) as one thread-block cluster (at most 16) merging in distributed shared memory."""
    B, T_q, S, D = _shape_qkv(q, k, v, h_q, h_kv)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if out is None:
        out = torch.empty_like(q)
    _h16(out, "out", q.dtype)
    nbytes = gqa_decode_workspace_size(B, T_q, S, h_q, h_kv, D, n_splits)
    if nbytes == 0:
        raise GQAError(GQA_ERR_INVALID_ARG, "gqa_decode_workspace_size")
    ws = workspace(nbytes, q.device, stream) if workspace_tensor is None else workspace_tensor
    opt = _opts(n_splits, merge_mode, timeout_us, test_stall_cta, causal=causal, bf16=q.dtype == torch.bfloat16,
                mma_path=mma_path)
    st = lib.gqa_decode_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, T_q, S, h_q, h_kv, D, scale,
                           _ptr(ws), ws.numel(), _stream(stream), ctypes.byref(opt))
    _check(st, "gqa_decode")
    return out


def gqa_decode_partial(q, k, v, h_q: int, h_kv: int, s_begin: int, s_len: int, scale: Optional[float] = None, *,
                       m=None, l=None, o_part=None, workspace_tensor=None, stream=None, n_splits: int = 0,
                       merge_mode: int = 0, causal: bool = False,
                       mma_path: int = 0) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Partial (m, l, O) over keys [s_begin, s_begin+s_len): m, l (B*T_q*h_q) and O (B*T_q*h_q, D) fp32."""
    B, T_q, S, D = _shape_qkv(q, k, v, h_q, h_kv)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    R = B * T_q * h_q
    dev = q.device
    m = torch.empty(R, dtype=torch.float32, device=dev) if m is None else m
    l = torch.empty(R, dtype=torch.float32, device=dev) if l is None else l
    o_part = torch.empty(R, D, dtype=torch.float32, device=dev) if o_part is None else o_part
    _f32(m, "m"), _f32(l, "l"), _f32(o_part, "o_part")
    nbytes = gqa_decode_workspace_size(B, T_q, max(int(s_len), 1), h_q, h_kv, D, n_splits)
    if nbytes == 0:
        raise GQAError(GQA_ERR_INVALID_ARG, "gqa_decode_workspace_size")
    ws = workspace(nbytes, dev, stream) if workspace_tensor is None else workspace_tensor
    opt = _opts(n_splits, merge_mode, causal=causal, bf16=q.dtype == torch.bfloat16, mma_path=mma_path)
    st = lib.gqa_decode_partial_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(m), _ptr(l), _ptr(o_part), B, T_q, S,
                                   int(s_begin), int(s_len), h_q, h_kv, D, scale, _ptr(ws), ws.numel(),
                                   _stream(stream), ctypes.byref(opt))
    _check(st, "gqa_decode_partial")
    return m, l, o_part


def gqa_merge(m: torch.Tensor, l: torch.Tensor, o_part: torch.Tensor, *, out=None, stream=None,
              dtype=torch.float16) -> torch.Tensor:
    """Merge partials m, l (n_parts, rows), o_part (n_parts, rows, D) into o (rows, D), float16 or
    bfloat16 (the dtype of ``out`` when given, else ``dtype``)."""
    _f32(m, "m"), _f32(l, "l"), _f32(o_part, "o_part")
    n_parts, rows, D = o_part.shape
    out = torch.empty(rows, D, dtype=dtype, device=o_part.device) if out is None else out
    _h16(out, "out")
    opt = _opts(bf16=out.dtype == torch.bfloat16)
    _check(lib.gqa_merge_ex(_ptr(m), _ptr(l), _ptr(o_part), n_parts, rows, D, _ptr(out), _stream(stream),
                            ctypes.byref(opt)), "gqa_merge")
    return out


def gqa_merge_partial(m, l, o_part, *, m_out=None, l_out=None, o_out=None, stream=None):
    """Merge partials into one partial (m, l, O), all fp32."""
    _f32(m, "m"), _f32(l, "l"), _f32(o_part, "o_part")
    n_parts, rows, D = o_part.shape
    dev = o_part.device
    m_out = torch.empty(rows, dtype=torch.float32, device=dev) if m_out is None else m_out
    l_out = torch.empty(rows, dtype=torch.float32, device=dev) if l_out is None else l_out
    o_out = torch.empty(rows, D, dtype=torch.float32, device=dev) if o_out is None else o_out
    _check(lib.gqa_merge_partial(_ptr(m), _ptr(l), _ptr(o_part), n_parts, rows, D, _ptr(m_out), _ptr(l_out),
                                 _ptr(o_out), _stream(stream)), "gqa_merge_partial")
    return m_out, l_out, o_out


def gqa_decode_paged(q, k_pool, v_pool, block_tables, seq_lens, h_q: int, h_kv: int, scale: Optional[float] = None,
                     *, max_seq_len: int, partition_size: int = 512, out=None, workspace_tensor=None,
                     stream=None, timeout_us: int = 0, test_stall_cta: int = -1,
                     head_group: int = 0) -> torch.Tensor:
    """Paged decode; q (N, h_q*D), pools (num_blocks, block_size, h_kv*D) float16 or bfloat16,
    tables (N, max_blocks) int32."""
    _h16(q, "q"), _h16(k_pool, "k_pool", q.dtype), _h16(v_pool, "v_pool", q.dtype)
    if not (block_tables.is_cuda and block_tables.dtype == torch.int32 and block_tables.is_contiguous()):
        raise ValueError("block_tables must be a contiguous int32 CUDA tensor")
    if not (seq_lens.is_cuda and seq_lens.dtype == torch.int32 and seq_lens.is_contiguous()):
        raise ValueError("seq_lens must be a contiguous int32 CUDA tensor")
    q2 = q.reshape(q.shape[0], -1)
    N, qc = q2.shape
    num_blocks, block_size, kc = k_pool.shape
    if qc % h_q or kc % h_kv or qc // h_q != kc // h_kv or v_pool.shape != k_pool.shape:
        raise ValueError("inconsistent head sizes")
    D = qc // h_q
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    out = torch.empty_like(q2) if out is None else out
    _h16(out, "out", q.dtype)
    nbytes = gqa_paged_workspace_size(N, h_q, h_kv, D, max_seq_len, partition_size)
    if nbytes == 0:
        raise GQAError(GQA_ERR_INVALID_ARG, "gqa_paged_workspace_size")
    ws = workspace(nbytes, q.device, stream) if workspace_tensor is None else workspace_tensor
    opt = _opts(0, 0, timeout_us, test_stall_cta, head_group, bf16=q.dtype == torch.bfloat16)
    st = lib.gqa_decode_paged_ex(_ptr(q2), _ptr(k_pool), _ptr(v_pool), _ptr(block_tables), _ptr(seq_lens),
                                 _ptr(out), N, block_tables.shape[1], num_blocks, block_size, partition_size,
                                 h_q, h_kv, D, scale, int(max_seq_len), _ptr(ws), ws.numel(), _stream(stream),
                                 ctypes.byref(opt))
    _check(st, "gqa_decode_paged")
    return out


def gqa_decode_paged_vllm(q, k_cache, v_cache, block_tables, seq_lens, h_q: int, h_kv: int,
                          scale: Optional[float] = None, *, max_seq_len: int, partition_size: int = 0, out=None,
                          workspace_tensor=None, stream=None, timeout_us: int = 0, test_stall_cta: int = -1,
                          head_group: int = 0) -> torch.Tensor:
    """Paged decode over vLLM's cache layout, read in place: q (N, h_q*D); k_cache
    (num_blocks, h_kv, D/8, block_size, 8), v_cache (num_blocks, h_kv, D, block_size), float16 or
    bfloat16; tables (N, max_blocks) int32.  partition_size 0: automatic (512-token partitions);
    partition_size >= max_seq_len: single pass (one launch)."""
    _h16(q, "q"), _h16(k_cache, "k_cache", q.dtype), _h16(v_cache, "v_cache", q.dtype)
    if not (block_tables.is_cuda and block_tables.dtype == torch.int32 and block_tables.is_contiguous()):
        raise ValueError("block_tables must be a contiguous int32 CUDA tensor")
    if not (seq_lens.is_cuda and seq_lens.dtype == torch.int32 and seq_lens.is_contiguous()):
        raise ValueError("seq_lens must be a contiguous int32 CUDA tensor")
    q2 = q.reshape(q.shape[0], -1)
    N, qc = q2.shape
    if k_cache.dim() != 5 or k_cache.shape[4] != 8 or v_cache.dim() != 4:
        raise ValueError("k_cache must be (num_blocks, h_kv, D/8, block_size, 8), v_cache (num_blocks, h_kv, D, block_size)")
    num_blocks, hk, d8, block_size, _ = k_cache.shape
    D = d8 * 8
    if hk != h_kv or qc != h_q * D or tuple(v_cache.shape) != (num_blocks, h_kv, D, block_size):
        raise ValueError("inconsistent head sizes")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    out = torch.empty_like(q2) if out is None else out
    _h16(out, "out", q.dtype)
    nbytes = gqa_paged_workspace_size(N, h_q, h_kv, D, max_seq_len, partition_size)
    if nbytes == 0:
        raise GQAError(GQA_ERR_INVALID_ARG, "gqa_paged_workspace_size")
    ws = workspace(nbytes, q.device, stream) if workspace_tensor is None else workspace_tensor
    opt = _opts(0, 0, timeout_us, test_stall_cta, head_group, bf16=q.dtype == torch.bfloat16)
    st = lib.gqa_decode_paged_vllm_ex(_ptr(q2), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(seq_lens),
                                      _ptr(out), N, block_tables.shape[1], num_blocks, block_size, partition_size,
                                      h_q, h_kv, D, scale, int(max_seq_len), _ptr(ws), ws.numel(), _stream(stream),
                                      ctypes.byref(opt))
    _check(st, "gqa_decode_paged_vllm")
    return out


GQA_NOALLOC_SCRATCH_BYTES = 8 * 1024 * 1024


def gqa_decode_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, h_q: int, h_kv: int,
                       scale: Optional[float] = None, *, out: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """gqa_decode without a caller workspace: the library's own per-GPU device array is used.

    For callers that cannot allocate device memory.  Calls on one device share that array,
    so they must not overlap on the GPU; shapes needing more than 8 MiB of workspace raise."""
    B, T_q, S, D = _shape_qkv(q, k, v, h_q, h_kv)
    _f16(q, "q")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if out is None:
        out = torch.empty_like(q)
    _f16(out, "out")
    st = lib.gqa_decode_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, T_q, S, h_q, h_kv, D, scale,
                                _stream(stream))
    _check(st, "gqa_decode_noalloc")
    return out


def gqa_decode_noalloc_check(stream=None) -> int:
    """Status of the gqa_decode_noalloc calls on the current device since the last check
    (synchronises ``stream``; GQA_OK or GQA_ERR_TIMEOUT); clears it."""
    return lib.gqa_decode_noalloc_check(_stream(stream))


# ---------------------------------------------------------------- filling a cache; the 8-bit cache
# These calls are made for every layer of every decode step, where the host's time is what counts: their checks
# are in ``_calls`` (csrc/torch_calls.cpp), which reads the tensors' fields directly.
_calls = None


def _load_calls():
    """The extension module, imported by the first call that needs it: it belongs to one torch and one Python, and the other
    calls of this module do without it."""
    global _calls
    again = "rebuild it with this Python and torch (python -c 'import __graft_entry__ as g; g.build()')"
    try:
        module = importlib.import_module("._calls", __package__)
    except ImportError as e:
        raise ImportError(f"the extension module _calls cannot be loaded ({e}): {again}") from e
    if module.torch_version != torch.__version__:
        raise ImportError(f"the extension module _calls was built against torch {module.torch_version}, "
                          f"this is {torch.__version__}: {again}")
    _calls = module
    return module


_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)


def _in_stream(stream):
    """The stream as a context, so that what a call allocates belongs to the stream it runs on."""
    return torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream)))


def _place(t: torch.Tensor, name: str) -> Tuple[int, int]:
    """Device of a tensor and its current stream."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev, _raw_stream(dev)


def _status_workspace(t: torch.Tensor, name: str) -> Optional[torch.Tensor]:
    """The status word of calls without a workspace, ``workspace(256, use="status")`` of the stream.  It never grows, so a
    graph that was captured with it may be replayed at any time (the kernels only set bits in it).  None, the library's own
    status word of the device, for a call that is captured on a stream that has none yet."""
    dev, raw = _place(t, name)
    ws = _ws_cache.get((dev, raw, "status"))
    if ws is not None or _capturing():
        return ws
    return workspace(256, t.device, use="status")


def gqa_status_check(device=None) -> int:
    """Status of the calls of the cache operators (gqa_append, gqa_decode_kv8, gqa_decode_kv4, gqa_decode_window, gqa_kv8_read,
    gqa_kv4_read) without a ``workspace_tensor`` on a device (the current one), of all streams, eager and replayed, since the
    last check; synchronises the device and clears it."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        torch.cuda.synchronize()
        index = torch.cuda.current_device()
        with _ws_lock:
            words = [t.data_ptr() for key, t in _ws_cache.items() if key[0] == index and key[2:] == ("status",)]
        own = lib.gqa_device_status()
        if own is None:
            return GQA_ERR_CUDA
        seen = [lib.gqa_workspace_check(ctypes.c_void_p(at), _stream(None)) for at in words + [own]]
    return next((s for s in (GQA_ERR_CUDA, GQA_ERR_BOUNDS, GQA_ERR_TIMEOUT, GQA_ERR_INVALID_ARG) if s in seen), GQA_OK)


def gqa_kv8_block_bytes(block_size: int, d_head: int) -> int:
    """Bytes of one (block, head) of the 8-bit cache; 0 for a block size or d_head it does not have."""
    return lib.gqa_kv8_block_bytes(int(block_size), int(d_head))


def gqa_kv8_cache(num_blocks: int, block_size: int, h_kv: int, d_head: int, device=None) -> torch.Tensor:
    """An empty 8-bit cache: uint8 (num_blocks, h_kv, block_size * (2 * d_head + 2))."""
    n = gqa_kv8_block_bytes(block_size, d_head)
    if n == 0:
        raise GQAError(GQA_ERR_UNSUPPORTED, "gqa_kv8_cache")
    return torch.zeros(num_blocks, h_kv, n, dtype=torch.uint8, device="cuda" if device is None else device)


def gqa_append(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, h_q: int, h_kv: int, slots: torch.Tensor,
               k_cache: torch.Tensor, v_cache: Optional[torch.Tensor] = None, *,
               positions: Optional[torch.Tensor] = None, cos_sin: Optional[torch.Tensor] = None,
               interleaved: bool = False, q_weight: Optional[torch.Tensor] = None,
               k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, q_out: Optional[torch.Tensor] = None,
               workspace_tensor: Optional[torch.Tensor] = None, stream=None,
               pair_axes: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """Put new tokens into a paged cache: per-head RMS norms of q and k (where ``q_weight`` / ``k_weight`` (D)
    are given), their rotation (where ``cos_sin`` (max_position, rot_dim) float32 and ``positions`` (T) int32
    are given: rot_dim/2 cosines then rot_dim/2 sines a row; ``interleaved``: pairs (2i, 2i+1) instead of
    (i, i + rot_dim/2); with ``pair_axes`` (rot_dim/2) uint8, as gqa_pair_axes makes it, ``positions`` are
    (axes, T) and pair i is turned by the position on axis pair_axes[i]), and the write of k and v into the cache rows ``slots`` (T) int64
    (block * block_size + row; negative: not stored; no slot twice).

    q (T, h_q*D) or None, k, v (T, h_kv*D) float16 or bfloat16, rows dense (views of a fused projection serve).
    The cache: ``k_cache, v_cache`` of gqa_decode_paged (num_blocks, block_size, h_kv*D) or of
    gqa_decode_paged_vllm, or one 8-bit or 4-bit cache (gqa_kv8_cache, gqa_kv4_cache), quantised as it is written.
    Returns the queries after norm and rotation (``q_out``, which may be q itself).  What the kernel reports is in the
    status word of ``workspace_tensor``; without one, gqa_status_check has it, for captured calls too."""
    if stream is not None:
        with _in_stream(stream):
            return gqa_append(q, k, v, h_q, h_kv, slots, k_cache, v_cache, positions=positions, cos_sin=cos_sin,
                              interleaved=interleaved, q_weight=q_weight, k_weight=k_weight, eps=eps, q_out=q_out,
                              workspace_tensor=workspace_tensor, pair_axes=pair_axes)
    ws = _status_workspace(k, "k") if workspace_tensor is None else workspace_tensor
    r = (_calls or _load_calls()).append(q, k, v, h_q, h_kv, slots, k_cache, v_cache, positions, cos_sin, interleaved,
                                         q_weight, k_weight, eps, q_out, ws, pair_axes)
    if r.__class__ is int:
        raise GQAError(r, "gqa_append")
    return r


def gqa_decode_kv8_workspace_size(num_seqs: int, T_q: int, h_q: int, h_kv: int, d_head: int) -> int:
    """Workspace bytes of gqa_decode_kv8 on the current device (0: invalid shape)."""
    return lib.gqa_decode_kv8_workspace_size(num_seqs, T_q, h_q, h_kv, d_head)


def _kv8_workspace_bytes(q: torch.Tensor, h_q: int, h_kv: int) -> int:
    n = gqa_decode_kv8_workspace_size(1, q.shape[1] if q.dim() == 3 else 1, h_q, h_kv, q.shape[-1] // h_q if h_q else 0)
    if n == 0:
        raise GQAError(GQA_ERR_UNSUPPORTED, "gqa_decode_kv8_workspace_size")
    return n


def gqa_decode_kv8(q: torch.Tensor, cache: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, h_q: int,
                   h_kv: int, scale: Optional[float] = None, *, causal: bool = False,
                   out: Optional[torch.Tensor] = None, workspace_tensor: Optional[torch.Tensor] = None, stream=None,
                   timeout_us: int = 0, test_stall_cta: int = -1) -> torch.Tensor:
    """Decode attention over the 8-bit cache: q (N, h_q*D) or (N, T_q, h_q*D) float16 or bfloat16 (the output too),
    cache (num_blocks, h_kv, block_size*(2D+2)) uint8, tables (N, max_blocks) and lens (N) int32; G*T_q <= 64.
    ``causal``: query token t sees keys j <= len - T_q + t only.

    Without ``workspace_tensor`` the stream's cached workspace of this call is used; a call that is being captured into
    a graph gets one of its own, so that graphs may be replayed side by side.  What such calls report, gqa_status_check has."""
    if stream is not None:
        with _in_stream(stream):
            return gqa_decode_kv8(q, cache, block_tables, seq_lens, h_q, h_kv, scale, causal=causal, out=out,
                                  workspace_tensor=workspace_tensor, timeout_us=timeout_us,
                                  test_stall_cta=test_stall_cta)
    ws = status = workspace_tensor
    if ws is None:
        dev, raw = _place(q, "q")
        status = _ws_cache.get((dev, raw, "status"))
        if _capturing():
            ws = torch.empty(_kv8_workspace_bytes(q, h_q, h_kv), dtype=torch.uint8, device=q.device)
        else:
            ws = _ws_cache.get((dev, raw, "kv8"))
            if ws is None or status is None:
                status = _status_workspace(q, "q")
                ws = workspace(_kv8_workspace_bytes(q, h_q, h_kv), q.device, use="kv8")
    r = (_calls or _load_calls()).decode(q, cache, block_tables, seq_lens, h_q, h_kv, scale, causal, out, ws, status,
                                         timeout_us, test_stall_cta)
    if r.__class__ is int:
        if r == GQA_ERR_WORKSPACE and workspace_tensor is None and ws.numel() < _kv8_workspace_bytes(q, h_q, h_kv):
            workspace(_kv8_workspace_bytes(q, h_q, h_kv), q.device, use="kv8")       # the cached one grows
            return gqa_decode_kv8(q, cache, block_tables, seq_lens, h_q, h_kv, scale, causal=causal, out=out,
                                  timeout_us=timeout_us, test_stall_cta=test_stall_cta)
        raise GQAError(r, "gqa_decode_kv8")
    return r


def gqa_kv8_read(cache: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, d_head: int,
                 out_len: Optional[int] = None, *, begins: Optional[torch.Tensor] = None, dtype=None,
                 k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
                 workspace_tensor: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Tokens [begins[b], min(begins[b] + out_len, seq_lens[b])) of every sequence of an 8-bit cache as 16-bit
    K and V (N, out_len, h_kv*D), the layout of gqa_decode.  Into ``k_out`` / ``v_out`` (the one left out is
    not read; rows past a sequence's last token stay as they were), or, with neither, into zeros of ``dtype``
    (float16) and ``out_len`` tokens.  begins (N) int32, default 0.  Reports as those of gqa_append."""
    return _read("gqa_kv8_read", cache, block_tables, seq_lens, d_head, out_len, begins, dtype, k_out, v_out, workspace_tensor,
                 stream)


def _read(name, cache, block_tables, seq_lens, d_head, out_len, begins, dtype, k_out, v_out, workspace_tensor, stream):
    """gqa_kv8_read and gqa_kv4_read."""
    if stream is not None:
        with _in_stream(stream):
            return _read(name, cache, block_tables, seq_lens, d_head, out_len, begins, dtype, k_out, v_out, workspace_tensor,
                         None)
    ws = _status_workspace(cache, "cache") if workspace_tensor is None else workspace_tensor
    if k_out is None and v_out is None:
        if out_len is None:
            raise ValueError("pass out_len, or k_out / v_out")
        shape = (block_tables.shape[0], out_len, cache.shape[1] * d_head)
        k_out, v_out = (torch.zeros(shape, dtype=dtype or torch.float16, device=cache.device) for _ in range(2))
    elif out_len is not None or dtype is not None:
        for t in (k_out, v_out):
            if t is not None and (out_len not in (None, t.shape[1]) or dtype not in (None, t.dtype)):
                raise ValueError("k_out and v_out must be (N, out_len, h_kv*d_head) of dtype")
    calls = _calls or _load_calls()
    r = (calls.read if name == "gqa_kv8_read" else calls.read4)(cache, block_tables, seq_lens, d_head, begins, k_out, v_out, ws)
    if r:
        raise GQAError(r, name)
    return k_out, v_out


# ---------------------------------------------------------------- several position axes; the 4-bit cache; windows
def gqa_pair_axes(sections: Sequence[int], *, in_turn: bool = False, device=None) -> torch.Tensor:
    """The axis of each rotated pair for gqa_append's ``pair_axes``, uint8 (sum(sections),): sections[i] pairs on axis i, as
    runs one after the other, or ``in_turn``: dealt out one to each axis in turn until its section is used up."""
    sections = [int(n) for n in sections]
    if not 1 <= len(sections) <= 32 or min(sections) < 0:
        raise ValueError("sections must be one to 32 whole numbers, none below 0")
    if in_turn:
        order = [i for k in range(max(sections)) for i, n in enumerate(sections) if k < n]
    else:
        order = [i for i, n in enumerate(sections) for _ in range(n)]
    return torch.tensor(order, dtype=torch.uint8, device="cuda" if device is None else device)


def gqa_kv4_block_bytes(block_size: int, d_head: int) -> int:
    """Bytes of one (block, head) of the 4-bit cache; 0 for a block size or d_head it does not have."""
    return lib.gqa_kv4_block_bytes(int(block_size), int(d_head))


def gqa_kv4_cache(num_blocks: int, block_size: int, h_kv: int, d_head: int, device=None) -> torch.Tensor:
    """An empty 4-bit cache: uint8 (num_blocks, h_kv, block_size * (d_head + d_head / 8))."""
    n = gqa_kv4_block_bytes(block_size, d_head)
    if n == 0:
        raise GQAError(GQA_ERR_UNSUPPORTED, "gqa_kv4_cache")
    return torch.zeros(num_blocks, h_kv, n, dtype=torch.uint8, device="cuda" if device is None else device)


def gqa_decode_window_workspace_size(num_seqs: int, T_q: int, h_q: int, h_kv: int, d_head: int,
                                     cache_layout: int = GQA_CACHE_ROWS) -> int:
    """Workspace bytes of gqa_decode_window (GQA_CACHE_ROWS) or gqa_decode_kv4 (GQA_CACHE_KV4) on the current device
    (0: invalid shape)."""
    return lib.gqa_decode_window_workspace_size(num_seqs, T_q, h_q, h_kv, d_head, cache_layout)


def _window_workspace_bytes(q: torch.Tensor, h_q: int, h_kv: int, layout: int) -> int:
    n = gqa_decode_window_workspace_size(1, q.shape[1] if q.dim() == 3 else 1, h_q, h_kv, q.shape[-1] // h_q if h_q else 0,
                                         layout)
    if n == 0:
        raise GQAError(GQA_ERR_UNSUPPORTED, "gqa_decode_window_workspace_size")
    return n


def _window(name, layout, q, k, v, block_tables, seq_lens, h_q, h_kv, scale, window, sinks, causal, out, workspace_tensor,
            timeout_us, test_stall_cta):
    """gqa_decode_kv4 (v None) and gqa_decode_window on the current stream."""
    ws = status = workspace_tensor
    if ws is None:
        dev, raw = _place(q, "q")
        status = _ws_cache.get((dev, raw, "status"))
        if _capturing():
            ws = torch.empty(_window_workspace_bytes(q, h_q, h_kv, layout), dtype=torch.uint8, device=q.device)
        else:
            ws = _ws_cache.get((dev, raw, "window"))
            if ws is None or status is None:
                status = _status_workspace(q, "q")
                ws = workspace(_window_workspace_bytes(q, h_q, h_kv, layout), q.device, use="window")
    r = (_calls or _load_calls()).window(q, k, v, block_tables, seq_lens, h_q, h_kv, scale, window, sinks, causal, out, ws,
                                         status, timeout_us, test_stall_cta)
    if r.__class__ is int:
        if r == GQA_ERR_WORKSPACE and workspace_tensor is None and ws.numel() < _window_workspace_bytes(q, h_q, h_kv, layout):
            workspace(_window_workspace_bytes(q, h_q, h_kv, layout), q.device, use="window")       # the cached one grows
            return _window(name, layout, q, k, v, block_tables, seq_lens, h_q, h_kv, scale, window, sinks, causal, out, None,
                           timeout_us, test_stall_cta)
        raise GQAError(r, name)
    return r


def gqa_decode_kv4(q: torch.Tensor, cache: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, h_q: int,
                   h_kv: int, scale: Optional[float] = None, *, causal: bool = False, window: int = 0, sinks: int = 0,
                   out: Optional[torch.Tensor] = None, workspace_tensor: Optional[torch.Tensor] = None, stream=None,
                   timeout_us: int = 0, test_stall_cta: int = -1) -> torch.Tensor:
    """Decode attention over the 4-bit cache: q (N, h_q*D) or (N, T_q, h_q*D) float16 or bfloat16 (the output too),
    cache (num_blocks, h_kv, block_size*(D + D/8)) uint8, tables (N, max_blocks) and lens (N) int32; G*T_q <= 64.
    ``causal``: query token t has the place len - T_q + t and sees the keys up to it only.  ``window`` > 0: of those only the
    ``window`` newest, its own among them, and the first ``sinks`` of the sequence; blocks that no token sees are not looked
    up in the table.  Workspaces and reports as those of gqa_decode_kv8."""
    if stream is not None:
        with _in_stream(stream):
            return _window("gqa_decode_kv4", GQA_CACHE_KV4, q, cache, None, block_tables, seq_lens, h_q, h_kv, scale, window,
                           sinks, causal, out, workspace_tensor, timeout_us, test_stall_cta)
    return _window("gqa_decode_kv4", GQA_CACHE_KV4, q, cache, None, block_tables, seq_lens, h_q, h_kv, scale, window, sinks,
                   causal, out, workspace_tensor, timeout_us, test_stall_cta)


def gqa_decode_window(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor, block_tables: torch.Tensor,
                      seq_lens: torch.Tensor, h_q: int, h_kv: int, scale: Optional[float] = None, *, window: int,
                      sinks: int = 0, causal: bool = False, out: Optional[torch.Tensor] = None,
                      workspace_tensor: Optional[torch.Tensor] = None, stream=None, timeout_us: int = 0,
                      test_stall_cta: int = -1) -> torch.Tensor:
    """gqa_decode_kv4 over the 16-bit pools of gqa_decode_paged: k_pool, v_pool (num_blocks, block_size, h_kv*D) of q's dtype.
    ``window`` 0: every key is visible."""
    if stream is not None:
        with _in_stream(stream):
            return _window("gqa_decode_window", GQA_CACHE_ROWS, q, k_pool, v_pool, block_tables, seq_lens, h_q, h_kv, scale,
                           window, sinks, causal, out, workspace_tensor, timeout_us, test_stall_cta)
    return _window("gqa_decode_window", GQA_CACHE_ROWS, q, k_pool, v_pool, block_tables, seq_lens, h_q, h_kv, scale, window,
                   sinks, causal, out, workspace_tensor, timeout_us, test_stall_cta)


def gqa_kv4_read(cache: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, d_head: int,
                 out_len: Optional[int] = None, *, begins: Optional[torch.Tensor] = None, dtype=None,
                 k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
                 workspace_tensor: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """gqa_kv8_read of a 4-bit cache."""
    return _read("gqa_kv4_read", cache, block_tables, seq_lens, d_head, out_len, begins, dtype, k_out, v_out, workspace_tensor,
                 stream)
