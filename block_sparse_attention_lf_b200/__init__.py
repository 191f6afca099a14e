"""Python binding of liblf_hsa.so, the B200 Light Forcing HSA library.

Argument marshalling only: every step of the HSA call runs in the library's
CUDA kernels (sm_100a). PyTorch supplies device memory and the current stream.
The functions carry the C names (``lf_pool``, ``lf_select_frames``,
``lf_select_blocks``, ``lf_block_sparse_attn``, ``lf_cag_budget``, ...) and
take preallocated torch tensors; ``HSACall`` is a convenience wrapper that
allocates the intermediate buffers and runs the four device steps in order.

The library is loaded from this directory (``liblf_hsa.so``, built by
``build.py``); importing this module fails loudly when it is missing, and the
device entry points raise when the tensors are not CUDA tensors. There is no
CPU fallback.

Typical use (q [B,H,n_cur*F,D], k and v [B,H,n_frames*F,D], bf16 on the GPU)::

    shape = LfShape.make(B, H, D, F, n_frames, n_sink, n_recent, n_cur)
    call = HSACall(shape, chunk_index, topk_frames, topk_blocks)
    out = call(q, k, v)          # pool, select frames, select blocks, attend

``HSACall.attend`` uses ``lf_block_sparse_attn_ws`` with a workspace sized by
``lf_attn_split_plan`` (the split of the attention's last, partial wave);
``tail_pieces=1`` turns the split off. ``lf_pool_range`` re-pools only some
frames (keep the pooled keys of past frames between calls),
``lf_select_blocks_1d`` gives the single-granularity lists of the ablation, and
``lf_cag_budget`` / ``lf_blocks_for_sparsity`` turn a sparsity target into
per-chunk block counts.

Fine-tuning a block under sparsity (the call's gradient, and what stands on both sides
of the call)::

    lf_norm_gate(NormGateShape.make(rows, dim, F, torch.float32, torch.bfloat16, pre="layer", post="none"),
                 x, y, r, h, gate=..., scale=..., shift=...)       # residual stream r, block input h
    call = HSACall(shape, chunk_index, topk_frames, topk_blocks, train=True)
    call.load(RopePlan.make(D, axis_dims=(44, 42, 42)), qkv, positions, q, k, v)
    out = call(q, k, v)                                            # also keeps lse and out_lo
    call.backward(q, k, v, dout, dq, dk, dv)                       # over the lists of the forward
    call.load_bwd(plan, dq, dk, dv, positions, dqkv)
    lf_norm_gate_bwd(..., x, y, dr, dh, dx, dy, grads, workspace)

Nothing here records an autograd graph; a training program calls the gradients where its
own does.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
from dataclasses import dataclass
from typing import Optional, Sequence, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblf_hsa.so")

__all__ = [
    "LfShape", "LfError", "lib", "lf_pool", "lf_pool_range", "lf_select_frames", "lf_select_blocks",
    "lf_select_blocks_1d", "lf_frame_index_build", "lf_select_frames_ivf", "FrameIndex", "lf_select_mask",
    "lf_quant_fp8_rows", "lf_block_sparse_attn_fp8",
    "lf_block_sparse_attn", "lf_block_sparse_attn_ws", "lf_attn_split_plan", "lf_cag_budget",
    "lf_blocks_for_sparsity", "lf_frames_selected", "lf_list_capacity", "lf_get_device_error",
    "lf_status_string", "lf_version", "HSACall",
    "lf_block_sparse_attn_lse", "lf_attn_lse_split_plan", "lf_block_sparse_attn_bwd", "lf_attn_bwd_workspace",
    "RopePlan", "lf_rope", "NormGateShape", "lf_norm_gate", "lf_norm_gate_bwd", "lf_norm_gate_bwd_workspace",
    "ABI_FUNCTIONS", "shard_units", "shard_shape", "unit_view",
]

# Names declared in include/lf_hsa.h.
ABI_FUNCTIONS = (
    "lf_pool", "lf_pool_range", "lf_frames_selected", "lf_select_frames", "lf_list_capacity", "lf_select_blocks",
    "lf_select_blocks_1d", "lf_frame_index_build", "lf_select_frames_ivf", "lf_select_mask", "lf_quant_fp8_rows",
    "lf_block_sparse_attn_fp8",
    "lf_block_sparse_attn", "lf_block_sparse_attn_ws", "lf_attn_split_plan", "lf_block_sparse_attn_static",
    "lf_cag_budget", "lf_blocks_for_sparsity", "lf_get_device_error", "lf_status_string", "lf_version",
    "lf_block_sparse_attn_lse", "lf_attn_lse_split_plan", "lf_attn_bwd_workspace", "lf_block_sparse_attn_bwd",
    "lf_rope_plan_init", "lf_rope", "lf_norm_gate", "lf_norm_gate_bwd_workspace", "lf_norm_gate_bwd",
)

LF_OK = 0
STATUS_NAMES = {
    0: "LF_OK", 1: "LF_ERR_NULL", 2: "LF_ERR_ALIGN", 3: "LF_ERR_SHAPE", 4: "LF_ERR_TOPK",
    5: "LF_ERR_CAP", 6: "LF_ERR_INFEASIBLE", 7: "LF_ERR_CUDA", 8: "LF_ERR_DEVICE_TIMEOUT",
    9: "LF_ERR_ARG", 10: "LF_ERR_LIST", 11: "LF_ERR_NO_DEVICE", 12: "LF_ERR_SCRATCH",
}


class LfError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} ({_lib.lf_status_string(status).decode()})")


class LfShape(ctypes.Structure):
    """Mirror of ``lf_hsa_shape``."""

    _fields_ = [
        ("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("frame_tokens", ctypes.c_int32), ("block_tokens", ctypes.c_int32),
        ("n_frames", ctypes.c_int32), ("n_sink", ctypes.c_int32), ("n_recent", ctypes.c_int32),
        ("n_cur", ctypes.c_int32), ("kv_stride", ctypes.c_int64),
    ]

    @classmethod
    def make(cls, batch, heads, head_dim, frame_tokens, n_frames, n_sink, n_recent, n_cur,
             block_tokens=64, kv_stride=0) -> "LfShape":
        return cls(batch, heads, head_dim, frame_tokens, block_tokens, n_frames, n_sink, n_recent,
                   n_cur, kv_stride)

    @property
    def bpf(self) -> int:
        return -(-self.frame_tokens // self.block_tokens)

    @property
    def Rq(self) -> int:
        return self.n_cur * self.bpf

    @property
    def Nkv(self) -> int:
        return self.n_frames * self.bpf

    @property
    def Lq(self) -> int:
        return self.n_cur * self.frame_tokens

    @property
    def Lkv(self) -> int:
        return self.n_frames * self.frame_tokens


class RopePlan(ctypes.Structure):
    """Mirror of ``lf_rope_plan``: a head's rotary frequencies (``make``), kept by the caller."""

    _fields_ = [
        ("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
        ("n_axes", ctypes.c_int32), ("axis_dims", ctypes.c_int32 * 3), ("amplitude", ctypes.c_float),
        ("turns", ctypes.c_double * 128),
    ]

    LAYOUTS = {"interleaved": 0, "half": 1}
    SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}

    @classmethod
    def make(cls, head_dim: int, rot_dim: Optional[int] = None, layout: str = "interleaved",
             axis_dims: Optional[Sequence[int]] = None, base: float = 10000.0, scaling: str = "none",
             factor: float = 1.0, original_length: float = 0.0, beta_fast: float = 32.0,
             beta_slow: float = 1.0) -> "RopePlan":
        """``axis_dims``: rotated dimensions of each position axis (one axis of ``rot_dim`` by default);
        ``scaling`` stretches axis 0 by ``factor`` (``original_length``: trained positions, for yarn)."""
        if layout not in cls.LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(cls.LAYOUTS)}")
        if scaling not in cls.SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(cls.SCALINGS)}")
        rot = head_dim if rot_dim is None else rot_dim
        dims = [rot] if axis_dims is None else [int(d) for d in axis_dims]
        plan = cls()
        arr = (ctypes.c_int32 * max(len(dims), 1))(*dims)
        _check(_lib.lf_rope_plan_init(ctypes.byref(plan), head_dim, rot, cls.LAYOUTS[layout], len(dims),
                                      ctypes.cast(arr, ctypes.c_void_p), float(base), cls.SCALINGS[scaling],
                                      float(factor), float(original_length), float(beta_fast), float(beta_slow)),
               "RopePlan.make")
        return plan


class _RopeIo(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("x_stride", ctypes.c_int64 * 3),
                ("out_stride", ctypes.c_int64 * 3), ("heads", ctypes.c_int32), ("rotate", ctypes.c_int32)]


class NormGateShape(ctypes.Structure):
    """Mirror of ``lf_norm_gate_shape``."""

    _fields_ = [
        ("rows", ctypes.c_int64), ("rows_per_group", ctypes.c_int64), ("dim", ctypes.c_int32),
        ("x_dtype", ctypes.c_int32), ("y_dtype", ctypes.c_int32), ("pre_norm", ctypes.c_int32),
        ("post_norm", ctypes.c_int32), ("eps", ctypes.c_float), ("residual_scale", ctypes.c_float),
    ]

    NORMS = {"none": 0, "rms": 1, "layer": 2}

    @classmethod
    def make(cls, rows: int, dim: int, rows_per_group: Optional[int] = None, x_dtype=None, y_dtype=None,
             pre: str = "layer", post: str = "none", eps: float = 1e-6, residual_scale: float = 1.0) -> "NormGateShape":
        """``rows_per_group``: consecutive rows that share gate, scale and shift (default: all rows);
        dtypes default to bf16."""
        if pre not in cls.NORMS or post not in cls.NORMS:
            raise ValueError(f"norms must be one of {sorted(cls.NORMS)}")
        bf = _bf16()
        return cls(rows, max(rows, 1) if rows_per_group is None else rows_per_group, dim, _dtype_code(x_dtype or bf),
                   _dtype_code(y_dtype or bf), cls.NORMS[pre], cls.NORMS[post], eps, residual_scale)

    @property
    def groups(self) -> int:
        return -(-self.rows // max(self.rows_per_group, 1))  # below 1: refused by the library


_NORM_VECTORS = ("gate", "scale", "shift", "pre_w", "pre_b", "post_w", "post_b")


class _NormVectors(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in _NORM_VECTORS]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m block_sparse_attention_lf_b200.build` "
            "(nvcc, sm_100a). There is no fallback implementation.")
    L = ctypes.CDLL(LIB_PATH)
    P, I32, F32, F64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_double
    S = ctypes.POINTER(LfShape)
    sig = {
        "lf_pool": ([S, P, P, P, P, P, P], I32),
        "lf_pool_range": ([S, P, P, I32, I32, I32, P, P, P, P], I32),
        "lf_frames_selected": ([S, I32, I32], I32),
        "lf_select_frames": ([S, I32, I32, P, P, P, P], I32),
        "lf_list_capacity": ([S, I32, I32, I32], I32),
        "lf_select_blocks": ([S, I32, I32, I32, P, P, P, P, P, I32, P], I32),
        "lf_select_blocks_1d": ([S, I32, I32, P, P, P, P, I32, P], I32),
        "lf_frame_index_build": ([S, I32, I32, P, P, P, P, P, P], I32),
        "lf_select_mask": ([S, I32, I32, I32, P, P, P, P, P, P, I32, P], I32),
        "lf_quant_fp8_rows": ([P, ctypes.c_int64, I32, P, P, P], I32),
        "lf_block_sparse_attn_fp8": ([S, P, P, P, P, P, P, P, I32, F32, P, I32, P, ctypes.c_int64, P], I32),
        "lf_select_frames_ivf": ([S, I32, I32, I32, I32, P, P, P, P, P, P, P], I32),
        "lf_block_sparse_attn": ([S, P, P, P, P, P, I32, F32, P, P], I32),
        "lf_block_sparse_attn_ws": ([S, P, P, P, P, P, I32, F32, P, I32, P, ctypes.c_int64, P], I32),
        "lf_attn_split_plan": ([S, I32, I32, ctypes.POINTER(I32), ctypes.POINTER(I32),
                                ctypes.POINTER(ctypes.c_int64)], I32),
        "lf_block_sparse_attn_static": ([S, P, P, P, P, P, I32, F32, P, I32, P], I32),
        "lf_cag_budget": ([I32, P, P, F64, F64, I32, P, P], I32),
        "lf_blocks_for_sparsity": ([F64, I32, I32, I32], I32),
        "lf_get_device_error": ([ctypes.POINTER(I32)], I32),
        "lf_block_sparse_attn_lse": ([S, P, P, P, P, P, I32, F32, P, P, P, I32, P, ctypes.c_int64, P], I32),
        "lf_attn_lse_split_plan": ([S, I32, I32, ctypes.POINTER(I32), ctypes.POINTER(I32),
                                   ctypes.POINTER(ctypes.c_int64)], I32),
        "lf_attn_bwd_workspace": ([S], ctypes.c_int64),
        "lf_block_sparse_attn_bwd": ([S, P, P, P, P, P, P, P, P, P, I32, F32, P, P, P, P, ctypes.c_int64, P], I32),
        "lf_rope_plan_init": ([P, I32, I32, I32, I32, P, F64, I32, F64, F64, F64, F64], I32),
        "lf_rope": ([P, I32, I32, I32, P, ctypes.c_int64, P, I32, I32, P], I32),
        "lf_norm_gate": ([P, P, P, P, P, P, P], I32),
        "lf_norm_gate_bwd_workspace": ([P], ctypes.c_int64),
        "lf_norm_gate_bwd": ([P, P, P, P, P, P, P, P, P, P, ctypes.c_int64, P], I32),
        "lf_status_string": ([I32], ctypes.c_char_p),
        "lf_version": ([], ctypes.c_char_p),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    return L


_lib = _load()
lib = _lib


def _check(status: int, where: str) -> None:
    if status != LF_OK:
        raise LfError(status, where)


def _dev_ptr(t, dtype, name: str):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _bf16():
    import torch
    return torch.bfloat16


def _dtype_code(dtype) -> int:
    import torch
    codes = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
    if dtype not in codes:
        raise TypeError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
    return codes[dtype]


def _sized_ptr(t, dtype, shape, device, name: str) -> int:
    """Address of a contiguous CUDA tensor of exactly this dtype and shape on ``device``."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _dev_ptr(t, dtype, name)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be on the current device (cuda:{device}), got {t.device}")


def _device() -> int:
    import torch
    return torch.cuda.current_device()


def _raw_stream(stream, device: int) -> int:
    """Handle of ``stream``, or of the device's current stream."""
    if stream is None:
        import torch
        get = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # without building a Stream object
        return get(device) if get is not None else torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def lf_version() -> str:
    return _lib.lf_version().decode()


def lf_status_string(status: int) -> str:
    return _lib.lf_status_string(status).decode()


def lf_frames_selected(shape: LfShape, chunk_index: int, topk_frames: int) -> int:
    return _lib.lf_frames_selected(ctypes.byref(shape), chunk_index, topk_frames)


def lf_list_capacity(shape: LfShape, chunk_index: int, topk_frames: int, topk_blocks: int) -> int:
    return _lib.lf_list_capacity(ctypes.byref(shape), chunk_index, topk_frames, topk_blocks)


def lf_blocks_for_sparsity(s: float, n_kv_blocks: int, n_sel_frames: int, bpf: int) -> int:
    return _lib.lf_blocks_for_sparsity(float(s), n_kv_blocks, n_sel_frames, bpf)


def lf_pool_range(shape: LfShape, q, k, frame_begin: int, frame_end: int, q_pool, k_pool, k_frame,
                  pool_q: bool = True, stream=None) -> None:
    """Pool KV frames [frame_begin, frame_end) (and q when ``pool_q``) into the
    same buffers lf_pool fills; other entries are left as they are."""
    import torch
    bf = _bf16()
    qp = _dev_ptr(q, bf, "q") if pool_q else None
    qpp = _dev_ptr(q_pool, torch.float32, "q_pool") if pool_q else None
    _check(_lib.lf_pool_range(ctypes.byref(shape), qp, _dev_ptr(k, bf, "k"), int(frame_begin), int(frame_end),
                              1 if pool_q else 0, qpp, _dev_ptr(k_pool, torch.float32, "k_pool"),
                              _dev_ptr(k_frame, torch.float32, "k_frame"), _stream(stream)), "lf_pool_range")


def lf_pool(shape: LfShape, q, k, q_pool, k_pool, k_frame, stream=None) -> None:
    import torch
    bf = _bf16()
    _check(_lib.lf_pool(ctypes.byref(shape), _dev_ptr(q, bf, "q"), _dev_ptr(k, bf, "k"),
                        _dev_ptr(q_pool, torch.float32, "q_pool"),
                        _dev_ptr(k_pool, torch.float32, "k_pool"),
                        _dev_ptr(k_frame, torch.float32, "k_frame"), _stream(stream)), "lf_pool")


def lf_select_frames(shape: LfShape, chunk_index: int, topk_frames: int, q_pool, k_frame,
                     frame_sel, stream=None) -> None:
    import torch
    _check(_lib.lf_select_frames(ctypes.byref(shape), chunk_index, topk_frames,
                                 _dev_ptr(q_pool, torch.float32, "q_pool"),
                                 _dev_ptr(k_frame, torch.float32, "k_frame"),
                                 _dev_ptr(frame_sel, torch.int32, "frame_sel"), _stream(stream)),
           "lf_select_frames")


def lf_select_blocks(shape: LfShape, chunk_index: int, topk_frames: int, topk_blocks: int, q_pool,
                     k_pool, frame_sel, block_list, block_count, list_cap: int, stream=None) -> None:
    import torch
    _check(_lib.lf_select_blocks(ctypes.byref(shape), chunk_index, topk_frames, topk_blocks,
                                 _dev_ptr(q_pool, torch.float32, "q_pool"),
                                 _dev_ptr(k_pool, torch.float32, "k_pool"),
                                 _dev_ptr(frame_sel, torch.int32, "frame_sel"),
                                 _dev_ptr(block_list, torch.int32, "block_list"),
                                 _dev_ptr(block_count, torch.int32, "block_count"), list_cap,
                                 _stream(stream)), "lf_select_blocks")


def lf_select_mask(shape: LfShape, chunk_index: int, topk_frames: int, topk_blocks: int, q_pool, k_frame, k_pool,
                   frame_sel, block_list, block_count, list_cap: int, stream=None) -> None:
    """Both selection levels in one launch (the results of lf_select_frames + lf_select_blocks)."""
    import torch
    f32, i32 = torch.float32, torch.int32
    _check(_lib.lf_select_mask(ctypes.byref(shape), chunk_index, topk_frames, topk_blocks,
                               _dev_ptr(q_pool, f32, "q_pool"), _dev_ptr(k_frame, f32, "k_frame"),
                               _dev_ptr(k_pool, f32, "k_pool"), _dev_ptr(frame_sel, i32, "frame_sel"),
                               _dev_ptr(block_list, i32, "block_list"), _dev_ptr(block_count, i32, "block_count"),
                               list_cap, _stream(stream)), "lf_select_mask")


def lf_quant_fp8_rows(x, x8, scales, stream=None) -> None:
    """Per-row e4m3 codes (uint8 tensor shaped like x) and fp32 scales (x.shape[:-1]) of bf16 x."""
    import torch
    D = x.shape[-1]
    n = x.numel() // D
    _check(_lib.lf_quant_fp8_rows(_dev_ptr(x, _bf16(), "x"), n, D, _dev_ptr(x8, torch.uint8, "x8"),
                                  _dev_ptr(scales, torch.float32, "scales"), _stream(stream)), "lf_quant_fp8_rows")


def lf_select_blocks_1d(shape: LfShape, chunk_index: int, topk_blocks: int, q_pool, k_pool,
                        block_list, block_count, list_cap: int, stream=None) -> None:
    import torch
    _check(_lib.lf_select_blocks_1d(ctypes.byref(shape), chunk_index, topk_blocks,
                                    _dev_ptr(q_pool, torch.float32, "q_pool"),
                                    _dev_ptr(k_pool, torch.float32, "k_pool"),
                                    _dev_ptr(block_list, torch.int32, "block_list"),
                                    _dev_ptr(block_count, torch.int32, "block_count"), list_cap,
                                    _stream(stream)), "lf_select_blocks_1d")


@dataclass
class FrameIndex:
    """Device buffers of a coarse frame index (lf_frame_index_build): fp32 centroids
    [B,H,n_clusters,D], int32 labels and members [B,H,max(n_mem,1)], int32 offsets
    [B,H,n_clusters+1]."""
    n_clusters: int
    centroids: "object"
    labels: "object"
    offsets: "object"
    members: "object"

    @classmethod
    def empty(cls, shape: LfShape, n_clusters: int, device="cuda") -> "FrameIndex":
        import torch
        n_mem = max(shape.n_frames - shape.n_sink - shape.n_recent - shape.n_cur, 1)
        bh = (shape.batch, shape.heads)
        return cls(n_clusters,
                   torch.empty(*bh, n_clusters, shape.head_dim, dtype=torch.float32, device=device),
                   torch.empty(*bh, n_mem, dtype=torch.int32, device=device),
                   torch.empty(*bh, n_clusters + 1, dtype=torch.int32, device=device),
                   torch.empty(*bh, n_mem, dtype=torch.int32, device=device))


def lf_frame_index_build(shape: LfShape, k_frame, index: FrameIndex, iters: int = 25, stream=None) -> None:
    """k-means index over each head's memory-frame means (k_frame from lf_pool)."""
    import torch
    i32 = torch.int32
    _check(_lib.lf_frame_index_build(ctypes.byref(shape), int(index.n_clusters), int(iters),
                                     _dev_ptr(k_frame, torch.float32, "k_frame"),
                                     _dev_ptr(index.centroids, torch.float32, "centroids"),
                                     _dev_ptr(index.labels, i32, "labels"), _dev_ptr(index.offsets, i32, "offsets"),
                                     _dev_ptr(index.members, i32, "members"), _stream(stream)),
           "lf_frame_index_build")


def lf_select_frames_ivf(shape: LfShape, chunk_index: int, topk_frames: int, index: FrameIndex, n_probe: int,
                         q_pool, k_frame, frame_sel, stream=None) -> None:
    """Frame selection probing the index (same output layout as lf_select_frames)."""
    import torch
    i32 = torch.int32
    _check(_lib.lf_select_frames_ivf(ctypes.byref(shape), chunk_index, topk_frames, int(index.n_clusters),
                                     int(n_probe), _dev_ptr(q_pool, torch.float32, "q_pool"),
                                     _dev_ptr(k_frame, torch.float32, "k_frame"),
                                     _dev_ptr(index.centroids, torch.float32, "centroids"),
                                     _dev_ptr(index.offsets, i32, "offsets"), _dev_ptr(index.members, i32, "members"),
                                     _dev_ptr(frame_sel, i32, "frame_sel"), _stream(stream)),
           "lf_select_frames_ivf")


def lf_block_sparse_attn(shape: LfShape, q, k, v, block_list, block_count, list_cap: int,
                         softmax_scale: float, out, stream=None) -> None:
    import torch
    bf = _bf16()
    _check(_lib.lf_block_sparse_attn(ctypes.byref(shape), _dev_ptr(q, bf, "q"), _dev_ptr(k, bf, "k"),
                                     _dev_ptr(v, bf, "v"),
                                     _dev_ptr(block_list, torch.int32, "block_list"),
                                     _dev_ptr(block_count, torch.int32, "block_count"), list_cap,
                                     float(softmax_scale), _dev_ptr(out, bf, "out"), _stream(stream)),
           "lf_block_sparse_attn")


def lf_block_sparse_attn_ws(shape: LfShape, q, k, v, block_list, block_count, list_cap: int,
                            softmax_scale: float, out, workspace=None, tail_pieces: int = 0,
                            stream=None) -> None:
    """``workspace``: a uint8 device tensor (or None: no split)."""
    import torch
    bf = _bf16()
    ws = _dev_ptr(workspace, torch.uint8, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() if workspace is not None else 0
    _check(_lib.lf_block_sparse_attn_ws(ctypes.byref(shape), _dev_ptr(q, bf, "q"), _dev_ptr(k, bf, "k"),
                                        _dev_ptr(v, bf, "v"),
                                        _dev_ptr(block_list, torch.int32, "block_list"),
                                        _dev_ptr(block_count, torch.int32, "block_count"), list_cap,
                                        float(softmax_scale), _dev_ptr(out, bf, "out"), int(tail_pieces),
                                        ws, ws_bytes, _stream(stream)),
           "lf_block_sparse_attn_ws")


def lf_block_sparse_attn_fp8(shape: LfShape, q8, k8, q_scale, k_scale, v, block_list, block_count, list_cap: int,
                             softmax_scale: float, out, workspace=None, tail_pieces: int = 0, stream=None) -> None:
    """Attention with e4m3 q8 / k8 (uint8 codes from lf_quant_fp8_rows) and fp32 per-token scales."""
    import torch
    bf = _bf16()
    u8, f32, i32 = torch.uint8, torch.float32, torch.int32
    ws = _dev_ptr(workspace, u8, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() if workspace is not None else 0
    _check(_lib.lf_block_sparse_attn_fp8(ctypes.byref(shape), _dev_ptr(q8, u8, "q8"), _dev_ptr(k8, u8, "k8"),
                                         _dev_ptr(q_scale, f32, "q_scale"), _dev_ptr(k_scale, f32, "k_scale"),
                                         _dev_ptr(v, bf, "v"), _dev_ptr(block_list, i32, "block_list"),
                                         _dev_ptr(block_count, i32, "block_count"), list_cap, float(softmax_scale),
                                         _dev_ptr(out, bf, "out"), int(tail_pieces), ws, ws_bytes, _stream(stream)),
           "lf_block_sparse_attn_fp8")


def _attn_args(shape: LfShape, dev: int, q, k, v, block_list, block_count, list_cap: int):
    import torch
    bf, i32 = torch.bfloat16, torch.int32
    B, H, D = shape.batch, shape.heads, shape.head_dim
    kv = (B, H, shape.kv_stride or shape.Lkv, D)
    return (_sized_ptr(q, bf, (B, H, shape.Lq, D), dev, "q"), _sized_ptr(k, bf, kv, dev, "k"),
            _sized_ptr(v, bf, kv, dev, "v"),
            _sized_ptr(block_list, i32, (B, H, shape.Rq, list_cap), dev, "block_list"),
            _sized_ptr(block_count, i32, (B, H, shape.Rq), dev, "block_count"))


def lf_block_sparse_attn_lse(shape: LfShape, q, k, v, block_list, block_count, list_cap: int, softmax_scale: float,
                             out, lse, workspace=None, tail_pieces: int = 0, stream=None, out_lo=None) -> None:
    """lf_block_sparse_attn_ws that also writes each row's log-sum-exp (fp32 [B,H,Lq]; -inf for an empty list)
    and, for the gradient, ``out_lo`` (like out): out + out_lo is the row under the rounded softmax weights. With
    ``out_lo`` the workspace of the automatic split is lf_attn_lse_split_plan's."""
    import torch
    dev = _device()
    qp, kp, vp, lp, cp = _attn_args(shape, dev, q, k, v, block_list, block_count, list_cap)
    ws = _sized_ptr(workspace, torch.uint8, workspace.shape, dev, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() if workspace is not None else 0
    _check(_lib.lf_block_sparse_attn_lse(
        ctypes.byref(shape), qp, kp, vp, lp, cp, list_cap, float(softmax_scale),
        _sized_ptr(out, torch.bfloat16, q.shape, dev, "out"),
        None if out_lo is None else _sized_ptr(out_lo, torch.bfloat16, q.shape, dev, "out_lo"),
        _sized_ptr(lse, torch.float32, q.shape[:3], dev, "lse"), int(tail_pieces), ws, ws_bytes,
        _raw_stream(stream, dev)), "lf_block_sparse_attn_lse")


def lf_attn_bwd_workspace(shape: LfShape) -> int:
    """Bytes of the workspace of lf_block_sparse_attn_bwd."""
    n = _lib.lf_attn_bwd_workspace(ctypes.byref(shape))
    if n < 0:
        raise LfError(3, "lf_attn_bwd_workspace")
    return n


def lf_block_sparse_attn_bwd(shape: LfShape, q, k, v, out, dout, lse, block_list, block_count, list_cap: int,
                             softmax_scale: float, dq, dk, dv, workspace, stream=None, out_lo=None) -> None:
    """Gradient of the attention in q, k and v over the same lists (out, out_lo and lse from
    lf_block_sparse_attn_lse; out_lo may be left out at some loss of accuracy); ``workspace``: a uint8 device tensor of lf_attn_bwd_workspace(shape) bytes."""
    import torch
    bf, dev = torch.bfloat16, _device()
    qp, kp, vp, lp, cp = _attn_args(shape, dev, q, k, v, block_list, block_count, list_cap)
    _check(_lib.lf_block_sparse_attn_bwd(
        ctypes.byref(shape), qp, kp, vp, _sized_ptr(out, bf, q.shape, dev, "out"),
        None if out_lo is None else _sized_ptr(out_lo, bf, q.shape, dev, "out_lo"),
        _sized_ptr(dout, bf, q.shape, dev, "dout"), _sized_ptr(lse, torch.float32, q.shape[:3], dev, "lse"), lp, cp,
        list_cap, float(softmax_scale), _sized_ptr(dq, bf, q.shape, dev, "dq"),
        _sized_ptr(dk, bf, k.shape, dev, "dk"), _sized_ptr(dv, bf, k.shape, dev, "dv"),
        _sized_ptr(workspace, torch.uint8, workspace.shape, dev, "workspace"), workspace.numel(), _raw_stream(stream, dev)),
        "lf_block_sparse_attn_bwd")


def lf_rope(plan: RopePlan, xs: Sequence, outs: Sequence, positions, rotate: Optional[Sequence[bool]] = None,
            backward: bool = False, stream=None) -> None:
    """Rotary positions of up to three tensors in one launch.

    ``xs`` and ``outs``: [batch, heads, tokens, head_dim] views of any strides (the last one 1) and
    one dtype (fp32, bf16, fp16), e.g. slices of a fused token-major projection and slots of the
    call's head-major tensors; an output may be its own input. ``positions``: int32
    [tokens, n_axes] or [batch, tokens, n_axes]. ``rotate[i]`` False copies tensor i. ``backward``:
    xs are gradients of the outputs, outs receive the gradients of the inputs."""
    n = len(xs)
    if len(outs) != n or not 1 <= n <= 3:
        raise ValueError("lf_rope takes one to three tensors and as many outputs")
    dev, first = _device(), xs[0]
    dtype = first.dtype
    if first.dim() != 4:
        raise ValueError("tensors must be [batch, heads, tokens, head_dim]")
    B, _, T, D = first.shape
    if D != plan.head_dim:
        raise ValueError(f"tensors have head_dim {D}, the plan {plan.head_dim}")
    io = b""
    for i in range(n):
        x, o = xs[i], outs[i]
        if x.dtype is not dtype or o.dtype is not dtype or x.get_device() != dev or o.get_device() != dev:
            _refuse_rope(x, o, dtype, dev)
        shape = x.shape
        if len(shape) != 4 or shape[0] != B or shape[2] != T or shape[3] != D or o.shape != shape:
            raise ValueError("every tensor and its output must be [batch, heads, tokens, head_dim] of the same sizes")
        xb, xh, xt, xe = x.stride()
        ob, oh, ot, oe = o.stride()
        if xe != 1 or oe != 1:
            raise ValueError("the last dimension must have stride 1")
        io += _ROPE_IO(x.data_ptr(), o.data_ptr(), xb, xh, xt, ob, oh, ot, shape[1], 1 if rotate is None or rotate[i] else 0)
    import torch
    shared = positions.dim() == 2
    pos = _sized_ptr(positions, torch.int32, (T, plan.n_axes) if shared else (B, T, plan.n_axes), dev, "positions")
    _check(_lib.lf_rope(ctypes.byref(plan), B, T, _dtype_code(dtype), pos, 0 if shared else T * plan.n_axes, io, n,
                        1 if backward else 0, _raw_stream(stream, dev)), "lf_rope")


_ROPE_IO = struct.Struct("@PP6qii").pack  # an lf_rope_io


def _refuse_rope(x, o, dtype, dev) -> None:
    for t, name in ((x, "x"), (o, "out")):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
        if t.device.index != dev:
            raise ValueError(f"{name} must be on the current device (cuda:{dev}), got {t.device}")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


_NORM_PACK = struct.Struct("@7P").pack  # an lf_norm_gate_vectors


def _norm_vectors(shape: NormGateShape, dev: int, gate=None, scale=None, shift=None, pre_w=None, pre_b=None, post_w=None,
                  post_b=None) -> bytes:
    import torch
    f32, group, row = torch.float32, (shape.groups, shape.dim), (shape.dim,)
    return _NORM_PACK(
        0 if gate is None else _sized_ptr(gate, f32, group, dev, "gate"),
        0 if scale is None else _sized_ptr(scale, f32, group, dev, "scale"),
        0 if shift is None else _sized_ptr(shift, f32, group, dev, "shift"),
        0 if pre_w is None else _sized_ptr(pre_w, f32, row, dev, "pre_w"),
        0 if pre_b is None else _sized_ptr(pre_b, f32, row, dev, "pre_b"),
        0 if post_w is None else _sized_ptr(post_w, f32, row, dev, "post_w"),
        0 if post_b is None else _sized_ptr(post_b, f32, row, dev, "post_b"))


def _norm_dtypes(shape: NormGateShape):
    import torch
    types = (torch.float32, torch.bfloat16, torch.float16)
    return types[shape.x_dtype], types[shape.y_dtype]


def lf_norm_gate(shape: NormGateShape, x, y, r, h, gate=None, scale=None, shift=None, pre_w=None, pre_b=None,
                 post_w=None, post_b=None, stream=None) -> None:
    """r = residual_scale x + gate post(y); h = pre(r) (1 + scale) + shift, in one pass over [rows, dim]
    (``y``, ``r`` or ``h`` may be None). gate, scale, shift: fp32 [groups, dim]; weights and biases fp32 [dim]."""
    dev = _device()
    xd, yd = _norm_dtypes(shape)
    want = (shape.rows, shape.dim)

    def opt(t, dtype, name):
        return None if t is None else _sized_ptr(t, dtype, want, dev, name)

    v = _norm_vectors(shape, dev, gate, scale, shift, pre_w, pre_b, post_w, post_b)
    _check(_lib.lf_norm_gate(ctypes.byref(shape), v, _sized_ptr(x, xd, want, dev, "x"), opt(y, yd, "y"),
                             opt(r, xd, "r"), opt(h, yd, "h"), _raw_stream(stream, dev)), "lf_norm_gate")


def lf_norm_gate_bwd_workspace(shape: NormGateShape) -> int:
    """Bytes of the workspace of lf_norm_gate_bwd."""
    n = _lib.lf_norm_gate_bwd_workspace(ctypes.byref(shape))
    if n < 0:
        raise LfError(3, "lf_norm_gate_bwd_workspace")
    return n


def lf_norm_gate_bwd(shape: NormGateShape, x, y, dr, dh, dx, dy, grads: dict, workspace, gate=None, scale=None,
                     shift=None, pre_w=None, pre_b=None, post_w=None, post_b=None, stream=None) -> None:
    """Gradients of lf_norm_gate from its own inputs. ``dr`` / ``dh``: gradients of r and h (None: none);
    ``dx`` / ``dy``: outputs (None: not wanted); ``grads``: fp32 outputs by vector name (gate, scale, shift,
    pre_w, ...), shaped as the vectors; ``workspace``: a uint8 device tensor of
    lf_norm_gate_bwd_workspace(shape) bytes."""
    import torch
    dev = _device()
    xd, yd = _norm_dtypes(shape)
    want = (shape.rows, shape.dim)

    def opt(t, dtype, name):
        return None if t is None else _sized_ptr(t, dtype, want, dev, name)

    for name in grads:
        if name not in _NORM_VECTORS:
            raise ValueError(f"unknown gradient {name}")
    v = _norm_vectors(shape, dev, gate, scale, shift, pre_w, pre_b, post_w, post_b)
    g = _norm_vectors(shape, dev, **grads)
    _check(_lib.lf_norm_gate_bwd(
        ctypes.byref(shape), v, _sized_ptr(x, xd, want, dev, "x"), opt(y, yd, "y"), opt(dr, xd, "dr"),
        opt(dh, yd, "dh"), opt(dx, xd, "dx"), opt(dy, yd, "dy"), g,
        _sized_ptr(workspace, torch.uint8, workspace.shape, dev, "workspace"), workspace.numel(), _raw_stream(stream, dev)),
        "lf_norm_gate_bwd")


def lf_attn_split_plan(shape: LfShape, list_cap: int, sm: int = 0) -> Tuple[int, int, int]:
    """(tail query blocks, pieces per list, workspace bytes) of the automatic split."""
    return _split_plan("lf_attn_split_plan", shape, list_cap, sm)


def lf_attn_lse_split_plan(shape: LfShape, list_cap: int, sm: int = 0) -> Tuple[int, int, int]:
    """lf_attn_split_plan for lf_block_sparse_attn_lse with out_lo, whose piece slots are larger."""
    return _split_plan("lf_attn_lse_split_plan", shape, list_cap, sm)


def _split_plan(name: str, shape: LfShape, list_cap: int, sm: int) -> Tuple[int, int, int]:
    t, p, b = ctypes.c_int32(0), ctypes.c_int32(0), ctypes.c_int64(0)
    _check(getattr(_lib, name)(ctypes.byref(shape), list_cap, sm, ctypes.byref(t), ctypes.byref(p),
                               ctypes.byref(b)), name)
    return t.value, p.value, b.value


def lf_cag_budget(T: Sequence[float], flops_w: Optional[Sequence[float]], s_base: float,
                  s_target: float, target_over_all: bool = True) -> Tuple[int, list, float]:
    """Host-only Chunk-Aware Growth solver: returns (status, s[n], beta)."""
    n = len(T)
    Ta = (ctypes.c_double * n)(*[float(x) for x in T])
    wa = (ctypes.c_double * n)(*[float(x) for x in flops_w]) if flops_w is not None else None
    s_out = (ctypes.c_double * max(n, 1))()
    beta = ctypes.c_double(0.0)
    st = _lib.lf_cag_budget(n, ctypes.cast(Ta, ctypes.c_void_p),
                            ctypes.cast(wa, ctypes.c_void_p) if wa is not None else None,
                            float(s_base), float(s_target), 1 if target_over_all else 0,
                            ctypes.cast(s_out, ctypes.c_void_p), ctypes.byref(beta))
    return st, list(s_out)[:n], beta.value


def lf_get_device_error() -> Tuple[int, int]:
    """(status, detail) of the current device's error word; clears it."""
    d = ctypes.c_int32(0)
    st = _lib.lf_get_device_error(ctypes.byref(d))
    return st, d.value


@dataclass
class HSABuffers:
    q_pool: "object"
    k_pool: "object"
    k_frame: "object"
    frame_sel: "object"
    block_list: "object"
    block_count: "object"
    out: "object"
    list_cap: int


class HSACall:
    """One HSA call's device buffers plus the device steps, in order: pooling, the
    two-level selection (one launch, lf_select_mask) and the attention.

    ``shape``: an ``LfShape``; ``chunk_index`` is 1-based (chunk 1 is dense);
    ``topk_frames`` / ``topk_blocks`` as in the C ABI. ``tail_pieces`` selects
    the attention's split of the last, partial wave (0: automatic plan for the
    current device, 1: none, k >= 2: k pieces); the workspace it needs is
    allocated here. ``train=True`` keeps each row's log-sum-exp, so that
    ``backward`` can give the gradients of the last call: until then its
    q, k, v and the output it returned stay as they are, so layers whose
    gradients are still to come have an HSACall each. ``load`` and
    ``load_bwd`` bring a chunk's fused projection into the call's tensors with
    rotary positions applied, and the gradients back.
    """

    def __init__(self, shape: LfShape, chunk_index: int, topk_frames: int, topk_blocks: int,
                 device="cuda", softmax_scale: float = 0.0, tail_pieces: int = 0, train: bool = False):
        import torch
        self.shape, self.chunk_index = shape, chunk_index
        self.topk_frames, self.topk_blocks = topk_frames, topk_blocks
        self.softmax_scale = softmax_scale
        s = shape
        D = s.head_dim
        n_sel = lf_frames_selected(s, chunk_index, topk_frames)
        cap = lf_list_capacity(s, chunk_index, topk_frames, topk_blocks)
        if n_sel < 0 or cap < 0:
            raise LfError(3, "HSACall")
        self.n_sel = n_sel
        f32, i32 = torch.float32, torch.int32
        self.buf = HSABuffers(
            q_pool=torch.empty(s.batch, s.heads, s.Rq, D, dtype=f32, device=device),
            k_pool=torch.empty(s.batch, s.heads, s.Nkv, D, dtype=f32, device=device),
            k_frame=torch.empty(s.batch, s.heads, s.n_frames, D, dtype=f32, device=device),
            frame_sel=torch.empty(s.batch, s.heads, s.Rq, n_sel, dtype=i32, device=device),
            block_list=torch.empty(s.batch, s.heads, s.Rq, cap, dtype=i32, device=device),
            block_count=torch.empty(s.batch, s.heads, s.Rq, dtype=i32, device=device),
            out=torch.empty(s.batch, s.heads, s.Lq, D, dtype=torch.bfloat16, device=device),
            list_cap=cap,
        )
        self.tail_pieces = tail_pieces
        if tail_pieces == 0:
            tail, pieces, _ = lf_attn_split_plan(s, cap)
        elif tail_pieces >= 2:
            # the same tail as the automatic plan, with the piece count given
            sm = torch.cuda.get_device_properties(torch.device(device)).multi_processor_count
            tail = (s.batch * s.heads * s.Rq) % sm
            pieces = min(tail_pieces, cap)
            if pieces < 2:
                tail, pieces = 0, 0
        else:
            tail, pieces = 0, 0
        ws_bytes = tail * pieces * 64 * (D + (3 if train else 2)) * 4  # a piece slot; training keeps one sum more
        self.workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=device) if ws_bytes else None
        self.split = (tail, pieces) if ws_bytes else (0, 0)
        self.lse = torch.empty(s.batch, s.heads, s.Lq, dtype=f32, device=device) if train else None
        self.out_lo = torch.empty_like(self.buf.out) if train else None
        self.bwd_workspace = torch.empty(lf_attn_bwd_workspace(s), dtype=torch.uint8, device=device) if train else None
        self.attended = False  # out, lse and out_lo are those of the lists that the buffers hold
        # kernels enqueued per call: pool, selection (both levels), attention (+ the merge of a split)
        self.launches_per_call = 3 + (1 if ws_bytes else 0)

    def pool(self, q, k, stream=None):
        b = self.buf
        lf_pool(self.shape, q, k, b.q_pool, b.k_pool, b.k_frame, stream)

    def select(self, stream=None):
        b = self.buf
        self.attended = False
        lf_select_mask(self.shape, self.chunk_index, self.topk_frames, self.topk_blocks, b.q_pool, b.k_frame,
                       b.k_pool, b.frame_sel, b.block_list, b.block_count, b.list_cap, stream)

    def load(self, plan: RopePlan, qkv, positions, q, k, v, stream=None):
        """The chunk's projection ``qkv`` [batch, Lq, 3, heads, head_dim] (bf16) into ``q`` and the
        current-chunk frames of ``k`` and ``v``, q and k rotated (one launch, lf_rope)."""
        xs, (kc, vc) = qkv.permute(2, 0, 3, 1, 4).unbind(0), self._current(k, v)
        lf_rope(plan, xs, (q, kc, vc), positions, rotate=(True, True, False), stream=stream)

    def load_bwd(self, plan: RopePlan, dq, dk, dv, positions, dqkv, stream=None):
        """Gradient of ``load``: ``dqkv`` from ``dq`` and the current-chunk frames of ``dk`` and ``dv``."""
        outs, (kc, vc) = dqkv.permute(2, 0, 3, 1, 4).unbind(0), self._current(dk, dv)
        lf_rope(plan, (dq, kc, vc), outs, positions, rotate=(True, True, False), backward=True, stream=stream)

    def _current(self, *ts):
        s = self.shape
        return [t[:, :, s.Lkv - s.Lq:s.Lkv] for t in ts]

    def backward(self, q, k, v, dout, dq, dk, dv, stream=None):
        """Gradients of the last call's output in q, k and v (``train=True``; the selected blocks are constants).
        Refused where the last attention failed or lists were selected since."""
        if self.lse is None or not self.attended:
            raise ValueError("HSACall.backward needs train=True and a call before it, with no selection in between")
        b = self.buf
        lf_block_sparse_attn_bwd(self.shape, q, k, v, b.out, dout, self.lse, b.block_list, b.block_count, b.list_cap,
                                 self.softmax_scale, dq, dk, dv, self.bwd_workspace, stream, out_lo=self.out_lo)

    def attend(self, q, k, v, stream=None):
        b = self.buf
        self.attended = False
        if self.lse is not None:
            lf_block_sparse_attn_lse(self.shape, q, k, v, b.block_list, b.block_count, b.list_cap,
                                     self.softmax_scale, b.out, self.lse, self.workspace, self.tail_pieces, stream,
                                     out_lo=self.out_lo)
            self.attended = True
            return
        lf_block_sparse_attn_ws(self.shape, q, k, v, b.block_list, b.block_count, b.list_cap,
                                self.softmax_scale, b.out, self.workspace, self.tail_pieces, stream)

    def __call__(self, q, k, v, stream=None):
        self.pool(q, k, stream)
        self.select(stream)
        self.attend(q, k, v, stream)
        return self.buf.out


def shard_units(batch: int, heads: int, world: int, rank: int) -> Tuple[int, int]:
    """Contiguous range [u0, u1) of the call's batch*heads (batch, head) units that
    process ``rank`` of ``world`` takes. Pooling, selection and attention of one unit
    never read another unit's data, so the ranges need no exchange; their sizes
    differ by at most one unit, and a rank past the unit count gets an empty range."""
    if world < 1 or not 0 <= rank < world:
        raise ValueError("rank outside the world")
    n = batch * heads
    return rank * n // world, (rank + 1) * n // world


def shard_shape(shape: LfShape, world: int, rank: int) -> Tuple[Optional[LfShape], int, int]:
    """(per-rank shape, u0, u1): the units [u0, u1) of ``shape`` as a call of their
    own (batch 1, u1 - u0 heads, same frames and head stride); None when the range
    is empty. The [B, H, L, D] tensors are contiguous over (batch, head), so the
    slice is a pointer offset (``unit_view``)."""
    u0, u1 = shard_units(shape.batch, shape.heads, world, rank)
    if u1 == u0:
        return None, u0, u1
    s = LfShape.make(1, u1 - u0, shape.head_dim, shape.frame_tokens, shape.n_frames, shape.n_sink,
                     shape.n_recent, shape.n_cur, block_tokens=shape.block_tokens, kv_stride=shape.kv_stride)
    return s, u0, u1


def unit_view(t, u0: int, u1: int):
    """Units [u0, u1) of a contiguous [B, H, L, D] tensor as a [1, u1 - u0, L, D] view."""
    if not t.is_contiguous():
        raise ValueError("unit_view needs a contiguous tensor")
    return t.reshape(-1, t.shape[-2], t.shape[-1])[u0:u1].unsqueeze(0)


def shape_from_workload(w) -> LfShape:
    """LfShape of an ``lf_synth.Workload`` (or anything with the same fields)."""
    return LfShape.make(w.batch, w.heads, w.head_dim, w.frame_tokens, w.n_frames, w.n_sink,
                        w.n_recent, w.n_cur, block_tokens=w.block_tokens)
