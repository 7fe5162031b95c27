"""Python binding of the block-sparse spatio-temporal attention library.

Argument marshalling only: every step runs in the CUDA library ``libbss.so``
(C ABI in ``include/bss.h`` and ``include/bss_block.h``).  PyTorch supplies device memory and the current
stream.  There is no CPU or PyTorch fallback: if the library is missing or was
not built for this GPU, every call raises.

Method: blog "Accelerating Spatio-Temporal Attention for Video Diffusion on
TPUs" (Google Developers) -- per-head spatial / temporal block-sparse
attention with full / boundary / skipped tiles, optional tile-aligned rounding,
and the (F,H,W) <-> (H,W,F) token permutation for temporal heads.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libbss.so")

KIND_SPATIAL, KIND_TEMPORAL = 0, 1
CLASS_FULL, CLASS_BOUNDARY, CLASS_PAD, CLASS_COLUMNS = 0, 1, 2, 3
ATTN_BQ, ATTN_BKV = 256, 128   # default tile shape of bss_sparse_attention's map
ATTN_BQ_SUPPORTED = (128, 256)  # query rows per tile it runs (one or two 128-row MMA halves)
ATTN_BKV_SUPPORTED = (64, 128)  # keys per tile it runs (routing, dense control and fused permutation: 128)
CLASS_SHIFT = 30
TILE_INDEX_MASK = (1 << 30) - 1
DTYPE_BF16, DTYPE_F32 = 0, 1
NORM_NONE, NORM_LAYER, NORM_RMS = 0, 1, 2                      # residual_norm
HEAD_NORM_NONE, HEAD_NORM_HEAD, HEAD_NORM_TOKEN = 0, 1, 2      # heads_from_tokens: Q/K norm over a head or a token
ACT_NONE, ACT_GELU_TANH, ACT_GELU, ACT_SILU = 0, 1, 2, 3       # linear
PAIR_INTERLEAVED, PAIR_HALVES = 0, 1                           # rotary pairs: channels (2p, 2p + 1) or (p, p + R/2)
STAT_NAMES = ("full", "boundary", "pad", "skip", "retained_pairs", "exact_retained_pairs", "columns")
STATUS_NAMES = {0: "BSS_OK", 1: "BSS_ERR_INVALID_ARG", 2: "BSS_ERR_UNSUPPORTED", 3: "BSS_ERR_CUDA",
                4: "BSS_ERR_TIMEOUT", 5: "BSS_ERR_OOM"}

_lib = None


class BssError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class _MaskParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("F", "Hs", "Ws", "head_dim", "spatial_frame_window",
                                               "temporal_raster_window", "sink_frames", "temporal_permuted",
                                               "rounding")]


@dataclass(frozen=True)
class MaskParams:
    """Video geometry and mask windows (see ``bss_mask_params`` in include/bss.h)."""
    F: int
    Hs: int
    Ws: int
    head_dim: int
    spatial_frame_window: int
    temporal_raster_window: int
    sink_frames: int = 1
    temporal_permuted: int = 1
    rounding: int = 0

    @property
    def S(self) -> int:
        return self.Hs * self.Ws

    @property
    def N(self) -> int:
        return self.F * self.S

    def c(self) -> _MaskParams:
        """The C form (made once: the fields do not change, the library only reads it)."""
        c = self.__dict__.get("_c")
        if c is None:
            c = self._make_c()
            object.__setattr__(self, "_c", c)
        return c

    def _make_c(self) -> _MaskParams:
        return _MaskParams(self.F, self.Hs, self.Ws, self.head_dim, self.spatial_frame_window,
                           self.temporal_raster_window, self.sink_frames, self.temporal_permuted, self.rounding)


class _Rotary(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p * 3), ("length", ctypes.c_int32 * 3), ("pairs", ctypes.c_int32 * 3),
                ("offset", ctypes.c_int32 * 3), ("pairing", ctypes.c_int32)]


class _TokenTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class _HeadsOptions(ctypes.Structure):
    _fields_ = [("norm", ctypes.c_int32), ("eps", ctypes.c_float), ("weight_dtype", ctypes.c_int32),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("rotary", ctypes.POINTER(_Rotary))]


# _Rotary's bytes: building them at once is quicker than its arrays element by element
_ROTARY_BYTES = struct.Struct("=3Q10i")


class _ResidualNormArgs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("rows", "rows_per_group")]
                + [(n, ctypes.c_int32) for n in ("channels", "stream_dtype", "branch_dtype", "param_dtype", "norm",
                                                 "y_norm")]
                + [(n, ctypes.c_float) for n in ("eps", "residual_scale")]
                + [(n, ctypes.c_void_p) for n in ("x", "y", "r", "h")]
                + [(n, ctypes.c_int64) for n in ("x_stride", "y_stride", "r_stride", "h_stride")]
                + [(n, ctypes.c_void_p) for n in ("gate", "scale", "shift")]
                + [(n, ctypes.c_int64) for n in ("gate_stride", "scale_stride", "shift_stride")]
                + [(n, ctypes.c_void_p) for n in ("weight", "bias", "y_weight", "stats", "y_stats")])


class _ResidualNormGrads(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("rows", "rows_per_group")]
                + [(n, ctypes.c_int32) for n in ("channels", "stream_dtype", "branch_dtype", "param_dtype", "norm",
                                                 "y_norm")]
                + [("residual_scale", ctypes.c_float)]
                + [(n, ctypes.c_void_p) for n in ("r", "y", "dr", "dh", "dx", "dy")]
                + [(n, ctypes.c_int64) for n in ("r_stride", "y_stride", "dr_stride", "dh_stride", "dx_stride",
                                                 "dy_stride")]
                + [(n, ctypes.c_void_p) for n in ("stats", "y_stats", "gate", "scale")]
                + [(n, ctypes.c_int64) for n in ("gate_stride", "scale_stride")]
                + [(n, ctypes.c_void_p) for n in ("weight", "bias", "y_weight", "dgate", "dscale", "dshift", "dweight",
                                                  "dbias", "dy_weight", "workspace")]
                + [("workspace_bytes", ctypes.c_int64)])


class _LinearArgs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("rows", "rows_per_group")]
                + [(n, ctypes.c_int32) for n in ("in_channels", "out_channels", "out_dtype", "param_dtype", "activation")]
                + [("residual_scale", ctypes.c_float)]
                + [(n, ctypes.c_void_p) for n in ("x", "weight", "bias", "gate", "residual", "out", "pre")]
                + [(n, ctypes.c_int64) for n in ("x_stride", "weight_stride", "gate_stride", "residual_stride",
                                                 "out_stride", "pre_stride")]
                + [("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64)])


class _LinearGrads(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("rows", "rows_per_group")]
                + [(n, ctypes.c_int32) for n in ("in_channels", "out_channels", "dout_dtype", "param_dtype",
                                                 "dweight_dtype", "activation")]
                + [(n, ctypes.c_void_p) for n in ("dout", "x", "weight", "pre", "gate", "dx", "dweight", "dbias", "dgate")]
                + [(n, ctypes.c_int64) for n in ("dout_stride", "x_stride", "weight_stride", "pre_stride", "gate_stride",
                                                 "dx_stride", "dweight_stride")]
                + [("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64)])


class _StateTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("group_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class _CrossArgs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("rows", "rows_per_group")]
                + [(n, ctypes.c_int32) for n in ("heads", "kv_heads", "head_dim", "keys")]
                + [("softmax_scale", ctypes.c_float)] + [(n, _TokenTensor) for n in ("q", "O")]
                + [(n, _StateTensor) for n in ("k", "v")] + [(n, ctypes.c_void_p) for n in ("lengths", "lse")])


class _CrossGrads(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("rows", "rows_per_group")]
                + [(n, ctypes.c_int32) for n in ("heads", "kv_heads", "head_dim", "keys")]
                + [("softmax_scale", ctypes.c_float)] + [(n, _TokenTensor) for n in ("dO", "q", "O", "dq")]
                + [(n, _StateTensor) for n in ("k", "v", "dk", "dv")]
                + [(n, ctypes.c_void_p) for n in ("lengths", "lse", "workspace")] + [("workspace_bytes", ctypes.c_int64)])


EXPORTED = ("bss_build_tile_map", "bss_tile_map_stats", "bss_tile_map_dims", "bss_tile_map_copy_csr",
            "bss_destroy_tile_map", "bss_permute", "bss_sparse_attention", "bss_dense_attention",
            "bss_get_device_status", "bss_status_string", "bss_last_error_message", "bss_version",
            "bss_diag_mma_tile", "bss_build_tile_map_csr_noalloc", "bss_route_heads",
            "bss_sparse_attention_fused", "bss_permute_flagged", "bss_sparse_attention_split",
            "bss_diag_wait_timeout", "bss_attention_step", "bss_step_workspace_create",
            "bss_step_workspace_destroy", "bss_step_workspace_wait_stream", "bss_attention_step_host",
            "bss_permute_flagged_multi", "bss_rotary_table", "bss_heads_from_tokens",
            "bss_heads_from_tokens_backward_workspace", "bss_heads_from_tokens_backward",
            "bss_attention_step_tokens", "bss_residual_norm", "bss_residual_norm_backward_workspace",
            "bss_residual_norm_backward", "bss_linear_workspace", "bss_linear", "bss_linear_backward_workspace",
            "bss_linear_backward", "bss_cross_attention",
            "bss_cross_attention_backward_workspace", "bss_cross_attention_backward")


def load(path: str | None = None):
    """Load libbss.so (raises if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m block_sparse_spatio_gb300.build`")
    lib = ctypes.CDLL(path)
    p, i32, st = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int
    MP = ctypes.POINTER(_MaskParams)
    lib.bss_build_tile_map.argtypes = [MP, i32, i32, ctypes.POINTER(p), p]
    lib.bss_build_tile_map.restype = st
    lib.bss_tile_map_stats.argtypes = [p, i32, ctypes.POINTER(ctypes.c_int64)]
    lib.bss_tile_map_stats.restype = st
    lib.bss_tile_map_dims.argtypes = [p, i32, ctypes.POINTER(ctypes.c_int32)]
    lib.bss_tile_map_dims.restype = st
    lib.bss_tile_map_copy_csr.argtypes = [p, i32, p, p]
    lib.bss_tile_map_copy_csr.restype = st
    lib.bss_destroy_tile_map.argtypes = [p]
    lib.bss_destroy_tile_map.restype = None
    lib.bss_permute.argtypes = [p, p, p, i32, MP, i32, p]
    lib.bss_permute.restype = st
    lib.bss_sparse_attention.argtypes = [p, p, p, p, p, p, p, i32, ctypes.c_float, p]
    lib.bss_sparse_attention.restype = st
    lib.bss_sparse_attention_fused.argtypes = [p, p, p, p, p, p, p, i32, ctypes.c_float, p]
    lib.bss_sparse_attention_fused.restype = st
    lib.bss_sparse_attention_split.argtypes = [p, p, p, p, p, p, p, p, p, p, p, i32, ctypes.c_float, p]
    lib.bss_sparse_attention_split.restype = st
    lib.bss_permute_flagged.argtypes = [p, p, p, i32, MP, i32, p]
    lib.bss_permute_flagged.restype = st
    lib.bss_diag_wait_timeout.argtypes = [ctypes.c_int64, p, p]
    lib.bss_diag_wait_timeout.restype = st
    lib.bss_dense_attention.argtypes = [p, p, p, p, p, i32, i32, i32, ctypes.c_float, p]
    lib.bss_dense_attention.restype = st
    lib.bss_get_device_status.argtypes = [p]
    lib.bss_get_device_status.restype = st
    lib.bss_status_string.argtypes = [st]
    lib.bss_status_string.restype = ctypes.c_char_p
    lib.bss_last_error_message.argtypes = []
    lib.bss_last_error_message.restype = ctypes.c_char_p
    lib.bss_version.argtypes = []
    lib.bss_version.restype = i32
    lib.bss_diag_mma_tile.argtypes = [p, p, p, p, p, p, i32, p]
    lib.bss_diag_mma_tile.restype = st
    lib.bss_build_tile_map_csr_noalloc.argtypes = [MP, i32, i32, i32, p, p, ctypes.c_int64, p, p]
    lib.bss_build_tile_map_csr_noalloc.restype = st
    lib.bss_route_heads.argtypes = [p, p, p, i32, MP, p, i32, p, p, p]
    lib.bss_route_heads.restype = st
    lib.bss_permute_flagged_multi.argtypes = [ctypes.POINTER(p), ctypes.POINTER(p), i32, p, i32, MP, i32, p]
    lib.bss_permute_flagged_multi.restype = st
    lib.bss_attention_step.argtypes = [p, p, p, p, p, p, p, i32, p, p, p, p]
    lib.bss_attention_step.restype = st
    lib.bss_step_workspace_create.argtypes = [MP, i32, i32, i32, ctypes.POINTER(p)]
    lib.bss_step_workspace_create.restype = st
    lib.bss_step_workspace_destroy.argtypes = [p]
    lib.bss_step_workspace_destroy.restype = None
    lib.bss_step_workspace_wait_stream.argtypes = [p, p]
    lib.bss_step_workspace_wait_stream.restype = st
    lib.bss_attention_step_host.argtypes = [p, p, p, p, p, p, p, p, p]
    lib.bss_attention_step_host.restype = st
    TT, HO, i64p = ctypes.POINTER(_TokenTensor), ctypes.POINTER(_HeadsOptions), ctypes.POINTER(ctypes.c_int64)
    lib.bss_rotary_table.argtypes = [p, i32, i32, i32, ctypes.c_double, p, p]
    lib.bss_rotary_table.restype = st
    lib.bss_heads_from_tokens.argtypes = [TT, TT, TT, p, p, p, p, i32, MP, HO, p]
    lib.bss_heads_from_tokens.restype = st
    lib.bss_heads_from_tokens_backward_workspace.argtypes = [i32, MP, i32, i64p]
    lib.bss_heads_from_tokens_backward_workspace.restype = st
    lib.bss_heads_from_tokens_backward.argtypes = [p, p, p, TT, TT, TT, TT, TT, p, p, p, i32, MP, HO, p,
                                                   ctypes.c_int64, p]
    lib.bss_heads_from_tokens_backward.restype = st
    lib.bss_attention_step_tokens.argtypes = [TT, TT, TT, p, p, p, p, i32, HO, p, p, p, p]
    lib.bss_attention_step_tokens.restype = st
    lib.bss_residual_norm.argtypes = [ctypes.POINTER(_ResidualNormArgs), p]
    lib.bss_residual_norm.restype = st
    lib.bss_residual_norm_backward_workspace.argtypes = [ctypes.POINTER(_ResidualNormGrads), i64p]
    lib.bss_residual_norm_backward_workspace.restype = st
    lib.bss_residual_norm_backward.argtypes = [ctypes.POINTER(_ResidualNormGrads), p]
    lib.bss_residual_norm_backward.restype = st
    lib.bss_cross_attention.argtypes = [ctypes.POINTER(_CrossArgs), p]
    lib.bss_cross_attention.restype = st
    for name, args in (("linear", _LinearArgs), ("linear_backward", _LinearGrads),
                       ("cross_attention_backward", _CrossGrads)):
        getattr(lib, f"bss_{name}").argtypes = [ctypes.POINTER(args), p]
        getattr(lib, f"bss_{name}_workspace").argtypes = [ctypes.POINTER(args), i64p]
        getattr(lib, f"bss_{name}").restype = getattr(lib, f"bss_{name}_workspace").restype = st
    _lib = lib
    return lib


def _check(status: int):
    if status != 0:
        raise BssError(status, load().bss_last_error_message().decode())


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dev_tensor(t, name, dtype=None):
    import torch
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _check_shapes(tile_map, lse, *named):
    """Every tensor [H][N][d] of the map's geometry (same H), lse [H][N]: a
    map built for another geometry is refused before any launch."""
    p = tile_map.params
    N, d = p.F * p.Hs * p.Ws, p.head_dim
    H = named[0][0].shape[0]
    for t, n in named:
        if tuple(t.shape) != (H, N, d):
            raise ValueError(f"{n} has shape {tuple(t.shape)}, the tile map wants ({H}, {N}, {d})")
    if lse is not None and tuple(lse.shape) != (H, N):
        raise ValueError(f"lse has shape {tuple(lse.shape)}, the tile map wants ({H}, {N})")
    return H


class TileMap:
    """Owning wrapper of a ``bss_tile_map`` handle."""

    def __init__(self, handle: ctypes.c_void_p, params: MaskParams, BQ: int, BKV: int):
        self._h = handle
        self.params, self.BQ, self.BKV = params, BQ, BKV

    @property
    def handle(self):
        if self._h is None:
            raise ValueError("tile map destroyed")
        return self._h

    def stats(self, kind: int) -> dict:
        return tile_map_stats(self, kind)

    def dims(self, kind: int):
        return tile_map_dims(self, kind)

    def csr(self, kind: int):
        return tile_map_copy_csr(self, kind)

    def destroy(self):
        if self._h is not None and _lib is not None:
            _lib.bss_destroy_tile_map(self._h)
        self._h = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.destroy()


def build_tile_map(params: MaskParams, BQ: int = ATTN_BQ, BKV: int = ATTN_BKV, stream=None) -> TileMap:
    lib = load()
    h = ctypes.c_void_p()
    mp = params.c()
    _check(lib.bss_build_tile_map(ctypes.byref(mp), BQ, BKV, ctypes.byref(h), _stream(stream)))
    return TileMap(h, params, BQ, BKV)


def _raw_handle(m):
    return m.handle if isinstance(m, TileMap) else m


def tile_map_stats(m, kind: int) -> dict:
    out = (ctypes.c_int64 * len(STAT_NAMES))()
    _check(load().bss_tile_map_stats(_raw_handle(m), kind, out))
    return dict(zip(STAT_NAMES, [int(x) for x in out]))


def tile_map_dims(m, kind: int):
    out = (ctypes.c_int32 * 4)()
    _check(load().bss_tile_map_dims(_raw_handle(m), kind, out))
    return tuple(int(x) for x in out)  # nq, nkv, nnz, ncols


def tile_map_copy_csr(m, kind: int):
    nq, nkv, nnz, ncols = tile_map_dims(m, kind)
    row_ptr = np.zeros(nq + 1, dtype=np.int32)
    entries = np.zeros(max(nnz, 1), dtype=np.int32)
    _check(load().bss_tile_map_copy_csr(_raw_handle(m), kind, row_ptr.ctypes.data, entries.ctypes.data))
    return row_ptr, entries[:nnz]


def destroy_tile_map(m):
    if isinstance(m, TileMap):
        m.destroy()
    else:
        load().bss_destroy_tile_map(m)


def permute(x, out, head_is_temporal, params: MaskParams, inverse: bool = False, stream=None,
            only_flagged: bool = False):
    """out <- per-head (F,H,W) -> (H,W,F) permutation of x (inverse=True: back).
    Heads with flag 0 are copied, or left untouched with ``only_flagged``."""
    import torch
    _dev_tensor(x, "x", torch.bfloat16)
    _dev_tensor(out, "out", torch.bfloat16)
    _dev_tensor(head_is_temporal, "head_is_temporal", torch.uint8)
    fn = load().bss_permute_flagged if only_flagged else load().bss_permute
    _check(fn(_ptr(x), _ptr(out), _ptr(head_is_temporal), x.shape[0], ctypes.byref(params.c()), int(bool(inverse)),
              _stream(stream)))
    return out


def permute_flagged_multi(xs, outs, head_is_temporal, params: MaskParams, inverse: bool = False, stream=None):
    """outs[i] <- the flagged heads of xs[i] permuted, 1 to 3 tensors in one launch
    (heads with flag 0 are left untouched in outs)."""
    import torch
    if len(xs) != len(outs) or not 1 <= len(xs) <= 3:
        raise ValueError("1 to 3 (input, output) pairs")
    for i, (x, o) in enumerate(zip(xs, outs)):
        _dev_tensor(x, f"xs[{i}]", torch.bfloat16)
        _dev_tensor(o, f"outs[{i}]", torch.bfloat16)
        if x.shape != xs[0].shape or o.shape != xs[0].shape:
            raise ValueError("every tensor must have the same shape")
    _dev_tensor(head_is_temporal, "head_is_temporal", torch.uint8)
    n = len(xs)
    ins = (ctypes.c_void_p * n)(*[x.data_ptr() for x in xs])
    ous = (ctypes.c_void_p * n)(*[o.data_ptr() for o in outs])
    _check(load().bss_permute_flagged_multi(ins, ous, n, _ptr(head_is_temporal), xs[0].shape[0],
                                            ctypes.byref(params.c()), int(bool(inverse)), _stream(stream)))
    return outs


def sparse_attention(Q, K, V, O, tile_map: TileMap, head_is_temporal=None, lse=None, softmax_scale: float = 0.0,
                     stream=None):
    """O <- block-sparse attention of [H][N][d] bf16 Q, K, V (temporal heads pre-permuted)."""
    import torch
    for t, n in ((Q, "Q"), (K, "K"), (V, "V"), (O, "O")):
        _dev_tensor(t, n, torch.bfloat16)
    _dev_tensor(head_is_temporal, "head_is_temporal", torch.uint8)
    _dev_tensor(lse, "lse", torch.float32)
    _check_shapes(tile_map, lse, (Q, "Q"), (K, "K"), (V, "V"), (O, "O"))
    _check(load().bss_sparse_attention(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(lse), tile_map.handle,
                                       _ptr(head_is_temporal), Q.shape[0], float(softmax_scale), _stream(stream)))
    return O


def sparse_attention_split(Q, K, V, O, Qt, Kt, Vt, Ot, tile_map: TileMap, head_is_temporal, lse=None,
                           softmax_scale: float = 0.0, stream=None):
    """Block-sparse attention with spatial heads in Q, K, V -> O and temporal
    heads (flag 1) in the permuted buffers Qt, Kt, Vt -> Ot.  Ot=None writes the
    temporal heads' output rows straight to O in (F,H,W) order (no inverse
    permutation needed)."""
    import torch
    named = [(Q, "Q"), (K, "K"), (V, "V"), (O, "O"), (Qt, "Qt"), (Kt, "Kt"), (Vt, "Vt")]
    if Ot is not None:
        named.append((Ot, "Ot"))
    for t, n in named:
        _dev_tensor(t, n, torch.bfloat16)
    _dev_tensor(head_is_temporal, "head_is_temporal", torch.uint8)
    _dev_tensor(lse, "lse", torch.float32)
    _check_shapes(tile_map, lse, *named)
    _check(load().bss_sparse_attention_split(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(Qt), _ptr(Kt), _ptr(Vt),
                                             _ptr(Ot), _ptr(lse), tile_map.handle, _ptr(head_is_temporal),
                                             Q.shape[0], float(softmax_scale), _stream(stream)))
    return O


def sparse_attention_fused(Q, K, V, O, tile_map: TileMap, head_is_temporal=None, lse=None,
                           softmax_scale: float = 0.0, stream=None):
    """O <- block-sparse attention of [H][N][d] bf16 Q, K, V, all heads in (F,H,W)
    order: the temporal heads' permutation is applied inside the kernel."""
    import torch
    for t, n in ((Q, "Q"), (K, "K"), (V, "V"), (O, "O")):
        _dev_tensor(t, n, torch.bfloat16)
    _dev_tensor(head_is_temporal, "head_is_temporal", torch.uint8)
    _dev_tensor(lse, "lse", torch.float32)
    _check_shapes(tile_map, lse, (Q, "Q"), (K, "K"), (V, "V"), (O, "O"))
    _check(load().bss_sparse_attention_fused(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(lse), tile_map.handle,
                                             _ptr(head_is_temporal), Q.shape[0], float(softmax_scale),
                                             _stream(stream)))
    return O


def dense_attention(Q, K, V, O, lse=None, softmax_scale: float = 0.0, stream=None):
    """O <- dense attention of [H][N][d] bf16 Q, K, V (the control)."""
    import torch
    for t, n in ((Q, "Q"), (K, "K"), (V, "V"), (O, "O")):
        _dev_tensor(t, n, torch.bfloat16)
    _dev_tensor(lse, "lse", torch.float32)
    H, N, d = Q.shape
    _check(load().bss_dense_attention(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(lse), H, N, d, float(softmax_scale),
                                      _stream(stream)))
    return O


def get_device_status(stream=None) -> int:
    """Synchronize and return (and clear) the device status word; 0 = OK."""
    return int(load().bss_get_device_status(_stream(stream)))


def status_string(status: int) -> str:
    return load().bss_status_string(status).decode()


def diag_wait_timeout(limit_ns: int, waited_ns=None, stream=None):
    """Run a bounded wait that nothing completes (see include/bss_diag.h); the
    device status word then holds BSS_ERR_TIMEOUT."""
    import torch
    _dev_tensor(waited_ns, "waited_ns", torch.int64)
    _check(load().bss_diag_wait_timeout(int(limit_ns), _ptr(waited_ns), _stream(stream)))


def diag_mma_tile(A, B, P, V, S, O, stream=None):
    """One-tile tensor-core self-test: S = A B^T, O = P V (see include/bss_diag.h)."""
    _check(load().bss_diag_mma_tile(_ptr(A), _ptr(B), _ptr(P), _ptr(V), _ptr(S), _ptr(O), A.shape[1],
                                    _stream(stream)))
    return S, O


def noalloc_map_dims(params: MaskParams, kind: int, BQ: int = ATTN_BQ, BKV: int = ATTN_BKV):
    """(nq, nkv) of the map bss_build_tile_map_csr_noalloc writes for one kind."""
    N, S = params.N, params.S
    ncols = (-(-S // BKV) * BKV + N) if (kind == KIND_TEMPORAL and params.temporal_permuted) else N
    return -(-N // BQ), -(-ncols // BKV)


def build_tile_map_csr_noalloc(params: MaskParams, kind: int, row_ptr, entries, stats, BQ: int = ATTN_BQ,
                               BKV: int = ATTN_BKV, stream=None):
    """Allocation-free CSR build of one kind into caller-owned device buffers
    (int32 row_ptr[nq + 1], int32 entries[>= nq * nkv], int64 stats[len(STAT_NAMES)])."""
    import torch
    _dev_tensor(row_ptr, "row_ptr", torch.int32)
    _dev_tensor(entries, "entries", torch.int32)
    _dev_tensor(stats, "stats", torch.int64)
    _check(load().bss_build_tile_map_csr_noalloc(ctypes.byref(params.c()), kind, BQ, BKV, _ptr(row_ptr),
                                                  _ptr(entries), entries.numel(), _ptr(stats), _stream(stream)))
    return row_ptr, entries, stats


def route_heads(Q, K, V, params: MaskParams, rows, head_is_temporal, errors, stream=None):
    """Per-head routing from sampled query rows (int32 device tensor of (F,H,W)
    token indices): writes head_is_temporal (uint8[H]) and errors (float32[H][2]:
    spatial and temporal deviation from the dense output)."""
    import torch
    for t, n in ((Q, "Q"), (K, "K"), (V, "V")):
        _dev_tensor(t, n, torch.bfloat16)
    _dev_tensor(rows, "rows", torch.int32)
    _dev_tensor(head_is_temporal, "head_is_temporal", torch.uint8)
    _dev_tensor(errors, "errors", torch.float32)
    _check(load().bss_route_heads(_ptr(Q), _ptr(K), _ptr(V), Q.shape[0], ctypes.byref(params.c()), _ptr(rows),
                                  rows.numel(), _ptr(head_is_temporal), _ptr(errors), _stream(stream)))
    return head_is_temporal, errors


def attention_step(Q, K, V, O, tile_map: TileMap, head_is_temporal, Qp, Kp, Vp, lse=None, stream=None):
    """The per-layer path of the blog's Figure 8 on one GPU (``bss_attention_step``):
    permute the temporal heads' Q, K, V to (H,W,F) into the workspaces Qp, Kp,
    Vp, run block-sparse attention, and store their O rows back in (F,H,W)
    order.  Q, K, V, O are in (F,H,W) order; Qp, Kp, Vp may be None when no
    head is permuted (no flags, or a map with temporal_permuted = 0).  lse, if
    given, is in each head's own layout."""
    import torch
    named = [(Q, "Q"), (K, "K"), (V, "V"), (O, "O")] + [(t, n) for t, n in ((Qp, "Qp"), (Kp, "Kp"), (Vp, "Vp"))
                                                          if t is not None]
    for t, n in named:
        _dev_tensor(t, n, torch.bfloat16)
    _dev_tensor(head_is_temporal, "head_is_temporal", torch.uint8)
    _dev_tensor(lse, "lse", torch.float32)
    _check_shapes(tile_map, lse, *named)
    _check(load().bss_attention_step(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(lse), tile_map.handle,
                                     _ptr(head_is_temporal), Q.shape[0], _ptr(Qp), _ptr(Kp), _ptr(Vp),
                                     _stream(stream)))
    return O


class StepWorkspace:
    """Owning wrapper of a ``bss_step_workspace`` (device buffer sets, copy
    streams and events of ``attention_step_host``)."""

    def __init__(self, handle, params: MaskParams, H: int, depth: int, heads_per_group: int):
        self._h = handle
        self.params, self.H, self.depth, self.heads_per_group = params, H, depth, heads_per_group

    @property
    def handle(self):
        if self._h is None:
            raise ValueError("step workspace destroyed")
        return self._h

    def wait_stream(self, stream=None):
        """Order the workspace's copy streams after the work enqueued on ``stream``."""
        _check(load().bss_step_workspace_wait_stream(self.handle, _stream(stream)))

    def destroy(self):
        if self._h is not None and _lib is not None:
            _lib.bss_step_workspace_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.destroy()


def step_workspace(params: MaskParams, H: int, depth: int = 3, heads_per_group: int = 2) -> StepWorkspace:
    """Workspace of ``attention_step_host`` (``bss_step_workspace_create``).

    depth buffer sets used in turn: with three (the default) the host-to-device
    copy of a call can start while the device-to-host copy of the call two back
    is still running; measured with two, steps were 2.4% slower (6.00 vs 5.86
    ms on the mixed 75.6K workload, against 5.78 ms for the kernels alone).
    heads_per_group heads are copied in and computed together: two (the
    default) cost nothing when the host link keeps up and shorten the step when
    it does not (6.07 ms per step against 7.22 ms for one group of all ten
    heads on a box whose host-to-device copies slowed down now and then);
    single-head groups were slower (7.2-7.4 ms: ten small attention launches,
    each with its own tail)."""
    h = ctypes.c_void_p()
    mp = params.c()
    _check(load().bss_step_workspace_create(ctypes.byref(mp), H, depth, heads_per_group, ctypes.byref(h)))
    return StepWorkspace(h, params, H, depth, heads_per_group)


def _host_tensor(t, name, dtype):
    import torch
    if not isinstance(t, torch.Tensor) or t.is_cuda:
        raise ValueError(f"{name} must be a CPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def attention_step_host(hQ, hK, hV, hO, tile_map: TileMap, head_is_temporal, workspace: StepWorkspace, stream=None):
    """The per-layer path from HOST buffers (``bss_attention_step_host``): H2D
    copies of Q, K, V, the ``attention_step`` kernels and the D2H copy of O,
    pipelined over groups of heads on the workspace's copy streams and
    ``stream`` (default: current).  hQ, hK, hV, hO: CPU bf16 [H][N][d], pinned
    for overlap; head_is_temporal: CPU uint8[H].  Returns a CUDA event that
    completes when hO is written; until then the host buffers must stay alive
    (the copies read and write them asynchronously) and the inputs unchanged."""
    import torch
    for t, n in ((hQ, "hQ"), (hK, "hK"), (hV, "hV"), (hO, "hO")):
        _host_tensor(t, n, torch.bfloat16)
    _host_tensor(head_is_temporal, "head_is_temporal", torch.uint8)
    p = tile_map.params
    shape = (workspace.H, p.N, p.head_dim)
    for t, n in ((hQ, "hQ"), (hK, "hK"), (hV, "hV"), (hO, "hO")):
        if tuple(t.shape) != shape:
            raise ValueError(f"{n} has shape {tuple(t.shape)}, the workspace and map want {shape}")
    if tuple(head_is_temporal.shape) != (workspace.H,):
        raise ValueError(f"head_is_temporal must have {workspace.H} entries")
    done = torch.cuda.Event()
    done.record()  # creates the event; the library records it again after the D2H copy
    _check(load().bss_attention_step_host(_ptr(hQ), _ptr(hK), _ptr(hV), _ptr(hO), _ptr(head_is_temporal),
                                          tile_map.handle, workspace.handle, ctypes.c_void_p(done.cuda_event),
                                          _stream(stream)))
    return done


# ---------------------------------------------------------------- around the attention step (include/bss_block.h)

def _current_device():
    import torch
    return torch.cuda.current_device()


def _stream_on(stream, device):
    """The address of a stream (None: the current one of the device)."""
    import torch
    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:  # the address alone: a Stream object costs 3 us
        return raw(device)
    return torch.cuda.current_stream().cuda_stream


def _on_device(t, name, device):
    """A tensor on the current device, where kernels are launched."""
    try:
        on = t.get_device()
    except AttributeError:
        on = -1
    if on != device:
        raise ValueError(f"{name} must be a CUDA tensor" if on < 0 else
                         f"{name} is on cuda:{on}, the current device is cuda:{device}")


def _exact(t, name, dtype, shape, device):
    """The address of a given contiguous tensor of this type and shape (None: None)."""
    if t is None:
        return None
    if getattr(t, "dtype", None) != dtype or t.get_device() != device:
        _on_device(t, name, device)
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, must be {shape}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _dtype_code(dtype, name):
    import torch
    if dtype == torch.bfloat16:
        return DTYPE_BF16
    if dtype == torch.float32:
        return DTYPE_F32
    raise ValueError(f"{name} must be bfloat16 or float32, got {dtype}")


def _one_dtype(*named):
    """The type that every given tensor has (None when none is given)."""
    dtype = None
    for t, n in named:
        if t is None:
            continue
        if dtype is None:
            dtype = getattr(t, "dtype", None)
            _dtype_code(dtype, n)
        elif getattr(t, "dtype", None) != dtype:
            raise ValueError(f"{', '.join(m for u, m in named if u is not None)} must have one type")
    return dtype


def _empty_on(stream, *shape, dtype):
    """Memory from torch's allocator that belongs to the stream the call runs on."""
    import torch
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device="cuda")
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(stream):
        return torch.empty(*shape, dtype=dtype, device="cuda")


def _workspace(workspace, nbytes, stream):
    """The caller's workspace, or one that belongs to the stream of the call."""
    import torch
    if workspace is not None:
        _on_device(workspace, "workspace", _current_device())
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        return workspace
    return None if nbytes == 0 else _empty_on(stream, nbytes, dtype=torch.uint8)


def rotary_table(length: int, pairs: int, base: float = 10000.0, dim: int | None = None, positions=None, out=None,
                 stream=None):
    """(cos, sin) of one rotary axis, float32 [length][pairs][2] (``bss_rotary_table``):
    position i (or positions[i], a float64 CUDA tensor) times base^(-2 j / dim) for
    pair j; dim defaults to 2 * pairs.  Angles are taken in 64 bits.  A table that
    the call makes (out None) belongs to its stream, like a tensor made there."""
    import torch
    if length <= 0 or pairs <= 0:
        raise ValueError("length and pairs must be positive")
    if out is None:
        out = _empty_on(stream, length, pairs, 2, dtype=torch.float32)
    device = _current_device()
    _check(load().bss_rotary_table(_exact(positions, "positions", torch.float64, (length,), device), length, pairs,
                                   2 * pairs if dim is None else dim, float(base),
                                   _exact(out, "out", torch.float32, (length, pairs, 2), device), _stream_on(stream, device)))
    return out


class Rotary:
    """Rotary positions of the (time, height, width) axes for ``heads_from_tokens``.

    time, height, width: float32 CUDA tables [positions][pairs][2] of (cos, sin)
    (``rotary_table`` makes one), None for an axis that turns nothing; the pairs
    of the three are dealt to the channels in this order.  Token (f, h, w) uses
    rows offset + (f, h, w).  pairing: PAIR_INTERLEAVED or PAIR_HALVES.  Holds
    the tables; what it was made from is not changed afterwards."""
    __slots__ = ("time", "height", "width", "offset", "pairing", "device", "_struct", "_pointer")

    def __init__(self, time=None, height=None, width=None, offset=(0, 0, 0), pairing: int = PAIR_INTERLEAVED):
        import torch
        self.time, self.height, self.width, self.offset, self.pairing = time, height, width, offset, pairing
        if len(offset) != 3:
            raise ValueError("offset must have three entries")
        device, address, sizes = None, [], []
        for t in (time, height, width):
            if t is None:
                address.append(0)
                sizes.append((0, 0))
                continue
            shape = getattr(t, "shape", ())
            if len(shape) != 3 or shape[2] != 2:
                raise ValueError("a rotary table must be a tensor [positions][pairs][2]")
            if device is None:
                device = t.get_device()
            address.append(_exact(t, "a rotary table", torch.float32, shape, device if device >= 0 else 0))
            sizes.append(shape)
        self.device = device
        time_, height_, width_ = sizes
        try:
            packed = _ROTARY_BYTES.pack(*address, time_[0], height_[0], width_[0], time_[1], height_[1], width_[1],
                                        *offset, pairing)
        except struct.error:
            raise ValueError("offset and pairing must be integers of 32 bits") from None
        self._struct = _Rotary.from_buffer_copy(packed)
        self._pointer = ctypes.pointer(self._struct)


def _token_tensor(t, name, shape, device):
    """A [N][H][d] bf16 tensor with any token and head strides -> its C form."""
    import torch
    if t is None:
        return None
    if t.dtype != torch.bfloat16 or t.get_device() != device:
        _on_device(t, name, device)
        raise ValueError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, must be {shape} (tokens, heads, channels)")
    tokens, heads, channels = t.stride()
    if channels != 1:
        raise ValueError(f"{name}: the channels of a head must be contiguous")
    return ctypes.byref(_TokenTensor(t.data_ptr(), tokens, heads))


def _heads_options(H, d, rotary, q_weight, k_weight, norm, eps, device):
    if norm == HEAD_NORM_NONE and (q_weight is not None or k_weight is not None):
        raise ValueError("weights are given without a norm")
    if rotary is not None:
        if not isinstance(rotary, Rotary):
            raise ValueError("rotary must be a Rotary")
        if rotary.device is not None and rotary.device != device:
            raise ValueError(f"the rotary tables are on cuda:{rotary.device}, the current device is cuda:{device}")
    width = H * d if norm == HEAD_NORM_TOKEN else d
    dtype = _one_dtype((q_weight, "q_weight"), (k_weight, "k_weight"))
    code = DTYPE_F32 if dtype is None else _dtype_code(dtype, "weights")
    return _HeadsOptions(norm, eps, code, _exact(q_weight, "q_weight", dtype, (width,), device),
                         _exact(k_weight, "k_weight", dtype, (width,), device),
                         None if rotary is None else rotary._pointer), width


def _heads_of(*tensors, axis):
    for t in tensors:
        if t is not None:
            if getattr(t, "ndim", 0) != 3:
                raise ValueError("Q, K and V must be CUDA tensors of three dimensions")
            return t.shape[axis]
    raise ValueError("no tensor given")


def heads_from_tokens(q, k, v, Qh, Kh, Vh, params: MaskParams, head_is_temporal=None, rotary: Rotary | None = None,
                      q_weight=None, k_weight=None, norm: int = HEAD_NORM_NONE, eps: float = 1e-6, stream=None):
    """Qh, Kh, Vh <- the heads of token-major q, k, v in one pass (``bss_heads_from_tokens``).

    q, k, v: bf16 [N][H][d] CUDA tensors whose tokens and heads may be strided
    (views of a packed projection, or of head-major tensors) or broadcast; Qh,
    Kh, Vh: contiguous bf16 [H][N][d], heads with flag 1 in (H,W,F) order, the
    others in (F,H,W) order -- what ``sparse_attention`` takes.  Q and K are
    RMS-normed over each head (HEAD_NORM_HEAD, weights [d]) or over all heads of a
    token (HEAD_NORM_TOKEN, weights [H * d]) and turned by ``rotary``.  Each pair
    (q, Qh), (k, Kh), (v, Vh) may be None."""
    import torch
    H, d, N = _heads_of(q, k, v, axis=1), params.head_dim, params.N
    device = _current_device()
    options, _ = _heads_options(H, d, rotary, q_weight, k_weight, norm, eps, device)
    shape, heads = (N, H, d), (H, N, d)
    _check(load().bss_heads_from_tokens(
        _token_tensor(q, "q", shape, device), _token_tensor(k, "k", shape, device), _token_tensor(v, "v", shape, device),
        _exact(Qh, "Qh", torch.bfloat16, heads, device), _exact(Kh, "Kh", torch.bfloat16, heads, device),
        _exact(Vh, "Vh", torch.bfloat16, heads, device), _exact(head_is_temporal, "head_is_temporal", torch.uint8, (H,), device), H,
        ctypes.byref(params.c()), ctypes.byref(options), _stream_on(stream, device)))
    return Qh, Kh, Vh


def heads_from_tokens_backward(dQh, dKh, dVh, dq, dk, dv, params: MaskParams, head_is_temporal=None,
                               rotary: Rotary | None = None, q=None, k=None, q_weight=None, k_weight=None,
                               dq_weight=None, dk_weight=None, norm: int = HEAD_NORM_NONE, eps: float = 1e-6,
                               workspace=None, stream=None):
    """Gradients of ``heads_from_tokens`` (``bss_heads_from_tokens_backward``).

    dQh, dKh, dVh: bf16 [H][N][d] in the layout of its outputs; dq, dk, dv: bf16
    [N][H][d] outputs, strided as the inputs may be (e.g. views of one packed
    gradient).  With a norm, q and k are the forward inputs, and dq_weight,
    dk_weight optional float32 outputs of the weights' shapes, overwritten.
    workspace: memory for the weights' partial sums (taken from torch's allocator
    when None)."""
    import torch
    H, d, N = _heads_of(dQh, dKh, dVh, axis=0), params.head_dim, params.N
    device = _current_device()
    options, width = _heads_options(H, d, rotary, q_weight, k_weight, norm, eps, device)
    shape, heads, lib, mp = (N, H, d), (H, N, d), load(), ctypes.byref(params.c())
    nbytes = 0
    if dq_weight is not None or dk_weight is not None:
        need = ctypes.c_int64()
        _check(lib.bss_heads_from_tokens_backward_workspace(H, mp, norm, ctypes.byref(need)))
        workspace = _workspace(workspace, need.value, stream)
        nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    else:
        workspace = None
    _check(lib.bss_heads_from_tokens_backward(
        _exact(dQh, "dQh", torch.bfloat16, heads, device), _exact(dKh, "dKh", torch.bfloat16, heads, device),
        _exact(dVh, "dVh", torch.bfloat16, heads, device), _token_tensor(q, "q", shape, device), _token_tensor(k, "k", shape, device),
        _token_tensor(dq, "dq", shape, device), _token_tensor(dk, "dk", shape, device), _token_tensor(dv, "dv", shape, device),
        _exact(dq_weight, "dq_weight", torch.float32, (width,), device), _exact(dk_weight, "dk_weight", torch.float32, (width,), device),
        _exact(head_is_temporal, "head_is_temporal", torch.uint8, (H,), device), H, mp, ctypes.byref(options),
        None if workspace is None else workspace.data_ptr(), nbytes, _stream_on(stream, device)))
    return dq, dk, dv


def attention_step_tokens(q, k, v, O, tile_map: TileMap, head_is_temporal, Qh, Kh, Vh, rotary: Rotary | None = None,
                          q_weight=None, k_weight=None, norm: int = HEAD_NORM_NONE, eps: float = 1e-6, lse=None,
                          stream=None):
    """The per-layer path from token-major projections (``bss_attention_step_tokens``):
    ``heads_from_tokens`` into the workspaces Qh, Kh, Vh, then block-sparse
    attention with every head's O rows in (F,H,W) order, in two launches.  lse as
    in ``attention_step``."""
    import torch
    p = tile_map.params
    H, d, N = _heads_of(q, axis=1), p.head_dim, p.N
    named = ((O, "O"), (Qh, "Qh"), (Kh, "Kh"), (Vh, "Vh"))
    device = _current_device()
    for t, n in named:
        if t is None:
            raise ValueError(f"{n} must be a CUDA tensor")
    options, _ = _heads_options(H, d, rotary, q_weight, k_weight, norm, eps, device)
    shape = (N, H, d)
    O_p, Q_p, K_p, V_p = (_exact(t, n, torch.bfloat16, (H, N, d), device) for t, n in named)
    _check(load().bss_attention_step_tokens(
        _token_tensor(q, "q", shape, device), _token_tensor(k, "k", shape, device), _token_tensor(v, "v", shape, device), O_p,
        _exact(lse, "lse", torch.float32, (H, N), device), tile_map.handle,
        _exact(head_is_temporal, "head_is_temporal", torch.uint8, (H,), device), H, ctypes.byref(options), Q_p, K_p, V_p,
        _stream_on(stream, device)))
    return O


def _row_tensor(t, name, dtype, shape, device):
    """(address, row stride) of a given [rows][channels] tensor with any row stride."""
    if t is None:
        return None, 0
    if t.get_device() != device:
        _on_device(t, name, device)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, must be {shape}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    rows, channels = t.stride()
    if channels != 1:
        raise ValueError(f"{name}: the channels of a row must be contiguous")
    return t.data_ptr(), rows


def _row_shape(t, name):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{name} must be a CUDA tensor [rows][channels]")
    return t.shape


def _groups(rows, rows_per_group, channels):
    """Rows per group and the shape of per-group parameters."""
    if rows_per_group is None:
        rows_per_group = rows
    if rows <= 0 or rows_per_group <= 0:
        raise ValueError("rows and rows_per_group must be positive")
    return rows_per_group, (-(-rows // rows_per_group), channels)


def residual_norm(x, y=None, r=None, h=None, gate=None, scale=None, shift=None, weight=None, bias=None, y_weight=None,
                  norm: int = NORM_LAYER, y_norm: int = NORM_NONE, rows_per_group: int | None = None,
                  residual_scale: float = 1.0, eps: float = 1e-6, stats=None, y_stats=None, stream=None):
    """The residual update of a block and the norm in front of the next one, in
    one pass (``bss_residual_norm``)::

        r = residual_scale * x + gate * y_norm(y) * y_weight
        h = (norm(r) * weight + bias) * (1 + scale) + shift

    x, r: [rows][channels] bf16 or float32 (the stream); y, h: bf16, or float32
    with a float32 stream.  Without y only h is made, from x.  r may be x, and h
    may be y (in place).  gate, scale, shift: [groups][channels], row i in group
    i // rows_per_group (default: one group); weight, bias, y_weight: [channels];
    all of these float32 or all bf16, all optional.  norm, y_norm: NORM_*.  stats,
    y_stats: float32 [rows][2] outputs, (mean, 1 / deviation) of each row, for the
    backward pass.  Returns (r, h)."""
    import torch
    shape = rows, channels = _row_shape(x, "x")
    device = _current_device()
    group, mods = _groups(rows, rows_per_group, channels)
    branch = _one_dtype((y, "y"), (h, "h"))
    param = _one_dtype((gate, "gate"), (scale, "scale"), (shift, "shift"), (weight, "weight"), (bias, "bias"),
                       (y_weight, "y_weight"))
    x_p, x_s = _row_tensor(x, "x", x.dtype, shape, device)
    y_p, y_s = _row_tensor(y, "y", branch, shape, device)
    r_p, r_s = _row_tensor(r, "r", x.dtype, shape, device)
    h_p, h_s = _row_tensor(h, "h", branch, shape, device)
    gate_p, gate_s = _row_tensor(gate, "gate", param, mods, device)
    scale_p, scale_s = _row_tensor(scale, "scale", param, mods, device)
    shift_p, shift_s = _row_tensor(shift, "shift", param, mods, device)
    a = _ResidualNormArgs(
        rows, group, channels, _dtype_code(x.dtype, "x"), DTYPE_BF16 if branch is None else _dtype_code(branch, "h"),
        DTYPE_F32 if param is None else _dtype_code(param, "weights"), norm, y_norm, eps, residual_scale, x_p, y_p, r_p,
        h_p, x_s, y_s, r_s, h_s, gate_p, scale_p, shift_p, gate_s, scale_s, shift_s,
        _exact(weight, "weight", param, (channels,), device), _exact(bias, "bias", param, (channels,), device),
        _exact(y_weight, "y_weight", param, (channels,), device), _exact(stats, "stats", torch.float32, (rows, 2), device),
        _exact(y_stats, "y_stats", torch.float32, (rows, 2), device))
    _check(load().bss_residual_norm(ctypes.byref(a), _stream_on(stream, device)))
    return r, h


def residual_norm_backward(r, y=None, dr=None, dh=None, dx=None, dy=None, stats=None, y_stats=None, gate=None,
                           scale=None, weight=None, bias=None, y_weight=None, dgate=None, dscale=None, dshift=None,
                           dweight=None, dbias=None, dy_weight=None, norm: int = NORM_LAYER, y_norm: int = NORM_NONE,
                           rows_per_group: int | None = None, residual_scale: float = 1.0, workspace=None,
                           stream=None):
    """Gradients of ``residual_norm`` (``bss_residual_norm_backward``).

    r: the updated stream it wrote (x when there was no y), with the stats it
    kept; dr, dh: gradients of r and h (one may be None).  Outputs: dx (required;
    may be dr), dy (with y; may be dh), and any of dgate, dscale, dshift (float32
    [groups][channels]) and dweight, dbias, dy_weight (float32 [channels]), all
    overwritten.  Every sum over rows is taken in a fixed order.  workspace:
    memory for partial sums (taken from torch's allocator when None)."""
    import torch
    shape = rows, channels = _row_shape(dx, "dx")
    device = _current_device()
    group, mods = _groups(rows, rows_per_group, channels)
    branch = _one_dtype((y, "y"), (dh, "dh"), (dy, "dy"))
    param = _one_dtype((gate, "gate"), (scale, "scale"), (weight, "weight"), (bias, "bias"), (y_weight, "y_weight"))
    r_p, r_s = _row_tensor(r, "r", dx.dtype, shape, device)
    y_p, y_s = _row_tensor(y, "y", branch, shape, device)
    dr_p, dr_s = _row_tensor(dr, "dr", dx.dtype, shape, device)
    dh_p, dh_s = _row_tensor(dh, "dh", branch, shape, device)
    dx_p, dx_s = _row_tensor(dx, "dx", dx.dtype, shape, device)
    dy_p, dy_s = _row_tensor(dy, "dy", branch, shape, device)
    gate_p, gate_s = _row_tensor(gate, "gate", param, mods, device)
    scale_p, scale_s = _row_tensor(scale, "scale", param, mods, device)
    f32, row = torch.float32, (channels,)
    a = _ResidualNormGrads(
        rows, group, channels, _dtype_code(dx.dtype, "dx"), DTYPE_BF16 if branch is None else _dtype_code(branch, "dh"),
        DTYPE_F32 if param is None else _dtype_code(param, "weights"), norm, y_norm, residual_scale, r_p, y_p, dr_p,
        dh_p, dx_p, dy_p, r_s, y_s, dr_s, dh_s, dx_s, dy_s, _exact(stats, "stats", f32, (rows, 2), device),
        _exact(y_stats, "y_stats", f32, (rows, 2), device), gate_p, scale_p, gate_s, scale_s, _exact(weight, "weight", param, row, device),
        _exact(bias, "bias", param, row, device), _exact(y_weight, "y_weight", param, row, device), _exact(dgate, "dgate", f32, mods, device),
        _exact(dscale, "dscale", f32, mods, device), _exact(dshift, "dshift", f32, mods, device), _exact(dweight, "dweight", f32, row, device),
        _exact(dbias, "dbias", f32, row, device), _exact(dy_weight, "dy_weight", f32, row, device))
    lib, need, args = load(), ctypes.c_int64(), ctypes.byref(a)
    _check(lib.bss_residual_norm_backward_workspace(args, ctypes.byref(need)))
    workspace = _workspace(workspace, need.value, stream)
    if workspace is not None:
        a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _check(lib.bss_residual_norm_backward(args, _stream_on(stream, device)))
    return dx, dy


# ---------------------------------------------------------------- matrix products

def _matrix(t, name):
    """(rows, width) of a given CUDA matrix."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{name} must be a CUDA tensor of two dimensions")
    return t.shape


def _with_workspace(args, need, call, workspace, stream, device):
    """Makes a call whose workspace `need` tells the size of."""
    ref = ctypes.byref(args)
    nbytes = ctypes.c_int64()
    _check(need(ref, ctypes.byref(nbytes)))
    if nbytes.value or workspace is not None:
        workspace = _workspace(workspace, nbytes.value, stream)
        args.workspace, args.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _check(call(ref, _stream_on(stream, device)))


def linear(x, weight, out, bias=None, activation: int = ACT_NONE, gate=None, residual=None,
           rows_per_group: int | None = None, residual_scale: float = 1.0, pre=None, workspace=None, stream=None):
    """A linear layer with what follows it (``bss_linear``)::

        z   = x weight^T + bias
        out = residual_scale * residual + gate * activation(z)

    x: bf16 [rows][in]; weight: bf16 [out][in]; out, residual: bf16 or float32
    [rows][out] (out may be residual); bias [out] and gate [groups][out], row i in
    group i // rows_per_group (default: one group), both float32 or both bf16;
    activation: ACT_*.  pre: optional bf16 [rows][out] output, z for the backward
    pass.  Rows may be strided.  workspace: memory for partial sums where the call
    needs some (taken from torch's allocator when None).  Returns out."""
    import torch
    rows, inner = _matrix(x, "x")
    outer = _matrix(weight, "weight")[0]
    device = _current_device()
    group, mods = _groups(rows, rows_per_group, outer)
    dtype = _one_dtype((out, "out"), (residual, "residual"))
    if dtype is None:
        raise ValueError("out must be a CUDA tensor")
    param = _one_dtype((bias, "bias"), (gate, "gate"))
    bf16, shape = torch.bfloat16, (rows, outer)
    x_p, x_s = _row_tensor(x, "x", bf16, (rows, inner), device)
    w_p, w_s = _row_tensor(weight, "weight", bf16, (outer, inner), device)
    g_p, g_s = _row_tensor(gate, "gate", param, mods, device)
    r_p, r_s = _row_tensor(residual, "residual", dtype, shape, device)
    o_p, o_s = _row_tensor(out, "out", dtype, shape, device)
    p_p, p_s = _row_tensor(pre, "pre", bf16, shape, device)
    a = _LinearArgs(rows, group, inner, outer, _dtype_code(dtype, "out"),
                    DTYPE_F32 if param is None else _dtype_code(param, "bias"), activation, residual_scale, x_p, w_p,
                    _exact(bias, "bias", param, (outer,), device), g_p, r_p, o_p, p_p, x_s, w_s, g_s, r_s, o_s, p_s)
    lib = load()
    _with_workspace(a, lib.bss_linear_workspace, lib.bss_linear, workspace, stream, device)
    return out


def linear_backward(dout, x=None, weight=None, dx=None, dweight=None, dbias=None, dgate=None, activation: int = ACT_NONE,
                    pre=None, gate=None, rows_per_group: int | None = None, workspace=None, stream=None):
    """Gradients of ``linear`` (``bss_linear_backward``)::

        dz = gate * dout * activation'(pre)
        dx = dz weight      dweight = dz^T x      dbias = sum of dz
        dgate = sum over a group's rows of dout * activation(pre)

    dout: bf16 or float32 [rows][out]; x, weight, gate: the forward inputs (x for
    dweight, weight for dx); pre: the z that ``linear`` kept, with an activation or
    for dgate.  Outputs, each optional, overwritten: dx bf16 [rows][in], dweight
    bf16 or float32 [out][in], dbias float32 [out], dgate float32 [groups][out].
    (The residual's gradient is residual_scale * dout.)  Sums over rows are taken in
    a fixed order.  workspace: taken from torch's allocator when None."""
    import torch
    rows, outer = _matrix(dout, "dout")
    inner = None
    for t, n, axis in ((x, "x", 1), (weight, "weight", 1), (dx, "dx", 1), (dweight, "dweight", 1)):
        if t is not None and inner is None:
            inner = _matrix(t, n)[axis]
    device = _current_device()
    group, mods = _groups(rows, rows_per_group, outer)
    bf16, f32 = torch.bfloat16, torch.float32
    param = _one_dtype((gate, "gate"))
    dw = _one_dtype((dweight, "dweight"))
    d_p, d_s = _row_tensor(dout, "dout", dout.dtype, (rows, outer), device)
    x_p, x_s = _row_tensor(x, "x", bf16, (rows, inner), device)
    w_p, w_s = _row_tensor(weight, "weight", bf16, (outer, inner), device)
    p_p, p_s = _row_tensor(pre, "pre", bf16, (rows, outer), device)
    g_p, g_s = _row_tensor(gate, "gate", param, mods, device)
    dx_p, dx_s = _row_tensor(dx, "dx", bf16, (rows, inner), device)
    dw_p, dw_s = _row_tensor(dweight, "dweight", dw, (outer, inner), device)
    a = _LinearGrads(rows, group, 8 if inner is None else inner, outer, _dtype_code(dout.dtype, "dout"),
                     DTYPE_F32 if param is None else _dtype_code(param, "gate"),
                     DTYPE_F32 if dw is None else _dtype_code(dw, "dweight"), activation, d_p, x_p, w_p, p_p, g_p, dx_p, dw_p,
                     _exact(dbias, "dbias", f32, (outer,), device), _exact(dgate, "dgate", f32, mods, device),
                     d_s, x_s, w_s, p_s, g_s, dx_s, dw_s)
    lib = load()
    _with_workspace(a, lib.bss_linear_backward_workspace, lib.bss_linear_backward, workspace, stream, device)
    return dx, dweight


# ---------------------------------------------------------------- cross attention

def _rows_heads(t, name, shape, device):
    """A [rows][heads][d] bf16 tensor's C form."""
    import torch
    if getattr(t, "dtype", None) != torch.bfloat16 or t.get_device() != device:
        _on_device(t, name, device)
        raise ValueError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, must be {tuple(shape)} (rows, heads, channels)")
    rows, heads, channels = t.stride()
    if channels != 1:
        raise ValueError(f"{name}: the channels of a head must be contiguous")
    return _TokenTensor(t.data_ptr(), rows, heads)


def _states(t, name, groups, d, device, like=None):
    """(C form, keys, heads) of [groups][keys][heads][d] states ([keys][heads][d]: one group's)."""
    import torch
    if getattr(t, "dtype", None) != torch.bfloat16 or t.get_device() != device:
        _on_device(t, name, device)
        raise ValueError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.dim() == 3:
        t = t.unsqueeze(0)
    if t.dim() != 4 or t.shape[0] != groups or t.shape[3] != d or (like is not None and t.shape[1:3] != like):
        want = "keys, kv heads" if like is None else f"{like[0]}, {like[1]}"
        raise ValueError(f"{name} has shape {tuple(t.shape)}, must be ({groups}, {want}, {d}) (groups, states, heads, channels)")
    group, token, head, channels = t.stride()
    if channels != 1:
        raise ValueError(f"{name}: the channels of a head must be contiguous")
    return _StateTensor(t.data_ptr(), group, token, head), t.shape[1:3]


def _rows_heads_shape(t, name):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 3:
        raise ValueError(f"{name} must be a CUDA tensor [rows][heads][channels]")
    return t.shape


def cross_attention(q, k, v, O, lengths=None, lse=None, rows_per_group: int | None = None,
                    softmax_scale: float | None = None, stream=None):
    """O <- attention of token-major q over an encoder's states (``bss_cross_attention``).

    q, O: bf16 [rows][heads][d], d 64 or 128, rows and heads may be strided (O may
    be q); k, v: bf16 [groups][states][kv_heads][d] (views of a packed projection
    too; [states][kv_heads][d] with one group; a group stride of 0 shares one set
    between the groups).  Row i attends to the states of group i // rows_per_group
    (default: one group), head h to key head h // (heads // kv_heads).  lengths:
    int32 [groups], the first so many states of a group are valid and the others
    are not looked at (None: all); without any a row's O is 0 and its lse -inf.
    softmax_scale: None or not positive: 1 / sqrt(d).  lse: optional float32 [heads][rows] output for the backward pass.  Returns O."""
    import torch
    shape = rows, heads, d = _rows_heads_shape(q, "q")
    device = _current_device()
    group, (groups, _) = _groups(rows, rows_per_group, d)
    k_t, like = _states(k, "k", groups, d, device)
    a = _CrossArgs(rows, group, heads, like[1], d, like[0], 0.0 if softmax_scale is None else softmax_scale,
                   _rows_heads(q, "q", shape, device), _rows_heads(O, "O", shape, device), k_t,
                   _states(v, "v", groups, d, device, like)[0], _exact(lengths, "lengths", torch.int32, (groups,), device),
                   _exact(lse, "lse", torch.float32, (heads, rows), device))
    _check(load().bss_cross_attention(ctypes.byref(a), _stream_on(stream, device)))
    return O


def cross_attention_backward(dO, q, k, v, O, lse, dq, dk, dv, lengths=None, rows_per_group: int | None = None,
                             softmax_scale: float | None = None, workspace=None, stream=None):
    """Gradients of ``cross_attention`` (``bss_cross_attention_backward``).

    dO: bf16 [rows][heads][d], the gradient of O; q, k, v, lengths: the forward
    call's inputs, O and lse what it wrote; dq [rows][heads][d], dk and dv
    [groups][states][kv_heads][d]: bf16 outputs, strided as the inputs may be
    (views of one packed gradient, say), overwritten; states that are not valid
    get zeros.  States shared by several groups (a group stride of 0) are refused.  Sums over rows are taken in a fixed order.  workspace: taken from
    torch's allocator when None.  Returns (dq, dk, dv)."""
    import torch
    shape = rows, heads, d = _rows_heads_shape(q, "q")
    device = _current_device()
    group, (groups, _) = _groups(rows, rows_per_group, d)
    k_t, like = _states(k, "k", groups, d, device)
    v_t, dk_t, dv_t = (_states(t, n, groups, d, device, like)[0] for t, n in ((v, "v"), (dk, "dk"), (dv, "dv")))
    dO_t, q_t, O_t, dq_t = (_rows_heads(t, n, shape, device) for t, n in ((dO, "dO"), (q, "q"), (O, "O"), (dq, "dq")))
    if lse is None:
        raise ValueError("lse must be given")
    a = _CrossGrads(rows, group, heads, like[1], d, like[0], 0.0 if softmax_scale is None else softmax_scale, dO_t, q_t,
                    O_t, dq_t, k_t, v_t, dk_t, dv_t, _exact(lengths, "lengths", torch.int32, (groups,), device),
                    _exact(lse, "lse", torch.float32, (heads, rows), device))
    lib = load()
    _with_workspace(a, lib.bss_cross_attention_backward_workspace, lib.bss_cross_attention_backward, workspace, stream, device)
    return dq, dk, dv
