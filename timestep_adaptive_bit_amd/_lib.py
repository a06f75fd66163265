"""ctypes binding of libtabit.so: argument marshalling only.

Every computation runs in the HIP library; this module checks tensor dtype,
device and contiguity, allocates outputs with torch when the caller passes
none, and forwards raw device pointers and the current HIP stream.  It fails
loudly if the library has not been built.
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtabit.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "tabit.h")

OK, EINVAL, ESHAPE, EALIGN, ERANGE, ENOSCHED, EHIP, ENOMEM = 0, -1, -2, -3, -4, -5, -6, -7
FMT_INT8, FMT_MXFP4, FMT_BF16 = 0, 1, 2
PATH_MASKED, PATH_BITSERIAL, PATH_PLANES, PATH_HQDM = 0, 1, 3, 4
OPT_GEMM_CONFIG, OPT_MXFP4_CONFIG, OPT_PLANE_CONFIG, OPT_HQDM_CONFIG = 0, 1, 2, 3
PATH_MXFP4_GEMM = 2
ACT_NONE, ACT_GELU = 0, 1
NORM_NONE, NORM_LAYER, NORM_RMS = 0, 1, 2

_c_int, _c_void_p, _c_size_t, _c_float = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
_c_int64 = ctypes.c_int64
_PINT = ctypes.POINTER(ctypes.c_int)

# name -> (restype, argtypes)
_SIGNATURES = {
    "tabit_create": (_c_int, [ctypes.POINTER(_c_void_p)]),
    "tabit_destroy": (None, [_c_void_p]),
    "tabit_last_error": (ctypes.c_char_p, [_c_void_p]),
    "tabit_version": (ctypes.c_char_p, []),
    "tabit_quantize_weights": (_c_int, [_c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_void_p,
                                        _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "tabit_set_step_schedule": (_c_int, [_c_void_p, _c_int, _c_int, _c_void_p, _c_void_p]),
    "tabit_schedule_lookup": (_c_int, [_c_void_p, _c_int, _c_int, _PINT, _PINT]),
    "tabit_hadamard_quant_act": (_c_int, [_c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_int,
                                          _c_void_p, _c_void_p, _c_void_p]),
    "tabit_masked_qgemm": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int,
                                    _c_int, _c_int, _c_int, _c_void_p, _c_void_p, _c_void_p]),
    "tabit_qgemm_bitserial": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                       _c_int, _c_int, _c_int, _c_int, _c_void_p, _c_void_p,
                                       _c_void_p]),
    "tabit_mxfp4_qgemm": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int,
                                   _c_int, _c_int, _c_float, _c_void_p, _c_void_p, _c_void_p]),
    "tabit_act_workspace_bytes": (_c_size_t, [_c_int, _c_int]),
    "tabit_scheduled_linear": (_c_int, [_c_void_p, _c_int, _c_int, _c_int, _c_void_p, _c_int,
                                        _c_int, _c_int, _c_int, _c_void_p, _c_void_p, _c_void_p,
                                        _c_void_p, _c_void_p, _c_size_t, _c_void_p, _c_void_p]),
    "tabit_noalloc_scratch_bytes": (_c_size_t, []),
    "tabit_scheduled_linear_noalloc": (_c_int, [_c_void_p, _c_int, _c_int, _c_int, _c_void_p,
                                                _c_int, _c_int, _c_int, _c_int, _c_void_p,
                                                _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                                _c_void_p]),
    "tabit_run_schedule": (_c_int, [_c_void_p, _c_int, _c_int, _c_void_p, _c_int, _c_void_p,
                                    _c_int, _c_int, _c_void_p, _c_size_t, _c_void_p, _c_void_p]),
    "tabit_autotune_gemm": (_c_int, [_c_void_p, _c_int, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                     _c_int, _c_int, _c_int, _c_int, _c_void_p, _c_int, _PINT,
                                     _c_void_p]),
    "tabit_set_option": (_c_int, [_c_void_p, _c_int, _c_int]),
    "tabit_gemm_config_info": (_c_int, [_c_int, _PINT, _PINT, _PINT]),
    "tabit_gemm_config_choose": (_c_int, [_c_int, _c_int, _c_int, _c_int]),
    "tabit_mxfp4_config_info": (_c_int, [_c_int, _PINT, _PINT]),
    "tabit_pack_weight_planes": (_c_int, [_c_void_p, _c_void_p, _c_int, _c_int, _c_void_p,
                                          _c_void_p]),
    "tabit_plane_qgemm": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int,
                                   _c_int, _c_int, _c_int, _c_void_p, _c_void_p, _c_void_p]),
    "tabit_plane_config_info": (_c_int, [_c_int, _PINT, _PINT, _PINT]),
    "tabit_plane_config_choose": (_c_int, [_c_int, _c_int, _c_int, _c_int]),
    "tabit_mxfp4_config_choose": (_c_int, [_c_int, _c_int, _c_int, _c_int]),
    "tabit_mfma_peak_probe": (_c_int, [_c_void_p, _c_int, _c_int, _c_void_p, _c_size_t,
                                       ctypes.POINTER(ctypes.c_double), _c_void_p]),
    "tabit_mfma_probe_sink_ints": (_c_size_t, [_c_int]),
    "tabit_weight_planes_bytes": (_c_size_t, [_c_int, _c_int]),
    "tabit_dmpq_workspace_bytes": (_c_size_t, [_c_int]),
    "tabit_gelu_quant_act": (_c_int, [_c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_int,
                                      _c_void_p, _c_void_p, _c_void_p]),
    "tabit_hqdm_quant_act": (_c_int, [_c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_void_p,
                                      _c_void_p, _c_void_p, _c_void_p]),
    "tabit_hqdm_qgemm": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                  _c_int, _c_int, _c_int, _c_int, _c_void_p, _c_void_p, _c_void_p]),
    "tabit_hqdm_config_info": (_c_int, [_c_int, _PINT, _PINT]),
    "tabit_dmpq_select": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int, _c_int, _c_void_p,
                                   _c_int, _c_void_p, _c_void_p, _c_void_p, _c_size_t, _c_void_p]),
    "tabit_gated_linear": (_c_int, [_c_void_p, _c_void_p, _c_int, _c_int, _c_void_p, _c_int, _c_int,
                                    _c_int, _c_int, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                    _c_void_p, _c_size_t, _c_void_p, _c_void_p]),
    "tabit_kv_append": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int64, _c_void_p, _c_int64,
                                 _c_int, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "tabit_kv_read": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int, _c_void_p, _c_void_p,
                               _c_void_p]),
    "tabit_kv_attention": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "tabit_kv_attention_workspace_bytes": (_c_size_t, [_c_int] * 7),
    "tabit_block_norm": (_c_int, [_c_void_p, _c_void_p, _c_void_p]),
    "tabit_kv_tree_attention": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int, _c_void_p]),
    "tabit_kv_tree_attention_workspace_bytes": (_c_size_t, [_c_int] * 7),
    "tabit_tree_mask": (_c_int, [_c_void_p, _c_void_p, _c_int, _c_void_p, _c_int, _c_int, _c_void_p,
                                 _c_int, _c_void_p, _c_void_p]),
    "tabit_kv_weigh": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "tabit_kv_weigh_workspace_bytes": (_c_size_t, [_c_int] * 7),
    "tabit_kv_evict": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int, _c_void_p, _c_int,
                                _c_int, _c_int, _c_int, _c_int, _c_void_p, _c_void_p, _c_void_p,
                                _c_size_t, _c_void_p]),
    "tabit_kv_evict_workspace_bytes": (_c_size_t, [_c_int] * 3),
    "tabit_kv_compact": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int, _c_int, _c_void_p, _c_int,
                                  _c_int, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_size_t,
                                  _c_void_p]),
    "tabit_kv_compact_workspace_bytes": (_c_size_t, [_c_int] * 4),
    "tabit_adapter_linear": (_c_int, [_c_void_p, _c_void_p, _c_void_p]),
    "tabit_adapter_workspace_bytes": (_c_size_t, [_c_int] * 3),
    "tabit_adapter_rotate": (_c_int, [_c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_void_p, _c_void_p]),
}



class Layer(ctypes.Structure):
    """tabit_layer: one linear of a stack (device pointers as integers)."""
    _fields_ = [("M", ctypes.c_int), ("N", ctypes.c_int), ("K", ctypes.c_int),
                ("w_q", ctypes.c_void_p), ("w_scale", ctypes.c_void_p),
                ("w_fp4", ctypes.c_void_p), ("w_e8m0", ctypes.c_void_p),
                ("y_bf16", ctypes.c_void_p), ("input_from", ctypes.c_int),
                ("input_act", ctypes.c_int)]


class _KvCache(ctypes.Structure):
    """tabit_kv_cache."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("num_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("had_block", ctypes.c_int)]


class _Rope(ctypes.Structure):
    """tabit_rope."""
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("num_positions", ctypes.c_int),
                ("rope_dim", ctypes.c_int), ("interleaved", ctypes.c_int)]


class _KvAttentionArgs(ctypes.Structure):
    """tabit_kv_attention_args."""
    _fields_ = [("q", ctypes.c_void_p), ("q_stride", ctypes.c_int64), ("num_tokens", ctypes.c_int),
                ("num_q_heads", ctypes.c_int), ("cu_q", ctypes.c_void_p), ("num_seqs", ctypes.c_int),
                ("max_q", ctypes.c_int), ("block_table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int), ("kv_lens", ctypes.c_void_p),
                ("max_kv", ctypes.c_int), ("scale", ctypes.c_float), ("causal", ctypes.c_int),
                ("rope", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("lse", ctypes.c_void_p), ("ws", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t)]


class _BlockNormArgs(ctypes.Structure):
    """tabit_block_norm_args."""
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("rows", ctypes.c_int),
                ("width", ctypes.c_int), ("post_kind", ctypes.c_int), ("pre_kind", ctypes.c_int),
                ("post_weight", ctypes.c_void_p), ("pre_weight", ctypes.c_void_p),
                ("gate", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("shift", ctypes.c_void_p),
                ("mod_stride", ctypes.c_int64), ("num_samples", ctypes.c_int),
                ("rows_per_sample", ctypes.c_int), ("res_scale", ctypes.c_float),
                ("eps", ctypes.c_float), ("x_out", ctypes.c_void_p), ("h", ctypes.c_void_p),
                ("h_scale", ctypes.c_void_p), ("fmt", ctypes.c_int), ("had_block", ctypes.c_int)]


class _AdapterArgs(ctypes.Structure):
    """tabit_adapter_args."""
    _fields_ = [("x", ctypes.c_void_p), ("x_scale", ctypes.c_void_p), ("x_fmt", ctypes.c_int),
                ("rows", ctypes.c_int), ("K", ctypes.c_int), ("N", ctypes.c_int),
                ("x_stride", ctypes.c_int64), ("a", ctypes.c_void_p), ("b", ctypes.c_void_p),
                ("scale", ctypes.c_void_p), ("num_adapters", ctypes.c_int), ("rank", ctypes.c_int),
                ("cu_rows", ctypes.c_void_p), ("adapter", ctypes.c_void_p),
                ("num_segments", ctypes.c_int), ("y", ctypes.c_void_p), ("y_stride", ctypes.c_int64),
                ("out", ctypes.c_void_p), ("out_stride", ctypes.c_int64), ("ws", ctypes.c_void_p),
                ("ws_bytes", ctypes.c_size_t)]


_lib = None


def header_functions() -> list:
    """Names of the functions include/tabit.h declares."""
    with open(HEADER_PATH) as f:
        text = f.read()
    return sorted(set(re.findall(r"\b(tabit_[a-z0-9_]+)\s*\(", text)))


def load() -> ctypes.CDLL:
    """Load libtabit.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with `python -m timestep_adaptive_bit_amd.build` "
            "(there is no fallback implementation)")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


class TabitError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"tabit status {status}: {message}")
        self.status = status


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


# The handle itself, where this torch has that call (it is not a public one): building a Stream
# object to ask for it takes longer than a small launch.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device: torch.device) -> int:
    if _raw_stream is None or device.index is None:
        return torch.cuda.current_stream(device).cuda_stream
    return _raw_stream(device.index)


def _dev(t: torch.Tensor, dtype, name: str, shape=None) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _counts(*values) -> None:
    """Refuses what a C int does not hold: ctypes would cut it without a word."""
    for v in values:
        if not -0x80000000 <= v <= 0x7FFFFFFF:
            raise ValueError(f"a count of {v} does not fit the library's 32 bits")


def _rows(t: torch.Tensor, name: str, tail, device) -> int:
    """bf16 [T][heads][head_dim] whose tokens may be apart (a slice of a fused output):
    the stride of a token in elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dim() != 3 or t.shape[1:] != tail:
        raise ValueError(f"{name} must have shape [tokens, {tail[0]}, {tail[1]}], got {tuple(t.shape)}")
    s = t.stride()
    if (s[2] != 1 and tail[1] > 1) or (s[1] != tail[1] and tail[0] > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return s[0] if t.shape[0] > 1 else tail[0] * tail[1]


def _on(t: torch.Tensor, dtype, name: str, shape, device) -> None:
    if (isinstance(t, torch.Tensor) and t.device == device and t.dtype == dtype and t.shape == shape
            and t.is_contiguous()):
        return
    _dev(t, dtype, name, shape)
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


class KVCache:
    """A paged MXFP4 key / value cache (tabit_kv_cache): its four tensors, kept alive here.

    k_codes, v_codes uint8 [pages][kv_heads][page_size][Dp/2]; k_scales, v_scales uint8
    [pages][kv_heads][page_size][Dp/32]; Dp = 32 ceil(head_dim / 32).
    """

    def __init__(self, k_codes, k_scales, v_codes, v_scales, head_dim: int, had_block: int = 0):
        dp = (head_dim + 31) // 32 * 32
        _dev(k_codes, torch.uint8, "k_codes")
        if k_codes.dim() != 4 or k_codes.shape[3] != dp // 2:
            raise ValueError(f"k_codes must be [pages][kv_heads][page_size][{dp // 2}]")
        lead = tuple(k_codes.shape[:3])
        _on(v_codes, torch.uint8, "v_codes", lead + (dp // 2,), k_codes.device)
        _on(k_scales, torch.uint8, "k_scales", lead + (dp // 32,), k_codes.device)
        _on(v_scales, torch.uint8, "v_scales", lead + (dp // 32,), k_codes.device)
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.num_pages, self.num_kv_heads, self.page_size = lead
        self.head_dim, self.had_block, self.device = head_dim, had_block, k_codes.device
        self._row = torch.Size((self.num_kv_heads, head_dim))
        self._c = _KvCache(k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(),
                           v_scales.data_ptr(), self.num_pages, self.page_size, self.num_kv_heads,
                           head_dim, had_block)
        self._ref = ctypes.addressof(self._c)

    @classmethod
    def empty(cls, num_pages: int, page_size: int, num_kv_heads: int, head_dim: int,
              had_block: int = 0, device="cuda:0") -> "KVCache":
        """A cache of zeros."""
        dp = (head_dim + 31) // 32 * 32
        t = [torch.zeros((num_pages, num_kv_heads, page_size, w), dtype=torch.uint8, device=device)
             for w in (dp // 2, dp // 32, dp // 2, dp // 32)]
        return cls(*t, head_dim=head_dim, had_block=had_block)


class Rope:
    """Rotation tables (tabit_rope): cos and sin fp32 [positions][rope_dim/2]; interleaved
    False: pairs (i, i + rope_dim/2), True: pairs (2i, 2i + 1)."""

    def __init__(self, cos: torch.Tensor, sin: torch.Tensor, interleaved: bool = False):
        _dev(cos, torch.float32, "cos")
        if cos.dim() != 2:
            raise ValueError("cos must be [positions][rope_dim/2]")
        _on(sin, torch.float32, "sin", cos.shape, cos.device)
        self.cos, self.sin, self.interleaved, self.device = cos, sin, interleaved, cos.device
        self._c = _Rope(cos.data_ptr(), sin.data_ptr(), cos.shape[0], 2 * cos.shape[1],
                        1 if interleaved else 0)
        self._ref = ctypes.addressof(self._c)


def _matrix(t: torch.Tensor, name: str, width, device) -> int:
    """bf16 [T][width] whose rows may be apart (a slice of a fused output): the stride of a row."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dim() != 2 or t.shape[1] != width:
        raise ValueError(f"{name} must have shape [rows, {width}], got {tuple(t.shape)}")
    if t.stride(1) != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else width


class Adapters:
    """Low-rank adapters that one projection's requests choose from, kept alive here.

    a bf16 [adapters][rank][K], b bf16 [adapters][N][rank], scale fp32 [adapters] or None (1); the
    rank 16, 32, 64 or 128.  For rows that are transformed before they are quantized, a is to be
    transformed too (Context.adapter_rotate).
    """

    def __init__(self, a: torch.Tensor, b: torch.Tensor, scale: Optional[torch.Tensor] = None):
        _dev(a, torch.bfloat16, "a")
        if a.dim() != 3:
            raise ValueError("a must be [adapters][rank][K]")
        self.num, self.rank, self.K = a.shape
        _dev(b, torch.bfloat16, "b")
        if b.dim() != 3 or b.shape[0] != self.num or b.shape[2] != self.rank:
            raise ValueError(f"b must be [{self.num}][N][{self.rank}], got {tuple(b.shape)}")
        if b.device != a.device:
            raise ValueError(f"b must be on {a.device}, got {b.device}")
        if scale is not None:
            _on(scale, torch.float32, "scale", (self.num,), a.device)
        self.N = b.shape[1]
        self.a, self.b, self.scale, self.device = a, b, scale, a.device

    @classmethod
    def of(cls, pairs, scale: Optional[torch.Tensor] = None) -> "Adapters":
        """From pairs of a [r][K] and b [N][r] bf16 of any ranks up to 128: smaller ones are filled up
        with zeros to the smallest rank the kernels take."""
        for a, b in pairs:
            if a.dim() != 2 or b.dim() != 2 or a.shape[0] != b.shape[1]:
                raise ValueError(f"a pair must be [r][K] and [N][r], got {tuple(a.shape)} and {tuple(b.shape)}")
        most = max(a.shape[0] for a, _ in pairs)
        if most > 128:
            raise ValueError(f"ranks are at most 128, got {most}")
        rank = next(r for r in (16, 32, 64, 128) if r >= most)
        pad = torch.nn.functional.pad
        return cls(torch.stack([pad(a, (0, 0, 0, rank - a.shape[0])) for a, _ in pairs]),
                   torch.stack([pad(b, (0, rank - b.shape[1])) for _, b in pairs]), scale)


def version() -> str:
    return load().tabit_version().decode()


def noalloc_scratch_bytes() -> int:
    return int(load().tabit_noalloc_scratch_bytes())


def act_workspace_bytes(M: int, K: int) -> int:
    return int(load().tabit_act_workspace_bytes(M, K))


def gemm_config_info(index: int = -1):
    """Number of INT8 GEMM configs (index < 0) or (bm, bn, k_groups) of one."""
    lib = load()
    if index < 0:
        return int(lib.tabit_gemm_config_info(-1, None, None, None))
    bm, bn, sk = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    st = lib.tabit_gemm_config_info(index, ctypes.byref(bm), ctypes.byref(bn), ctypes.byref(sk))
    if st != OK:
        raise TabitError(st, "bad config index")
    return bm.value, bn.value, sk.value


def mxfp4_config_info(index: int = -1):
    """Number of MXFP4 GEMM configs (index < 0) or (bm, bn) of one."""
    lib = load()
    if index < 0:
        return int(lib.tabit_mxfp4_config_info(-1, None, None))
    bm, bn = ctypes.c_int(), ctypes.c_int()
    st = lib.tabit_mxfp4_config_info(index, ctypes.byref(bm), ctypes.byref(bn))
    if st != OK:
        raise TabitError(st, "bad config index")
    return bm.value, bn.value


def hqdm_config_info(index: int = -1):
    """Number of HQ-DM GEMM configs (index < 0) or (bm, bn) of one."""
    lib = load()
    if index < 0:
        return int(lib.tabit_hqdm_config_info(-1, None, None))
    bm, bn = ctypes.c_int(), ctypes.c_int()
    st = lib.tabit_hqdm_config_info(index, ctypes.byref(bm), ctypes.byref(bn))
    if st != OK:
        raise TabitError(st, "bad config index")
    return bm.value, bn.value


def dmpq_workspace_bytes(M: int) -> int:
    return int(load().tabit_dmpq_workspace_bytes(M))


def weight_planes_bytes(N: int, K: int) -> int:
    return int(load().tabit_weight_planes_bytes(N, K))


def plane_config_info(index: int = -1):
    """Number of plane-major GEMM configs (index < 0) or (bm, bn, k_groups) of one."""
    lib = load()
    if index < 0:
        return int(lib.tabit_plane_config_info(-1, None, None, None))
    bm, bn, kg = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    st = lib.tabit_plane_config_info(index, ctypes.byref(bm), ctypes.byref(bn), ctypes.byref(kg))
    if st != OK:
        raise TabitError(st, "bad config index")
    return bm.value, bn.value, kg.value


def plane_config_choose(M: int, N: int, K: int, num_cus: int = 0) -> int:
    """Index of the plane-major GEMM configuration the library picks for M x N x K."""
    st = int(load().tabit_plane_config_choose(M, N, K, num_cus))
    if st < 0:
        raise TabitError(st, "bad shape")
    return st


def mxfp4_config_choose(M: int, N: int, K: int, num_cus: int = 0) -> int:
    """Index of the MXFP4 GEMM configuration the library picks for M x N x K."""
    st = int(load().tabit_mxfp4_config_choose(M, N, K, num_cus))
    if st < 0:
        raise TabitError(st, "bad shape")
    return st


def gemm_config_choose(M: int, N: int, K: int, num_cus: int = 0) -> int:
    return int(load().tabit_gemm_config_choose(M, N, K, num_cus))


class Context:
    """A tabit_ctx: schedule table, options and last error (host state only)."""

    def __init__(self):
        self._lib = load()
        h = ctypes.c_void_p()
        st = self._lib.tabit_create(ctypes.byref(h))
        if st != OK:
            raise TabitError(st, "tabit_create failed")
        self._h = h

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            self._lib.tabit_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self):
        return self._h

    def last_error(self) -> str:
        return self._lib.tabit_last_error(self._h).decode()

    def _check(self, st: int) -> None:
        if st != OK:
            raise TabitError(st, self.last_error())

    # ------------------------------------------------------------ options
    def set_option(self, option: int, value: int) -> None:
        self._check(self._lib.tabit_set_option(self._h, option, value))

    # ------------------------------------------------------------ schedule
    def set_step_schedule(self, k_bits, fmt=None) -> None:
        import numpy as np
        k = np.ascontiguousarray(k_bits, dtype=np.uint8)
        if k.ndim != 2:
            raise ValueError("k_bits must be [steps, layers]")
        f = None if fmt is None else np.ascontiguousarray(fmt, dtype=np.uint8)
        if f is not None and f.shape != k.shape:
            raise ValueError("fmt must match k_bits' shape")
        st = self._lib.tabit_set_step_schedule(self._h, k.shape[0], k.shape[1],
                                               k.ctypes.data, None if f is None else f.ctypes.data)
        self._check(st)

    def schedule_lookup(self, step: int, layer: int) -> Tuple[int, int]:
        k, f = ctypes.c_int(), ctypes.c_int()
        self._check(self._lib.tabit_schedule_lookup(self._h, step, layer, ctypes.byref(k), ctypes.byref(f)))
        return k.value, f.value

    # ------------------------------------------------------------ kernels
    def quantize_weights(self, w: torch.Tensor, had_block: int, int8: bool = True, mx: bool = False,
                         out=None):
        """bf16 [N, K] -> dict with w_q/w_scale (int8) and/or w_fp4/w_e8m0 (mx)."""
        N, K = w.shape
        _dev(w, torch.bfloat16, "w")
        out = dict(out or {})
        dev = w.device
        if int8:
            out.setdefault("w_q", torch.empty((N, K), dtype=torch.int8, device=dev))
            out.setdefault("w_scale", torch.empty((N,), dtype=torch.float32, device=dev))
            _dev(out["w_q"], torch.int8, "w_q", (N, K))
            _dev(out["w_scale"], torch.float32, "w_scale", (N,))
        if mx:
            out.setdefault("w_fp4", torch.empty((N, K // 2), dtype=torch.uint8, device=dev))
            out.setdefault("w_e8m0", torch.empty((N, K // 32), dtype=torch.uint8, device=dev))
            _dev(out["w_fp4"], torch.uint8, "w_fp4", (N, K // 2))
            _dev(out["w_e8m0"], torch.uint8, "w_e8m0", (N, K // 32))
        st = self._lib.tabit_quantize_weights(
            self._h, w.data_ptr(), N, K, had_block,
            _ptr(out.get("w_q")) if int8 else None, _ptr(out.get("w_scale")) if int8 else None,
            _ptr(out.get("w_fp4")) if mx else None, _ptr(out.get("w_e8m0")) if mx else None,
            _stream(dev))
        self._check(st)
        return out

    def hadamard_quant_act(self, x: torch.Tensor, had_block: int, fmt: int = FMT_INT8,
                           x_q: Optional[torch.Tensor] = None, x_scale: Optional[torch.Tensor] = None):
        """bf16 [M, K] -> (codes, scales): int8 [M, K] + fp32 [M], or fp4 [M, K/2] + e8m0 [M, K/32]."""
        _dev(x, torch.bfloat16, "x")
        M, K = x.shape
        dev = x.device
        if fmt == FMT_INT8:
            x_q = torch.empty((M, K), dtype=torch.int8, device=dev) if x_q is None else x_q
            x_scale = torch.empty((M,), dtype=torch.float32, device=dev) if x_scale is None else x_scale
            _dev(x_q, torch.int8, "x_q", (M, K))
            _dev(x_scale, torch.float32, "x_scale", (M,))
        else:
            x_q = torch.empty((M, K // 2), dtype=torch.uint8, device=dev) if x_q is None else x_q
            x_scale = torch.empty((M, K // 32), dtype=torch.uint8, device=dev) if x_scale is None else x_scale
            _dev(x_q, torch.uint8, "x_q", (M, K // 2))
            _dev(x_scale, torch.uint8, "x_scale", (M, K // 32))
        st = self._lib.tabit_hadamard_quant_act(self._h, x.data_ptr(), M, K, had_block, fmt,
                                                x_q.data_ptr(), x_scale.data_ptr(), _stream(dev))
        self._check(st)
        return x_q, x_scale

    def _gemm_i8(self, fn, x_q, x_scale, w_q, w_scale, k_bits, y=None, acc=None, want_y=True,
                 want_acc=False, planes=False):
        _dev(x_q, torch.int8, "x_q")
        M, K = x_q.shape
        if planes:
            _dev(w_q, torch.int32, "w_planes")
            if w_q.dim() != 4 or w_q.shape[0] != 8 or w_q.shape[1] != (K + 127) // 128 or w_q.shape[3] != 4:
                raise ValueError("w_planes must be [8][ceil(K/128)][N][4] words")
            N = w_q.shape[2]
        else:
            _dev(w_q, torch.int8, "w_q")
            N = w_q.shape[0]
            if w_q.shape[1] != K:
                raise ValueError("x_q and w_q disagree on K")
        _dev(x_scale, torch.float32, "x_scale", (M,))
        _dev(w_scale, torch.float32, "w_scale", (N,))
        dev = x_q.device
        if want_y and y is None:
            y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        if want_acc and acc is None:
            acc = torch.empty((M, N), dtype=torch.int32, device=dev)
        if y is not None:
            _dev(y, torch.bfloat16, "y", (M, N))
        if acc is not None:
            _dev(acc, torch.int32, "acc", (M, N))
        st = fn(self._h, x_q.data_ptr(), x_scale.data_ptr(), w_q.data_ptr(), w_scale.data_ptr(),
                M, N, K, k_bits, _ptr(y), _ptr(acc), _stream(dev))
        self._check(st)
        return y, acc

    def masked_qgemm(self, x_q, x_scale, w_q, w_scale, k_bits, y=None, acc=None, want_y=True,
                     want_acc=False):
        return self._gemm_i8(self._lib.tabit_masked_qgemm, x_q, x_scale, w_q, w_scale, k_bits, y,
                             acc, want_y, want_acc)

    def qgemm_bitserial(self, x_q, x_scale, w_q, w_scale, k_bits, y=None, acc=None, want_y=True,
                        want_acc=False):
        return self._gemm_i8(self._lib.tabit_qgemm_bitserial, x_q, x_scale, w_q, w_scale, k_bits, y,
                             acc, want_y, want_acc)

    def gelu_quant_act(self, x: torch.Tensor, had_block: int, x_q=None, x_scale=None,
                       fmt: int = FMT_INT8):
        """Down projection's input codes with the GELU folded in: int8 [M, K] + fp32 [M], or
        (fmt = FMT_MXFP4) fp4 [M, K/2] + e8m0 [M, K/32]."""
        _dev(x, torch.bfloat16, "x")
        M, K = x.shape
        dev = x.device
        if fmt == FMT_INT8:
            x_q = torch.empty((M, K), dtype=torch.int8, device=dev) if x_q is None else x_q
            x_scale = torch.empty((M,), dtype=torch.float32, device=dev) if x_scale is None else x_scale
            _dev(x_q, torch.int8, "x_q", (M, K))
            _dev(x_scale, torch.float32, "x_scale", (M,))
        else:
            x_q = torch.empty((M, K // 2), dtype=torch.uint8, device=dev) if x_q is None else x_q
            x_scale = torch.empty((M, K // 32), dtype=torch.uint8, device=dev) if x_scale is None else x_scale
            _dev(x_q, torch.uint8, "x_q", (M, K // 2))
            _dev(x_scale, torch.uint8, "x_scale", (M, K // 32))
        st = self._lib.tabit_gelu_quant_act(self._h, x.data_ptr(), M, K, had_block, fmt,
                                            x_q.data_ptr(), x_scale.data_ptr(), _stream(dev))
        self._check(st)
        return x_q, x_scale

    def hqdm_quant_act(self, x: torch.Tensor, had_block: int):
        """HQ-DM single-Hadamard codes: (x_hi int8 [M,K], x_lo int8 [M,K], x_scale fp32 [M])."""
        _dev(x, torch.bfloat16, "x")
        M, K = x.shape
        hi = torch.empty((M, K), dtype=torch.int8, device=x.device)
        lo = torch.empty((M, K), dtype=torch.int8, device=x.device)
        sc = torch.empty((M,), dtype=torch.float32, device=x.device)
        st = self._lib.tabit_hqdm_quant_act(self._h, x.data_ptr(), M, K, had_block, hi.data_ptr(),
                                            lo.data_ptr(), sc.data_ptr(), _stream(x.device))
        self._check(st)
        return hi, lo, sc

    def hqdm_qgemm(self, x_hi, x_lo, x_scale, w_q, w_scale, k_bits, y=None, want_y=True,
                   want_acc=False):
        """y bf16 [M,N] and/or the exact int64 accumulator of Z . W_k^T."""
        _dev(x_hi, torch.int8, "x_hi")
        M, K = x_hi.shape
        _dev(x_lo, torch.int8, "x_lo", (M, K))
        _dev(w_q, torch.int8, "w_q")
        N = w_q.shape[0]
        if w_q.shape[1] != K:
            raise ValueError("x and w_q disagree on K")
        _dev(x_scale, torch.float32, "x_scale", (M,))
        _dev(w_scale, torch.float32, "w_scale", (N,))
        if want_y and y is None:
            y = torch.empty((M, N), dtype=torch.bfloat16, device=x_hi.device)
        acc = torch.empty((M, N), dtype=torch.int64, device=x_hi.device) if want_acc else None
        st = self._lib.tabit_hqdm_qgemm(self._h, x_hi.data_ptr(), x_lo.data_ptr(), x_scale.data_ptr(),
                                        w_q.data_ptr(), w_scale.data_ptr(), M, N, K, k_bits, _ptr(y),
                                        _ptr(acc), _stream(x_hi.device))
        self._check(st)
        return y, acc

    def pack_weight_planes(self, w_q: torch.Tensor, out: Optional[torch.Tensor] = None):
        """Plane-major copy of int8 codes [N][K]: int32 tensor [8][ceil(K/128)][N][4] (uint32 words)."""
        _dev(w_q, torch.int8, "w_q")
        N, K = w_q.shape
        shape = (8, (K + 127) // 128, N, 4)
        if out is None:
            out = torch.empty(shape, dtype=torch.int32, device=w_q.device)
        _dev(out, torch.int32, "w_planes", shape)
        st = self._lib.tabit_pack_weight_planes(self._h, w_q.data_ptr(), N, K, out.data_ptr(),
                                                _stream(w_q.device))
        self._check(st)
        return out

    def plane_qgemm(self, x_q, x_scale, w_planes, w_scale, k_bits, y=None, acc=None, want_y=True,
                    want_acc=False):
        return self._gemm_i8(self._lib.tabit_plane_qgemm, x_q, x_scale, w_planes, w_scale, k_bits,
                             y, acc, want_y, want_acc, planes=True)

    def mxfp4_qgemm(self, x_fp4, x_e8m0, w_fp4, w_e8m0, out_scale: float, y=None, acc=None,
                    want_y=True, want_acc=False):
        for t, n in ((x_fp4, "x_fp4"), (x_e8m0, "x_e8m0"), (w_fp4, "w_fp4"), (w_e8m0, "w_e8m0")):
            _dev(t, torch.uint8, n)
        M, KB = x_fp4.shape
        N = w_fp4.shape[0]
        K = 2 * KB
        if w_fp4.shape[1] != KB or x_e8m0.shape != (M, K // 32) or w_e8m0.shape != (N, K // 32):
            raise ValueError("inconsistent MXFP4 operand shapes")
        dev = x_fp4.device
        if want_y and y is None:
            y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        if want_acc and acc is None:
            acc = torch.empty((M, N), dtype=torch.float32, device=dev)
        if y is not None:
            _dev(y, torch.bfloat16, "y", (M, N))
        if acc is not None:
            _dev(acc, torch.float32, "acc", (M, N))
        st = self._lib.tabit_mxfp4_qgemm(self._h, x_fp4.data_ptr(), x_e8m0.data_ptr(),
                                         w_fp4.data_ptr(), w_e8m0.data_ptr(), M, N, K,
                                         float(out_scale), _ptr(y), _ptr(acc), _stream(dev))
        self._check(st)
        return y, acc

    def scheduled_linear(self, step: int, layer: int, x: torch.Tensor, weights: dict,
                         had_block: int, act_ws: torch.Tensor, y: Optional[torch.Tensor] = None,
                         path: int = PATH_MASKED):
        """One linear at (step, layer): schedule lookup, quantize, GEMM -- all in the library."""
        _dev(x, torch.bfloat16, "x")
        M, K = x.shape
        wq = weights.get("w_planes") if path == PATH_PLANES else weights.get("w_q")
        wf = weights.get("w_fp4")
        if wq is not None:
            N = wq.shape[2] if path == PATH_PLANES else wq.shape[0]   # planes: [8][S][N][4]
        else:
            N = wf.shape[0]
        if y is None:
            y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
        _dev(y, torch.bfloat16, "y", (M, N))
        st = self._lib.tabit_scheduled_linear(
            self._h, step, layer, path, x.data_ptr(), M, N, K, had_block,
            _ptr(wq), _ptr(weights.get("w_scale")), _ptr(wf), _ptr(weights.get("w_e8m0")),
            act_ws.data_ptr(), act_ws.numel() * act_ws.element_size(), y.data_ptr(),
            _stream(x.device))
        self._check(st)
        return y

    def scheduled_linear_noalloc(self, step: int, layer: int, x: torch.Tensor, weights: dict,
                                 had_block: int, y: torch.Tensor, path: int = PATH_MASKED):
        """As scheduled_linear, with the library's static device scratch instead of a
        workspace; `y` [M, N] bf16 must be given (nothing is allocated here)."""
        _dev(x, torch.bfloat16, "x")
        M, K = x.shape
        N = y.shape[1]
        _dev(y, torch.bfloat16, "y", (M, N))
        wq = weights.get("w_planes") if path == PATH_PLANES else weights.get("w_q")
        st = self._lib.tabit_scheduled_linear_noalloc(
            self._h, step, layer, path, x.data_ptr(), M, N, K, had_block,
            _ptr(wq), _ptr(weights.get("w_scale")), _ptr(weights.get("w_fp4")),
            _ptr(weights.get("w_e8m0")), y.data_ptr(), _stream(x.device))
        self._check(st)
        return y

    def dmpq_select(self, x_in: torch.Tensor, x_out: torch.Tensor, theta: Optional[torch.Tensor],
                    fmt: Optional[torch.Tensor], gamma: Optional[torch.Tensor],
                    ws: Optional[torch.Tensor] = None):
        """Gamma of a block (device fp64) and fmt[l] = Gamma > theta[l] ? INT8 : MXFP4 (device)."""
        _dev(x_in, torch.bfloat16, "x_in")
        M, H = x_in.shape
        _dev(x_out, torch.bfloat16, "x_out", (M, H))
        n = 0
        if theta is not None:
            n = theta.numel()
            _dev(theta, torch.float32, "theta", (n,))
            _dev(fmt, torch.uint8, "fmt", (n,))
        if gamma is not None:
            _dev(gamma, torch.float64, "gamma", (1,))
        if ws is None:
            ws = torch.empty(dmpq_workspace_bytes(M), dtype=torch.uint8, device=x_in.device)
        st = self._lib.tabit_dmpq_select(self._h, x_in.data_ptr(), x_out.data_ptr(), M, H,
                                         _ptr(theta), n, _ptr(fmt), _ptr(gamma), ws.data_ptr(),
                                         ws.numel() * ws.element_size(), _stream(x_in.device))
        self._check(st)

    def gated_linear(self, fmt_dev: torch.Tensor, k_bits: int, x: torch.Tensor, weights: dict,
                     had_block: int, act_ws: torch.Tensor, y: Optional[torch.Tensor] = None,
                     path: int = PATH_MASKED):
        """One linear whose format is the device byte fmt_dev (both weight formats needed)."""
        _dev(x, torch.bfloat16, "x")
        M, K = x.shape
        wq = weights["w_planes"] if path == PATH_PLANES else weights["w_q"]
        N = wq.shape[2] if path == PATH_PLANES else wq.shape[0]
        if y is None:
            y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
        _dev(y, torch.bfloat16, "y", (M, N))
        st = self._lib.tabit_gated_linear(
            self._h, fmt_dev.data_ptr(), k_bits, path, x.data_ptr(), M, N, K, had_block,
            wq.data_ptr(), weights["w_scale"].data_ptr(), weights["w_fp4"].data_ptr(),
            weights["w_e8m0"].data_ptr(), act_ws.data_ptr(), act_ws.numel() * act_ws.element_size(),
            y.data_ptr(), _stream(x.device))
        self._check(st)
        return y

    def run_schedule(self, first_step: int, num_steps: int, layers, x_ptrs, had_block: int,
                     act_ws: torch.Tensor, path: int = PATH_MASKED, gemm_events=None,
                     stream: Optional[int] = None):
        """Native driver over steps [first_step, first_step+num_steps) x all layers.

        layers: a ctypes array of Layer; x_ptrs: a ctypes array of c_void_p of
        length num_steps * len(layers); gemm_events: None or a ctypes array of
        2 * num_steps * len(layers) hipEvent_t handles (c_void_p).
        """
        if stream is None:
            stream = _stream(act_ws.device)
        st = self._lib.tabit_run_schedule(
            self._h, first_step, num_steps, ctypes.cast(layers, ctypes.c_void_p), len(layers),
            ctypes.cast(x_ptrs, ctypes.c_void_p), had_block, path, act_ws.data_ptr(),
            act_ws.numel() * act_ws.element_size(),
            None if gemm_events is None else ctypes.cast(gemm_events, ctypes.c_void_p), stream)
        self._check(st)

    def mfma_peak_probe(self, kind: int = 0, iters: int = 20000, device="cuda:0") -> float:
        """Sustained matrix-core rate (ops or flops per second) of the device at its
        running clock: kind 0 INT8 MFMA, 1 FP4 scaled MFMA.  Synchronizes."""
        dev = torch.device(device)
        cus = torch.cuda.get_device_properties(dev).multi_processor_count
        n = int(self._lib.tabit_mfma_probe_sink_ints(cus))
        sink = torch.empty(n, dtype=torch.int32, device=dev)
        out = ctypes.c_double()
        st = self._lib.tabit_mfma_peak_probe(self._h, kind, iters, sink.data_ptr(), n,
                                             ctypes.byref(out), _stream(dev))
        self._check(st)
        return out.value

    def autotune_gemm(self, path: int, x_q, x_scale, w_q, w_scale, M: int, N: int, K: int,
                      k_bits: int, y: torch.Tensor, reps: int = 3) -> int:
        """Time every tile configuration for (path, M, N, K); the ctx keeps the fastest."""
        best = ctypes.c_int(-1)
        st = self._lib.tabit_autotune_gemm(self._h, path, x_q.data_ptr(), x_scale.data_ptr(),
                                           w_q.data_ptr(), w_scale.data_ptr(), M, N, K, k_bits,
                                           y.data_ptr(), reps, ctypes.byref(best), _stream(y.device))
        self._check(st)
        return best.value

    # ------------------------------------------------------------ between the linears
    def _rope(self, cache: KVCache, rope: Optional[Rope], positions, tokens: int):
        if rope is None:
            return None, None
        if rope.device != cache.device:
            raise ValueError(f"rope must be on {cache.device}, got {rope.device}")
        _on(positions, torch.int32, "positions", (tokens,), cache.device)
        return rope._ref, positions.data_ptr()

    def kv_append(self, cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                  rope: Optional[Rope] = None, positions: Optional[torch.Tensor] = None) -> None:
        """Rotate k to `positions`, quantize k and v, write them at `slots` (int64 [T]; negative:
        skipped).  k, v bf16 [T][kv_heads][head_dim], tokens of any stride of 8 elements."""
        ks = _rows(k, "k", cache._row, cache.device)
        vs = _rows(v, "v", cache._row, cache.device)
        n = k.shape[0]
        if v.shape[0] != n:
            raise ValueError("k and v disagree on the number of tokens")
        _on(slots, torch.int64, "slots", (n,), cache.device)
        r, pos = self._rope(cache, rope, positions, n)
        _counts(n)
        if n == 0:
            return
        self._check(self._lib.tabit_kv_append(self._h, cache._ref, k.data_ptr(), ks, v.data_ptr(), vs,
                                              n, slots.data_ptr(), r, pos, _stream(cache.device)))

    def kv_read(self, cache: KVCache, slots: torch.Tensor, k: Optional[torch.Tensor] = None,
                v: Optional[torch.Tensor] = None):
        """The keys and values held at `slots` as bf16 [T][kv_heads][head_dim] each."""
        n = slots.shape[0]
        _on(slots, torch.int64, "slots", (n,), cache.device)
        _counts(n)
        shape = (n,) + tuple(cache._row)
        k = torch.empty(shape, dtype=torch.bfloat16, device=cache.device) if k is None else k
        v = torch.empty(shape, dtype=torch.bfloat16, device=cache.device) if v is None else v
        _on(k, torch.bfloat16, "k", shape, cache.device)
        _on(v, torch.bfloat16, "v", shape, cache.device)
        if n:
            self._check(self._lib.tabit_kv_read(self._h, cache._ref, slots.data_ptr(), n, k.data_ptr(),
                                                v.data_ptr(), _stream(cache.device)))
        return k, v

    def kv_attention_workspace(self, cache: KVCache, q: torch.Tensor, num_seqs: int, max_q: int,
                               max_kv: int) -> Optional[torch.Tensor]:
        """A workspace for such calls (None where none is needed)."""
        _counts(q.shape[0], num_seqs, max_q, max_kv)
        n = int(self._lib.tabit_kv_attention_workspace_bytes(
            q.shape[0], q.shape[1], cache.num_kv_heads, cache.head_dim, num_seqs, max_q, max_kv))
        return torch.empty(n, dtype=torch.uint8, device=cache.device) if n else None

    def kv_attention(self, cache: KVCache, q: torch.Tensor, cu_q: torch.Tensor,
                     block_table: torch.Tensor, kv_lens: torch.Tensor, max_q: int, max_kv: int,
                     scale: Optional[float] = None, causal: bool = False,
                     rope: Optional[Rope] = None, positions: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                     ws: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Softmax attention of the ragged query rows q bf16 [T][q_heads][head_dim] over the cache.

        cu_q int32 [B+1] row bounds, block_table int32 [B][pages], kv_lens int32 [B]; max_q and
        max_kv bound the sequences' rows and keys.  scale defaults to head_dim ** -0.5.  Rows that
        no sequence covers are left unwritten in `out`; lse fp32 [T][q_heads] is filled if given.
        """
        dev = cache.device
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q must be [tokens][q_heads][head_dim]")
        T, hq = q.shape[0], q.shape[1]
        stride = _rows(q, "q", torch.Size((hq, cache.head_dim)), dev)
        B = kv_lens.shape[0]
        _counts(T, B, max_q, max_kv)
        _on(kv_lens, torch.int32, "kv_lens", (B,), dev)
        _on(cu_q, torch.int32, "cu_q", (B + 1,), dev)
        _on(block_table, torch.int32, "block_table", (B, block_table.shape[1]), dev)
        r, pos = self._rope(cache, rope, positions, T)
        if out is None:
            out = torch.empty((T, hq, cache.head_dim), dtype=torch.bfloat16, device=dev)
        else:
            _on(out, torch.bfloat16, "out", (T, hq, cache.head_dim), dev)
        if lse is not None:
            _on(lse, torch.float32, "lse", (T, hq), dev)
        if T == 0 or B == 0:
            return out
        if ws is None:
            ws = self.kv_attention_workspace(cache, q, B, max_q, max_kv)
        elif ws.device != dev or not ws.is_contiguous():
            raise ValueError(f"ws must be contiguous and on {dev}")
        a = _KvAttentionArgs(q.data_ptr(), stride, T, hq, cu_q.data_ptr(), B, max_q,
                             block_table.data_ptr(), block_table.shape[1], kv_lens.data_ptr(), max_kv,
                             cache.head_dim ** -0.5 if scale is None else scale, 1 if causal else 0,
                             r, pos, out.data_ptr(), _ptr(lse), _ptr(ws),
                             0 if ws is None else ws.numel() * ws.element_size())
        self._check(self._lib.tabit_kv_attention(self._h, cache._ref, ctypes.addressof(a),
                                                 _stream(dev)))
        return out

    def _launch(self, device: torch.device, fn, *args) -> None:
        """fn on the tensors' device, whichever is the current one, and on torch's stream of it."""
        if device.index == torch.cuda.current_device():
            self._check(fn(self._h, *args, _stream(device)))
        else:
            with torch.cuda.device(device):
                self._check(fn(self._h, *args, _stream(device)))

    def _rows_args(self, cache: KVCache, q, cu_q, block_table, kv_lens, max_q, max_kv, scale, causal,
                   rope, positions, out, lse, ws):
        """Checks and the argument structure of an attention-like call; ws given."""
        dev = cache.device
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q must be [tokens][q_heads][head_dim]")
        T, hq = q.shape[0], q.shape[1]
        stride = _rows(q, "q", torch.Size((hq, cache.head_dim)), dev)
        B = kv_lens.shape[0]
        _counts(T, B, max_q, max_kv)
        _on(kv_lens, torch.int32, "kv_lens", (B,), dev)
        _on(cu_q, torch.int32, "cu_q", (B + 1,), dev)
        _on(block_table, torch.int32, "block_table", (B, block_table.shape[1]), dev)
        r, pos = self._rope(cache, rope, positions, T)
        if lse is not None:
            _on(lse, torch.float32, "lse", (T, hq), dev)
        if ws is not None and (ws.device != dev or not ws.is_contiguous()):
            raise ValueError(f"ws must be contiguous and on {dev}")
        return _KvAttentionArgs(q.data_ptr(), stride, T, hq, cu_q.data_ptr(), B, max_q,
                                block_table.data_ptr(), block_table.shape[1], kv_lens.data_ptr(), max_kv,
                                cache.head_dim ** -0.5 if scale is None else scale, 1 if causal else 0,
                                r, pos, _ptr(out), _ptr(lse), _ptr(ws),
                                0 if ws is None else ws.numel() * ws.element_size())

    def _rows_workspace(self, fn, cache: KVCache, q, num_seqs, max_q, max_kv):
        _counts(q.shape[0], num_seqs, max_q, max_kv)
        n = int(fn(q.shape[0], q.shape[1], cache.num_kv_heads, cache.head_dim, num_seqs, max_q, max_kv))
        return torch.empty(n, dtype=torch.uint8, device=cache.device) if n else None

    # ------------------------------------------------------------ drafted trees
    def tree_mask(self, parents: torch.Tensor, cu_q: torch.Tensor, max_q: int):
        """Masks int64 [T][ceil(max_q / 64)] (bit j: the row sees node j of its sequence: itself and
        its ancestors) and depths int32 [T] of trees given by parents int32 [T]: the index of each
        row's parent among its sequence's rows (smaller than its own), -1 for none."""
        if not isinstance(parents, torch.Tensor) or parents.dim() != 1:
            raise ValueError("parents must be [tokens]")
        _dev(parents, torch.int32, "parents")
        T = parents.shape[0]
        _counts(T, max_q)
        _on(cu_q, torch.int32, "cu_q", (cu_q.shape[0],), parents.device)
        if cu_q.dim() != 1 or cu_q.shape[0] < 1:
            raise ValueError("cu_q must be [sequences + 1]")
        words = max((max_q + 63) // 64, 1)
        mask = torch.zeros((T, words), dtype=torch.int64, device=parents.device)
        depth = torch.zeros((T,), dtype=torch.int32, device=parents.device)
        if T:
            self._launch(parents.device, self._lib.tabit_tree_mask, parents.data_ptr(), T, cu_q.data_ptr(),
                         cu_q.shape[0] - 1, max_q, mask.data_ptr(), words, depth.data_ptr())
        return mask, depth

    def kv_tree_attention_workspace(self, cache: KVCache, q: torch.Tensor, num_seqs: int, max_q: int,
                                    max_kv: int) -> Optional[torch.Tensor]:
        """A workspace for such calls (None where none is needed)."""
        return self._rows_workspace(self._lib.tabit_kv_tree_attention_workspace_bytes, cache, q, num_seqs,
                                    max_q, max_kv)

    def kv_tree_attention(self, cache: KVCache, q: torch.Tensor, mask: torch.Tensor, cu_q: torch.Tensor,
                          block_table: torch.Tensor, kv_lens: torch.Tensor, max_q: int, max_kv: int,
                          scale: Optional[float] = None, rope: Optional[Rope] = None,
                          positions: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                          lse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Softmax attention of trees of drafted tokens: as kv_attention, but row i of a sequence's n
        sees the tokens before the last n, and of those the nodes that its row of mask (int64
        [T][words], bit j % 64 of word j / 64 for node j; see tree_mask) names."""
        dev = cache.device
        if out is None and isinstance(q, torch.Tensor):
            out = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
        B = kv_lens.shape[0]
        if ws is None and isinstance(q, torch.Tensor) and q.dim() == 3 and q.shape[0] and B:
            ws = self.kv_tree_attention_workspace(cache, q, B, max_q, max_kv)
        a = self._rows_args(cache, q, cu_q, block_table, kv_lens, max_q, max_kv, scale, False, rope, positions,
                            out, lse, ws)
        T = a.num_tokens
        _on(out, torch.bfloat16, "out", (T, q.shape[1], cache.head_dim), dev)
        if not isinstance(mask, torch.Tensor) or mask.dim() != 2:
            raise ValueError("mask must be [tokens][words]")
        _on(mask, torch.int64, "mask", (T, mask.shape[1]), dev)
        if T and B:
            self._launch(dev, self._lib.tabit_kv_tree_attention, cache._ref, ctypes.addressof(a), mask.data_ptr(),
                         mask.shape[1])
        return out

    # ------------------------------------------------------------ eviction
    def kv_sums(self, cache: KVCache) -> torch.Tensor:
        """Zeros for the accumulated attention weights of a cache's tokens, a number a key head."""
        return torch.zeros((cache.num_pages, cache.num_kv_heads, cache.page_size), dtype=torch.float32,
                           device=cache.device)

    def _sums(self, cache: KVCache, sums) -> None:
        _on(sums, torch.float32, "sums", (cache.num_pages, cache.num_kv_heads, cache.page_size), cache.device)

    def kv_weigh_workspace(self, cache: KVCache, q: torch.Tensor, num_seqs: int, max_q: int,
                           max_kv: int) -> Optional[torch.Tensor]:
        """A workspace for such calls."""
        return self._rows_workspace(self._lib.tabit_kv_weigh_workspace_bytes, cache, q, num_seqs, max_q, max_kv)

    def kv_weigh(self, cache: KVCache, sums: torch.Tensor, q: torch.Tensor, cu_q: torch.Tensor,
                 block_table: torch.Tensor, kv_lens: torch.Tensor, max_q: int, max_kv: int,
                 scale: Optional[float] = None, causal: bool = True, rope: Optional[Rope] = None,
                 positions: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                 ws: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Add to sums (fp32 [pages][kv_heads][page_size], see kv_sums) the attention weights that the
        rows q give to the cached tokens; with causal, the sums of a sequence's last n tokens (n
        its rows) are set instead.  Arguments as kv_attention; lse fp32 [T][q_heads] is filled if
        given.  Returns sums."""
        B = kv_lens.shape[0]
        if ws is None and isinstance(q, torch.Tensor) and q.dim() == 3 and q.shape[0] and B:
            ws = self.kv_weigh_workspace(cache, q, B, max_q, max_kv)
        a = self._rows_args(cache, q, cu_q, block_table, kv_lens, max_q, max_kv, scale, causal, rope, positions,
                            None, lse, ws)
        self._sums(cache, sums)
        if a.num_tokens and B:
            self._launch(cache.device, self._lib.tabit_kv_weigh, cache._ref, ctypes.addressof(a), sums.data_ptr())
        return sums

    def kv_evict_workspace(self, cache: KVCache, num_seqs: int, max_kv: int) -> Optional[torch.Tensor]:
        """A workspace for such kv_evict calls (None where none is needed)."""
        _counts(num_seqs, max_kv)
        n = int(self._lib.tabit_kv_evict_workspace_bytes(num_seqs, cache.num_kv_heads, max_kv))
        return torch.empty(n, dtype=torch.uint8, device=cache.device) if n else None

    def kv_evict(self, cache: KVCache, sums: torch.Tensor, block_table: torch.Tensor, kv_lens: torch.Tensor,
                 max_kv: int, budget: int, sinks: int = 0, recent: int = 0, ws: Optional[torch.Tensor] = None):
        """Which tokens each head keeps of sequences longer than budget: the first sinks, the last
        recent and the largest sums between.  Returns (keep int32 [B][kv_heads][budget], rising, -1
        behind the last; new lengths int32 [B]); kv_compact then moves them."""
        dev, B = cache.device, kv_lens.shape[0]
        _counts(B, max_kv, budget, sinks, recent)
        self._sums(cache, sums)
        _on(kv_lens, torch.int32, "kv_lens", (B,), dev)
        _on(block_table, torch.int32, "block_table", (B, block_table.shape[1]), dev)
        keep = torch.empty((B, cache.num_kv_heads, max(budget, 0)), dtype=torch.int32, device=dev)
        lens = torch.empty((B,), dtype=torch.int32, device=dev)
        if B:
            if ws is None:
                ws = self.kv_evict_workspace(cache, B, max_kv)
            elif ws.device != dev or not ws.is_contiguous():
                raise ValueError(f"ws must be contiguous and on {dev}")
            self._launch(dev, self._lib.tabit_kv_evict, cache._ref, sums.data_ptr(), block_table.data_ptr(),
                         block_table.shape[1], kv_lens.data_ptr(), B, max_kv, budget, sinks, recent, keep.data_ptr(),
                         lens.data_ptr(), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size())
        return keep, lens

    def kv_compact_workspace(self, cache: KVCache, num_seqs: int, most: int) -> Optional[torch.Tensor]:
        """A workspace for kv_compact calls of num_seqs lists of up to `most` tokens (None where none is
        needed)."""
        _counts(num_seqs, most)
        n = int(self._lib.tabit_kv_compact_workspace_bytes(num_seqs, cache.num_kv_heads, cache.head_dim, most))
        return torch.empty(n, dtype=torch.uint8, device=cache.device) if n else None

    def kv_compact(self, cache: KVCache, block_table: torch.Tensor, keep: torch.Tensor, counts: torch.Tensor,
                   starts: Optional[torch.Tensor] = None, sums: Optional[torch.Tensor] = None,
                   ws: Optional[torch.Tensor] = None) -> None:
        """Move tokens inside their sequences: token starts[b] + j becomes what token keep[b][h][j] was,
        j < counts[b], with its sum where sums are given.  keep int32 [B][kv_heads or 1][most], each
        list rising and none before its place; counts, starts (None: 0) int32 [B]."""
        dev = cache.device
        if not isinstance(keep, torch.Tensor) or keep.dim() != 3:
            raise ValueError("keep must be [sequences][kv_heads or 1][tokens]")
        B, heads, most = keep.shape
        _counts(B, most)
        _on(keep, torch.int32, "keep", (B, heads, most), dev)
        _on(counts, torch.int32, "counts", (B,), dev)
        _on(block_table, torch.int32, "block_table", (B, block_table.shape[1]), dev)
        if starts is not None:
            _on(starts, torch.int32, "starts", (B,), dev)
        if sums is not None:
            self._sums(cache, sums)
        if B == 0 or most == 0:
            return
        if ws is None:
            ws = self.kv_compact_workspace(cache, B, most)
        elif ws.device != dev or not ws.is_contiguous():
            raise ValueError(f"ws must be contiguous and on {dev}")
        self._launch(dev, self._lib.tabit_kv_compact, cache._ref, block_table.data_ptr(), block_table.shape[1], B,
                     keep.data_ptr(), heads, most, counts.data_ptr(), _ptr(starts), _ptr(sums), _ptr(ws),
                     0 if ws is None else ws.numel() * ws.element_size())

    # ------------------------------------------------------------ adapters
    def adapter_rotate(self, a: torch.Tensor, had_block: int, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """A matrices bf16 [..][K] of adapters, transformed for rows that are quantized after a block
        Hadamard transform: (1 / b) A H, rounded to bf16."""
        _dev(a, torch.bfloat16, "a")
        if a.dim() < 1:
            raise ValueError("a must be [..][K]")
        out = torch.empty_like(a) if out is None else out
        _on(out, torch.bfloat16, "out", a.shape, a.device)
        rows = a.numel() // a.shape[-1] if a.numel() else 0
        _counts(rows, a.shape[-1])
        if rows:
            self._launch(a.device, self._lib.tabit_adapter_rotate, a.data_ptr(), rows, a.shape[-1], had_block,
                         out.data_ptr())
        return out

    def adapter_workspace(self, adapters: Adapters, x: torch.Tensor, num_segments: int) -> Optional[torch.Tensor]:
        """A workspace for adapter_linear calls of as many rows."""
        _counts(x.shape[0], num_segments)
        n = int(self._lib.tabit_adapter_workspace_bytes(x.shape[0], adapters.rank, num_segments))
        return torch.empty(n, dtype=torch.uint8, device=adapters.device) if n else None

    def adapter_linear(self, adapters: Adapters, x: torch.Tensor, y: torch.Tensor, cu_rows: torch.Tensor,
                       which: torch.Tensor, x_scale: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
        """out = y + scale (x A^T) B^T, with the adapter which[i] of the rows [cu_rows[i], cu_rows[i+1]).

        x bf16 [T][K] (rows of any stride of 8 elements), int8 [T][K] with x_scale fp32 [T], or packed
        uint8 [T][K/2] with x_scale E8M0 uint8 [T][K/32]: what the projection reads.  y bf16
        [T][N], the projection's output; out may be y.  cu_rows int32 [S+1], which int32 [S] (outside
        the adapters: out = y).  Rows of no segment are left unwritten in out.
        """
        dev, K, N = adapters.device, adapters.K, adapters.N
        if not isinstance(x, torch.Tensor) or x.dim() != 2:
            raise ValueError("x must be [rows][features]")
        T, xs = x.shape[0], K
        if x.dtype == torch.bfloat16:
            fmt, xs = FMT_BF16, _matrix(x, "x", K, dev)
            if x_scale is not None:
                raise ValueError("bf16 rows have no scales")
        elif x.dtype == torch.int8:
            fmt = FMT_INT8
            _on(x, torch.int8, "x", (T, K), dev)
            _on(x_scale, torch.float32, "x_scale", (T,), dev)
        else:
            fmt = FMT_MXFP4
            _on(x, torch.uint8, "x", (T, K // 2), dev)
            _on(x_scale, torch.uint8, "x_scale", (T, K // 32), dev)
        ys = _matrix(y, "y", N, dev)
        if y.shape[0] != T:
            raise ValueError("x and y disagree on the number of rows")
        if out is None:
            out = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
        os_ = _matrix(out, "out", N, dev)
        if out.shape[0] != T:
            raise ValueError("x and out disagree on the number of rows")
        S = which.shape[0]
        _counts(T, S, K, N)
        _on(which, torch.int32, "which", (S,), dev)
        _on(cu_rows, torch.int32, "cu_rows", (S + 1,), dev)
        if T == 0 or S == 0:
            return out
        if ws is None:
            ws = self.adapter_workspace(adapters, x, S)
        elif ws.device != dev or not ws.is_contiguous():
            raise ValueError(f"ws must be contiguous and on {dev}")
        a = _AdapterArgs(x.data_ptr(), _ptr(x_scale), fmt, T, K, N, xs, adapters.a.data_ptr(),
                         adapters.b.data_ptr(), _ptr(adapters.scale), adapters.num, adapters.rank,
                         cu_rows.data_ptr(), which.data_ptr(), S, y.data_ptr(), ys, out.data_ptr(), os_,
                         _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size())
        self._launch(dev, self._lib.tabit_adapter_linear, ctypes.addressof(a))
        return out

    def block_norm(self, x: torch.Tensor, y: Optional[torch.Tensor] = None, post: int = NORM_NONE,
                   post_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                   res_scale: float = 1.0, pre: int = NORM_NONE,
                   pre_weight: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                   shift: Optional[torch.Tensor] = None, eps: float = 1e-6, fmt: int = FMT_BF16,
                   had_block: int = 0, want_x: bool = True, want_h: bool = True,
                   x_out: Optional[torch.Tensor] = None):
        """x' = res_scale x + gate N_post(y); h = N_pre(x') (1 + scale) + shift.

        x, y bf16 [M][H]; weights bf16 [H]; gate, scale, shift bf16 [samples][H] with one row
        stride for all three (slices of one conditioning output), M a multiple of samples.
        Returns (x', h, h_scale): h bf16, or int8 with fp32 [M] scales (FMT_INT8), or packed
        uint8 [M][H/2] with E8M0 uint8 [M][H/32] (FMT_MXFP4); None for what is not wanted.
        """
        _dev(x, torch.bfloat16, "x")
        if x.dim() != 2:
            raise ValueError("x must be [M][H]")
        M, H = x.shape
        dev = x.device
        _counts(M, H)
        if y is not None:
            _on(y, torch.bfloat16, "y", (M, H), dev)
        for w, name in ((post_weight, "post_weight"), (pre_weight, "pre_weight")):
            if w is not None:
                _on(w, torch.bfloat16, name, (H,), dev)
        samples, stride = 0, 0
        for t, name in ((gate, "gate"), (scale, "scale"), (shift, "shift")):
            if t is None:
                continue
            if t.dtype != torch.bfloat16:
                raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
            if t.device != dev or t.dim() != 2 or t.shape[1] != H or t.stride(1) != 1:
                raise ValueError(f"{name} must be [samples][{H}] on {dev}, its rows contiguous")
            s = t.stride(0) if t.shape[0] > 1 else H
            if samples and (t.shape[0] != samples or s != stride):
                raise ValueError("gate, scale and shift must have the same rows and row stride")
            samples, stride = t.shape[0], s
        if samples and M % samples != 0:
            raise ValueError(f"{M} rows are not a multiple of {samples} samples")
        if not samples and (gate is not None or scale is not None or shift is not None) and M:
            raise ValueError("gate, scale and shift must have a row")
        if x_out is not None:
            _on(x_out, torch.bfloat16, "x_out", (M, H), dev)
        elif want_x:
            x_out = torch.empty_like(x)
        h = hs = None
        if want_h:
            if fmt == FMT_INT8:
                h = torch.empty_like(x, dtype=torch.int8)
                hs = torch.empty((M,), dtype=torch.float32, device=dev)
            elif fmt == FMT_MXFP4:
                h = torch.empty((M, H // 2), dtype=torch.uint8, device=dev)
                hs = torch.empty((M, H // 32), dtype=torch.uint8, device=dev)
            else:
                h = torch.empty_like(x)
        if M == 0:
            return x_out, h, hs
        a = _BlockNormArgs(x.data_ptr(), _ptr(y), M, H, post, pre, _ptr(post_weight), _ptr(pre_weight),
                           _ptr(gate), _ptr(scale), _ptr(shift), stride, samples,
                           M // samples if samples else 0, res_scale, eps, _ptr(x_out), _ptr(h),
                           _ptr(hs), fmt, had_block)
        self._check(self._lib.tabit_block_norm(self._h, ctypes.addressof(a), _stream(dev)))
        return x_out, h, hs
