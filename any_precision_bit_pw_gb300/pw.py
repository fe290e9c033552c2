"""Thin Python binding of libpw's C ABI (include/pw.h): same names, argument
marshalling only.  Every step of the path runs in libpw's CUDA kernels; there
is no Python or CPU fallback.  Tensors are torch tensors (device memory);
``stream`` defaults to torch's current CUDA stream.

Importing this module loads ``libpw.so`` from the package directory and fails
loudly if it is missing (build it with ``python -m any_precision_bit_pw_gb300.build``).
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional, Sequence

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libpw.so")

PW_OK = 0
PW_ERR_INVALID_ARG = -1
PW_ERR_UNSUPPORTED = -2
PW_ERR_NOT_RESIDENT = -3
PW_ERR_CUDA = -4
PW_ERR_TIMEOUT = -5
PW_ERR_WORKSPACE = -6
PW_ERR_BUSY = -7
PW_PAGE_GPU, PW_PAGE_CPU, PW_PAGE_TO_CPU, PW_PAGE_TO_GPU = 1, 2, 4, 8


def PW_PAGE_LUT(b: int) -> int:
    return 8 + b

PW_LAYOUT_TILED = 1
PW_MAX_BITS = 8
PW_PATH_AUTO, PW_PATH_DECODE, PW_PATH_PREFILL = 0, 1, 2
PW_KERNEL_AUTO, PW_KERNEL_TENSOR, PW_KERNEL_CUDA_CORES = 0, 1, 2
PW_FFN_FLAG_TEST_DROP_ONE_ARRIVAL = 1
PW_FFN_FLAG_STRIP_COMBINE = 2
PW_DTYPE_F16, PW_DTYPE_BF16, PW_DTYPE_F32 = 0, 1, 2
PW_ACT_SILU, PW_ACT_GELU_TANH = 0, 1
PW_ROPE_PLAIN, PW_ROPE_LINEAR, PW_ROPE_NTK, PW_ROPE_YARN, PW_ROPE_BANDS = 0, 1, 2, 3, 4

ERR_NAMES = {0: "PW_OK", -1: "PW_ERR_INVALID_ARG", -2: "PW_ERR_UNSUPPORTED", -3: "PW_ERR_NOT_RESIDENT",
             -4: "PW_ERR_CUDA", -5: "PW_ERR_TIMEOUT", -6: "PW_ERR_WORKSPACE", -7: "PW_ERR_BUSY"}

EXPORTS = (
    "pw_last_error", "pw_plane_bytes", "pw_pack_bitplanes", "pw_pack_lut", "pw_desc_bytes", "pw_page_table_create",
    "pw_page_table_destroy", "pw_page_table_attach_plane", "pw_page_table_attach_lut",
    "pw_page_table_set_desired", "pw_page_table_set_bits", "pw_page_table_get", "pw_page_table_bytes",
    "pw_page_table_resident_bytes", "pw_page_table_sync", "pw_moe_route_topk", "pw_moe_route_topk_shared",
    "pw_page_bytes", "pw_page_offload", "pw_page_reload", "pw_page_table_poll", "pw_page_table_take_released",
    "pw_page_state",
    "pw_moe_apl_ffn_workspace", "pw_moe_apl_ffn", "pw_moe_apl_ffn_ex", "pw_moe_apl_ffn_noalloc",
    "pw_moe_route_apl_ffn", "pw_moe_route_apl_ffn_ex", "pw_moe_route_apl_ffn_layers",
    "pw_add_rmsnorm", "pw_quantize_fp8", "pw_fp8_linear", "pw_rope_turns", "pw_rope_append",
    "pw_paged_attention_workspace", "pw_paged_attention", "pw_paged_attention_ex",
    "pw_norm_add_norm", "pw_fp8_gated_linear", "pw_token_logprobs",
    "pw_unpack_indices",
    "pw_apl_linear",
)


class PwError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{ERR_NAMES.get(code, code)}: {msg}")
        self.code = code


class pw_block_info(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("parent_bits", ctypes.c_int32),
                ("seed_bits", ctypes.c_int32), ("layout", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class pw_ffn_options(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int32), ("flags", ctypes.c_uint32), ("wait_timeout_us", ctypes.c_uint32),
                ("shared_experts", ctypes.c_int32), ("kernel", ctypes.c_int32), ("reserved", ctypes.c_int32 * 3)]


class pw_rope_scaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("reserved", ctypes.c_int32), ("scale", ctypes.c_double),
                ("original_positions", ctypes.c_double), ("fast", ctypes.c_double), ("slow", ctypes.c_double)]


class pw_norm_args(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("x", "residual", "weight", "residual_out", "y", "q", "scale")]
                + [(n, ctypes.c_int64) for n in ("x_stride", "residual_stride", "residual_out_stride", "y_stride",
                                                 "q_stride", "scale_stride", "rows")]
                + [("cols", ctypes.c_int32), ("dtype", ctypes.c_int32), ("eps", ctypes.c_float),
                   ("reserved", ctypes.c_int32)])


class pw_quant_args(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("x", "q", "scale")]
                + [(n, ctypes.c_int64) for n in ("x_stride", "q_stride", "scale_stride", "rows")]
                + [(n, ctypes.c_int32) for n in ("cols", "dtype", "block_rows", "reserved")])


class pw_linear_args(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("a", "a_scale", "b", "b_scale", "y", "status")]
                + [(n, ctypes.c_int64) for n in ("lda", "a_scale_stride", "ldb", "b_scale_stride", "ldy")]
                + [(n, ctypes.c_int32) for n in ("m", "n", "k", "dtype")])


class pw_rope_args(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q", "q_out", "k", "v", "k_cache", "v_cache", "turns", "positions",
                                                "page_table", "q_offsets", "kv_lens", "status")]
                + [(n, ctypes.c_int64) for n in (
                    "q_stride_token", "q_stride_head", "q_out_stride_token", "q_out_stride_head", "k_stride_token",
                    "k_stride_head", "v_stride_token", "v_stride_head", "k_cache_stride_page", "k_cache_stride_token",
                    "k_cache_stride_head", "v_cache_stride_page", "v_cache_stride_token", "v_cache_stride_head",
                    "page_table_stride")]
                + [(n, ctypes.c_int32) for n in ("tokens", "batch", "heads", "kv_heads", "head_dim", "rotary_dim",
                                                 "page_size", "num_pages", "pages_per_seq", "dtype", "interleaved")]
                + [("factor", ctypes.c_float)])


class pw_attn_args(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q", "out", "lse", "k_cache", "v_cache", "page_table", "q_offsets",
                                                "kv_lens", "status")]
                + [(n, ctypes.c_int64) for n in (
                    "q_stride_token", "q_stride_head", "out_stride_token", "out_stride_head", "k_stride_page",
                    "k_stride_token", "k_stride_head", "v_stride_page", "v_stride_token", "v_stride_head",
                    "page_table_stride")]
                + [(n, ctypes.c_int32) for n in ("tokens", "batch", "heads", "kv_heads", "head_dim", "page_size",
                                                 "num_pages", "pages_per_seq", "max_q_len", "max_kv_len", "dtype",
                                                 "causal", "window")]
                + [("scale", ctypes.c_float)])


class pw_attn_options(ctypes.Structure):
    _fields_ = [("sinks", ctypes.c_int32), ("reserved", ctypes.c_int32 * 7)]


class pw_norms_args(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("x", "residual", "post_weight", "gate", "weight", "residual_out", "y", "q",
                                                "scale")]
                + [(n, ctypes.c_int64) for n in ("x_stride", "residual_stride", "gate_stride", "residual_out_stride",
                                                 "y_stride", "q_stride", "scale_stride", "rows")]
                + [(n, ctypes.c_int32) for n in ("cols", "dtype")]
                + [(n, ctypes.c_float) for n in ("eps", "residual_scale", "block_scale")] + [("reserved", ctypes.c_int32)])


class pw_gated_args(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("a", "a_scale", "gate", "gate_scale", "up", "up_scale", "y", "q", "scale",
                                                "status")]
                + [(n, ctypes.c_int64) for n in ("lda", "a_scale_stride", "ld_gate", "gate_scale_stride", "ld_up",
                                                 "up_scale_stride", "ldy", "ldq", "scale_stride")]
                + [(n, ctypes.c_int32) for n in ("m", "n", "k", "dtype", "activation", "reserved")])


class pw_logprob_args(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("logits", "targets", "logprobs", "lse", "entropy", "top_ids",
                                                "top_logprobs")]
                + [(n, ctypes.c_int64) for n in ("stride", "targets_stride", "logprobs_stride", "top_ids_stride",
                                                 "top_logprobs_stride", "rows")]
                + [(n, ctypes.c_int32) for n in ("vocab", "given", "top", "dtype")]
                + [("scale", ctypes.c_float), ("reserved", ctypes.c_int32)])


_lib: Optional[ctypes.CDLL] = None
P, I32, I64, U64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint64, ctypes.c_size_t
F32, F64 = ctypes.c_float, ctypes.c_double


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libpw.so not built at {LIB_PATH}; run python -m any_precision_bit_pw_gb300.build")
        L = ctypes.CDLL(LIB_PATH)
        sig = {
            "pw_last_error": (ctypes.c_char_p, []),
            "pw_plane_bytes": (SZ, [I64, I64, I32]),
            "pw_pack_bitplanes": (I32, [P, I64, I64, I32, ctypes.POINTER(P), I32, P]),
            "pw_pack_lut": (I32, [P, I64, I32, P, P]),
            "pw_desc_bytes": (SZ, [I32]),
            "pw_page_table_create": (I32, [ctypes.POINTER(P), I32, ctypes.POINTER(pw_block_info)]),
            "pw_page_table_destroy": (I32, [P]),
            "pw_page_table_attach_plane": (I32, [P, I32, I32, P]),
            "pw_page_table_attach_lut": (I32, [P, I32, I32, P]),
            "pw_page_table_set_desired": (I32, [P, I32, I32]),
            "pw_page_table_set_bits": (I32, [P, I32, I32, ctypes.POINTER(U64)]),
            "pw_page_table_get": (I32, [P, I32, ctypes.POINTER(I32), ctypes.POINTER(I32), ctypes.POINTER(U64)]),
            "pw_page_table_bytes": (I64, [P, I32, I32]),
            "pw_page_table_resident_bytes": (I64, [P]),
            "pw_page_table_sync": (I32, [P, P, SZ, P]),
            "pw_page_bytes": (I64, [P, I32, I32]),
            "pw_page_offload": (I32, [P, I32, I32, P, P]),
            "pw_page_reload": (I32, [P, I32, I32, P, P, P]),
            "pw_page_table_poll": (I32, [P, ctypes.POINTER(I32)]),
            "pw_page_table_take_released": (I32, [P, I32, ctypes.POINTER(U64)]),
            "pw_page_state": (I32, [P, I32, I32, ctypes.POINTER(I32), ctypes.POINTER(P), ctypes.POINTER(P)]),
            "pw_moe_route_topk": (I32, [P, I32, I32, I32, P, P, P, P, P, P, P]),
            "pw_moe_route_topk_shared": (I32, [P, I32, I32, I32, I32, P, P, P, P, P, P, P]),
            "pw_moe_apl_ffn_workspace": (SZ, [I32, I32, I32, I32, I32]),
            "pw_moe_apl_ffn": (I32, [P, I32, P, I32, I32, I32, I32, I32, P, P, P, P, P, P, SZ, P, P, P]),
            "pw_moe_apl_ffn_ex": (I32, [P, I32, P, I32, I32, I32, I32, I32, P, P, P, P, P, P, SZ, P, P,
                                        ctypes.POINTER(pw_ffn_options), P]),
            "pw_moe_apl_ffn_noalloc": (I32, [P, I32, P, I32, I32, I32, I32, I32, P, P, P, P, P, P, P, P]),
            "pw_moe_route_apl_ffn": (I32, [P, I32, P, P, I32, I32, I32, I32, I32, P, P, P, P, P, P, P, SZ, P, P,
                                           P]),
            "pw_moe_route_apl_ffn_ex": (I32, [P, I32, P, P, I32, I32, I32, I32, I32, P, P, P, P, P, P, P, SZ, P,
                                              P, ctypes.POINTER(pw_ffn_options), P]),
            "pw_moe_route_apl_ffn_layers": (I32, [P, I32, I32, P, P, I32, I32, I32, I32, I32, P, P, P, P, P, P, P,
                                                  SZ, P, P, ctypes.POINTER(pw_ffn_options), P]),
            "pw_add_rmsnorm": (I32, [P, P]),
            "pw_quantize_fp8": (I32, [P, P]),
            "pw_fp8_linear": (I32, [P, P]),
            "pw_rope_turns": (I32, [I32, F64, ctypes.POINTER(pw_rope_scaling), P, ctypes.POINTER(F32)]),
            "pw_rope_append": (I32, [P, P]),
            "pw_paged_attention_workspace": (SZ, [I32, I32, I32, I32, I32]),
            "pw_paged_attention": (I32, [P, P, SZ, P]),
            "pw_paged_attention_ex": (I32, [P, P, P, SZ, P]),
            "pw_norm_add_norm": (I32, [P, P]),
            "pw_fp8_gated_linear": (I32, [P, P]),
            "pw_token_logprobs": (I32, [P, P]),
            "pw_unpack_indices": (I32, [P, I32, I32, P, P]),
            "pw_apl_linear": (I32, [P, I32, P, I32, P, P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(rc: int) -> int:
    if rc != PW_OK:
        raise PwError(rc, pw_last_error())
    return rc


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    if stream is None:   # the raw handle: a Stream object per call costs as much as a small kernel
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dev(t: torch.Tensor, dtype, name: str) -> None:
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name}: need a contiguous CUDA tensor of {dtype}, got {t.dtype} on {t.device}")


# ---------------------------------------------------------------------------
def pw_last_error() -> str:
    return lib().pw_last_error().decode(errors="replace")


def pw_plane_bytes(rows: int, cols: int, layout: int = PW_LAYOUT_TILED) -> int:
    return int(lib().pw_plane_bytes(rows, cols, layout))


def pw_pack_bitplanes(idx: torch.Tensor, parent_bits: int, planes: Sequence[torch.Tensor],
                      layout: int = PW_LAYOUT_TILED, stream=None) -> None:
    _dev(idx, torch.uint8, "idx")
    if len(planes) != parent_bits:
        raise ValueError("need one plane buffer per parent bit")
    arr = (P * parent_bits)(*[p.data_ptr() for p in planes])
    _check(lib().pw_pack_bitplanes(_ptr(idx), idx.shape[0], idx.shape[1], parent_bits, arr, layout,
                                   _stream(stream)))


def pw_pack_lut(lut: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """fp16 [rows][2^b] row-major LUT -> `out` (same size) in the tiled LUT layout."""
    _dev(lut, torch.float16, "lut")
    rows, C = lut.shape
    bits = C.bit_length() - 1
    if C != 1 << bits or not out.is_cuda or out.numel() * out.element_size() < rows * C * 2:
        raise ValueError("pack_lut: need lut [rows][2^b] and an output of the same size")
    _check(lib().pw_pack_lut(_ptr(lut), rows, bits, _ptr(out), _stream(stream)))


def pw_desc_bytes(n_blocks: int) -> int:
    return int(lib().pw_desc_bytes(n_blocks))


def pw_page_table_create(infos: Sequence[pw_block_info]) -> ctypes.c_void_p:
    arr = (pw_block_info * len(infos))(*infos)
    h = ctypes.c_void_p()
    _check(lib().pw_page_table_create(ctypes.byref(h), len(infos), arr))
    return h


def pw_page_table_destroy(t) -> None:
    _check(lib().pw_page_table_destroy(t))


def pw_page_table_attach_plane(t, block: int, plane: int, d_plane_ptr: int) -> None:
    _check(lib().pw_page_table_attach_plane(t, block, plane, ctypes.c_void_p(d_plane_ptr)))


def pw_page_table_attach_lut(t, block: int, bits: int, d_lut_ptr: int) -> None:
    _check(lib().pw_page_table_attach_lut(t, block, bits, ctypes.c_void_p(d_lut_ptr)))


def pw_page_table_set_desired(t, block: int, d: int) -> None:
    _check(lib().pw_page_table_set_desired(t, block, d))


def pw_page_table_set_bits(t, block: int, q: int) -> int:
    """Returns the released-page mask (bit p: plane p; bit 8+b: LUT b)."""
    m = U64(0)
    _check(lib().pw_page_table_set_bits(t, block, q, ctypes.byref(m)))
    return int(m.value)


def pw_page_table_get(t, block: int):
    q, d, m = I32(0), I32(0), U64(0)
    _check(lib().pw_page_table_get(t, block, ctypes.byref(q), ctypes.byref(d), ctypes.byref(m)))
    return int(q.value), int(d.value), int(m.value)


def pw_page_table_bytes(t, block: int, b: int) -> int:
    return int(lib().pw_page_table_bytes(t, block, b))


def pw_page_table_resident_bytes(t) -> int:
    return int(lib().pw_page_table_resident_bytes(t))


def pw_page_table_sync(t, d_desc: torch.Tensor, stream=None) -> None:
    _check(lib().pw_page_table_sync(t, _ptr(d_desc), d_desc.numel() * d_desc.element_size(), _stream(stream)))


def pw_page_bytes(t, block: int, page: int) -> int:
    return int(lib().pw_page_bytes(t, block, page))


def pw_page_offload(t, block: int, page: int, host: torch.Tensor, stream=None) -> None:
    """Start copying a GPU-resident page into `host` (pinned, >= pw_page_bytes bytes)."""
    if host.is_cuda or host.numel() * host.element_size() < pw_page_bytes(t, block, page):
        raise ValueError("offload: need a host tensor of at least the page's bytes")
    _check(lib().pw_page_offload(t, block, page, _ptr(host), _stream(stream)))


def pw_page_reload(t, block: int, page: int, host: Optional[torch.Tensor], dev: torch.Tensor, stream=None) -> None:
    """Start copying a page from `host` (None: the page's own host copy) into `dev`."""
    if not dev.is_cuda or dev.numel() * dev.element_size() < pw_page_bytes(t, block, page):
        raise ValueError("reload: need a device tensor of at least the page's bytes")
    _check(lib().pw_page_reload(t, block, page, _ptr(host), _ptr(dev), _stream(stream)))


def pw_page_table_poll(t) -> int:
    """Advance finished transfers; returns the number still in flight."""
    n = I32(0)
    _check(lib().pw_page_table_poll(t, ctypes.byref(n)))
    return int(n.value)


def pw_page_table_take_released(t, block: int) -> int:
    m = U64(0)
    _check(lib().pw_page_table_take_released(t, block, ctypes.byref(m)))
    return int(m.value)


def pw_page_state(t, block: int, page: int):
    """(state bits, attached device address or 0, host address or 0)."""
    st, d, h = I32(0), P(), P()
    _check(lib().pw_page_state(t, block, page, ctypes.byref(st), ctypes.byref(d), ctypes.byref(h)))
    return int(st.value), int(d.value or 0), int(h.value or 0)


def pw_moe_route_topk(logits: torch.Tensor, k: int, ids: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor,
                      perm: torch.Tensor, inv_perm: torch.Tensor, mass_accum: Optional[torch.Tensor] = None,
                      stream=None) -> None:
    _dev(logits, torch.float32, "logits")
    T, E = logits.shape
    _check(lib().pw_moe_route_topk(_ptr(logits), T, E, k, _ptr(ids), _ptr(w), _ptr(offsets), _ptr(perm),
                                   _ptr(inv_perm), _ptr(mass_accum), _stream(stream)))


def pw_moe_route_topk_shared(logits: torch.Tensor, k: int, shared: int, ids: torch.Tensor, w: torch.Tensor,
                             offsets: torch.Tensor, perm: torch.Tensor, inv_perm: torch.Tensor,
                             mass_accum: Optional[torch.Tensor] = None, stream=None) -> None:
    """Top-k routing plus `shared` always-on experts (ids E..E+S-1, weight 1)."""
    _dev(logits, torch.float32, "logits")
    T, E = logits.shape
    _check(lib().pw_moe_route_topk_shared(_ptr(logits), T, E, k, shared, _ptr(ids), _ptr(w), _ptr(offsets),
                                          _ptr(perm), _ptr(inv_perm), _ptr(mass_accum), _stream(stream)))


def pw_moe_apl_ffn_workspace(T: int, H: int, I: int, E: int, k: int) -> int:
    return int(lib().pw_moe_apl_ffn_workspace(T, H, I, E, k))


def pw_moe_apl_ffn(d_desc: torch.Tensor, layer: int, x: torch.Tensor, I: int, E: int, k: int,
                   ids: Optional[torch.Tensor], w: torch.Tensor, offsets: torch.Tensor, perm: torch.Tensor,
                   inv_perm: torch.Tensor, ws: torch.Tensor, y: torch.Tensor, status: torch.Tensor,
                   options: Optional[pw_ffn_options] = None, stream=None) -> None:
    _dev(x, torch.float16, "x")
    _dev(y, torch.float16, "y")
    T, H = x.shape
    args = (_ptr(d_desc), layer, _ptr(x), T, H, I, E, k, _ptr(ids), _ptr(w), _ptr(offsets), _ptr(perm),
            _ptr(inv_perm), _ptr(ws), ws.numel() * ws.element_size(), _ptr(y), _ptr(status))
    if options is None:
        _check(lib().pw_moe_apl_ffn(*args, _stream(stream)))
    else:
        _check(lib().pw_moe_apl_ffn_ex(*args, ctypes.byref(options), _stream(stream)))


def pw_moe_route_apl_ffn(d_desc: torch.Tensor, layer: int, x: torch.Tensor, logits: torch.Tensor, I: int, E: int,
                         k: int, ids: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, perm: torch.Tensor,
                         inv_perm: torch.Tensor, mass_accum: Optional[torch.Tensor], ws: torch.Tensor,
                         y: torch.Tensor, status: torch.Tensor, options: Optional[pw_ffn_options] = None,
                         stream=None) -> None:
    """Routing and the fused expert layer (the routing arrays are outputs):
    one launch for batches one warp routes (at most 32 tokens, 8 experts and
    4 slots per token), else a routing launch and the fused launch."""
    _dev(x, torch.float16, "x")
    _dev(y, torch.float16, "y")
    _dev(logits, torch.float32, "logits")
    T, H = x.shape
    if tuple(logits.shape) != (T, E):
        raise ValueError(f"logits: need shape ({T}, {E}), got {tuple(logits.shape)}")
    args = (_ptr(d_desc), layer, _ptr(x), _ptr(logits), T, H, I, E, k, _ptr(ids), _ptr(w), _ptr(offsets),
            _ptr(perm), _ptr(inv_perm), _ptr(mass_accum), _ptr(ws), ws.numel() * ws.element_size(), _ptr(y),
            _ptr(status))
    if options is None:
        _check(lib().pw_moe_route_apl_ffn(*args, _stream(stream)))
    else:
        _check(lib().pw_moe_route_apl_ffn_ex(*args, ctypes.byref(options), _stream(stream)))


def pw_moe_route_apl_ffn_layers(d_desc: torch.Tensor, layer0: int, x: torch.Tensor, logits: torch.Tensor, I: int,
                                E: int, k: int, ids: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor,
                                perm: torch.Tensor, inv_perm: torch.Tensor, mass_accum: Optional[torch.Tensor],
                                ws: torch.Tensor, y: torch.Tensor, status: torch.Tensor,
                                options: Optional[pw_ffn_options] = None, stream=None) -> None:
    """Routing and the fused expert layer of L independent layers in one
    launch: x [L][T][H], logits [L][T][E], y [L][T][H]; the routing arrays
    are outputs in the layers' concatenated index space (see pw.h)."""
    _dev(x, torch.float16, "x")
    _dev(y, torch.float16, "y")
    _dev(logits, torch.float32, "logits")
    L, T, H = x.shape
    if tuple(logits.shape) != (L, T, E) or tuple(y.shape[:2]) != (L, T) or y.shape[2] != H:
        raise ValueError(f"layers call: x {tuple(x.shape)}, logits {tuple(logits.shape)}, y {tuple(y.shape)}")
    opts = options if options is not None else pw_ffn_options()
    _check(lib().pw_moe_route_apl_ffn_layers(_ptr(d_desc), layer0, L, _ptr(x), _ptr(logits), T, H, I, E, k, _ptr(ids),
                                             _ptr(w), _ptr(offsets), _ptr(perm), _ptr(inv_perm), _ptr(mass_accum),
                                             _ptr(ws), ws.numel() * ws.element_size(), _ptr(y), _ptr(status),
                                             ctypes.byref(opts), _stream(stream)))


PW_NOALLOC_SCRATCH_BYTES = 32 << 20


def pw_moe_apl_ffn_noalloc(d_desc: torch.Tensor, layer: int, x: torch.Tensor, I: int, E: int, k: int,
                           ids: Optional[torch.Tensor], w: torch.Tensor, offsets: torch.Tensor,
                           perm: torch.Tensor, inv_perm: torch.Tensor, y: torch.Tensor, status: torch.Tensor,
                           stream=None) -> None:
    """pw_moe_apl_ffn without a caller workspace: libpw's built-in scratch
    array is used instead (see include/pw.h for its size and sharing rules)."""
    _dev(x, torch.float16, "x")
    _dev(y, torch.float16, "y")
    T, H = x.shape
    _check(lib().pw_moe_apl_ffn_noalloc(_ptr(d_desc), layer, _ptr(x), T, H, I, E, k, _ptr(ids), _ptr(w),
                                        _ptr(offsets), _ptr(perm), _ptr(inv_perm), _ptr(y), _ptr(status),
                                        _stream(stream)))


def pw_unpack_indices(t, block: int, b: int, out: torch.Tensor, stream=None) -> None:
    _dev(out, torch.uint8, "out")
    _check(lib().pw_unpack_indices(t, block, b, _ptr(out), _stream(stream)))


def pw_apl_linear(t, block: int, x: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    _dev(x, torch.float16, "x")
    _dev(out, torch.float32, "out")
    _check(lib().pw_apl_linear(t, block, _ptr(x), x.shape[0], _ptr(out), _stream(stream)))


# ---------------------------------------------------------------------------
# The attention half of a decoder layer.  A single token's kernels run for a
# few microseconds, so these calls keep to plain integers and tuples: pointers
# are passed as numbers, the argument structures are packed in one go.
# ---------------------------------------------------------------------------
_DTYPE = {torch.float16: PW_DTYPE_F16, torch.bfloat16: PW_DTYPE_BF16}
_CODES = (torch.float8_e4m3fn, torch.uint8)
_F32 = (torch.float32,)
_I32 = (torch.int32,)


def _dtype16(t: torch.Tensor, name: str) -> int:
    d = _DTYPE.get(t.dtype)
    if d is None:
        raise ValueError(f"{name}: need fp16 or bf16, got {t.dtype}")
    return d


def _refuse(t: torch.Tensor, shape, dtypes, name: str, rows: str):
    raise ValueError(f"{name}: need a tensor {tuple(shape)} of {dtypes[0]} with {rows}, on the GPU of the call's first one, "
                     f"got {tuple(t.shape)} of {t.dtype} with strides {t.stride()} on {t.device}")


def _queue(stream, dev: int) -> int:
    """The stream of a call whose tensors are on GPU `dev`: its kernel runs on the
    current GPU, which has to be that one."""
    if dev < 0 or torch._C._cuda_getDevice() != dev:
        raise ValueError("need tensors on a GPU" if dev < 0 else
                         f"tensors on cuda:{dev}, but the current device is cuda:{torch._C._cuda_getDevice()}")
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _matrix(t: Optional[torch.Tensor], rows: int, cols: int, dtypes, name: str, dev: int):
    """(pointer, row stride) of a CUDA matrix whose rows are contiguous; (0, 0)
    for None."""
    if t is None:
        return 0, 0
    st = t.stride()
    if t.dtype not in dtypes or t.get_device() != dev or t.shape != (rows, cols) or (st[1] != 1 and cols > 1):
        _refuse(t, (rows, cols), dtypes, name, "contiguous rows")
    # the stride of a single row says nothing
    return t.data_ptr(), st[0] if rows > 1 or st[0] > cols else cols


def _vector(t: torch.Tensor, n: int, dtypes, name: str, dev: int) -> int:
    if t.dtype not in dtypes or t.get_device() != dev or t.shape != (n,) or (n > 1 and t.stride() != (1,)):
        _refuse(t, (n,), dtypes, name, "contiguous values")
    return t.data_ptr()


def _status(t: torch.Tensor, dev: int) -> int:
    if t.dtype is not torch.int32 or t.get_device() != dev or t.numel() < 1:
        _refuse(t, (1,), _I32, "status", "one value")
    return t.data_ptr()


# the structures of pw.h, packed in one go: pointers, strides, sizes
_NORM_ARGS = struct.Struct("@7P7q2ifi")
_QUANT_ARGS = struct.Struct("@3P4q4i")
_LINEAR_ARGS = struct.Struct("@6P5q4i")
_ROPE_ARGS = struct.Struct("@12P15q11if")
_ATTN_ARGS = struct.Struct("@9P11q13if")
_ATTN_OPTIONS = struct.Struct("@8i")
_NORMS_ARGS = struct.Struct("@9P8q2i3fi")
_GATED_ARGS = struct.Struct("@10P9q6i")
_LOGPROB_ARGS = struct.Struct("@7P6q4ifi")
for _packed, _struct in ((_NORM_ARGS, pw_norm_args), (_QUANT_ARGS, pw_quant_args), (_LINEAR_ARGS, pw_linear_args),
                         (_ROPE_ARGS, pw_rope_args), (_ATTN_ARGS, pw_attn_args), (_ATTN_OPTIONS, pw_attn_options),
                         (_NORMS_ARGS, pw_norms_args), (_GATED_ARGS, pw_gated_args), (_LOGPROB_ARGS, pw_logprob_args)):
    assert _packed.size == ctypes.sizeof(_struct)


def pw_add_rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float, residual: Optional[torch.Tensor] = None,
                   residual_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                   q: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None, stream=None) -> None:
    """y = r * rsqrt(mean(r^2) + eps) * weight with r = x + residual; `y` in
    x's type and/or `q` (e4m3) with `scale` (fp32, a scale per 128 columns);
    `residual_out` receives r."""
    dt, dev = _dtype16(x, "x"), x.get_device()
    rows, cols = x.shape
    same = (x.dtype,)
    xp, xs = _matrix(x, rows, cols, same, "x", dev)
    wp = _vector(weight, cols, same, "weight", dev)
    rp, rs = _matrix(residual, rows, cols, same, "residual", dev)
    rop, ros = _matrix(residual_out, rows, cols, same, "residual_out", dev)
    yp, ys = _matrix(y, rows, cols, same, "y", dev)
    qp, qs = _matrix(q, rows, cols, _CODES, "q", dev)
    sp, ss = _matrix(scale, rows, -(-cols // 128), _F32, "scale", dev)
    args = _NORM_ARGS.pack(xp, rp, wp, rop, yp, qp, sp, xs, rs, ros, ys, qs, ss, rows, cols, dt, eps, 0)
    _check(lib().pw_add_rmsnorm(args, _queue(stream, dev)))


def pw_quantize_fp8(x: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, block_rows: int = 1, stream=None) -> None:
    """x (fp16 or bf16 matrix) to e4m3 codes `q` and fp32 `scale`: groups of
    128 columns of one row (block_rows 1) or of 128 rows (block_rows 128)."""
    dt, dev = _dtype16(x, "x"), x.get_device()
    rows, cols = x.shape
    if block_rows < 1:
        raise ValueError(f"block_rows: {block_rows}")
    xp, xs = _matrix(x, rows, cols, (x.dtype,), "x", dev)
    qp, qs = _matrix(q, rows, cols, _CODES, "q", dev)
    sp, ss = _matrix(scale, -(-rows // block_rows), -(-cols // 128), _F32, "scale", dev)
    args = _QUANT_ARGS.pack(xp, qp, sp, xs, qs, ss, rows, cols, dt, block_rows, 0)
    _check(lib().pw_quantize_fp8(args, _queue(stream, dev)))


def pw_fp8_linear(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor, y: torch.Tensor,
                  status: torch.Tensor, stream=None) -> None:
    """y [M][N] = a [M][K] b [N][K]^T of e4m3 codes with their scales:
    a_scale [M][ceil(K/128)], b_scale [ceil(N/128)][ceil(K/128)]."""
    dt, dev = _dtype16(y, "y"), y.get_device()
    M, K = a.shape
    N = b.shape[0]
    kb = -(-K // 128)
    ap, lda = _matrix(a, M, K, _CODES, "a", dev)
    bp, ldb = _matrix(b, N, K, _CODES, "b", dev)
    yp, ldy = _matrix(y, M, N, (y.dtype,), "y", dev)
    sap, sa = _matrix(a_scale, M, kb, _F32, "a_scale", dev)
    sbp, sb = _matrix(b_scale, -(-N // 128), kb, _F32, "b_scale", dev)
    # a single row may have any stride: the row's own alignment is what counts
    if M == 1:
        lda = (lda + 15) // 16 * 16
    if N == 1:
        ldb = (ldb + 15) // 16 * 16
    args = _LINEAR_ARGS.pack(ap, sap, bp, sbp, yp, _status(status, dev), lda, sa, ldb, sb, ldy, M, N, K, dt)
    _check(lib().pw_fp8_linear(args, _queue(stream, dev)))


def pw_rope_turns(rotary_dim: int, base: float = 10000.0, scaling: Optional[pw_rope_scaling] = None):
    """(int64 CPU tensor [rotary_dim/2], factor): the table of pw_rope_append."""
    turns = torch.empty(max(rotary_dim, 0) // 2, dtype=torch.int64)
    factor = F32(0)
    _check(lib().pw_rope_turns(rotary_dim, base, ctypes.byref(scaling) if scaling is not None else None, _ptr(turns),
                               ctypes.byref(factor)))
    return turns, float(factor.value)


def _heads(t: torch.Tensor, shape, dtypes, name: str, dev: int):
    """(pointer, outer strides) of a CUDA tensor whose last dimension is contiguous."""
    st = t.stride()
    if t.dtype not in dtypes or t.get_device() != dev or t.shape != shape or (st[-1] != 1 and shape[-1] > 1):
        _refuse(t, shape, dtypes, name, "a contiguous last dimension")
    return t.data_ptr(), st


def _sequences(q_offsets: torch.Tensor, kv_lens: torch.Tensor, dev: int):
    """(q_offsets, kv_lens, batch)"""
    batch = kv_lens.shape[0]
    return (_vector(q_offsets, batch + 1, _I32, "q_offsets", dev), _vector(kv_lens, batch, _I32, "kv_lens", dev), batch)


def pw_rope_append(q: Optional[torch.Tensor], k: Optional[torch.Tensor], v: Optional[torch.Tensor],
                   turns: torch.Tensor, k_cache: Optional[torch.Tensor], v_cache: Optional[torch.Tensor],
                   page_table: Optional[torch.Tensor], q_offsets: torch.Tensor, kv_lens: torch.Tensor,
                   q_out: Optional[torch.Tensor], status: torch.Tensor, interleaved: bool = False, factor: float = 1.0,
                   positions: Optional[torch.Tensor] = None, stream=None) -> None:
    """Rotates q into q_out [T][heads][D] and k into the cache
    [pages][page_size][kv_heads][D] (any outer strides), and appends v there.
    The rotated part of a head is 2 * len(turns) wide."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("rope_append: neither q nor k")
    dt, dev, same = _dtype16(x, "q"), x.get_device(), (x.dtype,)
    T, _, D = x.shape
    offsets, lens, batch = _sequences(q_offsets, kv_lens, dev)
    qp = qop = kp = vp = kcp = vcp = table = pos = 0
    qs = qos = ks = vs = kcs = vcs = (0, 0, 0)
    heads = kv_heads = ts = pages = page_size = width = 0
    if q is not None:
        if q_out is None:
            raise ValueError("rope_append: q needs q_out")
        heads = q.shape[1]
        qp, qs = _heads(q, (T, heads, D), same, "q", dev)
        qop, qos = _heads(q_out, (T, heads, D), same, "q_out", dev)
    if k is not None:
        if v is None or k_cache is None or v_cache is None or page_table is None:
            raise ValueError("rope_append: k, v, the caches and the page table come together")
        kv_heads, (pages, page_size) = k.shape[1], k_cache.shape[:2]
        kp, ks = _heads(k, (T, kv_heads, D), same, "k", dev)
        vp, vs = _heads(v, (T, kv_heads, D), same, "v", dev)
        kcp, kcs = _heads(k_cache, (pages, page_size, kv_heads, D), same, "k_cache", dev)
        vcp, vcs = _heads(v_cache, (pages, page_size, kv_heads, D), same, "v_cache", dev)
        width = page_table.shape[1]
        table, ts = _matrix(page_table, batch, width, _I32, "page_table", dev)
    elif v is not None or k_cache is not None or v_cache is not None:
        raise ValueError("rope_append: k, v, the caches and the page table come together")
    half = turns.shape[0]
    tp = _vector(turns, half, (torch.int64,), "turns", dev)
    if positions is not None:
        pos = _vector(positions, T, _I32, "positions", dev)
    args = _ROPE_ARGS.pack(qp, qop, kp, vp, kcp, vcp, tp, pos, table, offsets, lens, _status(status, dev), qs[0], qs[1],
                           qos[0], qos[1], ks[0], ks[1], vs[0], vs[1], kcs[0], kcs[1], kcs[2], vcs[0], vcs[1], vcs[2],
                           ts, T, batch, heads, kv_heads, D, 2 * half, page_size, pages, width, dt, interleaved, factor)
    _check(lib().pw_rope_append(args, _queue(stream, dev)))


def pw_paged_attention_workspace(tokens: int, batch: int, heads: int, kv_heads: int, head_dim: int) -> int:
    return int(lib().pw_paged_attention_workspace(tokens, batch, heads, kv_heads, head_dim))


def pw_paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                       q_offsets: torch.Tensor, kv_lens: torch.Tensor, out: torch.Tensor, ws: torch.Tensor,
                       status: torch.Tensor, scale: float, causal: bool = True, window: int = 0, max_q_len: int = 0,
                       max_kv_len: int = 0, lse: Optional[torch.Tensor] = None, stream=None, sinks: int = 0) -> None:
    """out [T][heads][D] = attention of the new tokens q over their sequences'
    keys in the paged cache [pages][page_size][kv_heads][D]; with a `window` a
    token sees that many keys up to its own, and the first `sinks` of its
    sequence.  `ws` must be zeroed before its first use.  max_q_len / max_kv_len: bounds of the lengths
    (0: the batch's tokens, and what the page table holds)."""
    dt, dev, same = _dtype16(q, "q"), q.get_device(), (q.dtype,)
    T, heads, D = q.shape
    pages, page_size, kv_heads, _ = k_cache.shape
    offsets, lens, batch = _sequences(q_offsets, kv_lens, dev)
    qp, qs = _heads(q, (T, heads, D), same, "q", dev)
    op, os_ = _heads(out, (T, heads, D), same, "out", dev)
    kp, ks = _heads(k_cache, (pages, page_size, kv_heads, D), same, "k_cache", dev)
    vp, vs = _heads(v_cache, (pages, page_size, kv_heads, D), same, "v_cache", dev)
    width = page_table.shape[1]
    table, ts = _matrix(page_table, batch, width, _I32, "page_table", dev)
    lp = 0
    if lse is not None:
        lp, ls = _matrix(lse, T, heads, _F32, "lse", dev)
        if ls != heads and T > 1:   # the stride of a single row says nothing
            raise ValueError("lse: need a contiguous tensor")
    if ws.get_device() != dev:
        raise ValueError("ws: need a tensor on q's GPU")
    args = _ATTN_ARGS.pack(qp, op, lp, kp, vp, table, offsets, lens, _status(status, dev), qs[0], qs[1], os_[0], os_[1],
                           ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], ts, T, batch, heads, kv_heads, D, page_size, pages,
                           width, max_q_len or T, max_kv_len or page_size * width, dt, causal, window, scale)
    if sinks:
        _check(lib().pw_paged_attention_ex(args, _ATTN_OPTIONS.pack(sinks, 0, 0, 0, 0, 0, 0, 0), ws.data_ptr(), ws.nbytes,
                                           _queue(stream, dev)))
    else:
        _check(lib().pw_paged_attention(args, ws.data_ptr(), ws.nbytes, _queue(stream, dev)))


# ---------------------------------------------------------------------------
# Around the attention half: norms on both sides of a block, the model's end.
# ---------------------------------------------------------------------------
def pw_norm_add_norm(x: torch.Tensor, residual: torch.Tensor, eps: float, post_weight: Optional[torch.Tensor] = None,
                     weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                     residual_scale: float = 1.0, block_scale: float = 1.0,
                     residual_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                     q: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None, stream=None) -> None:
    """r = residual_scale * residual + block_scale * gate * u with u the
    RMS norm of x by `post_weight` (x itself without it); `residual_out` receives
    r, `y` and/or `q` (e4m3) with `scale` its RMS norm by `weight`.  `gate`:
    a row for all rows [cols], or [rows][cols]."""
    dt, dev = _dtype16(x, "x"), x.get_device()
    rows, cols = x.shape
    same = (x.dtype,)
    xp, xs = _matrix(x, rows, cols, same, "x", dev)
    rp, rs = _matrix(residual, rows, cols, same, "residual", dev)
    pp = 0 if post_weight is None else _vector(post_weight, cols, same, "post_weight", dev)
    wp = 0 if weight is None else _vector(weight, cols, same, "weight", dev)
    gp = gs = 0
    if gate is not None:
        if gate.dim() == 1:
            gp = _vector(gate, cols, same, "gate", dev)
        else:
            gp, gs = _matrix(gate, rows, cols, same, "gate", dev)
    rop, ros = _matrix(residual_out, rows, cols, same, "residual_out", dev)
    yp, ys = _matrix(y, rows, cols, same, "y", dev)
    qp, qs = _matrix(q, rows, cols, _CODES, "q", dev)
    sp, ss = _matrix(scale, rows, -(-cols // 128), _F32, "scale", dev)
    args = _NORMS_ARGS.pack(xp, rp, pp, gp, wp, rop, yp, qp, sp, xs, rs, gs, ros, ys, qs, ss, rows, cols, dt, eps,
                            residual_scale, block_scale, 0)
    _check(lib().pw_norm_add_norm(args, _queue(stream, dev)))


def pw_fp8_gated_linear(a: torch.Tensor, a_scale: torch.Tensor, gate: torch.Tensor, gate_scale: torch.Tensor,
                        up: torch.Tensor, up_scale: torch.Tensor, status: torch.Tensor, y: Optional[torch.Tensor] = None,
                        q: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                        activation: int = PW_ACT_SILU, stream=None) -> None:
    """h [M][N] = act(a gate^T) * (a up^T) of e4m3 codes a [M][K], gate and up
    [N][K] with scales as in pw_fp8_linear; `y` receives h (fp16 or bf16),
    and/or `q` its e4m3 codes with `scale` [M][ceil(N/128)]."""
    dt, dev = PW_DTYPE_F16 if y is None else _dtype16(y, "y"), a.get_device()
    M, K = a.shape
    N = gate.shape[0]
    kb, nb = -(-K // 128), -(-N // 128)
    ap, lda = _matrix(a, M, K, _CODES, "a", dev)
    gp, ldg = _matrix(gate, N, K, _CODES, "gate", dev)
    up_, ldu = _matrix(up, N, K, _CODES, "up", dev)
    sap, sa = _matrix(a_scale, M, kb, _F32, "a_scale", dev)
    sgp, sg = _matrix(gate_scale, nb, kb, _F32, "gate_scale", dev)
    sup, su = _matrix(up_scale, nb, kb, _F32, "up_scale", dev)
    yp, ldy = (0, 0) if y is None else _matrix(y, M, N, (y.dtype,), "y", dev)
    qp, ldq = _matrix(q, M, N, _CODES, "q", dev)
    sp, ss = _matrix(scale, M, nb, _F32, "scale", dev)
    # a single row may have any stride: the row's own alignment is what counts
    if M == 1:
        lda, ldq = (lda + 15) // 16 * 16, (ldq + 15) // 16 * 16
    if N == 1:
        ldg, ldu = (ldg + 15) // 16 * 16, (ldu + 15) // 16 * 16
    args = _GATED_ARGS.pack(ap, sap, gp, sgp, up_, sup, yp, qp, sp, _status(status, dev), lda, sa, ldg, sg, ldu, su, ldy, ldq,
                            ss, M, N, K, dt, activation, 0)
    _check(lib().pw_fp8_gated_linear(args, _queue(stream, dev)))


def pw_token_logprobs(logits: torch.Tensor, targets: Optional[torch.Tensor] = None,
                      logprobs: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                      entropy: Optional[torch.Tensor] = None, top_ids: Optional[torch.Tensor] = None,
                      top_logprobs: Optional[torch.Tensor] = None, scale: float = 1.0, stream=None) -> None:
    """Of softmax(scale * logits) by rows [T][V] (fp16, bf16 or fp32): the log
    probabilities of int32 `targets` [T][n] into `logprobs`, the logarithm of its
    sum into `lse` [T], its `entropy` [T], and the most probable tokens with
    their log probabilities into `top_ids`, `top_logprobs` [T][k]."""
    dt, dev = PW_DTYPE_F32 if logits.dtype is torch.float32 else _dtype16(logits, "logits"), logits.get_device()
    rows, vocab = logits.shape
    zp, zs = _matrix(logits, rows, vocab, (logits.dtype,), "logits", dev)
    if (targets is None) != (logprobs is None) or (top_ids is None) != (top_logprobs is None):
        raise ValueError("token_logprobs: targets and logprobs, top_ids and top_logprobs come together")
    given = 0 if targets is None else targets.shape[1]
    top = 0 if top_ids is None else top_ids.shape[1]
    tp, ts = _matrix(targets, rows, given, _I32, "targets", dev)
    lp, ls = _matrix(logprobs, rows, given, _F32, "logprobs", dev)
    ip, is_ = _matrix(top_ids, rows, top, _I32, "top_ids", dev)
    op, os_ = _matrix(top_logprobs, rows, top, _F32, "top_logprobs", dev)
    sp = 0 if lse is None else _vector(lse, rows, _F32, "lse", dev)
    ep = 0 if entropy is None else _vector(entropy, rows, _F32, "entropy", dev)
    args = _LOGPROB_ARGS.pack(zp, tp, lp, sp, ep, ip, op, zs, ts, ls, is_, os_, rows, vocab, given, top, dt, scale, 0)
    _check(lib().pw_token_logprobs(args, _queue(stream, dev)))
