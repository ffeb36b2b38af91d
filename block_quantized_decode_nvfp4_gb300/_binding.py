"""ctypes binding of libbqd.so: the C ABI of include/bqd.h, same names.

Argument marshalling only. Array arguments are torch tensors (device memory)
or raw integer device addresses; sizes are passed through unchanged; the
stream defaults to torch's current stream. A non-zero status raises BqdError.
There is no fallback: if libbqd.so is missing every call raises.
"""
from __future__ import annotations

import ctypes as C
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libbqd.so")

BQD_OK = 0
STATUS_NAMES = {0: "BQD_OK", 1: "BQD_ERR_NULL", 2: "BQD_ERR_SHAPE", 3: "BQD_ERR_ALIGN", 4: "BQD_ERR_ARCH",
                5: "BQD_ERR_LAUNCH", 6: "BQD_ERR_WORKSPACE", 7: "BQD_ERR_PATH", 8: "BQD_ERR_DEVICE"}
BQD_PATH_AUTO = 0
BQD_PATH_CUDA_CORE = 1
BQD_PATH_STREAM = 2
BQD_PATH_MMA = 3
BQD_PATH_DIRECT = 4
BQD_PATH_TILES = 5
BQD_LAUNCH_PDL = 1
BQD_F32 = 0
BQD_BF16 = 1
BQD_E4M3 = 2
BQD_SLOTS_TABLE_FULL = 1
BQD_SLOTS_TOKENS_CUT = 2
BQD_ROPE_HALVES = 0
BQD_ROPE_PAIRS = 1

_lib = None


class BqdError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = lib().bqd_status_string(status).decode() if _lib is not None else "?"
        if status == 5 and _lib is not None:
            msg += ": " + lib().bqd_last_cuda_error().decode()
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} ({msg})")


class KVCache(C.Structure):
    """bqd_kv_cache: the paged K and V arrays of one layer (see bqd.h)."""
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("num_pages", C.c_int64), ("page_stride", C.c_int64), ("token_stride", C.c_int64),
                ("head_stride", C.c_int64), ("page_size", C.c_int32), ("heads", C.c_int32),
                ("head_dim", C.c_int32), ("type", C.c_int32)]


_vp, _i64, _i32, _f32, _sz = C.c_void_p, C.c_int64, C.c_int, C.c_float, C.c_size_t
SIGNATURES = {
    "bqd_status_string": (C.c_char_p, [_i32]),
    "bqd_version": (_i32, []),
    "bqd_last_cuda_error": (C.c_char_p, []),
    "bqd_set_launch_flags": (C.c_uint, [C.c_uint]),
    "bqd_get_launch_flags": (C.c_uint, []),
    "nvfp4_gemv": (_i32, [_vp, _vp, _f32, _vp, _vp, _i64, _i64, _i32, _vp]),
    "nvfp4_gemv_path": (_i32, [_vp, _vp, _f32, _vp, _vp, _i64, _i64, _i32, _i32, _vp]),
    "q8_0_gemv": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _vp]),
    "q8_0_gemv_path": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _i32, _vp]),
    "nvfp4_gemm": (_i32, [_vp, _vp, _f32, _vp, _vp, _i64, _i64, _i64, _vp]),
    "moe_prefill_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32]),
    "moe_prefill_layer": (_i32, [_vp] * 10 + [_sz, _i32, _i32, _i32, _i32, _i32, _vp]),
    "nvfp4_gemm_grouped": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i64, _vp]),
    "q4_0_gemv": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _vp]),
    "q4_0_gemv_path": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _i32, _vp]),
    "q4_0_dequant": (_i32, [_vp, _vp, _vp, _i64, _i64, _vp]),
    "q4_1_gemv": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _vp]),
    "q4_1_dequant": (_i32, [_vp, _vp, _vp, _i64, _i64, _vp]),
    "fp8_b128_gemv": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _vp]),
    "fp8_b128_gemv_path": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _i32, _vp]),
    "fp8_b128_dequant": (_i32, [_vp, _vp, _vp, _i64, _i64, _vp]),
    "nvfp4_gemv_add": (_i32, [_vp, _vp, _f32, _vp, _vp, _vp, _i64, _i64, _i32, _vp]),
    "nvfp4_encode": (_i32, [_vp, _f32, _vp, _vp, _i64, _i64, _vp]),
    "q8_0_encode": (_i32, [_vp, _vp, _vp, _i64, _i64, _vp]),
    "q8_0_gemv_add": (_i32, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i32, _vp]),
    "nvfp4_gemv_silu_mul": (_i32, [_vp, _vp, _f32, _vp, _vp, _i64, _i64, _i32, _vp]),
    "q8_0_gemv_silu_mul": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _vp]),
    "bqd_device_error": (_i32, [C.POINTER(C.c_uint)]),
    "bqd_debug_stream_fault": (_i32, [_i32, C.c_longlong]),
    "nvfp4_dequant": (_i32, [_vp, _vp, _f32, _vp, _i64, _i64, _vp]),
    "q8_0_dequant": (_i32, [_vp, _vp, _vp, _i64, _i64, _vp]),
    "moe_route_topk": (_i32, [_vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp]),
    "moe_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32]),
    "moe_grouped_gemv": (_i32, [_vp] * 13 + [_sz, _i32, _i32, _i32, _i32, _i32, _vp]),
    "bqd_moe_read_status": (_i32, [_vp, C.POINTER(C.c_int32), _vp]),
    "moe_grouped_gemv_noalloc": (_i32, [_vp] * 12 + [_i32, _i32, _i32, _i32, _i32, _vp]),
    "moe_layer": (_i32, [_vp] * 10 + [_sz, _i32, _i32, _i32, _i32, _i32, _vp]),
    "moe_layer_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32]),
    "paged_slots": (_i32, [_vp, _vp, _vp, _i64, _vp, _i64, _i64, _i32, _vp, _vp, _vp, _vp, _i64, _vp, _vp]),
    "qk_norm_rope_cache": (_i32, [_vp, _vp, _vp, _i32, _i64, _i64, _i64, _vp, _vp, _f32, _vp, _i64, _i32, _i32, _vp,
                                  _vp, _vp, C.POINTER(KVCache), _i64, _i32, _vp]),
    "tree_attention": (_i32, [_vp, _i64, C.POINTER(KVCache), _vp, _i64, _vp, _vp, _vp, _i32, _f32, _vp, _vp, _vp, _sz,
                              _i64, _i64, _i32, _vp]),
    "tree_attention_workspace_bytes": (_sz, [_i64, _i64, _i32, _i32, _i32]),
    "token_logprobs": (_i32, [_vp, _i32, _i64, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _sz, _i64, _i64, _vp]),
    "token_logprobs_workspace_bytes": (_sz, [_i64, _i64, _i32]),
    "fp8_x_encode": (_i32, [_vp, _i32, _i64, _vp, _vp, _i64, _i64, _vp]),
    "residual_norm": (_i32, [_vp, _i32, _i64, _vp, _vp, _i32, _i64, _f32, _vp, _vp, _i32, _vp, _f32, _vp, _i32, _vp,
                             _i64, _i64, _vp]),
    "fp8_b128_gemm": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i64, _vp]),
    "fp8_b128_gemm_silu_mul": (_i32, [_vp] * 7 + [_i32, _vp, _i64, _i64, _i64, _vp]),
}


def lib() -> C.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it first (python -c 'import __graft_entry__ as g; "
                               "g.build()'); there is no CPU fallback")
        L = C.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _ptr(a):
    if a is None:
        return None
    if isinstance(a, int):
        return a
    return a.data_ptr()


_current_raw_stream = None  # handle of torch's current stream on the current device


def _find_current_raw_stream():
    """torch's own shortcut to the handle where it has one (0.2 us a call), else through a Stream object (2.9 us)."""
    global _current_raw_stream
    import torch
    torch.cuda.current_stream()  # initialises CUDA, or raises
    raw, dev = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
    if raw is None or dev is None:
        _current_raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    else:
        _current_raw_stream = lambda: raw(dev())  # noqa: E731


def _stream(s):
    if s is None:
        if _current_raw_stream is None:
            _find_current_raw_stream()
        return _current_raw_stream()
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(status: int, where: str) -> None:
    if status != BQD_OK:
        raise BqdError(status, where)


def version() -> int:
    return lib().bqd_version()


def set_launch_flags(flags: int) -> int:
    """Process-wide launch options (BQD_LAUNCH_*); returns the previous value."""
    return lib().bqd_set_launch_flags(flags)


def get_launch_flags() -> int:
    return lib().bqd_get_launch_flags()


def nvfp4_gemv(codes, scales, tensor_scale, x, y, M, K, N, stream=None):
    _check(lib().nvfp4_gemv(_ptr(codes), _ptr(scales), tensor_scale, _ptr(x), _ptr(y), M, K, N, _stream(stream)),
           "nvfp4_gemv")


def nvfp4_gemv_path(codes, scales, tensor_scale, x, y, M, K, N, path, stream=None):
    _check(lib().nvfp4_gemv_path(_ptr(codes), _ptr(scales), tensor_scale, _ptr(x), _ptr(y), M, K, N, path,
                                 _stream(stream)), "nvfp4_gemv_path")


def q8_0_gemv(q, d, x, y, M, K, N, stream=None):
    _check(lib().q8_0_gemv(_ptr(q), _ptr(d), _ptr(x), _ptr(y), M, K, N, _stream(stream)), "q8_0_gemv")


def q8_0_gemv_path(q, d, x, y, M, K, N, path, stream=None):
    _check(lib().q8_0_gemv_path(_ptr(q), _ptr(d), _ptr(x), _ptr(y), M, K, N, path, _stream(stream)),
           "q8_0_gemv_path")


def nvfp4_gemv_add(codes, scales, tensor_scale, x, residual, y, M, K, N=1, stream=None):
    _check(lib().nvfp4_gemv_add(_ptr(codes), _ptr(scales), tensor_scale, _ptr(x), _ptr(residual), _ptr(y), M, K, N,
                                _stream(stream)), "nvfp4_gemv_add")


def q8_0_gemv_add(q, d, x, residual, y, M, K, N=1, stream=None):
    _check(lib().q8_0_gemv_add(_ptr(q), _ptr(d), _ptr(x), _ptr(residual), _ptr(y), M, K, N, _stream(stream)),
           "q8_0_gemv_add")


def nvfp4_gemv_silu_mul(codes, scales, tensor_scale, x, h, I, K, N=1, stream=None):
    _check(lib().nvfp4_gemv_silu_mul(_ptr(codes), _ptr(scales), tensor_scale, _ptr(x), _ptr(h), I, K, N,
                                     _stream(stream)), "nvfp4_gemv_silu_mul")


def q8_0_gemv_silu_mul(q, d, x, h, I, K, N=1, stream=None):
    _check(lib().q8_0_gemv_silu_mul(_ptr(q), _ptr(d), _ptr(x), _ptr(h), I, K, N, _stream(stream)),
           "q8_0_gemv_silu_mul")


def nvfp4_encode(w, tensor_scale, codes, scales, M, K, stream=None):
    _check(lib().nvfp4_encode(_ptr(w), tensor_scale, _ptr(codes), _ptr(scales), M, K, _stream(stream)),
           "nvfp4_encode")


def q8_0_encode(w, q, d, M, K, stream=None):
    _check(lib().q8_0_encode(_ptr(w), _ptr(q), _ptr(d), M, K, _stream(stream)), "q8_0_encode")


def bqd_device_error() -> int:
    """Device error bits of the streaming kernels (synchronising; clears them)."""
    out = C.c_uint(0)
    st = lib().bqd_device_error(C.byref(out))
    if st not in (BQD_OK, 8):
        raise BqdError(st, "bqd_device_error")
    return out.value


def debug_stream_fault(withhold_last_stage: bool, wait_limit_cycles: int = 0) -> None:
    """Failure-path test switch of the streaming GEMV kernel (see bqd.h)."""
    _check(lib().bqd_debug_stream_fault(1 if withhold_last_stage else 0, wait_limit_cycles),
           "bqd_debug_stream_fault")


def nvfp4_dequant(codes, scales, tensor_scale, w, M, K, stream=None):
    _check(lib().nvfp4_dequant(_ptr(codes), _ptr(scales), tensor_scale, _ptr(w), M, K, _stream(stream)),
           "nvfp4_dequant")


def q8_0_dequant(q, d, w, M, K, stream=None):
    _check(lib().q8_0_dequant(_ptr(q), _ptr(d), _ptr(w), M, K, _stream(stream)), "q8_0_dequant")


def nvfp4_gemm(codes, scales, tensor_scale, x, y, M, K, T, stream=None):
    _check(lib().nvfp4_gemm(_ptr(codes), _ptr(scales), tensor_scale, _ptr(x), _ptr(y), M, K, T, _stream(stream)),
           "nvfp4_gemm")


def nvfp4_gemm_grouped(codes, scales, tensor_scales, x, expert_offsets, y, E, M, K, P, stream=None):
    _check(lib().nvfp4_gemm_grouped(_ptr(codes), _ptr(scales), _ptr(tensor_scales), _ptr(x), _ptr(expert_offsets),
                                    _ptr(y), E, M, K, P, _stream(stream)), "nvfp4_gemm_grouped")


def moe_prefill_workspace_bytes(T, topk, H, I, E):
    return int(lib().moe_prefill_workspace_bytes(T, topk, H, I, E))


def moe_prefill_layer(logits, gu_codes, gu_scales, gu_ts, dn_codes, dn_scales, dn_ts, x, y, workspace,
                      workspace_bytes, E, H, I, T, topk, stream=None):
    _check(lib().moe_prefill_layer(_ptr(logits), _ptr(gu_codes), _ptr(gu_scales), _ptr(gu_ts), _ptr(dn_codes),
                                   _ptr(dn_scales), _ptr(dn_ts), _ptr(x), _ptr(y), _ptr(workspace), workspace_bytes,
                                   E, H, I, T, topk, _stream(stream)), "moe_prefill_layer")


def q4_0_gemv(codes, d, x, y, M, K, N, stream=None):
    _check(lib().q4_0_gemv(_ptr(codes), _ptr(d), _ptr(x), _ptr(y), M, K, N, _stream(stream)), "q4_0_gemv")


def q4_0_gemv_path(codes, d, x, y, M, K, N, path, stream=None):
    _check(lib().q4_0_gemv_path(_ptr(codes), _ptr(d), _ptr(x), _ptr(y), M, K, N, path, _stream(stream)),
           "q4_0_gemv_path")


def q4_0_dequant(codes, d, w, M, K, stream=None):
    _check(lib().q4_0_dequant(_ptr(codes), _ptr(d), _ptr(w), M, K, _stream(stream)), "q4_0_dequant")


def q4_1_gemv(codes, dm, x, y, M, K, N, stream=None):
    """Q4_1 GEMV: codes [M][K/2] (Q4_0 nibble order), dm [M][K/32][2] fp16 (d, m)."""
    _check(lib().q4_1_gemv(_ptr(codes), _ptr(dm), _ptr(x), _ptr(y), M, K, N, _stream(stream)), "q4_1_gemv")


def q4_1_dequant(codes, dm, w, M, K, stream=None):
    _check(lib().q4_1_dequant(_ptr(codes), _ptr(dm), _ptr(w), M, K, _stream(stream)), "q4_1_dequant")


def fp8_b128_gemv(codes, scales, x, y, M, K, N, stream=None):
    """FP8 block-128 GEMV: E4M3 codes [M][K], fp32 tile scales [ceil(M/128)][ceil(K/128)]."""
    _check(lib().fp8_b128_gemv(_ptr(codes), _ptr(scales), _ptr(x), _ptr(y), M, K, N, _stream(stream)),
           "fp8_b128_gemv")


def fp8_b128_gemv_path(codes, scales, x, y, M, K, N, path, stream=None):
    _check(lib().fp8_b128_gemv_path(_ptr(codes), _ptr(scales), _ptr(x), _ptr(y), M, K, N, path, _stream(stream)),
           "fp8_b128_gemv_path")


def fp8_b128_dequant(codes, scales, w, M, K, stream=None):
    _check(lib().fp8_b128_dequant(_ptr(codes), _ptr(scales), _ptr(w), M, K, _stream(stream)), "fp8_b128_dequant")


def moe_route_topk(logits, T, E, topk, expert_offsets, pair_token, pair_weight, pair_slot, stream=None):
    _check(lib().moe_route_topk(_ptr(logits), T, E, topk, _ptr(expert_offsets), _ptr(pair_token),
                                _ptr(pair_weight), _ptr(pair_slot), _stream(stream)), "moe_route_topk")


def moe_workspace_bytes(T, topk, H, I) -> int:
    return lib().moe_workspace_bytes(T, topk, H, I)


def moe_grouped_gemv(gu_codes, gu_scales, gu_ts, dn_codes, dn_scales, dn_ts, x, expert_offsets, pair_token,
                     pair_weight, pair_slot, y, workspace, workspace_bytes, E, H, I, T, topk, stream=None):
    _check(lib().moe_grouped_gemv(_ptr(gu_codes), _ptr(gu_scales), _ptr(gu_ts), _ptr(dn_codes), _ptr(dn_scales),
                                  _ptr(dn_ts), _ptr(x), _ptr(expert_offsets), _ptr(pair_token), _ptr(pair_weight),
                                  _ptr(pair_slot), _ptr(y), _ptr(workspace), workspace_bytes, E, H, I, T, topk,
                                  _stream(stream)), "moe_grouped_gemv")


def moe_grouped_gemv_noalloc(gu_codes, gu_scales, gu_ts, dn_codes, dn_scales, dn_ts, x, expert_offsets,
                             pair_token, pair_weight, pair_slot, y, E, H, I, T, topk, stream=None):
    """moe_grouped_gemv without a caller workspace (scratch inside the library)."""
    _check(lib().moe_grouped_gemv_noalloc(_ptr(gu_codes), _ptr(gu_scales), _ptr(gu_ts), _ptr(dn_codes),
                                          _ptr(dn_scales), _ptr(dn_ts), _ptr(x), _ptr(expert_offsets),
                                          _ptr(pair_token), _ptr(pair_weight), _ptr(pair_slot), _ptr(y), E, H, I, T,
                                          topk, _stream(stream)), "moe_grouped_gemv_noalloc")


def moe_layer(logits, gu_codes, gu_scales, gu_ts, dn_codes, dn_scales, dn_ts, x, y, workspace, workspace_bytes,
              E, H, I, T, topk, stream=None):
    """Router and routed MoE layer from logits (moe_route_topk + moe_grouped_gemv in one call)."""
    _check(lib().moe_layer(_ptr(logits), _ptr(gu_codes), _ptr(gu_scales), _ptr(gu_ts), _ptr(dn_codes),
                           _ptr(dn_scales), _ptr(dn_ts), _ptr(x), _ptr(y), _ptr(workspace), workspace_bytes, E, H, I,
                           T, topk, _stream(stream)), "moe_layer")


def moe_layer_workspace_bytes(T, topk, H, I, E) -> int:
    return lib().moe_layer_workspace_bytes(T, topk, H, I, E)


def bqd_moe_read_status(workspace, stream=None) -> int:
    """Device status word of a MoE workspace (synchronising). Returns the bits."""
    out = C.c_int32(0)
    st = lib().bqd_moe_read_status(_ptr(workspace), C.byref(out), _stream(stream))
    if st not in (BQD_OK, 8):
        raise BqdError(st, "bqd_moe_read_status")
    return out.value


def kv_cache(k, v, k_scale=None, v_scale=None) -> KVCache:
    """Descriptor of a paged cache: k and v tensors [pages][page_size][heads][head_dim], bfloat16, or float8_e4m3fn
    (or its bytes, uint8) with fp32 scales per head. A cache that holds a page's tokens by heads is passed as a view
    with its dimensions in this order (k.transpose(1, 2)). The tensors must outlive the descriptor."""
    import torch
    types = {torch.bfloat16: BQD_BF16, torch.float8_e4m3fn: BQD_E4M3, torch.uint8: BQD_E4M3}
    if k.dtype not in types or v.dtype != k.dtype or k.dim() != 4 or v.shape != k.shape or v.stride() != k.stride():
        raise ValueError("kv_cache: k and v are [pages][page_size][heads][head_dim], of one type (bfloat16 or "
                         "float8_e4m3fn) and one layout")
    if k.shape[3] > 1 and k.stride(3) != 1:
        raise ValueError("kv_cache: a head's elements are contiguous")
    return KVCache(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), k.shape[0], k.stride(0), k.stride(1), k.stride(2),
                   k.shape[1], k.shape[2], k.shape[3], types[k.dtype])


def paged_slots(context_lens, new_lens, free_pages, num_free, block_table, R, table_width, page_size, depths,
                token_offsets, slots, positions, token_capacity, counts, stream=None):
    """Block table, slots and positions of a step's new tokens from the requests' lengths."""
    _check(lib().paged_slots(_ptr(context_lens), _ptr(new_lens), _ptr(free_pages), num_free, _ptr(block_table), R,
                             table_width, page_size, _ptr(depths), _ptr(token_offsets), _ptr(slots), _ptr(positions),
                             token_capacity, _ptr(counts), _stream(stream)), "paged_slots")


def qk_norm_rope_cache(q, k, v, in_type, q_pitch, k_pitch, v_pitch, q_weight, k_weight, eps, cos_sin, max_pos,
                       rot_dim, rot_style, positions, slots, q_out, cache, T, Hq, stream=None):
    """Norm and rotation of q and k heads, q to q_out (bf16), k and v into the cache at each token's slot."""
    _check(lib().qk_norm_rope_cache(_ptr(q), _ptr(k), _ptr(v), in_type, q_pitch, k_pitch, v_pitch, _ptr(q_weight),
                                    _ptr(k_weight), eps, _ptr(cos_sin), max_pos, rot_dim, rot_style, _ptr(positions),
                                    _ptr(slots), _ptr(q_out), C.byref(cache), T, Hq, _stream(stream)),
           "qk_norm_rope_cache")


def tree_attention(q, q_pitch, cache, block_table, table_width, context_lens, token_offsets, mask, mask_words, scale,
                   out, lse, workspace, workspace_bytes, R, T, Hq, stream=None):
    """Attention of a step's new tokens (decode, a drafted chain or a drafted tree) over the paged cache."""
    _check(lib().tree_attention(_ptr(q), q_pitch, C.byref(cache), _ptr(block_table), table_width, _ptr(context_lens),
                                _ptr(token_offsets), _ptr(mask), mask_words, scale, _ptr(out), _ptr(lse),
                                _ptr(workspace), workspace_bytes, R, T, Hq, _stream(stream)), "tree_attention")


def tree_attention_workspace_bytes(R, T, Hq, Hkv, D) -> int:
    return lib().tree_attention_workspace_bytes(R, T, Hq, Hkv, D)


def token_logprobs(logits, in_type, pitch, tokens, logprob, entropy, top_ids, top_logprobs, topk, workspace,
                   workspace_bytes, T, V, stream=None):
    """Log probability of given tokens, entropy and the topk alternatives of logits rows."""
    _check(lib().token_logprobs(_ptr(logits), in_type, pitch, _ptr(tokens), _ptr(logprob), _ptr(entropy),
                                _ptr(top_ids), _ptr(top_logprobs), topk, _ptr(workspace), workspace_bytes, T, V,
                                _stream(stream)), "token_logprobs")


def token_logprobs_workspace_bytes(T, V, topk) -> int:
    return lib().token_logprobs_workspace_bytes(T, V, topk)


def _elsewhere(where, a, dev):
    raise ValueError(f"{where}: a tensor on {a.device}, the current device is cuda:{dev}")


_current_device = None  # torch's current device, by its own shortcut


def _here(where, stream, *tensors):
    """Addresses of a call's tensors (None and integers as they are), all of the current device, and the handle of its
    stream, the current one of that device where none is given."""
    global _current_device
    if _current_device is None:
        import torch
        _find_current_raw_stream()  # initialises CUDA, or raises
        _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    dev = _current_device()
    at = [a if a is None or type(a) is int else a.data_ptr() if a.get_device() == dev else _elsewhere(where, a, dev)
          for a in tensors]
    at.append(_current_raw_stream() if stream is None else _stream(stream))
    return at


def fp8_x_encode(x, x_type, x_pitch, codes, scales, K, T, stream=None):
    """8-bit activations of rows [T][K]: E4M3 codes [T][K], fp32 scales [ceil(K/128)][T]."""
    x, codes, scales, stream = _here("fp8_x_encode", stream, x, codes, scales)
    status = (_lib or lib()).fp8_x_encode(x, x_type, x_pitch, codes, scales, K, T, stream)
    if status:
        raise BqdError(status, "fp8_x_encode")


def residual_norm(x, x_type, x_pitch, post_weight, gate, gate_type, gate_pitch, residual_scale, residual, residual_out,
                  residual_type, pre_weight, eps, y, y_type, y_scales, H, T, stream=None):
    """Residual add of a block's output (its norm, gate and scale), then the next block's norm: y bf16 or E4M3."""
    x, post_weight, gate, residual, residual_out, pre_weight, y, y_scales, stream = _here(
        "residual_norm", stream, x, post_weight, gate, residual, residual_out, pre_weight, y, y_scales)
    status = (_lib or lib()).residual_norm(x, x_type, x_pitch, post_weight, gate, gate_type, gate_pitch, residual_scale,
                                           residual, residual_out, residual_type, pre_weight, eps, y, y_type, y_scales, H,
                                           T, stream)
    if status:
        raise BqdError(status, "residual_norm")


def fp8_b128_gemm(codes, scales, x, x_scales, y, y_type, M, K, T, stream=None):
    """8-bit activations [T][K] times FP8 block-128 weights [M][K]: y [T][M], fp32 or bf16."""
    codes, scales, x, x_scales, y, stream = _here("fp8_b128_gemm", stream, codes, scales, x, x_scales, y)
    status = (_lib or lib()).fp8_b128_gemm(codes, scales, x, x_scales, y, y_type, M, K, T, stream)
    if status:
        raise BqdError(status, "fp8_b128_gemm")


def fp8_b128_gemm_silu_mul(gate_codes, gate_scales, up_codes, up_scales, x, x_scales, h, h_type, h_scales, I, K, T,
                           stream=None):
    """SiLU(gate) * up of 8-bit activations in one kernel: h [T][I], fp32, bf16 or E4M3 with scales."""
    gate_codes, gate_scales, up_codes, up_scales, x, x_scales, h, h_scales, stream = _here(
        "fp8_b128_gemm_silu_mul", stream, gate_codes, gate_scales, up_codes, up_scales, x, x_scales, h, h_scales)
    status = (_lib or lib()).fp8_b128_gemm_silu_mul(gate_codes, gate_scales, up_codes, up_scales, x, x_scales, h, h_type,
                                                    h_scales, I, K, T, stream)
    if status:
        raise BqdError(status, "fp8_b128_gemm_silu_mul")
