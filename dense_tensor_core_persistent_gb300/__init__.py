"""Python binding of the GB300 (sm_103a) dense tensor-core GEMM library.

Argument marshalling only: every step of the GEMM runs in the CUDA kernels of
``_lib/libdtcp_gemm.so`` (built by ``build.py``), called through its C ABI
(``include/gemm.h``). There is no CPU or PyTorch fallback: if the library is
missing, importing the binding's functions raises.

Functions take raw device pointers (ints) or torch CUDA tensors; ``stream``
defaults to torch's current CUDA stream when torch is importable, else the
legacy default stream.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libdtcp_gemm.so")

GEMM_OK = 0
GEMM_ERR_INVALID_ARG = 1
GEMM_ERR_UNSUPPORTED_SHAPE = 2
GEMM_ERR_MISALIGNED = 3
GEMM_ERR_NO_DEVICE = 4
GEMM_ERR_ARCH = 5
GEMM_ERR_DRIVER = 6
GEMM_ERR_LAUNCH = 7
GEMM_ERR_TIMEOUT = 8
GEMM_ERR_OUT_OF_MEMORY = 9
GEMM_ERR_SCRATCH_TOO_SMALL = 10
NVFP4_NOALLOC_SCRATCH_BYTES = 16 << 20

GEMM_KERNEL_DEFAULT = 0
GEMM_KERNEL_BF16_1CTA = 1
GEMM_KERNEL_BF16_2CTA = 2
GEMM_KERNEL_BF16_2CTA_K64 = 3
GEMM_KERNEL_BF16_2CTA_WIDE = 4

# Entry points declared in include/gemm.h (the CPU tests check the library exports all of them).
EXPORTS = (
    "gemm_bf16", "gemm_nvfp4", "gemm_status_string", "gemm_get_device_status", "gemm_bf16_ex",
    "gemm_nvfp4_ex", "gemm_tile_coord", "gemm_choose_group_m", "gemm_launch_count",
    "gemm_nvfp4_blocked_scale_bytes", "gemm_nvfp4_pack_scales", "gemm_nvfp4_blocked", "gemm_nvfp4_blocked_ex",
    "gemm_nvfp4_noalloc", "gemm_measure_mma_rate", "gemm_bf16_fused", "gemm_nvfp4_fused", "gemm_nvfp4_blocked_fused",
    "gemm_bf16_plan", "gemm_clc_rule", "gemm_nvfp4_plan", "gemm_bf16_wide_rule",
    "gemm_rms_norm", "gemm_rms_norm_backward", "gemm_token_logprobs", "gemm_token_logprobs_backward",
    "gemm_glu_bf16", "gemm_glu_e4m3", "gemm_glu_bf16_backward", "gemm_glu_plan",
    "gemm_layer_norm", "gemm_layer_norm_backward", "gemm_embedding", "gemm_embedding_backward",
    "gemm_cross_entropy", "gemm_cross_entropy_backward", "gemm_cross_entropy_piece",
    "gemm_cross_entropy_plan",
)

# gemm_activation_t
GEMM_ACT_NONE = 0
GEMM_ACT_RELU = 1
GEMM_ACT_GELU_TANH = 2


class GemmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class gemm_options_t(ctypes.Structure):
    _fields_ = [
        ("kernel", ctypes.c_int),
        ("persistent", ctypes.c_int),
        ("group_m", ctypes.c_int),
        ("max_clusters", ctypes.c_int),
        ("wait_limit_us", ctypes.c_uint32),
        ("debug_flags", ctypes.c_uint32),
        ("no_tail_split", ctypes.c_int),
        ("no_pdl", ctypes.c_int),
        ("no_swap_ab", ctypes.c_int),
        ("no_split_k", ctypes.c_int),
        ("clc", ctypes.c_int),
        ("no_pad_a", ctypes.c_int),
        ("clock_probe", ctypes.c_void_p),
        ("clock_probe_ctas", ctypes.c_int),
    ]


# gemm_options_t.clc
GEMM_CLC_AUTO = 0
GEMM_CLC_ON = 1
GEMM_CLC_OFF = 2


def options(kernel=GEMM_KERNEL_DEFAULT, persistent=1, group_m=0, max_clusters=0, wait_limit_us=0, debug_flags=0,
            no_tail_split=0, no_pdl=0, no_swap_ab=0, no_split_k=0, clc=GEMM_CLC_AUTO, no_pad_a=0, clock_probe=None):
    """`clock_probe`: None, or a CUDA int64 tensor of 4 values per CTA (see clock_probe_mhz)."""
    probe, probe_ctas = None, 0
    if clock_probe is not None:
        probe, probe_ctas = _ptr(clock_probe), clock_probe.numel() // 4
    return gemm_options_t(kernel, persistent, group_m, max_clusters, wait_limit_us, debug_flags, no_tail_split, no_pdl,
                          no_swap_ab, no_split_k, clc, no_pad_a, probe, probe_ctas)


def clock_probe_mhz(probe) -> dict:
    """Reads a clock probe after the launch completed (gemm_options_t.clock_probe): each CTA's
    SM clock over its work (clock64 difference / %globaltimer difference), the median and
    range over the CTAs that recorded, and the span from the first start to the last end."""
    v = probe.view(-1, 4).cpu().tolist()
    rec = [r for r in v if r[0] and r[2] > r[0]]
    if not rec:
        return {"ctas": 0}
    mhz = sorted((r[3] - r[1]) / (r[2] - r[0]) * 1e3 for r in rec)
    span_us = (max(r[2] for r in rec) - min(r[0] for r in rec)) / 1e3
    return {"ctas": len(rec), "sm_mhz": mhz[len(mhz) // 2], "sm_mhz_min": mhz[0], "sm_mhz_max": mhz[-1],
            "span_us": span_us}


class gemm_epilogue_t(ctypes.Structure):
    _fields_ = [
        ("alpha", ctypes.c_float),
        ("beta", ctypes.c_float),
        ("bias", ctypes.c_void_p),
        ("activation", ctypes.c_int),
        ("reserved", ctypes.c_int),
    ]


def epilogue(alpha=1.0, beta=0.0, bias=None, activation=GEMM_ACT_NONE) -> gemm_epilogue_t:
    """C = act(alpha * A B^T + beta * C + bias[col]); `bias` is a device tensor of N BF16 values or None."""
    return gemm_epilogue_t(alpha, beta, None if bias is None else _ptr(bias), activation, 0)


GEMM_NORM_BF16 = 0
GEMM_NORM_E4M3 = 1
GEMM_NORM_NVFP4 = 2


GEMM_LOGITS_BF16 = 0
GEMM_LOGITS_F32 = 1


GEMM_GLU_SILU = 0
GEMM_GLU_GELU_TANH = 1
GEMM_GLU_RELU = 2


GEMM_TABLE_BF16 = 0
GEMM_TABLE_F32 = 1


class gemm_glu_strides_t(ctypes.Structure):
    _fields_ = [("x", ctypes.c_longlong), ("h", ctypes.c_longlong), ("dh", ctypes.c_longlong),
                ("dx", ctypes.c_longlong)]


class gemm_cross_entropy_strides_t(ctypes.Structure):
    _fields_ = [("x", ctypes.c_longlong), ("dx", ctypes.c_longlong)]


class gemm_norm_strides_t(ctypes.Structure):
    _fields_ = [("x", ctypes.c_longlong), ("residual", ctypes.c_longlong), ("sum", ctypes.c_longlong),
                ("y", ctypes.c_longlong)]


class gemm_norm_backward_strides_t(ctypes.Structure):
    _fields_ = [("dy", ctypes.c_longlong), ("sum", ctypes.c_longlong), ("dsum", ctypes.c_longlong),
                ("dx", ctypes.c_longlong)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded C library; raises if it has not been built (no fallback exists)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it with `python -m dense_tensor_core_persistent_gb300.build` "
                "(the GEMM has no CPU fallback)")
        l = ctypes.CDLL(LIB_PATH)
        P, I = ctypes.c_void_p, ctypes.c_int
        l.gemm_bf16.argtypes = [P, P, P, I, I, I, P]
        l.gemm_bf16.restype = I
        l.gemm_bf16_ex.argtypes = [P, P, P, I, I, I, P, ctypes.POINTER(gemm_options_t)]
        l.gemm_bf16_ex.restype = I
        l.gemm_nvfp4.argtypes = [P, P, P, P, P, I, I, I, P]
        l.gemm_nvfp4.restype = I
        l.gemm_nvfp4_ex.argtypes = [P, P, P, P, P, I, I, I, P, ctypes.POINTER(gemm_options_t)]
        l.gemm_nvfp4_ex.restype = I
        l.gemm_status_string.argtypes = [I]
        l.gemm_status_string.restype = ctypes.c_char_p
        l.gemm_get_device_status.argtypes = [P, ctypes.POINTER(ctypes.c_uint32)]
        l.gemm_get_device_status.restype = I
        l.gemm_tile_coord.argtypes = [I, I, I, I, I, I, ctypes.POINTER(I), ctypes.POINTER(I)]
        l.gemm_tile_coord.restype = I
        l.gemm_choose_group_m.argtypes = [I, I, I, I, I, I, I, ctypes.c_longlong]
        l.gemm_choose_group_m.restype = I
        l.gemm_clc_rule.argtypes = [I, I, I, I]
        l.gemm_clc_rule.restype = I
        l.gemm_nvfp4_blocked_scale_bytes.argtypes = [I, I]
        l.gemm_nvfp4_blocked_scale_bytes.restype = ctypes.c_longlong
        l.gemm_nvfp4_pack_scales.argtypes = [P, P, I, I, P]
        l.gemm_nvfp4_pack_scales.restype = I
        l.gemm_nvfp4_blocked.argtypes = [P, P, P, P, P, I, I, I, P]
        l.gemm_nvfp4_blocked.restype = I
        l.gemm_nvfp4_blocked_ex.argtypes = [P, P, P, P, P, I, I, I, P, ctypes.POINTER(gemm_options_t)]
        l.gemm_nvfp4_blocked_ex.restype = I
        l.gemm_nvfp4_noalloc.argtypes = [P, P, P, P, P, I, I, I, P]
        l.gemm_nvfp4_noalloc.restype = I
        l.gemm_launch_count.argtypes = []
        l.gemm_launch_count.restype = ctypes.c_ulonglong
        l.gemm_measure_mma_rate.argtypes = [I, ctypes.POINTER(ctypes.c_double)]
        EP, OP = ctypes.POINTER(gemm_epilogue_t), ctypes.POINTER(gemm_options_t)
        l.gemm_bf16_fused.argtypes = [P, P, P, I, I, I, P, EP, OP]
        l.gemm_bf16_fused.restype = I
        l.gemm_nvfp4_fused.argtypes = [P, P, P, P, P, I, I, I, P, EP, OP]
        l.gemm_nvfp4_fused.restype = I
        l.gemm_nvfp4_blocked_fused.argtypes = [P, P, P, P, P, I, I, I, P, EP, OP]
        l.gemm_nvfp4_blocked_fused.restype = I
        l.gemm_bf16_plan.argtypes = [I, I, I, OP, EP, ctypes.POINTER(I), ctypes.POINTER(I)]
        l.gemm_bf16_plan.restype = I
        l.gemm_nvfp4_plan.argtypes = [I, I, I, OP, ctypes.POINTER(I)]
        l.gemm_nvfp4_plan.restype = I
        l.gemm_bf16_wide_rule.argtypes = [I, I, I, I]
        l.gemm_bf16_wide_rule.restype = I
        l.gemm_measure_mma_rate.restype = I
        F = ctypes.c_float
        l.gemm_rms_norm.argtypes = [P, P, P, P, P, P, P, I, I, F, I, P, ctypes.POINTER(gemm_norm_strides_t)]
        l.gemm_rms_norm.restype = I
        l.gemm_rms_norm_backward.argtypes = [P, P, P, P, P, P, P, I, I, P, ctypes.POINTER(gemm_norm_backward_strides_t)]
        l.gemm_rms_norm_backward.restype = I
        LL = ctypes.c_longlong
        l.gemm_token_logprobs.argtypes = [P, I, P, P, P, P, I, P, P, I, I, LL, F, P]
        l.gemm_token_logprobs.restype = I
        l.gemm_token_logprobs_backward.argtypes = [P, I, P, P, P, P, P, P, I, I, LL, LL, F, P]
        l.gemm_token_logprobs_backward.restype = I
        GS = ctypes.POINTER(gemm_glu_strides_t)
        l.gemm_glu_bf16.argtypes = [P, P, P, P, P, I, I, I, I, P, GS]
        l.gemm_glu_bf16.restype = I
        l.gemm_glu_e4m3.argtypes = [P, P, P, P, P, P, P, I, I, I, I, P, GS]
        l.gemm_glu_e4m3.restype = I
        l.gemm_glu_bf16_backward.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, P, GS]
        l.gemm_glu_bf16_backward.restype = I
        l.gemm_glu_plan.argtypes = [I, I, I, I, ctypes.POINTER(I), ctypes.POINTER(I)]
        l.gemm_glu_plan.restype = I
        NS, NB = ctypes.POINTER(gemm_norm_strides_t), ctypes.POINTER(gemm_norm_backward_strides_t)
        l.gemm_layer_norm.argtypes = [P, P, P, P, P, P, P, P, P, I, I, F, I, P, NS]
        l.gemm_layer_norm.restype = I
        l.gemm_layer_norm_backward.argtypes = [P, P, P, P, P, P, P, P, P, I, I, P, NB]
        l.gemm_layer_norm_backward.restype = I
        l.gemm_embedding.argtypes = [P, I, P, P, I, I, I, LL, LL, F, P]
        l.gemm_embedding.restype = I
        l.gemm_embedding_backward.argtypes = [P, I, P, P, P, I, I, I, I, LL, F, P]
        l.gemm_embedding_backward.restype = I
        CS = ctypes.POINTER(gemm_cross_entropy_strides_t)
        l.gemm_cross_entropy.argtypes = [P, P, P, P, P, I, I, I, F, P, CS]
        l.gemm_cross_entropy.restype = I
        l.gemm_cross_entropy_backward.argtypes = [P, P, P, P, P, P, P, P, I, I, I, F, ctypes.c_size_t, P, CS]
        l.gemm_cross_entropy_backward.restype = I
        l.gemm_cross_entropy_piece.argtypes = [I, I, ctypes.c_size_t]
        l.gemm_cross_entropy_piece.restype = I
        l.gemm_cross_entropy_plan.argtypes = [I, I, I, I, ctypes.c_size_t, I, I, ctypes.POINTER(I), ctypes.POINTER(I)]
        l.gemm_cross_entropy_plan.restype = I
        _lib = l
    return _lib


def _ptr(x) -> int:
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    return x.data_ptr()


_current_stream = None


def _find_current_stream():
    """A function without arguments that gives the handle of torch's current CUDA stream (0 without torch or a GPU).
    The raw-handle call skips the Stream object that current_stream() builds: 0.4 us instead of 3 us a call."""
    try:
        import torch
        raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), torch.cuda.current_device
        if raw is None:
            return lambda: torch.cuda.current_stream().cuda_stream
        raw(device())
        return lambda: raw(device())
    except Exception:
        return None


def _stream(stream) -> int:
    global _current_stream
    if stream is None:
        if _current_stream is None:
            _current_stream = _find_current_stream()
        return _current_stream() if _current_stream is not None else 0
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str) -> None:
    if status != GEMM_OK:
        raise GemmError(status, where)


def status_string(status: int) -> str:
    return lib().gemm_status_string(status).decode()


def gemm_bf16(A, B, C, M: int, N: int, K: int, stream=None, opts: gemm_options_t | None = None) -> None:
    """C[M,N] = A[M,K] @ B[N,K]^T in BF16 (FP32 accumulation); see include/gemm.h."""
    l = lib()
    if opts is None:
        st = l.gemm_bf16(_ptr(A), _ptr(B), _ptr(C), M, N, K, _stream(stream))
    else:
        st = l.gemm_bf16_ex(_ptr(A), _ptr(B), _ptr(C), M, N, K, _stream(stream), ctypes.byref(opts))
    _check(st, "gemm_bf16")


def gemm_nvfp4(A, SFA, B, SFB, C, M: int, N: int, K: int, stream=None, opts: gemm_options_t | None = None) -> None:
    """C[M,N] = dequant(A, SFA) @ dequant(B, SFB)^T for packed E2M1 with per-16 E4M3 scales."""
    l = lib()
    if opts is None:
        st = l.gemm_nvfp4(_ptr(A), _ptr(SFA), _ptr(B), _ptr(SFB), _ptr(C), M, N, K, _stream(stream))
    else:
        st = l.gemm_nvfp4_ex(_ptr(A), _ptr(SFA), _ptr(B), _ptr(SFB), _ptr(C), M, N, K, _stream(stream),
                             ctypes.byref(opts))
    _check(st, "gemm_nvfp4")


def nvfp4_blocked_scale_bytes(rows: int, K: int) -> int:
    n = lib().gemm_nvfp4_blocked_scale_bytes(rows, K)
    if n < 0:
        raise GemmError(GEMM_ERR_UNSUPPORTED_SHAPE, "gemm_nvfp4_blocked_scale_bytes")
    return n


def gemm_nvfp4_pack_scales(SF, SF_blocked, rows: int, K: int, stream=None) -> None:
    """Row-major scales [rows][K/16] -> the blocked tensor-core layout (see include/gemm.h)."""
    _check(lib().gemm_nvfp4_pack_scales(_ptr(SF), _ptr(SF_blocked), rows, K, _stream(stream)),
           "gemm_nvfp4_pack_scales")


def gemm_nvfp4_blocked(A, SFA_blocked, B, SFB_blocked, C, M: int, N: int, K: int, stream=None,
                       opts: gemm_options_t | None = None) -> None:
    """gemm_nvfp4 with scales already in the blocked layout (the fast path)."""
    l = lib()
    if opts is None:
        st = l.gemm_nvfp4_blocked(_ptr(A), _ptr(SFA_blocked), _ptr(B), _ptr(SFB_blocked), _ptr(C), M, N, K,
                                  _stream(stream))
    else:
        st = l.gemm_nvfp4_blocked_ex(_ptr(A), _ptr(SFA_blocked), _ptr(B), _ptr(SFB_blocked), _ptr(C), M, N, K,
                                     _stream(stream), ctypes.byref(opts))
    _check(st, "gemm_nvfp4_blocked")


def _byref_or_null(x):
    return None if x is None else ctypes.byref(x)


def gemm_bf16_fused(A, B, C, M: int, N: int, K: int, epi: gemm_epilogue_t | None = None, stream=None,
                    opts: gemm_options_t | None = None) -> None:
    """gemm_bf16 with the fused epilogue C = act(alpha * A B^T + beta * C + bias)."""
    _check(lib().gemm_bf16_fused(_ptr(A), _ptr(B), _ptr(C), M, N, K, _stream(stream), _byref_or_null(epi),
                                 _byref_or_null(opts)), "gemm_bf16_fused")


def gemm_nvfp4_fused(A, SFA, B, SFB, C, M: int, N: int, K: int, epi: gemm_epilogue_t | None = None, stream=None,
                     opts: gemm_options_t | None = None) -> None:
    """gemm_nvfp4 with the fused epilogue."""
    _check(lib().gemm_nvfp4_fused(_ptr(A), _ptr(SFA), _ptr(B), _ptr(SFB), _ptr(C), M, N, K, _stream(stream),
                                  _byref_or_null(epi), _byref_or_null(opts)), "gemm_nvfp4_fused")


def gemm_nvfp4_blocked_fused(A, SFA_blocked, B, SFB_blocked, C, M: int, N: int, K: int,
                             epi: gemm_epilogue_t | None = None, stream=None,
                             opts: gemm_options_t | None = None) -> None:
    """gemm_nvfp4_blocked with the fused epilogue."""
    _check(lib().gemm_nvfp4_blocked_fused(_ptr(A), _ptr(SFA_blocked), _ptr(B), _ptr(SFB_blocked), _ptr(C), M, N, K,
                                          _stream(stream), _byref_or_null(epi), _byref_or_null(opts)),
           "gemm_nvfp4_blocked_fused")


def bf16_plan(M: int, N: int, K: int, opts: gemm_options_t | None = None, epi: gemm_epilogue_t | None = None):
    """(swap_ab, tile_n) that gemm_bf16 uses for this problem (host only)."""
    swap, tile_n = ctypes.c_int(), ctypes.c_int()
    _check(lib().gemm_bf16_plan(M, N, K, _byref_or_null(opts), _byref_or_null(epi), ctypes.byref(swap),
                                ctypes.byref(tile_n)), "gemm_bf16_plan")
    return swap.value, tile_n.value


def bf16_wide_rule(M: int, N: int, K: int, wave: int = 76) -> bool:
    """Whether gemm_bf16's default kernel takes the 512 x 256 pair tile for this problem
    (static schedule, not swapped), with `wave` co-resident clusters."""
    r = lib().gemm_bf16_wide_rule(M, N, K, wave)
    if r < 0:
        raise GemmError(-r, "gemm_bf16_wide_rule")
    return r == 1


def nvfp4_plan(M: int, N: int, K: int, opts: gemm_options_t | None = None) -> int:
    """Rows of A the NVFP4 GEMM kernel reads for this problem: 32 when A is copied into a
    padded workspace first, else M (host only)."""
    a_rows = ctypes.c_int()
    _check(lib().gemm_nvfp4_plan(M, N, K, _byref_or_null(opts), ctypes.byref(a_rows)), "gemm_nvfp4_plan")
    return a_rows.value


def gemm_nvfp4_noalloc(A, SFA, B, SFB, C, M: int, N: int, K: int, stream=None) -> None:
    """gemm_nvfp4 without any device allocation: the rearranged scales live in a fixed
    16 MiB array inside the library (see include/gemm.h for the size limit and the
    rule that calls overlapping on the GPU must be ordered)."""
    _check(lib().gemm_nvfp4_noalloc(_ptr(A), _ptr(SFA), _ptr(B), _ptr(SFB), _ptr(C), M, N, K, _stream(stream)),
           "gemm_nvfp4_noalloc")


def get_device_status(stream=None) -> tuple[int, int]:
    """(status, detail word) reported by kernels since the last call; synchronises the stream."""
    detail = ctypes.c_uint32(0)
    st = lib().gemm_get_device_status(_stream(stream), ctypes.byref(detail))
    return st, detail.value


def tile_coord(M, N, tile_m, tile_n, group_m, t) -> tuple[int, int]:
    mb, nb = ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().gemm_tile_coord(M, N, tile_m, tile_n, group_m, t, ctypes.byref(mb), ctypes.byref(nb)),
           "gemm_tile_coord")
    return mb.value, nb.value


def choose_group_m(M, N, K, tile_m, tile_n, elem_bytes_x2, concurrent_tiles, l2_bytes) -> int:
    g = lib().gemm_choose_group_m(M, N, K, tile_m, tile_n, elem_bytes_x2, concurrent_tiles, l2_bytes)
    if g < 0:
        raise GemmError(-g, "gemm_choose_group_m")
    return g


def clc_rule(items: int, wave: int, K: int, nvfp4: bool = False) -> bool:
    """Whether a persistent launch with the default options schedules its items with cluster launch control."""
    r = lib().gemm_clc_rule(items, wave, K, int(nvfp4))
    if r < 0:
        raise GemmError(-r, "gemm_clc_rule")
    return r == 1


def launch_count() -> int:
    return lib().gemm_launch_count()


GEMM_MMA_BF16 = 0
GEMM_MMA_NVFP4 = 1
GEMM_MMA_NVFP4_1CTA_N128 = 2
GEMM_MMA_NVFP4_1CTA_N192 = 3
GEMM_MMA_NVFP4_1CTA_N256 = 4
GEMM_MMA_NVFP4_PAIR_N128 = 5
GEMM_MMA_NVFP4_PAIR_N128_2ACC = 6
GEMM_MMA_MXF4_PAIR_N256 = 7


def measure_mma_rate(kind: int) -> float:
    """FLOP per SM clock of back-to-back M=256 N=256 MMAs of `kind` on the current device."""
    out = ctypes.c_double(0.0)
    _check(lib().gemm_measure_mma_rate(kind, ctypes.byref(out)), "gemm_measure_mma_rate")
    return out.value


def gemm_rms_norm(X, R, W, S, Y, scales, rstd, rows: int, cols: int, eps: float, fmt: int = GEMM_NORM_BF16,
                  stream=None, strides: gemm_norm_strides_t | None = None) -> None:
    """s = bf16(X + R), Y = s / sqrt(mean(s^2) + eps) * W in one of three formats; see include/gemm.h."""
    _check(lib().gemm_rms_norm(_ptr(X), _ptr(R), _ptr(W), _ptr(S), _ptr(Y), _ptr(scales), _ptr(rstd), rows, cols, eps,
                               fmt, _stream(stream), _byref_or_null(strides)), "gemm_rms_norm")


def gemm_rms_norm_backward(dY, S, W, rstd, dS, dX, dW, rows: int, cols: int, stream=None,
                           strides: gemm_norm_backward_strides_t | None = None) -> None:
    """Gradient of gemm_rms_norm's BF16 form; see include/gemm.h."""
    _check(lib().gemm_rms_norm_backward(_ptr(dY), _ptr(S), _ptr(W), _ptr(rstd), _ptr(dS), _ptr(dX), _ptr(dW), rows,
                                        cols, _stream(stream), _byref_or_null(strides)), "gemm_rms_norm_backward")


def gemm_token_logprobs(logits, kind: int, tokens, logprob, entropy, lse, top: int, top_logprobs, top_ids, rows: int,
                        vocab: int, ld: int = 0, scale: float = 1.0, stream=None) -> None:
    """Log probabilities of given tokens, entropy and the `top` alternatives of each row; see include/gemm.h."""
    _check(lib().gemm_token_logprobs(_ptr(logits), kind, _ptr(tokens), _ptr(logprob), _ptr(entropy), _ptr(lse), top,
                                     _ptr(top_logprobs), _ptr(top_ids), rows, vocab, ld, scale, _stream(stream)),
           "gemm_token_logprobs")


def gemm_token_logprobs_backward(logits, kind: int, tokens, lse, entropy, dlogprob, dentropy, dlogits, rows: int,
                                 vocab: int, ld: int = 0, ldd: int = 0, scale: float = 1.0, stream=None) -> None:
    """Gradient of logprob and entropy with respect to the logits; see include/gemm.h."""
    _check(lib().gemm_token_logprobs_backward(_ptr(logits), kind, _ptr(tokens), _ptr(lse), _ptr(entropy),
                                              _ptr(dlogprob), _ptr(dentropy), _ptr(dlogits), rows, vocab, ld, ldd,
                                              scale, _stream(stream)), "gemm_token_logprobs_backward")


def gemm_glu_bf16(X, Wg, Wu, H, preact, M: int, N: int, K: int, act: int = GEMM_GLU_SILU, stream=None,
                  strides: gemm_glu_strides_t | None = None) -> None:
    """H = act(X Wg^T) * (X Wu^T) in BF16, keeping [g | u] in preact if given; see include/gemm.h."""
    _check(lib().gemm_glu_bf16(_ptr(X), _ptr(Wg), _ptr(Wu), _ptr(H), _ptr(preact), M, N, K, act, _stream(stream),
                               _byref_or_null(strides)), "gemm_glu_bf16")


def gemm_glu_e4m3(X, x_scale, Wg, wg_scale, Wu, wu_scale, H, M: int, N: int, K: int, act: int = GEMM_GLU_SILU,
                  stream=None, strides: gemm_glu_strides_t | None = None) -> None:
    """gemm_glu_bf16 from E4M3 operands with a scale per row; see include/gemm.h."""
    _check(lib().gemm_glu_e4m3(_ptr(X), _ptr(x_scale), _ptr(Wg), _ptr(wg_scale), _ptr(Wu), _ptr(wu_scale), _ptr(H), M,
                               N, K, act, _stream(stream), _byref_or_null(strides)), "gemm_glu_e4m3")


def gemm_glu_bf16_backward(dH, X, Wg, Wu, preact, dX, dWg, dWu, M: int, N: int, K: int, act: int = GEMM_GLU_SILU,
                           stream=None, strides: gemm_glu_strides_t | None = None) -> None:
    """Gradient of gemm_glu_bf16; see include/gemm.h."""
    _check(lib().gemm_glu_bf16_backward(_ptr(dH), _ptr(X), _ptr(Wg), _ptr(Wu), _ptr(preact), _ptr(dX), _ptr(dWg),
                                        _ptr(dWu), M, N, K, act, _stream(stream), _byref_or_null(strides)),
           "gemm_glu_bf16_backward")


def glu_plan(M: int, N: int, K: int, wave: int = 76) -> tuple[int, int]:
    """Rows of the pair tile that glu_bf16 (0: the kernel for few rows) and its gradient use for this problem (host only)."""
    fwd, bwd = ctypes.c_int(), ctypes.c_int()
    _check(lib().gemm_glu_plan(M, N, K, wave, ctypes.byref(fwd), ctypes.byref(bwd)), "gemm_glu_plan")
    return fwd.value, bwd.value


def gemm_layer_norm(X, R, W, B, S, Y, scales, mean, rstd, rows: int, cols: int, eps: float, fmt: int = GEMM_NORM_BF16,
                    stream=None, strides: gemm_norm_strides_t | None = None) -> None:
    """s = bf16(X + R), Y = (s - mean) / sqrt(var + eps) * W + B in one of three formats; see include/gemm.h."""
    _check(lib().gemm_layer_norm(_ptr(X), _ptr(R), _ptr(W), _ptr(B), _ptr(S), _ptr(Y), _ptr(scales), _ptr(mean),
                                 _ptr(rstd), rows, cols, eps, fmt, _stream(stream), _byref_or_null(strides)),
           "gemm_layer_norm")


def gemm_layer_norm_backward(dY, S, W, mean, rstd, dS, dX, dW, dB, rows: int, cols: int, stream=None,
                             strides: gemm_norm_backward_strides_t | None = None) -> None:
    """Gradient of gemm_layer_norm's BF16 form; see include/gemm.h."""
    _check(lib().gemm_layer_norm_backward(_ptr(dY), _ptr(S), _ptr(W), _ptr(mean), _ptr(rstd), _ptr(dS), _ptr(dX),
                                          _ptr(dW), _ptr(dB), rows, cols, _stream(stream), _byref_or_null(strides)),
           "gemm_layer_norm_backward")


def gemm_embedding(table, kind: int, tokens, Y, rows: int, vocab: int, cols: int, ldt: int = 0, ldy: int = 0,
                   scale: float = 1.0, stream=None) -> None:
    """Y[i] = scale * table[tokens[i]]; see include/gemm.h."""
    _check(lib().gemm_embedding(_ptr(table), kind, _ptr(tokens), _ptr(Y), rows, vocab, cols, ldt, ldy, scale,
                                _stream(stream)), "gemm_embedding")


def gemm_embedding_backward(dY, dy_kind: int, tokens, base, dtable, table_kind: int, rows: int, vocab: int, cols: int,
                            ldd: int = 0, scale: float = 1.0, stream=None) -> None:
    """dtable[v] = base[v] + scale * sum of dY over the positions of token v; see include/gemm.h."""
    _check(lib().gemm_embedding_backward(_ptr(dY), dy_kind, _ptr(tokens), _ptr(base), _ptr(dtable), table_kind, rows,
                                         vocab, cols, ldd, scale, _stream(stream)), "gemm_embedding_backward")


def gemm_cross_entropy(X, W, targets, loss, lse, M: int, vocab: int, K: int, scale: float = 1.0, stream=None,
                       strides: gemm_cross_entropy_strides_t | None = None) -> None:
    """Softmax cross entropy of X W^T against targets, without storing the logits; see include/gemm.h."""
    _check(lib().gemm_cross_entropy(_ptr(X), _ptr(W), _ptr(targets), _ptr(loss), _ptr(lse), M, vocab, K, scale,
                                    _stream(stream), _byref_or_null(strides)), "gemm_cross_entropy")


def gemm_cross_entropy_backward(X, W, targets, lse, dloss, dlse, dX, dW, M: int, vocab: int, K: int, scale: float = 1.0,
                                workspace: int = 0, stream=None,
                                strides: gemm_cross_entropy_strides_t | None = None) -> None:
    """Gradient of gemm_cross_entropy; see include/gemm.h."""
    _check(lib().gemm_cross_entropy_backward(_ptr(X), _ptr(W), _ptr(targets), _ptr(lse), _ptr(dloss), _ptr(dlse),
                                             _ptr(dX), _ptr(dW), M, vocab, K, scale, workspace, _stream(stream),
                                             _byref_or_null(strides)), "gemm_cross_entropy_backward")


def cross_entropy_piece(M: int, vocab: int, workspace: int = 0) -> int:
    """Columns of the vocabulary that the gradient of cross_entropy takes at a time (host only)."""
    n = lib().gemm_cross_entropy_piece(M, vocab, workspace)
    if n < 0:
        raise GemmError(-n, "gemm_cross_entropy_piece")
    return n


def cross_entropy_plan(M: int, vocab: int, K: int, workspace: int = 0, input_grad: bool = True, weight_grad: bool = True,
                       wave: int = 76) -> tuple[int, bool]:
    """(rows of the pair tile of the gradient's products, whether a contiguous X is copied) of cross_entropy_backward for
    this problem (host only)."""
    rows, copy = ctypes.c_int(), ctypes.c_int()
    _check(lib().gemm_cross_entropy_plan(M, vocab, K, wave, workspace, input_grad, weight_grad, ctypes.byref(rows),
                                         ctypes.byref(copy)), "gemm_cross_entropy_plan")
    return rows.value, bool(copy.value)


# ---------------------------------------------------------------- torch-tensor conveniences
# `stream`: a torch stream or a handle; torch's current stream if it is None. The matrix products allocate `out`, where it
# is not given, on the current stream; the operators allocate on `stream` (see _on_stream).

def matmul_bf16(A, B, out=None, stream=None, opts=None):
    """A (M x K) and B (N x K) BF16 CUDA tensors -> C = A @ B^T (M x N BF16)."""
    import torch
    M, K = A.shape
    N = B.shape[0]
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=A.device)
    gemm_bf16(A, B, out, M, N, K, stream, opts)
    return out


def pack_scales(SF, stream=None):
    """Row-major E4M3 scales (rows x K/16 uint8 CUDA tensor) -> blocked-layout uint8 tensor."""
    import torch
    rows, kb = SF.shape
    K = 16 * kb
    out = torch.empty(nvfp4_blocked_scale_bytes(rows, K), dtype=torch.uint8, device=SF.device)
    gemm_nvfp4_pack_scales(SF, out, rows, K, stream)
    return out


def matmul_nvfp4_blocked(A, SFA_blocked, B, SFB_blocked, out=None, stream=None, opts=None):
    """Like matmul_nvfp4, with scales from pack_scales."""
    import torch
    M = A.shape[0]
    N = B.shape[0]
    K = 2 * A.shape[1]
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=A.device)
    gemm_nvfp4_blocked(A, SFA_blocked, B, SFB_blocked, out, M, N, K, stream, opts)
    return out


def matmul_nvfp4(A, SFA, B, SFB, out=None, stream=None, opts=None):
    """Packed E2M1 A (M x K/2), B (N x K/2) with E4M3 scales (M x K/16, N x K/16) -> BF16 C."""
    import torch
    M = A.shape[0]
    N = B.shape[0]
    K = 2 * A.shape[1]
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=A.device)
    gemm_nvfp4(A, SFA, B, SFB, out, M, N, K, stream, opts)
    return out


_device = None


def _elsewhere(t) -> bool:
    """Whether a CUDA tensor lies on another device than the current one, on which the call would run."""
    global _device
    if _device is None:
        import torch
        _device = torch._C._cuda_getDevice
    return t.get_device() != _device()


_MOST = 0x7FFFFFFF  # sizes of the library's calls have 32 bits (ctypes would cut a larger one without a word)


def _matrix(t, what, dtype, shape=None):
    """A CUDA matrix of `dtype` on the current device whose rows are contiguous -> its row stride (0: rows follow one
    another)."""
    if t is None:
        raise ValueError(f"{what}: a CUDA {dtype} matrix is needed, got None")
    size = t.shape
    if t.dtype is not dtype or len(size) != 2 or not t.is_cuda or (shape is not None and size != shape):
        want = "" if shape is None else f" of shape {tuple(shape)}"
        raise ValueError(f"{what}: a CUDA {dtype} matrix{want} is needed, got {t.dtype} {tuple(size)} on {t.device}")
    if size[0] > _MOST or size[1] > _MOST:
        raise ValueError(f"{what}: sizes below 2^31 are needed, got {tuple(size)}")
    if _elsewhere(t):
        raise ValueError(f"{what}: lies on {t.device}, which is not the current device")
    if t.is_contiguous():
        return 0
    rows, cols = size
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{what}: the elements of a row must be contiguous (strides {t.stride()})")
    if rows <= 1 or cols == 0 or t.stride(0) == cols:
        return 0
    if t.stride(0) < cols:
        raise ValueError(f"{what}: rows must not overlap (strides {t.stride()})")
    return t.stride(0)


def _address(t):
    """A tensor's device address, or NULL for None (the conveniences call the library directly: 2 us less a call)."""
    return None if t is None else t.data_ptr()


def _vector(t, what, dtype, n):
    if t is None:
        raise ValueError(f"{what}: a CUDA {dtype} vector of {n} is needed, got None")
    if t.dtype is not dtype or t.shape != (n,) or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous CUDA {dtype} vector of {n} is needed, got {t.dtype} {tuple(t.shape)}")
    if n > _MOST:
        raise ValueError(f"{what}: sizes below 2^31 are needed, got {n}")
    if _elsewhere(t):
        raise ValueError(f"{what}: lies on {t.device}, which is not the current device")
    return t


def _on_stream(stream, call, *args):
    """call(*args) on `stream` (a torch stream, a handle or an object that has one), as under torch.cuda.stream: what it
    allocates is that stream's memory. Its tensors are recorded on the streams that use them, so none is given away while
    a kernel still reads or writes it; that its inputs are ready on `stream`, and its outputs where they are read, is the
    caller's to order."""
    import torch
    here = torch.cuda.current_stream()
    handle = _stream(stream)
    if handle == here.cuda_stream:
        return call(*args)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        got = call(*args)
    for t in args:
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)
    for t in (got,) if isinstance(got, torch.Tensor) else got:
        if t is not None:
            t.record_stream(here)
    return got


class NormOutput(NamedTuple):
    """y: BF16, float8_e4m3fn, or packed E2M1 bytes; scales: None, FP32 a row, or E4M3 bytes per 16;
    sum: the residual stream after the addition; rstd: FP32 a row, or None."""
    y: object
    scales: object
    sum: object
    rstd: object


_NORM_FORMATS = {"bf16": GEMM_NORM_BF16, "e4m3": GEMM_NORM_E4M3, "nvfp4": GEMM_NORM_NVFP4}


def rms_norm(x, weight=None, residual=None, eps: float = 1e-5, out: str = "bf16", save: bool = False,
             inplace: bool = False, stream=None) -> NormOutput:
    """RMS norm of the rows of x + residual (rows x cols BF16). `out`: "bf16", "e4m3" (scales: FP32 a row)
    or "nvfp4" (y and scales are A and SFA of matmul_nvfp4). `save`: keep rstd for rms_norm_backward.
    `inplace`: the sum overwrites `residual`."""
    if stream is not None:
        return _on_stream(stream, rms_norm, x, weight, residual, eps, out, save, inplace)
    import torch
    fmt = _NORM_FORMATS.get(out)
    if fmt is None:
        raise ValueError(f"out: one of {sorted(_NORM_FORMATS)} is needed, got {out!r}")
    bf16 = torch.bfloat16
    ldx, ldr, lds = _matrix(x, "x", bf16), 0, 0
    size = x.shape
    rows, cols = size
    total, written = x, None
    if residual is not None:
        ldr = _matrix(residual, "residual", bf16, size)
        if inplace:
            total, lds = residual, ldr
        else:
            total = torch.empty_like(x, memory_format=torch.contiguous_format)
        written = total
    elif inplace:
        raise ValueError("inplace: there is no residual to overwrite")
    if weight is not None:
        _vector(weight, "weight", bf16, cols)
    scales = rstd = strides = None
    if fmt == GEMM_NORM_BF16:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
    elif fmt == GEMM_NORM_E4M3:
        y = torch.empty_like(x, dtype=torch.float8_e4m3fn, memory_format=torch.contiguous_format)
        scales = torch.empty(rows, dtype=torch.float32, device=x.device)
    else:
        y = torch.empty((rows, cols // 2), dtype=torch.uint8, device=x.device)
        scales = torch.empty((rows, cols // 16), dtype=torch.uint8, device=x.device)
    if save:
        rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
    if ldx or ldr or lds:
        strides = gemm_norm_strides_t(ldx, ldr, lds, 0)
    status = lib().gemm_rms_norm(x.data_ptr(), _address(residual), _address(weight), _address(written), y.data_ptr(),
                                 _address(scales), _address(rstd), rows, cols, eps, fmt, _stream(None),
                                 _byref_or_null(strides))
    if status:
        raise GemmError(status, "gemm_rms_norm")
    return NormOutput(y, scales, total, rstd)


def rms_norm_backward(dy, total, weight, rstd, dsum=None, weight_grad: bool = True, stream=None):
    """(dx, dweight) of rms_norm with BF16 output: `total` and `rstd` are NormOutput.sum and .rstd, `dsum` the
    gradient that reaches the sum past the norm. dx is the gradient of x and of the residual; dweight is FP32."""
    if stream is not None:
        return _on_stream(stream, rms_norm_backward, dy, total, weight, rstd, dsum, weight_grad)
    import torch
    bf16 = torch.bfloat16
    lds = _matrix(total, "total", bf16)
    rows, cols = total.shape
    lddy = _matrix(dy, "dy", bf16, total.shape)
    ldds = _matrix(dsum, "dsum", bf16, total.shape) if dsum is not None else 0
    _vector(rstd, "rstd", torch.float32, rows)
    if weight is not None:
        _vector(weight, "weight", bf16, cols)
    dx = torch.empty_like(dy, memory_format=torch.contiguous_format)
    dw = torch.empty(cols, dtype=torch.float32, device=dy.device) if weight_grad else None
    strides = gemm_norm_backward_strides_t(lddy, lds, ldds, 0) if lddy or lds or ldds else None
    status = lib().gemm_rms_norm_backward(dy.data_ptr(), total.data_ptr(), _address(weight), rstd.data_ptr(),
                                          _address(dsum), dx.data_ptr(), _address(dw), rows, cols, _stream(None),
                                          _byref_or_null(strides))
    if status:
        raise GemmError(status, "gemm_rms_norm_backward")
    return dx, dw


class LayerNormOutput(NamedTuple):
    """As NormOutput, with the rows' means: mean and rstd are FP32 a row, or None."""
    y: object
    scales: object
    sum: object
    mean: object
    rstd: object


def layer_norm(x, weight=None, bias=None, residual=None, eps: float = 1e-5, out: str = "bf16", save: bool = False,
               inplace: bool = False, stream=None) -> LayerNormOutput:
    """Layer norm of the rows of x + residual (rows x cols BF16). `out`: "bf16", "e4m3" (scales: FP32 a row) or "nvfp4"
    (y and scales are A and SFA of matmul_nvfp4). `save`: keep mean and rstd for layer_norm_backward. `inplace`: the sum
    overwrites `residual`."""
    if stream is not None:
        return _on_stream(stream, layer_norm, x, weight, bias, residual, eps, out, save, inplace)
    import torch
    fmt = _NORM_FORMATS.get(out)
    if fmt is None:
        raise ValueError(f"out: one of {sorted(_NORM_FORMATS)} is needed, got {out!r}")
    bf16 = torch.bfloat16
    ldx, ldr, lds = _matrix(x, "x", bf16), 0, 0
    size = x.shape
    rows, cols = size
    total, written = x, None
    if residual is not None:
        ldr = _matrix(residual, "residual", bf16, size)
        if inplace:
            total, lds = residual, ldr
        else:
            total = torch.empty_like(x, memory_format=torch.contiguous_format)
        written = total
    elif inplace:
        raise ValueError("inplace: there is no residual to overwrite")
    if weight is not None:
        _vector(weight, "weight", bf16, cols)
    if bias is not None:
        _vector(bias, "bias", bf16, cols)
    scales = mean = rstd = strides = None
    if fmt == GEMM_NORM_BF16:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
    elif fmt == GEMM_NORM_E4M3:
        y = torch.empty_like(x, dtype=torch.float8_e4m3fn, memory_format=torch.contiguous_format)
        scales = torch.empty(rows, dtype=torch.float32, device=x.device)
    else:
        y = torch.empty((rows, cols // 2), dtype=torch.uint8, device=x.device)
        scales = torch.empty((rows, cols // 16), dtype=torch.uint8, device=x.device)
    if save:
        mean = torch.empty(rows, dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
    if ldx or ldr or lds:
        strides = gemm_norm_strides_t(ldx, ldr, lds, 0)
    status = lib().gemm_layer_norm(x.data_ptr(), _address(residual), _address(weight), _address(bias), _address(written),
                                   y.data_ptr(), _address(scales), _address(mean), _address(rstd), rows, cols, eps, fmt,
                                   _stream(None), _byref_or_null(strides))
    if status:
        raise GemmError(status, "gemm_layer_norm")
    return LayerNormOutput(y, scales, total, mean, rstd)


def layer_norm_backward(dy, total, weight, mean, rstd, dsum=None, weight_grads: bool = True, stream=None):
    """(dx, dweight, dbias) of layer_norm with BF16 output: `total`, `mean` and `rstd` are LayerNormOutput.sum, .mean and
    .rstd, `dsum` the gradient that reaches the sum past the norm. dx is the gradient of x and of the residual; dweight
    and dbias are FP32 (None without weight_grads)."""
    if stream is not None:
        return _on_stream(stream, layer_norm_backward, dy, total, weight, mean, rstd, dsum, weight_grads)
    import torch
    bf16 = torch.bfloat16
    lds = _matrix(total, "total", bf16)
    rows, cols = total.shape
    lddy = _matrix(dy, "dy", bf16, total.shape)
    ldds = _matrix(dsum, "dsum", bf16, total.shape) if dsum is not None else 0
    _vector(mean, "mean", torch.float32, rows)
    _vector(rstd, "rstd", torch.float32, rows)
    if weight is not None:
        _vector(weight, "weight", bf16, cols)
    dx = torch.empty_like(dy, memory_format=torch.contiguous_format)
    dw = torch.empty(cols, dtype=torch.float32, device=dy.device) if weight_grads else None
    db = torch.empty_like(dw) if weight_grads else None
    strides = gemm_norm_backward_strides_t(lddy, lds, ldds, 0) if lddy or lds or ldds else None
    status = lib().gemm_layer_norm_backward(dy.data_ptr(), total.data_ptr(), _address(weight), mean.data_ptr(),
                                            rstd.data_ptr(), _address(dsum), dx.data_ptr(), _address(dw), _address(db),
                                            rows, cols, _stream(None), _byref_or_null(strides))
    if status:
        raise GemmError(status, "gemm_layer_norm_backward")
    return dx, dw, db


class TokenLogprobs(NamedTuple):
    """FP32 per row: logprob (None without tokens), entropy, lse; rows x top: top_logprobs (FP32), top_ids (int32)."""
    logprob: object
    entropy: object
    lse: object
    top_logprobs: object
    top_ids: object


def _logits_kind(logits):
    import torch
    if logits.dtype == torch.bfloat16:
        return GEMM_LOGITS_BF16
    if logits.dtype == torch.float32:
        return GEMM_LOGITS_F32
    raise ValueError(f"logits: BF16 or FP32 is needed, got {logits.dtype}")


def token_logprobs(logits, tokens=None, top: int = 0, scale: float = 1.0, stream=None) -> TokenLogprobs:
    """Log probabilities of `tokens` (rows int64; negative: none) under softmax(scale * logits) of each row, the
    entropy, and the `top` most likely alternatives (equal logits: the lower index first)."""
    if stream is not None:
        return _on_stream(stream, token_logprobs, logits, tokens, top, scale)
    import torch
    kind = _logits_kind(logits)
    ld = _matrix(logits, "logits", logits.dtype)
    rows, vocab = logits.shape
    if tokens is not None:
        _vector(tokens, "tokens", torch.int64, rows)
    lse = torch.empty(rows, dtype=torch.float32, device=logits.device)
    entropy = torch.empty_like(lse)
    logprob = torch.empty_like(lse) if tokens is not None else None
    top_logprobs = top_ids = None
    if top > 0:
        top_logprobs = torch.empty((rows, top), dtype=torch.float32, device=logits.device)
        top_ids = torch.empty((rows, top), dtype=torch.int32, device=logits.device)
    status = lib().gemm_token_logprobs(logits.data_ptr(), kind, _address(tokens), _address(logprob), entropy.data_ptr(),
                                       lse.data_ptr(), top, _address(top_logprobs), _address(top_ids), rows, vocab, ld,
                                       scale, _stream(None))
    if status:
        raise GemmError(status, "gemm_token_logprobs")
    return TokenLogprobs(logprob, entropy, lse, top_logprobs, top_ids)


def token_logprobs_backward(logits, tokens, lse, entropy, dlogprob, dentropy=None, scale: float = 1.0,
                            inplace: bool = False, stream=None):
    """dlogits of token_logprobs, in the type of the logits; `inplace` overwrites them. tokens and dlogprob may
    both be None, and dentropy."""
    if stream is not None:
        return _on_stream(stream, token_logprobs_backward, logits, tokens, lse, entropy, dlogprob, dentropy, scale,
                          inplace)
    import torch
    kind = _logits_kind(logits)
    ld = _matrix(logits, "logits", logits.dtype)
    rows, vocab = logits.shape
    _vector(lse, "lse", torch.float32, rows)
    for t, what, dtype in ((tokens, "tokens", torch.int64), (entropy, "entropy", torch.float32),
                           (dlogprob, "dlogprob", torch.float32), (dentropy, "dentropy", torch.float32)):
        if t is not None:
            _vector(t, what, dtype, rows)
    dlogits = logits if inplace else torch.empty((rows, vocab), dtype=logits.dtype, device=logits.device)
    status = lib().gemm_token_logprobs_backward(logits.data_ptr(), kind, _address(tokens), lse.data_ptr(),
                                                _address(entropy), _address(dlogprob), _address(dentropy),
                                                dlogits.data_ptr(), rows, vocab, ld, ld if inplace else 0, scale,
                                                _stream(None))
    if status:
        raise GemmError(status, "gemm_token_logprobs_backward")
    return dlogits


_GLU_ACTS = {"silu": GEMM_GLU_SILU, "gelu_tanh": GEMM_GLU_GELU_TANH, "relu": GEMM_GLU_RELU}


def _glu_act(act):
    if act not in _GLU_ACTS:
        raise ValueError(f"act: one of {sorted(_GLU_ACTS)} is needed, got {act!r}")
    return _GLU_ACTS[act]


def _contiguous(t, what, dtype, shape):
    if _matrix(t, what, dtype, shape):
        raise ValueError(f"{what}: rows must follow one another (strides {t.stride()})")
    return t


def glu_bf16(x, wg, wu, act: str = "silu", save: bool = False, stream=None):
    """act(x wg^T) * (x wu^T) for BF16 x (M x K), wg and wu (N x K) -> M x N BF16. `save`: also what
    glu_bf16_backward needs, as (h, saved)."""
    if stream is not None:
        return _on_stream(stream, glu_bf16, x, wg, wu, act, save)
    import torch
    kind, bf16 = _glu_act(act), torch.bfloat16
    ldx = _matrix(x, "x", bf16)
    M, K = x.shape
    N = wg.shape[0]
    _contiguous(wg, "wg", bf16, (N, K))
    _contiguous(wu, "wu", bf16, (N, K))
    h = torch.empty((M, N), dtype=bf16, device=x.device)
    saved = torch.empty((M, 2 * N), dtype=torch.float32, device=x.device) if save else None
    status = lib().gemm_glu_bf16(x.data_ptr(), wg.data_ptr(), wu.data_ptr(), h.data_ptr(), _address(saved), M, N, K, kind,
                                 _stream(None), gemm_glu_strides_t(ldx, 0, 0, 0) if ldx else None)
    if status:
        raise GemmError(status, "gemm_glu_bf16")
    return (h, saved) if save else h


def glu_e4m3(x, x_scale, wg, wg_scale, wu, wu_scale, act: str = "silu", stream=None):
    """glu_bf16 from float8_e4m3fn operands with an FP32 scale per row (x: rms_norm(..., out="e4m3"))."""
    if stream is not None:
        return _on_stream(stream, glu_e4m3, x, x_scale, wg, wg_scale, wu, wu_scale, act)
    import torch
    kind, e4m3 = _glu_act(act), torch.float8_e4m3fn
    ldx = _matrix(x, "x", e4m3)
    M, K = x.shape
    N = wg.shape[0]
    _contiguous(wg, "wg", e4m3, (N, K))
    _contiguous(wu, "wu", e4m3, (N, K))
    for t, what, n in ((x_scale, "x_scale", M), (wg_scale, "wg_scale", N), (wu_scale, "wu_scale", N)):
        _vector(t, what, torch.float32, n)
    h = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    status = lib().gemm_glu_e4m3(x.data_ptr(), x_scale.data_ptr(), wg.data_ptr(), wg_scale.data_ptr(), wu.data_ptr(),
                                 wu_scale.data_ptr(), h.data_ptr(), M, N, K, kind, _stream(None),
                                 gemm_glu_strides_t(ldx, 0, 0, 0) if ldx else None)
    if status:
        raise GemmError(status, "gemm_glu_e4m3")
    return h


def glu_bf16_backward(dh, x, wg, wu, saved, act: str = "silu", input_grad: bool = True, weight_grads: bool = True,
                      stream=None):
    """(dx, dwg, dwu) of glu_bf16(..., save=True); None in the place of a gradient that is not asked for."""
    if stream is not None:
        return _on_stream(stream, glu_bf16_backward, dh, x, wg, wu, saved, act, input_grad, weight_grads)
    import torch
    kind, bf16 = _glu_act(act), torch.bfloat16
    ldx = _matrix(x, "x", bf16)
    M, K = x.shape
    N = wg.shape[0]
    lddh = _matrix(dh, "dh", bf16, (M, N))
    _contiguous(wg, "wg", bf16, (N, K))
    _contiguous(wu, "wu", bf16, (N, K))
    _contiguous(saved, "saved", torch.float32, (M, 2 * N))
    dx = torch.empty((M, K), dtype=bf16, device=x.device) if input_grad else None
    dwg = torch.empty_like(wg) if weight_grads else None
    dwu = torch.empty_like(wg) if weight_grads else None
    status = lib().gemm_glu_bf16_backward(dh.data_ptr(), x.data_ptr(), wg.data_ptr(), wu.data_ptr(), saved.data_ptr(),
                                          _address(dx), _address(dwg), _address(dwu), M, N, K, kind, _stream(None),
                                          gemm_glu_strides_t(ldx, 0, lddh, 0) if ldx or lddh else None)
    if status:
        raise GemmError(status, "gemm_glu_bf16_backward")
    return dx, dwg, dwu


class CrossEntropy(NamedTuple):
    """FP32 per row: loss (None without targets; 0 where there is none), lse."""
    loss: object
    lse: object


def cross_entropy(x, head, targets=None, scale: float = 1.0, stream=None) -> CrossEntropy:
    """Softmax cross entropy of scale * x head^T (x: rows x width, head: vocab x width, BF16) against `targets` (rows
    int64; negative: none), without storing the logits."""
    if stream is not None:
        return _on_stream(stream, cross_entropy, x, head, targets, scale)
    import torch
    bf16 = torch.bfloat16
    ldx = _matrix(x, "x", bf16)
    rows, width = x.shape
    _contiguous(head, "head", bf16, None)
    vocab = head.shape[0]
    if head.shape[1] != width:
        raise ValueError(f"head: rows of {width} are needed, got {tuple(head.shape)}")
    if targets is not None:
        _vector(targets, "targets", torch.int64, rows)
    lse = torch.empty(rows, dtype=torch.float32, device=x.device)
    loss = torch.empty_like(lse) if targets is not None else None
    status = lib().gemm_cross_entropy(x.data_ptr(), head.data_ptr(), _address(targets), _address(loss), lse.data_ptr(),
                                      rows, vocab, width, scale, _stream(None),
                                      gemm_cross_entropy_strides_t(ldx, 0) if ldx else None)
    if status:
        raise GemmError(status, "gemm_cross_entropy")
    return CrossEntropy(loss, lse)


def cross_entropy_backward(x, head, targets, lse, dloss, dlse=None, scale: float = 1.0, input_grad: bool = True,
                           weight_grad: bool = True, workspace: int = 0, stream=None):
    """(dx, dhead) of cross_entropy, BF16; None in the place of a gradient that is not asked for. targets and dloss may
    both be None, and dlse. `workspace`: bytes that a piece of the logits' gradient may take (0: 512 MiB)."""
    if stream is not None:
        return _on_stream(stream, cross_entropy_backward, x, head, targets, lse, dloss, dlse, scale, input_grad,
                          weight_grad, workspace)
    import torch
    bf16 = torch.bfloat16
    ldx = _matrix(x, "x", bf16)
    rows, width = x.shape
    _contiguous(head, "head", bf16, None)
    vocab = head.shape[0]
    if head.shape[1] != width:
        raise ValueError(f"head: rows of {width} are needed, got {tuple(head.shape)}")
    if workspace < 0:
        raise ValueError(f"workspace: bytes, or 0, are needed, got {workspace}")
    _vector(lse, "lse", torch.float32, rows)
    for t, what, dtype in ((targets, "targets", torch.int64), (dloss, "dloss", torch.float32),
                           (dlse, "dlse", torch.float32)):
        if t is not None:
            _vector(t, what, dtype, rows)
    dx = torch.empty((rows, width), dtype=bf16, device=x.device) if input_grad else None
    dhead = torch.empty_like(head) if weight_grad else None
    status = lib().gemm_cross_entropy_backward(x.data_ptr(), head.data_ptr(), _address(targets), lse.data_ptr(),
                                               _address(dloss), _address(dlse), _address(dx), _address(dhead), rows,
                                               vocab, width, scale, workspace, _stream(None),
                                               gemm_cross_entropy_strides_t(ldx, 0) if ldx else None)
    if status:
        raise GemmError(status, "gemm_cross_entropy_backward")
    return dx, dhead


def _table_kind(t, what):
    import torch
    dtype = getattr(t, "dtype", t)
    if dtype == torch.bfloat16:
        return GEMM_TABLE_BF16
    if dtype == torch.float32:
        return GEMM_TABLE_F32
    raise ValueError(f"{what}: BF16 or FP32 is needed, got {dtype}")


def embedding(table, tokens, scale: float = 1.0, stream=None):
    """scale * table[tokens] (table: vocab x width, BF16 or FP32; tokens: rows int64) in the type of the table. A negative
    token gives zeros, one past the table NaN."""
    if stream is not None:
        return _on_stream(stream, embedding, table, tokens, scale)
    import torch
    kind = _table_kind(table, "table")
    ldt = _matrix(table, "table", table.dtype)
    vocab, width = table.shape
    rows = 0 if tokens is None else tokens.numel()
    _vector(tokens, "tokens", torch.int64, rows)
    y = torch.empty((rows, width), dtype=table.dtype, device=table.device)
    status = lib().gemm_embedding(table.data_ptr(), kind, tokens.data_ptr(), y.data_ptr(), rows, vocab, width, ldt, 0,
                                  scale, _stream(None))
    if status:
        raise GemmError(status, "gemm_embedding")
    return y


def embedding_backward(dy, tokens, vocab: int, scale: float = 1.0, base=None, inplace: bool = False, dtype=None,
                       stream=None):
    """The dense gradient of embedding's table (vocab x width): base + scale * the sum of dy (rows x width, BF16 or FP32)
    over each token's positions. `base`: what is there already (the head's gradient, with tied weights), zeros if None;
    `inplace` adds to it. `dtype`: BF16 or FP32, base's or else dy's if None."""
    if stream is not None:
        return _on_stream(stream, embedding_backward, dy, tokens, vocab, scale, base, inplace, dtype)
    import torch
    dy_kind = _table_kind(dy, "dy")
    ldd = _matrix(dy, "dy", dy.dtype)
    rows, width = dy.shape
    _vector(tokens, "tokens", torch.int64, rows)
    if not 0 <= vocab <= _MOST:
        raise ValueError(f"vocab: a size below 2^31 is needed, got {vocab}")
    if dtype is None:
        dtype = dy.dtype if base is None else base.dtype
    kind = _table_kind(dtype, "dtype")
    if base is not None:
        _contiguous(base, "base", dtype, (vocab, width))
    elif inplace:
        raise ValueError("inplace: there is no base to add to")
    out = base if inplace else torch.empty((vocab, width), dtype=dtype, device=dy.device)
    status = lib().gemm_embedding_backward(dy.data_ptr(), dy_kind, tokens.data_ptr(), _address(base), out.data_ptr(), kind,
                                           rows, vocab, width, ldd, scale, _stream(None))
    if status:
        raise GemmError(status, "gemm_embedding_backward")
    return out
