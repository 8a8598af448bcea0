"""GB300 (sm_103a) single-precision GEMM: C = A . B on row-major FP32 matrices.

This package is a thin ctypes binding over the C ABI in ``include/sgemm.h``
(``_build/libsgemm.so``, compiled from ``csrc/`` by ``build.py``). Its
functions carry the same names and arguments as the C functions and only
marshal arguments: pointers are plain integers (device addresses, e.g. a
torch tensor's ``data_ptr()``), streams are integers (``cudaStream_t``,
e.g. ``torch.cuda.current_stream().cuda_stream``; 0 is the default stream).
Every step of the product runs in the library's CUDA kernels; there is no
CPU fallback, and loading fails loudly if the library cannot be built or
loaded.
"""

from __future__ import annotations

import ctypes
import threading

from . import build as _build

SGEMM_OK = 0
SGEMM_ERR_INVALID_VALUE = 1
SGEMM_ERR_OVERFLOW = 2
SGEMM_ERR_ALLOC = 3
SGEMM_ERR_LAUNCH = 4
SGEMM_ERR_TIMEOUT = 5
SGEMM_ERR_CUDA = 6
SGEMM_ERR_UNSUPPORTED = 7
SGEMM_ERR_SCRATCH_LIMIT = 8

# Every function declared in include/sgemm.h.
EXPORTED = ("sgemm", "sgemm_ex", "sgemm_check_status", "sgemm_error_string",
            "sgemm_num_configs", "sgemm_config_name", "sgemm_plan", "sgemm_noalloc",
            "sgemm_test_withhold_copy", "sgemm_test_schedule", "sgemm_plan_row_tail",
            "sgemm_test_fail_next_allocs", "sgemm_general", "sgemm_general_ex", "sgemm_general_plan",
            "sgemm_general_plan_launches")

# Every function declared in include/sgemm_experts.h.
EXPORTED_EXPERTS = ("sgemm_fp8_quantize_rows", "sgemm_fp8_quantize_cols", "sgemm_fp8_quantize_both",
                    "sgemm_fp8_quantize_blocks", "sgemm_fp8", "sgemm_fp8_grouped", "sgemm_fp8_grouped_k",
                    "sgemm_fp8_plan", "sgemm_route", "sgemm_route_backward", "sgemm_dispatch", "sgemm_combine",
                    "sgemm_combine_backward", "sgemm_test_fail_next_setups")

# Every function declared in include/sgemm_layers.h.
EXPORTED_LAYERS = ("sgemm_bf16", "sgemm_bf16_grouped", "sgemm_bf16_grouped_k", "sgemm_bf16_plan",
                   "sgemm_epilogue_backward", "sgemm_rms_norm", "sgemm_rms_norm_backward")

# Matrix types, scale forms of B, router scores and product modes of sgemm_experts.h.
SGEMM_F32, SGEMM_BF16 = 0, 1
SGEMM_SCALE_BLOCKS, SGEMM_SCALE_ROWS = 0, 1
SGEMM_SCORE_SOFTMAX, SGEMM_SCORE_SIGMOID = 0, 1
SGEMM_FP8_DENSE, SGEMM_FP8_GROUPED, SGEMM_FP8_GROUPED_K = 0, 1, 2

# Activations, joins and product modes of sgemm_layers.h.
SGEMM_ACT_NONE, SGEMM_ACT_RELU, SGEMM_ACT_GELU, SGEMM_ACT_GELU_TANH, SGEMM_ACT_SILU = 0, 1, 2, 3, 4
SGEMM_JOIN_NONE, SGEMM_JOIN_ADD, SGEMM_JOIN_MUL = 0, 1, 2
SGEMM_BF16_DENSE, SGEMM_BF16_GROUPED, SGEMM_BF16_GROUPED_K = 0, 1, 2

_lock = threading.Lock()
_lib = None

_i64 = ctypes.c_int64
_vp = ctypes.c_void_p


class SgemmError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {sgemm_error_string(code)} ({code})")
        self.code = code


def load(rebuild: bool = False):
    """Build (if needed) and load the library; raises if either fails."""
    global _lib
    if _lib is not None and not rebuild:
        return _lib
    with _lock:
        if _lib is None or rebuild:
            path = _build.build(force=rebuild)
            lib = ctypes.CDLL(path)
            lib.sgemm.restype = ctypes.c_int
            lib.sgemm.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp]
            lib.sgemm_ex.restype = ctypes.c_int
            lib.sgemm_ex.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64,
                                     ctypes.c_int, _vp]
            lib.sgemm_noalloc.restype = ctypes.c_int
            lib.sgemm_noalloc.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp]
            lib.sgemm_test_withhold_copy.restype = ctypes.c_int
            lib.sgemm_test_withhold_copy.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp,
                                                     _i64, ctypes.c_int, _vp]
            lib.sgemm_test_schedule.restype = ctypes.c_int
            lib.sgemm_test_schedule.argtypes = [_i64, _i64, _i64, ctypes.c_int, ctypes.c_int, ctypes.c_int, _i64,
                                                ctypes.c_int, _i64, _vp, _i64, _vp, _vp]
            lib.sgemm_plan_row_tail.restype = ctypes.c_int
            lib.sgemm_plan_row_tail.argtypes = [ctypes.c_int, _i64, _i64, _i64, _i64, _vp]
            lib.sgemm_test_fail_next_allocs.restype = ctypes.c_int
            lib.sgemm_test_fail_next_allocs.argtypes = [ctypes.c_int]
            gen = [ctypes.c_int, ctypes.c_int, _i64, _i64, _i64, ctypes.c_float, _vp, _i64, _i64,
                   _vp, _i64, _i64, ctypes.c_float, _vp, _i64, _i64, _i64]
            lib.sgemm_general.restype = ctypes.c_int
            lib.sgemm_general.argtypes = gen + [_vp]
            lib.sgemm_general_ex.restype = ctypes.c_int
            lib.sgemm_general_ex.argtypes = gen + [ctypes.c_int, _vp]
            _pi = ctypes.POINTER(ctypes.c_int)
            lib.sgemm_general_plan.restype = ctypes.c_int
            lib.sgemm_general_plan.argtypes = [ctypes.c_int, ctypes.c_int, _i64, _i64, _i64, ctypes.c_float,
                                               _i64, _i64, _i64, _i64, ctypes.c_float, _i64, _i64, _i64,
                                               ctypes.c_uint64, ctypes.c_uint64, ctypes.c_uint64, ctypes.c_int,
                                               ctypes.c_int, _pi, _pi, _pi]
            lib.sgemm_general_plan_launches.restype = ctypes.c_int
            lib.sgemm_general_plan_launches.argtypes = lib.sgemm_general_plan.argtypes[:19] + [_pi]
            lib.sgemm_check_status.restype = ctypes.c_int
            lib.sgemm_check_status.argtypes = [_vp]
            lib.sgemm_error_string.restype = ctypes.c_char_p
            lib.sgemm_error_string.argtypes = [ctypes.c_int]
            lib.sgemm_num_configs.restype = ctypes.c_int
            lib.sgemm_num_configs.argtypes = []
            lib.sgemm_config_name.restype = ctypes.c_char_p
            lib.sgemm_config_name.argtypes = [ctypes.c_int]
            lib.sgemm_plan.restype = ctypes.c_int
            lib.sgemm_plan.argtypes = [_i64, _i64, _i64, _i64, _i64, _i64,
                                       ctypes.c_uint64, ctypes.c_uint64, ctypes.c_uint64,
                                       ctypes.c_int,
                                       ctypes.POINTER(ctypes.c_int),
                                       ctypes.POINTER(ctypes.c_int),
                                       ctypes.POINTER(ctypes.c_int)]
            i, f = ctypes.c_int, ctypes.c_float
            for name, args in {
                "sgemm_fp8_quantize_rows": [_i64, _i64, _vp, i, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp],
                "sgemm_fp8_quantize_cols": [_i64, _i64, _vp, i, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _i64, _vp,
                                            _i64, _vp],
                "sgemm_fp8_quantize_both": [_i64, _i64, _vp, i, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _i64, _vp,
                                            _i64, _vp, _i64, _vp, _i64, _vp],
                "sgemm_fp8_quantize_blocks": [_i64, _i64, _vp, i, _i64, _i64, i, _vp, _i64, _i64, _vp, _i64, _i64,
                                              _i64, _vp],
                "sgemm_fp8": [i, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, f, _vp, i, _i64, _vp],
                "sgemm_fp8_grouped": [_i64, _vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _i64,
                                      _i64, f, _vp, i, _i64, _vp],
                "sgemm_fp8_grouped_k": [_i64, _vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, f,
                                        _vp, i, _i64, _i64, _vp],
                "sgemm_fp8_plan": [i, _i64, _i64, _i64, _i64, i, _vp, _vp, _vp, _vp],
                "sgemm_route": [_i64, _i64, _vp, i, _i64, _vp, i, i, i, i, i, i, f, _vp, _vp, _vp],
                "sgemm_route_backward": [_i64, _i64, _vp, i, _i64, i, i, i, f, _vp, _vp, _vp, _i64, _vp],
                "sgemm_dispatch": [_i64, i, _i64, _vp, _vp, _vp, _vp, _vp],
                "sgemm_combine": [_i64, i, _i64, _i64, _vp, i, _i64, _vp, _vp, _vp, _i64, _vp],
                "sgemm_combine_backward": [_i64, i, _i64, _i64, _vp, i, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp,
                                           _vp],
                "sgemm_test_fail_next_setups": [i],
                "sgemm_bf16": [i, i, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, i, _vp, _i64, i, _vp, _i64, _vp, i,
                               _i64, _vp],
                "sgemm_bf16_grouped": [i, _i64, _vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _i64, i, _vp,
                                       _i64, i, _vp, _i64, _vp, i, _i64, _vp],
                "sgemm_bf16_grouped_k": [_i64, _vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, i, _vp, i, _i64, _i64, _vp],
                "sgemm_bf16_plan": [i, _i64, _i64, _i64, _i64, i, _vp, _vp, _vp, _vp, _vp],
                "sgemm_epilogue_backward": [_i64, _i64, i, _vp, _i64, _vp, _i64, i, i, _vp, _i64, _i64, _vp, _vp, _i64,
                                            _vp, _i64, _vp, _i64, _vp],
                "sgemm_rms_norm": [_i64, _i64, i, _vp, _i64, _vp, _i64, _vp, f, _vp, _i64, _vp, _i64, _vp, _i64, _vp,
                                   _i64, _vp],
                "sgemm_rms_norm_backward": [_i64, _i64, i, _vp, _i64, _vp, _i64, _vp, f, _vp, _i64, _vp, _i64, _vp,
                                            _vp],
            }.items():
                getattr(lib, name).restype = ctypes.c_int
                getattr(lib, name).argtypes = args
            _lib = lib
    return _lib


def library_path() -> str:
    return _build.LIB


def sgemm(M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    """C = A . B on device pointers; returns the status code (0 = OK)."""
    return load().sgemm(M, N, K, A, lda, B, ldb, C, ldc, stream)


def sgemm_ex(M, N, K, A, lda, B, ldb, C, ldc, config, stream=0) -> int:
    """sgemm() with a forced kernel configuration (-1 = automatic)."""
    return load().sgemm_ex(M, N, K, A, lda, B, ldb, C, ldc, config, stream)


def sgemm_noalloc(M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    """sgemm() for callers that cannot allocate: misaligned operands are
    packed into the library's fixed 64 MiB scratch array instead of
    allocated scratch (SGEMM_ERR_SCRATCH_LIMIT if they would not fit), and
    stream-K partial sums go in a fixed 24 MiB array. All calls on a device
    share those arrays, so calls that overlap on the GPU race on them."""
    return load().sgemm_noalloc(M, N, K, A, lda, B, ldb, C, ldc, stream)


def sgemm_test_fail_next_allocs(n) -> int:
    """Test hook: the next `n` scratch allocations are treated as failed (host only)."""
    return load().sgemm_test_fail_next_allocs(n)


def sgemm_test_withhold_copy(M, N, K, A, lda, B, ldb, C, ldc, slab, stream=0) -> int:
    """Test hook: the 128x256 TMA product whose first CTA never issues the copy of its
    `slab`-th K slab, so the kernel's bounded waits expire (about a second)
    and sgemm_check_status() reports SGEMM_ERR_TIMEOUT."""
    return load().sgemm_test_withhold_copy(M, N, K, A, lda, B, ldb, C, ldc, slab, stream)


def sgemm_test_schedule(M, N, K, bm, bn, bk, slots, policy, batch=1):
    """Test hook (host only): the persistent kernels' work schedule. Returns
    (items, info): items an (n, 10) int64 array of CTA, tile, first slab, end
    slab, batch entry, tile row, tile column, and for a part of a split tile
    its first CTA, last CTA and partial-sum slot (-1 otherwise); info a dict
    of grid, tiles, dp_tiles, sk_ctas, nk, tiles_m, tiles_n."""
    import numpy as np
    count = ctypes.c_int64(0)
    info = np.zeros(7, dtype=np.int64)
    cap = 1024
    while True:
        items = np.zeros((cap, 10), dtype=np.int64)
        rc = load().sgemm_test_schedule(M, N, K, bm, bn, bk, slots, policy, batch,
                                        items.ctypes.data, cap, ctypes.addressof(count), info.ctypes.data)
        if rc == SGEMM_OK:
            keys = ("grid", "tiles", "dp_tiles", "sk_ctas", "nk", "tiles_m", "tiles_n")
            return items[: count.value], dict(zip(keys, (int(x) for x in info)))
        if count.value <= cap:
            raise SgemmError(rc, "sgemm_test_schedule")
        cap = int(count.value)


def sgemm_general(op_a, op_b, M, N, K, alpha, A, lda, stride_a, B, ldb, stride_b,
                  beta, C, ldc, stride_c, batch, stream=0) -> int:
    """C_b = alpha * op(A_b) . op(B_b) + beta * C_b for b < batch."""
    return load().sgemm_general(op_a, op_b, M, N, K, alpha, A, lda, stride_a, B, ldb, stride_b,
                                beta, C, ldc, stride_c, batch, stream)


def sgemm_general_ex(op_a, op_b, M, N, K, alpha, A, lda, stride_a, B, ldb, stride_b,
                     beta, C, ldc, stride_c, batch, config, stream=0) -> int:
    """sgemm_general() with a forced kernel configuration (-1 = automatic)."""
    return load().sgemm_general_ex(op_a, op_b, M, N, K, alpha, A, lda, stride_a, B, ldb, stride_b,
                                   beta, C, ldc, stride_c, batch, config, stream)


def sgemm_check_status(stream=0) -> int:
    """Waits for `stream`, reads and clears the device error word."""
    return load().sgemm_check_status(stream)


def sgemm_error_string(code: int) -> str:
    return load().sgemm_error_string(code).decode()


def sgemm_num_configs() -> int:
    return load().sgemm_num_configs()


def sgemm_config_name(config: int) -> str:
    return load().sgemm_config_name(config).decode()


def sgemm_plan(M, N, K, lda, ldb, ldc, a_addr, b_addr, c_addr, num_sms):
    """Host-only: (status, config, pack_a, pack_b) that sgemm() would use."""
    cfg, pa, pb = ctypes.c_int(-1), ctypes.c_int(-1), ctypes.c_int(-1)
    rc = load().sgemm_plan(M, N, K, lda, ldb, ldc, a_addr, b_addr, c_addr, num_sms,
                           ctypes.byref(cfg), ctypes.byref(pa), ctypes.byref(pb))
    return rc, cfg.value, pa.value, pb.value


def sgemm_plan_row_tail(config, M, N, K, batch=1):
    """Host-only: (status, rows) — the last rows of C that a call on this
    configuration computes with the row-tail kernel (0: none)."""
    rows = ctypes.c_int64(-1)
    rc = load().sgemm_plan_row_tail(config, M, N, K, batch, ctypes.addressof(rows))
    return rc, rows.value


def sgemm_general_plan(op_a, op_b, M, N, K, alpha, lda, stride_a, ldb, stride_b, beta, ldc, stride_c,
                       batch, a_addr, b_addr, c_addr, num_sms, config=-1):
    """Host-only: (status, config, pack_a, pack_b) that sgemm_general_ex() would use
    (config -1 when the call runs no product)."""
    cfg, pa, pb = ctypes.c_int(-1), ctypes.c_int(-1), ctypes.c_int(-1)
    rc = load().sgemm_general_plan(op_a, op_b, M, N, K, alpha, lda, stride_a, ldb, stride_b, beta, ldc,
                                   stride_c, batch, a_addr, b_addr, c_addr, num_sms, config,
                                   ctypes.byref(cfg), ctypes.byref(pa), ctypes.byref(pb))
    return rc, cfg.value, pa.value, pb.value


def sgemm_general_plan_launches(op_a, op_b, M, N, K, alpha, lda, stride_a, ldb, stride_b, beta, ldc, stride_c,
                                batch, a_addr, b_addr, c_addr, num_sms, config=-1):
    """Host-only: (status, kernels of this library that sgemm_general_ex() would launch)."""
    n = ctypes.c_int(-1)
    rc = load().sgemm_general_plan_launches(op_a, op_b, M, N, K, alpha, lda, stride_a, ldb, stride_b, beta, ldc,
                                            stride_c, batch, a_addr, b_addr, c_addr, num_sms, config,
                                            ctypes.byref(n))
    return rc, n.value


def config_ids() -> dict:
    """Map of configuration name -> id."""
    return {sgemm_config_name(i): i for i in range(sgemm_num_configs())}


# ---------------------------------------------------------------------------
# include/sgemm_experts.h: routing, 8-bit quantisation and products, the sum of
# the experts' outputs. Arguments and status codes as there.


def sgemm_fp8_quantize_rows(rows, cols, src, type, ld, gather, src_rows, q, ldq, scales, lds, stream=0) -> int:
    """e4m3 with a scale per row and 128 columns, of rows of src (gathered by `gather` unless 0)."""
    return load().sgemm_fp8_quantize_rows(rows, cols, src, type, ld, gather, src_rows, q, ldq, scales, lds, stream)


def sgemm_fp8_quantize_cols(rows, cols, src, type, ld, gather, src_rows, groups, offsets, padded, q_t, ldq_t,
                            scales_t, lds_t, stream=0) -> int:
    """The transpose with a scale per column and 128 rows of a group, each group from a multiple of 128 on."""
    return load().sgemm_fp8_quantize_cols(rows, cols, src, type, ld, gather, src_rows, groups, offsets, padded, q_t,
                                          ldq_t, scales_t, lds_t, stream)


def sgemm_fp8_quantize_both(rows, cols, src, type, ld, gather, src_rows, groups, offsets, padded, q, ldq, scales,
                            lds, q_t, ldq_t, scales_t, lds_t, stream=0) -> int:
    """sgemm_fp8_quantize_rows() and sgemm_fp8_quantize_cols() from one read of src."""
    return load().sgemm_fp8_quantize_both(rows, cols, src, type, ld, gather, src_rows, groups, offsets, padded, q,
                                          ldq, scales, lds, q_t, ldq_t, scales_t, lds_t, stream)


def sgemm_fp8_quantize_blocks(rows, cols, src, type, ld, stride_src, transpose, q, ldq, stride_q, scales, lds,
                              stride_s, batch, stream=0) -> int:
    """e4m3 with a scale per 128 x 128 block (weights), or the transpose of that."""
    return load().sgemm_fp8_quantize_blocks(rows, cols, src, type, ld, stride_src, transpose, q, ldq, stride_q,
                                            scales, lds, stride_s, batch, stream)


def sgemm_fp8(b_form, M, N, K, A, lda, sa, ld_sa, B, ldb, sb, ld_sb, beta, C, c_type, ldc, stream=0) -> int:
    """C = A . B^T + beta * C on e4m3 operands with a scale per block of 128."""
    return load().sgemm_fp8(b_form, M, N, K, A, lda, sa, ld_sa, B, ldb, sb, ld_sb, beta, C, c_type, ldc, stream)


def sgemm_fp8_grouped(groups, offsets, rows, N, K, A, lda, sa, ld_sa, B, ldb, stride_b, sb, ld_sb, stride_sb, beta,
                      C, c_type, ldc, stream=0) -> int:
    """Each group of rows of A times its own B: the experts' products."""
    return load().sgemm_fp8_grouped(groups, offsets, rows, N, K, A, lda, sa, ld_sa, B, ldb, stride_b, sb, ld_sb,
                                    stride_sb, beta, C, c_type, ldc, stream)


def sgemm_fp8_grouped_k(groups, offsets, padded, M, N, A, lda, sa, ld_sa, B, ldb, sb, ld_sb, beta, C, c_type, ldc,
                        stride_c, stream=0) -> int:
    """One product per group over that group's rows: the experts' weight gradients."""
    return load().sgemm_fp8_grouped_k(groups, offsets, padded, M, N, A, lda, sa, ld_sa, B, ldb, sb, ld_sb, beta, C,
                                      c_type, ldc, stride_c, stream)


def sgemm_fp8_plan(mode, groups, M, N, K, num_sms):
    """Host-only: (status, columns, swap, split, grid) of the kernel an 8-bit product takes."""
    cols, swap, split, grid = ctypes.c_int(-1), ctypes.c_int(-1), ctypes.c_int(-1), ctypes.c_int64(-1)
    rc = load().sgemm_fp8_plan(mode, groups, M, N, K, num_sms, ctypes.addressof(cols), ctypes.addressof(swap),
                               ctypes.addressof(split), ctypes.addressof(grid))
    return rc, cols.value, swap.value, split.value, grid.value


def sgemm_route(T, E, logits, type, ld, bias, score, groups, kept, two, k, renorm, scale, weights, indices,
                stream=0) -> int:
    """The k experts of each token and their weights."""
    return load().sgemm_route(T, E, logits, type, ld, bias, score, groups, kept, two, k, renorm, scale, weights,
                              indices, stream)


def sgemm_route_backward(T, E, logits, type, ld, score, k, renorm, scale, indices, grad_w, grad_logits, ld_g,
                         stream=0) -> int:
    """Gradient of sgemm_route()'s weights with respect to the logits."""
    return load().sgemm_route_backward(T, E, logits, type, ld, score, k, renorm, scale, indices, grad_w, grad_logits,
                                       ld_g, stream)


def sgemm_dispatch(T, k, E, indices, offsets, row_of, token_of, stream=0) -> int:
    """The (token, slot) pairs sorted by expert."""
    return load().sgemm_dispatch(T, k, E, indices, offsets, row_of, token_of, stream)


def sgemm_combine(T, k, cols, rows, Y, type, ldy, row_of, weights, out, ld_out, stream=0) -> int:
    """out[t] = sum_j weights[t, j] * Y[row_of[t, j]]."""
    return load().sgemm_combine(T, k, cols, rows, Y, type, ldy, row_of, weights, out, ld_out, stream)


def sgemm_combine_backward(T, k, cols, rows, grad_out, type, ld_go, Y, ldy, row_of, weights, grad_y, ld_gy, grad_w,
                           stream=0) -> int:
    """Gradients of sgemm_combine() with respect to Y and the weights."""
    return load().sgemm_combine_backward(T, k, cols, rows, grad_out, type, ld_go, Y, ldy, row_of, weights, grad_y,
                                         ld_gy, grad_w, stream)


def sgemm_test_fail_next_setups(n) -> int:
    """Test hook: the next `n` set-ups of the kernels above are treated as failed (host only)."""
    return load().sgemm_test_fail_next_setups(n)


# ---------------------------------------------------------------------------
# include/sgemm_layers.h: 16-bit products with an epilogue, its gradient, the
# root-mean-square norm. Arguments and status codes as there.


def sgemm_bf16(op_a, op_b, M, N, K, A, lda, B, ldb, bias, act, pre, ld_pre, join, D, ldd, C, c_type, ldc,
               stream=0) -> int:
    """C = act(op(A) . op(B) + bias), plus or times D, on bfloat16 A and B."""
    return load().sgemm_bf16(op_a, op_b, M, N, K, A, lda, B, ldb, bias, act, pre, ld_pre, join, D, ldd, C, c_type, ldc,
                             stream)


def sgemm_bf16_grouped(op_b, groups, offsets, rows, N, K, A, lda, B, ldb, stride_b, bias, stride_bias, act, pre, ld_pre,
                       join, D, ldd, C, c_type, ldc, stream=0) -> int:
    """sgemm_bf16() of each group of rows of A with its own B and bias: the experts' products."""
    return load().sgemm_bf16_grouped(op_b, groups, offsets, rows, N, K, A, lda, B, ldb, stride_b, bias, stride_bias,
                                     act, pre, ld_pre, join, D, ldd, C, c_type, ldc, stream)


def sgemm_bf16_grouped_k(groups, offsets, rows, M, N, A, lda, B, ldb, accumulate, C, c_type, ldc, stride_c,
                         stream=0) -> int:
    """A_g^T . B_g over each group's rows: the experts' weight gradients."""
    return load().sgemm_bf16_grouped_k(groups, offsets, rows, M, N, A, lda, B, ldb, accumulate, C, c_type, ldc,
                                       stride_c, stream)


def sgemm_bf16_plan(mode, groups, M, N, K, num_sms):
    """Host-only: (status, columns, pair, swap, split, grid) of the kernel a 16-bit product takes."""
    cols, pair, swap, split = (ctypes.c_int(-1) for _ in range(4))
    grid = ctypes.c_int64(-1)
    rc = load().sgemm_bf16_plan(mode, groups, M, N, K, num_sms, *(ctypes.addressof(x) for x in
                                                                  (cols, pair, swap, split, grid)))
    return rc, cols.value, pair.value, swap.value, split.value, grid.value


def sgemm_epilogue_backward(rows, cols, type, grad_out, ld_go, pre, ld_pre, act, join, D, ldd, groups, offsets,
                            grad_pre, ld_gp, grad_D, ld_gd, grad_bias, stride_gb, stream=0) -> int:
    """Gradients of a product's epilogue: of its sums, of the factor D, and of the bias per group of rows."""
    return load().sgemm_epilogue_backward(rows, cols, type, grad_out, ld_go, pre, ld_pre, act, join, D, ldd, groups,
                                          offsets, grad_pre, ld_gp, grad_D, ld_gd, grad_bias, stride_gb, stream)


def sgemm_rms_norm(rows, cols, type, x, ldx, residual, ld_res, weight, eps, sum, ld_sum, y, ldy, q, ldq, scales, lds,
                   stream=0) -> int:
    """x + residual, and its rows over their root mean square times weight, in `type` and in 8 bits."""
    return load().sgemm_rms_norm(rows, cols, type, x, ldx, residual, ld_res, weight, eps, sum, ld_sum, y, ldy, q, ldq,
                                 scales, lds, stream)


def sgemm_rms_norm_backward(rows, cols, type, grad_y, ld_gy, s, ld_s, weight, eps, grad_sum, ld_gsum, grad_s, ld_gs,
                            grad_weight, stream=0) -> int:
    """Gradients of sgemm_rms_norm() with respect to the sum and the weight."""
    return load().sgemm_rms_norm_backward(rows, cols, type, grad_y, ld_gy, s, ld_s, weight, eps, grad_sum, ld_gsum,
                                          grad_s, ld_gs, grad_weight, stream)
