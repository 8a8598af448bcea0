"""A training step of a layer of experts, with every product in the library.

Each token goes to k of E experts, each a two-layer network D -> F -> D:

    logits = x . Wr                                    FP32 product (sgemm)
    weights, indices = route(logits)                   softmax, top k, renormalised
    rows sorted by expert                              dispatch
    h = x[token_of] . W1_e^T, a = silu(h)              8-bit product over the experts
    y = a . W2_e^T                                     the same
    out[t] = sum_j weights[t, j] y[row_of[t, j]]       combine

and backward, with the same operators: the gradients of the inputs of the 8-bit
products are 8-bit products with the transposed weights, those of the weights
8-bit products over each expert's rows. torch holds the tensors and does the
elementwise silu; run as a script, the step is compared with FP32 autograd.
"""

from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dense_fp32_matrix_07_gb300 as sg  # noqa: E402

FP8, BLOCK = torch.float8_e4m3fn, 128
KIND = {torch.float32: sg.SGEMM_F32, torch.bfloat16: sg.SGEMM_BF16}


def ok(code):
    if code != sg.SGEMM_OK:
        raise sg.SgemmError(code, "experts_layer")


def stream():
    return torch.cuda.current_stream().cuda_stream


def up(n, m=BLOCK):
    return (n + m - 1) // m * m


def new(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="cuda")


def product(a, b, op_a=0, op_b=0):
    """op(a) . op(b) in FP32 (row-major; op 1: transposed)."""
    M, K = a.shape if op_a == 0 else a.shape[::-1]
    N = b.shape[1] if op_b == 0 else b.shape[0]
    c = new(M, N)
    ok(sg.sgemm_general(op_a, op_b, M, N, K, 1.0, a.data_ptr(), a.stride(0), 0, b.data_ptr(), b.stride(0), 0, 0.0,
                        c.data_ptr(), N, 0, 1, stream()))
    return c


def weights_in_8_bits(w, transpose):
    """(E, N, K) weights, or their transposes, in 128 x 128 blocks: (q, scales, rows, columns)."""
    E, N, K = w.shape
    rows, cols = (K, N) if transpose else (N, K)
    ld, sr, sc = up(cols, 16), up(rows) // BLOCK, up(cols) // BLOCK
    q, s = new(E, rows, ld, dtype=FP8), new(E, sr, sc)
    ok(sg.sgemm_fp8_quantize_blocks(N, K, w.data_ptr(), KIND[w.dtype], K, N * K, int(transpose), q.data_ptr(), ld,
                                    rows * ld, s.data_ptr(), sc, sr * sc, E, stream()))
    return q, s, rows, cols


def rows_in_8_bits(x, rows, gather=None, offsets=None):
    """x (gathered) in rows form and, with the experts' offsets, in column form: ((q, s), (q_t, s_t))."""
    cols, ld = x.shape[1], up(x.shape[1], 16)
    q, s = new(rows, ld, dtype=FP8), new(up(cols) // BLOCK, rows)
    at = gather.data_ptr() if gather is not None else 0
    if offsets is None:
        ok(sg.sgemm_fp8_quantize_rows(rows, cols, x.data_ptr(), KIND[x.dtype], x.stride(0), at, x.shape[0],
                                      q.data_ptr(), ld, s.data_ptr(), rows, stream()))
        return (q, s), None
    E = offsets.numel() - 1
    padded = up(rows + (BLOCK - 1) * min(rows, E))   # room for each expert's rows from a multiple of 128 on
    q_t, s_t = new(cols, padded, dtype=FP8), new(padded // BLOCK, cols)
    ok(sg.sgemm_fp8_quantize_both(rows, cols, x.data_ptr(), KIND[x.dtype], x.stride(0), at, x.shape[0], E,
                                  offsets.data_ptr(), padded, q.data_ptr(), ld, s.data_ptr(), rows, q_t.data_ptr(),
                                  padded, s_t.data_ptr(), cols, stream()))
    return (q, s), (q_t, s_t)


def over_experts(a, offsets, b):
    """Rows of a times their experts' matrices, in bfloat16."""
    (q, s), (bq, bs, N, K) = a, b
    rows, E = q.shape[0], bq.shape[0]
    c = new(rows, N, dtype=torch.bfloat16)
    ok(sg.sgemm_fp8_grouped(E, offsets.data_ptr(), rows, N, K, q.data_ptr(), q.stride(0), s.data_ptr(), rows,
                            bq.data_ptr(), bq.stride(1), bq.stride(0), bs.data_ptr(), bs.stride(1), bs.stride(0), 0.0,
                            c.data_ptr(), sg.SGEMM_BF16, N, stream()))
    return c


def weight_gradient(dy, x, offsets):
    """dy^T . x over each expert's rows (both in column form), in FP32."""
    (qa, sa), (qb, sb) = dy, x
    E, M, N, padded = offsets.numel() - 1, qa.shape[0], qb.shape[0], qa.shape[1]
    c = new(E, M, N)
    ok(sg.sgemm_fp8_grouped_k(E, offsets.data_ptr(), padded, M, N, qa.data_ptr(), padded, sa.data_ptr(), M, qb.data_ptr(),
                              padded, sb.data_ptr(), N, 0.0, c.data_ptr(), sg.SGEMM_F32, N, M * N, stream()))
    return c


def combine(y, row_of, weights=None):
    (T, k), (R, cols) = row_of.shape, y.shape
    out = new(T, cols, dtype=y.dtype)
    ok(sg.sgemm_combine(T, k, cols, R, y.data_ptr(), KIND[y.dtype], y.stride(0), row_of.data_ptr(),
                        weights.data_ptr() if weights is not None else 0, out.data_ptr(), cols, stream()))
    return out


def step(x, Wr, W1, W2, k, grad_out):
    """Forward and backward: the output and the gradients of x, Wr, W1 and W2, and the experts chosen."""
    (T, D), E, F = x.shape, Wr.shape[1], W1.shape[1]
    R = T * k
    # Forward. Router in FP32.
    xf = x.float()
    logits = product(xf, Wr)
    weights, indices = new(T, k), new(T, k, dtype=torch.int32)
    ok(sg.sgemm_route(T, E, logits.data_ptr(), sg.SGEMM_F32, E, 0, sg.SGEMM_SCORE_SOFTMAX, 1, 1, 0, k, 1, 1.0,
                      weights.data_ptr(), indices.data_ptr(), stream()))
    offsets, row_of, token_of = new(E + 1, dtype=torch.int32), new(T, k, dtype=torch.int32), new(R, dtype=torch.int32)
    ok(sg.sgemm_dispatch(T, k, E, indices.data_ptr(), offsets.data_ptr(), row_of.data_ptr(), token_of.data_ptr(), stream()))
    x_rows, x_cols = rows_in_8_bits(x, R, token_of, offsets)
    h = over_experts(x_rows, offsets, weights_in_8_bits(W1, False))
    hf = h.float()
    gate = torch.sigmoid(hf)
    a = (hf * gate).bfloat16()
    a_rows, a_cols = rows_in_8_bits(a, R, None, offsets)
    y = over_experts(a_rows, offsets, weights_in_8_bits(W2, False))
    out = combine(y, row_of, weights)
    # Backward.
    dy, dw = torch.empty_like(y), torch.empty_like(weights)
    ok(sg.sgemm_combine_backward(T, k, D, R, grad_out.data_ptr(), KIND[grad_out.dtype], D, y.data_ptr(), D,
                                 row_of.data_ptr(), weights.data_ptr(), dy.data_ptr(), D, dw.data_ptr(), stream()))
    dy_rows, dy_cols = rows_in_8_bits(dy, R, None, offsets)
    da = over_experts(dy_rows, offsets, weights_in_8_bits(W2, True))
    dW2 = weight_gradient(dy_cols, a_cols, offsets)
    dh = (da.float() * gate * (1 + hf * (1 - gate))).bfloat16()
    dh_rows, dh_cols = rows_in_8_bits(dh, R, None, offsets)
    dW1 = weight_gradient(dh_cols, x_cols, offsets)
    dx = combine(over_experts(dh_rows, offsets, weights_in_8_bits(W1, True)), row_of).float()
    dlogits = torch.empty_like(logits)
    ok(sg.sgemm_route_backward(T, E, logits.data_ptr(), sg.SGEMM_F32, E, sg.SGEMM_SCORE_SOFTMAX, k, 1, 1.0,
                               indices.data_ptr(), dw.data_ptr(), dlogits.data_ptr(), E, stream()))
    dx += product(dlogits, Wr, op_b=1)
    dWr = product(xf, dlogits, op_a=1)
    return dict(out=out, x=dx, Wr=dWr, W1=dW1, W2=dW2), indices


def reference(x, Wr, W1, W2, indices, grad_out):
    """The same step by FP32 autograd, for the given choice of experts."""
    x, Wr, W1, W2 = (t.float().requires_grad_(True) for t in (x, Wr, W1, W2))
    at = indices.long()
    w = torch.softmax(x @ Wr, 1).gather(1, at)
    w = w / w.sum(1, keepdim=True)
    out = torch.zeros_like(x)
    for e in range(W1.shape[0]):
        t, j = (at == e).nonzero(as_tuple=True)
        y = torch.nn.functional.silu(x[t] @ W1[e].t()) @ W2[e].t()
        out = out.index_add(0, t, w[t, j, None] * y)
    g = torch.autograd.grad((out * grad_out.float()).sum(), (x, Wr, W1, W2))
    return dict(out=out.detach(), x=g[0], Wr=g[1], W1=g[2], W2=g[3])


def inputs(T, D, F, E, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    return (normal(T, D).bfloat16(), normal(D, E) / math.sqrt(D), normal(E, F, D) / math.sqrt(D),
            normal(E, D, F) / math.sqrt(F), normal(T, D).bfloat16())


def main(T=2000, D=1024, F=1536, E=16, k=4):
    x, Wr, W1, W2, grad_out = inputs(T, D, F, E)
    got, indices = step(x, Wr, W1, W2, k, grad_out)
    status = sg.sgemm_check_status(stream())
    if status != sg.SGEMM_OK:
        raise sg.SgemmError(status, "experts_layer")
    want = reference(x, Wr, W1, W2, indices, grad_out)
    off = {n: float((got[n].float() - want[n]).norm() / want[n].norm()) for n in want}
    for n, v in off.items():
        print(f"{n:4s} relative difference to FP32: {v:.4f}")
    return off


if __name__ == "__main__":
    main()
