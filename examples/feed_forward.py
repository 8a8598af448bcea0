"""A training step of a gated feed-forward block in 16 bits, all of it in the library.

    s = x + r,  y = rms_norm(s) * w          norm with the residual's addition
    u = y . Wu^T                             16-bit product
    h = silu(y . Wg^T + b) * u               the same, with bias, activation and the factor u in its epilogue
    out = h . Wd^T + s                       the same, with the residual

and backward, with the same operators: gradients of a product's inputs are
products with the weights as they are stored, those of the weights products
over the tokens, in FP32; the epilogue's gradient gives those of the sums
before the activation, of the factor and of the bias; the norm's adds the
gradient that comes along the residual. torch holds the tensors. Run as a
script, the step is compared with FP32 autograd.
"""

from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dense_fp32_matrix_07_gb300 as sg  # noqa: E402

EPS = 1e-6
KIND = {torch.float32: sg.SGEMM_F32, torch.bfloat16: sg.SGEMM_BF16}


def ok(code):
    if code != sg.SGEMM_OK:
        raise sg.SgemmError(code, "feed_forward")


def stream():
    return torch.cuda.current_stream().cuda_stream


def new(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda")


def at(t):
    return 0 if t is None else t.data_ptr()


def product(a, b, op_a=0, op_b=0, bias=None, act=sg.SGEMM_ACT_NONE, pre=None, join=sg.SGEMM_JOIN_NONE, d=None, out=None,
            dtype=torch.bfloat16):
    """act(op(a) . op(b) + bias), plus or times d; op 1: stored transposed. Rows of a and b begin on 16 bytes."""
    M, K = a.shape if op_a == 0 else a.shape[::-1]
    N = b.shape[1] if op_b == 0 else b.shape[0]
    c = out if out is not None else new(M, N, dtype=dtype)
    ok(sg.sgemm_bf16(op_a, op_b, M, N, K, a.data_ptr(), a.stride(0), b.data_ptr(), b.stride(0), at(bias), act, at(pre), N,
                     join, at(d), N, c.data_ptr(), KIND[c.dtype], N, stream()))
    return c


def step(x, r, w, b, Wu, Wg, Wd, grad_out):
    """Forward and backward: the output, the sum s, and the gradients of x (and r), w, b and the weights."""
    T, D = x.shape
    F = Wu.shape[0]
    s, y = torch.empty_like(x), torch.empty_like(x)
    ok(sg.sgemm_rms_norm(T, D, sg.SGEMM_BF16, x.data_ptr(), D, r.data_ptr(), D, w.data_ptr(), EPS, s.data_ptr(), D,
                         y.data_ptr(), D, 0, 0, 0, 0, stream()))
    u, z = product(y, Wu, op_b=1), new(T, F)
    h = product(y, Wg, op_b=1, bias=b, act=sg.SGEMM_ACT_SILU, pre=z, join=sg.SGEMM_JOIN_MUL, d=u)
    out = product(h, Wd, op_b=1, join=sg.SGEMM_JOIN_ADD, d=s)
    # Backward.
    dh, dWd = product(grad_out, Wd), product(grad_out, h, op_a=1, dtype=torch.float32)
    dz, du, db = torch.empty_like(z), torch.empty_like(u), new(F, dtype=torch.float32)
    ok(sg.sgemm_epilogue_backward(T, F, sg.SGEMM_BF16, dh.data_ptr(), F, z.data_ptr(), F, sg.SGEMM_ACT_SILU,
                                  sg.SGEMM_JOIN_MUL, u.data_ptr(), F, 1, 0, dz.data_ptr(), F, du.data_ptr(), F,
                                  db.data_ptr(), F, stream()))
    dWg, dWu = product(dz, y, op_a=1, dtype=torch.float32), product(du, y, op_a=1, dtype=torch.float32)
    dy = product(dz, Wg)
    product(du, Wu, join=sg.SGEMM_JOIN_ADD, d=dy, out=dy)      # added in place
    dx, dw = torch.empty_like(x), new(D, dtype=torch.float32)
    ok(sg.sgemm_rms_norm_backward(T, D, sg.SGEMM_BF16, dy.data_ptr(), D, s.data_ptr(), D, w.data_ptr(), EPS,
                                  grad_out.data_ptr(), D, dx.data_ptr(), D, dw.data_ptr(), stream()))
    return dict(out=out, x=dx, w=dw, b=db, Wu=dWu, Wg=dWg, Wd=dWd)


def reference(x, r, w, b, Wu, Wg, Wd, grad_out, dtype=torch.float32):
    """The same step by autograd."""
    x, r, w, b, Wu, Wg, Wd = (t.to(dtype) for t in (x, r, w, b, Wu, Wg, Wd))
    leaves = [t.requires_grad_(True) for t in (x, w, b, Wu, Wg, Wd)]
    s = x + r
    y = s / torch.sqrt((s * s).mean(1, keepdim=True) + EPS) * w
    out = torch.nn.functional.silu(y @ Wg.t() + b) * (y @ Wu.t()) @ Wd.t() + s
    g = torch.autograd.grad((out * grad_out.to(dtype)).sum(), leaves)
    return dict(out=out.detach(), **dict(zip(("x", "w", "b", "Wu", "Wg", "Wd"), g)))


def inputs(T, D, F, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    return (normal(T, D).bfloat16(), normal(T, D).bfloat16(), 1.0 + 0.1 * normal(D), 0.1 * normal(F),
            (normal(F, D) / math.sqrt(D)).bfloat16(), (normal(F, D) / math.sqrt(D)).bfloat16(),
            (normal(D, F) / math.sqrt(F)).bfloat16(), normal(T, D).bfloat16())


def main(T=2000, D=1024, F=2048):
    args = inputs(T, D, F)
    got = step(*args)
    status = sg.sgemm_check_status(stream())
    if status != sg.SGEMM_OK:
        raise sg.SgemmError(status, "feed_forward")
    want = reference(*args)
    off = {n: float((got[n].float() - want[n]).norm() / want[n].norm()) for n in want}
    for n, v in off.items():
        print(f"{n:4s} relative difference to FP32: {v:.5f}")
    return off


if __name__ == "__main__":
    main()
