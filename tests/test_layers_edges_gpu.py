"""Calls of the operators of layers that their documentation allows and whose
shape is out of the ordinary: matrices of one call aligned differently, the
largest number of groups, one very long side, the same matrix in two places,
offsets that change between replays of a captured call. Products of small whole
numbers are exact; the norm is held to test_layers_gpu's bounds."""

import pytest
import torch

import dense_fp32_matrix_07_gb300 as sg
import layers_ref as ref
from test_experts_gpu import Guarded, finish, ok, stream
from test_layers_gpu import BF16, F32, TYPES, gen, norm_error, normal, operand, up

pytestmark = pytest.mark.gpu


def whole(g, *shape):
    return torch.randint(-3, 4, shape, generator=g, device="cuda").double()


@pytest.mark.parametrize("shape", [(3, 1), (17, 7), (40, 250), (9, 1000), (33, 2047), (5, 4095), (6, 8191), (3, 12001), (2, 16384)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("type", [F32, BF16], ids=["f32", "bf16"])
def test_norm_of_matrices_that_lie_differently(cuda_device, shape, type):
    (rows, cols), dtype, half, eps = shape, TYPES[type], ref.half_step(TYPES[type]), 1e-6
    g = gen(rows, cols, type)
    places = iter([(up(cols, 8), 0), (cols, 1), (cols + 2, 2), (up(cols, 8) + 8, 3), (cols + 1, 5), (cols, 0), (cols + 7, 7), (up(cols, 8), 0)])

    def place(x=None):
        apart, shift = next(places)
        m = Guarded(rows, cols, apart, dtype, shift=shift)
        return m if x is None else m.put(x.to(dtype))
    x, r, s_out, y_out = place(normal(g, rows, cols)), place(normal(g, rows, cols)), place(), place()
    w = normal(g, cols)
    ok(sg.sgemm_rms_norm(rows, cols, type, x.ptr, x.ld, r.ptr, r.ld, w.data_ptr(), eps, s_out.ptr, s_out.ld, y_out.ptr, y_out.ld, 0, 0,
                         0, 0, stream()))
    gy, gs, d, dw = place(normal(g, rows, cols)), place(normal(g, rows, cols)), place(), Guarded(1, cols, cols, torch.float32)
    ok(sg.sgemm_rms_norm_backward(rows, cols, type, gy.ptr, gy.ld, s_out.ptr, s_out.ld, w.data_ptr(), eps, gs.ptr, gs.ld, d.ptr, d.ld,
                                  dw.ptr, stream()))
    finish()
    s = x.view().double() + r.view().double()
    y = ref.rms_norm(s, w.double(), eps)
    e = norm_error(s, y, cols)
    ref.close(s_out.view(), s, (half + 2.0 ** -24) * s.abs(), "sum")
    ref.close(y_out.view(), y, e + half * (y.abs() + e) + 2.0 ** -126, "y")
    # The gradient, from the sum as it was stored; bounds as in test_layers_gpu.
    S, G, W = s_out.view().double(), gy.view().double(), w.double()
    want, want_dw = ref.rms_norm_backward(G, S, W, eps, gs.view().double())
    rel = (cols + 1) * 2.0 ** -25 + 2.0 ** -22 + 6 * 2.0 ** -24
    i = 1.0 / torch.sqrt((S * S).mean(1, keepdim=True) + eps)
    h, gw = S * i, G * W
    e = i * (gw.abs() + h.abs() * (gw * h).abs().mean(1, keepdim=True)) * (4 * rel + (cols + 4) * 2.0 ** -24)
    e = e + 2.0 ** -24 * (want.abs() + e)
    ref.close(d.view(), want, e + half * (want.abs() + e) + 2.0 ** -126, "d")
    ref.close(dw.view()[0], want_dw, (G * h).abs().sum(0) * (rel + (rows + 2) * 2.0 ** -24) + 2.0 ** -126, "dw")
    for m in (s_out, y_out, d, dw):
        assert m.outside_untouched()


@pytest.mark.parametrize("E", [511, 512])
@pytest.mark.parametrize("type", [F32, BF16], ids=["f32", "bf16"])
def test_the_largest_number_of_groups(cuda_device, E, type):
    g = gen(E, type)
    counts = torch.randint(0, 9, (E,), generator=g, device="cuda").tolist()
    counts[0], counts[E - 1], counts[255], counts[256] = 0, 300, 1, 0
    R, N, K, dtype = sum(counts), 136, 72, TYPES[type]
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    o = off.tolist()
    a, b, bias, c = whole(g, R, K), whole(g, E, N, K), whole(g, E, N), whole(g, R, N)
    A, lda = operand(a.bfloat16())
    B, ldb = operand(b.bfloat16())
    G, ldg = operand(c.bfloat16())
    C, dW = Guarded(R, N, N, dtype), Guarded(E * N, K, K, dtype)
    dz, db = Guarded(R, N, N, dtype), Guarded(E, N, N, torch.float32)
    bias32, cc = bias.float(), c.to(dtype)
    ok(sg.sgemm_bf16_grouped(1, E, off.data_ptr(), R, N, K, A.data_ptr(), lda, B.data_ptr(), ldb, B.stride(0), bias32.data_ptr(), N,
                             sg.SGEMM_ACT_RELU, 0, 0, 0, 0, 0, C.ptr, type, N, stream()))
    ok(sg.sgemm_bf16_grouped_k(E, off.data_ptr(), R, N, K, G.data_ptr(), ldg, A.data_ptr(), lda, 0, dW.ptr, type, K, N * K, stream()))
    ok(sg.sgemm_epilogue_backward(R, N, type, cc.data_ptr(), N, C.ptr, N, sg.SGEMM_ACT_RELU, 0, 0, 0, E, off.data_ptr(), dz.ptr, N, 0, 0,
                                  db.ptr, N, stream()))
    finish()
    for e in range(E):
        rows = slice(o[e], o[e + 1])
        z = (a[rows] @ b[e].t() + bias[e]).clamp(min=0)
        grad = c[rows] * (z > 0)
        assert torch.equal(C.view()[rows], z.to(dtype)), e
        assert torch.equal(dW.view()[e * N:(e + 1) * N], (c[rows].t() @ a[rows]).to(dtype)), e
        assert torch.equal(dz.view()[rows], grad.to(dtype)) and torch.equal(db.view()[e], grad.sum(0).float()), e
    for m in (C, dW, dz, db):
        assert m.outside_untouched()


@pytest.mark.parametrize("M,N,K", [(300001, 8, 16), (8, 300001, 16), (1, 1, 100000), (300001, 1, 1), (1, 300001, 1)], ids=str)
@pytest.mark.parametrize("type", [F32, BF16], ids=["f32", "bf16"])
def test_one_long_side(cuda_device, M, N, K, type):
    g = gen(M, N, K)
    a, b, dtype = whole(g, M, K), whole(g, N, K), TYPES[type]
    A, lda = operand(a.bfloat16())
    B, ldb = operand(b.bfloat16())
    C, z = Guarded(M, N, N, dtype), a @ b.t()
    ok(sg.sgemm_bf16(0, 1, M, N, K, A.data_ptr(), lda, B.data_ptr(), ldb, 0, 0, 0, 0, 0, 0, 0, C.ptr, type, N, stream()))
    db = Guarded(1, N, N, torch.float32)
    ok(sg.sgemm_epilogue_backward(M, N, type, C.ptr, N, 0, 0, 0, 0, 0, 0, 1, 0, 0, 0, 0, 0, db.ptr, N, stream()))
    finish()
    assert torch.equal(C.view(), z.to(dtype)) and C.outside_untouched()
    # Sums of up to 300001 rounded values: each in FP32 order of its own.
    C64 = C.view().double()
    assert bool(((db.view()[0].double() - C64.sum(0)).abs() <= M * 2.0 ** -24 * C64.abs().sum(0)).all()) and db.outside_untouched()


@pytest.mark.parametrize("type", [F32, BF16], ids=["f32", "bf16"])
def test_the_same_matrix_in_two_places(cuda_device, type):
    dtype = TYPES[type]
    g = gen(type)
    R, K = 300, 200
    a = whole(g, R, K).bfloat16()
    x = whole(g, R, K).to(dtype)
    C, s, y = torch.empty(R, R, device="cuda").to(dtype), torch.empty_like(x), torch.empty_like(x)
    dz, dD = torch.empty_like(x), torch.empty_like(x)
    ok(sg.sgemm_bf16(0, 1, R, R, K, a.data_ptr(), K, a.data_ptr(), K, 0, 0, 0, 0, 0, 0, 0, C.data_ptr(), type, R, stream()))
    ok(sg.sgemm_rms_norm(R, K, type, x.data_ptr(), K, x.data_ptr(), K, 0, 1e-6, s.data_ptr(), K, y.data_ptr(), K, 0, 0, 0, 0, stream()))
    ok(sg.sgemm_epilogue_backward(R, K, type, x.data_ptr(), K, x.data_ptr(), K, sg.SGEMM_ACT_RELU, sg.SGEMM_JOIN_MUL, x.data_ptr(), K, 1, 0,
                                  dz.data_ptr(), K, dD.data_ptr(), K, 0, 0, stream()))
    d = x.clone()      # all three of the norm's gradients in one place
    ok(sg.sgemm_rms_norm_backward(R, K, type, d.data_ptr(), K, s.data_ptr(), K, 0, 1e-6, d.data_ptr(), K, d.data_ptr(), K, 0, stream()))
    apart = torch.empty_like(x)
    ok(sg.sgemm_rms_norm_backward(R, K, type, x.data_ptr(), K, s.data_ptr(), K, 0, 1e-6, x.data_ptr(), K, apart.data_ptr(), K, 0, stream()))
    finish()
    A, X = a.double(), x.double()
    assert torch.equal(C, (A @ A.t()).to(dtype)) and torch.equal(s, 2 * x)
    on = (X > 0).double()
    assert torch.equal(dz, (X * X * on).to(dtype)) and torch.equal(dD, (X * X * on).to(dtype))
    assert torch.equal(d, apart)


def test_replays_with_other_offsets(cuda_device):
    """A captured step over groups follows the offsets that are there when it runs."""
    E, R, N, K = 6, 700, 264, 136
    g = gen(3)
    a, b, c = whole(g, R, K), whole(g, E, N, K), whole(g, R, N)
    A, B, G = a.bfloat16(), b.bfloat16(), c.bfloat16()
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    C, dz, db, dW = (torch.empty(s, device="cuda") for s in ((R, N), (R, N), (E, N), (E, N, K)))
    G32 = c.float()

    def step(st):
        ok(sg.sgemm_bf16_grouped(1, E, off.data_ptr(), R, N, K, A.data_ptr(), K, B.data_ptr(), K, N * K, 0, 0, 0, 0, 0, 0, 0, 0, C.data_ptr(),
                                 F32, N, st))
        ok(sg.sgemm_epilogue_backward(R, N, F32, G32.data_ptr(), N, C.data_ptr(), N, sg.SGEMM_ACT_RELU, 0, 0, 0, E, off.data_ptr(),
                                      dz.data_ptr(), N, 0, 0, db.data_ptr(), N, st))
        ok(sg.sgemm_bf16_grouped_k(E, off.data_ptr(), R, N, K, G.data_ptr(), N, A.data_ptr(), K, 0, dW.data_ptr(), F32, K, N * K, st))
    step(stream())
    finish()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(stream())
    for counts in ([100, 0, 300, 1, 250, 49], [0, 0, 0, 0, 0, 700], [1, 2, 3, 4, 5, 6], [0] * 6, [700, 0, 0, 0, 0, 0]):
        off.copy_(torch.tensor([0] + counts).cumsum(0).to(torch.int32))
        for t in (C, dz, db, dW):
            t.fill_(7.0)
        graph.replay()
        finish()
        o = off.tolist()
        for e in range(E):
            rows = slice(o[e], o[e + 1])
            z = a[rows] @ b[e].t()
            grad = c[rows] * (z > 0)
            assert torch.equal(C[rows].double(), z) and torch.equal(dz[rows].double(), grad), (counts, e)
            assert torch.equal(db[e].double(), grad.sum(0)) and torch.equal(dW[e].double(), c[rows].t() @ a[rows]), (counts, e)
        assert bool((C[o[-1]:] == 7).all()) and bool((dz[o[-1]:] == 7).all()), counts
