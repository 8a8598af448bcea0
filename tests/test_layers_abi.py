"""include/sgemm_layers.h without a GPU: every declared function is exported
and bound, bad arguments are refused before anything is enqueued, and the
host-only plan follows its rule."""

import ctypes
import os
import re

import pytest

import dense_fp32_matrix_07_gb300 as sg

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "sgemm_layers.h")
BAD, OVER, OK = sg.SGEMM_ERR_INVALID_VALUE, sg.SGEMM_ERR_OVERFLOW, sg.SGEMM_OK
F32, BF16 = sg.SGEMM_F32, sg.SGEMM_BF16
ADD, MUL = sg.SGEMM_JOIN_ADD, sg.SGEMM_JOIN_MUL

# Addresses far apart that are never followed: a refused call touches nothing.
P = [(i + 1) << 40 for i in range(9)]


def test_header_declares_the_binding_functions(sgemm_lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"^\s*int\s+(sgemm\w*)\s*\(", text, flags=re.M)))
    assert declared == sorted(sg.EXPORTED_LAYERS)
    for name in declared:
        assert isinstance(getattr(sgemm_lib, name), ctypes._CFuncPtr)
        assert callable(getattr(sg, name))
    for name, value in re.findall(r"(SGEMM_(?:ACT|JOIN|BF16)_\w+) = (\d+)", text):
        assert getattr(sg, name) == int(value)


def call(name, good, **change):
    return getattr(sg, name)(**dict(good, **change))


DENSE = dict(op_a=0, op_b=1, M=300, N=200, K=260, A=P[0], lda=264, B=P[1], ldb=264, bias=P[2], act=4, pre=P[3], ld_pre=200,
             join=ADD, D=P[4], ldd=200, C=P[5], c_type=BF16, ldc=200)


@pytest.mark.parametrize("change,code", [
    (dict(op_a=2), BAD), (dict(op_b=-1), BAD), (dict(M=-1), BAD), (dict(K=-1), BAD), (dict(A=0), BAD), (dict(A=P[0] + 8), BAD),
    (dict(B=P[1] + 2), BAD), (dict(lda=256), BAD), (dict(lda=262), BAD), (dict(ldb=260), BAD), (dict(op_a=1), BAD),
    (dict(op_b=0, ldb=192), BAD), (dict(act=5), BAD), (dict(act=-1), BAD), (dict(join=3), BAD), (dict(D=0), BAD),
    (dict(ldd=199), BAD), (dict(ld_pre=199), BAD), (dict(C=0), BAD), (dict(ldc=199), BAD), (dict(c_type=2), BAD),
    (dict(C=P[0]), BAD), (dict(C=P[3]), BAD), (dict(pre=P[4]), BAD), (dict(D=P[5], ldd=208), BAD), (dict(D=P[5] + 2), BAD),
    (dict(pre=P[5]), BAD), (dict(C=P[2] + 16), BAD), (dict(C=P[5] + 1), BAD), (dict(bias=P[2] + 2), BAD),
    (dict(M=2 ** 31), OVER), (dict(ldc=2 ** 62), OVER), (dict(ldd=2 ** 62), OVER), (dict(lda=2 ** 62), OVER),
    (dict(M=0), OK), (dict(N=0), OK),
])
def test_product_refusals(change, code):
    assert call("sgemm_bf16", DENSE, **change) == code


GROUPED = dict(op_b=1, groups=4, offsets=P[6], rows=300, N=200, K=260, A=P[0], lda=264, B=P[1], ldb=264, stride_b=200 * 264,
               bias=P[2], stride_bias=200, act=0, pre=0, ld_pre=0, join=MUL, D=P[4], ldd=200, C=P[5], c_type=F32, ldc=200)


@pytest.mark.parametrize("change,code", [
    (dict(groups=-1), BAD), (dict(groups=513), BAD), (dict(offsets=0), BAD), (dict(stride_b=1000), BAD),
    (dict(stride_b=200 * 264 + 4), BAD), (dict(stride_b=-8), BAD), (dict(stride_bias=199), BAD), (dict(stride_bias=-1), BAD),
    (dict(op_b=0), BAD), (dict(C=P[6]), BAD), (dict(C=P[1]), BAD), (dict(lda=256), BAD), (dict(offsets=P[6] + 2), BAD),
    (dict(join=ADD, D=0), BAD), (dict(rows=2 ** 31), OVER), (dict(groups=0), OK), (dict(rows=0), OK), (dict(N=0), OK),
])
def test_grouped_refusals(change, code):
    assert call("sgemm_bf16_grouped", GROUPED, **change) == code


GROUPED_K = dict(groups=4, offsets=P[6], rows=500, M=300, N=200, A=P[0], lda=304, B=P[1], ldb=200, accumulate=1, C=P[5],
                 c_type=F32, ldc=200, stride_c=60000)


@pytest.mark.parametrize("change,code", [
    (dict(groups=-1), BAD), (dict(groups=513), BAD), (dict(offsets=0), BAD), (dict(accumulate=2), BAD), (dict(lda=296), BAD),
    (dict(ldb=204), BAD), (dict(A=P[0] + 2), BAD), (dict(B=0), BAD), (dict(C=0), BAD), (dict(ldc=199), BAD),
    (dict(stride_c=59999), BAD), (dict(stride_c=-1), BAD), (dict(c_type=9), BAD), (dict(C=P[0] + 4), BAD), (dict(rows=-1), BAD),
    (dict(M=2 ** 31, lda=2 ** 31), OVER), (dict(groups=0), OK), (dict(M=0), OK), (dict(N=0), OK),
])
def test_grouped_k_refusals(change, code):
    assert call("sgemm_bf16_grouped_k", GROUPED_K, **change) == code


BACKWARD = dict(rows=300, cols=200, type=BF16, grad_out=P[0], ld_go=200, pre=P[1], ld_pre=200, act=4, join=MUL, D=P[2], ldd=200,
                groups=4, offsets=P[6], grad_pre=P[3], ld_gp=200, grad_D=P[4], ld_gd=200, grad_bias=P[5], stride_gb=200)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), BAD), (dict(type=2), BAD), (dict(act=5), BAD), (dict(join=-1), BAD), (dict(join=ADD), BAD),
    (dict(groups=513), BAD), (dict(groups=-1), BAD), (dict(offsets=0), BAD), (dict(grad_out=0), BAD), (dict(ld_go=199), BAD),
    (dict(pre=0), BAD), (dict(pre=0, act=0), BAD), (dict(ld_pre=199), BAD), (dict(D=0), BAD), (dict(ldd=199), BAD),
    (dict(ld_gp=199), BAD), (dict(ld_gd=199), BAD), (dict(stride_gb=199), BAD), (dict(grad_pre=P[0]), BAD),
    (dict(grad_D=P[3]), BAD), (dict(grad_bias=P[6]), BAD), (dict(grad_pre=P[3] + 1), BAD), (dict(grad_bias=P[5] + 2), BAD),
    (dict(rows=2 ** 31), OVER), (dict(ld_go=2 ** 62), OVER), (dict(cols=0), OK), (dict(groups=0), OK),
    (dict(grad_pre=0, grad_D=0, grad_bias=0), OK), (dict(rows=0, grad_bias=0), OK),
])
def test_epilogue_backward_refusals(change, code):
    assert call("sgemm_epilogue_backward", BACKWARD, **change) == code


NORM = dict(rows=300, cols=200, type=BF16, x=P[0], ldx=200, residual=P[1], ld_res=200, weight=P[2], eps=1e-6, sum=P[3], ld_sum=200,
            y=P[4], ldy=200, q=P[5], ldq=208, scales=P[6], lds=300)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), BAD), (dict(type=3), BAD), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD),
    (dict(x=0), BAD), (dict(ldx=199), BAD), (dict(ld_res=199), BAD), (dict(ld_sum=199), BAD), (dict(ldy=199), BAD),
    (dict(q=P[5] + 8), BAD), (dict(ldq=200), BAD), (dict(scales=0), BAD), (dict(lds=299), BAD), (dict(sum=P[4]), BAD),
    (dict(sum=P[0], ld_sum=208), BAD), (dict(y=P[1] + 2), BAD), (dict(sum=P[2]), BAD), (dict(q=P[0]), BAD), (dict(scales=P[1]), BAD),
    (dict(x=P[0] + 1), BAD), (dict(weight=P[2] + 2), BAD), (dict(cols=16385, ldx=20000, ld_res=20000, ld_sum=20000, ldy=20000, ldq=20000), OVER),
    (dict(rows=2 ** 31, lds=2 ** 31), OVER), (dict(ldx=2 ** 62), OVER), (dict(rows=0), OK), (dict(cols=0), OK),
    (dict(sum=0, y=0, q=0), OK),
])
def test_rms_norm_refusals(change, code):
    assert call("sgemm_rms_norm", NORM, **change) == code


NORM_BACKWARD = dict(rows=300, cols=200, type=BF16, grad_y=P[0], ld_gy=200, s=P[1], ld_s=200, weight=P[2], eps=1e-6, grad_sum=P[3],
                     ld_gsum=200, grad_s=P[4], ld_gs=200, grad_weight=P[5])


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), BAD), (dict(type=3), BAD), (dict(eps=-1.0), BAD), (dict(grad_y=0), BAD), (dict(s=0), BAD), (dict(grad_s=0), BAD),
    (dict(ld_gy=199), BAD), (dict(ld_s=199), BAD), (dict(ld_gsum=199), BAD), (dict(ld_gs=199), BAD), (dict(grad_s=P[1]), BAD),
    (dict(grad_s=P[0], ld_gs=208), BAD), (dict(grad_s=P[3] + 2), BAD), (dict(grad_weight=P[2]), BAD), (dict(grad_weight=P[4]), BAD),
    (dict(cols=16385, ld_gy=20000, ld_s=20000, ld_gsum=20000, ld_gs=20000), OVER), (dict(rows=2 ** 31), OVER),
    (dict(cols=0), OK), (dict(rows=0, grad_weight=0), OK),
])
def test_rms_norm_backward_refusals(change, code):
    assert call("sgemm_rms_norm_backward", NORM_BACKWARD, **change) == code


SMS = 152


def plan(mode, groups, M, N, K, sms=SMS):
    rc, *p = sg.sgemm_bf16_plan(mode, groups, M, N, K, sms)
    assert rc == OK
    return p


def test_plan_refusals():
    for bad in ((3, 1, 1, 1, 1, SMS), (-1, 1, 1, 1, 1, SMS), (0, 2, 1, 1, 1, SMS), (1, 0, 1, 1, 1, SMS), (1, 513, 1, 1, 1, SMS),
                (0, 1, -1, 1, 1, SMS), (0, 1, 1, 1, 1, 0)):
        assert sg.sgemm_bf16_plan(*bad)[0] == BAD
    assert sg.sgemm_bf16_plan(0, 1, 2 ** 31, 1, 1, SMS)[0] == OVER
    assert plan(0, 1, 0, 5, 5)[4] == 0


@pytest.mark.parametrize("mode,groups", [(0, 1), (1, 1), (1, 7), (1, 64), (2, 1), (2, 16)])
def test_plans_cover_c_with_one_wave_or_a_persistent_grid(mode, groups):
    for M in (1, 16, 17, 64, 100, 129, 500, 1000, 5000, 100000):
        for N in (1, 16, 100, 300, 2048, 5000):
            for K in (0, 1, 64, 500, 4096):
                for sms in (1, 2, 7, 152):
                    cols, pair, swap, split, grid = plan(mode, groups, M, N, K, sms)
                    cluster = 2 if pair else split
                    assert cols in (16, 32, 64, 128, 256) and split in (1, 2, 4, 8)
                    assert 0 < grid and grid % cluster == 0 and grid <= max(sms // cluster, 1) * cluster
                    assert not pair or split == 1
                    if split > 1:      # swapped, one tile per cluster, at least four slabs of 64 along K each
                        assert swap and mode != 2 and (K + 63) // 64 >= 4 * split
                        tiles = -(-M // cols) * -(-N // 128)
                        assert mode == 1 or grid == tiles * split
