"""include/sgemm_experts.h without a GPU: every declared function is exported
and bound, bad arguments are refused before anything is enqueued, and the
host-only plan follows its rule."""

import ctypes
import os
import re

import pytest

import dense_fp32_matrix_07_gb300 as sg

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "sgemm_experts.h")
BAD, OVER, OK = sg.SGEMM_ERR_INVALID_VALUE, sg.SGEMM_ERR_OVERFLOW, sg.SGEMM_OK


def test_header_declares_the_binding_functions(sgemm_lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"^\s*int\s+(sgemm\w*)\s*\(", text, flags=re.M)))
    assert declared == sorted(sg.EXPORTED_EXPERTS)
    for name in declared:
        assert isinstance(getattr(sgemm_lib, name), ctypes._CFuncPtr)
        assert callable(getattr(sg, name))


# Addresses far apart that are never followed: a refused call touches nothing.
P = [(i + 1) << 40 for i in range(8)]
F32, BF16 = sg.SGEMM_F32, sg.SGEMM_BF16


def call(name, good, **change):
    args = dict(good, **change)
    return getattr(sg, name)(**args)


ROWS = dict(rows=10, cols=200, src=P[0], type=BF16, ld=200, gather=0, src_rows=10, q=P[1], ldq=208, scales=P[2], lds=10)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), BAD), (dict(cols=-1), BAD), (dict(type=7), BAD), (dict(ld=199), BAD), (dict(src=0), BAD),
    (dict(q=0), BAD), (dict(q=P[1] + 8), BAD), (dict(ldq=200), BAD), (dict(ldq=192), BAD), (dict(scales=0), BAD),
    (dict(lds=9), BAD), (dict(src_rows=9), BAD), (dict(q=P[0]), BAD), (dict(scales=P[1]), BAD),
    (dict(rows=2 ** 31, src_rows=2 ** 31, lds=2 ** 31), OVER), (dict(ld=2 ** 62), OVER),
    (dict(cols=2 ** 24, ld=2 ** 24, ldq=2 ** 24), OVER), (dict(rows=0), OK), (dict(cols=0), OK),
])
def test_quantize_rows_refusals(change, code):
    assert call("sgemm_fp8_quantize_rows", ROWS, **change) == code


BOTH = dict(rows=10, cols=200, src=P[0], type=F32, ld=200, gather=0, src_rows=10, groups=3, offsets=P[5], padded=384,
            q=P[1], ldq=208, scales=P[2], lds=10, q_t=P[3], ldq_t=384, scales_t=P[4], lds_t=200)


@pytest.mark.parametrize("change,code", [
    (dict(padded=100), BAD), (dict(padded=-128), BAD), (dict(groups=0), BAD), (dict(groups=513), BAD),
    (dict(q_t=0), BAD), (dict(ldq_t=368), BAD), (dict(scales_t=0), BAD), (dict(lds_t=199), BAD), (dict(ldq=199), BAD),
    (dict(lds=9), BAD), (dict(scales=0), BAD), (dict(offsets=0, rows=400, src_rows=400, lds=400), BAD),
    (dict(q_t=P[1]), BAD), (dict(scales_t=P[5]), BAD), (dict(ld=100), BAD), (dict(cols=0), OK), (dict(padded=0), OK),
])
def test_quantize_both_refusals(change, code):
    assert call("sgemm_fp8_quantize_both", BOTH, **change) == code


BLOCKS = dict(rows=300, cols=200, src=P[0], type=F32, ld=200, stride_src=60000, transpose=0, q=P[1], ldq=208,
              stride_q=300 * 208, scales=P[2], lds=2, stride_s=6, batch=2)


@pytest.mark.parametrize("change,code", [
    (dict(transpose=2), BAD), (dict(ldq=192), BAD), (dict(lds=1), BAD), (dict(stride_q=100), BAD),
    (dict(stride_q=300 * 208 + 8), BAD), (dict(stride_s=5), BAD), (dict(src=0), BAD), (dict(batch=-1), BAD),
    (dict(stride_src=-1), BAD), (dict(transpose=1), BAD),          # the transpose needs ldq >= 300
    (dict(batch=0), OK), (dict(rows=0), OK),
])
def test_quantize_blocks_refusals(change, code):
    assert call("sgemm_fp8_quantize_blocks", BLOCKS, **change) == code


DENSE = dict(b_form=sg.SGEMM_SCALE_BLOCKS, M=300, N=200, K=260, A=P[0], lda=272, sa=P[1], ld_sa=300, B=P[2], ldb=272,
             sb=P[3], ld_sb=3, beta=0.0, C=P[4], c_type=F32, ldc=200)


@pytest.mark.parametrize("change,code", [
    (dict(b_form=2), BAD), (dict(M=-1), BAD), (dict(A=0), BAD), (dict(B=P[2] + 4), BAD), (dict(lda=260), BAD),
    (dict(ldb=256), BAD), (dict(ld_sa=299), BAD), (dict(ld_sb=2), BAD), (dict(sa=0), BAD), (dict(sb=0), BAD),
    (dict(C=0), BAD), (dict(ldc=199), BAD), (dict(c_type=3), BAD), (dict(C=P[0]), BAD), (dict(C=P[3]), BAD),
    (dict(b_form=sg.SGEMM_SCALE_ROWS), BAD),                        # rows form needs ld_sb >= N
    (dict(M=2 ** 31, ld_sa=2 ** 31), OVER), (dict(ldc=2 ** 61), OVER), (dict(M=0), OK), (dict(N=0), OK),
])
def test_product_refusals(change, code):
    assert call("sgemm_fp8", DENSE, **change) == code


GROUPED = dict(groups=4, offsets=P[5], rows=300, N=200, K=260, A=P[0], lda=272, sa=P[1], ld_sa=300, B=P[2], ldb=272,
               stride_b=200 * 272, sb=P[3], ld_sb=3, stride_sb=6, beta=0.0, C=P[4], c_type=F32, ldc=200)


@pytest.mark.parametrize("change,code", [
    (dict(groups=-1), BAD), (dict(groups=513), BAD), (dict(offsets=0), BAD), (dict(stride_b=1000), BAD),
    (dict(stride_b=200 * 272 + 8), BAD), (dict(stride_sb=5), BAD), (dict(ld_sa=299), BAD), (dict(C=P[5]), BAD),
    (dict(lda=264), BAD), (dict(ld_sb=2), BAD), (dict(groups=0), OK), (dict(rows=0), OK), (dict(N=0), OK),
])
def test_grouped_refusals(change, code):
    assert call("sgemm_fp8_grouped", GROUPED, **change) == code


GROUPED_K = dict(groups=4, offsets=P[5], padded=512, M=300, N=200, A=P[0], lda=512, sa=P[1], ld_sa=300, B=P[2], ldb=512,
                 sb=P[3], ld_sb=200, beta=0.0, C=P[4], c_type=F32, ldc=200, stride_c=60000)


@pytest.mark.parametrize("change,code", [
    (dict(padded=500), BAD), (dict(stride_c=59999), BAD), (dict(lda=496), BAD), (dict(ld_sb=199), BAD),
    (dict(offsets=0), BAD), (dict(C=P[1]), BAD), (dict(groups=0), OK), (dict(M=0), OK),
])
def test_grouped_k_refusals(change, code):
    assert call("sgemm_fp8_grouped_k", GROUPED_K, **change) == code


ROUTE = dict(T=10, E=64, logits=P[0], type=F32, ld=64, bias=P[1], score=sg.SGEMM_SCORE_SIGMOID, groups=8, kept=4, two=1,
             k=6, renorm=1, scale=1.0, weights=P[2], indices=P[3])


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), BAD), (dict(E=0), BAD), (dict(E=1025, ld=1025, groups=1, kept=1), BAD), (dict(ld=63), BAD),
    (dict(groups=7), BAD), (dict(groups=64), BAD), (dict(kept=9), BAD), (dict(kept=0), BAD), (dict(k=0), BAD),
    (dict(k=33), BAD), (dict(E=4, ld=4, groups=1, kept=1, k=5), BAD), (dict(two=2), BAD), (dict(score=2), BAD),
    (dict(renorm=2), BAD), (dict(weights=0), BAD), (dict(indices=P[2]), BAD), (dict(weights=P[0]), BAD),
    (dict(E=8, ld=8, groups=8, kept=4), BAD),                       # two best of groups of one
    (dict(T=2 ** 31), OVER), (dict(ld=2 ** 61), OVER), (dict(T=0), OK),
])
def test_route_refusals(change, code):
    assert call("sgemm_route", ROUTE, **change) == code


BACK = dict(T=10, E=64, logits=P[0], type=BF16, ld=64, score=sg.SGEMM_SCORE_SOFTMAX, k=6, renorm=0, scale=1.0,
            indices=P[1], grad_w=P[2], grad_logits=P[3], ld_g=64)


@pytest.mark.parametrize("change,code", [
    (dict(ld_g=63), BAD), (dict(grad_w=0), BAD), (dict(indices=0), BAD), (dict(grad_logits=0), BAD),
    (dict(grad_logits=P[0]), BAD), (dict(type=2), BAD), (dict(T=0), OK),
])
def test_route_backward_refusals(change, code):
    assert call("sgemm_route_backward", BACK, **change) == code


DISPATCH = dict(T=10, k=6, E=64, indices=P[0], offsets=P[1], row_of=P[2], token_of=P[3])


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), BAD), (dict(k=0), BAD), (dict(E=0), BAD), (dict(E=1025), BAD), (dict(offsets=0), BAD),
    (dict(row_of=0), BAD), (dict(token_of=P[2]), BAD), (dict(row_of=P[0]), BAD), (dict(T=2 ** 30, k=4), OVER),
])
def test_dispatch_refusals(change, code):
    assert call("sgemm_dispatch", DISPATCH, **change) == code


COMBINE = dict(T=10, k=6, cols=64, rows=60, Y=P[0], type=BF16, ldy=64, row_of=P[1], weights=P[2], out=P[3], ld_out=64)


@pytest.mark.parametrize("change,code", [
    (dict(k=0), BAD), (dict(k=33), BAD), (dict(Y=0), BAD), (dict(row_of=0), BAD), (dict(out=0), BAD), (dict(ldy=63), BAD),
    (dict(ld_out=63), BAD), (dict(out=P[0]), BAD), (dict(rows=-1), BAD), (dict(T=0), OK), (dict(cols=0), OK),
    (dict(cols=2 ** 24, ldy=2 ** 24, ld_out=2 ** 24), OVER),
])
def test_combine_refusals(change, code):
    assert call("sgemm_combine", COMBINE, **change) == code


CBACK = dict(T=10, k=6, cols=64, rows=60, grad_out=P[0], type=BF16, ld_go=64, Y=P[1], ldy=64, row_of=P[2], weights=P[3],
             grad_y=P[4], ld_gy=64, grad_w=P[5])


@pytest.mark.parametrize("change,code", [
    (dict(grad_out=0), BAD), (dict(Y=0), BAD), (dict(ld_gy=63), BAD), (dict(row_of=0), BAD), (dict(grad_y=P[1]), BAD),
    (dict(grad_w=P[3]), BAD), (dict(k=33), BAD), (dict(T=0), OK), (dict(grad_y=0, grad_w=0), OK),
])
def test_combine_backward_refusals(change, code):
    assert call("sgemm_combine_backward", CBACK, **change) == code


def test_plan_refusals_and_empty():
    assert sg.sgemm_fp8_plan(3, 1, 10, 10, 10, 152)[0] == BAD
    assert sg.sgemm_fp8_plan(0, 2, 10, 10, 10, 152)[0] == BAD
    assert sg.sgemm_fp8_plan(0, 1, 10, 10, 10, 0)[0] == BAD
    assert sg.sgemm_fp8_plan(1, 513, 10, 10, 10, 152)[0] == BAD
    assert sg.sgemm_fp8_plan(0, 1, 0, 10, 10, 152)[4] == 0


def test_plan_puts_few_rows_on_the_columns():
    # 65 to 128 rows: split tiles of 64 columns while 128 x 128 ones would leave half the SMs idle.
    assert sg.sgemm_fp8_plan(sg.SGEMM_FP8_DENSE, 1, 128, 4096, 4096, 152)[1:4] == (64, 1, 2)
    assert sg.sgemm_fp8_plan(sg.SGEMM_FP8_DENSE, 1, 128, 16384, 4096, 152)[1:4] == (128, 0, 1)
    # More: by waves of CTAs (1024 rows: one wave of 256-column tiles; 512 rows: one of either).
    assert sg.sgemm_fp8_plan(sg.SGEMM_FP8_DENSE, 1, 1024, 4096, 4096, 152)[1:3] == (256, 0)
    assert sg.sgemm_fp8_plan(sg.SGEMM_FP8_DENSE, 1, 512, 4096, 4096, 152)[1:3] == (128, 0)
    for M, cols in ((1, 16), (16, 16), (17, 32), (33, 64)):
        rc, c, swap, split, grid = sg.sgemm_fp8_plan(sg.SGEMM_FP8_DENSE, 1, M, 4096, 4096, 152)
        assert (rc, c, swap) == (OK, cols, 1) and grid <= 152 and grid % split == 0
    rc, c, swap, split, grid = sg.sgemm_fp8_plan(sg.SGEMM_FP8_DENSE, 1, 16384, 4096, 4096, 152)
    assert (rc, swap, split) == (OK, 0, 1) and grid <= 152
    # A grouped product goes by the rows of a group.
    assert sg.sgemm_fp8_plan(sg.SGEMM_FP8_GROUPED, 64, 96, 2048, 2048, 152)[1:3] == (16, 1)
    assert sg.sgemm_fp8_plan(sg.SGEMM_FP8_GROUPED, 64, 16384, 2048, 2048, 152)[2] == 0
