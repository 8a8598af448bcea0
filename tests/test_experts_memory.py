"""What the experts' operators may touch, checked on the host: a call whose
output would be written where another of its matrices lies is refused."""

import pytest

import dense_fp32_matrix_07_gb300 as sg

BAD = sg.SGEMM_ERR_INVALID_VALUE
# Addresses far apart that are never followed: a refused call touches nothing.
P = [(i + 1) << 40 for i in range(8)]


# The quantisers store 8 bytes at a time along a row (16 in a transposed one),
# in the last row too: up to 7 (15) bytes past its last value.
ROW = dict(rows=1, cols=2041, src=P[0], type=sg.SGEMM_BF16, ld=2048, gather=0, src_rows=1, q=P[1], ldq=2048, scales=P[2],
           lds=1)
BOTH = dict(rows=3, cols=130, src=P[0], type=sg.SGEMM_F32, ld=130, gather=P[6], src_rows=3, groups=2, offsets=P[5],
            padded=256, q=P[1], ldq=144, scales=P[2], lds=3, q_t=P[3], ldq_t=256, scales_t=P[4], lds_t=130)
BLOCKS = dict(rows=130, cols=130, src=P[0], type=sg.SGEMM_F32, ld=130, stride_src=0, transpose=0, q=P[1], ldq=144,
              stride_q=0, scales=P[2], lds=2, stride_s=0, batch=1)


@pytest.mark.parametrize("name,args,change", [
    ("sgemm_fp8_quantize_rows", ROW, dict(scales=P[1] + 2044)),
    ("sgemm_fp8_quantize_rows", ROW, dict(src=P[1] + 2046)),
    ("sgemm_fp8_quantize_rows", ROW, dict(gather=P[1] + 2044)),
    ("sgemm_fp8_quantize_both", BOTH, dict(scales=P[1] + 2 * 144 + 132)),
    ("sgemm_fp8_quantize_both", BOTH, dict(scales_t=P[1] + 2 * 144 + 132)),
    ("sgemm_fp8_quantize_both", BOTH, dict(offsets=P[1] + 2 * 144 + 132)),
    ("sgemm_fp8_quantize_both", BOTH, dict(gather=P[1] + 2 * 144 + 132)),
    ("sgemm_fp8_quantize_blocks", BLOCKS, dict(scales=P[1] + 129 * 144 + 132)),
    ("sgemm_fp8_quantize_blocks", BLOCKS, dict(src=P[1] + 129 * 144 + 132)),
    ("sgemm_fp8_quantize_blocks", BLOCKS, dict(scales=P[1] + 129 * 144 + 140, transpose=1)),
    ("sgemm_fp8_quantize_blocks", BLOCKS, dict(scales=P[1] + 129 * 144 + 140 + 5 * 20736, transpose=1, batch=6,
                                               stride_q=20736, stride_s=4)),
])
def test_outputs_in_the_last_rows_padding_are_refused(name, args, change):
    assert getattr(sg, name)(**dict(args, **change)) == BAD


# Every array lies on multiples of its elements' size: the kernels read and
# write whole elements, which the GPU refuses elsewhere.
DENSE = dict(b_form=sg.SGEMM_SCALE_BLOCKS, M=300, N=200, K=260, A=P[0], lda=272, sa=P[1], ld_sa=300, B=P[2], ldb=272,
             sb=P[3], ld_sb=3, beta=0.0, C=P[4], c_type=sg.SGEMM_BF16, ldc=200)
GROUPED = dict(groups=4, offsets=P[5], rows=300, N=200, K=260, A=P[0], lda=272, sa=P[1], ld_sa=300, B=P[2], ldb=272,
               stride_b=200 * 272, sb=P[3], ld_sb=3, stride_sb=6, beta=0.0, C=P[4], c_type=sg.SGEMM_F32, ldc=200)
GROUPED_K = dict(groups=4, offsets=P[5], padded=512, M=300, N=200, A=P[0], lda=512, sa=P[1], ld_sa=300, B=P[2], ldb=512,
                 sb=P[3], ld_sb=200, beta=0.0, C=P[4], c_type=sg.SGEMM_F32, ldc=200, stride_c=60000)
ROUTE = dict(T=10, E=64, logits=P[0], type=sg.SGEMM_F32, ld=64, bias=P[1], score=sg.SGEMM_SCORE_SIGMOID, groups=8, kept=4,
             two=1, k=6, renorm=1, scale=1.0, weights=P[2], indices=P[3])
BACK = dict(T=10, E=64, logits=P[0], type=sg.SGEMM_BF16, ld=64, score=sg.SGEMM_SCORE_SOFTMAX, k=6, renorm=0, scale=1.0,
            indices=P[1], grad_w=P[2], grad_logits=P[3], ld_g=64)
DISPATCH = dict(T=10, k=6, E=64, indices=P[0], offsets=P[1], row_of=P[2], token_of=P[3])
COMBINE = dict(T=10, k=6, cols=64, rows=60, Y=P[0], type=sg.SGEMM_BF16, ldy=64, row_of=P[1], weights=P[2], out=P[3],
               ld_out=64)
CBACK = dict(T=10, k=6, cols=64, rows=60, grad_out=P[0], type=sg.SGEMM_F32, ld_go=64, Y=P[1], ldy=64, row_of=P[2],
             weights=P[3], grad_y=P[4], ld_gy=64, grad_w=P[5])
ARRAYS = [
    ("sgemm_fp8_quantize_rows", dict(ROW, gather=P[6]), dict(src=2, gather=4, scales=4)),
    ("sgemm_fp8_quantize_both", BOTH, dict(src=4, gather=4, offsets=4, scales=4, scales_t=4)),
    ("sgemm_fp8_quantize_blocks", BLOCKS, dict(src=4, scales=4)),
    ("sgemm_fp8", DENSE, dict(sa=4, sb=4, C=2)),
    ("sgemm_fp8_grouped", GROUPED, dict(sa=4, sb=4, offsets=4, C=4)),
    ("sgemm_fp8_grouped_k", GROUPED_K, dict(sa=4, sb=4, offsets=4, C=4)),
    ("sgemm_route", ROUTE, dict(logits=4, bias=4, weights=4, indices=4)),
    ("sgemm_route_backward", BACK, dict(logits=2, indices=4, grad_w=4, grad_logits=2)),
    ("sgemm_dispatch", DISPATCH, dict(indices=4, offsets=4, row_of=4, token_of=4)),
    ("sgemm_combine", COMBINE, dict(Y=2, row_of=4, weights=4, out=2)),
    ("sgemm_combine_backward", CBACK, dict(grad_out=4, Y=4, row_of=4, weights=4, grad_y=4, grad_w=4)),
]


@pytest.mark.parametrize("name,args,array,off", [(name, args, array, off) for name, args, sizes in ARRAYS
                                                 for array, size in sizes.items() for off in {1, size // 2}])
def test_arrays_between_elements_are_refused(name, args, array, off):
    assert getattr(sg, name)(**dict(args, **{array: args[array] + off})) == BAD
