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
