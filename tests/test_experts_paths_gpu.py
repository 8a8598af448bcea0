"""Paths of the experts' operators that the sizes, strides and types of
test_experts_gpu.py do not reach."""

import pytest
import torch

import dense_fp32_matrix_07_gb300 as sg
import experts_ref as ref

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn
TYPES = {sg.SGEMM_F32: torch.float32, sg.SGEMM_BF16: torch.bfloat16}


def stream():
    return torch.cuda.current_stream().cuda_stream


def ok(rc):
    assert rc == sg.SGEMM_OK, sg.sgemm_error_string(rc)


def finish():
    torch.cuda.synchronize()
    assert sg.sgemm_check_status(stream()) == sg.SGEMM_OK


# ---------------------------------------------------------------- quantisers

@pytest.mark.parametrize("form", ["rows", "both", "blocks", "blocks transposed"])
def test_scales_right_behind_the_values(cuda_device, form):
    """One buffer: 8-bit values, and the scales from where the last row's stores end. Exact in every bit."""
    rows, cols = 9, 130
    x = torch.randn(rows, cols, generator=torch.Generator().manual_seed(0))
    src = x.cuda()
    turned = form == "blocks transposed"
    qr, qc, ld = (cols, rows, 16) if turned else (rows, cols, 144)
    end = (qr - 1) * ld + (16 if turned else 136)
    shape = (2, rows) if form in ("rows", "both") else (-(-qr // 128), -(-qc // 128))
    buf = torch.zeros(end + 4 * shape[0] * shape[1], dtype=torch.uint8, device="cuda")
    q, s = buf.data_ptr(), buf.data_ptr() + end
    if form == "rows":
        ok(sg.sgemm_fp8_quantize_rows(rows, cols, src.data_ptr(), sg.SGEMM_F32, cols, 0, rows, q, ld, s, rows, stream()))
    elif form == "both":
        qt, st = torch.zeros(cols, 128, dtype=FP8, device="cuda"), torch.zeros(1, cols, device="cuda")
        ok(sg.sgemm_fp8_quantize_both(rows, cols, src.data_ptr(), sg.SGEMM_F32, cols, 0, rows, 1, 0, 128, q, ld, s, rows,
                                      qt.data_ptr(), 128, st.data_ptr(), cols, stream()))
    else:
        ok(sg.sgemm_fp8_quantize_blocks(rows, cols, src.data_ptr(), sg.SGEMM_F32, cols, 0, int(turned), q, ld, 0, s,
                                        shape[1], 0, 1, stream()))
    finish()
    wq, ws = ref.quantize(x.t().contiguous() if turned else x, 1 if form in ("rows", "both") else None)
    got = torch.zeros(qr * ld, dtype=torch.uint8)
    got[:end] = buf.cpu()[:end]
    assert torch.equal(got.view(qr, ld)[:, :qc].contiguous().view(FP8).float(), wq.float())
    scales = buf[end:].cpu().view(torch.float32).view(shape)
    assert torch.equal(scales, ws.t() if form in ("rows", "both") else ws)
