"""The operators of layers called from several host threads, each on its own
stream and with sizes of its own: what one call sets up for its launch is not
undone by another's. ctypes releases the GIL during each call."""

import threading

import pytest
import torch

import dense_fp32_matrix_07_gb300 as sg
from test_experts_gpu import ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("type,dtype", [(sg.SGEMM_F32, torch.float32), (sg.SGEMM_BF16, torch.bfloat16)], ids=["f32", "bf16"])
def test_norms_of_different_widths_side_by_side(cuda_device, type, dtype):
    """Rows that lie apart from each other on 16 bytes pass through shared memory: 43 to 64 KB of it here."""
    rows, calls = 2, 1500
    widths, wrong = (11001, 16383, 13333, 16000), []

    def worker(cols):
        try:
            g = torch.Generator(device="cuda").manual_seed(cols)
            ld = cols + 1
            x, gy = (torch.randn(rows * ld + 8, generator=g, device="cuda").to(dtype) for _ in range(2))
            out = [torch.full((rows * ld + 8,), 5.0, device="cuda", dtype=dtype) for _ in range(4)]
            dw = [torch.full((cols,), 5.0, device="cuda") for _ in range(2)]
            at = x.element_size()                # y and the gradient begin one value further
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.current_stream())

            def both(i):
                return (sg.sgemm_rms_norm(rows, cols, type, x.data_ptr(), ld, 0, 0, 0, 1e-6, 0, 0, out[2 * i].data_ptr() + at, ld, 0, 0,
                                          0, 0, stream.cuda_stream),
                        sg.sgemm_rms_norm_backward(rows, cols, type, gy.data_ptr(), ld, x.data_ptr(), ld, 0, 1e-6, 0, 0,
                                                   out[2 * i + 1].data_ptr() + at, ld, dw[i].data_ptr(), stream.cuda_stream))
            first = both(0)
            start.wait()
            codes = {c for _ in range(calls) for c in both(1)} | set(first)
            stream.synchronize()
            if codes != {sg.SGEMM_OK}:
                wrong.append((cols, [sg.sgemm_error_string(c) for c in codes]))
            elif not all(torch.equal(a, b) for a, b in ((out[0], out[2]), (out[1], out[3]), (dw[0], dw[1]))):
                wrong.append((cols, "other values"))
        except Exception as e:        # surfaced by the assertion below
            wrong.append((cols, repr(e)))
            start.abort()
    start = threading.Barrier(len(widths))
    threads = [threading.Thread(target=worker, args=(c,)) for c in widths]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong, wrong
    ok(sg.sgemm_check_status(torch.cuda.current_stream().cuda_stream))
