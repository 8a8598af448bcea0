"""The set-up of the experts' kernels on a device: by their own first call, and
without the FP32 products. Each case runs in a process of its own, whose first
calls are what is tested."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu

PRELUDE = """
import torch
import dense_fp32_matrix_07_gb300 as sg

n = 96
g = torch.Generator().manual_seed(0)
A, B = (torch.randint(-4, 5, (n, n), generator=g).float() for _ in range(2))
dA, dB, C = A.cuda(), B.cuda(), torch.full((n, n), float("nan"), device="cuda")
q, s = torch.zeros(n, n, dtype=torch.uint8, device="cuda"), torch.zeros(1, n, device="cuda")
w, sw = torch.zeros(n, n, dtype=torch.uint8, device="cuda"), torch.zeros(1, 1, device="cuda")
off = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
ix, row, tok = (torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(3))
wt, P = torch.zeros(n, device="cuda"), torch.full((n, n), float("nan"), device="cuda")


def fp32(st=0):
    return sg.sgemm(n, n, n, dA.data_ptr(), n, dB.data_ptr(), n, C.data_ptr(), n, st)


def experts(st=0):
    return [sg.sgemm_fp8_quantize_rows(n, n, dA.data_ptr(), 0, n, 0, n, q.data_ptr(), n, s.data_ptr(), n, st),
            sg.sgemm_fp8_quantize_blocks(n, n, dB.data_ptr(), 0, n, 0, 0, w.data_ptr(), n, 0, sw.data_ptr(), 1, 0, 1, st),
            sg.sgemm_fp8(0, n, n, n, q.data_ptr(), n, s.data_ptr(), n, w.data_ptr(), n, sw.data_ptr(), 1, 0.0,
                         P.data_ptr(), 0, n, st),
            sg.sgemm_route(n, n, dA.data_ptr(), 0, n, 0, 0, 1, 1, 0, 1, 1, 1.0, wt.data_ptr(), ix.data_ptr(), st),
            sg.sgemm_dispatch(n, 1, n, ix.data_ptr(), off.data_ptr(), row.data_ptr(), tok.data_ptr(), st)]


def check(c, p):
    torch.cuda.synchronize()
    assert sg.sgemm_check_status(0) == 0
    if c:
        assert torch.equal(C.cpu(), A @ B)
    if p:
        # In blocks whose largest is 4, values are held as multiples of 1 / 112: 1, 2 and 4 as 7, 14 and 28 times 16,
        # exact; 3 as 21 times 16, whose fifth bit is rounded off (to even: 20).
        a = torch.where(A.abs() == 3, A * (20.0 / 21.0), A)
        b = torch.where(B.abs() == 3, B * (20.0 / 21.0), B)
        assert bool(((P.cpu() - a @ b.t()).abs() <= 1e-5 * (a.abs() @ b.abs().t()) + 1e-5).all())
        assert int(off[n]) == n and bool((wt == 1).all())
"""


def run(body):
    r = subprocess.run([sys.executable, "-c", PRELUDE + body], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]


def test_products_in_fp32_do_not_set_up_the_experts_kernels(cuda_device):
    run("""
assert sg.sgemm_test_fail_next_setups(1) == sg.SGEMM_OK
assert fp32() == sg.SGEMM_OK
check(True, False)
assert experts()[0] == sg.SGEMM_ERR_CUDA                       # the pending failure is theirs
C.fill_(0)
assert fp32() == sg.SGEMM_OK and experts() == [sg.SGEMM_OK] * 5
check(True, True)
""")


def test_first_experts_call_in_a_capture(cuda_device):
    """A product in FP32 has run; the experts' first calls are captured, then replayed."""
    run("""
side = torch.cuda.Stream()
assert fp32(side.cuda_stream) == sg.SGEMM_OK
side.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=side):
    codes = experts(torch.cuda.current_stream().cuda_stream)
assert codes == [sg.SGEMM_OK] * 5, codes
graph.replay()
check(True, True)
""")


def test_first_calls_of_several_threads(cuda_device):
    run("""
import threading
streams = [torch.cuda.Stream() for _ in range(4)]
codes = [None] * 4
x = torch.randn(n, n).cuda()
outs = [(torch.zeros(n, n, dtype=torch.uint8, device="cuda"), torch.zeros(1, n, device="cuda")) for _ in range(4)]
torch.cuda.synchronize()


def work(i):
    codes[i] = [sg.sgemm_fp8_quantize_rows(n, n, x.data_ptr(), 0, n, 0, n, outs[i][0].data_ptr(), n, outs[i][1].data_ptr(),
                                           n, streams[i].cuda_stream) for _ in range(5)]


threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
for t in threads:
    t.start()
for t in threads:
    t.join()
assert codes == [[sg.SGEMM_OK] * 5] * 4
torch.cuda.synchronize()
assert all(torch.equal(o[0], outs[0][0]) and torch.equal(o[1], outs[0][1]) for o in outs) and bool(outs[0][0].any())
""")
