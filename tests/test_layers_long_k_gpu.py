"""Sums over a long K into bfloat16 are FP32 sums, whatever the length: the
tensor cores cut a running sum off with each 16 of K, and what that adds up to
has to stay far below the rounding to bfloat16 (half a step, 2^-8): CUT = 2^-11
is allowed in any result, a quarter of it on average.

Operands are positive, so that every cut is a loss (summed over all of K in
tensor memory, 6e-9 K of a result). Rows and columns differ in size by random
factors within a power of two, so that the roundings to bfloat16 (2^-8 at most,
evenly spread) average out: the mean of n results is off by 6 * 2^-8 / sqrt(3 n)
at most."""

import pytest
import torch

import dense_fp32_matrix_07_gb300 as sg
from test_experts_gpu import finish, ok, stream

pytestmark = pytest.mark.gpu

BF16 = sg.SGEMM_BF16
CUT = 2.0 ** -11


def positive(g, k, n):
    """K x N values in [0.5, 2), each column with a size of its own."""
    x = torch.rand(k, n, generator=g, device="cuda", dtype=torch.float32).add_(1.0)
    return x.mul_(0.5 + 0.5 * torch.rand(n, generator=g, device="cuda")).bfloat16()


def product(a, b):
    """a^T . b in 64 bits, a part of K at a time."""
    return sum(p.double().t() @ q.double() for p, q in zip(a.split(1 << 18), b.split(1 << 18)))


def check(got, want):
    off = (got.double() - want) / want
    half = torch.finfo(torch.bfloat16).eps / 2
    assert float(off.abs().max()) <= half + CUT * (1 + half)
    assert abs(float(off.mean())) <= CUT / 4 + 6 * half / (3 * off.numel()) ** 0.5, float(off.mean())


@pytest.mark.parametrize("counts", [[1 << 22], [1 << 21, 0, (1 << 20) + 37, 65, 1 << 16]], ids=["one", "ragged"])
@pytest.mark.parametrize("accumulate", [0, 1])
def test_weight_gradients_of_many_rows(cuda_device, counts, accumulate):
    M, N, E, R = 128, 136, len(counts), sum(counts)
    g = torch.Generator(device="cuda").manual_seed(E)
    a, b = positive(g, R, M), positive(g, R, N)
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    C = torch.ones(E, M, N, device="cuda").bfloat16()
    ok(sg.sgemm_bf16_grouped_k(E, off.data_ptr(), R, M, N, a.data_ptr(), M, b.data_ptr(), N, accumulate, C.data_ptr(), BF16, N, M * N,
                               stream()))
    finish()
    at = 0
    for e, n in enumerate(counts):
        if n == 0:
            assert bool((C[e] == accumulate).all())
        else:
            check(C[e], product(a[at:at + n], b[at:at + n]) + accumulate)
        at += n


@pytest.mark.parametrize("M,N,K", [(1104, 1304, 1 << 18), (2104, 200, (1 << 19) + 8)], ids=str)
@pytest.mark.parametrize("join", [sg.SGEMM_JOIN_NONE, sg.SGEMM_JOIN_ADD], ids=["none", "add"])
def test_dense_products_of_a_long_k(cuda_device, M, N, K, join):
    g = torch.Generator(device="cuda").manual_seed(K + M)
    a, b = positive(g, K, M), positive(g, K, N)
    want = product(a, b)
    d = (want * 0.5).bfloat16()
    C, pre = torch.empty(M, N, device="cuda").bfloat16(), torch.empty(M, N, device="cuda").bfloat16()
    ok(sg.sgemm_bf16(1, 0, M, N, K, a.data_ptr(), a.stride(0), b.data_ptr(), N, 0, 0, pre.data_ptr(), N, join, d.data_ptr(), N,
                     C.data_ptr(), BF16, N, stream()))
    finish()
    check(pre, want)
    check(C, want + d.double() if join else want)


def test_groups_of_rows_of_a_long_k(cuda_device):
    counts, N, K = [1200, 0, 1300], 1304, 1 << 18
    E, R = len(counts), sum(counts)
    g = torch.Generator(device="cuda").manual_seed(7)
    a = positive(g, K, R).t().contiguous()
    b = torch.stack([positive(g, K, N) if n else torch.zeros(K, N, device="cuda").bfloat16() for n in counts])
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    C = torch.empty(R, N, device="cuda").bfloat16()
    ok(sg.sgemm_bf16_grouped(0, E, off.data_ptr(), R, N, K, a.data_ptr(), K, b.data_ptr(), N, K * N, 0, 0, 0, 0, 0, 0, 0, 0, C.data_ptr(),
                             BF16, N, stream()))
    finish()
    check(C[:1200], product(a[:1200].t(), b[0]))
    check(C[1200:], product(a[1200:].t(), b[2]))
