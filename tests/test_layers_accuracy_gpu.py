"""How near the activations and their slopes come to their formulas relative to
their own size, down to where they vanish, in both output types.

Sums that are exact (an empty product plus the bias) leave the activation's own
error. By their formulas in FP32, in units u = 2^-24: the hardware's 2^x is off
by 4 u, its reciprocal by 2 u, a sum or product by 1 u, a constant by u / 2; an
exponential's argument x has x times its relative error.
  silu       -z log2(e): 1.5 u |z|; exponential, sum, reciprocal, product 8 u.
  gelu_tanh  the argument x = 1.596 |z| + 0.0714 |z|^3 is five roundings and two
             constants, the one for 2^x 1.5 more: 7 u x < (12 |z| + 0.5 |z|^3) u; 8 u.
  gelu       exp(-z^2 / 2): z^2 / 2 (2.5 u); t = 1 / (1 + p |z|): 4.5 u, of which
             a polynomial in t with d ln q / d ln t <= 2.7 makes 12 u; its fit
             2.5 u and steps 6 u, the exponential 4 u, three products 3 u:
             (28 + 1.25 z^2) u; (32 + 2 z^2) u is asked for.
Below 2^-126 a sigmoid or an exponential may be 0, which times |z| is lost.
Storing a value rounds it by half a step of its type."""

import math

import pytest
import torch

import dense_fp32_matrix_07_gb300 as sg
from test_experts_gpu import finish, ok, stream

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {sg.SGEMM_F32: torch.float32, sg.SGEMM_BF16: torch.bfloat16}
GELU, GELU_TANH, SILU = sg.SGEMM_ACT_GELU, sg.SGEMM_ACT_GELU_TANH, sg.SGEMM_ACT_SILU


def argument(z):
    return 2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)


def formula(z, act):
    """(activation, relative bound) in 64 bits, without cancellation."""
    if act == GELU:
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0)), (32 + 2 * z * z) * U
    if act == GELU_TANH:
        return z / (1.0 + torch.exp(-argument(z))), (8 + 12 * z.abs() + 0.5 * z.abs() ** 3) * U
    return z / (1.0 + torch.exp(-z)), (8 + 2 * z.abs()) * U


def grid(low, high):
    return torch.linspace(low, high, 4001, device="cuda", dtype=torch.float64).float()


def held(got, want, bound, z):
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    assert not bool(bad.any()), (int(bad.sum()), float(z[bad][0]), float(got.double()[bad][0]), float(want[bad][0]),
                                 float((off / want.abs())[bad].max()))


@pytest.mark.parametrize("act", [GELU, GELU_TANH, SILU], ids=["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("type", TYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 300])
def test_activations_relative_to_themselves(cuda_device, act, type, M):
    z, dtype = grid(-12, 12), TYPES[type]
    C = torch.full((M, z.numel()), 7.0, device="cuda", dtype=dtype)
    ok(sg.sgemm_bf16(0, 1, M, z.numel(), 0, 0, 0, 0, 0, z.data_ptr(), act, 0, 0, 0, 0, 0, C.data_ptr(), type, z.numel(), stream()))
    finish()
    x = z.double()
    want, rel = formula(x, act)
    half = torch.finfo(dtype).eps / 2
    bound = want.abs() * (rel + half * (1 + rel)) + x.abs() * 2.0 ** -125
    for row in C[:: max(1, M - 1)]:
        held(row, want, bound, z)


@pytest.mark.parametrize("act", [GELU, GELU_TANH, SILU], ids=["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("type", TYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("low,high", [(-12, -2), (-2, 12)], ids=["tail", "rest"])
def test_slopes_relative_to_their_terms(cuda_device, act, type, low, high):
    """The slopes are sums of two terms with the activations' relative errors, and at most eight more roundings:
    Phi + z phi; s + z s (1 - s) x'(z) for a sigmoid s of x. Where s is near 1 it is off by 2.5 u, and so is 1 - s:
    2.5 u z x' = (4 z + 0.54 z^3) u for gelu_tanh (up to z = 5.4, where s is 1 in FP32) and 2.5 u z for silu are within
    the same bounds, as the terms are at least s."""
    dtype = TYPES[type]
    z = grid(low, high).to(dtype)
    n = z.numel()
    g, dz = torch.ones(n, device="cuda", dtype=dtype), torch.empty(n, device="cuda", dtype=dtype)
    ok(sg.sgemm_epilogue_backward(1, n, type, g.data_ptr(), n, z.data_ptr(), n, act, 0, 0, 0, 1, 0, dz.data_ptr(), n, 0, 0, 0, 0, stream()))
    finish()
    x = z.double()
    _, rel = formula(x, act)
    if act == GELU:
        terms = 0.5 * torch.special.erfc(-x / math.sqrt(2.0)), x * torch.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)
    else:
        a, rise = (x, 1.0) if act == SILU else (argument(x), 2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 3 * 0.044715 * x * x))
        s = 1.0 / (1.0 + torch.exp(-a))
        terms = s, x * s * (1.0 - s) * rise
    want, size = terms[0] + terms[1], terms[0].abs() + terms[1].abs()
    e = size * (rel + 8 * U)
    # What a sigmoid or an exponential of 0 loses, times |z| x'(z) <= 12 * 33.
    held(dz, want, e + torch.finfo(dtype).eps / 2 * (want.abs() + e) + 400 * 2.0 ** -125, z.float())
