"""Renormalised router weights and their gradients where the scores themselves
are far below what 32 bits hold: the weights are ratios, so a common factor of
the scores (exp of the row's largest logit, of a very negative logit) must not
cost range or digits.

Tolerances. Each of the k scores is an exponential of a rounded difference of
logits (2 ulp, and 2^-24 of the logits' distance), for the sigmoid over a sum
of two numbers (2 ulp); the weights divide by their sum (k + 1 roundings): with
distances below 16, (16 + 4 + k + 2) 2^-23 relative. The gradient is a weight
times the scale times a difference of two numbers of the gradients' magnitude:
the same bound on scale * weight * 2 max |g|, and k + 4 roundings more."""

import numpy as np
import pytest
import torch

import dense_fp32_matrix_07_gb300 as sg

pytestmark = pytest.mark.gpu

SOFTMAX, SIGMOID = sg.SGEMM_SCORE_SOFTMAX, sg.SGEMM_SCORE_SIGMOID


def stream():
    return torch.cuda.current_stream().cuda_stream


def ok(rc):
    assert rc == sg.SGEMM_OK, sg.sgemm_error_string(rc)


def finish():
    torch.cuda.synchronize()
    assert sg.sgemm_check_status(stream()) == sg.SGEMM_OK


def tolerance(k):
    return (16 + 4 + k + 2) * 2.0 ** -23


def shares(l, kind):
    """64-bit ratios of the scores of the logits l, by logarithms: log sigmoid(l) = -log(1 + exp(-l))."""
    l = l.astype(np.float64)
    log = l if kind == SOFTMAX else -np.logaddexp(0.0, -l)
    x = np.exp(log - log.max(1, keepdims=True))
    return x / x.sum(1, keepdims=True)


def gradient(l, kind, g, scale):
    """dl_j = scale w_j (g_j - sum w_i g_i), for the sigmoid times its own 1 - s_j."""
    w = shares(l, kind)
    d = scale * w * (g - (w * g).sum(1, keepdims=True))
    return d if kind == SOFTMAX else d / (1.0 + np.exp(l.astype(np.float64)))


def backward(l, kind, indices, g, scale):
    """The library's gradient, as a (T, E) array."""
    T, E = l.shape
    dl, di = torch.tensor(l).cuda(), torch.tensor(indices, dtype=torch.int32).cuda()
    dg, out = torch.tensor(g).cuda(), torch.empty(T, E, device="cuda")
    ok(sg.sgemm_route_backward(T, E, dl.data_ptr(), sg.SGEMM_F32, E, kind, indices.shape[1], 1, scale, di.data_ptr(),
                               dg.data_ptr(), out.data_ptr(), E, stream()))
    finish()
    return out.cpu().numpy().astype(np.float64)


# Chosen logits: near the sum that scale / sum overflows at, below the least
# normal score, below the least score, and ordinary ones.
LOGITS = [[-88.3, -88.5], [-90.0, -91.5], [-110.0, -104.25], [-5.0, 2.5], [-3.0, -88.0], [30.0, 31.0]]


@pytest.mark.parametrize("scale", [1.0, 16.0])
@pytest.mark.parametrize("k", [1, 2])
def test_sigmoid_gradient_of_very_small_scores(cuda_device, k, scale):
    T, E = len(LOGITS), 4
    l = np.full((T, E), -200.0, np.float32)
    l[:, 1:3] = LOGITS
    indices = np.tile(np.array([[1, 2]]), (T, 1))[:, :k].copy()
    g = np.random.RandomState(0).randn(T, k).astype(np.float32)
    got = backward(l, SIGMOID, indices, g, scale)
    at = l[np.arange(T)[:, None], indices]
    w, want = shares(at, SIGMOID), np.zeros((T, E))
    np.put_along_axis(want, indices, gradient(at, SIGMOID, g, scale), 1)
    bound = np.zeros((T, E))
    # (distances of up to 85 in one row: 2^-24 of that, in the exponent)
    np.put_along_axis(bound, indices, scale * w * 2 * np.abs(g).max() * (tolerance(k) + 85 * 2.0 ** -23), 1)
    assert np.isfinite(got).all()
    assert np.all(np.abs(got - want) <= bound + 1e-38), np.abs(got - want).max()


def forward(l, kind, bias, k, scale):
    """The library's renormalised weights and choice for logits l (T, E)."""
    T, E = l.shape
    dl, db = torch.tensor(l).cuda(), torch.tensor(bias).cuda() if bias is not None else None
    w, ix = torch.empty(T, k, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda")
    ok(sg.sgemm_route(T, E, dl.data_ptr(), sg.SGEMM_F32, E, db.data_ptr() if bias is not None else 0, kind, 1, 1, 0, k, 1,
                      scale, w.data_ptr(), ix.data_ptr(), stream()))
    finish()
    return w.cpu().numpy().astype(np.float64), ix.cpu().numpy()


@pytest.mark.parametrize("E", [8, 64, 128, 512])
def test_softmax_weights_of_a_biased_choice_far_below_the_best(cuda_device, E):
    """A bias chooses experts whose scores are denormal or zero in 32 bits; the gradient is that of these weights."""
    k, scale = 3, 2.0
    chosen = np.array([[-100.0, -101.0, -102.5], [-104.0, -105.0, -103.0], [-300.0, -301.0, -302.0],
                       [-1.0, -2.0, -3.0], [-86.0, -88.0, -90.0]], np.float32)
    T = len(chosen)
    l = np.full((T, E), -9.0, np.float32)
    l[:, 0], l[:, 1:4] = 0.0, chosen
    bias = np.zeros(E, np.float32)
    bias[1:4] = 9.0, 7.0, 5.0
    w, ix = forward(l, SOFTMAX, bias, k, scale)
    assert (ix == [1, 2, 3]).all()
    want = scale * shares(chosen, SOFTMAX)
    assert np.all(np.abs(w - want) <= tolerance(k) * want), np.abs(w / want - 1).max()
    g = np.random.RandomState(1).randn(T, k).astype(np.float32)
    d = np.zeros((T, E))
    d[:, 1:4] = gradient(chosen, SOFTMAX, g, scale)
    got = backward(l, SOFTMAX, ix, g, scale)
    bound = np.zeros((T, E))
    bound[:, 1:4] = want * 2 * np.abs(g).max() * tolerance(k)
    assert np.all(np.abs(got - d) <= bound)


@pytest.mark.parametrize("E", [8, 64, 128, 512])
@pytest.mark.parametrize("biased", [False, True], ids=["by_logit", "biased"])
def test_sigmoid_weights_of_very_small_scores(cuda_device, E, biased):
    k, scale = 2, 2.5
    T = len(LOGITS)
    l = np.full((T, E), -200.0, np.float32)
    l[:, 1:3] = LOGITS
    bias = None
    if biased:
        bias = np.zeros(E, np.float32)
        bias[1:3] = 3.0, 5.0
    w, ix = forward(l, SIGMOID, bias, k, scale)
    at = np.take_along_axis(l, ix, 1)
    assert (np.sort(ix, 1) == [1, 2]).all()
    want = scale * shares(at, SIGMOID)
    assert np.all(np.abs(w - want) <= (tolerance(k) + 85 * 2.0 ** -23) * want + 1e-38), np.abs(w / want - 1).max()
