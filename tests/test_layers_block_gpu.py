"""The example feed-forward block: a whole training step through the library
against autograd in 64 bits.

A value kept in bfloat16 is off by at most 2^-9 of itself after rounding to
nearest (half a step of 2^-8), by 2^-9 / sqrt(3) in the mean square of a spread
of values. No result of the step depends on more than nine such roundings one
after the other (s, y, u, z, h, the output's or dh, dz or du, dy twice, the
result), each of which reaches it with a factor of about one in the mean square
(the activations' slopes are at most 1.1, and products of independent values
keep relative errors): together 3 * 2^-9 / sqrt(3); four times that is asked for."""

import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu

BOUND = 4 * 3 * 2.0 ** -9 / 3 ** 0.5


@pytest.mark.parametrize("shape", [(2000, 1024, 2048), (37, 200, 136), (1, 128, 256), (4097, 512, 640), (130, 2048, 1000)], ids=str)
def test_training_step_follows_64_bits(cuda_device, shape):
    import feed_forward
    args = feed_forward.inputs(*shape)
    got = feed_forward.step(*args)
    want = feed_forward.reference(*args, dtype=torch.float64)
    for name in want:
        off = float((got[name].double() - want[name]).norm() / want[name].norm())
        assert off < BOUND, (name, off)


def test_gradients_follow_differences(cuda_device):
    """Along a random direction of each parameter, in 64 bits, the loss's difference quotient against the step's gradients."""
    import feed_forward
    args = list(feed_forward.inputs(200, 256, 320, seed=3))
    got = feed_forward.step(*args)
    wide = [a.double() for a in args]

    def loss(params):
        x, r, w, b, Wu, Wg, Wd, grad_out = params
        s = x + r
        y = s / torch.sqrt((s * s).mean(1, keepdim=True) + feed_forward.EPS) * w
        z = y @ Wg.t() + b
        return float((((z / (1 + torch.exp(-z))) * (y @ Wu.t()) @ Wd.t() + s) * grad_out).sum())
    for name, i in (("x", 0), ("w", 2), ("b", 3), ("Wu", 4), ("Wg", 5), ("Wd", 6)):
        # The gradient's own direction: its length is what the quotient gives.
        grad = got[name].double()
        d = grad / grad.norm()
        h = 1e-4 * float(wide[i].norm())
        ends = []
        for sign in (1, -1):
            moved = list(wide)
            moved[i] = wide[i] + sign * h * d
            ends.append(loss(moved))
        quotient = (ends[0] - ends[1]) / (2 * h)
        assert abs(quotient - float(grad.norm())) < BOUND * float(grad.norm()), (name, quotient, float(grad.norm()))


@pytest.mark.parametrize("T", [300, 16])
def test_a_captured_step_replays_beside_an_eager_one(cuda_device, T):
    """A step captured into a graph while an eager one's tensors live, replayed on new inputs: the same bits as eager."""
    import feed_forward
    static = feed_forward.inputs(T, 256, 512, seed=1)
    eager = feed_forward.step(*static)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured = feed_forward.step(*static)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(captured[n], eager[n]) for n in eager)
    fresh = feed_forward.inputs(T, 256, 512, seed=2)
    for a, b in zip(static, fresh):
        a.copy_(b)
    graph.replay()
    want = feed_forward.step(*fresh)
    torch.cuda.synchronize()
    assert all(torch.equal(captured[n], want[n]) for n in want)
