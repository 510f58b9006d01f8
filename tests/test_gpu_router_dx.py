"""The router's gradient in its activations, dx = dl W, against 64 bits where
the router's weights are what makes it hard.

Tolerances (u = 2^-24).  More than a few tokens take dl and W to f16, each row
of dl and each 32 columns of W first times the power of two that puts their
largest magnitude in [2^14, 2^15): half a step of f16 is 2^-11 relative, so the
products lose at most 2^-10 (1 + 2^-10) of sum |dl| |W|, and 2^-25 absolute
below f16's normal range, that is 2^-39 of the largest magnitude on either side.
The fp32 sums of up to 256 products lose (3 E / 8 + 64) u of sum |dl| |W|, and
the result is rounded to bf16, half a step 2^-8.
"""
import math

import pytest

torch = pytest.importorskip("torch")

from quantized_routed_expert_04_b200 import binding  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def normal(*shape, seed):
    return torch.randn(*shape, device="cuda", generator=gen(seed))


def dx_of(W, x, dlogits):
    """dx as the layer computes it, and the status of the call."""
    E, H = W.shape
    layer = binding.StrataMoE(H, 128, E, 1, 0, E)
    layer.set_router(W, None)
    dx = torch.full_like(x, 7.0)
    ws = torch.empty(layer.route_backward_workspace(x.shape[0]), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)
    layer.route_backward(x, None, None, None, dlogits, None, None, dx, ws)
    status = layer.status()
    layer.close()
    return dx, status


def check(W, dlogits, operand, what):
    """operand: what the rounding of the operands may lose of sum |dl| |W|."""
    (T, E), H = dlogits.shape, W.shape[1]
    x = normal(T, H, seed=1).bfloat16()
    dx, status = dx_of(W, x, dlogits)
    # (weights past the limit are reported, and dx is had all the same)
    large = float(W.abs().max()) >= 65520 / 256
    assert status == (binding.Status.RANGE, 16) if large else int(status[0]) == 0, status
    dl, w = dlogits.double(), W.double()
    want = dl @ w
    top = w.abs().view(E, H // 32, 32).amax((0, 2)).repeat_interleave(32)
    tol = (dl.abs() @ w.abs()) * (operand + (3 * E / 8 + 64) * U) + want.abs() * 2.0 ** -8 + \
        dl.abs().amax(1, keepdim=True) * w.abs().sum(0) * 2.0 ** -39 + \
        dl.abs().sum(1, keepdim=True) * top * 2.0 ** -39
    err = (dx.double() - want).abs()
    assert bool((err <= tol).all()), "%s: worst ratio %.3g" % (what, float((err / tol.clamp(min=1e-300)).max()))


SHAPES = [(3, 16, 256), (600, 64, 256), (1030, 256, 384), (700, 100, 1152), (5000, 8, 128)]


@pytest.mark.parametrize("T,E,H", SHAPES)
@pytest.mark.parametrize("size", [1e-5, 1e-7, 1e-9, 1e-20])
def test_dx_of_small_router_weights(T, E, H, size):
    check(normal(E, H, seed=2) * size, normal(T, E, seed=3), 2.0 ** -10 * (1 + 2.0 ** -9), size)


@pytest.mark.parametrize("T,E,H", SHAPES)
def test_dx_of_columns_of_every_size(T, E, H):
    size = 10.0 ** (torch.arange(H, device="cuda") // 32 % 24 - 22.0)
    check(normal(E, H, seed=4) * size, normal(T, E, seed=5), 2.0 ** -10 * (1 + 2.0 ** -9), "columns")
    # and gradients whose rows are as far apart
    rows = 10.0 ** (torch.arange(T, device="cuda") % 16 - 8.0)
    check(normal(E, H, seed=4) * 1e-6, normal(T, E, seed=5) * rows[:, None], 2.0 ** -10 * (1 + 2.0 ** -9), "rows")


# Rows of W with something in common, and rows of dl that sum to zero, as those of
# a softmax do: what is common cancels, and what the operands' rounding loses of it
# does not.  Each operand is two f16 numbers: 2^-22 relative each, and 2^-22 for the
# product of the two small parts, which is left out; 16 u for 12 u and its squares.
@pytest.mark.parametrize("T,E,H", SHAPES)
@pytest.mark.parametrize("common", [0, 4, 64, 1000])
def test_dx_of_router_weights_with_a_common_part(T, E, H, common):
    W = (normal(E, H, seed=6) + common * normal(1, H, seed=7)) / math.sqrt(H)
    p = torch.softmax(normal(T, E, seed=8), 1).double()
    f = torch.rand(E, device="cuda", generator=gen(9)).double()
    dlogits = (p * (f - p @ f[:, None])).float()
    check(W, dlogits, 16 * U, "common %g" % common)
    # and rows far from the others: one expert's, an eighth of them
    W[0] *= 1e4
    check(W, dlogits, 16 * U, "one large")
    W[::8] *= -300
    check(W, dlogits, 16 * U, "some large")
