"""The low-rank delta of the projection with pooled adapters keeps its bits: s v (and u of the gradient) enter the
second product as two bf16 terms, not as one rounding of 2^-8."""

import numpy as np
import pytest
import torch

from gpu_util import dev, f64, say
from oracle import operators_ref as ref
from test_gpu_project import HALF, ULP, Case

pytestmark = pytest.mark.gpu

# A value as two bf16 terms: the first leaves at most 2^-8 of it, the second at most 2^-8 of that.
TWO = 2.0 ** -16

# T, K, N, R: each tile of the few-token product, then the LDS tiles of 64, 128 and 256; ranks that share a step of the
# expand and ranks that fill several
SHAPES = [(1, 512, 1024, 16), (16, 136, 712, 128), (16, 136, 8200, 8), (31, 264, 4104, 24), (64, 512, 4104, 16),
          (250, 72, 2056, 40), (513, 328, 4104, 8), (700, 136, 4104, 16), (700, 136, 4104, 64), (2049, 72, 2400, 24),
          (2049, 200, 2400, 128), (3200, 136, 4104, 32), (3200, 136, 4104, 72)]


@pytest.mark.parametrize("T,K,N,R", SHAPES)
def test_the_delta_alone(T, K, N, R):
    """W = 0, so that y is the delta: sums of R terms that cancel show what each term has lost."""
    say(f"[delta] T={T} K={K} N={N} R={R}")
    c = Case(T, K, N, 4, R, seed=31)
    c.w.zero_()
    y, v = c.forward()
    a, b = c.clean
    x = f64(c.x)
    want, want_v = ref.project(x, np.zeros((N, K)), c.slot, c.rank, c.scaling, a, b)
    # the terms of each output without their signs (v itself is an fp32 sum of K products)
    size, v_size = np.zeros_like(want), np.zeros_like(want)
    for s in range(c.S):
        rows, r = np.flatnonzero(c.slot == s), min(max(c.rank[s], 0), R)
        scale, b_abs = float(c.scaling[s]), np.abs(b[s, :, :r]).T
        size[rows] = scale * np.abs(want_v[rows, :r]) @ b_abs
        v_size[rows] = scale * (np.abs(x[rows]) @ np.abs(a[s, :r]).T) @ b_abs
    tol = HALF * np.abs(want) + 1.01 * TWO * size + 2 * (K + 2 * R + 16) * ULP * v_size
    err = np.abs(f64(y) - want)
    assert (err <= tol).all(), float((err - tol).max())


@pytest.mark.parametrize("T,K,N,R", [(64, 1032, 264, 16), (64, 4104, 72, 128), (300, 1032, 200, 24), (700, 2056, 136, 8),
                                     (2049, 2400, 72, 32), (3200, 4104, 136, 72)])
def test_the_delta_of_the_input_gradient_alone(T, K, N, R):
    say(f"[delta of dx] T={T} K={K} N={N} R={R}")
    c = Case(T, K, N, 4, R, seed=32)
    c.w.zero_()
    dx = f64(c.backward(want=("dx",))["dx"])
    a, b = c.clean
    dy = f64(c.dy)
    want, size, u_size = np.zeros((T, K)), np.zeros((T, K)), np.zeros((T, K))
    for s in range(c.S):
        rows, r = np.flatnonzero(c.slot == s), min(max(c.rank[s], 0), R)
        scale, a_abs = float(c.scaling[s]), np.abs(a[s, :r])
        u = scale * (dy[rows] @ b[s, :, :r])
        want[rows] = u @ a[s, :r]
        size[rows] = np.abs(u) @ a_abs
        u_size[rows] = scale * (np.abs(dy[rows]) @ np.abs(b[s, :, :r])) @ a_abs
    tol = HALF * np.abs(want) + 1.01 * TWO * size + 2 * (N + 2 * R + 16) * ULP * u_size
    err = np.abs(dx - want)
    assert (err <= tol).all(), float((err - tol).max())


@pytest.mark.parametrize("T", [40, 700])
def test_an_infinite_v_stays_an_infinity(T):
    """A token whose v overflows: its second term is zero, so that the outputs keep the sign of the product."""
    c = Case(T, 64, 4104, 2, 16, mixed=True, dirty=False)
    c.slot[:], c.rank[:] = 1, 16
    c.pool.token_slot.fill_(1)
    c.pool.rank.fill_(16)
    c.pool.scaling.fill_(1.0)
    c.w.zero_()
    c.a.zero_()
    c.b[1].zero_()
    c.a[1, 3, 0], c.b[1, :, 3] = 2.0, 1.0
    c.b[1, 1::2, 3] = -1.0
    c.x[:, 0] = 1.0
    c.x[5, 0] = 3e38
    y = c.forward()[0]
    assert (y[5, 0::2] == float("inf")).all() and (y[5, 1::2] == float("-inf")).all()
    keep = torch.ones(T, dtype=torch.bool, device=dev())
    keep[5] = False
    assert (y[keep][:, 0::2] == 2.0).all() and (y[keep][:, 1::2] == -2.0).all()


