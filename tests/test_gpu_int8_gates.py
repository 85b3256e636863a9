"""The gate of the INT8 products far out on both sides, in each of their kernels: silu(g) u from its
definition in 64 bits."""
import numpy as np
import pytest
import torch

from qwtest import dev
from test_gpu_int8 import call, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [16, 4096])
@pytest.mark.parametrize("M", [1, 2, 3, 16, 17, 64, 200, 700])
def test_far_gates(M, K):
    """Gates of -120 to 120 before up values of 2^100 and 1: silu(g) u with 2^-19 relative error (expf
    2 ulp, a product, a division of 2 ulp, scales) beside what an FP32 below its normal range may lose,
    2^-149 of e^g times g u, and the result's BF16 rounding."""
    gates = np.array([-120, -104, -103, -100, -95, -90, -89, -88, -87, -86, -80, -40, -1, 0, 1, 40, 87,
                      88, 89, 100, 120])
    n = len(gates)
    p = problem(M, 4 * n, K, 5, a="int8")
    q = np.zeros((M, K), dtype=np.int8)
    q[:, K // 2] = 1
    w = np.zeros((4 * n, K), dtype=np.int8)
    w[:2 * n, K // 2] = np.tile(gates, 2)
    w[2 * n:, K // 2] = 1
    sw = np.ones(4 * n, dtype=np.float32)
    sw[2 * n:3 * n] = 2.0 ** 100
    p.update(w=w, sw=sw, A=dev(q), sa_t=torch.ones(M, device="cuda"))
    out = call(p, gated=True)
    g = np.tile(gates, 2).astype(np.float64)
    u = sw[2 * n:].astype(np.float64)
    want = g / (1 + np.exp(-g)) * u
    tol = np.abs(want) * (2.0 ** -8 + 2.0 ** -19) + 2.0 ** -149 * (1 + np.abs(g)) * np.abs(u) + 2.0 ** -133
    bad = ~(np.abs(out - want) <= tol)
    assert not bad.any(), sorted({(gates[c % n], out[r, c], want[c]) for r, c in np.argwhere(bad)})
