"""The INT8 quantiser over the range of its inputs, from the definition: a code times its row's scale is the
value to half a scale."""
import numpy as np
import pytest
import torch

from qwtest import dev, host, qw
from test_gpu_int8 import bf16

pytestmark = pytest.mark.gpu

MIN_NORMAL = 2.0 ** -126


@pytest.mark.parametrize("K", [16, 1040, 5008])
def test_codes_times_scale_are_the_values(K):
    """Rows of every magnitude from 2^-133 to the largest BF16.  Bound: half a scale, plus what the scale
    (amax / 127 rounded to FP32, to 2^-24 or 2^-150) and the code's quotient and product (2^-22 of 127)
    may be off.  Rows without a normal number count as zeros."""
    Q = qw()
    rng = np.random.default_rng(K)
    tops = [3.3895e38, 1e38, 1e30, 1.0, 1e-30, 1e-36, 4e-37, 3.8e-37, 3.76e-37, 3.745e-37, 3.73e-37, 3.7e-37,
            2e-37, 1e-37, 5e-38, 2e-38, 1.2e-38, MIN_NORMAL, MIN_NORMAL / 2, 1e-39, 2.0 ** -133, 0.0]
    x = rng.uniform(-1, 1, (len(tops), K)) * np.array(tops)[:, None]
    x[np.arange(len(tops)), rng.integers(0, K, len(tops))] = tops
    x, xt = bf16(x)
    rows = len(tops)
    q = torch.full((rows, K), 99, dtype=torch.int8, device="cuda")
    s = torch.empty(rows, device="cuda")
    err = Q.new_error_flag()
    Q.qw_quantize_int8(xt.cuda(), K, rows, K, q, s, err)
    assert Q.qw_read_error(err) == 0
    q, s, x = host(q).astype(np.float64), host(s).astype(np.float64), x.astype(np.float64)
    amax = np.abs(x).max(axis=1)
    some = amax >= MIN_NORMAL
    assert (np.abs(q[some]).max(axis=1) == 127).all()  # the codes' whole range is used
    tol = (amax / 127 * (0.5 + 127 * 2.0 ** -21) + 127 * 2.0 ** -150)[:, None]
    off = np.abs(q * s[:, None] - x)
    assert (off[some] <= np.broadcast_to(tol, x.shape)[some]).all(), \
        [(amax[r], off[r].max() / amax[r]) for r in range(rows) if (off[r] > tol[r]).any()]
    assert (q[~some] == 0).all() and (s[~some] <= MIN_NORMAL / 127).all()


@pytest.mark.parametrize("M", [1, 2, 9, 40])
def test_product_of_small_rows(M):
    """The quantisers inside the product are the same: the product of a row of 1e-37 is that row's.
    Bound: half a scale per value, the scales' product (FP32, 2^-24 or 2^-150) and the sum."""
    Q = qw()
    K, N = 1040, 24
    rng = np.random.default_rng(M)
    x, xt = bf16(rng.uniform(-1, 1, (M, K)) * np.array([[1e-37], [2e-38], [1e-30]])[np.arange(M) % 3])
    w = rng.integers(-127, 128, (N, K)).astype(np.int8)
    sw = np.full(N, 2.0 ** 40, dtype=np.float32)
    C = torch.empty((M, N), device="cuda")
    n = Q.qgemm_int8_workspace_size(Q.QW_A_BF16, M, N, K)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    Q.qgemm_int8(Q.QW_A_BF16, xt.cuda(), K, None, dev(w), dev(sw), None, Q.QW_T_F32, C, N, M, N, K, ws, n)
    amax = np.abs(x).max(axis=1).astype(np.float64)
    want = x.astype(np.float64) @ w.T.astype(np.float64) * sw
    tol = (amax / 127)[:, None] * 0.51 * np.abs(w).sum(axis=1)[None, :] * sw + 2.0 ** -20 * np.abs(want)
    assert (np.abs(host(C) - want) <= tol).all()
