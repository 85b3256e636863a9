"""qw_logprobs over more rows than fit the GPU at once, where smaller CTAs take a row each: the
checks, bounds and reference of test_gpu_logprobs.  (A thread of the smallest CTA sums at most V / 64
terms in two chains, which is the bound's V / 128.)"""
import numpy as np
import pytest
import torch

from test_gpu_logprobs import TYPES, normal, run_and_check

pytestmark = pytest.mark.gpu


def many():
    """Rows that are more than the CTAs of 256 threads that fit at once."""
    return 4 * torch.cuda.get_device_properties(0).multi_processor_count + 3


# vocabularies around the widths where the CTA's size changes (256 and 1024 vectors of 16 bytes), one
# logit to several blocks
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V,k", [(1, 1), (5, 5), (33, 32), (250, 20), (968, 20), (1023, 32), (1100, 5),
                                 (2049, 32), (2060, 0), (4097, 20), (8190, 32), (8300, 3)])
def test_many_rows(V, k, dtype):
    run_and_check(normal(many(), V, V + k), dtype, k, pad=V % 3, shift=V % 5)


def test_many_long_rows():
    """Past twice as many rows, vocabularies of more blocks than are noted one by one."""
    T, V = 2 * many() + 1, 9001
    run_and_check(normal(T, V, 1), "f32", 20, pad=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [40, 900, 3001])
def test_many_rows_of_ties_and_masks(V, dtype):
    T = many()
    rng = np.random.default_rng(V)
    x = normal(T, V, V)
    low = float(torch.finfo(TYPES[dtype]).min)
    rows = np.arange(T) % 9
    x[rows == 1] = 1.25                                             # all equal
    x[rows == 2] = rng.integers(-2, 3, (int((rows == 2).sum()), V))  # few values
    x[rows == 3] = (np.arange(V) / V * 8 - 4).astype(np.float32)     # ascending
    x[(rows == 4)[:, None] & (rng.random((T, V)) < 0.95)] = -np.inf  # few left
    x[rows == 5] = -np.inf                                          # nothing left
    x[rows == 6] = low
    x[rows == 7] = low
    x[rows == 7, V // 2] = 60.0
    x[rows == 8] = -np.inf
    x[rows == 8, V - 1] = 3.0                                        # one id left
    run_and_check(x, dtype, 20, pad=3, seed=V)
