"""The INT8 products over shapes that end inside every unit of their kernels (rows of a block, boxes and
chunks of k, token groups and tiles, slices of a split K), and over shapes drawn at random: the checks,
bounds and reference of test_gpu_int8."""
import numpy as np
import pytest

from qwtest import qw
from test_gpu_int8 import call, check, check_gated, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [16, 48, 128, 144, 512, 528, 1040, 1536, 4112])
@pytest.mark.parametrize("M,N", [(3, 2), (4, 34), (7, 66), (8, 200), (9, 30), (16, 1030)])
def test_few_tokens(M, N, K):
    p = problem(M, N, K, M * 131 + N + K, bias=K % 32 == 0, pad=16 * (M % 3))
    check(p, call(p, ldc_pad=M % 2))
    check_gated(p, call(p, gated=True))
    p = problem(M, N, K, M + K, a="int8", extreme=M % 2 == 0)
    check(p, call(p, afmt=qw().QW_A_INT8_TOKEN, c_type=qw().QW_T_F32), f32=True)


# K around the limits where a split leaves a CTA with one stage or would leave it with none
@pytest.mark.parametrize("M,N,K", [(20, 64, 1024), (20, 64, 1168), (33, 130, 2064), (40, 96, 4624),
                                   (40, 260, 6160), (64, 1000, 8192), (64, 1930, 4112), (64, 2050, 8208),
                                   (100, 300, 9232), (128, 258, 2192), (200, 1026, 4112)])
def test_split_sums(M, N, K):
    p = problem(M, N, K, M + N + K, bias=True)
    check(p, call(p))
    check_gated(p, call(p, gated=True))
    check(p, call(p, c_type=qw().QW_T_F32, ldc_pad=3), f32=True)


@pytest.mark.parametrize("seed", range(40))
def test_drawn_shapes(seed):
    rng = np.random.default_rng(1000 + seed)

    def size(lo, hi):
        return int(round(np.exp(rng.uniform(np.log(lo), np.log(hi)))))

    M, N, K = size(1, 1500), 2 * size(1, 2000), 16 * size(1, 500)
    a = "int8" if seed % 2 else "bf16"
    p = problem(M, N, K, seed, a=a, bias=seed % 3 == 0, pad=16 * (seed % 4))
    afmt = qw().QW_A_INT8_TOKEN if seed % 2 else None
    check(p, call(p, afmt=afmt, ldc_pad=seed % 5))
    check_gated(p, call(p, afmt=afmt, gated=True))


@pytest.mark.parametrize("M,N", [(1, 20), (2, 34), (9, 20), (40, 36), (130, 30)])
def test_longest_k(M, N):
    """K = 131056: the largest 32-bit sum (every code -128) among them."""
    K = 131056
    p = problem(M, N, K, M, a="int8", extreme=True)
    check(p, call(p, c_type=qw().QW_T_F32), f32=True)
    check_gated(p, call(p, gated=True))
    p = problem(M, N, K, M + 1, bias=True)
    check(p, call(p))
