"""qw_logprobs of rows that have logits beside their 16-byte vectors (short, odd or shifted rows) and are
far from 0, where the rounding of the running reference counts: the reference and the bound are
test_gpu_logprobs's."""
import numpy as np
import pytest

from test_gpu_logprobs import run_and_check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 3, 5, 7, 15, 22, 41, 301])
def test_logits_beside_the_vectors(V, dtype):
    rng = np.random.default_rng(V)
    rows = []
    for v in (777.0, 3e3, 2.5e4, 5.3e4) + (() if dtype == "f16" else (3.1e5, 1.1e6)):
        for sign in (1, -1):
            rows += [np.full(V, sign * v), sign * v + rng.normal(0, 2.5, V),
                     np.where(rng.random(V) < 0.5, sign * v, -sign * v)]
    x = np.array(rows, dtype=np.float32)
    for shift in range(4):
        run_and_check(x, dtype, min(V, 5), shift=shift, seed=shift)
