"""qw_logprobs: NaN and +inf wherever a logit can be - beside the 16-byte vectors, in either half of a
packed pair, in the first and the last vector - for every type and CTA size; ties of FP16 rows."""
import numpy as np
import pytest
import torch

from qwtest import qw
from test_gpu_logprobs import TYPES, call, normal, run_and_check
from test_gpu_logprobs_rows import many

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("what", [np.nan, np.inf])
@pytest.mark.parametrize("T,V", [(40, 7), (40, 301), (40, 5003), (3, 70001), (None, 250), (None, 3001)])
def test_flagged_wherever_it_is(T, V, what, dtype):
    Q = qw()
    T = many() if T is None else T
    # rows start at every offset within a vector (pitch V + 1 is odd or V is)
    ld = V + 1 - V % 2 + 1 if V % 2 else V + 1
    x = torch.full((T, ld), 5.0, dtype=TYPES[dtype], device="cuda")
    x[:, :V] = torch.from_numpy(normal(T, V, V)).to(TYPES[dtype]).cuda()
    places = sorted({0, 1, 2, 3, 5, 7, 8, 9, V // 2, V // 2 + 1, V - 9, V - 2, V - 1} & set(range(V)))
    bad = np.zeros(T, dtype=bool)
    for i, at in enumerate(places):
        for r in range(2 * i, T, 2 * len(places) + 3):
            x[r, at] = what
            bad[r] = True
    k = min(V, 4)
    lp, rank, ent, ids, top = call(x, T, V, ld, dtype, [0] * T, k, want_err=Q.QW_ERR_VALUE)
    for a in (lp, ent, top):
        assert np.isnan(a[bad]).all()
        assert np.isfinite(a[~bad]).all()
    assert ((ids >= 0) & (ids < V)).all()


@pytest.mark.parametrize("what", [np.nan, np.inf])
def test_flagged_beside_masks(what):
    """The rest of the row, or of its vector, masked; the token itself is the bad one."""
    Q = qw()
    for dtype in ("bf16", "f16", "f32"):
        for V in (9, 5003, 70001):
            for at in (0, V // 2, V - 1):
                x = torch.full((2, V), -np.inf, dtype=TYPES[dtype], device="cuda")
                x[0, at] = what
                x[1, at] = 2.0
                lp, rank, ent, ids, top = call(x, 2, V, V, dtype, [at, at], 4, want_err=Q.QW_ERR_VALUE)
                assert np.isnan(lp[0]) and np.isnan(ent[0]) and np.isnan(top[0]).all()
                assert lp[1] == 0 and ent[1] == 0 and rank[1] == 1
                assert ids[1, 0] == at and top[1, 0] == 0 and (top[1, 1:] == -np.inf).all()


@pytest.mark.parametrize("V", [40, 6000, 70001])
def test_ties_f16(V):
    rng = np.random.default_rng(V)
    x = np.array([np.full(V, 1.25), rng.integers(-2, 3, V), np.arange(V) / V * 8 - 4,
                  -np.arange(V) / V * 8, np.where(rng.random(V) < 0.5, -0.0, 0.0),
                  rng.integers(0, 2, V) * 1e-3], dtype=np.float32)
    for tok in (0, V // 2, V - 1):
        run_and_check(x, "f16", 20, tokens=[tok] * len(x), shift=1)


def test_ties_f16_many_rows():
    for V in (250, 3001):
        x = np.random.default_rng(V).integers(-2, 3, (many(), V)).astype(np.float32)
        run_and_check(x, "f16", 20, pad=3, seed=V)
