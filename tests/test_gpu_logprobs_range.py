"""qw_logprobs over the whole range of finite logits: masks of any large negative number, rows of huge
logits, rows at the types' limits.  The 64-bit reference and the bound are test_gpu_logprobs's; a log
probability below FP32's range is -inf."""
import numpy as np
import pytest
import torch

from test_gpu_logprobs import TYPES, call, normal, reference
from test_gpu_logprobs_rows import many

pytestmark = pytest.mark.gpu

SIZES = [1e6, 1.6e7, 1.7e7, 4e7, 1e8, 1e9, 2.5e9, 1e10, 1e20, 9e29, 2e30, 2.3e38, 2.5e38, None]


def size(v, dtype):
    return float(torch.finfo(TYPES[dtype]).max) if v is None else v


def check(x, dtype, k, tokens, pad=0):
    T, V = x.shape
    view = torch.zeros((T, V + pad), dtype=TYPES[dtype], device="cuda")
    view[:, :V] = torch.from_numpy(x).to(TYPES[dtype]).cuda()
    xs = view[:, :V].double().cpu().numpy()
    assert (np.isfinite(xs) | (xs == -np.inf)).all()
    got = call(view, T, V, V + pad, dtype, tokens, k)
    lp, rank, ent, ids, top, tol_lp, tol_ent = reference(xs, np.asarray(tokens), k)
    assert np.array_equal(got[3], ids) and np.array_equal(got[1], rank)

    def near(a, b, tol):
        b = np.where(b < -float(np.finfo(np.float32).max), -np.inf, b)
        fine = np.isfinite(b)
        assert np.array_equal(a[~fine], b[~fine]), (a[~fine], b[~fine])
        t = np.broadcast_to(tol, b.shape)[fine] + 2.0 ** -23 * np.abs(b[fine])
        bad = ~(np.abs(a[fine] - b[fine]) <= t)
        assert not bad.any(), (a[fine][bad][:5], b[fine][bad][:5], t[bad][:5])
    near(got[0], lp, tol_lp)
    near(got[2], ent, tol_ent)
    near(got[4], top, tol_lp[:, None])


def rows_of(v, V, dtype, seed):
    """Rows that a logit of size v makes hard."""
    rng = np.random.default_rng(seed)
    x = normal(9, V, seed)
    ulp = 2 * float(np.spacing(np.float32(v / 2))) if dtype == "f32" else v / 128
    x[0] = v                                            # all equal
    x[1] = -v                                           # a mask that leaves nothing
    x[2, V // 3] = v                                    # certain
    x[3, rng.random(V) < 0.9] = -v                      # a mask, the rest ordinary
    x[4] = -v
    x[4, V - 1] = 3.0                                   # one id left, the last
    x[5] = np.where(rng.random(V) < 0.5, v, -v)         # both signs
    x[6] = v - 3 * ulp * rng.integers(1, 4, V)          # neighbours of each other
    x[7] = -v + 3 * ulp * rng.integers(1, 4, V)
    x[8] = -v
    x[8, ::5] = -np.inf                                 # two masks, nothing left by either
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [40, 6000, 70001])
@pytest.mark.parametrize("v", SIZES)
def test_huge_logits(v, V, dtype):
    x = rows_of(size(v, dtype), V, dtype, V)
    for tok in (0, V // 3, V - 1):
        check(x, dtype, 5, [tok] * len(x), pad=V % 3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v", [4e7, 1e10, 1e20, 2.5e38])
@pytest.mark.parametrize("V", [40, 900, 3001])
def test_huge_logits_in_many_rows(v, V, dtype):
    """More rows than fit at once: smaller CTAs."""
    T = many()
    x = normal(T, V, V)
    hard = rows_of(v, V, dtype, V)
    for r in range(len(hard)):
        x[r::11] = hard[r]
    check(x, dtype, 5, np.random.default_rng(1).integers(0, V, T), pad=1)


@pytest.mark.parametrize("V", [40, 6000, 70001])
def test_f16_limits(V):
    for v in (59999.0, 60000.0, 60032.0, 65504.0):
        x = rows_of(v, V, "f16", V)
        x[6] = v - 96 * (np.arange(V) % 3)
        x[7] = -x[6]
        check(x, "f16", 5, [V // 3] * len(x), pad=1)


def test_growing_logits():
    """Every block of the row beats all before it, through every power of two up to the limit."""
    V = 40000
    x = np.empty((2, V), dtype=np.float32)
    x[0] = -np.exp2(127.0 - np.arange(V) / V * 250)
    x[1] = x[0] * -1.0
    x[1] = x[1][::-1]
    for dtype in ("f32", "bf16"):
        check(x, dtype, 8, [V - 1, 0])
