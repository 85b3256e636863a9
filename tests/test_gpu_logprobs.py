"""qw_logprobs on the GPU against a 64-bit restatement: ids, ranks and ties exactly, the log
probabilities and entropies within a derived bound.

Bound.  exp's relative error is a few ulp plus that of its argument (2^-23 |d| for d = x - m,
and e^d |d| <= 0.37); s is a sum of V positive terms in chains of at most V/128 + 64, so its
relative error is at most e_s = 2^-24 (V/128 + 96), and so is that of t = sum e^d d against
sum e^d |d| (plus 2^-23 for d).  lp = (x - m) - log s adds the rounding of two FP32 values."""
import numpy as np
import pytest
import torch

from qwtest import qw

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def kind(dtype):
    Q = qw()
    return {"bf16": Q.QW_T_BF16, "f16": Q.QW_T_F16, "f32": Q.QW_T_F32}[dtype]


def reference(x, tokens, k):
    """x float64 [T][V] (the exact input values)."""
    T, V = x.shape
    lp, rank, ent = np.zeros(T), np.zeros(T, dtype=np.int64), np.zeros(T)
    ids, top = np.zeros((T, k), dtype=np.int64), np.zeros((T, k))
    tol_lp, tol_ent = np.zeros(T), np.zeros(T)
    e_s = 2.0 ** -24 * (V / 128 + 96)
    for t in range(T):
        r = x[t]
        order = np.lexsort((np.arange(V), -(r + 0.0)))  # value descending, id ascending
        ids[t] = order[:k]
        rank[t] = 1 + np.flatnonzero(order == tokens[t])[0]
        m = r.max()
        if m == -np.inf:
            lp[t], ent[t], top[t] = -np.inf, 0.0, -np.inf
            continue
        d = r - m
        e = np.exp(d)
        s = e.sum()
        ed = np.where(e > 0, e * np.where(np.isfinite(d), d, 0.0), 0.0)
        logp = d - np.log(s)
        lp[t], top[t] = logp[tokens[t]], logp[ids[t]]
        ent[t] = np.log(s) - ed.sum() / s
        tol_lp[t] = e_s + 2.0 ** -23 * np.log(s)
        tol_ent[t] = e_s * (1 + 3 * np.abs(ed).sum() / s) + 2.0 ** -22 * (np.log(s) + np.abs(ed).sum() / s)
    return lp, rank, ent, ids, top, tol_lp, tol_ent


def call(logits, T, V, ld, dtype, tokens, k, want_err=0, stream=None):
    Q = qw()
    lp = torch.full((max(T, 1),), 7.0, device="cuda")
    rank = torch.full((max(T, 1),), -7, dtype=torch.int32, device="cuda")
    ent = torch.full((max(T, 1),), 7.0, device="cuda")
    ids = torch.full((max(T, 1), k), -7, dtype=torch.int32, device="cuda")
    top = torch.full((max(T, 1), k), 7.0, device="cuda")
    tok = torch.from_numpy(np.asarray(tokens, dtype=np.int32)).cuda()
    err = Q.new_error_flag()
    torch.cuda.synchronize()
    Q.qw_logprobs(kind(dtype), logits, ld, T, V, tok, k, lp, rank, ent, ids, top, err, stream)
    assert Q.qw_read_error(err, stream) == want_err
    return [t.cpu().numpy() for t in (lp, rank, ent, ids, top)]


def run_and_check(x, dtype, k, pad=0, shift=0, tokens=None, seed=0):
    """x float32 [T][V]; stored in dtype at pitch V + pad, `shift` elements into a buffer."""
    T, V = x.shape
    rng = np.random.default_rng(seed)
    buf = torch.full((T * (V + pad) + shift,), float("nan"), dtype=TYPES[dtype], device="cuda")
    view = buf[shift:].view(T, V + pad)
    view[:, :V] = torch.from_numpy(x).to(TYPES[dtype]).cuda()
    xs = view[:, :V].double().cpu().numpy()
    tokens = rng.integers(0, V, T) if tokens is None else np.asarray(tokens)
    got = call(view, T, V, V + pad, dtype, tokens, k)
    lp, rank, ent, ids, top, tol_lp, tol_ent = reference(xs, tokens, k)
    assert np.array_equal(got[3], ids)
    assert np.array_equal(got[1], rank)

    def near(a, b, tol):
        fine = np.isfinite(b)
        assert np.array_equal(a[~fine], b[~fine])
        t = np.broadcast_to(tol, b.shape)[fine] + 2.0 ** -23 * np.abs(b[fine])
        assert (np.abs(a[fine] - b[fine]) <= t).all(), (a[fine], b[fine], t)
    near(got[0], lp, tol_lp)
    near(got[2], ent, tol_ent)
    near(got[4], top, tol_lp[:, None])
    return got


def normal(T, V, seed, scale=2.5):
    return (np.random.default_rng(seed).normal(0, scale, (T, V))).astype(np.float32)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,V,k", [(1, 1, 1), (1, 2, 2), (3, 7, 5), (2, 31, 31), (5, 33, 32), (1, 1000, 20),
                                   (4, 4095, 8), (3, 4097, 32), (1, 32003, 5), (2, 50021, 20),
                                   (1, 131072, 32), (1, 200001, 1), (70, 5003, 3), (700, 1025, 4),
                                   (9, 20000, 0)])
def test_random_rows(T, V, k, dtype):
    run_and_check(normal(T, V, T + V + k), dtype, k, pad=(T + V) % 3, shift=V % 5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [40, 6000, 70001])
def test_ties_and_orders(V, dtype):
    """All equal; few distinct values; ascending and descending rows (every element of the one
    beats all before it); -0 against 0; the largest at either end."""
    rng = np.random.default_rng(V)
    rows = [np.full(V, 1.25), rng.integers(-2, 3, V), np.arange(V) / V * 8 - 4, -np.arange(V) / V * 8,
            np.where(rng.random(V) < 0.5, -0.0, 0.0), np.zeros(V), np.zeros(V), rng.integers(0, 2, V) * 1e-3]
    x = np.array(rows, dtype=np.float32)
    x[5, 0] = 30.0
    x[6, -1] = 30.0
    for tok in (0, V - 1, V // 2):
        run_and_check(x, dtype, 20, tokens=[tok] * len(rows))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_masks(dtype):
    """-inf and the type's lowest value as masks; one id left; nothing left; fewer ids left
    than alternatives asked for."""
    V = 9001
    low = float(torch.finfo(TYPES[dtype]).min)
    rng = np.random.default_rng(3)
    x = normal(8, V, 5)
    x[0, rng.random(V) < 0.95] = -np.inf
    x[1] = -np.inf
    x[1, 4321] = -3.0
    x[2] = -np.inf
    x[3, rng.random(V) < 0.95] = low
    x[4] = low
    x[5] = low
    x[5, 17] = 60.0
    x[6] = -np.inf
    x[6, :10] = np.arange(10)
    x[7, ::2] = -np.inf
    for tok in (17, 4321, 0):
        run_and_check(x, dtype, 20, tokens=[tok] * 8, pad=3)


@pytest.mark.parametrize("T,V", [(1, 131072), (3, 5000), (300, 2000)])
def test_large_and_peaked(T, V):
    """Logits of +-1e4 and rows that are nearly certain (entropy near 0)."""
    x = normal(T, V, 1, scale=1.0)
    x[0] *= 3e3
    x[T // 2, 5] = 40.0
    run_and_check(x, "f32", 8)


def test_nan_and_inf_are_flagged():
    Q = qw()
    for T, V in ((3, 300), (3, 70000)):
        for what in (np.nan, np.inf):
            x = torch.from_numpy(normal(T, V, 2)).cuda()
            x[1, V - 3] = what
            lp, rank, ent, ids, top = call(x, T, V, V, "f32", [0, 1, 2], 4, want_err=Q.QW_ERR_VALUE)
            for a in (lp, ent, top):
                assert np.isnan(a[1]).all() and np.isfinite(a[[0, 2]]).all()
            assert ((ids >= 0) & (ids < V)).all()


def test_token_out_of_range():
    Q = qw()
    x = torch.from_numpy(normal(4, 500, 2)).cuda()
    lp, rank, ent, ids, top = call(x, 4, 500, 500, "f32", [0, -1, 500, 499], 2,
                                   want_err=Q.QW_ERR_INVALID_ARG)
    assert np.isnan(lp[[1, 2]]).all() and (rank[[1, 2]] == 0).all()
    assert np.isfinite(lp[[0, 3]]).all() and np.isfinite(ent).all() and np.isfinite(top).all()


def test_outputs_may_be_left_out():
    Q = qw()
    x = normal(3, 20000, 2)
    xt = torch.from_numpy(x).cuda()
    lp0, rank0, ent0, ids0, top0 = call(xt, 3, 20000, 20000, "f32", [1, 2, 3], 6)
    tok = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    lp = torch.empty(3, device="cuda")
    Q.qw_logprobs(Q.QW_T_F32, xt, 20000, 3, 20000, tok, 0, lp, None, None, None, None)
    assert np.array_equal(lp.cpu().numpy(), lp0)
    ent = torch.empty(3, device="cuda")
    Q.qw_logprobs(Q.QW_T_F32, xt, 20000, 3, 20000, None, 0, None, None, ent, None, None)
    assert np.array_equal(ent.cpu().numpy(), ent0)
    ids, top = torch.empty((3, 6), dtype=torch.int32, device="cuda"), torch.empty((3, 6), device="cuda")
    Q.qw_logprobs(Q.QW_T_F32, xt, 20000, 3, 20000, None, 6, None, None, None, ids, top)
    assert np.array_equal(ids.cpu().numpy(), ids0) and np.array_equal(top.cpu().numpy(), top0)


def test_pitch_past_two_to_the_31_elements():
    Q = qw()
    V, ld = 3001, 2**30 + 8
    buf = torch.empty(2 * ld + V, dtype=torch.bfloat16, device="cuda")
    x = torch.from_numpy(normal(3, V, 4)).to(torch.bfloat16)
    for r in range(3):
        buf[r * ld:r * ld + V] = x[r].cuda()
    tokens = [5, 3000, 77]
    lp, rank, ent, ids, top = call(buf, 3, V, ld, "bf16", tokens, 5)
    rlp, rrank, rent, rids, rtop, tol, _ = reference(x.double().numpy(), np.array(tokens), 5)
    assert np.array_equal(ids, rids) and np.array_equal(rank, rrank)
    assert (np.abs(lp - rlp) <= tol + 2.0 ** -23 * np.abs(rlp)).all()


def test_another_stream_and_repeatable():
    x = torch.from_numpy(normal(5, 40001, 6)).cuda()
    a = call(x, 5, 40001, 40001, "f32", [1] * 5, 20)
    st = torch.cuda.Stream()
    for s in (st, None, None):
        b = call(x, 5, 40001, 40001, "f32", [1] * 5, 20, stream=s)
        for u, v in zip(a, b):
            assert np.array_equal(u, v)
