"""qgemm_lora on the GPU against 64 bits.

Bound.  With t = A x and |t| = |A| |x|: products of BF16 values are exact in FP32, sums are taken 16
products at a time at the coarsest, in at most K / 16 + 16 steps (joins of slices included), each of
which may lose 2^-22 of what is summed (tensor cores may cut instead of round, more than once a step):
e_t = 2^-22 (K / 16 + 16).  t times the scale is rounded to FP32 and then held as a sum of BF16 numbers,
three (FP32 results, 2^-23) or two of them (BF16 results, 2^-17).  The second sum has at most
3 (R / 16 + 1) such steps.  All of it is relative to |B| |t|; then one rounding of the result."""
import numpy as np
import pytest
import torch

from qwtest import qw

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def pool(L, R, N, K, seed, junk=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    a = (torch.randn((L, R, K), generator=g, device="cuda") / K ** 0.5).to(torch.bfloat16)
    b = (torch.randn((L, N, R), generator=g, device="cuda") / R ** 0.5).to(torch.bfloat16)
    scales = torch.rand(L, generator=g, device="cuda") + 0.5
    ranks = torch.randint(1, R + 1, (L,), generator=g, device="cuda", dtype=torch.int32)
    ranks[0] = R
    if L > 2:
        ranks[2] = 0
    if junk:  # what lies beyond an adapter's rank is nobody's business
        for i, r in enumerate(ranks.tolist()):
            a[i, r:] = float("nan")
            b[i, :, r:] = float("nan")
    return a, b, scales, ranks


def reference(x, a, b, scales, ranks, ids, base):
    """(result in 64 bits, |base| + |B| |A| |x|, bound before the result's rounding) with e as above."""
    M, K = x.shape
    L, N, R = b.shape
    out = torch.zeros((M, N), dtype=torch.float64, device="cuda") if base is None else base.double()
    size = out.abs()
    tol = torch.zeros_like(out)
    e_t = 2.0 ** -22 * (K / 16 + 16)
    for i in range(L):
        rows = torch.nonzero(ids == i)[:, 0]
        r = R if ranks is None else int(ranks[i])
        if rows.numel() == 0 or r == 0:
            continue
        s = 1.0 if scales is None else float(scales[i].double())
        xa, ad, bd = x[rows].double(), a[i, :r].double(), b[i, :, :r].double()
        out[rows] += s * (xa @ ad.t()) @ bd.t()
        big = abs(s) * (xa.abs() @ ad.abs().t()) @ bd.abs().t()
        size[rows] += big
        tol[rows] = (e_t + 2.0 ** -22 * 3 * (R / 16 + 1) + 2.0 ** -22) * big
    return out, size, tol


def call(x, a, b, scales, ranks, ids, base, c, pad_x=0, pad_c=0, in_place=False, want_err=0,
         stream=None, shift=0):
    """base: values [M][N] or None; -> C [M][N]."""
    Q = qw()
    M, K = x.shape
    L, N, R = b.shape
    X = torch.full((M, K + pad_x), float("nan"), dtype=torch.bfloat16, device="cuda")
    X[:, :K] = x
    C = torch.full((M * (N + pad_c) + shift,), float("nan"), dtype=TYPES[c], device="cuda")[shift:]
    C = C.view(M, N + pad_c)
    source = base
    if in_place:
        C[:, :N] = base
        source = C
    kind = Q.QW_T_F32 if c == "f32" else Q.QW_T_BF16
    err = Q.new_error_flag()
    torch.cuda.synchronize()
    Q.qgemm_lora(X, K + pad_x, a, b, scales, ranks, L, R, ids, source, N + pad_c if in_place else N,
                 kind, C, N + pad_c, M, N, K, err, stream)
    assert Q.qw_read_error(err, stream) == want_err
    assert bool(torch.isnan(C[:, N:]).all())
    return C[:, :N]


def check(got, want, c, none=None, base=None):
    out, size, tol = want
    half = 2.0 ** -24 if c == "f32" else 2.0 ** -8
    split = 2.0 ** -23 if c == "f32" else 2.0 ** -17
    limit = tol + split * size + half * (out.abs() + tol) + 2.0 ** -133
    off = (got.double() - out).abs()
    assert bool((off <= limit).all()), float((off / limit).max())
    if none is not None and bool(none.any()):
        rows = got[none]
        assert torch.equal(rows, torch.zeros_like(rows) if base is None else base[none])


def problem(M, N, K, L, R, c, seed, runs=False, base=True, plain=False):
    a, b, scales, ranks = pool(L, R, N, K, seed, junk=not plain)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.randint(-1, L, (M,), generator=g, device="cuda", dtype=torch.int32)
    if runs:
        ids = ids.sort().values
    y = (3 * torch.randn((M, N), generator=g, device="cuda")).to(TYPES[c]) if base else None
    if plain:
        scales = ranks = None
    return x, a, b, scales, ranks, ids, y


def run_and_check(M, N, K, L, R, c, seed=0, runs=False, base=True, plain=False, **kw):
    x, a, b, scales, ranks, ids, y = problem(M, N, K, L, R, c, seed, runs, base, plain)
    got = call(x, a, b, scales, ranks, ids, y, c, **kw)
    none = ids == -1
    if ranks is not None:
        none = none | (ranks[ids.clamp(min=0).long()] == 0)
    check(got, reference(x, a, b, scales, ranks, ids, y), c, none, y)
    return got


SHAPES = [(1, 1, 8, 1, 8), (1, 4096, 4096, 3, 16), (2, 17, 72, 2, 8), (3, 1000, 1040, 5, 24),
          (16, 256, 512, 4, 64), (17, 129, 264, 3, 32), (33, 48, 8, 3, 40), (64, 2048, 1024, 32, 16),
          (100, 333, 2056, 7, 128), (129, 1001, 1040, 4, 72), (300, 640, 4096, 2, 256),
          (777, 1000, 520, 9, 24), (1500, 264, 128, 3, 64)]


@pytest.mark.parametrize("M,N,K,L,R", SHAPES)
@pytest.mark.parametrize("c", ["bf16", "f32"])
@pytest.mark.parametrize("runs", [False, True])
def test_shapes(M, N, K, L, R, c, runs):
    run_and_check(M, N, K, L, R, c, M + N, runs, in_place=runs)


# more adapters than tokens of a window, ranks past 128, windows of 512 tokens and their last few, few columns
# and many, K of one stage and of many
MORE = [(1100, 600, 640, 700, 16), (513, 264, 264, 2, 200), (40, 136, 64, 1, 256), (1023, 8, 136, 2, 40),
        (515, 1000, 1032, 1, 64), (2048, 520, 264, 40, 40), (130, 9000, 64, 1, 16), (700, 4096, 4096, 1, 64),
        (520, 130, 8, 5, 136), (257, 2000, 2048, 6, 8), (4096, 2048, 2048, 8, 64), (3000, 1001, 1032, 20, 128)]


@pytest.mark.parametrize("M,N,K,L,R", MORE)
@pytest.mark.parametrize("c", ["bf16", "f32"])
@pytest.mark.parametrize("runs", [False, True])
def test_many_tokens(M, N, K, L, R, c, runs):
    run_and_check(M, N, K, L, R, c, M + N, runs, in_place=not runs)


@pytest.mark.parametrize("c", ["bf16", "f32"])
@pytest.mark.parametrize("most", [1, 7, 8, 9, 31, 32, 33, 64, 65, 127, 128, 129])
def test_runs_of_every_length(c, most):
    """Adapters whose tokens stand together, from odd places on, and one whose tokens stand between."""
    M, N, K = 600, 392, 328
    x, a, b, scales, ranks, ids, y = problem(M, N, K, 5, 24, c, 20)
    ids[:] = -1
    at, i = 3, 0
    while at + most <= M:
        ids[at:at + most] = i % 4
        at, i = at + most + 1, i + 1
    ids[ids == -1] = 4
    ids[0] = -1
    for in_place in (False, True):
        got = call(x, a, b, scales, ranks, ids, y, c, in_place=in_place)
        none = (ids == -1) | (ranks[ids.clamp(min=0).long()] == 0)
        check(got, reference(x, a, b, scales, ranks, ids, y), c, none, y)


@pytest.mark.parametrize("M", [5, 70, 300, 1166])
@pytest.mark.parametrize("N,pad", [(7, 1), (132, 4), (131, 5), (66, 6), (1153, 7), (127, 1), (190, 2)])
@pytest.mark.parametrize("c", ["bf16", "f32"])
def test_rows_that_end_within_16_bytes(M, N, pad, c):
    """What lies behind them, up to the pitch, stays as it was."""
    for in_place in (False, True):
        run_and_check(M, N, 136, 2, 16, c, M + N, True, pad_c=pad, in_place=in_place)
    run_and_check(M, N, 136, 2, 16, c, M + N, True, pad_c=pad, base=False)


@pytest.mark.parametrize("M", [1, 5, 40, 200, 600])
@pytest.mark.parametrize("c", ["bf16", "f32"])
def test_strides_and_alignment(M, c):
    run_and_check(M, 203, 264, 3, 16, c, 1, pad_x=8, pad_c=5)
    run_and_check(M, 200, 264, 3, 16, c, 2, pad_x=24, pad_c=8, shift=1)
    run_and_check(M, 200, 264, 3, 16, c, 3, pad_c=8, in_place=True)
    run_and_check(M, 201, 264, 3, 16, c, 4, pad_c=1, in_place=True, shift=3)


@pytest.mark.parametrize("M", [1, 20, 150, 520])
@pytest.mark.parametrize("c", ["bf16", "f32"])
def test_without_base_scales_or_ranks(M, c):
    run_and_check(M, 320, 512, 3, 32, c, 5, base=False)
    run_and_check(M, 320, 512, 3, 32, c, 6, plain=True)
    run_and_check(M, 320, 512, 3, 32, c, 7, base=False, plain=True, runs=True)


@pytest.mark.parametrize("M", [1, 16, 130, 700])
@pytest.mark.parametrize("c", ["bf16", "f32"])
def test_tokens_without_an_adapter(M, c):
    """Their rows are the base's, bit for bit: negative zeros, infinities and NaN among them."""
    x, a, b, scales, ranks, ids, y = problem(M, 72, 128, 2, 16, c, 8)
    ids[:] = -1
    y[:, ::7] = -0.0
    y[:, 1::7] = float("inf")
    y[:, 2::7] = float("nan")
    for in_place in (False, True):
        got = call(x, a, b, scales, ranks, ids, y, c, in_place=in_place)
        bits = torch.int32 if c == "f32" else torch.int16
        assert torch.equal(got.contiguous().view(bits), y.view(bits))


@pytest.mark.parametrize("M", [3, 64, 257])
def test_bad_ids_and_ranks(M):
    """Said so, and the tokens are taken as ones without adapter; the others are right."""
    Q = qw()
    x, a, b, scales, ranks, ids, y = problem(M, 136, 128, 4, 16, "bf16", 9)
    ids[M // 2] = 4
    ids[0] = -2
    got = call(x, a, b, scales, ranks, ids, y, "bf16", want_err=Q.QW_ERR_INVALID_ARG)
    ok = ids.clone()
    ok[M // 2] = ok[0] = -1
    check(got, reference(x, a, b, scales, ranks, ok, y), "bf16", ok == -1, y)
    ids = ok
    ids[1] = 1
    bad = ranks.clone()
    bad[1] = 17
    got = call(x, a, b, scales, bad, ids, y, "bf16", want_err=Q.QW_ERR_INVALID_ARG)
    bad[1] = 0
    check(got, reference(x, a, b, scales, bad, ids, y), "bf16", (ids == -1) | (ids == 1), y)


@pytest.mark.parametrize("M", [8, 200])
def test_a_token_that_is_not_finite_stays_alone(M):
    x, a, b, scales, ranks, ids, y = problem(M, 136, 512, 3, 16, "bf16", 10)
    ids[:] = 1
    want = call(x, a, b, scales, ranks, ids, y, "bf16")
    x[2, 5] = float("inf")
    x[5, 100] = float("nan")
    got = call(x, a, b, scales, ranks, ids, y, "bf16")
    rest = [i for i in range(M) if i not in (2, 5)]
    assert torch.equal(got[rest], want[rest])
    assert bool(torch.isnan(got[5]).all()) and not bool(torch.isfinite(got[2]).any())


@pytest.mark.parametrize("M", [1, 7, 64, 333, 1000])
def test_repeats_give_the_same_bits(M):
    x, a, b, scales, ranks, ids, y = problem(M, 1000, 2048, 4, 64, "f32", 11)
    want = call(x, a, b, scales, ranks, ids, y, "f32")
    for _ in range(3):
        assert torch.equal(call(x, a, b, scales, ranks, ids, y, "f32"), want)


def test_pools_past_32_bits():
    """Adapters whose weights lie past 2^31 elements."""
    Q = qw()
    L, R, N, K, M = 5, 128, 4096, 1 << 22, 3
    a = torch.empty((L, R, K), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(12)
    for i in range(L):
        for r in range(0, R, 32):
            a[i, r:r + 32] = torch.randn((32, K), generator=g, device="cuda") / 2048
    b = (torch.randn((L, N, R), generator=g, device="cuda") / 16).to(torch.bfloat16)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.tensor([4, 0, 4], dtype=torch.int32, device="cuda")
    ranks = torch.full((L,), 8, dtype=torch.int32, device="cuda")  # (few rows: the reference is in 64 bits)
    got = call(x, a, b, None, ranks, ids, None, "f32")
    check(got, reference(x, a, b, None, ranks, ids, None), "f32")
    assert Q.QW_OK == 0 and np.isfinite(got.sum().item())


def test_rows_past_32_bits():
    """C rows whose offsets pass 2^31 elements."""
    Q = qw()
    M, N, K, ld = 5, 512, 256, 1 << 29
    x, a, b, scales, ranks, ids, _ = problem(M, N, K, 2, 16, "bf16", 13)
    ids[:] = torch.tensor([0, 1, -1, 0, 1], device="cuda")
    buf = torch.empty(4 * ld + N, dtype=torch.bfloat16, device="cuda")
    C = buf.as_strided((M, N), (ld, 1))
    y = torch.randn((M, N), device="cuda").to(torch.bfloat16)
    C.copy_(y)
    Q.qgemm_lora(x, K, a, b, scales, ranks, 2, 16, ids, C, ld, Q.QW_T_BF16, C, ld, M, N, K)
    check(C, reference(x, a, b, scales, ranks, ids, y), "bf16", ids == -1, y)
