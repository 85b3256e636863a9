"""The adapters where offsets pass 32 bits in calls of more than a few tokens of an adapter, FP32 results of high ranks
in runs of one adapter, and the norm in place with more rows than run at once."""
import pytest
import torch

from qwtest import qw
from test_gpu_lora import check as check_lora, pool, reference as adapters
from test_gpu_norm import EPS, call as call_norm, problem as norm_problem

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def far(values, ld, dtype):
    """values as rows of pitch ld in a buffer that ends with them, and what lies behind each row (8 numbers)."""
    M, N = values.shape
    buf = torch.empty((M - 1) * ld + N + 8, dtype=dtype, device="cuda")
    rows = buf.as_strided((M, N), (ld, 1))
    rows.copy_(values)
    behind = buf.as_strided((M, 8), (ld, 1), N)
    behind.fill_(7.0)
    return rows, behind


def ids_of(kind, M):
    """One adapter's tokens: all that stand together, every other one, or eight together out of nine."""
    i = torch.arange(M, device="cuda")
    keep = {"all": i >= 0, "every other": i % 2 == 0, "eights": i % 9 != 8}[kind]
    return torch.where(keep, 0, -1).to(torch.int32)


# 24 tokens of one loaded adapter go to the tensor cores: in boxes, in pieces, and rows that 16 bytes do not fit
@pytest.mark.parametrize("c,odd", [("bf16", 0), ("bf16", 1), ("f32", 0), ("f32", 1)])
@pytest.mark.parametrize("ids", ["all", "every other", "eights"])
@pytest.mark.parametrize("in_place", [False, True])
def test_rows_past_32_bits_on_tensor_cores(c, odd, ids, in_place):
    Q = qw()
    M, N, K, R, ld = 24, 264, 328, 16, (1 << 27) + 8 + odd
    a, b, scales, _ = pool(1, R, N, K, 31)
    g = torch.Generator(device="cuda").manual_seed(32)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    y = torch.randn((M, N), generator=g, device="cuda").to(TYPES[c])
    which = ids_of(ids, M)
    X, _ = far(x, 1 << 27, torch.bfloat16)
    C, behind = far(y if in_place else torch.zeros_like(y), ld, TYPES[c])
    base = C if in_place else far(y, ld + 8, TYPES[c])[0]
    err = Q.new_error_flag()
    Q.qgemm_lora(X, 1 << 27, a, b, scales, None, 1, R, which, base, ld if in_place else ld + 8,
                 Q.QW_T_F32 if c == "f32" else Q.QW_T_BF16, C, ld, M, N, K, err)
    assert Q.qw_read_error(err) == 0
    check_lora(C, adapters(x, a, b, scales, None, which, y), c, which == -1, y)
    assert bool((behind == 7.0).all())


def test_tall_items_past_32_bits():
    """128 tokens an item, so that rows go by whole boxes: the last rows lie past 2^31 elements."""
    Q = qw()
    M, N, K, R, ld = 300, 520, 136, 16, 1 << 23
    a, b, scales, _ = pool(1, R, N, K, 33)
    g = torch.Generator(device="cuda").manual_seed(34)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    y = torch.randn((M, N), generator=g, device="cuda").to(torch.bfloat16)
    for kind in ("all", "eights"):
        which = ids_of(kind, M)
        C, behind = far(y, ld, torch.bfloat16)
        Q.qgemm_lora(x, K, a, b, scales, None, 1, R, which, C, ld, Q.QW_T_BF16, C, ld, M, N, K)
        check_lora(C, adapters(x, a, b, scales, None, which, y), "bf16", which == -1, y)
        assert bool((behind == 7.0).all())


@pytest.mark.parametrize("L,R,N,K", [(2, 128, 72, (1 << 23) + 64), (2, 256, (1 << 22) + 8, 64)])
def test_pools_past_32_bits_on_tensor_cores(L, R, N, K):
    """The second adapter's weights, of which few ranks are used, end past 2^31 elements.  Weights and tokens of -1, 0
    and 1, tokens of 64 k at the beginning and 64 at the end: all sums are exact."""
    Q = qw()
    M, used = 40, 8
    g = torch.Generator(device="cuda").manual_seed(35)

    def draw(*shape):
        return torch.randint(-1, 2, shape, generator=g, device="cuda").to(torch.bfloat16)
    a = torch.zeros((L, R, K), dtype=torch.bfloat16, device="cuda")
    b = torch.zeros((L, N, R), dtype=torch.bfloat16, device="cuda")
    a[:, :used] = draw(L, used, K)
    b[:, :, :used] = draw(L, N, used)
    assert max(a.numel(), b.numel()) > 1 << 31
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    x[:, :64] = draw(M, 64)
    x[:, K - 64:] = draw(M, 64)
    ids = torch.randint(0, L, (M,), generator=g, device="cuda", dtype=torch.int32)
    ranks = torch.full((L,), used, dtype=torch.int32, device="cuda")
    C = torch.empty((M, N), device="cuda")
    err = Q.new_error_flag()
    Q.qgemm_lora(x, K, a, b, None, ranks, L, R, ids, None, 0, Q.QW_T_F32, C, N, M, N, K, err)
    assert Q.qw_read_error(err) == 0
    for i in range(L):
        mine = ids == i
        t = sum(x[mine][:, k].double() @ a[i, :used, k].double().t() for k in (slice(0, 64), slice(K - 64, K))) \
            if K > 64 else x[mine].double() @ a[i, :used].double().t()
        assert torch.equal(C[mine].double(), t @ b[i, :, :used].double().t())


def test_pools_whose_rows_pass_32_bits():
    """L * N above 2^31: the few-token kernel takes the call, whatever the number of tokens."""
    Q = qw()
    L, R, N, K, M = 2100, 8, 1 << 20, 64, 530
    g = torch.Generator(device="cuda").manual_seed(36)
    a = torch.randn((L, R, K), generator=g, device="cuda").to(torch.bfloat16)
    b = torch.zeros((L, N, R), dtype=torch.bfloat16, device="cuda")
    some = [0, 1050, 2099]
    for i in some:
        b[i] = torch.randn((N, R), generator=g, device="cuda")
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.tensor(some, dtype=torch.int32, device="cuda")[torch.randint(0, 3, (M,), generator=g, device="cuda")]
    C = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    err = Q.new_error_flag()
    Q.qgemm_lora(x, K, a, b, None, None, L, R, ids, None, 0, Q.QW_T_BF16, C, N, M, N, K, err)
    assert Q.qw_read_error(err) == 0
    for at in range(0, N, N // 8):  # (in columns' parts: the reference is in 64 bits)
        part = b[some, at:at + N // 8]
        where = torch.zeros(L, dtype=torch.int32, device="cuda")
        where[some] = torch.arange(3, dtype=torch.int32, device="cuda")
        check_lora(C[:, at:at + N // 8], adapters(x, a[some], part, None, None, where[ids.long()], None), "bf16")


@pytest.mark.parametrize("M,R", [(600, 136), (1100, 256), (40, 200)])
@pytest.mark.parametrize("together", [True, False])
def test_fp32_results_of_high_ranks(M, R, together):
    """One adapter's tokens over more than a window, in a run and every other."""
    Q = qw()
    N, K = 520, 1032
    a, b, scales, _ = pool(2, R, N, K, 37, junk=False)
    g = torch.Generator(device="cuda").manual_seed(38)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    y = torch.randn((M, N), generator=g, device="cuda")
    ids = torch.ones(M, dtype=torch.int32, device="cuda")
    if not together:
        ids[::2] = -1
    C = torch.empty_like(y)
    Q.qgemm_lora(x, K, a, b, scales, None, 2, R, ids, y, N, Q.QW_T_F32, C, N, M, N, K)
    check_lora(C, adapters(x, a, b, scales, None, ids, y), "f32", ids == -1, y)


@pytest.mark.parametrize("rows,K", [(5000, 160), (1300, 1056), (700, 4096), (400, 7200), (320, 16384)])
@pytest.mark.parametrize("q", ["mxfp8", "int8", None])
@pytest.mark.parametrize("over", ["r", "x"])
def test_norm_in_place_with_many_rows(rows, K, q, over):
    """R_out over R and Y over X, or R_out over X: the same bits as with buffers of their own, where a CTA has the
    next row on its way while it writes one."""
    Q = qw()
    xv, rv, w = norm_problem(rows, K, "bf16", "bf16", 39)
    want = call_norm(xv, rv, w, q)
    X, R = xv.clone(), rv.clone()
    out = R if over == "r" else X
    Y = X if over == "r" else torch.empty_like(X)
    fmt = {None: Q.QW_A_BF16, "int8": Q.QW_A_INT8_TOKEN, "mxfp8": Q.QW_A_MXFP8_G32}[q]
    codes = None if q is None else torch.empty_like(want["codes"])
    sf = None if q is None else torch.empty_like(want["sf"])
    Q.qw_rmsnorm(Q.QW_T_BF16, X, K, Q.QW_T_BF16, R, K, out, K, w, 0.0, EPS, rows, K, Y, K, fmt, codes, sf)
    assert torch.equal(out, want["h"]) and torch.equal(Y, want["y"])
    assert q is None or (torch.equal(codes, want["codes"]) and torch.equal(sf, want["sf"]))


@pytest.mark.parametrize("rows,K", [(5000, 160), (700, 4096), (400, 7200)])
def test_fp32_norm_in_place_with_many_rows(rows, K):
    Q = qw()
    xv, rv, w = norm_problem(rows, K, "f32", "f32", 40)
    want = call_norm(xv, rv, w, "mxfp8")
    for over in ("r", "x"):
        X, R = xv.clone(), rv.clone()
        out = R if over == "r" else X
        Y = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda")
        codes, sf = torch.empty_like(want["codes"]), torch.empty_like(want["sf"])
        Q.qw_rmsnorm(Q.QW_T_F32, X, K, Q.QW_T_F32, R, K, out, K, w, 0.0, EPS, rows, K, Y, K, Q.QW_A_MXFP8_G32, codes,
                     sf)
        assert torch.equal(out, want["h"]) and torch.equal(Y, want["y"])
        assert torch.equal(codes, want["codes"]) and torch.equal(sf, want["sf"])
