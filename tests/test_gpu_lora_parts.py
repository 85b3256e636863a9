"""How qgemm_lora holds t = s A x between its two products: as BF16 numbers that add up to it, three of them for
FP32 results (all 24 bits) and two for BF16 ones (2^-17 t at most is lost).

Inputs whose sums lose nothing or next to nothing, so that what is left is the parts'.  Calls of a few tokens and of
many take different kernels, calls of few k and columns lone CTAs, others clusters."""
import pytest
import torch

from qwtest import qw

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
TOP = (2 - 2.0 ** -7) * 2.0 ** 127  # BF16's largest number
# (tokens, N, K): lone CTAs and clusters, the few-token kernel and (over 16 tokens of one adapter) tcgen05
SIZES = [(3, 64, 64), (9, 1032, 2048), (40, 64, 64), (200, 1032, 2048), (600, 264, 1040)]


def call(x, a, b, c, base=None, scale=None):
    """x [M][K], a [1][R][K], b [1][N][R], base [M][N] or None in 64 bits, exact in their types."""
    Q = qw()
    M, K = x.shape
    _, N, R = b.shape
    low = [t.to(torch.bfloat16) for t in (x, a, b)]
    assert all(torch.equal(t.double(), w) for t, w in zip(low, (x, a, b)))
    y = None if base is None else base.to(TYPES[c]).contiguous()
    s = None if scale is None else torch.tensor([scale], device="cuda")
    C = torch.full((M, N), float("nan"), dtype=TYPES[c], device="cuda")
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    err = Q.new_error_flag()
    Q.qgemm_lora(low[0], K, low[1], low[2], s, None, 1, R, ids, y, N, Q.QW_T_F32 if c == "f32" else Q.QW_T_BF16,
                 C, N, M, N, K, err)
    assert Q.qw_read_error(err) == 0
    return C


def sparse(M, N, K, R, seed):
    """Zeros for x, a and b, three k apart from one another, and the column that each r goes to alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, a, b = (torch.zeros(s, dtype=torch.float64, device="cuda") for s in ((M, K), (1, R, K), (1, N, R)))
    ks = torch.randperm(K, generator=g, device="cuda")[:3]
    r_of = torch.randint(0, R, (N,), generator=g, device="cuda")
    return x, a, b, ks, r_of, g


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("c", ["bf16", "f32"])
def test_t_above_the_largest_bf16_number(M, N, K, c):
    """t between BF16's and FP32's largest number, negative for some tokens: a finite result, t's parts exact."""
    R = 24
    x, a, b, ks, r_of, _ = sparse(M, N, K, R, M)
    sign = torch.where(torch.arange(M, device="cuda") % 3 == 1, -1.0, 1.0).double()
    x[:, ks[0]], x[:, ks[1]] = sign, sign
    a[0, :, ks[0]], a[0, :, ks[1]] = TOP, 2.0 ** 119  # t = (2 - 2^-8) 2^127: rounded to BF16, 2^128
    b[0, torch.arange(N, device="cuda"), r_of] = 2.0 ** -100
    want = (sign * (2 - 2.0 ** -8) * 2.0 ** 27)[:, None].expand(M, N)
    assert torch.equal(call(x, a, b, c), want.to(TYPES[c]))
    # what passes FP32 is infinite, and NaN stays NaN
    x[0, ks[0]], x[0, ks[1]] = 1, 64
    got = call(x, a, b, c)
    assert bool((got[0] != got[0]).logical_or(got[0].isinf()).all())
    assert torch.equal(got[1:], want[1:].to(TYPES[c]))
