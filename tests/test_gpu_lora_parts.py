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


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("scale", [None, 0.25])
def test_three_parts_for_fp32_results(M, N, K, scale):
    """t = 1 + 2^-9 + 2^-18, one bit in each of three BF16 numbers (two would lose the last): sums of 19 bits, which
    neither cut nor round, so the results are exact."""
    R = 24
    x, a, b, ks, r_of, g = sparse(M, N, K, R, M + 1)
    x[:, ks] = 1
    a[0, :, ks[0]], a[0, :, ks[1]], a[0, :, ks[2]] = 1, 2.0 ** -9, 2.0 ** -18
    power = torch.exp2(torch.randint(-3, 4, (N,), generator=g, device="cuda").double())
    b[0, torch.arange(N, device="cuda"), r_of] = power
    base = -power.expand(M, N)
    t = (1 + 2.0 ** -9 + 2.0 ** -18) * (scale or 1.0)
    assert torch.equal(call(x, a, b, "f32", None, scale).double(), (t * power).expand(M, N))
    assert torch.equal(call(x, a, b, "f32", base, scale).double(), t * power + base)


@pytest.mark.parametrize("M,N,K", SIZES)
def test_all_bits_of_t_for_fp32_results(M, N, K):
    """t of 24 random bits out of three products (of 8 bits each: 1.xxxxxxx, and the next ones 2^-8 and 2^-16 of
    that).  A tensor core may cut each number of a sum to FP32's 24 bits of the largest, 2^-23: four numbers to make
    t, two in each of the two sums that join its parts.  FP32 additions round, 2^-24: two for a cluster's slices, and
    the result.  10 * 2^-23 in all; without t's third part it would be up to 2^-17."""
    R = 24
    x, a, b, ks, r_of, g = sparse(M, N, K, R, M + 2)
    bits = torch.randint(0, 128, (3, R), generator=g, device="cuda").double() / 128 + 1
    x[:, ks] = 1
    for i in range(3):
        a[0, :, ks[i]] = bits[i] * 2.0 ** (-8 * i)
    b[0, torch.arange(N, device="cuda"), r_of] = 1
    want = a[0][:, ks].sum(dim=1)[r_of].expand(M, N)
    off = (call(x, a, b, "f32").double() - want).abs() / want
    assert float(off.max()) <= 10 * 2.0 ** -23, float(off.max() * 2.0 ** 23)


@pytest.mark.parametrize("M,N,K", SIZES)
def test_two_parts_for_bf16_results(M, N, K):
    """16 bits of t are exact (1 + 2^-9 + 2^-16, of which base leaves the last two), and of 19 bits no more than
    2^-17 t is lost beside the result's rounding."""
    R = 24
    x, a, b, ks, r_of, g = sparse(M, N, K, R, M + 3)
    x[:, ks] = 1
    power = torch.exp2(torch.randint(-3, 4, (N,), generator=g, device="cuda").double())
    b[0, torch.arange(N, device="cuda"), r_of] = power
    base = -power.expand(M, N)
    a[0, :, ks[0]], a[0, :, ks[1]], a[0, :, ks[2]] = 1, 2.0 ** -9, 2.0 ** -16
    want = (2.0 ** -9 + 2.0 ** -16) * power.expand(M, N)
    assert torch.equal(call(x, a, b, "bf16", base).double(), want)
    a[0, :, ks[2]] = 2.0 ** -18
    want = (2.0 ** -9 + 2.0 ** -18) * power.expand(M, N)
    off = (call(x, a, b, "bf16", base).double() - want).abs()
    assert bool((off <= 2.0 ** -17 * (1 + 2.0 ** -8) * power + 2.0 ** -8 * want).all())


@pytest.mark.parametrize("M,N,K", [(5, 200, 4096), (64, 520, 2048), (200, 1032, 4096), (1100, 392, 1040)])
@pytest.mark.parametrize("c", ["bf16", "f32"])
def test_small_whole_numbers(M, N, K, c):
    """x and a of -1, 0 and 1, b of one -1 or 1 in eight: |t| <= 4096 takes 13 bits, which two parts hold, sums stay
    below 2^24, so FP32 results are exact and BF16 ones rounded once."""
    R = 64
    g = torch.Generator(device="cuda").manual_seed(M)

    def draw(*shape):
        return torch.randint(-1, 2, shape, generator=g, device="cuda").double()
    x, a = draw(M, K), draw(1, R, K)
    b = draw(1, N, R) * (torch.rand((1, N, R), generator=g, device="cuda") < 0.125)
    base = torch.randint(-100, 101, (M, N), generator=g, device="cuda").double()
    want = base + (x @ a[0].t()) @ b[0].t()
    assert float(want.abs().max()) < 2 ** 24
    assert torch.equal(call(x, a, b, c, base), want.float().to(TYPES[c]))
