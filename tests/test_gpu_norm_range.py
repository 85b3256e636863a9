"""The norm's INT8 rows over the range of y: a code times its row's scale is y to half a scale, as qw_quantize_int8's
codes are, down to rows without a normal number."""
import pytest
import torch

from qwtest import qw
from test_gpu_norm import bound, call, reference

pytestmark = pytest.mark.gpu

MIN_NORMAL = 2.0 ** -126


@pytest.mark.parametrize("K", [16, 1040, 4112, 20000])
@pytest.mark.parametrize("rows", [1, 700])
@pytest.mark.parametrize("power", [-90, -117, -118, -119, -120, -121, -122, -123, -124, -125, -126, -129])
def test_codes_times_scale_are_the_values(K, rows, power):
    """Rows whose largest |y| is about 2^power, by their weights.  h is within 4, 1 / rms below 1: h w below 2^-126
    is off by up to 2^-150, and y, after a rounding of its own, by no more than 2^-148.  Bound: half a step,
    the quotient's and the product's roundings (127 * 4 * 2^-24 of one), e |y|, the scale's rounding (2^-24 or
    2^-150) 127 times."""
    Q = qw()
    g = torch.Generator(device="cuda").manual_seed(K + rows)
    x = (torch.rand((rows, K), generator=g, device="cuda") * 2 - 1) * 4
    w = (torch.rand(K, generator=g, device="cuda") * 0.5 + 0.5).double() * 2.0 ** power
    w = w.to(torch.bfloat16)
    _, y = reference(x, None, w)
    got = call(x, None, w, "int8", y=rows > 1)
    codes, sf = got["codes"].double(), got["sf"].double()[:, None]
    top = y.abs().amax(dim=1, keepdim=True)
    e = bound(K)
    off = (codes * sf - y).abs()
    tol = top / 127 * (0.5 + 127 * 4 * 2.0 ** -24) + 2 * e * y.abs() + 127 * 2.0 ** -150 + 127 * 2.0 ** -24 * top / 127 \
        + 2.0 ** -148
    some = (top >= MIN_NORMAL * (1 + 2.0 ** -16)).expand_as(y)  # (y is off by 2^-148 at most)
    assert bool((off <= tol)[some].all()), float((off / tol)[some].max())
    normal = some[:, 0]
    assert bool((got["codes"][normal].abs().amax(dim=1) == 127).all())  # the codes' whole range is used
    none = (top < MIN_NORMAL * (1 - 2.0 ** -16))[:, 0]
    assert bool((got["codes"][none] == 0).all())  # rows without a normal number count as zeros
    assert int(normal.sum()) + int(none.sum()) > 0 or rows == 1
    if rows > 1:  # BF16 rows beside the codes: half a step of the value, or of BF16's smallest numbers
        assert bool(((got["y"].double() - y).abs() <= (2.0 ** -8 * (1 + e) + e) * y.abs() + 2.0 ** -134 + 2.0 ** -148).all())


def test_the_same_codes_as_the_quantisers():
    """Rows of ordinary size and of every small one: the norm's codes are qw_quantize_int8's of y, where y is exact in
    BF16 (h = 2^j and eps chosen so that 1 / rms is a power of two)."""
    Q = qw()
    K = 1040
    x = torch.ones((64, K), device="cuda")  # mean h^2 = 1, eps = 3: rms is 2
    w = (torch.randint(-127, 128, (K,), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")).double()
    w[0] = 127
    for power in (0, -100, -115, -118, -119, -120, -124, -130):
        wp = (w * 2.0 ** power).to(torch.bfloat16)
        got = call(x, None, wp, "int8", y=True, eps=3.0)
        assert torch.equal(got["y"].double(), (wp.double() / 2).expand(64, K))
        q = torch.empty((64, K), dtype=torch.int8, device="cuda")
        s = torch.empty(64, device="cuda")
        Q.qw_quantize_int8(got["y"].contiguous(), K, 64, K, q, s, None)
        assert torch.equal(got["codes"], q) and torch.equal(got["sf"], s), power
