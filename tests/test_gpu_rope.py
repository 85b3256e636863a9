"""qw_rope on the GPU against 64 bits and more.

Bound.  An angle is held to 2^-32 turns (2^-29 rad) and its rest within an eighth of a turn rounded to
FP32 (2^-24 * pi / 4); sine and cosine are within an ulp (2^-24 here), times the scale 2^-24 more: less than
3.5 * 2^-24 s in all.  The two products and their sum add 1.5 * 2^-24 of the products' magnitudes.  So
a value is within 5 * 2^-24 s (|a| + |b|) before it is rounded to its type (half a step of it)."""
import numpy as np
import pytest
import torch

from qwtest import qw

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
LEAST = {"bf16": 2.0 ** -133, "f16": 2.0 ** -25, "f32": 2.0 ** -149}
TWO_PI = 2 * np.longdouble("3.14159265358979323846264338327950288419717")


def reference(x, heads, D, rot, layout, positions, freqs, scale):
    """x float64 [T][heads * D] -> (result, bound before rounding); angles in extended precision."""
    T = x.shape[0]
    angle = positions.astype(np.longdouble)[:, None] * freqs.astype(np.longdouble)
    angle = np.fmod(angle, TWO_PI)
    cos = np.cos(angle).astype(np.float64)[:, None] * scale
    sin = np.sin(angle).astype(np.float64)[:, None] * scale
    x = x.reshape(T, heads, D)
    out, tol = x.copy(), np.zeros_like(x)
    a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else \
        (slice(0, rot, 2), slice(1, rot, 2))
    out[:, :, a] = x[:, :, a] * cos - x[:, :, b] * sin
    out[:, :, b] = x[:, :, b] * cos + x[:, :, a] * sin
    tol[:, :, a] = tol[:, :, b] = 5 * 2.0 ** -24 * abs(scale) * (np.abs(x[:, :, a]) + np.abs(x[:, :, b]))
    return out.reshape(T, -1), tol.reshape(T, -1)


def run(T, heads, D, rot, layout, kind, pad=0, shift=0, positions=None, freqs=None, scale=1.0,
        in_place=False, seed=0, check=True):
    Q = qw()
    rng = np.random.default_rng(seed)
    n = heads * D
    if positions is None:
        positions = rng.integers(0, 1 << 17, T)
    if freqs is None:
        freqs = 10000.0 ** (-np.arange(rot // 2) * 2.0 / rot)
    buf = torch.full((T * (n + pad) + shift,), float("nan"), dtype=TYPES[kind], device="cuda")
    X = buf[shift:].view(T, n + pad)
    X[:, :n] = torch.from_numpy(rng.standard_normal((T, n))).to(TYPES[kind]).cuda()
    values = X[:, :n].clone()
    Y = X if in_place else torch.full((T * (n + pad) + shift,), float("nan"), dtype=TYPES[kind],
                                      device="cuda")[shift:].view(T, n + pad)
    pos = torch.from_numpy(np.asarray(positions, dtype=np.int32)).cuda()
    fr = torch.from_numpy(np.asarray(freqs, dtype=np.float64)).cuda()
    err = Q.new_error_flag()
    kinds = {"bf16": Q.QW_T_BF16, "f16": Q.QW_T_F16, "f32": Q.QW_T_F32}
    Q.qw_rope(kinds[kind], X, n + pad, Y, n + pad, T, heads, D, rot,
              Q.QW_ROPE_HALF if layout == "half" else Q.QW_ROPE_INTERLEAVED, pos, fr, scale, err)
    assert Q.qw_read_error(err) == 0
    assert bool(torch.isnan(Y[:, n:]).all())
    if not in_place:
        assert torch.equal(X[:, :n], values)
    if check:
        want, tol = reference(values.double().cpu().numpy(), heads, D, rot, layout,
                              np.asarray(positions, dtype=np.int64), np.asarray(freqs, dtype=np.float64),
                              float(np.float32(scale)))
        got = Y[:, :n].double().cpu().numpy()
        still = tol == 0
        assert np.array_equal(got[still], want[still])  # copied as they are
        assert (np.abs(got - want) <= tol + HALF_STEP[kind] * (np.abs(want) + tol) + LEAST[kind]).all()
    return Y[:, :n]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,heads,D,rot,pad,shift", [
    (1, 1, 2, 2, 0, 0), (1, 40, 128, 128, 0, 0), (5, 3, 64, 32, 8, 0), (7, 2, 80, 20, 0, 0),
    (3, 5, 72, 46, 5, 0), (4, 1, 128, 64, 0, 1), (67, 9, 96, 96, 16, 0), (130, 4, 256, 128, 0, 0),
    (2, 1, 1024, 1024, 0, 0), (1025, 2, 64, 64, 0, 0), (3, 700, 64, 64, 0, 0), (6, 2, 7, 6, 0, 0)])
def test_shapes(layout, kind, T, heads, D, rot, pad, shift):
    for in_place in (False, True):
        run(T, heads, D, rot, layout, kind, pad, shift, in_place=in_place, seed=T + D)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,heads,D,rot,pad", [
    (3001, 5, 256, 126, 0), (2500, 6, 72, 36, 0), (5003, 1, 64, 64, 0), (2049, 3, 80, 80, 3),
    (400, 33, 256, 256, 64), (1777, 4, 10, 10, 1)])
def test_many_tokens(layout, kind, T, heads, D, rot, pad):
    run(T, heads, D, rot, layout, kind, pad, seed=T, in_place=T % 2 == 0)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_and_negative_positions(layout):
    positions = [0, 1, -1, 1 << 20, (1 << 24) + 1, (1 << 31) - 1, -(1 << 31), -12345678, 1000003]
    run(len(positions), 3, 128, 128, layout, "f32", positions=positions, scale=1.25)


def test_frequencies_of_any_size():
    freqs = np.array([0.0, 1.0, -1.0, 6.283185307179586, 3.141592653589793, 1e-12, 1e-3, 123456.789,
                      -4e9, 2.0 ** -40, 0.5, 1.5707963267948966])
    positions = [0, 1, 2, 3, 1000, 123457]
    run(6, 2, 24, 24, "half", "f32", positions=positions, freqs=freqs)


def test_a_negative_position_turns_back():
    """Turned there and back: two roundings of FP32 values and twice the bound above."""
    Q = qw()
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((33, 512), generator=g, device="cuda")
    y = x.clone()
    pos = torch.arange(33, dtype=torch.int32, device="cuda") * 31337
    freqs = Q.qw_rope_frequencies(Q.QW_ROPE_YARN, 5e5, 128, 8.0, 8192.0)[0].cuda()
    for p in (pos, -pos):
        Q.qw_rope(Q.QW_T_F32, y, 512, y, 512, 33, 4, 128, 128, Q.QW_ROPE_HALF, p, freqs)
    size = x.view(33, 4, 2, 64).abs().sum(dim=2, keepdim=True).expand(33, 4, 2, 64).reshape(33, 512)
    assert bool(((x - y).abs() <= 2 * 8 * 2.0 ** -24 * 2 * size).all())


def test_frequencies_that_are_not_finite():
    Q = qw()
    x = torch.randn((3, 16), device="cuda")
    y = torch.zeros_like(x)
    freqs = torch.ones(8, dtype=torch.float64, device="cuda")
    freqs[3] = float("nan")
    freqs[5] = 1e10
    pos = torch.arange(3, dtype=torch.int32, device="cuda")
    err = Q.new_error_flag()
    Q.qw_rope(Q.QW_T_F32, x, 16, y, 16, 3, 1, 16, 16, Q.QW_ROPE_HALF, pos, freqs, 1.0, err)
    assert Q.qw_read_error(err) == Q.QW_ERR_VALUE
    gone = torch.isnan(y)
    assert bool(gone[:, [3, 5, 11, 13]].all()) and int(gone.sum()) == 12


def test_rows_past_32_bits():
    Q = qw()
    ld = 1 << 29
    buf = torch.empty(4 * ld + 256, dtype=torch.bfloat16, device="cuda")
    X = buf.as_strided((5, 256), (ld, 1))
    X.copy_(torch.randn(5, 256, device="cuda"))
    want = X.contiguous()
    pos = torch.tensor([5, 6, 7, 8, 9], dtype=torch.int32, device="cuda")
    freqs = Q.qw_rope_frequencies(Q.QW_ROPE_NONE, 1e4, 128)[0].cuda()
    Q.qw_rope(Q.QW_T_BF16, X, ld, X, ld, 5, 2, 128, 128, Q.QW_ROPE_HALF, pos, freqs)
    Q.qw_rope(Q.QW_T_BF16, want, 256, want, 256, 5, 2, 128, 128, Q.QW_ROPE_HALF, pos, freqs)
    assert torch.equal(X.contiguous(), want)
