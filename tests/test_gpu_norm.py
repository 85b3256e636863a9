"""qw_rmsnorm on the GPU against 64 bits.

Bound.  The sum of squares is one of positive terms in chains of at most c = 8 ceil(K / 8 / lanes) + 10
additions, lanes being 32 up to K = 1024 and at least min(K / 32, 512) beyond (a thread has four vectors
of eight values where a call has many rows: 32 additions, ten for the joins); each adds 2^-24, and
1 / rms has half of that, the division and the addition of eps 2^-24 each, 1 / rms itself no more than
2^-23.  h w, w_offset + w and y add 2^-24 each.  So y is within e |y|, e = 2^-24 (c / 2 + 7), before it is
rounded: to BF16 (2^-8 |y|), to E4M3 (2^-4 |y|, below 2^-6 of its scale 2^-10 of it) or to a step of the
row's INT8 scale (half a step; the quotient's roundings add at most 127 * 3 * 2^-24 of one)."""
import math

import numpy as np
import pytest
import torch

from qwtest import qw

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def bound(K):
    lanes = 32 if K <= 1024 else min(K // 32, 512)
    return 2.0 ** -24 * ((8 * math.ceil(K / 8 / lanes) + 10) / 2 + 7)


def wide(values, pad, dtype):
    """values as the first columns of a wider tensor that is NaN elsewhere."""
    t = torch.full((values.shape[0], values.shape[1] + pad), float("nan"), dtype=dtype, device="cuda")
    t[:, :values.shape[1]] = values
    return t


def call(x, r, w, q, y=True, pad=0, offset=0.0, eps=EPS, keep=True, want_err=0, stream=None):
    """x, r (or None): values [rows][K] in their types; -> dict of outputs."""
    Q = qw()
    kinds = {torch.bfloat16: Q.QW_T_BF16, torch.float32: Q.QW_T_F32}
    rows, K = x.shape
    X = wide(x, pad, x.dtype)
    R = None if r is None else wide(r, 2 * pad, r.dtype)
    out = wide(torch.zeros_like(r), pad, r.dtype) if r is not None and keep else None
    Y = wide(torch.zeros_like(x, dtype=torch.bfloat16), pad, torch.bfloat16) if y else None
    fmt, codes, sf = Q.QW_A_BF16, None, None
    if q == "int8":
        fmt = Q.QW_A_INT8_TOKEN
        codes = torch.full((rows, K), 99, dtype=torch.int8, device="cuda")
        sf = torch.full((rows,), 7.0, device="cuda")
    elif q == "mxfp8":
        fmt = Q.QW_A_MXFP8_G32
        codes = torch.full((rows, K), 99, dtype=torch.uint8, device="cuda")
        sf = torch.full((rows, K // 32), 99, dtype=torch.uint8, device="cuda")
    err = Q.new_error_flag()
    torch.cuda.synchronize()
    Q.qw_rmsnorm(kinds[x.dtype], X, K + pad, kinds[r.dtype] if r is not None else 0, R, K + 2 * pad,
                 out, K + pad, w, offset, eps, rows, K, Y, K + pad, fmt, codes, sf, err, stream)
    assert Q.qw_read_error(err, stream) == want_err
    for t in (out, Y):  # what lies beside the rows is as it was
        assert t is None or bool(torch.isnan(t[:, K:]).all())
    return dict(h=None if out is None else out[:, :K], y=None if Y is None else Y[:, :K],
                codes=codes, sf=sf)


def reference(x, r, w, offset=0.0, eps=EPS):
    """(h as stored or None, y in 64 bits)"""
    h = None if r is None else (x.float() + r.float()).to(r.dtype)
    d = (x if h is None else h).double()
    rms = (d.square().mean(dim=1, keepdim=True) + eps).sqrt()
    return h, d * (w.double() + offset) / rms


def check(got, h, y, q, e):
    if got["h"] is not None:
        assert torch.equal(got["h"], h)
    tiny = 2.0 ** -133
    if got["y"] is not None:
        assert bool(((got["y"].double() - y).abs() <= (2.0 ** -8 * (1 + e) + e) * y.abs() + tiny).all())
    if q == "int8":
        top = y.abs().amax(dim=1)
        assert bool(((got["sf"].double() - top / 127).abs() <= (e + 2.0 ** -23) * top / 127).all())
        step = got["sf"].double()[:, None]
        off = (got["codes"].double() * step - y).abs()
        assert bool((off <= step * (0.5 + 127 * 4 * 2.0 ** -24) + 2 * e * y.abs()).all())
        assert int(got["codes"].min()) >= -127
    elif q == "mxfp8":
        rows, K = y.shape
        g = y.view(rows, K // 32, 32)
        top = g.abs().amax(dim=2)
        power = got["sf"].double() - 127
        fl = torch.floor(torch.log2(top)) - 8
        near = (torch.floor(torch.log2(top * (1 - e))) != torch.floor(torch.log2(top * (1 + e))))
        assert bool(((power == fl) | (near & ((power - fl).abs() <= 1)) | (top == 0)).all())
        assert bool((got["sf"][top == 0] == 0).all())
        unit = torch.exp2(power)[:, :, None]
        v = got["codes"].view(torch.float8_e4m3fn).double().view(rows, K // 32, 32) * unit
        off = (v - g).abs()
        full = g.abs() > 448 * unit * (1 - e)
        assert bool((v.abs()[full] <= 448 * unit.expand_as(v)[full]).all())
        assert bool((v.abs()[full] >= 416 * unit.expand_as(v)[full]).all())
        ok = off <= (2.0 ** -4 * (1 + e) + e) * g.abs() + 2.0 ** -10 * unit
        assert bool((ok | full).all())


def problem(rows, K, x, r, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def draw(dtype):
        t = torch.randn((rows, K), generator=g, device="cuda")
        t *= torch.exp2(torch.randint(-6, 7, (rows, 1), generator=g, device="cuda").float())
        return t.to(dtype)
    w = (1 + 0.3 * torch.randn(K, generator=g, device="cuda")).to(torch.bfloat16)
    return draw(TYPES[x]), None if r is None else draw(TYPES[r]), w


SHAPES = [(1, 32), (3, 64), (9, 96), (2, 1024), (5, 1056), (1, 4096), (333, 1056), (64, 7168),
          (2, 16384), (3, 16416), (2, 32800), (1, 131072), (5000, 160)]


@pytest.mark.parametrize("rows,K", SHAPES)
@pytest.mark.parametrize("q", ["mxfp8", "int8", None])
def test_shapes(rows, K, q):
    i = rows + K
    x, r = [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16"), ("bf16", None),
            ("f32", None)][i % 6]
    xv, rv, w = problem(rows, K, x, r, i)
    h, y = reference(xv, rv, w)
    check(call(xv, rv, w, q, y=q is None or i % 2 == 0, pad=[0, 8, 40][i % 3]), h, y, q, bound(K))


@pytest.mark.parametrize("rows,K", [(1300, 1056), (320, 4096), (200, 7200), (160, 16384), (155, 16352)])
@pytest.mark.parametrize("x,r", [("bf16", "bf16"), ("bf16", None), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("q", ["mxfp8", "int8", None])
def test_more_rows_than_run_at_once(rows, K, x, r, q):
    xv, rv, w = problem(rows, K, x, r, rows)
    xv[rows - 1] *= 1e30  # (its squares pass FP32; the row before it is the same CTA's or another's)
    h, y = reference(xv, rv, w, 1.0)
    check(call(xv, rv, w, q, y=True, pad=8, offset=1.0), h, y, q, bound(K))


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("r", [None, "bf16", "f32"])
@pytest.mark.parametrize("q", ["mxfp8", "int8", None])
def test_types(x, r, q):
    for K in (128, 2080):
        xv, rv, w = problem(7, K, x, r, 11)
        for offset, keep in ((0.0, True), (1.0, False)):
            h, y = reference(xv, rv, w, offset)
            check(call(xv, rv, w, q, y=True, pad=8, offset=offset, keep=keep), h, y, q, bound(K))


@pytest.mark.parametrize("K", [8, 24, 1000, 1016, 1032, 4104])
def test_widths_of_bf16_rows(K):
    xv, rv, w = problem(5, K, "bf16", "bf16", K)
    h, y = reference(xv, rv, w)
    check(call(xv, rv, w, None), h, y, None, bound(K))


@pytest.mark.parametrize("K", [64, 4096, 20000])
@pytest.mark.parametrize("q", ["mxfp8", "int8", None])
def test_extremes(K, q):
    """Zeros, squares that pass FP32 or vanish in it, one loud value, residuals that cancel."""
    xv, rv, w = problem(8, K, "f32", "f32", 5)
    xv[0], rv[0] = 0, 0
    xv[1] *= 1e30
    xv[2] *= 1e-30
    rv[2] *= 1e-30
    xv[3] = 0
    rv[3] = 0
    xv[3, K // 2] = 3e38
    rv[4] = -xv[4]
    xv[5], rv[5] = 1e-3, 0
    xv[5, 0] = 1e4
    for eps in (1e-5, 1e-12):
        h, y = reference(xv, rv, w, eps=eps)
        got = call(xv, rv, w, q, eps=eps)
        # (row 2: y below 1e-21; its INT8 codes and scale follow the bound as well)
        check(got, h, y, q, bound(K))
        assert bool((got["y"][0] == 0).all()) and bool((got["y"][4] == 0).all())


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("K", [96, 4096, 20000])
@pytest.mark.parametrize("q", ["mxfp8", "int8", None])
def test_rows_that_are_not_finite(value, K, q):
    """The row says so and the others are right."""
    Q = qw()
    xv, rv, w = problem(6, K, "bf16", "bf16", 3)
    xv[2, K - 5] = value
    rv[4, 0] = value
    xv[5, 1], rv[5, 1] = 3.38e38, 3.38e38  # the sum passes the type
    got = call(xv, rv, w, q, want_err=Q.QW_ERR_VALUE)
    for row in (2, 4, 5):
        assert bool(torch.isnan(got["y"][row]).all())
        if q == "int8":
            assert bool(torch.isnan(got["sf"][row])) and bool((got["codes"][row] == 0).all())
        elif q == "mxfp8":
            assert bool((got["sf"][row] == 255).all()) and bool((got["codes"][row] == 0).all())
    fine = [0, 1, 3]
    h, y = reference(xv[fine], rv[fine], w)
    part = {k: None if v is None else v[fine] for k, v in got.items()}
    check(part, h, y, q, bound(K))


@pytest.mark.parametrize("K", [256, 4096, 20000])
def test_in_place(K):
    """R_out over R, or over X; Y over X: the same values as with buffers of their own."""
    Q = qw()
    xv, rv, w = problem(5, K, "bf16", "bf16", 9)
    want = call(xv, rv, w, "int8")
    for over in ("r", "x"):
        X, R = xv.clone(), rv.clone()
        out = R if over == "r" else X
        Y = X if over == "r" else torch.empty_like(X)
        codes = torch.empty((5, K), dtype=torch.int8, device="cuda")
        sf = torch.empty(5, device="cuda")
        Q.qw_rmsnorm(Q.QW_T_BF16, X, K, Q.QW_T_BF16, R, K, out, K, w, 0.0, EPS, 5, K, Y, K,
                     Q.QW_A_INT8_TOKEN, codes, sf)
        assert torch.equal(out, want["h"]) and torch.equal(Y, want["y"])
        assert torch.equal(codes, want["codes"]) and torch.equal(sf, want["sf"])


def test_rows_past_32_bits():
    """A pitch that takes the last rows past 2^31 elements."""
    Q = qw()
    rows, K, ld = 5, 1024, 1 << 29
    buf = torch.empty(4 * ld + K, dtype=torch.bfloat16, device="cuda")
    X = buf.as_strided((rows, K), (ld, 1))
    xv, _, w = problem(rows, K, "bf16", None, 2)
    X.copy_(xv)
    Y = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda")
    Q.qw_rmsnorm(Q.QW_T_BF16, X, ld, 0, None, 0, None, 0, w, 0.0, EPS, rows, K, Y, K)
    _, y = reference(xv, None, w)
    check(dict(h=None, y=Y, codes=None, sf=None), None, y, None, bound(K))


def test_many_rows_are_each_their_own():
    """More rows than a grid of one wave; each equal to the row alone."""
    xv, rv, w = problem(40000, 256, "bf16", "bf16", 21)
    got = call(xv, rv, w, "mxfp8")
    pick = [0, 1, 17777, 39998, 39999]
    alone = call(xv[pick], rv[pick], w, "mxfp8")
    for k in got:
        assert torch.equal(got[k][pick], alone[k]), k
    assert np.isfinite(got["y"].float().sum().item())
