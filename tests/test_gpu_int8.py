"""The INT8 product, its gated form and the per-token quantiser on the GPU, against 64-bit
restatements of their formulas.

Tolerance (derived, not fitted).  Codes are bit-exact.  With S the exact integer sum and
B = sum |a w|: while B < 2^24 every partial sum is an FP32 integer, so the sum is exact; beyond
that each of the K/16 tensor-core steps may lose 2^-23 of a partial sum of at most B.  The scale
product, its multiplication and the bias addition round to FP32 three times, and the result
rounds once to BF16 (2^-8 relative) or not at all.  The gate adds expf (2 ulp), a division and
two products, and |silu'| <= 1.1."""
import numpy as np
import pytest
import torch

from qwtest import dev, host, qw

pytestmark = pytest.mark.gpu


def bf16(x):
    """float32 array -> (values rounded to BF16, their bits)."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)
    return t.float().numpy(), t


def quantize_ref(a):
    """FP32 restatement, operation for operation (codes must match bit for bit)."""
    a = a.astype(np.float32)
    amax = np.abs(a).max(axis=1, keepdims=True)
    with np.errstate(divide="ignore", over="ignore"):
        inv = np.minimum(np.float32(127.0) / amax, np.finfo(np.float32).max)
    q = np.rint((a * inv).astype(np.float32))
    return q.astype(np.int64), (amax[:, 0] / np.float32(127.0)).astype(np.float32)


def product_ref(q, sa, w, sw, bias):
    """64-bit value and error bound before the output's rounding."""
    S = q.astype(np.float64) @ w.astype(np.float64).T
    B = np.abs(q).astype(np.float64) @ np.abs(w).astype(np.float64).T
    K = q.shape[1]
    sc = sa.astype(np.float64)[:, None] * sw.astype(np.float64)[None, :]
    R = S * sc
    E = 2.0 ** -22 * np.abs(R) + np.where(B < 2.0 ** 24, 0.0, 2.0 ** -23 * (K / 16 + 2) * B * sc)
    if bias is not None:
        b = bias.astype(np.float64)[None, :]
        E = E + 2.0 ** -22 * (np.abs(R) + np.abs(b))
        R = R + b
    return R, E


def problem(M, N, K, seed, a="bf16", bias=False, pad=0, extreme=False):
    rng = np.random.default_rng(seed)
    lo, hi = (-128, 128) if extreme else (-127, 128)
    w = rng.integers(lo, hi, (N, K)).astype(np.int8)
    if extreme:
        w[: N // 2] = -128
    sw = rng.uniform(0.5, 1.5, N).astype(np.float32) / np.float32(64 * np.sqrt(K))
    p = dict(M=M, N=N, K=K, w=w, sw=sw, bias=None, pad=pad)
    if bias:
        p["bias"], p["bias_t"] = bf16(rng.normal(0, 1, N))
    if a == "int8":
        q = rng.integers(lo, hi, (M, K + pad)).astype(np.int8)
        if extreme:
            q[: M // 2 + 1] = -128
        sa = rng.uniform(0.01, 0.05, M).astype(np.float32)
        p.update(q=q[:, :K].astype(np.int64), sa=sa, A=dev(q), sa_t=dev(sa))
    else:
        x = rng.normal(0, 1, (M, K + pad)) * np.exp2(rng.integers(-6, 6, (M, 1)))
        x, xt = bf16(x)
        q, sa = quantize_ref(x[:, :K])
        p.update(q=q, sa=sa, A=xt.cuda(), sa_t=None)
    return p


def call(p, afmt=None, c_type=None, gated=False, ldc_pad=0, stream=None):
    Q = qw()
    M, N, K = p["M"], p["N"], p["K"]
    afmt = (Q.QW_A_BF16 if p["sa_t"] is None else Q.QW_A_INT8_TOKEN) if afmt is None else afmt
    c_type = Q.QW_T_BF16 if c_type is None else c_type
    cols = N // 2 if gated else N
    dt = torch.float32 if c_type == Q.QW_T_F32 else torch.bfloat16
    C = torch.full((max(M, 1), cols + ldc_pad), 776.0, dtype=dt, device="cuda")
    n = Q.qgemm_int8_workspace_size(afmt, M, N, K)
    ws = torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda")
    err = Q.new_error_flag()
    bias = p["bias_t"].cuda() if p["bias"] is not None else None
    W, sw = dev(p["w"]), dev(p["sw"])
    torch.cuda.synchronize()
    lda = K + p["pad"]
    if gated:
        Q.qgemm_int8_gated(afmt, p["A"], lda, p["sa_t"], W, sw, bias, C, cols + ldc_pad, M,
                           N // 2, K, ws, n, err, stream)
    else:
        Q.qgemm_int8(afmt, p["A"], lda, p["sa_t"], W, sw, bias, c_type, C, cols + ldc_pad, M, N,
                     K, ws, n, err, stream)
    assert Q.qw_read_error(err, stream) == 0
    out = C.float().cpu().numpy().astype(np.float64)
    assert (out[:, cols:] == 776.0).all()  # nothing written past a row's columns
    return out[:M, :cols]


def check(p, out, f32=False):
    R, E = product_ref(p["q"], p["sa"], p["w"], p["sw"], p["bias"])
    tol = E if f32 else E + 2.0 ** -8 * (np.abs(R) + E) + 1e-38
    bad = np.abs(out - R) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], out[bad][:5], R[bad][:5], tol[bad][:5])


def check_gated(p, out):
    R, E = product_ref(p["q"], p["sa"], p["w"], p["sw"], p["bias"])
    n = p["N"] // 2
    g, u, eg, eu = R[:, :n], R[:, n:], E[:, :n], E[:, n:]
    with np.errstate(over="ignore"):
        silu = g / (1.0 + np.exp(-g))
    y = silu * u
    tol = (1.1 * eg * (np.abs(u) + eu) + (np.abs(silu) + eg) * eu) * 1.01 \
        + np.abs(y) * (2.0 ** -8 + 2.0 ** -20) + 1e-38
    bad = np.abs(out - y) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], out[bad][:5], y[bad][:5], tol[bad][:5])


# one row up to several token tiles; widths that end inside every tile; K that ends inside a
# stage (multiples of 16 only) and K long enough to be split
SHAPES = [(1, 1, 16), (1, 130, 4096), (2, 17, 48), (3, 1000, 1040), (5, 129, 8208), (8, 64, 512),
          (9, 33, 2064), (16, 300, 14336), (17, 128, 64), (31, 257, 272), (33, 96, 6160),
          (48, 1111, 1040), (64, 4099, 512), (65, 31, 80), (127, 200, 1296), (128, 128, 128),
          (129, 385, 656), (255, 259, 336), (256, 512, 1024), (257, 130, 4112), (300, 1, 96),
          (513, 640, 208), (700, 1029, 2048)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_from_bf16(M, N, K):
    p = problem(M, N, K, M * 31 + N + K, bias=(M + N) % 2 == 1, pad=8 * (M % 3))
    check(p, call(p))


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_from_codes_f32(M, N, K):
    p = problem(M, N, K, M * 37 + N + K, a="int8", bias=(M + N) % 2 == 0, pad=16 * (M % 3))
    check(p, call(p, c_type=qw().QW_T_F32, ldc_pad=M % 4), f32=True)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gated(M, N, K):
    a = "int8" if (M + K) % 3 == 0 else "bf16"
    p = problem(M, 2 * N, K, M * 41 + N + K, a=a, bias=(M + N) % 2 == 1, pad=16 * (M % 2))
    check_gated(p, call(p, gated=True, ldc_pad=M % 3))


@pytest.mark.parametrize("M", [1, 4, 16, 40, 200])
def test_extreme_codes(M):
    """-128 on both sides: sums of 2^14 K pass 2^24 at K = 1024."""
    p = problem(M, 96, 8192, 5 + M, a="int8", extreme=True)
    check(p, call(p, c_type=qw().QW_T_F32), f32=True)


@pytest.mark.parametrize("M", [1, 16, 40, 300])
def test_contiguous_output_and_pitched_output_agree(M):
    p = problem(M, 264, 528, 11, bias=True)
    assert np.array_equal(call(p), call(p, ldc_pad=5))


@pytest.mark.parametrize("rows,K", [(1, 16), (3, 1040), (37, 4096), (5, 14336), (2, 40000), (130, 272)])
def test_quantizer_bit_exact(rows, K):
    Q = qw()
    rng = np.random.default_rng(rows + K)
    x = rng.normal(0, 1, (rows, K + 24)) * np.exp2(rng.integers(-120, 100, (rows, 1)))
    if rows > 1:
        x[1] = 0.0
        x[0, :4] = [0.5, 2.5, -1.5, 127.0]  # ties once the row is scaled
        x[0, 4:] = np.clip(x[0, 4:], -1, 1)
    if rows > 2:
        x[2] = np.exp2(-133.0) * rng.integers(-1, 2, K + 24)  # subnormals
    x, xt = bf16(x)
    q = torch.full((rows, K), 99, dtype=torch.int8, device="cuda")
    s = torch.empty(rows, device="cuda")
    err = Q.new_error_flag()
    Q.qw_quantize_int8(xt.cuda(), K + 24, rows, K, q, s, err)
    assert Q.qw_read_error(err) == 0
    rq, rs = quantize_ref(x[:, :K])
    assert np.array_equal(host(q), rq)
    assert np.array_equal(host(s), rs)


def test_product_from_bf16_equals_quantise_then_product():
    Q = qw()
    for M in (1, 7, 16, 90, 300):
        p = problem(M, 520, 1040, M, bias=True)
        q = torch.empty((M, 1040), dtype=torch.int8, device="cuda")
        s = torch.empty(M, device="cuda")
        Q.qw_quantize_int8(p["A"], 1040, M, 1040, q, s)
        assert np.array_equal(call(p), call(dict(p, A=q, sa_t=s)))


@pytest.mark.parametrize("M", [1, 12, 70])
@pytest.mark.parametrize("what", [np.inf, -np.inf, np.nan])
def test_non_finite_rows_are_nan_and_flagged(M, what):
    Q = qw()
    p = problem(M, 72, 256, 3, bias=True)
    p["A"][M // 2, 200] = what
    C = torch.zeros((M, 72), dtype=torch.float32, device="cuda")
    n = Q.qgemm_int8_workspace_size(Q.QW_A_BF16, M, 72, 256)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    err = Q.new_error_flag()
    Q.qgemm_int8(Q.QW_A_BF16, p["A"], 256, None, dev(p["w"]), dev(p["sw"]), p["bias_t"].cuda(),
                 Q.QW_T_F32, C, 72, M, 72, 256, ws, n, err)
    assert Q.qw_read_error(err) == Q.QW_ERR_VALUE
    out = C.cpu().numpy()
    assert np.isnan(out[M // 2]).all()
    assert np.isfinite(np.delete(out, M // 2, axis=0)).all()


def test_gate_saturates_without_nan():
    """Gates far out on both sides: silu(-1e6) = -0, silu(1e6) = 1e6."""
    for M in (2, 40):
        p = problem(M, 64, 64, 9, a="int8")
        p["sw"][:] = 10.0
        out = call(p, gated=True)
        assert np.isfinite(out).all()
        check_gated(p, out)


def test_weights_and_rows_past_two_to_the_31():
    """Byte offsets beyond 2^31 in the weights, the activations' pitch and the output's pitch;
    sampled rows and columns against the reference."""
    Q = qw()
    rng = np.random.default_rng(7)
    K, N = 65536, 33000  # 2.16e9 weight bytes
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    W = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    sw = torch.rand(N, device="cuda", generator=g) * 1e-4
    for M in (2, 24):
        x, xt = bf16(rng.normal(0, 1, (M, K)))
        q, sa = quantize_ref(x)
        C = torch.empty((M, N), dtype=torch.float32, device="cuda")
        n = Q.qgemm_int8_workspace_size(Q.QW_A_BF16, M, N, K)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        Q.qgemm_int8(Q.QW_A_BF16, xt.cuda(), K, None, W, sw, None, Q.QW_T_F32, C, N, M, N, K, ws, n)
        cols = np.array([0, 1, N // 2, 32767, 32768, 32769, N - 2, N - 1])
        ci = torch.from_numpy(cols).cuda()
        w, s, out = W[ci].cpu().numpy(), sw[ci].cpu().numpy(), C[:, ci].cpu().numpy()
        R, E = product_ref(q, sa, w, s, None)
        assert (np.abs(out - R) <= E).all()
    del W
    pitch = 2**30 + 16
    for M in (3, 18):
        p = problem(M, 40, 64, 21, a="int8")
        wide = torch.empty((M - 1) * (pitch // (1 if M == 3 else 8)) + 64, dtype=torch.int8, device="cuda")
        lda = pitch // (1 if M == 3 else 8) // 16 * 16
        for r in range(M):
            wide[r * lda:r * lda + 64] = p["A"][r]
        ldc = lda
        C = torch.empty((M - 1) * ldc + 40, dtype=torch.bfloat16, device="cuda")
        n = Q.qgemm_int8_workspace_size(Q.QW_A_INT8_TOKEN, M, 40, 64)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        Q.qgemm_int8(Q.QW_A_INT8_TOKEN, wide, lda, p["sa_t"], dev(p["w"]), dev(p["sw"]), None,
                     Q.QW_T_BF16, C, ldc, M, 40, 64, ws, n)
        out = torch.stack([C[r * ldc:r * ldc + 40] for r in range(M)]).float().cpu().numpy()
        check(p, out)


def test_on_another_stream_and_in_a_graph():
    Q = qw()
    p = problem(40, 300, 528, 4)
    want = call(p)
    st = torch.cuda.Stream()
    assert np.array_equal(call(p, stream=st), want)
    W, sw = dev(p["w"]), dev(p["sw"])
    C = torch.zeros((40, 300), dtype=torch.bfloat16, device="cuda")
    n = Q.qgemm_int8_workspace_size(Q.QW_A_BF16, 40, 300, 528)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q.qgemm_int8(Q.QW_A_BF16, p["A"], 528, None, W, sw, None, Q.QW_T_BF16, C, 300, 40, 300, 528, ws, n)
    graph.replay()
    assert np.array_equal(C.float().cpu().numpy(), want)


def test_deterministic():
    for M in (1, 16, 40, 300):
        p = problem(M, 520, 6160, 8, bias=True)
        a = call(p)
        for _ in range(3):
            assert np.array_equal(call(p), a)
