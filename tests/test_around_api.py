"""Host-side refusals of the norm, adapter and rotary entry points (no GPU: every call below fails
validation, or is a no-op, before any CUDA call), and the rotary frequencies."""
import math

import pytest
import torch


@pytest.fixture(scope="module")
def Q():
    import moe_qw_repack_gb300.qw as q
    return q


G = 1 << 20  # a 256-byte aligned fake pointer, never dereferenced


def status(fn, *args):
    try:
        fn(*args)
    except Exception as e:  # QwError
        return e.status
    return 0


def test_norm_refusals(Q):
    inv, uns, ali = Q.QW_ERR_INVALID_ARG, Q.QW_ERR_UNSUPPORTED, Q.QW_ERR_ALIGNMENT
    nan, inf = float("nan"), float("inf")

    def norm(**kw):
        a = dict(x_type=Q.QW_T_BF16, X=G, ldx=64, r_type=Q.QW_T_BF16, R=G, ldr=64, R_out=G, ldro=64,
                 W=G, w_offset=0.0, eps=1e-6, rows=4, K=64, Y=G, ldy=64, q_fmt=Q.QW_A_MXFP8_G32, Q=G,
                 Q_sf=G, d_err=None, stream=0)
        a.update(kw)
        return status(Q.qw_rmsnorm, *a.values())
    assert norm(rows=0) == Q.QW_OK
    assert norm(rows=0, X=None, R=None, R_out=None, W=None, Y=None, Q=None, Q_sf=None) == Q.QW_OK
    none = dict(q_fmt=Q.QW_A_BF16, Q=None, Q_sf=None)
    for kw, want in [
            (dict(x_type=Q.QW_T_F16), uns), (dict(r_type=Q.QW_T_F16), uns),
            (dict(q_fmt=Q.QW_A_NVFP4_G16), uns), (dict(q_fmt=9), uns),
            (dict(rows=-1), inv), (dict(K=0), inv), (dict(ldx=56), inv), (dict(ldr=56), inv),
            (dict(ldro=56), inv), (dict(ldy=56), inv), (dict(rows=1 << 31), uns),
            (dict(K=48), uns), (dict(K=40, q_fmt=Q.QW_A_INT8_TOKEN), uns), (dict(K=60, **none), uns),
            (dict(eps=0.0), inv), (dict(eps=-1e-6), inv), (dict(eps=nan), inv), (dict(eps=inf), inv),
            (dict(w_offset=nan), inv), (dict(w_offset=inf), inv),
            (dict(X=None), inv), (dict(W=None), inv), (dict(R=None), inv),  # R_out without R
            (dict(Q=None), inv), (dict(Q_sf=None), inv), (dict(q_fmt=Q.QW_A_BF16), inv),
            (dict(Y=None, **none), inv),
            (dict(X=G + 8), ali), (dict(ldx=68), ali), (dict(R=G + 8), ali), (dict(ldr=68), ali),
            (dict(R_out=G + 8), ali), (dict(ldro=68), ali), (dict(W=G + 2), ali), (dict(Y=G + 8), ali),
            (dict(ldy=68), ali), (dict(Q=G + 8), ali),
            (dict(q_fmt=Q.QW_A_INT8_TOKEN, Q_sf=G + 2), ali),
            (dict(x_type=Q.QW_T_F32, ldx=66), ali), (dict(r_type=Q.QW_T_F32, ldr=66), ali)]:
        assert norm(**kw) == want, kw


def test_norm_refuses_buffers_in_each_others_place(Q):
    """What the declaration allows in place has one pitch and type; the rest is refused before any launch."""
    def norm(**kw):
        a = dict(x_type=Q.QW_T_BF16, X=G, ldx=64, r_type=Q.QW_T_BF16, R=2 * G, ldr=72, R_out=3 * G, ldro=80,
                 W=4 * G, w_offset=0.0, eps=1e-6, rows=4, K=64, Y=5 * G, ldy=88, q_fmt=Q.QW_A_MXFP8_G32,
                 Q=6 * G, Q_sf=7 * G, d_err=None, stream=0)
        a.update(kw)
        return status(Q.qw_rmsnorm, *a.values())
    for kw in (dict(R_out=2 * G), dict(R_out=G), dict(R_out=G, ldro=64, r_type=Q.QW_T_F32), dict(Y=G),
               dict(Y=G, ldy=64, x_type=Q.QW_T_F32), dict(Y=2 * G, ldy=72), dict(Y=3 * G, ldy=80),
               dict(Q=G), dict(Q=2 * G), dict(Q=3 * G), dict(Q=5 * G), dict(Q=7 * G)):
        assert norm(**kw) == Q.QW_ERR_INVALID_ARG, kw


def test_adapter_refusals(Q):
    inv, uns, ali = Q.QW_ERR_INVALID_ARG, Q.QW_ERR_UNSUPPORTED, Q.QW_ERR_ALIGNMENT

    def lora(**kw):
        a = dict(X=G, ldx=64, A=G, B=G, scales=G, ranks=G, L=2, R=16, ids=G, base=G, ld_base=32,
                 c_type=Q.QW_T_BF16, C=G, ldc=32, M=4, N=32, K=64, d_err=None, stream=0)
        a.update(kw)
        return status(Q.qgemm_lora, *a.values())
    assert lora(M=0) == Q.QW_OK
    assert lora(M=0, X=None, A=None, B=None, ids=None, base=None, C=None) == Q.QW_OK
    for kw, want in [
            (dict(c_type=Q.QW_T_F16), uns), (dict(M=-1), inv), (dict(N=0), inv), (dict(K=0), inv),
            (dict(L=0), inv), (dict(R=0), inv), (dict(ldx=56), inv), (dict(ldc=31), inv),
            (dict(ld_base=31), inv), (dict(K=60), uns), (dict(R=12), uns), (dict(R=264), uns),
            (dict(M=(1 << 26) + 1), uns), (dict(N=(1 << 31) - 1, ldc=1 << 31, ld_base=1 << 31), uns),
            (dict(X=None), inv), (dict(A=None), inv), (dict(B=None), inv), (dict(ids=None), inv),
            (dict(C=None), inv), (dict(ldc=40), inv),  # C is base, at another pitch
            (dict(X=G + 8), ali), (dict(ldx=68), ali), (dict(A=G + 8), ali), (dict(B=G + 8), ali),
            (dict(scales=G + 2), ali), (dict(ranks=G + 2), ali), (dict(ids=G + 1), ali),
            (dict(base=G + 1), ali), (dict(C=G + 1), ali), (dict(c_type=Q.QW_T_F32, C=G + 2), ali)]:
        assert lora(**kw) == want, kw


def test_rotary_refusals(Q):
    inv, uns, ali = Q.QW_ERR_INVALID_ARG, Q.QW_ERR_UNSUPPORTED, Q.QW_ERR_ALIGNMENT

    def rope(**kw):
        a = dict(type=Q.QW_T_BF16, X=G, ldx=256, Y=G, ldy=256, T=4, heads=2, head_dim=128, rot_dim=64,
                 layout=Q.QW_ROPE_HALF, positions=G, freqs=G, scale=1.0, d_err=None, stream=0)
        a.update(kw)
        return status(Q.qw_rope, *a.values())
    assert rope(T=0) == Q.QW_OK
    assert rope(T=0, X=None, Y=None, positions=None, freqs=None) == Q.QW_OK
    for kw, want in [
            (dict(type=3), uns), (dict(layout=2), uns), (dict(layout=-1), uns), (dict(T=-1), inv),
            (dict(heads=0), inv), (dict(head_dim=0), inv), (dict(rot_dim=0), inv),
            (dict(rot_dim=63), inv), (dict(rot_dim=130), inv), (dict(ldx=255), inv),
            (dict(ldy=255), inv), (dict(ldy=264), inv),  # in place, at another pitch
            (dict(T=1 << 31), uns), (dict(head_dim=1032, ldx=4096, ldy=4096), uns),
            (dict(heads=1 << 20, ldx=1 << 30, ldy=1 << 30), uns),
            (dict(scale=float("nan")), inv), (dict(scale=float("inf")), inv),
            (dict(X=None), inv), (dict(Y=None), inv), (dict(positions=None), inv),
            (dict(freqs=None), inv), (dict(X=G + 1), ali), (dict(Y=G + 1), ali),
            (dict(type=Q.QW_T_F32, X=G + 2), ali), (dict(positions=G + 2), ali),
            (dict(freqs=G + 4), ali)]:
        assert rope(**kw) == want, kw


def test_frequency_refusals(Q):
    for args in [(5, 1e4, 64), (-1, 1e4, 64), (Q.QW_ROPE_NONE, 1e4, 63), (Q.QW_ROPE_NONE, 1e4, 0),
                 (Q.QW_ROPE_NONE, 1.0, 64), (Q.QW_ROPE_NONE, float("nan"), 64),
                 (Q.QW_ROPE_LINEAR, 1e4, 64, 0.5), (Q.QW_ROPE_YARN, 1e4, 64, 8.0),
                 (Q.QW_ROPE_BANDS, 1e4, 64, 8.0, 8192.0, 4.0, 4.0)]:
        with pytest.raises(Q.QwError):
            Q.qw_rope_frequencies(*args)


@pytest.mark.parametrize("rot", [2, 64, 128])
def test_frequencies(Q, rot):
    """Against the definitions; FP64 powers and divisions are good to 2^-50 here."""
    def close(got, want):
        want = torch.tensor(want, dtype=torch.float64)
        return bool(((got - want).abs() <= 2.0 ** -48 * want).all())
    plain = [1e4 ** (-2 * j / rot) for j in range(rot // 2)]
    f, s = Q.qw_rope_frequencies(Q.QW_ROPE_NONE, 1e4, rot)
    assert close(f, plain) and s == 1.0
    f, s = Q.qw_rope_frequencies(Q.QW_ROPE_LINEAR, 1e4, rot, 8.0)
    assert close(f, [v / 8 for v in plain]) and s == 1.0
    f, s = Q.qw_rope_frequencies(Q.QW_ROPE_NTK, 1e4, rot, 8.0)
    if rot > 2:  # the slowest frequency is stretched by the whole factor, the fastest not at all
        assert f[0] == 1.0 and abs(f[-1] * 8 / plain[-1] - 1) < 1e-12 and s == 1.0
    f, s = Q.qw_rope_frequencies(Q.QW_ROPE_YARN, 1e4, rot, 16.0, 4096.0, 1.0, 32.0)
    assert abs(s - (0.1 * math.log(16.0) + 1.0)) < 1e-6
    for v, w in zip(f.tolist(), plain):
        turns = 4096.0 * w / (2 * math.pi)
        if turns > 32:
            assert abs(v / w - 1) < 1e-12
        elif turns < 1:
            assert abs(v * 16 / w - 1) < 1e-12
        else:
            assert w / 16 < v < w
    g, s = Q.qw_rope_frequencies(Q.QW_ROPE_BANDS, 1e4, rot, 16.0, 4096.0, 1.0, 32.0)
    assert torch.equal(f, g) and s == 1.0
