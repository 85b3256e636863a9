"""Host-side refusals of the INT8 and log-probability entry points (no GPU: every call below
fails validation, or is a no-op, before any CUDA call)."""
import pytest


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


def product(Q, **kw):
    a = dict(afmt=Q.QW_A_BF16, A=G, lda=64, a_scale=None, W=G, w_scale=G, bias=None,
             c_type=Q.QW_T_BF16, C=G, ldc=32, M=4, N=32, K=64, workspace=G, ws_bytes=1 << 20,
             d_err=None, stream=0)
    a.update(kw)
    return status(Q.qgemm_int8, *a.values())


def test_product_refusals(Q):
    inv, uns, ali, wsp = (Q.QW_ERR_INVALID_ARG, Q.QW_ERR_UNSUPPORTED, Q.QW_ERR_ALIGNMENT,
                          Q.QW_ERR_WORKSPACE)
    assert product(Q, M=0) == Q.QW_OK
    assert product(Q, M=0, A=None, C=None, workspace=None, ws_bytes=0) == Q.QW_OK
    for kw, want in [
            (dict(M=-1), inv), (dict(M=1 << 31), inv), (dict(N=0), inv), (dict(K=0), inv),
            (dict(K=72, lda=72), uns), (dict(K=131072, lda=131072), uns),
            (dict(afmt=Q.QW_A_MXFP8_G32), uns), (dict(c_type=Q.QW_T_F16), uns),
            (dict(lda=56), inv), (dict(ldc=31), inv),
            (dict(a_scale=G), inv),                               # BF16 rows bring no scales
            (dict(afmt=Q.QW_A_INT8_TOKEN), inv),                  # INT8 rows have to
            (dict(A=None), inv), (dict(W=None), inv), (dict(w_scale=None), inv), (dict(C=None), inv),
            (dict(A=G + 8), ali), (dict(lda=68), ali), (dict(W=G + 8), ali), (dict(w_scale=G + 2), ali),
            (dict(afmt=Q.QW_A_INT8_TOKEN, a_scale=G, lda=72), ali), (dict(bias=G + 1), ali),
            (dict(afmt=Q.QW_A_INT8_TOKEN, a_scale=G + 2), ali),
            (dict(C=G + 1), ali), (dict(c_type=Q.QW_T_F32, C=G + 2), ali),
            (dict(workspace=None), wsp), (dict(ws_bytes=16), wsp), (dict(workspace=G + 16), ali)]:
        assert product(Q, **kw) == want, kw


def test_gated_refusals(Q):
    def gated(**kw):
        a = dict(afmt=Q.QW_A_BF16, A=G, lda=64, a_scale=None, W=G, w_scale=G, bias=None, Y=G,
                 ldy=32, M=4, I=32, K=64, workspace=G, ws_bytes=1 << 20, d_err=None, stream=0)
        a.update(kw)
        return status(Q.qgemm_int8_gated, *a.values())
    assert gated(M=0) == Q.QW_OK
    for kw, want in [(dict(I=0), Q.QW_ERR_INVALID_ARG), (dict(I=1 << 30), Q.QW_ERR_INVALID_ARG),
                     (dict(ldy=31), Q.QW_ERR_INVALID_ARG), (dict(Y=G + 1), Q.QW_ERR_ALIGNMENT),
                     (dict(K=24, lda=24), Q.QW_ERR_UNSUPPORTED),
                     (dict(workspace=None), Q.QW_ERR_WORKSPACE)]:
        assert gated(**kw) == want, kw


def test_quantizer_refusals(Q):
    def quant(**kw):
        a = dict(A=G, lda=64, rows=4, K=64, A_q=G, A_scale=G, d_err=None, stream=0)
        a.update(kw)
        return status(Q.qw_quantize_int8, *a.values())
    assert quant(rows=0) == Q.QW_OK
    for kw, want in [(dict(rows=-1), Q.QW_ERR_INVALID_ARG), (dict(lda=48), Q.QW_ERR_INVALID_ARG),
                     (dict(K=40), Q.QW_ERR_UNSUPPORTED), (dict(rows=1 << 31), Q.QW_ERR_UNSUPPORTED),
                     (dict(A=None), Q.QW_ERR_INVALID_ARG), (dict(A=G + 2), Q.QW_ERR_ALIGNMENT),
                     (dict(lda=66), Q.QW_ERR_ALIGNMENT), (dict(A_q=G + 8), Q.QW_ERR_ALIGNMENT),
                     (dict(A_scale=G + 1), Q.QW_ERR_ALIGNMENT)]:
        assert quant(**kw) == want, kw


def test_workspace_sizes(Q):
    for fmt in (Q.QW_A_BF16, Q.QW_A_INT8_TOKEN):
        last = 0
        for M in (0, 1, 8, 16, 17, 64, 4096, 100000):
            n = Q.qgemm_int8_workspace_size(fmt, M, 512, 4096)
            assert n >= last and n <= M * 4096 * 2 + 4 * M + 256
            last = n
    for args in [(Q.QW_A_NVFP4_G16, 4, 32, 64), (Q.QW_A_BF16, -1, 32, 64), (Q.QW_A_BF16, 4, 0, 64),
                 (Q.QW_A_BF16, 4, 32, 100)]:
        with pytest.raises(Q.QwError):
            Q.qgemm_int8_workspace_size(*args)


def test_logprobs_refusals(Q):
    def lp(**kw):
        a = dict(l_type=Q.QW_T_BF16, logits=G, ld=100, T=4, V=100, tokens=G, topk=5,
                 token_logprobs=G, token_ranks=G, entropy=G, top_ids=G, top_logprobs=G, d_err=None,
                 stream=0)
        a.update(kw)
        return status(Q.qw_logprobs, *a.values())
    inv, ali = Q.QW_ERR_INVALID_ARG, Q.QW_ERR_ALIGNMENT
    assert lp(T=0) == Q.QW_OK
    for kw, want in [(dict(l_type=3), Q.QW_ERR_UNSUPPORTED), (dict(T=-1), inv), (dict(V=0), inv),
                     (dict(ld=99), inv), (dict(topk=-1), inv), (dict(topk=33), inv),
                     (dict(V=4, topk=5), inv), (dict(T=(1 << 26) + 1), inv), (dict(logits=None), inv),
                     (dict(tokens=None), inv), (dict(top_ids=None), inv), (dict(top_logprobs=None), inv),
                     (dict(logits=G + 1), ali), (dict(l_type=Q.QW_T_F32, logits=G + 2), ali),
                     (dict(tokens=G + 2), ali), (dict(entropy=G + 2), ali), (dict(top_ids=G + 2), ali)]:
        assert lp(**kw) == want, kw
