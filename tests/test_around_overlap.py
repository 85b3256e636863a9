"""The adapters' result in the place of one of their inputs: refused before any launch (no GPU), since slices of K
are read while other clusters already write columns of C."""
import pytest

G = 1 << 20  # a 256-byte aligned fake pointer, never dereferenced


@pytest.fixture(scope="module")
def lora():
    import moe_qw_repack_gb300.qw as Q

    def call(**kw):
        a = dict(X=G, ldx=64, A=2 * G, B=3 * G, scales=4 * G, ranks=5 * G, L=2, R=16, ids=6 * G, base=7 * G,
                 ld_base=64, c_type=Q.QW_T_BF16, C=8 * G, ldc=64, M=4, N=64, K=64, d_err=None, stream=0)
        a.update(kw)
        try:
            Q.qgemm_lora(*a.values())
        except Q.QwError as e:
            return e.status
        return Q.QW_OK
    return Q, call


@pytest.mark.parametrize("over", ["X", "A", "B", "scales", "ranks", "ids"])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M", [1, 4, 1000])
def test_adapter_results_over_an_input(lora, over, f32, M):
    Q, call = lora
    kind = Q.QW_T_F32 if f32 else Q.QW_T_BF16
    at = 9 * G
    assert call(**{over: at}, C=at, c_type=kind, M=M) == Q.QW_ERR_INVALID_ARG
    assert call(**{over: at}, C=at, base=at, c_type=kind, M=M) == Q.QW_ERR_INVALID_ARG  # in place too
    assert call(**{over: at}, C=at, base=None, c_type=kind, M=M) == Q.QW_ERR_INVALID_ARG


def test_the_other_refusals_with_pointers_of_their_own(lora):
    Q, call = lora
    inv, uns, ali = Q.QW_ERR_INVALID_ARG, Q.QW_ERR_UNSUPPORTED, Q.QW_ERR_ALIGNMENT
    for kw, want in [
            (dict(C=7 * G, ldc=72), inv),  # C is base, at another pitch
            (dict(X=None), inv), (dict(A=None), inv), (dict(B=None), inv), (dict(ids=None), inv),
            (dict(C=None), inv), (dict(C=None, base=None), inv), (dict(ldx=56), inv), (dict(ldc=63), inv),
            (dict(ld_base=63), inv), (dict(R=264), uns), (dict(K=60), uns), (dict(X=G + 8), ali),
            (dict(C=8 * G + 1), ali), (dict(scales=G + 1), ali)]:
        assert call(**kw) == want, kw
