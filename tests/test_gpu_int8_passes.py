"""Passes of the INT8 products queued without a pause, over different activations that share one
workspace: every pass's whole output has to be that of its own activations.  (Codes or scales of the
pass before, a product that starts before its quantiser is done, a barrier that passes out of turn.)"""
import pytest
import torch

from qwtest import qw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,gated,codes,f32,passes", [
    (1, 14336, 4096, False, False, False, 240),
    (2, 4096, 8192, True, False, False, 240),      # slices over a cluster
    (1, 520, 1040, False, True, True, 240),
    (16, 4096, 14336, False, False, False, 240),   # split over clusters
    (9, 2050, 1040, True, True, False, 240),
    (64, 32003, 4096, False, True, True, 240),     # widened codes, two tiles to a CTA
    (64, 2048, 14336, False, False, False, 240),   # split over clusters
    (40, 300, 528, False, True, False, 240),
    (300, 8200, 4096, True, False, False, 120),    # 256 tokens a tile
    (700, 14336, 2048, False, False, False, 120),
])
def test_every_pass_is_its_own(M, N, K, gated, codes, f32, passes):
    Q = qw()
    g = torch.Generator(device="cuda").manual_seed(M + N)
    cols = N // 2 if gated else N
    kinds, ring = 3, 24
    if codes:
        A = [torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
             for _ in range(kinds)]
        S = [torch.rand(M, generator=g, device="cuda") + 0.5 for _ in range(kinds)]
    else:
        A = [(torch.randn(M, K, generator=g, device="cuda") * 2.0 ** (3 * i)).to(torch.bfloat16)
             for i in range(kinds)]
        S = [None] * kinds
    W = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.full((N,), 2.0 ** -12, device="cuda")
    afmt = Q.QW_A_INT8_TOKEN if codes else Q.QW_A_BF16
    dt = torch.float32 if f32 else torch.bfloat16
    n = Q.qgemm_int8_workspace_size(afmt, M, N, K)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    err = Q.new_error_flag()

    def run(i, C):
        if gated:
            Q.qgemm_int8_gated(afmt, A[i], K, S[i], W, sw, None, C, cols, M, cols, K, ws, n, err)
        else:
            Q.qgemm_int8(afmt, A[i], K, S[i], W, sw, None, Q.QW_T_F32 if f32 else Q.QW_T_BF16, C,
                         cols, M, N, K, ws, n, err)

    want = []
    for i in range(kinds):  # each alone
        ws.fill_(255)
        torch.cuda.synchronize()
        want.append(torch.empty(M, cols, dtype=dt, device="cuda"))
        run(i, want[i])
        torch.cuda.synchronize()
    assert not any(torch.equal(want[i], want[i - 1]) for i in range(kinds))
    outs = [torch.empty(M, cols, dtype=dt, device="cuda") for _ in range(ring)]
    order = torch.randint(kinds, (passes,), generator=torch.Generator().manual_seed(1)).tolist()
    for start in range(0, passes, ring):
        batch = order[start:start + ring]
        for C, i in zip(outs, batch):
            C.fill_(float("nan"))
        for C, i in zip(outs, batch):
            run(i, C)
        for j, (C, i) in enumerate(zip(outs, batch)):
            assert torch.equal(C, want[i]), (start + j, i)
    assert Q.qw_read_error(err) == 0


def test_log_probabilities_follow_their_logits():
    """The chain head -> log probabilities queued over three activations: each pass's answer is that of
    its own logits and tokens."""
    Q = qw()
    g = torch.Generator(device="cuda").manual_seed(5)
    V, K = 32003, 512
    W = torch.randint(-127, 128, (V, K), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.full((V,), 2.0 ** -9, device="cuda")
    for M in (1, 12, 64):
        A = [torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3)]
        T = [torch.randint(V, (M,), generator=g, device="cuda", dtype=torch.int32) for _ in range(3)]
        n = Q.qgemm_int8_workspace_size(Q.QW_A_BF16, M, V, K)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        logits = torch.empty(M, V, device="cuda")
        err = Q.new_error_flag()

        def new():
            return [torch.zeros(M, device="cuda"), torch.zeros(M, dtype=torch.int32, device="cuda"),
                    torch.zeros(M, device="cuda"), torch.zeros(M, 5, dtype=torch.int32, device="cuda"),
                    torch.zeros(M, 5, device="cuda")]

        def run(i, o):
            Q.qgemm_int8(Q.QW_A_BF16, A[i], K, None, W, sw, None, Q.QW_T_F32, logits, V, M, V, K, ws,
                         n, err)
            Q.qw_logprobs(Q.QW_T_F32, logits, V, M, V, T[i], 5, *o, err)

        want = []
        for i in range(3):
            torch.cuda.synchronize()
            want.append(new())
            run(i, want[i])
            torch.cuda.synchronize()
        outs = [new() for _ in range(60)]
        torch.cuda.synchronize()
        for j, o in enumerate(outs):
            run(j * 7 % 3, o)
        for j, o in enumerate(outs):
            assert all(torch.equal(a, b) for a, b in zip(o, want[j * 7 % 3])), j
        assert Q.qw_read_error(err) == 0
