"""examples/int8_decode.py: the INT8 products and the log probabilities together, and repeated passes
of the products whose weights come from HBM (several tiles per CTA, deep queues)."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from qwtest import qw

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "int8_decode.py")
    spec = importlib.util.spec_from_file_location("int8_decode", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens", [2, 12, 60, 300])
def test_prompt_scores_are_the_logits_softmax(tokens):
    """Tolerance: logits of at most 64 in magnitude; x log2(e) rounds once (2^-24 of 93, which is
    6e-6), 2^y and the FP32 sums of positive terms stay within 2^-21 relative per step of a tree of
    at most 16 levels (8e-6), the logarithm and the differences add 1e-6."""
    E = example()
    model = E.Model(vocab=5003, hidden=256, inner=512, seed=tokens)
    prompt = torch.randint(5003, (tokens,), device="cuda", dtype=torch.int32,
                           generator=torch.Generator(device="cuda").manual_seed(7))
    s = E.score(model, prompt, top=4)
    x = s.logits.double()
    assert x.abs().max() < 64
    lp = torch.log_softmax(x, dim=1)
    want = lp.gather(1, s.next.long()[:, None])[:, 0]
    assert (s.logprob.double() - want).abs().max() < 3e-5
    top, ids = torch.sort(x, dim=1, descending=True, stable=True)
    assert torch.equal(s.top_ids.long(), ids[:, :4])
    assert (s.top_logprobs.double() - lp.gather(1, ids[:, :4])).abs().max() < 3e-5
    rank = (x > x.gather(1, s.next.long()[:, None])).sum(1) + 1
    ties = (x == x.gather(1, s.next.long()[:, None])).sum(1) - 1
    assert ((s.rank >= rank) & (s.rank <= rank + ties)).all()
    entropy = -(lp.exp() * lp).sum(1)
    assert (s.entropy.double() - entropy).abs().max() < 2e-4  # a difference of numbers below 16


def test_decoding_by_graph_is_decoding_by_calls():
    E = example()
    model = E.Model(vocab=5003, hidden=256, inner=512, seed=3)
    ids, lp = E.decode(model, 17, 12, graph=True)
    ids2, lp2 = E.decode(model, 17, 12, graph=False)
    assert torch.equal(ids, ids2) and torch.equal(lp, lp2)


@pytest.mark.parametrize("M,N,K,gated,f32,passes", [
    (64, 32003, 4096, False, True, 400),     # two tiles to a CTA, 131 MB of weights
    (300, 8200, 4096, True, False, 200),     # gated, 256 tokens a tile
    (700, 14336, 2048, False, False, 200),
    (16, 4096, 14336, False, False, 400),    # a ring over a long K, clusters
    (1, 14336, 4096, True, False, 400),
])
def test_many_passes_give_one_result(M, N, K, gated, f32, passes):
    """Queued without a pause: barriers' phases, rings and workspaces are used over and over while
    copies come late; sums are added in a fixed order, so every pass gives the same bits."""
    Q = qw()
    g = torch.Generator(device="cuda").manual_seed(M)
    cols = N // 2 if gated else N
    A = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    W = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.full((N,), 2.0 ** -12, device="cuda")
    dt = torch.float32 if f32 else torch.bfloat16
    outs = [torch.empty(M, cols, dtype=dt, device="cuda") for _ in range(2)]
    n = Q.qgemm_int8_workspace_size(Q.QW_A_BF16, M, N, K)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    err = Q.new_error_flag()

    def run(C):
        if gated:
            Q.qgemm_int8_gated(Q.QW_A_BF16, A, K, None, W, sw, None, C, cols, M, N // 2, K, ws, n,
                               err)
        else:
            Q.qgemm_int8(Q.QW_A_BF16, A, K, None, W, sw, None,
                         Q.QW_T_F32 if f32 else Q.QW_T_BF16, C, cols, M, N, K, ws, n, err)

    run(outs[0])
    differs = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(passes):
        run(outs[1])
        if i % 50 == 49:
            differs += (outs[1] != outs[0]).sum()
    assert Q.qw_read_error(err) == 0
    assert differs.item() == 0
    # a few columns against 64 bits
    x = A.float()
    amax = x.abs().amax(1, keepdim=True)
    # (tensor / tensor: a number / tensor multiplies by a rounded reciprocal)
    q = torch.round(x * (torch.full_like(amax, 127.0) / amax)).double()
    sa = (amax / torch.full_like(amax, 127.0)).double()[:, 0]
    pick = torch.linspace(0, cols - 1, 40, device="cuda").long()

    def product(rows):
        return (q @ W[rows].double().T) * sa[:, None] * 2.0 ** -12, \
            (q.abs() @ W[rows].double().abs().T) * sa[:, None] * 2.0 ** -12

    R, B = product(pick)
    E = 2.0 ** -22 * R.abs() + 2.0 ** -23 * (K / 16 + 2) * B
    if gated:
        U, BU = product(pick + cols)
        EU = 2.0 ** -22 * U.abs() + 2.0 ** -23 * (K / 16 + 2) * BU
        silu = R / (1 + torch.exp(-R))
        Eg = 1.1 * E + 2.0 ** -20 * silu.abs()
        E = 1.01 * (Eg * (U.abs() + EU) + (silu.abs() + Eg) * EU) + 2.0 ** -22 * (silu * U).abs()
        R = silu * U
    tol = E if f32 else E + 2.0 ** -8 * (R.abs() + E)
    assert ((outs[0][:, pick].double() - R).abs() <= tol).all()
