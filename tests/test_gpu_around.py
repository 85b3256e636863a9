"""The operators around a projection one after the other, as a decoder layer has them: residual and norm to
BF16 and the projection's 8-bit operand, the projection, the requests' adapters onto ranges of its columns,
rotary positions of the query and key heads; on one stream, on two and in a graph.

Each step is checked against 64 bits of what the step before it left, with the bounds of its own tests."""
import numpy as np
import pytest
import torch

import synth
from oracle import qgemm as OQ
from qwtest import qw, repack, u16_view
from test_gpu_lora import check as check_lora, pool, reference as adapters
from test_gpu_norm import bound, check as check_norm, reference as norm
from test_gpu_rope import reference as rotary

pytestmark = pytest.mark.gpu

K, D, HQ, HKV, L, R = 512, 64, 6, 2, 4, 16
NQ, NKV = HQ * D, HKV * D
N = NQ + 2 * NKV
EPS, BASE = 1e-6, 1e6


class Layer:
    """Buffers and weights of a layer; run() is what a serving step launches."""

    def __init__(self, M, q, seed):
        Q = self.Q = qw()
        self.M, self.q = M, q
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.w = (1 + 0.3 * torch.randn(K, generator=g, device="cuda")).to(torch.bfloat16)
        if q == "int8":
            self.W = torch.randint(-127, 128, (N, K), generator=g, device="cuda").to(torch.int8)
            self.sw = torch.rand(N, generator=g, device="cuda") / 1000 + 0.001
            self.codes = torch.zeros((M, K), dtype=torch.int8, device="cuda")
            self.sf = torch.zeros(M, device="cuda")
            n = Q.qgemm_int8_workspace_size(Q.QW_A_INT8_TOKEN, M, N, K)
        else:
            self.p = synth.w8a8_problem(M, N, K, cfg_id=seed)
            self.desc, self.wp, self.sp = repack(Q.QW_W_MXFP8_G32, 1, N, K, self.p["w_canon"],
                                                 self.p["s_canon"])
            self.codes = torch.zeros((M, K), dtype=torch.uint8, device="cuda")
            self.sf = torch.zeros((M, K // 32), dtype=torch.uint8, device="cuda")
            n = Q.qgemm_workspace_size(self.desc, Q.QW_A_MXFP8_G32, M)
        self.ws, self.ws_n = torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda"), n
        self.for_q, self.for_v = pool(L, R, NQ, K, seed + 1), pool(L, R, NKV, K, seed + 2)
        self.freqs = Q.qw_rope_frequencies(Q.QW_ROPE_LINEAR, BASE, D, 2.0)[0].cuda()
        self.x, self.r = (torch.zeros((M, K), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.ids, self.pos = (torch.zeros(M, dtype=torch.int32, device="cuda") for _ in range(2))
        self.y = torch.zeros_like(self.x)
        self.C = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
        self.err = Q.new_error_flag()
        self.fill(seed + 3)

    def fill(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (self.x, self.r):
            t.copy_(torch.randn((self.M, K), generator=g, device="cuda"))
        self.ids.copy_(torch.randint(-1, L, (self.M,), generator=g, device="cuda"))
        self.pos.copy_(torch.randint(0, 1 << 17, (self.M,), generator=g, device="cuda"))

    def run(self, stream=None, after=lambda: None):
        """after() is called behind each step."""
        Q, M = self.Q, self.M
        T = Q.QW_T_BF16
        fmt = Q.QW_A_INT8_TOKEN if self.q == "int8" else Q.QW_A_MXFP8_G32
        Q.qw_rmsnorm(T, self.x, K, T, self.r, K, self.r, K, self.w, 0.0, EPS, M, K, self.y, K, fmt, self.codes,
                     self.sf, self.err, stream)
        after()
        if self.q == "int8":
            Q.qgemm_int8(fmt, self.codes, K, self.sf, self.W, self.sw, None, T, self.C, N, M, N, K, self.ws,
                         self.ws_n, self.err, stream)
        else:
            Q.qgemm_dense(self.desc, self.wp, self.sp, fmt, self.codes, self.sf, None, self.C, M, self.ws,
                          self.ws_n, self.err, stream)
        after()
        for (a, b, scales, ranks), n0, n in ((self.for_q, 0, NQ), (self.for_v, NQ + NKV, NKV)):
            part = self.C[:, n0:]
            Q.qgemm_lora(self.y, K, a, b, scales, ranks, L, R, self.ids, part, N, T, part, N, M, n, K, self.err,
                         stream)
            after()
        Q.qw_rope(T, self.C, N, self.C, N, M, HQ + HKV, D, D, Q.QW_ROPE_HALF, self.pos, self.freqs, 1.0,
                  self.err, stream)
        after()

    def results(self):
        return [t.clone() for t in (self.r, self.y, self.codes, self.sf, self.C)]


@pytest.mark.parametrize("M", [1, 24, 300])
@pytest.mark.parametrize("q", ["int8", "mxfp8"])
def test_step_by_step(M, q):
    s = Layer(M, q, 40 + M)
    x, r = s.x.clone(), s.r.clone()
    steps = []
    s.run(after=lambda: steps.append(s.C.clone()))
    assert s.Q.qw_read_error(s.err) == 0
    h, y = norm(x, r, s.w, eps=EPS)
    check_norm(dict(h=s.r, y=s.y, codes=s.codes, sf=s.sf), h, y, q, bound(K))
    after = steps[1]
    if q == "int8":
        # an exact sum, made FP32, times two scales: three roundings and the result's
        want = (s.codes.double() @ s.W.double().t()) * s.sf.double()[:, None] * s.sw.double()
        assert bool(((after.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -22) * want.abs()).all())
    else:
        want, size = OQ.gemm_w8a8(s.codes.cpu().numpy(), s.sf.cpu().numpy(), s.p["w_canon"][0],
                                  s.p["s_canon"][0])
        ok, ratio, frob = OQ.check_bf16_result(u16_view(after.view(torch.int16)), want, size)
        assert ok, (ratio, frob)
    for (a, b, scales, ranks), n0, n, i in ((s.for_q, 0, NQ, 2), (s.for_v, NQ + NKV, NKV, 3)):
        before, after = steps[i - 1], steps[i]
        base = before[:, n0:n0 + n]
        none = (s.ids == -1) | (ranks[s.ids.clamp(min=0).long()] == 0)
        check_lora(after[:, n0:n0 + n], adapters(s.y, a, b, scales, ranks, s.ids, base), "bf16", none, base)
        others = [j for j in range(N) if not n0 <= j < n0 + n]
        assert torch.equal(after[:, others], before[:, others])
    before, after = steps[3], steps[4]
    heads = NQ + NKV
    want, tol = rotary(before[:, :heads].double().cpu().numpy(), HQ + HKV, D, D, "half",
                       s.pos.cpu().numpy().astype(np.int64), s.freqs.cpu().numpy(), 1.0)
    got = after[:, :heads].double().cpu().numpy()
    assert (np.abs(got - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol) + 2.0 ** -133).all()
    assert torch.equal(after[:, heads:], before[:, heads:])


@pytest.mark.parametrize("M", [1, 24, 300])
@pytest.mark.parametrize("q", ["int8", "mxfp8"])
def test_in_a_graph(M, q):
    """Captured once and replayed with other inputs: the bits of a plain run."""
    s = Layer(M, q, 50 + M)
    s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
        s.run()  # (the second on the residual that the first left)
    for seed in (1, 2):
        s.fill(seed)
        graph.replay()
        got = s.results()
        s.fill(seed)
        s.run()
        s.run()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, s.results()))
    assert s.Q.qw_read_error(s.err) == 0


def test_two_streams_at_once():
    """Layers of their own on two streams, beside each other, and many times over."""
    layers = [Layer(300, "int8", 60), Layer(24, "mxfp8", 61)]
    want = []
    for s in layers:
        s.run()
        want.append(s.results())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for turn in range(5):
        for s, seed in zip(layers, (63, 64)):
            s.fill(seed)
        torch.cuda.synchronize()
        for s, st in zip(layers, streams):
            s.run(st)
        torch.cuda.synchronize()
        for s, w in zip(layers, want):
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(s.results(), w))
            assert s.Q.qw_read_error(s.err) == 0


def test_no_tokens():
    """Calls of no rows leave everything as it is."""
    Q = qw()
    T = Q.QW_T_BF16
    buf = torch.full((64,), 7.0, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    freqs = torch.ones(8, dtype=torch.float64, device="cuda")
    err = Q.new_error_flag()
    Q.qw_rmsnorm(T, buf, 16, 0, None, 16, None, 16, buf, 0.0, EPS, 0, 16, buf, 16, Q.QW_A_BF16, None, None, err)
    Q.qgemm_lora(buf, 16, buf, buf, None, None, 1, 8, ids, None, 16, T, buf, 16, 0, 16, 16, err)
    Q.qw_rope(T, buf, 16, buf, 16, 0, 1, 16, 16, Q.QW_ROPE_HALF, ids, freqs, 1.0, err)
    assert Q.qw_read_error(err) == 0 and bool((buf == 7).all())
