"""The INT8 products and the log probabilities behind a kernel that lets its dependents start at once and
runs on for longer than a wait inside a kernel may take: their own waits begin after that kernel has ended,
so they finish, without an error and with its writes seen."""
import ctypes
import os
import subprocess

import pytest
import torch

from qwtest import qw

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include <cstdint>
// lets the next kernel start, works for ns nanoseconds (and no more than `most` looks at the clock), and
// only then writes
__global__ void busy(uint64_t ns, uint64_t most, const uint4* src, uint4* dst, int64_t n) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint64_t t0, t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  do {
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    __nanosleep(1000);
  } while (t - t0 < ns && --most > 0);
  for (int64_t i = threadIdx.x; i < n; i += blockDim.x) dst[i] = src[i];
}
extern "C" int run_busy(uint64_t ns, const void* src, void* dst, int64_t bytes, void* stream) {
  busy<<<1, 256, 0, (cudaStream_t)stream>>>(ns, 10000000, (const uint4*)src, (uint4*)dst, bytes / 16);
  return (int)cudaGetLastError();
}
"""
NS = 1_400_000_000  # waits are limited to a second


@pytest.fixture(scope="module")
def busy(tmp_path_factory):
    from moe_qw_repack_gb300.build import ARCH, nvcc
    d = tmp_path_factory.mktemp("busy")
    src, lib = os.path.join(d, "busy.cu"), os.path.join(d, "libbusy.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run([nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-cudart", "shared", "-o", lib, src],
                   check=True)
    fn = ctypes.CDLL(lib).run_busy
    fn.argtypes = [ctypes.c_uint64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]

    def run(src, dst):
        n = src.numel() * src.element_size()
        assert n == dst.numel() * dst.element_size() and n % 16 == 0
        assert fn(NS, src.data_ptr(), dst.data_ptr(), n, torch.cuda.current_stream().cuda_stream) == 0
    return run


@pytest.mark.parametrize("M,codes,gated", [(1, True, False), (1, False, False), (2, False, True),
                                           (8, True, False), (16, True, True), (16, False, False),
                                           (40, True, False), (40, False, True), (300, False, False)])
def test_product_behind_a_long_kernel(busy, M, codes, gated):
    Q = qw()
    g = torch.Generator(device="cuda").manual_seed(M)
    N, K = 520, 2064
    cols = N // 2 if gated else N
    afmt = Q.QW_A_INT8_TOKEN if codes else Q.QW_A_BF16
    if codes:
        x = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
        s = torch.rand(M, generator=g, device="cuda") + 0.5
    else:
        x, s = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16), None
    W = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.full((N,), 2.0 ** -12, device="cuda")
    n = Q.qgemm_int8_workspace_size(afmt, M, N, K)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    err = Q.new_error_flag()

    def run(a):
        C = torch.full((M, cols), 776.0, dtype=torch.bfloat16, device="cuda")
        if gated:
            Q.qgemm_int8_gated(afmt, a, K, s, W, sw, None, C, cols, M, cols, K, ws, n, err)
        else:
            Q.qgemm_int8(afmt, a, K, s, W, sw, None, Q.QW_T_BF16, C, cols, M, N, K, ws, n, err)
        return C

    want = run(x)
    late = torch.zeros_like(x)
    C = torch.full((M, cols), 776.0, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    busy(x, late)
    if gated:
        Q.qgemm_int8_gated(afmt, late, K, s, W, sw, None, C, cols, M, cols, K, ws, n, err)
    else:
        Q.qgemm_int8(afmt, late, K, s, W, sw, None, Q.QW_T_BF16, C, cols, M, N, K, ws, n, err)
    assert Q.qw_read_error(err) == Q.QW_OK
    assert torch.equal(C, want)


def test_log_probabilities_behind_a_long_kernel(busy):
    Q = qw()
    for T, V in ((1, 70000), (64, 5008)):
        x = torch.randn(T, V, device="cuda")
        late = torch.zeros_like(x)
        out = [[torch.zeros(T, device="cuda"), torch.zeros(T, 4, dtype=torch.int32, device="cuda"),
                torch.zeros(T, 4, device="cuda")] for _ in range(2)]
        err = Q.new_error_flag()
        Q.qw_logprobs(Q.QW_T_F32, x, V, T, V, None, 4, None, None, *out[0], err)
        torch.cuda.synchronize()
        busy(x, late)
        Q.qw_logprobs(Q.QW_T_F32, late, V, T, V, None, 4, None, None, *out[1], err)
        assert Q.qw_read_error(err) == Q.QW_OK
        assert all(torch.equal(a, b) for a, b in zip(*out))
