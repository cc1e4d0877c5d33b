"""mla_window_decode right behind the kernel that writes its lengths: the call
starts while that kernel still runs, and must not have looked at cache_seqlens
or new_lens before it ends.  The writer here lets its dependents start at once
and writes 200 us later; the results have to be the bits of a call made after a
synchronisation on the same lengths."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from mla_decode_attention_gb300 import binding, build, workloads
from tests.test_gpu_append import DEV, library  # noqa: F401

pytestmark = pytest.mark.gpu

BF16, FP8_656, FP8_528 = binding.MLA_KV_BF16, binding.MLA_KV_FP8_656, binding.MLA_KV_FP8_528
SCALE = workloads.SOFTMAX_SCALE
KINDS = [(BF16, 128, 100), (BF16, 128, 1500), (BF16, 64, 130), (BF16, 16, 300), (FP8_656, 64, 500), (FP8_656, 128, 100), (FP8_528, 32, 200)]
SOURCE = r"""
#include <cstdint>
#include <cuda_runtime.h>
__global__ void late(int32_t* to, const int32_t* from, int n, int us) {
  asm volatile("griddepcontrol.launch_dependents;");
  uint64_t t0, t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
  for (int i = 0; i < 1000000; ++i) {
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    if (t - t0 >= 1000ull * us) break;
  }
  for (int i = threadIdx.x; i < n; i += blockDim.x) to[i] = from[i];
}
extern "C" int late_write(int32_t* to, const int32_t* from, int n, int us, cudaStream_t stream) {
  late<<<1, 32, 0, stream>>>(to, from, n, us);
  return static_cast<int>(cudaGetLastError());
}
"""


@pytest.fixture(scope="module")
def late_write(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    d = tmp_path_factory.mktemp("late")
    (d / "late.cu").write_text(SOURCE)
    lib = str(d / "late.so")
    subprocess.run([nvcc, *build.ARCH, "-shared", "-Xcompiler", "-fPIC", str(d / "late.cu"), "-o", lib], check=True, env=dict(os.environ))
    fn = ctypes.CDLL(lib).late_write
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]

    def write(to, values):
        assert fn(to.data_ptr(), values.data_ptr(), to.numel(), 200, torch.cuda.current_stream().cuda_stream) == 0
    return write


class Call:
    """Requests whose tables cover `most` tokens, every cache slot finite."""

    def __init__(self, fmt, h, window, b, s, most, seed=1):
        g = torch.Generator().manual_seed(seed)
        slots, d = (most + 63) // 64, 512 if fmt == FP8_528 else 576
        x = torch.randn(b * slots, 64, d, generator=g)
        cache = x.to(torch.bfloat16) if fmt == BF16 else (workloads.quantize_fp8_tokens(x) if fmt == FP8_656 else workloads.quantize_fp8_v41_tokens(x))
        self.fmt, self.window = fmt, window
        self.cache, self.table = cache.to(DEV), torch.randperm(b * slots, generator=g).view(b, slots).int().to(DEV)
        self.q = torch.randn(b, s, h, d, generator=g).to(torch.bfloat16).to(DEV)
        self.lens = torch.zeros(b, dtype=torch.int32, device=DEV)
        self.new = torch.full((b,), s, dtype=torch.int32, device=DEV)
        self.buf = binding.WindowBuffers(b, s, h, window, 4, DEV)

    def __call__(self, out=None, lse=None, ragged=False):
        binding.mla_window_decode(self.q, self.cache, self.fmt, self.table, self.lens, SCALE, self.window, 4, self.buf.num_sm_parts,
                                  self.buf.workspace, self.buf.out if out is None else out, self.buf.lse if lse is None else lse,
                                  self.buf.err, new_lens=self.new if ragged else None)


@pytest.mark.parametrize("fmt,h,window", KINDS)
@pytest.mark.parametrize("ragged", [False, True])
def test_lengths_written_by_the_kernel_before(late_write, fmt, h, window, ragged):
    """Old and new lengths (and counts of new tokens) on either side of page and
    tile borders, among them requests that begin or end empty."""
    after = [0, 1, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700, 1000, 1023, 1024, 1025, 64, 128, 2000, 1900]
    before = [5, 0, 62, 63, 64, 126, 127, 128, 254, 255, 256, 699, 999, 1022, 1023, 1024, 1900, 0, 64, 2000]
    b, s = len(after), 3
    c = Call(fmt, h, window, b, s, 2000)
    lens = [torch.tensor(v, dtype=torch.int32, device=DEV) for v in (before, after)]
    fresh = [torch.tensor([(i + k) % (s + 1) for i in range(b)], dtype=torch.int32, device=DEV) for k in (0, 2)]
    c.lens.copy_(lens[1]); c.new.copy_(fresh[1])
    torch.cuda.synchronize()
    c(ragged=ragged)
    torch.cuda.synchronize()
    want = c.buf.out.clone(), c.buf.lse.clone()
    written = [(c.lens, lens)] + ([(c.new, fresh)] if ragged else [])
    for to, values in written * 4:
        c.lens.copy_(lens[1]); c.new.copy_(fresh[1])
        to.copy_(values[0])
        c.buf.out.fill_(9.0); c.buf.lse.fill_(9.0)
        torch.cuda.synchronize()
        late_write(to, values[1])
        c(ragged=ragged)
        torch.cuda.synchronize()
        assert torch.equal(c.buf.lse, want[1]) and torch.equal(c.buf.out, want[0])
    assert int(c.buf.err.item()) == 0


@pytest.mark.parametrize("fmt,h,window", KINDS)
def test_captured_lengths_that_grow(fmt, h, window):
    """lens.add_(1) directly before every call, captured and replayed without a
    synchronisation; every step's output is that of a call of its own."""
    start, steps, replays = [0, 60, 61, 124, 126, 250, 700, 1020], 4, 5
    b = len(start)
    c = Call(fmt, h, window, b, 1, max(start) + steps * replays)
    outs = torch.zeros(steps, *c.buf.out.shape, dtype=torch.bfloat16, device=DEV)
    lses = torch.zeros(steps, *c.buf.lse.shape, device=DEV)
    c()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(steps):
            c.lens.add_(1)
            c(outs[i], lses[i])
    c.lens.copy_(torch.tensor(start, dtype=torch.int32))
    torch.cuda.synchronize()
    seen = []
    for _ in range(replays):
        graph.replay()
        seen.append((outs.clone(), lses.clone()))
    torch.cuda.synchronize()
    c.lens.copy_(torch.tensor(start, dtype=torch.int32))
    for o, l in seen:
        for i in range(steps):
            c.lens.add_(1)
            torch.cuda.synchronize()
            c()
            torch.cuda.synchronize()
            assert torch.equal(l[i], c.buf.lse) and torch.equal(o[i], c.buf.out)
    assert int(c.buf.err.item()) == 0
