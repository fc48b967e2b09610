"""Inputs that the kernel just before a call is still writing.

The kernels are launched so that they may start while the kernel before them on the stream still runs.  A producer of
lengths, tables or activations that lets its dependents start early (griddepcontrol.launch_dependents ahead of its
stores) is the strictest case: the call behind it has to give the bits that it gives for the same inputs at rest.
"""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from workloads import Dims, V2_LITE
from test_shared_parity import Call, make_shared

PRODUCER = r"""
#include <cuda_runtime.h>
#include <stdint.h>
// Lets the next kernel on the stream start, waits `ns` nanoseconds, then copies n words.
__global__ void produce_kernel(const uint32_t *src, uint32_t *dst, int n, unsigned long long ns) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  unsigned long long t0, t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
  do asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t)); while (t - t0 < ns);
  for (int i = threadIdx.x; i < n; i += blockDim.x) dst[i] = src[i];
}
extern "C" int produce(const void *src, void *dst, int n, unsigned long long ns, void *stream) {
  produce_kernel<<<1, 256, 0, (cudaStream_t)stream>>>((const uint32_t *)src, (uint32_t *)dst, n, ns);
  return (int)cudaGetLastError();
}
"""


@pytest.fixture(scope="module")
def produce(tmp_path_factory):
    """produce(src, dst): dst = src, 50 us later, from a kernel that lets its dependents start at once."""
    d = tmp_path_factory.mktemp("producer")
    src, out = d / "producer.cu", d / "producer.so"
    src.write_text(PRODUCER)
    nvcc = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
    subprocess.run([nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-shared", "-Xcompiler", "-fPIC", "-o", str(out),
                    str(src)], check=True, capture_output=True)
    so = ctypes.CDLL(str(out))
    so.produce.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_ulonglong, ctypes.c_void_p]

    def run(a, b):
        assert a.is_contiguous() and b.is_contiguous() and a.numel() * a.element_size() % 4 == 0 and a.shape == b.shape
        assert so.produce(a.data_ptr(), b.data_ptr(), a.numel() * a.element_size() // 4, 50000,
                          torch.cuda.current_stream().cuda_stream) == 0

    return run


def late(produce, keys, run, result, dev, before):
    """Results of run() for dev[k] at rest, and again where each holds before[k] until a producer writes it."""
    run()
    want = result()
    for k in keys:
        final = dev[k].clone()
        for _ in range(3):
            dev[k].copy_(before[k])
            torch.cuda.synchronize()
            produce(final, dev[k])
            run()
            got = result()
            assert torch.equal(dev[k], final)
            for a, b in zip(got, want):
                assert np.array_equal(a, b), k


@pytest.mark.gpu
@pytest.mark.parametrize("heads,n_q", [(16, 1), (128, 1)])
def test_shared_decode_behind_a_producer_of_lengths_and_groups(lib, produce, heads, n_q):
    inp = make_shared(Dims(**{**V2_LITE, "n_heads": heads}), [(640, [700, 650, 900, 641]), (128, [300, 129])], n_q, 64, seed=51)
    c = Call(lib, inp)
    before = dict(seqlens=torch.full_like(c.dev["seqlens"], 70), prefix_lens=torch.zeros_like(c.dev["prefix_lens"]),
                  group_offsets=torch.tensor([0, 1, 6], dtype=torch.int32, device="cuda"))
    late(produce, sorted(before), c.run, c.result, c.dev, before)
