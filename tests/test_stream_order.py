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

from helpers import device_pool, dims_of
from test_shared_parity import Call, make_shared
from workloads import DecodeCase, Dims, V2_LITE, make_decode_step_inputs

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
    """produce(src, dst): dst = src, 50 us (or `ns`) later, from a kernel that lets its dependents start at once."""
    d = tmp_path_factory.mktemp("producer")
    src, out = d / "producer.cu", d / "producer.so"
    src.write_text(PRODUCER)
    nvcc = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
    subprocess.run([nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-shared", "-Xcompiler", "-fPIC", "-o", str(out),
                    str(src)], check=True, capture_output=True)
    so = ctypes.CDLL(str(out))
    so.produce.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_ulonglong, ctypes.c_void_p]

    def run(a, b, ns=50000):
        assert a.is_contiguous() and b.is_contiguous() and a.numel() * a.element_size() % 4 == 0 and a.shape == b.shape
        assert so.produce(a.data_ptr(), b.data_ptr(), a.numel() * a.element_size() // 4, ns,
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
            assert torch.equal(dev[k].view(torch.uint8), final.view(torch.uint8))
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


class Step:
    """One decode step's inputs on the device, and a call of each entry point that takes lengths or positions."""

    def __init__(self, mla, n_q):
        d = Dims(**{**V2_LITE, "d_model": 256})
        case = DecodeCase("late", d, 7, n_q, ("list", (63, 64, 165, 511, 1500, 700, 901)), 64, True, 77)
        self.inp = inp = make_decode_step_inputs(case)
        self.mla, self.d, self.n_q, self.B, self.H = mla, d, n_q, 7, d.n_heads
        self.dims = dims_of(mla, d, 64, 1)
        self.dev = {k: inp[k].cuda() for k in ("q_nope", "q_pe", "block_table", "seqlens", "w_uk", "w_uv", "h_new", "w_dkv", "w_kr",
                                               "gamma", "seq_idx", "pos")}
        # The pool's unused rows hold NaN; any finite rows will do here.
        self.pool0, _, _ = device_pool(mla, d, 64, torch.nan_to_num(inp["pool"].float()).to(torch.bfloat16), 1)
        self.pool = self.pool0.clone()
        self.S, B, H = int(inp["seqlens"].max()), 7, d.n_heads
        bf = lambda *shape: torch.empty(*shape, dtype=torch.bfloat16, device="cuda")   # noqa: E731
        self.out, self.o_lat, self.q_abs = bf(B, n_q, H, 128), bf(B, n_q, H, 512), bf(B, n_q, H, 576)
        self.lse = torch.empty(B, n_q, H, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.dev["topk"] = torch.tensor(np.random.default_rng(1).integers(0, 60, (B, n_q, 100)), dtype=torch.int32).cuda()
        size = max(mla.mla_decode_step_workspace_size(self.dims, B, n_q, self.S),
                   mla.mla_decode_sparse_workspace_size(self.dims, B, n_q, 100))
        self.ws = mla.alloc_workspace(size)
        self.append_ws = mla.alloc_workspace(mla.mla_append_workspace_size(self.dims, B * n_q))

    def call(self, entry):
        m, v, i = self.mla, self.dev, self.inp
        pool = (self.pool, self.pool, v["block_table"], i["max_blocks_per_seq"], i["num_blocks"])
        q, cache = (v["q_nope"], v["q_pe"]), (*pool, v["seqlens"], self.S)
        if entry == "decode":
            m.mla_decode(self.dims, *q, *cache, v["w_uk"], v["w_uv"], self.out, self.lse, self.ws, self.status)
        elif entry == "latent":
            m.mla_decode_latent(self.dims, *q, *cache, v["w_uk"], self.o_lat, self.lse, self.ws, self.status)
        elif entry == "partial":
            m.mla_decode_partial(self.dims, *q, *cache, 64, 640, v["w_uk"], self.o_lat, self.lse, self.ws, self.status)
        elif entry == "attention":
            m.mla_decode_attention(self.dims, self.q_abs, *cache, self.ws, self.status)
            m.mla_decode_combine(self.dims, self.B, self.n_q, v["seqlens"], self.S, v["w_uv"], self.out, self.lse, self.ws)
        elif entry == "sparse":
            m.mla_decode_sparse(self.dims, *q, *cache, v["topk"], v["w_uk"], v["w_uv"], self.out, self.lse, self.ws, self.status)
        elif entry == "step":
            m.mla_decode_step(self.dims, v["h_new"].view(self.B, self.n_q, -1), v["w_dkv"], v["w_kr"], v["gamma"], *q, *cache,
                              v["w_uk"], v["w_uv"], self.out, self.lse, self.ws, self.status)
        elif entry == "append":
            m.mla_append_latent(self.dims, v["h_new"], v["w_dkv"], v["w_kr"], v["gamma"], v["seq_idx"], v["pos"], self.pool, self.pool,
                                v["block_table"], self.B, i["max_blocks_per_seq"], i["num_blocks"], self.status,
                                workspace=self.append_ws)
        else:
            m.mla_absorb_q(self.dims, *q, v["w_uk"], v["seqlens"], self.q_abs)

    def reset(self):
        self.pool.copy_(self.pool0)
        for t in (self.out, self.o_lat, self.lse, self.q_abs):
            t.zero_()
        if self.entry == "attention":   # (its queries are an input)
            self.q_abs.copy_(self.keep_q)

    def check(self, entry, produce, before):
        self.entry = entry
        self.call("absorb")
        self.keep_q = self.q_abs.clone()

        def run():
            self.call(entry)

        def result():
            torch.cuda.synchronize()
            assert int(self.status.item()) == 0
            got = [t.view(torch.int16).cpu().numpy() for t in (self.out, self.o_lat, self.q_abs, self.pool)]
            got.append(self.lse.view(torch.int32).cpu().numpy())
            self.reset()
            return got

        self.reset()
        late(produce, sorted(before), run, result, self.dev, before)


@pytest.mark.gpu
@pytest.mark.parametrize("n_q", [1, 3])
@pytest.mark.parametrize("entry", ["decode", "latent", "partial", "attention", "sparse", "step", "append", "absorb"])
def test_entry_points_behind_a_producer_of_lengths_tables_and_positions(lib, produce, entry, n_q):
    s = Step(lib, n_q)
    if entry == "append":
        before = dict(seq_idx=torch.zeros_like(s.dev["seq_idx"]), pos=torch.zeros_like(s.dev["pos"]))
    else:
        before = dict(seqlens=torch.full_like(s.dev["seqlens"], 40))
        if entry != "absorb":
            before["block_table"] = torch.zeros_like(s.dev["block_table"])
    s.check(entry, produce, before)


@pytest.mark.gpu
@pytest.mark.parametrize("n_q", [1, 3])
@pytest.mark.parametrize("entry", ["decode", "partial", "sparse", "step", "append", "absorb"])
def test_entry_points_behind_a_producer_of_queries_and_hidden_states(lib, produce, entry, n_q):
    s = Step(lib, n_q)
    names = {"append": ["h_new"], "step": ["h_new", "q_nope", "q_pe"]}.get(entry, ["q_nope", "q_pe"])
    s.check(entry, produce, {k: torch.flip(s.dev[k], [-1]) for k in names})


@pytest.mark.gpu
def test_shared_decode_behind_a_producer_of_queries_tables_and_keys(lib, produce):
    inp = make_shared(Dims(**V2_LITE), [(640, [700, 650, 900, 641]), (128, [300, 129])], 1, 64, seed=52)
    c = Call(lib, inp)
    c.dev["pool"] = c.c_kv
    before = {k: torch.flip(c.dev[k], [-1]) for k in ("q_nope", "q_pe")}
    before.update(block_table=torch.zeros_like(c.dev["block_table"]), pool=torch.zeros_like(c.c_kv))
    late(produce, sorted(before), c.run, c.result, c.dev, before)


@pytest.mark.gpu
def test_a_decode_that_takes_what_the_call_ahead_wrote(lib):
    """The output of one call as the hidden states of the append behind it, and these rows decoded by the next: the bits of
    the same calls with the device at rest between them."""
    s = Step(lib, 1)
    dims = s.dims
    dims.d_model = 16 * 128   # a token's heads side by side
    g = torch.Generator(device="cuda").manual_seed(5)
    s.dev["w_dkv"] = (torch.randn(2048, 512, generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    s.dev["w_kr"] = (torch.randn(2048, 64, generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    s.dev["h_new"] = s.out.view(s.B, 2048)
    s.append_ws = lib.alloc_workspace(lib.mla_append_workspace_size(dims, s.B))
    s.entry = "decode"

    def chain(pause):
        s.reset()
        for entry in ("decode", "append", "decode", "append", "decode"):
            s.call(entry)
            if pause:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert int(s.status.item()) == 0
        return s.out.view(torch.int16).clone(), s.pool.view(torch.int16).clone()

    want = chain(True)
    for _ in range(20):
        for a, b in zip(chain(False), want):
            assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("entry", ["append", "step", "decode", "attention", "shared"])
def test_a_producer_that_takes_longer_than_a_bounded_wait(lib, produce, entry):
    """The waits inside the kernels give up after 2 s; what is ahead on the stream may take longer."""
    if entry == "shared":
        inp = make_shared(Dims(**V2_LITE), [(640, [700, 650, 900, 641]), (128, [300, 129])], 1, 64, seed=53)
        c = Call(lib, inp)
        run, lens = c.run, c.dev["seqlens"]

        def result():
            return c.result()
    else:
        s = Step(lib, 1)
        s.entry = entry
        s.call("absorb")
        s.keep_q = s.q_abs.clone()
        s.reset()
        lens = s.dev["h_new"] if entry in ("append", "step") else s.dev["seqlens"]

        def run():
            s.call(entry)

        def result():
            torch.cuda.synchronize()
            got = s.out.float().cpu().numpy(), s.pool.view(torch.int16).cpu().numpy(), int(s.status.item())
            s.reset()
            return got

    run()
    want = result()
    produce(lens.clone(), lens, 2300000000)
    run()
    got = result()
    assert got[2] == want[2] == 0
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
