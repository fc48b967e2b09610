"""The shared-prefix operators as a serving loop uses them: mla_plan_step, mla_append_latent, mla_decode_shared and
mla_release_blocks, eagerly and as one replayed graph per step, against the fp64 oracle over the cache that the loop
has built (whole numbers: against the model of tests/test_step_plan.py)."""
import numpy as np
import pytest
import torch

import oracle
from workloads import Dims, V2_LITE
from helpers import check_close, dims_of
from test_step_plan import model_plan, model_release

pytestmark = pytest.mark.gpu
BS = 64
D = Dims(**{**V2_LITE, "d_model": 256})


class Loop:
    """Two prompts of 2 and 3 blocks; requests 0-3 behind the first, 4-6 behind the second, 7 by itself."""

    def __init__(self, mla):
        self.mla = mla
        self.dims = dims_of(mla, D, BS, 1)
        g = torch.Generator().manual_seed(7)
        rnd = lambda *shape, scale=1.0: (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16).cuda()   # noqa: E731
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
        self.i32, self.rnd = i32, rnd
        self.B, self.mb, self.num_blocks = 8, 8, 40
        self.pool = torch.zeros(self.num_blocks * BS, D.latent_width, dtype=torch.bfloat16, device="cuda")
        self.w_dkv, self.w_kr = rnd(D.d_model, D.d_c, scale=D.d_model ** -0.5), rnd(D.d_model, D.d_rope, scale=D.d_model ** -0.5)
        self.gamma = torch.ones(D.d_c, dtype=torch.bfloat16, device="cuda")
        self.w_uk, self.w_uv = rnd(D.n_heads, D.d_c, D.d_nope, scale=D.d_c ** -0.5), rnd(D.n_heads, D.d_c, D.d_v, scale=D.d_c ** -0.5)
        self.offsets, self.prefixes = i32([0, 4, 7, 8]), i32([2 * BS, 3 * BS, 0])
        self.prefix_table = i32([[0, 1, -1], [2, 3, 4], [-1, -1, -1]])
        self.free_list = i32(np.random.default_rng(1).permutation(np.arange(5, self.num_blocks)).tolist() + [-1] * 5)
        self.free_count = i32([self.num_blocks - 5])
        self.table = i32([[-1] * self.mb] * self.B)
        self.lens = i32([2 * BS] * 4 + [3 * BS] * 3 + [0])
        self.status = i32([0])
        # The prompts themselves: appended once, through a table of their own.
        for row, p in ((0, 2 * BS), (1, 3 * BS)):
            self.append(rnd(p, D.d_model), i32([row] * p), i32(list(range(p))), self.prefix_table, 3)

    def append(self, h, seq_idx, pos, table, mb):
        ws = self.mla.mla_append_workspace_size(self.dims, h.shape[0])
        self.mla.mla_append_latent(self.dims, h, self.w_dkv, self.w_kr, self.gamma, seq_idx, pos, self.pool, self.pool, table,
                                   table.shape[0], mb, self.num_blocks, self.status,
                                   workspace=self.mla.alloc_workspace(ws) if ws else None)

    def plan(self, new, T):
        """Buffers of a step of T tokens; the call updates lengths, table and free count in place."""
        b = dict(new=self.i32(new), cu=self.i32([0] * (self.B + 1)), seq_idx=self.i32([-1] * T), pos=self.i32([-1] * T),
                 slots=torch.full((T,), -1, dtype=torch.int64, device="cuda"))
        self.call_plan(b)
        return b

    def call_plan(self, b):
        self.mla.mla_plan_step(self.dims, self.lens, b["new"], self.offsets, self.prefixes, self.prefix_table, self.free_list,
                               self.free_count, self.table, self.num_blocks, self.lens, b["cu"], b["seq_idx"], b["pos"],
                               b["slots"], self.free_count, self.status)

    def decode_buffers(self):
        B, H = self.B, D.n_heads
        return dict(q_nope=self.rnd(B, 1, H, D.d_nope), q_pe=self.rnd(B, 1, H, D.d_rope),
                    out=torch.empty(B, 1, H, D.d_v, dtype=torch.bfloat16, device="cuda"),
                    lse=torch.empty(B, 1, H, dtype=torch.float32, device="cuda"),
                    ws=self.mla.alloc_workspace(self.mla.mla_decode_shared_workspace_size(self.dims, B, 1, self.mb * BS, 3)))

    def call_decode(self, d):
        self.mla.mla_decode_shared(self.dims, d["q_nope"], d["q_pe"], self.pool, None, self.table, self.mb, self.num_blocks,
                                   self.lens, self.mb * BS, self.offsets, self.prefixes, self.w_uk, self.w_uv, d["out"],
                                   d["lse"], d["ws"], self.status)

    def check_decode(self, d):
        rows = torch.empty_like(self.pool)
        self.mla.mla_cache_unpack(self.dims, self.pool, rows)
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        picks = [(b, 0, s) for b in range(self.B) for s in (0, 5, D.n_heads - 1)]
        ref, ref_lse = oracle.decode(D, d["q_nope"].cpu(), d["q_pe"].cpu(), rows.cpu(), self.table.cpu(), BS, self.lens.cpu(),
                                     self.w_uk.cpu(), self.w_uv.cpu(), picks=picks)
        idx = tuple(np.array(picks).T)
        check_close(d["out"].float().cpu().numpy()[idx], ref[idx], "bf16", "step")
        assert np.max(np.abs(d["lse"].cpu().numpy()[idx] - ref_lse[idx])) <= 3e-2

    def state(self):
        return (self.lens.cpu().numpy(), self.table.cpu().numpy(), int(self.free_count.item()))


def test_serving_loop(lib):
    """Requests join behind their prompts with texts of their own, decode, some finish and their blocks go to new ones."""
    L = Loop(lib)
    fl, pre, off, pt = (x.cpu().numpy() for x in (L.free_list, L.prefixes, L.offsets, L.prefix_table))
    new = [5, 64, 0, 130, 1, 70, 63, 90]
    lens, table, free = L.state()
    b = L.plan(new, sum(new))
    m_table, m_lens, m_cu, m_seq, m_pos, m_slots, m_free, err = model_plan(BS, lens, new, off, pre, pt, fl, free, table, 40, sum(new))
    lens, table, free = L.state()
    assert not err and free == m_free and lens.tolist() == m_lens and np.array_equal(table, m_table)
    assert np.array_equal(b["slots"].cpu().numpy(), m_slots) and np.array_equal(b["seq_idx"].cpu().numpy(), m_seq)
    h = L.rnd(sum(new), D.d_model)
    L.append(h, b["seq_idx"], b["pos"], L.table, L.mb)
    rows = torch.empty_like(L.pool)
    lib.mla_cache_unpack(L.dims, L.pool, rows)
    c_ref, k_ref = oracle.append_latent(h.cpu(), L.w_dkv.cpu(), L.w_kr.cpu(), L.gamma.cpu(), b["pos"].cpu(), D.rms_eps, D.rope_base)
    got = rows[b["slots"]].float().cpu().numpy()   # the slot map names the rows that the append wrote
    check_close(got, np.concatenate([c_ref, k_ref], 1), "bf16", "appended rows")
    d = L.decode_buffers()
    for step in range(3):
        b = L.plan([1] * 8, 8)
        L.append(L.rnd(8, D.d_model), b["seq_idx"], b["pos"], L.table, L.mb)
        L.call_decode(d)
        L.check_decode(d)
    # Requests 1 and 5 finish; their blocks are the next to be taken.
    done = [0, 1, 0, 0, 0, 1, 0, 0]
    lens, table, free = L.state()
    w_fl, w_lens, w_free, err = model_release(BS, done, lens, off, pre, table, 40, L.free_list.cpu().numpy(), free)
    lib.mla_release_blocks(L.dims, L.i32(done), L.lens, L.offsets, L.prefixes, L.table, 40, L.free_list, L.free_count, L.lens,
                           L.free_count, L.status)
    lens, table, free = L.state()
    assert not err and free == w_free and lens.tolist() == w_lens and np.array_equal(L.free_list.cpu().numpy(), w_fl)
    L.lens[1], L.lens[5] = 2 * BS, 3 * BS          # new requests in their places, behind the same prompts
    new = [1, 100, 1, 1, 1, 3, 1, 1]
    b = L.plan(new, sum(new))
    L.append(L.rnd(sum(new), D.d_model), b["seq_idx"], b["pos"], L.table, L.mb)
    own = set()
    for r in range(8):                             # no block is in two places but the prompts'
        p = int(pre[[0, 0, 0, 0, 1, 1, 1, 2][r]]) // BS
        ids = L.table[r].cpu().tolist()[p:-(-int(L.lens[r]) // BS)]
        assert not own & set(ids) and not set(ids) & {0, 1, 2, 3, 4}
        own |= set(ids)
    L.call_decode(d)
    L.check_decode(d)


def test_serving_step_as_one_graph(lib):
    """Plan, append and decode captured together; each replay is the next step."""
    L = Loop(lib)
    new = [5, 64, 3, 130, 1, 70, 63, 90]
    b = L.plan(new, sum(new))
    L.append(L.rnd(sum(new), D.d_model), b["seq_idx"], b["pos"], L.table, L.mb)
    b, d, h = L.plan([1] * 8, 8), L.decode_buffers(), L.rnd(8, D.d_model)
    nws = lib.mla_append_workspace_size(L.dims, 8)
    ws = lib.alloc_workspace(nws) if nws else None

    def step():
        L.call_plan(b)
        lib.mla_append_latent(L.dims, h, L.w_dkv, L.w_kr, L.gamma, b["seq_idx"], b["pos"], L.pool, L.pool, L.table, 8, L.mb,
                              L.num_blocks, L.status, workspace=ws)
        L.call_decode(d)

    L.append(h, b["seq_idx"], b["pos"], L.table, L.mb)   # the tokens that the first plan made room for
    step()                                               # (also sets the kernels up before the capture)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    before = L.state()[0]
    for k in range(1, 4):
        h.copy_(L.rnd(8, D.d_model))
        d["q_nope"].copy_(L.rnd(*d["q_nope"].shape))
        g.replay()
        torch.cuda.synchronize()
        assert (L.state()[0] == before + k).all()
        L.check_decode(d)


def test_append_from_odd_addresses(lib):
    """Hidden states and weights behind addresses that no 16-byte copy can start at: the same rows but for fp32 sums of 256
    products in another order (256 * 2^-24 = 2^-16 of the sum of magnitudes, 2^-12 of a row's norm is ample) and so a bf16
    rounding that may fall the other way (a whole step, 2^-7 of the value at most)."""
    a, b = Loop(lib), Loop(lib)
    for k in ("w_dkv", "w_kr"):
        w = getattr(b, k)
        flat = torch.empty(w.numel() + 1, dtype=w.dtype, device="cuda")
        flat[1:].copy_(w.flatten())
        setattr(b, k, flat[1:].view(w.shape))
    g = torch.Generator().manual_seed(3)
    h = torch.randn(5, D.d_model, generator=g).to(torch.bfloat16).cuda()
    odd = torch.empty(h.numel() + 1, dtype=h.dtype, device="cuda")
    odd[1:].copy_(h.flatten())
    for loop, x in ((a, h), (b, odd[1:].view(h.shape))):
        loop.append(x, loop.i32([0, 0, 1, 1, 1]), loop.i32([0, 70, 3, 64, 191]), loop.prefix_table, 3)
    torch.cuda.synchronize()
    assert int(a.status.item()) == int(b.status.item()) == 0
    want, got = a.pool.float(), b.pool.float()
    assert ((got - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -12 * want.norm(dim=1, keepdim=True)).all()
    assert want.abs().sum() > 0
