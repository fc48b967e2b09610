"""GPU parity of mla_decode_shared (groups of sequences that share their first tokens) against the fp64 oracle.

The result is that of an ordinary decode of every sequence through its own block table row, so the oracle's decode is
the reference.  Bars: those of the other decode tests (tests/helpers.py): queries, P, partial outputs and the merged
o_lat are each rounded to bf16 once (2^-8 relative at most each, fp32 between), four independent roundings of random
sign: 2 * 2^-8 / sqrt(3) = 4.5e-3 of the output's norm, below the 1e-2 bar; fp32 paths keep 1e-4.
(Partials are in fp32 by now and the merged row meets W_UV in two bf16 parts: queries, P and the output remain, some 2.5e-3.
The bar counts more than is rounded; tests/test_shared_rows.py has bounds of every row by its own arithmetic.)
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from workloads import Dims, V2_LITE, V3
from helpers import check_close, device_pool, dims_of, tiled_ok

SMALL = dict(n_heads=8, d_c=64, d_rope=16, d_nope=32, d_v=32, d_model=256, dtype="f32")


def make_shared(dims, groups, n_q, bs, seed=0, spread=1.0):
    """groups: list of (prefix tokens, [total tokens of each sequence]).  Whole blocks among the prefix tokens are the
    same blocks for the group; everything else is each sequence's own.  Unused pool rows hold NaN."""
    g = torch.Generator().manual_seed(seed)
    lens = [n for _, seqs in groups for n in seqs]
    B = len(lens)
    mb = max(-(-n // bs) for n in lens)
    need = sum(p // bs for p, _ in groups) + sum(-(-n // bs) for n in lens) + 2
    ids = torch.randperm(need, generator=g).tolist()
    table = torch.full((B, mb), -1, dtype=torch.int32)
    dt = dims.torch_dtype
    pool = torch.full((need * bs, dims.latent_width), float("nan"), dtype=dt)
    b, offs = 0, [0]
    for p, seqs in groups:
        whole = min(p, max(seqs, default=0)) // bs
        shared = [ids.pop() for _ in range(whole)]
        for blk in shared:
            pool[blk * bs:(blk + 1) * bs] = (torch.randn(bs, dims.latent_width, generator=g) * spread).to(dt)
        for n in seqs:
            for i in range(-(-n // bs)):
                if i < whole and (i + 1) * bs <= n:
                    table[b, i] = shared[i]
                else:
                    blk = table[b, i] = ids.pop()
                    k = min(n - i * bs, bs)
                    pool[blk * bs:blk * bs + k] = (torch.randn(k, dims.latent_width, generator=g) * spread).to(dt)
            b += 1
        offs.append(b)

    def rnd(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g) * scale).to(dt)

    H = dims.n_heads
    return dict(dims=dims, n_q=n_q, block_size=bs, seqlens=torch.tensor(lens, dtype=torch.int32), block_table=table,
                num_blocks=need, max_blocks_per_seq=mb, pool=pool, group_offsets=torch.tensor(offs, dtype=torch.int32),
                prefix_lens=torch.tensor([p for p, _ in groups], dtype=torch.int32),
                q_nope=rnd(B, n_q, H, dims.d_nope), q_pe=rnd(B, n_q, H, dims.d_rope),
                w_uk=rnd(H, dims.d_c, dims.d_nope, scale=dims.d_c ** -0.5),
                w_uv=rnd(H, dims.d_c, dims.d_v, scale=dims.d_c ** -0.5))


class Call:
    """One prepared device call (buffers kept, so that it can be repeated or captured)."""

    def __init__(self, mla, inp, layout=None, latent=False, max_seqlen=None, groups=True):
        d, bs = inp["dims"], inp["block_size"]
        layout = (1 if tiled_ok(d, bs) else 0) if layout is None else layout
        self.mla, self.dims = mla, dims_of(mla, d, bs, layout)
        self.dev = {k: v.cuda() for k, v in inp.items() if isinstance(v, torch.Tensor) and k != "pool"}
        self.c_kv, self.k_pe, self.keep = device_pool(mla, d, bs, inp["pool"], layout)
        B, n_q, H = inp["q_nope"].shape[:3]
        self.inp, self.latent = inp, latent
        self.max_seqlen = max_seqlen or int(inp["seqlens"].max())
        self.out = torch.full((B, n_q, H, d.d_c if latent else d.d_v), float("nan"), dtype=d.torch_dtype, device="cuda")
        self.lse = torch.full((B, n_q, H), float("nan"), dtype=torch.float32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.groups = groups
        G = inp["prefix_lens"].numel() if groups else 0
        self.ws = mla.alloc_workspace(mla.mla_decode_shared_workspace_size(self.dims, B, n_q, self.max_seqlen, G))
        self.ws.fill_(0xFF)   # no reliance on what the workspace holds
        torch.cuda.synchronize()

    def run(self, stream=None):
        v, i = self.dev, self.inp
        self.mla.mla_decode_shared(self.dims, v["q_nope"], v["q_pe"], self.c_kv, self.k_pe, v["block_table"],
                                   i["max_blocks_per_seq"], i["num_blocks"], v["seqlens"], self.max_seqlen,
                                   v["group_offsets"] if self.groups else None, v["prefix_lens"] if self.groups else None,
                                   v["w_uk"], None if self.latent else v["w_uv"], self.out, self.lse, self.ws,
                                   self.status, stream=stream)

    def result(self):
        torch.cuda.synchronize()
        return self.out.float().cpu().numpy(), self.lse.cpu().numpy(), int(self.status.item())


def reference(inp, picks=None):
    return oracle.decode(inp["dims"], inp["q_nope"], inp["q_pe"], inp["pool"], inp["block_table"], inp["block_size"],
                         inp["seqlens"], inp["w_uk"], inp["w_uv"], picks=picks)


def check(inp, got, picks=None):
    out, lse, st = got
    assert st == 0, st
    ref, ref_lse = reference(inp, picks)
    idx = tuple(np.array(picks).T) if picks is not None else ...
    check_close(out[idx], ref[idx], inp["dims"].dtype, "shared")
    assert np.max(np.abs(lse[idx] - ref_lse[idx])) <= (1e-4 if inp["dims"].dtype == "f32" else 3e-2)


def some(inp, n_seq, n_head, seed=0):
    """Every head of a few sequences would take long at 128 heads: some (b, j, s)."""
    r = np.random.default_rng(seed)
    B, n_q, H = inp["q_nope"].shape[:3]
    seqs = sorted({0, B - 1} | set(r.choice(B, min(B, n_seq), replace=False).tolist()))
    return [(b, j, int(s)) for b in seqs for j in range(n_q)
            for s in sorted({0, H - 1} | set(r.choice(H, min(H, n_head), replace=False).tolist()))]


V2L, V3D = Dims(**V2_LITE), Dims(**V3)
H20 = Dims(**{**V2_LITE, "n_heads": 20})
GROUPS = {
    # (prefix, totals): whole pages, ends inside a page and a block, one sequence inside the prefix, prefixes of 0.
    "one": [(128, [130, 129, 200, 391])],
    "ragged": [(200, [201, 260, 230]), (0, [5, 77]), (64, [65]), (640, [640, 641, 1000, 703, 900])],
    "inside": [(512, [300, 512, 700, 2])],
    "empty": [(64, []), (256, [257, 300, 320]), (1 << 20, [70, 500, 900]), (128, [])],
    "lone": [(448, [450]), (64, [66, 100])],
}


@pytest.mark.gpu
@pytest.mark.parametrize("shape", sorted(GROUPS))
@pytest.mark.parametrize("dims,n_q,bs,layout", [(Dims(**SMALL), 1, 16, 0), (Dims(**SMALL), 2, 7, 0), (V2L, 1, 64, 1),
                                                (V2L, 2, 64, 0), (V2L, 4, 128, 1), (H20, 2, 64, 1)])
def test_shared_small_all_outputs(lib, shape, dims, n_q, bs, layout):
    groups = [(p, [max(n, n_q) for n in seqs]) for p, seqs in GROUPS[shape]]
    inp = make_shared(dims, groups, n_q, bs, seed=len(shape) + n_q)
    c = Call(lib, inp, layout)
    c.run()
    picks = None if dims.n_heads <= 8 else some(inp, 16, 4)
    check(inp, c.result(), picks)


@pytest.mark.gpu
@pytest.mark.parametrize("n_q,layout", [(1, 1), (2, 1), (1, 0)])
def test_shared_v3_heads(lib, n_q, layout):
    inp = make_shared(V3D, [(704, [705, 900, 706]), (1024, [1030, 1100, 1300, 1026, 1029]), (0, [40])], n_q, 64, seed=3)
    inp["seqlens"] = torch.clamp(inp["seqlens"], min=n_q)
    c = Call(lib, inp, layout)
    c.run()
    check(inp, c.result(), some(inp, 9, 3))


@pytest.mark.gpu
def test_shared_matches_the_plain_decode_and_the_latent_form(lib):
    """Against mla_decode / mla_decode_latent over the same table (bf16: both within the bar of the oracle)."""
    inp = make_shared(V2L, GROUPS["ragged"], 1, 64, seed=5)
    full, plain = Call(lib, inp), Call(lib, inp, groups=False)
    lat = Call(lib, inp, latent=True)
    for c in (full, plain, lat):
        c.run()
    (o1, l1, s1), (o2, l2, s2), (o3, l3, s3) = (c.result() for c in (full, plain, lat))
    assert s1 == s2 == s3 == 0
    check_close(o1, o2, "bf16", "shared vs ungrouped")
    o_from_lat = np.einsum("bjhc,hcv->bjhv", o3, inp["w_uv"].float().numpy())
    check_close(o_from_lat, o1, "bf16", "latent form")
    assert np.max(np.abs(l1 - l2)) <= 3e-2
    # The two merges add at most 2 x 75 positive weights in different orders (150 * 2^-24 relative) whose exponentials
    # may differ by a few ulps (2^-21), and round the logarithm (lse < 16: 2^-21): below 1.1e-5 together.
    assert np.max(np.abs(l1 - l3)) <= 1.1e-5


@pytest.mark.gpu
def test_shared_peaked_scores(lib):
    """Scores spread over hundreds (one key takes all the weight, in the prefix or in the tail): the running maximum
    moves often, and partials whose share is nil leave no trace."""
    inp = make_shared(V2L, [(640, [700, 650, 900, 641, 1100, 800, 777, 690])], 1, 64, seed=9, spread=24.0)
    c = Call(lib, inp)
    c.run()
    out, lse, st = c.result()
    ref, ref_lse = reference(inp)
    assert st == 0
    # Scores are N(0, 24^2): a bf16 query moves each by up to 24 * 2^-8 * a few = 0.3, so weights near the top shift
    # by as much; rows whose largest score leads by 8 are decided (the rest weighs e^-8), and their output is the
    # leading row's value within bf16 steps.
    d = np.abs(out - ref).max(-1) / np.abs(ref).max(-1)
    assert np.median(d) < 2e-2
    assert np.max(np.abs(lse - ref_lse)) <= 0.5


@pytest.mark.gpu
def test_shared_on_a_stream_in_a_graph_and_repeated(lib):
    """Same bits again from another stream, from a replayed graph (with other lengths written between replays) and
    after the workspace was overwritten."""
    inp = make_shared(V2L, [(640, [700, 650, 900, 641]), (128, [300, 129])], 1, 64, seed=11)
    c = Call(lib, inp)
    c.run()
    o0, l0, st = c.result()
    assert st == 0
    c.out.fill_(float("nan"))
    c.ws.fill_(0x7F)
    torch.cuda.synchronize()
    c.run(stream=torch.cuda.Stream())
    o1, l1, _ = c.result()
    assert np.array_equal(o0, o1) and np.array_equal(l0, l1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    keep = c.dev["prefix_lens"].clone()
    c.dev["prefix_lens"].zero_()
    g.replay()
    o2, _, st = c.result()
    assert st == 0
    check_close(o2, o0, "bf16", "nothing shared")
    c.dev["prefix_lens"].copy_(keep)
    g.replay()
    o3, l3, _ = c.result()
    assert np.array_equal(o0, o3) and np.array_equal(l0, l3)


@pytest.mark.gpu
@pytest.mark.parametrize("spoil", ["first", "last", "falls", "negative"])
def test_shared_bad_groups_are_reported_and_share_nothing(lib, spoil):
    inp = make_shared(V2L, [(128, [200, 300]), (64, [100, 90])], 1, 64, seed=13)
    if spoil == "first":
        inp["group_offsets"][0] = 1
    elif spoil == "last":
        inp["group_offsets"][2] = 1 << 30
    elif spoil == "falls":
        inp["group_offsets"][1] = -7
    else:
        inp["prefix_lens"][1] = -64
    c = Call(lib, inp)
    c.run()
    out, lse, st = c.result()
    assert st == -6
    ref, _ = reference(inp, some(inp, 4, 3))
    idx = tuple(np.array(some(inp, 4, 3)).T)
    check_close(out[idx], ref[idx], "bf16", "bad groups")


@pytest.mark.gpu
def test_shared_bad_block_of_the_prefix_is_reported(lib):
    inp = make_shared(V2L, [(256, [300, 310, 290])], 1, 64, seed=15)
    for blk in (-1, inp["num_blocks"]):
        bad = dict(inp, block_table=inp["block_table"].clone())
        bad["block_table"][:, 2] = blk
        c = Call(lib, bad)
        c.run()
        assert c.result()[2] == -6


def _heads(h):
    return Dims(**{**V2_LITE, "n_heads": h})


@pytest.mark.gpu
@pytest.mark.parametrize("heads,n_q", [(1, 1), (4, 1), (7, 1), (8, 1), (9, 1), (80, 2), (96, 2), (128, 2), (255, 1), (256, 1)])
def test_shared_head_counts(lib, heads, n_q):
    """Units of up to 32 sequences, units that cut a sequence's rows, one sequence per unit: 70 sequences (7 at many
    heads) in three groups, tails of one to three pages, one page shared and many."""
    r = np.random.default_rng(heads)
    n = 70 if heads <= 9 else 7
    cut = sorted(r.choice(np.arange(1, n), 2, replace=False).tolist())
    lens = r.integers(n_q, 190, n)
    groups, at = [], 0
    for p, end in zip((64, 1280, 192), cut + [n]):
        groups.append((p, [int(p + x) for x in lens[at:end]]))
        at = end
    inp = make_shared(_heads(heads), groups, n_q, 64, seed=heads)
    c = Call(lib, inp, heads % 2)
    c.run()
    check(inp, c.result(), some(inp, 12, 3, seed=heads))


@pytest.mark.gpu
def test_shared_many_sequences_and_groups(lib):
    """3000 sequences in some 1200 groups (empty ones too): the plan works outside shared memory."""
    r = np.random.default_rng(3)
    B = 3000
    bounds = np.concatenate(([0], np.sort(r.integers(0, B + 1, 1199)), [B]))
    groups = [(int(r.integers(0, 3)) * 64, [int(x) for x in r.integers(1, 200, b - a)]) for a, b in zip(bounds, bounds[1:])]
    inp = make_shared(_heads(2), groups, 1, 64, seed=4)
    c = Call(lib, inp)
    c.run()
    check(inp, c.result(), some(inp, 60, 2))


@pytest.mark.gpu
def test_shared_long_runs_of_pages(lib):
    """A unit per cluster and 74 pages each: the page lookups move on, and every barrier goes round many times."""
    inp = make_shared(V3D, [(4608, [4608 + 1 + 3 * i for i in range(68)])], 1, 64, seed=21)
    c = Call(lib, inp)
    c.run()
    check(inp, c.result(), some(inp, 3, 2))


@pytest.mark.gpu
@pytest.mark.parametrize("n,longer", [(64, 0), (66, 0), (66, 2000), (68, 0), (7, 0)])
def test_shared_units_that_have_a_cluster_each_or_are_cut(lib, n, longer):
    """As many units as clusters and fewer, alike in length (none is cut) and not (they are); one unit more; a group of one
    sequence whose length is refused leaves a unit with nothing to do."""
    groups = [(1024, [1025 + i % 3 for i in range(n - 1)]), (0, [64 + longer])]
    inp = make_shared(V3D, groups, 1, 64, seed=n)
    c = Call(lib, inp)
    c.run()
    check(inp, c.result(), some(inp, 4, 2))
    picks = [x for x in some(inp, 4, 2) if x[0] < n - 1]
    ref, _ = reference(inp, picks)
    c.dev["seqlens"][n - 1] = 0
    c.run()
    out, _, st = c.result()
    assert st == -6
    idx = tuple(np.array(picks).T)
    check_close(out[idx], ref[idx], "bf16", "beside a refused length")
    assert not out[n - 1].any()


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(8))
def test_shared_random_batches(lib, seed):
    r = np.random.default_rng(100 + seed)
    heads, bs = int(r.choice([12, 16, 20, 64, 128])), int(r.choice([64, 128, 192]))
    n_q = int(r.integers(1, 256 // heads + 1)) if heads <= 64 else int(r.integers(1, 3))
    n_q = min(n_q, 5)
    groups = []
    for _ in range(int(r.integers(1, 5))):
        p = int(r.choice([0, r.integers(1, 300), 64 * r.integers(1, 20)]))
        groups.append((p, [int(max(n_q, p + r.integers(-40, 400))) for _ in range(int(r.integers(1, 8)))]))
    inp = make_shared(_heads(heads), groups, n_q, bs, seed=seed)
    c = Call(lib, inp, seed % 2)
    c.run()
    check(inp, c.result(), some(inp, 6, 3, seed))


@pytest.mark.gpu
def test_shared_bad_lengths_are_reported(lib):
    """A length below n_q or beyond max_seqlen is reported; the other groups' results stand."""
    inp = make_shared(V2L, [(128, [200, 300, 150]), (64, [100, 90])], 2, 64, seed=17)
    picks = [x for x in some(inp, 5, 3) if x[0] >= 3]
    idx = tuple(np.array(picks).T)
    ref, _ = reference(inp, picks)
    for bad in (1, 0, -5, 100000):
        c = Call(lib, inp)
        c.dev["seqlens"][1] = bad
        c.run()
        out, lse, st = c.result()
        assert st == -6
        check_close(out[idx], ref[idx], "bf16", "other group")


@pytest.mark.gpu
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("heads,n_q", [(4, 1), (16, 2), (96, 1), (128, 1)])
def test_shared_values_that_are_not_finite_stay_with_their_sequence(lib, heads, n_q, layout):
    """NaN and infinities among one sequence's own keys: the other sequences of the group, whose rows meet these keys
    with a weight of 0, keep their bits, and the sequence itself has NaN, as in a decode of its own."""
    groups = [(192, [250, 330, 193 + n_q, 500, 196, 260]), (0, [70, 40])]
    inp = make_shared(_heads(heads), groups, n_q, 64, seed=heads)
    c = Call(lib, inp, layout)
    c.run()
    want, _, st = c.result()
    assert st == 0
    for seq, key, dims, value in ((1, 200, slice(0, 576), float("nan")), (3, 450, slice(300, 301), float("inf")),
                                  (3, 200, slice(511, 512), float("nan")), (4, 193, slice(10, 12), float("-inf")),
                                  (0, 192, slice(520, 521), float("nan")), (7, 0, slice(0, 8), float("nan"))):
        bad = dict(inp, pool=inp["pool"].clone())
        row = int(inp["block_table"][seq, key // 64]) * 64 + key % 64
        bad["pool"][row, dims] = value
        c = Call(lib, bad, layout)
        c.run()
        got, _, st = c.result()
        assert st == 0
        others = [b for b in range(8) if b != seq]
        assert np.array_equal(got[others], want[others]), (seq, value)
        if np.isnan(value):
            assert np.isnan(got[seq]).all(), seq


def _shifted(t):
    """The same values behind an address that is no multiple of 4 bytes."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    flat[1:].copy_(t.flatten())
    return flat[1:].view(t.shape)


@pytest.mark.gpu
@pytest.mark.parametrize("d_nope,shift", [(128, True), (40, False), (96, False), (96, True)])
def test_shared_queries_that_the_tensor_core_absorption_does_not_take(lib, d_nope, shift):
    """Odd addresses and widths of the queries: the plan is a launch of its own, and another kernel absorbs."""
    dims = Dims(**{**V2_LITE, "d_nope": d_nope})
    inp = make_shared(dims, GROUPS["ragged"], 2, 64, seed=d_nope)
    inp["seqlens"] = torch.clamp(inp["seqlens"], min=2)
    c = Call(lib, inp)
    if shift:
        for k in ("q_nope", "q_pe", "w_uk"):
            c.dev[k] = _shifted(c.dev[k])
    c.run()
    check(inp, c.result(), some(inp, 8, 4))


@pytest.mark.gpu
def test_shared_refuses_odd_addresses_of_outputs_weights_and_pools(lib):
    inp = make_shared(V2L, [(64, [100, 90])], 1, 64, seed=43)
    for key, groups in (("out", True), ("w_uv", True), ("c_kv", True), ("out", False), ("w_uv", False), ("c_kv", False)):
        c = Call(lib, inp, groups=groups)
        if key == "out":
            c.out = _shifted(c.out)
        elif key == "w_uv":
            c.dev["w_uv"] = _shifted(c.dev["w_uv"])
        else:
            c.c_kv = _shifted(c.c_kv)
        with pytest.raises(RuntimeError):
            c.run()


@pytest.mark.gpu
def test_shared_two_calls_at_once(lib):
    """Two calls on two streams with workspaces of their own, many times over: the bits of each call alone."""
    calls = [Call(lib, make_shared(V2L, [(640, [700, 650, 900, 641]), (128, [300, 129])], 1, 64, seed=31)),
             Call(lib, make_shared(_heads(64), [(1024, [1100, 1030, 1500])], 2, 64, seed=32))]
    alone = []
    for c in calls:
        c.run()
        alone.append(c.result())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for c, st in zip(calls, streams):
            c.run(stream=st)
    for c, (o, l, _) in zip(calls, alone):
        o1, l1, st = c.result()
        assert st == 0 and np.array_equal(o, o1) and np.array_equal(l, l1)


@pytest.mark.gpu
def test_shared_graphs_that_share_a_workspace(lib):
    """Two captured graphs with one workspace, replayed in turn on one stream."""
    a = Call(lib, make_shared(V2L, [(640, [700, 650, 900, 641]), (128, [300, 129])], 1, 64, seed=33))
    b = Call(lib, make_shared(V2L, [(192, [200, 250]), (0, [30])], 1, 64, seed=34))
    for c in (a, b):
        c.run()
    want = [a.result(), b.result()]
    if b.ws.numel() > a.ws.numel():
        a.ws = b.ws
    b.ws = a.ws
    graphs = []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    for c in (a, b):
        c.out.fill_(float("nan"))
    for _ in range(5):
        for g in graphs:
            g.replay()
    for c, (o, l, _) in zip((a, b), want):
        o1, l1, st = c.result()
        assert st == 0 and np.array_equal(o, o1) and np.array_equal(l, l1)


@pytest.mark.gpu
def test_shared_refuses_wrong_tensors(lib):
    inp = make_shared(V2L, [(64, [100, 90])], 1, 64, seed=41)
    for key, bad in (("q_nope", lambda t: t.float()), ("q_pe", lambda t: t[:, :, :8]), ("seqlens", lambda t: t.long()),
                     ("block_table", lambda t: t[:, :1]), ("w_uk", lambda t: t.transpose(1, 2)), ("prefix_lens", lambda t: t.repeat(2)),
                     ("group_offsets", lambda t: t.cpu()), ("q_nope", lambda t: None), ("prefix_lens", lambda t: None)):
        c = Call(lib, inp)
        c.dev[key] = bad(c.dev[key])
        with pytest.raises((TypeError, ValueError, AttributeError)):
            c.run()


def test_shared_host_refusals():
    import mla_latent_kv_40_b200 as mla
    lib = mla._lib
    d = mla.make_dims(16, 512, 64, 128, 128, 2048, 64, "bf16", cache_layout=1)
    f, n = ctypes.c_void_p(0x1000), ctypes.c_size_t(0)
    size = lambda *a: lib.mla_decode_shared_workspace_size(ctypes.byref(d), *a, ctypes.byref(n))   # noqa: E731
    assert size(4, 1, 100, 2) == 0 and n.value > 0
    assert size(0, 1, 100, 0) == size(4, 1, 0, 1) == size(4, 1, 100, -1) == size(4, 1, 100, 5) == -1
    assert size(4, 17, 100, 1) == -2
    base = dict(dims=ctypes.byref(d), B=4, n_q=1, qn=f, qp=f, ckv=f, kpe=None, bt=f, mb=4, nb=9, sl=f, ms=100, G=2, offs=f,
                pl=f, wuk=f, wuv=f, out=f, lse=None, ws=f, bytes=ctypes.c_size_t(1 << 40), st=None, stream=None)
    for over, rc in [(dict(qn=None), -1), (dict(qp=None), -1), (dict(ckv=None), -1), (dict(bt=None), -1), (dict(sl=None), -1),
                     (dict(wuk=None), -1), (dict(out=None), -1), (dict(G=-1), -1), (dict(G=5), -1), (dict(offs=None), -1),
                     (dict(pl=None), -1), (dict(mb=1), -1), (dict(n_q=17), -2), (dict(ws=None), -3),
                     (dict(bytes=ctypes.c_size_t(8)), -3), (dict(ws=ctypes.c_void_p(0x1010)), -3), (dict(B=0), -1)]:
        assert lib.mla_decode_shared(*{**base, **over}.values()) == rc, over
