"""mla_decode_shared, mla_plan_step and mla_release_blocks at the ends of their ranges: lengths that are no lengths, plans
that do not fit into shared memory, idle requests, rows past 2^31."""
import numpy as np
import pytest
import torch

from helpers import check_close
from test_shared_parity import Call, V2L, _heads, make_shared, reference, some
from test_shared_serving import D as loop_dims, Loop

INT_MIN, INT_MAX = -2**31, 2**31 - 1


@pytest.mark.gpu
@pytest.mark.parametrize("n_q", [1, 2, 5])
@pytest.mark.parametrize("bad", [INT_MIN, INT_MIN + 1, INT_MIN + 3, -1, INT_MAX])
def test_shared_lengths_at_the_ends_of_their_type(lib, bad, n_q):
    """Reported like any other length that is none: S - n_q + 1 must not wrap to a long one.  The other groups' results
    stand."""
    inp = make_shared(V2L, [(128, [200, 300, 150]), (64, [100, 90])], n_q, 64, seed=17)
    picks = [x for x in some(inp, 5, 3) if x[0] >= 3]
    idx = tuple(np.array(picks).T)
    ref, _ = reference(inp, picks)
    c = Call(lib, inp)
    c.dev["seqlens"][1] = bad
    c.run()
    out, lse, st = c.result()
    assert st == -6
    check_close(out[idx], ref[idx], "bf16", "other group")


@pytest.mark.gpu
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("heads,n_q", [(4, 1), (16, 2), (96, 1), (128, 1)])
def test_shared_infinite_latents_leave_their_sequence_no_finite_row(lib, heads, n_q, layout):
    """0 * inf is NaN also where the infinite latent makes the score -inf: every row that sees such a key has NaN, as in a
    decode of its own and whoever shares its unit; the other sequences keep their bits."""
    groups = [(192, [250, 330, 193 + n_q, 500, 196, 260]), (0, [70, 40])]
    inp = make_shared(_heads(heads), groups, n_q, 64, seed=heads)
    c = Call(lib, inp, layout)
    c.run()
    want, _, st = c.result()
    assert st == 0
    inf = float("inf")
    for seq, key, dim, value in ((3, 450, 300, inf), (3, 450, 300, -inf), (1, 200, 0, -inf), (1, 329, 511, inf), (4, 192, 10, -inf),
                                 (7, 0, 255, inf), (5, 256, 256, -inf), (0, 249, 575, inf)):
        bad = dict(inp, pool=inp["pool"].clone())
        row = int(inp["block_table"][seq, key // 64]) * 64 + key % 64
        bad["pool"][row, dim] = value
        c, plain = Call(lib, bad, layout), Call(lib, bad, layout, groups=False)
        c.run()
        plain.run()
        (got, _, st), (alone, _, _) = c.result(), plain.result()
        assert st == 0
        others = [b for b in range(8) if b != seq]
        assert np.array_equal(got[others], want[others]), (seq, value)
        S = int(inp["seqlens"][seq])
        for j in range(n_q):
            if key > S - n_q + j:   # (a row that does not see the key: mla_decode multiplies it by 0)
                continue
            # (a RoPE key of -inf is a key of no weight: nothing of it is in the values)
            if dim < 512:
                assert np.isnan(got[seq, j]).all(), (seq, key, dim, j)
            assert np.array_equal(np.isnan(got[seq, j]), np.isnan(alone[seq, j])), (seq, key, dim, j)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
def test_plan_and_release_of_nearly_2_to_31_tokens_and_blocks(lib):
    """Four requests of 2^29 - 1 tokens in blocks of one token: 2^31 - 4 tokens, table entries and free ids, so that the last
    step of every thread's walk passes 2^31."""
    n, B = 2**29 - 1, 4
    total = n * B
    dims = lib.make_dims(16, 512, 64, 128, 128, 7168, 1, "bf16")
    free_list = torch.arange(total, dtype=torch.int32, device="cuda")
    free, lens, cu, st = _i32([total]), _i32([0] * B), _i32([0] * (B + 1)), _i32([0])
    table = torch.full((B, n), -1, dtype=torch.int32, device="cuda")
    seq_idx = torch.full((total,), -7, dtype=torch.int32, device="cuda")
    pos = torch.full((total,), -7, dtype=torch.int32, device="cuda")
    lib.mla_plan_step(dims, lens, _i32([n] * B), None, None, None, free_list, free, table, total, lens, cu, seq_idx, pos, None, free, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and int(free.item()) == 0
    assert lens.tolist() == [n] * B and cu.tolist() == [b * n for b in range(B + 1)]
    steps = torch.arange(n, dtype=torch.int32, device="cuda")
    for b in range(B):   # the k-th new block is free_list[total - 1 - k] = total - 1 - k
        assert torch.equal(table[b], total - 1 - b * n - steps)
        assert torch.equal(pos[b * n:(b + 1) * n], steps)
        assert bool((seq_idx[b * n:(b + 1) * n] == b).all())
    del seq_idx, pos, steps
    free_list.fill_(-1)
    lib.mla_release_blocks(dims, _i32([1] * B), lens, None, None, table, total, free_list, free, lens, free, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and int(free.item()) == total and lens.tolist() == [0] * B
    assert torch.equal(free_list, table.view(-1))


@pytest.mark.gpu
def test_a_serving_loop_with_idle_slots_reports_nothing(lib):
    """Requests finish and their slots stay free for some steps: the plan passes over them (length 0, no token), the decode is
    given the prefix's length for them, and dev_status stays 0 at every step; later others join in their places."""
    loop = Loop(lib)
    new = [5, 64, 3, 130, 1, 70, 63, 90]
    b = loop.plan(new, sum(new))
    loop.append(loop.rnd(sum(new), loop_dims.d_model), b["seq_idx"], b["pos"], loop.table, loop.mb)
    done = [0, 1, 0, 0, 0, 0, 1, 0]          # (not the groups' first, whose rows name the prompts)
    lib.mla_release_blocks(loop.dims, _i32(done), loop.lens, loop.offsets, loop.prefixes, loop.table, 40, loop.free_list,
                           loop.free_count, loop.lens, loop.free_count, loop.status)
    assert loop.lens.tolist()[1] == loop.lens.tolist()[6] == 0
    prefix = torch.repeat_interleave(loop.prefixes, (loop.offsets[1:] - loop.offsets[:-1]).long())
    d, lens = loop.decode_buffers(), loop.lens
    for step in range(3):
        b = loop.plan([1 - x for x in done], 6)
        loop.append(loop.rnd(6, loop_dims.d_model), b["seq_idx"], b["pos"], loop.table, loop.mb)
        loop.lens = torch.where(lens == 0, prefix, lens)     # what the decode sees
        loop.call_decode(d)
        loop.check_decode(d)                                 # (the idle slots' rows are those of the prompt alone)
        loop.lens = lens
        torch.cuda.synchronize()
        assert int(loop.status.item()) == 0 and lens.tolist()[1] == lens.tolist()[6] == 0
        assert b["cu"].tolist() == [0, 1, 1, 2, 3, 4, 5, 5, 6]
    lens[1], lens[6] = 128, 192                              # new requests behind the same prompts
    b = loop.plan([1, 7, 1, 1, 1, 1, 2, 1], 15)
    loop.append(loop.rnd(15, loop_dims.d_model), b["seq_idx"], b["pos"], loop.table, loop.mb)
    loop.call_decode(d)
    loop.check_decode(d)


@pytest.mark.gpu
def test_plan_idle_slots_beside_what_is_refused(lib):
    """Length 0 without tokens behind a prefix is idle; with a token, or with tokens short of the prefix, refused."""
    lens, new = _i32([0, 0, 64, 128, 0]), _i32([0, 1, 0, 1, 0])
    for rows, status in (([0, 4], 0), ([0, 1], -6), ([2, 4], -6), ([3], 0)):
        B = len(rows)
        pick = torch.tensor(rows, device="cuda")
        c, n, st = lens[pick].contiguous(), new[pick].contiguous(), _i32([0])
        table, cu, free = torch.full((B, 4), -1, dtype=torch.int32, device="cuda"), _i32([0] * (B + 1)), _i32([4])
        seq_idx, pos, out = _i32([-7] * 4), _i32([-7] * 4), torch.full_like(c, -9)
        dims = lib.make_dims(16, 512, 64, 128, 128, 7168, 64, "bf16")
        lib.mla_plan_step(dims, c, n, _i32([0, B]), _i32([128]), _i32([[5, 6]]), _i32([0, 1, 2, 3]), free, table, 7, out, cu, seq_idx,
                          pos, None, free, st)
        torch.cuda.synchronize()
        assert int(st.item()) == status, rows
        if rows == [0, 4]:
            assert out.tolist() == [0, 0] and cu.tolist() == [0, 0, 0] and (table == -1).all() and int(free.item()) == 4
            assert (seq_idx == -7).all()


@pytest.mark.gpu
def test_the_current_stream_with_and_without_torch_s_private_handle(lib, monkeypatch):
    """The small calls ask for the current stream's handle directly, or, where this torch has no such call, as the others do:
    the same stream, by default, in a stream context and where one is given."""
    side = torch.cuda.Stream()
    dev = torch.cuda.current_device()

    def handles():
        default = lib._raw_stream(None, dev)
        with torch.cuda.stream(side):
            inside = lib._raw_stream(None, dev)
        return default, inside, lib._raw_stream(side, dev)

    want = (torch.cuda.current_stream().cuda_stream, side.cuda_stream, side.cuda_stream)
    assert handles() == want
    monkeypatch.setattr(lib, "_current_handle", None)
    assert handles() == want
    inp = make_shared(V2L, [(128, [200, 300, 150])], 1, 64, seed=19)
    c = Call(lib, inp)
    with torch.cuda.stream(side):
        c.run()
    side.synchronize()
    first = c.out.clone()
    monkeypatch.undo()
    c.out.zero_()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        c.run()
    side.synchronize()
    assert torch.equal(first, c.out)


@pytest.mark.gpu
@pytest.mark.parametrize("n_q", [1, 2, 4])
def test_shared_idle_slots_as_the_header_says(lib, n_q):
    """A slot given the prefix's length plus n_q - 1, with a table row that names nothing of the prefix (it is not the first) and
    for n_q > 1 one block behind it: nothing is reported, and the others have the bits that they have beside a real
    member of that length."""
    P = 256
    inp = make_shared(V2L, [(P, [300, P + n_q - 1, 320, 500])], n_q, 64, seed=23)
    full = Call(lib, inp)
    full.run()
    want, want_lse, st = full.result()
    assert st == 0
    table = inp["block_table"].clone()
    table[1] = -1
    table[1, P // 64 if n_q > 1 else 0] = 0
    idle = Call(lib, dict(inp, block_table=table))
    idle.run()
    got, lse, st = idle.result()
    others = [0, 2, 3]
    assert st == 0 and np.array_equal(got[others], want[others]) and np.array_equal(lse[others], want_lse[others])
