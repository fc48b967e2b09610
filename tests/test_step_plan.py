"""mla_plan_step and mla_release_blocks: the host's refusals, and every output word against a plain model that walks the
requests one by one (whole numbers: equal, no tolerance)."""
import ctypes

import numpy as np
import pytest
import torch

INT_MAX = 2**31 - 1


# ---------------------------------------------------------------- the model
def model_groups(B, offsets):
    """Group of every request, or None where the offsets do not rise from 0 to B."""
    if offsets is None:
        return [-1] * B, False
    o = list(offsets)
    if o[0] != 0 or o[-1] != B or any(x > y for x, y in zip(o, o[1:])):
        return [-1] * B, True
    return [g for g in range(len(o) - 1) for _ in range(o[g], o[g + 1])], False


def model_plan(bs, cached, new, offsets, prefixes, prefix_table, free_list, free, table, num_blocks, max_tokens):
    """(table, seqlens, cu, seq_idx, pos, slots, free, errors); token entries behind the last token are -7."""
    B, mb = table.shape
    table = table.copy()
    gid, bad_groups = model_groups(B, offsets)
    errors = {-6} if bad_groups else set()
    if not 0 <= free <= len(free_list):
        errors.add(-6)
        free = min(max(free, 0), len(free_list))
    seq_idx, pos, slots = (np.full(max_tokens, -7, np.int64) for _ in range(3))
    seqlens, cu, left, out_of = [], [0], free, False
    for b in range(B):
        c, n = int(cached[b]), int(new[b])
        P = int(prefixes[gid[b]]) if gid[b] >= 0 else 0
        bad = n < 0 or n > max_tokens
        n = 0 if bad else n
        bad |= c < 0 or c + n > min(mb * bs, INT_MAX) or P < 0 or P % bs != 0 or c < P
        if gid[b] >= 0 and P >= 0:
            bad |= P // bs > prefix_table.shape[1]
        lo, hi = cu[-1], cu[-1] + n
        bad |= n > 0 and hi > max_tokens
        cu.append(hi)
        lo, hi = min(lo, max_tokens), min(hi, max_tokens)
        need = 0 if bad else -(-(c + n) // bs) - -(-c // bs)
        if bad:
            errors.add(-6)
        elif need and (out_of or need > left):
            errors.add(-8)
            out_of = bad = True
        if bad:
            seqlens.append(max(c, 0))
            seq_idx[lo:hi] = pos[lo:hi] = slots[lo:hi] = -1
            continue
        for i in range(-(-c // bs), -(-(c + n) // bs)):
            left -= 1
            ident = int(free_list[left])
            if not 0 <= ident < num_blocks:
                errors.add(-6)
                ident = -1
            table[b, i] = ident
        if P > 0 and c == P:
            table[b, :P // bs] = prefix_table[gid[b], :P // bs]
        seqlens.append(c + n)
        for t in range(n):
            p = c + t
            blk = int(table[b, p // bs])
            ok = 0 <= blk < num_blocks
            if not ok:
                errors.add(-6)
            seq_idx[lo + t], pos[lo + t], slots[lo + t] = (b, p, blk * bs + p % bs) if ok else (-1, -1, -1)
    return table, seqlens, [min(x, max_tokens) for x in cu], seq_idx, pos, slots, left, errors


def model_release(bs, done, seqlens, offsets, prefixes, table, num_blocks, free_list, free):
    B, mb = table.shape
    fl, out = free_list.copy(), list(int(x) for x in seqlens)
    gid, bad_groups = model_groups(B, offsets)
    errors, full = ({-6} if bad_groups else set()), False
    if not 0 <= free <= len(fl):
        errors.add(-6)
        free = min(max(free, 0), len(fl))
    for b in range(B):
        P = int(prefixes[gid[b]]) if gid[b] >= 0 else 0
        if not done[b]:
            continue
        n = out[b]
        if n < 0 or P < 0 or P % bs or -(-n // bs) > mb:
            errors.add(-6)
            continue
        ids = table[b, P // bs:-(-n // bs)]
        if len(ids) and (full or free + len(ids) > len(fl)):
            errors.add(-6)
            full = True
            continue
        if np.any((ids < 0) | (ids >= num_blocks)):
            errors.add(-6)
        fl[free:free + len(ids)] = ids
        free += len(ids)
        out[b] = 0
    return fl, out, free, errors


# ---------------------------------------------------------------- random states
def make_state(seed, B, bs, G, prefix_blocks, own_hi, new_hi, short=False, spoil=False):
    """A pool in mid-flight.  spoil: some lengths, prefixes and ids that the call has to refuse."""
    r = np.random.default_rng(seed)
    offsets = prefixes = pt = None
    gid = [-1] * B
    if G:
        offsets = np.concatenate(([0], np.sort(r.integers(0, B + 1, G - 1)), [B])).astype(np.int32)   # empty groups too
        prefixes = (r.integers(0, prefix_blocks + 1, G) * bs).astype(np.int32)
        gid = [g for g in range(G) for _ in range(offsets[g], offsets[g + 1])]
    own = r.integers(0, own_hi + 1, B)
    own[r.random(B) < 0.3] = 0
    new = r.integers(0, new_hi + 1, B)
    P = np.array([prefixes[g] if g >= 0 else 0 for g in gid])
    cached = P + own
    mb = int(max(-(-(cached + new) // bs))) + 1
    held = int(sum(-(-own // bs))) + (int(sum(prefixes // bs)) if G else 0)
    need = int(sum(-(-(cached + new) // bs) + (-cached // bs)))
    free = need * 2 // 3 if short else need + 3
    num_blocks = held + max(free, need) + 3
    ids = r.permutation(num_blocks).astype(np.int32)
    k = 0
    if G:
        pt = np.full((G, prefix_blocks), -1, np.int32)
        for g in range(G):
            pt[g, :prefixes[g] // bs] = ids[k:k + prefixes[g] // bs]
            k += prefixes[g] // bs
    table = np.full((B, mb), -5, np.int32)
    for b in range(B):
        n, p = -(-own[b] // bs), P[b] // bs
        if own[b]:
            table[b, :p] = pt[gid[b], :p] if p else table[b, :p]
            table[b, p:p + n] = ids[k:k + n]
            k += n
    fl = np.full(num_blocks, -1, np.int32)
    fl[:free] = ids[k:k + free]
    s = dict(bs=bs, B=B, cached=cached.astype(np.int32), new=new.astype(np.int32), offsets=offsets, prefixes=prefixes,
             pt=pt, fl=fl, free=free, table=table, num_blocks=num_blocks, max_tokens=int(new.sum()) + 5)
    if spoil:
        for x, v in ((s["cached"], -3), (s["new"], -1), (s["new"], s["max_tokens"] + 1), (s["cached"], mb * bs - 1),
                     (s["cached"], INT_MAX)):
            x[r.integers(B)] = v
        if free > 2:
            fl[free - 2] = num_blocks
        if G > 1:
            prefixes[r.integers(G)] += 1
    return s


def run_plan(mla, s, stream=None, slots=True, offset=0, in_place=False):
    """Device call on fresh buffers; `offset` elements of misalignment on the token arrays."""
    cu = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()   # noqa: E731
    dims = mla.make_dims(16, 512, 64, 128, 128, 7168, s["bs"], "bf16")
    T = s["max_tokens"]
    cached, table, free = cu(s["cached"]), cu(s["table"]), torch.tensor([s["free"]], dtype=torch.int32, device="cuda")
    tok = lambda dt: torch.full((T + offset,), -7, dtype=dt, device="cuda")[offset:]   # noqa: E731
    seq_idx, pos, sl = tok(torch.int32), tok(torch.int32), tok(torch.int64) if slots else None
    seqlens = cached if in_place else torch.full_like(cached, -9)
    fout = free if in_place else torch.full_like(free, -9)
    cul = torch.full((s["B"] + 1,), -9, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (dims, cached, cu(s["new"]), cu(s["offsets"]), cu(s["prefixes"]), cu(s["pt"]), cu(s["fl"]), free, table,
            s["num_blocks"], seqlens, cul, seq_idx, pos, sl, fout, st)
    torch.cuda.synchronize()
    mla.mla_plan_step(*args, stream=stream)
    torch.cuda.synchronize()
    n = lambda x: x.cpu().numpy()   # noqa: E731
    return n(table), n(seqlens), n(cul), n(seq_idx), n(pos), n(sl) if slots else None, int(fout.item()), int(st.item())


def check_plan(got, s):
    want = model_plan(s["bs"], s["cached"], s["new"], s["offsets"], s["prefixes"], s["pt"], s["fl"], s["free"], s["table"],
                      s["num_blocks"], s["max_tokens"])
    for name, a, b in zip(("table", "seqlens", "cu_seqlens", "seq_idx", "pos", "slots"), got, want):
        if a is not None:
            np.testing.assert_array_equal(a, np.asarray(b), err_msg=name)
    assert got[6] == want[6]
    assert (got[7] in want[7]) if want[7] else got[7] == 0


CASES = [  # B, block, groups, prefix blocks, own tokens, new tokens
    (1, 64, 0, 0, 0, 1), (1, 64, 1, 3, 100, 1), (2, 16, 1, 1, 40, 70), (33, 64, 4, 9, 500, 3), (64, 1, 5, 4, 9, 5),
    (100, 7, 7, 6, 200, 90), (257, 16, 257, 5, 300, 40), (1023, 64, 31, 20, 900, 2), (1025, 128, 3, 2, 1000, 65),
    (4096, 16, 40, 8, 300, 9), (8192, 64, 100, 3, 200, 3),
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,bs,G,pb,own,new", CASES)
@pytest.mark.parametrize("kind", ["plain", "short", "spoiled"])
def test_plan_matches_the_model(lib, B, bs, G, pb, own, new, kind):
    s = make_state(B * 7 + bs, B, bs, G, pb, own, new, short=kind != "plain", spoil=kind == "spoiled")
    check_plan(run_plan(lib, s), s)


@pytest.mark.gpu
def test_plan_in_place_unaligned_without_slots_and_on_another_stream(lib):
    s = make_state(5, 300, 16, 6, 5, 200, 33, short=True)
    check_plan(run_plan(lib, s, in_place=True), s)
    check_plan(run_plan(lib, s, offset=1), s)
    check_plan(run_plan(lib, s, slots=False), s)
    check_plan(run_plan(lib, s, stream=torch.cuda.Stream()), s)


@pytest.mark.gpu
def test_plan_refuses_tokens_beyond_the_arrays_and_bad_groups(lib):
    s = make_state(6, 40, 16, 3, 4, 100, 30)
    s["max_tokens"] //= 2
    check_plan(run_plan(lib, s), s)
    s = make_state(6, 40, 16, 0, 0, 100, 30)
    s["max_tokens"] = 0
    check_plan(run_plan(lib, s), s)
    for spoil in (lambda o: o.__setitem__(0, 1), lambda o: o.__setitem__(-1, 41), lambda o: o.__setitem__(1, 1 << 30),
                  lambda o: o.__setitem__(2, -5)):
        s = make_state(7, 40, 16, 5, 4, 100, 30)
        spoil(s["offsets"])
        check_plan(run_plan(lib, s), s)
    for free in (-1, 1 << 30):
        s = make_state(8, 40, 16, 0, 0, 100, 30)
        s["free"] = free
        check_plan(run_plan(lib, s), s)


@pytest.mark.gpu
@pytest.mark.parametrize("B,bs,G,pb,own,new", CASES)
@pytest.mark.parametrize("kind", ["plain", "full", "spoiled"])
def test_release_matches_the_model(lib, B, bs, G, pb, own, new, kind):
    s = make_state(B + bs, B, bs, G, pb, own, new)
    r = np.random.default_rng(B)
    done = (r.random(B) < 0.6).astype(np.int32) * r.integers(1, 9, B).astype(np.int32)
    lens, fl, free = s["cached"], s["fl"], s["free"]
    if kind == "full":
        fl = fl[:free + 7].copy()
    if kind == "spoiled":
        for v in (-1, INT_MAX):
            lens[r.integers(B)] = v
        free = len(fl) + 1
    for in_place in (False, True):
        cu = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()   # noqa: E731
        dims = lib.make_dims(16, 512, 64, 128, 128, 7168, bs, "bf16")
        dl, dfl, df = cu(lens), cu(fl), torch.tensor([free], dtype=torch.int32, device="cuda")
        out, fout = (dl, df) if in_place else (torch.full_like(dl, -9), torch.full_like(df, -9))
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        lib.mla_release_blocks(dims, cu(done), dl, cu(s["offsets"]), cu(s["prefixes"]), cu(s["table"]), s["num_blocks"],
                               dfl, df, out, fout, st)
        torch.cuda.synchronize()
        w_fl, w_out, w_free, errors = model_release(bs, done, lens, s["offsets"], s["prefixes"], s["table"],
                                                    s["num_blocks"], fl, free)
        np.testing.assert_array_equal(dfl.cpu().numpy(), w_fl)
        np.testing.assert_array_equal(out.cpu().numpy(), np.asarray(w_out))
        assert int(fout.item()) == w_free
        assert int(st.item()) in errors if errors else int(st.item()) == 0


@pytest.mark.gpu
def test_a_replayed_graph_advances_the_state_in_place(lib):
    """Captured once, replayed per step: lengths, free count and table advance as the model's, until the pool is empty;
    a release then gives every block back."""
    B, bs, mb = 9, 16, 6
    dims = lib.make_dims(16, 512, 64, 128, 128, 7168, bs, "bf16")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    num_blocks = 25
    fl = np.random.default_rng(1).permutation(num_blocks).astype(np.int32)
    lens, new, table, dfl, free = i32([0] * B), i32([7] * B), i32([[-1] * mb] * B), torch.from_numpy(fl.copy()).cuda(), i32([num_blocks])
    cul, seq_idx, pos, slots = i32([0] * (B + 1)), i32([0] * 7 * B), i32([0] * 7 * B), torch.zeros(7 * B, dtype=torch.int64, device="cuda")
    st = i32([0])
    args = (dims, lens, new, None, None, None, dfl, free, table, num_blocks, lens, cul, seq_idx, pos, slots, free, st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.mla_plan_step(*args)
    m_lens, m_table, m_free = np.zeros(B, np.int32), np.full((B, mb), -1, np.int32), num_blocks
    for _ in range(8):
        st.zero_()
        g.replay()
        torch.cuda.synchronize()
        m_table, m_lens, m_cu, m_seq, m_pos, m_slots, m_free, err = model_plan(
            bs, m_lens, np.full(B, 7), None, None, None, fl, m_free, m_table, num_blocks, 7 * B)
        np.testing.assert_array_equal(table.cpu().numpy(), m_table)
        np.testing.assert_array_equal(lens.cpu().numpy(), np.asarray(m_lens))
        np.testing.assert_array_equal(slots.cpu().numpy(), m_slots)
        np.testing.assert_array_equal(seq_idx.cpu().numpy(), m_seq)
        np.testing.assert_array_equal(pos.cpu().numpy(), m_pos)
        assert int(free.item()) == m_free and (int(st.item()) in err if err else int(st.item()) == 0)
    assert m_free < B                              # the last steps were refused for some
    st.zero_()
    lib.mla_release_blocks(dims, i32([1] * B), lens, None, None, table, num_blocks, dfl, free, lens, free, st)
    torch.cuda.synchronize()
    assert int(free.item()) == num_blocks and int(st.item()) == 0 and not lens.any()
    assert sorted(dfl.cpu().tolist()) == list(range(num_blocks))


# ---------------------------------------------------------------- host checks (CPU)
def _plan_rc(mla, **over):
    d = mla.make_dims(16, 512, 64, 128, 128, 7168, 64, "bf16")
    P = ctypes.c_void_p
    f = P(0x1000)
    a = dict(dims=ctypes.byref(d), B=4, cached=f, new=f, G=1, offs=f, lens=f, pt=f, mpb=4, fl=f, cap=10, fc=f, bt=f, mb=8,
             nb=20, T=16, sl=f, cu=f, seq=f, pos=f, slots=f, out=f, st=None, stream=None)
    a.update(over)
    return mla._lib.mla_plan_step(*a.values())


def test_plan_host_refusals():
    import mla_latent_kv_40_b200 as mla
    bad = [dict(dims=None), dict(B=0), dict(G=-1), dict(G=5), dict(mb=0), dict(nb=0), dict(cap=-1), dict(T=-1), dict(mpb=-1),
           dict(cached=None), dict(new=None), dict(offs=None), dict(lens=None), dict(pt=None), dict(fl=None), dict(fc=None),
           dict(bt=None), dict(sl=None), dict(cu=None), dict(seq=None), dict(pos=None), dict(out=None)]
    for over in bad:
        assert _plan_rc(mla, **over) == -1, over
    assert _plan_rc(mla, B=8193, G=1) == -2


def test_release_host_refusals():
    import mla_latent_kv_40_b200 as mla
    d = mla.make_dims(16, 512, 64, 128, 128, 7168, 64, "bf16")
    f = ctypes.c_void_p(0x1000)
    base = dict(dims=ctypes.byref(d), B=4, done=f, lens=f, G=1, offs=f, pl=f, bt=f, mb=8, nb=20, fl=f, cap=10, fc=f, out=f,
                fout=f, st=None, stream=None)
    for over in [dict(dims=None), dict(B=0), dict(G=-1), dict(G=5), dict(mb=0), dict(nb=0), dict(cap=-1), dict(done=None),
                 dict(lens=None), dict(offs=None), dict(pl=None), dict(bt=None), dict(fl=None), dict(fc=None),
                 dict(out=None), dict(fout=None)]:
        assert mla._lib.mla_release_blocks(*{**base, **over}.values()) == -1, over
    assert mla._lib.mla_release_blocks(*{**base, "B": 8193}.values()) == -2


def test_no_blocks_status_string():
    import mla_latent_kv_40_b200 as mla
    assert mla.STATUS[-8] == "MLA_ERR_NO_BLOCKS" and "block" in mla.mla_status_string(-8)


def test_model_serves_in_order_until_the_list_ends():
    """The model itself, by hand: blocks of 4, three free; request 1 needs two, request 2 two (refused), request 3 none."""
    table, lens, cu, seq, pos, slots, left, err = model_plan(
        4, [3, 4, 0, 1], [1, 8, 5, 2], None, None, None, np.array([7, 5, 9]), 3,
        np.array([[2, -1, -1], [0, -1, -1], [-1, -1, -1], [6, -1, -1]]), 10, 16)
    assert table.tolist() == [[2, -1, -1], [0, 9, 5], [-1, -1, -1], [6, -1, -1]]
    assert lens == [4, 12, 0, 3] and cu == [0, 1, 9, 14, 16] and left == 1 and err == {-8}
    assert seq.tolist() == [0] + [1] * 8 + [-1] * 5 + [3, 3]
    assert slots.tolist() == [11, 36, 37, 38, 39, 20, 21, 22, 23] + [-1] * 5 + [25, 26]
