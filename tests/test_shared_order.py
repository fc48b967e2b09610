"""What one CTA of the shared decode's clusters stores and another one's MMAs or copies use: RoPE queries, tidied pages, the
slots that the epilogue borrows, and the slots' way round.  Each would show as other bits in some call of many."""
import numpy as np
import pytest
import torch

from test_shared_parity import Call, _heads, check, make_shared, some


def again_and_again(calls, times):
    """The calls in turn, many times over, against the bits that each had with the device at rest."""
    want = []
    for c in calls:
        c.run()
        want.append(c.result())
    for _ in range(times):
        for c in calls:
            c.out.fill_(float("nan"))
            c.run()
        for c, (o, l, _) in zip(calls, want):
            got, lse, st = c.result()
            assert st == 0 and np.array_equal(got, o) and np.array_equal(lse, l)


@pytest.mark.gpu
@pytest.mark.parametrize("heads,layout", [(16, 1), (128, 1), (128, 0)])
def test_shared_rope_queries_of_every_unit(lib, heads, layout):
    """Scores from the RoPE part alone, three units a cluster and other queries in every unit and call: a unit that met the
    queries of the one before it would have other scores."""
    n = 100 * 256 // heads
    calls = []
    for seed in (61, 62):
        inp = make_shared(_heads(heads), [(192, [193 + i % 60 for i in range(n)])], 1, 64, seed=seed)
        inp["q_nope"].zero_()
        inp["q_pe"] *= 3
        calls.append(Call(lib, inp, layout))
        calls[-1].run()
        check(inp, calls[-1].result(), some(inp, 8, 2))
    again_and_again(calls, 40)


@pytest.mark.gpu
@pytest.mark.parametrize("heads,layout", [(16, 1), (64, 0), (128, 1)])
def test_shared_tidied_pages(lib, heads, layout):
    """Every page of own keys ends inside (NaN behind the last key), page after page: a page that reached the MMAs untidied
    would make every row of its unit NaN."""
    n = 60 * 256 // heads
    calls = [Call(lib, make_shared(_heads(heads), [(64 * (seed % 3), [64 * (seed % 3) + 1 + (7 * i) % 63 for i in range(n)])], 1, 64,
                                   seed=seed), layout) for seed in (64, 65, 66)]
    for c in calls:
        c.run()
        check(c.inp, c.result(), some(c.inp, 8, 2))
    again_and_again(calls, 40)


@pytest.mark.gpu
@pytest.mark.parametrize("pages", [1, 2, 3, 4, 5, 6, 7, 11, 12])
def test_shared_short_runs(lib, pages):
    """Some five units a cluster of so many pages each, in one launch: fewer, as many and more than P has slots and staging
    tiles."""
    inp = make_shared(_heads(128), [(64 * pages, [64 * pages] * 330)], 1, 64, seed=pages)
    inp["prefix_lens"] += 64   # (the last query token sees the whole of the last page)
    c = Call(lib, inp)
    c.run()
    check(inp, c.result(), some(inp, 6, 2))
    again_and_again([c], 10)


@pytest.mark.gpu
def test_shared_runs_of_mixed_lengths(lib):
    """Runs of one to nine pages after one another on every cluster."""
    r = np.random.default_rng(8)
    groups = [(0, [int(x)]) for x in r.integers(1, 9 * 64, 400)]
    calls = [Call(lib, make_shared(_heads(h), groups, 1, 64, seed=h)) for h in (128, 256)]
    for c in calls:
        c.run()
        check(c.inp, c.result(), some(c.inp, 12, 2))
    again_and_again(calls, 10)


def _slots_in_order(runs, rng, seen_barrier):
    """A model of the value CTA's P slots over runs of so many pages: the sender fills freed slots in order, the MMAs of a page
    follow its P, the slots' thread frees a page's slot when it has seen its MMAs' phase (by parity, as an mbarrier is waited
    for), but a run's last two pages' slots are freed by the issuing warp once the run's epilogue is through.  Threads move in
    random order.  True if every page gets through; False if nobody can move on."""
    slots = 5
    last = [r >= 2 and i >= r - 2 for r in runs for i in range(r)]
    end_of = [i == r - 1 for r in runs for i in range(r)]
    first_of = [i == 0 for r in runs for i in range(r)]
    run_of = [k for k, r in enumerate(runs) for _ in range(r)]
    total = len(last)
    freed = [0] * slots          # phases of "may be written"
    done = [0] * slots           # phases of "its MMAs are complete"
    sent = issued = watched = seen_runs = 0

    def send():
        nonlocal sent
        q, s = sent // slots, sent % slots
        if sent < total and (q == 0 or freed[s] >= q):
            sent += 1
            return True
        return False

    def issue():
        nonlocal issued
        if issued >= total or issued >= sent:
            return False
        if first_of[issued] and issued > 0:
            if seen_barrier and seen_runs < run_of[issued]:
                return False
            n = runs[run_of[issued] - 1]
            if n >= 2:
                for page in (issued - 2, issued - 1):
                    freed[page % slots] += 1
        done[issued % slots] += 1
        issued += 1
        return True

    def watch():
        nonlocal watched, seen_runs
        if watched >= total:
            return False
        if done[watched % slots] % 2 != (watched // slots + 1) % 2:   # the phase of this parity is not the last one completed
            return False
        if not last[watched]:
            freed[watched % slots] += 1
        if end_of[watched]:
            seen_runs += 1
        watched += 1
        return True

    while watched < total:
        moves = [send, issue, watch]
        rng.shuffle(moves)
        if rng.random() < 0.7:      # the slots' thread is held up
            moves.sort(key=lambda f: f is watch)
        if not any(f() for f in moves):
            return False
    return True


def test_slots_of_the_value_side_go_round_whoever_is_late():
    """The protocol of B_PVDONE, B_PEMPTY and B_RUNSEEN on the CPU, with a thread that is held up: every page gets through.
    Without the last of the three the parity is lapped in some of these orders."""
    import random
    lapped = 0
    for seed in range(400):
        rng = random.Random(seed)
        runs = [rng.randint(1, 9) for _ in range(12)]
        assert _slots_in_order(runs, random.Random(seed), True), (seed, runs)
        lapped += not _slots_in_order(runs, random.Random(seed), False)
    assert lapped > 0
