"""What one CTA of the shared decode's clusters stores and another one's MMAs or copies use: RoPE queries, tidied pages, the
slots that the epilogue borrows.  Each would show as other bits in some call of many."""
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
