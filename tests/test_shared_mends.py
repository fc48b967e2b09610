"""mla_decode_shared, mla_plan_step and mla_release_blocks at the ends of their ranges: lengths that are no lengths, plans
that do not fit into shared memory, idle requests, rows past 2^31."""
import numpy as np
import pytest
import torch

from helpers import check_close
from test_shared_parity import Call, V2L, make_shared, reference, some

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
