"""mla_decode_shared row by row where the running maximum moves most, and plans that do not fit into shared memory."""
import numpy as np
import pytest
import torch

import oracle
from test_shared_parity import Call, _heads, _shifted, check, make_shared, some


@pytest.mark.gpu
@pytest.mark.parametrize("heads,n_q,layout", [(16, 1, 1), (128, 1, 1), (64, 2, 0)])
def test_shared_every_row_of_peaked_scores(lib, heads, n_q, layout):
    """Scores N(0, 39^2), so that one key takes nearly all the weight of a row and the reference maximum moves again and
    again; queries that the absorption leaves exact (W_UK repeats the identity, no RoPE part), so that every row has a bound:

    * a score is 36 fp32 MMAs of 16 products: with partial sums up to A (in units of the score, after the scale) it is off by at
      most d = 600 * 2^-23 * A (a truncated addition per product), and a weight by 2 d of itself after the division by the sum;
    * a weight is rounded to bf16 (2^-9 of it; the row sum is not), the output likewise (2^-9 of it);
    * o_lat reaches W_UV with 16 bits, 512 products in fp32 (2^-17 and 512 * 2^-24 of the sum of magnitudes: 2^-14 together).
    """
    dims = _heads(heads)
    inp = make_shared(dims, [(640, [700, 650, 900, 641 + n_q, 1100, 800, 777, 690]), (64, [300, 70])], n_q, 64, seed=9, spread=24.0)
    inp["w_uk"] = torch.eye(128).repeat(4, 1).expand(heads, 512, 128).contiguous().to(torch.bfloat16)
    inp["q_pe"].zero_()
    c = Call(lib, inp, layout)
    c.run()
    out, lse, st = c.result()
    assert st == 0
    w_uv = inp["w_uv"].double().numpy()
    scale, decided, rows = 192 ** -0.5, 0, 0
    for b in range(out.shape[0]):
        S = int(inp["seqlens"][b])
        keys = oracle.gather_rows(inp["pool"], inp["block_table"], 64, b, S)[:, :512]
        q = np.tile(inp["q_nope"][b].double().numpy(), 4)   # [n_q, H, 512]
        for j in range(n_q):
            seen = keys[:S - n_q + j + 1]
            A = np.abs(np.cumsum((q[j][:, None, :] * seen[None, :64] * scale).reshape(heads, -1, 32, 16).sum(-1), -1)).max() * 2
            d = 600 * 2.0 ** -23 * A
            z = scale * q[j] @ seen.T
            top = z.max(1, keepdims=True)
            p = np.exp(z - top)
            L = p.sum(1, keepdims=True)
            p /= L
            decided += int((np.sort(z, 1)[:, -1] - np.sort(z, 1)[:, -2] > 8).sum())
            rows += heads
            want = np.einsum("hc,hcv->hv", p @ seen, w_uv)
            spread = np.einsum("hc,hcv->hv", p @ np.abs(seen), np.abs(w_uv))   # sum of p |c| |W|
            bound = (2 * d + 2.0 ** -9 + 2.0 ** -14) * spread + 2.0 ** -9 * np.abs(want)
            err = np.abs(out[b, j] - want)
            assert (err <= bound).all(), (b, j, float((err / bound).max()))
            # exp2 and log2 of the library are good to a few 2^-22; lse itself is rounded to fp32
            assert (np.abs(lse[b, j] - (top + np.log(L))[:, 0]) <= d + 2.0 ** -20 + 2.0 ** -23 * np.abs(top[:, 0])).all()
    assert decided > rows // 4


def _plan_bytes(B, heads, groups):
    """What the plan of B sequences of one query token works on (shared_plan_words)."""
    unit_rows = 256 if heads >= 8 else 32 * heads
    units = B * heads // unit_rows + groups
    return 4 * (3 * B + 1 + 4 * units + 1 + 3 * groups + 2)


@pytest.mark.gpu
@pytest.mark.parametrize("B,G,shift", [(4000, 2000, False), (6000, 4000, True)])
def test_shared_plan_outside_shared_memory(lib, B, G, shift):
    """As a block of the absorption the plan has the 50,176 bytes of its operand tiles, as a launch of its own (queries at
    odd addresses) up to 160 KB; beyond that it works in the workspace."""
    assert _plan_bytes(B, 2, G) > (160 * 1024 if shift else 50176)
    r = np.random.default_rng(B)
    bounds = np.concatenate(([0], np.sort(r.integers(0, B + 1, G - 1)), [B]))
    groups = [(int(r.integers(0, 2)) * 64, [int(x) for x in r.integers(1, 90, b - a)]) for a, b in zip(bounds, bounds[1:])]
    inp = make_shared(_heads(2), groups, 1, 64, seed=B)
    c = Call(lib, inp)
    if shift:
        for k in ("q_nope", "q_pe", "w_uk"):
            c.dev[k] = _shifted(c.dev[k])
    c.run()
    first = c.result()
    check(inp, first, some(inp, 60, 2))
    c.out.fill_(float("nan"))
    c.ws.fill_(0x7F)
    torch.cuda.synchronize()
    c.run()
    again = c.result()
    assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])
