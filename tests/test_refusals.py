"""Addresses that the tensor-core decode cannot copy 16 bytes at a time from or to are refused before anything is launched
(host checks on made-up addresses: nothing may be read or run for these answers)."""
import ctypes

import pytest
import torch

INVALID, UNSUPPORTED = -1, -2
P = ctypes.c_void_p
GOOD, ODD, WS = P(0x100000), P(0x100002), P(0x200000)
BIG = ctypes.c_size_t(1 << 40)


def _call(entry, layout, **over):
    import mla_latent_kv_40_b200 as mla
    d = mla.make_dims(16, 512, 64, 128, 128, 2048, 64, "bf16", cache_layout=layout)
    a = dict(c_kv=GOOD, k_pe=GOOD, w_uv=GOOD, out=GOOD)
    a.update(over)
    q, cache = (4, 1, GOOD, GOOD, a["c_kv"], a["k_pe"]), (GOOD, 4, 20, GOOD, 200)
    tail = (None, WS, BIG, None, None)
    lib, ref = mla._lib, ctypes.byref(d)
    if entry == "decode":
        return lib.mla_decode(ref, *q, *cache, GOOD, a["w_uv"], a["out"], *tail)
    if entry == "latent":
        return lib.mla_decode_latent(ref, *q, *cache, GOOD, a["out"], *tail)
    if entry == "partial":
        return lib.mla_decode_partial(ref, *q, *cache, 0, 128, GOOD, a["out"], GOOD, WS, BIG, None, None)
    if entry == "step":
        return lib.mla_decode_step(ref, 4, 1, *([GOOD] * 4), GOOD, GOOD, a["c_kv"], a["k_pe"], *cache, GOOD, a["w_uv"], a["out"], *tail)
    if entry == "shared":
        return lib.mla_decode_shared(ref, *q, *cache, 2, GOOD, GOOD, GOOD, a["w_uv"], a["out"], *tail)
    if entry == "shared without groups":
        return lib.mla_decode_shared(ref, *q, *cache, 0, None, None, GOOD, a["w_uv"], a["out"], *tail)
    if entry == "sparse":
        return lib.mla_decode_sparse(ref, *q, *cache, GOOD, 64, GOOD, a["w_uv"], a["out"], *tail)
    return lib.mla_decode_absorbed(ref, 512, 4, 1, GOOD, GOOD, GOOD, GOOD, a["c_kv"], a["k_pe"], *cache, GOOD, a["out"], *tail)


ENTRIES = ["decode", "latent", "partial", "step", "shared", "shared without groups", "sparse", "absorbed"]


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("entry", ENTRIES)
def test_odd_addresses_are_refused_before_anything_is_launched(entry, layout):
    if entry != "absorbed":   # (its output is a product of its own, at any address)
        assert _call(entry, layout, out=ODD) == UNSUPPORTED
    if entry in ("decode", "step", "shared", "shared without groups", "sparse"):
        assert _call(entry, layout, w_uv=ODD) == UNSUPPORTED
    pool = UNSUPPORTED if entry == "sparse" else INVALID   # (the gather copies whole 16-byte groups)
    assert _call(entry, layout, c_kv=ODD) == pool
    if layout == 0:
        assert _call(entry, layout, k_pe=ODD) == pool


@pytest.mark.gpu
def test_a_refused_step_leaves_the_cache_alone(lib):
    """mla_decode_step appends first: with an output that it cannot write, it must not have."""
    from test_stream_order import Step
    s = Step(lib, 1)
    odd = torch.empty(s.out.numel() + 1, dtype=s.out.dtype, device="cuda")
    s.out = odd[1:].view(s.out.shape)
    before = s.pool.clone()
    with pytest.raises(lib.MlaError):
        s.call("step")
    torch.cuda.synchronize()
    assert torch.equal(s.pool, before) and int(s.status.item()) == 0
