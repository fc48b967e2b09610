"""Measured cases of the shared-prefix operators: decode over a shared prefix, and the paged-cache bookkeeping around it.

Three operators of the library, used together by a serving loop:

* ``plan``: block tables, sequence lengths and slot maps of a step, from the requests' lengths (``mla_plan_step``);
* ``decode``: one decode step of a batch whose groups of sequences share the first tokens of the cache
  (``mla_decode_shared``);
* ``release``: the blocks of finished requests go back to the free list (``mla_release_blocks``).

``run`` computes each in plain torch (32 bits, elementary operations) or, where ``own`` is true, calls the library.
``exact`` computes the decode from its definition in 64 bits (keys and values decompressed per head) and the
bookkeeping request by request on the host.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

D_C, D_ROPE, D_NOPE, D_V, D_MODEL = 512, 64, 128, 128, 7168   # latent, RoPE, per-head key and value widths, hidden width
W = D_C + D_ROPE
ROPE_BASE = 10000.0
SCALE = 1.0 / math.sqrt(D_NOPE + D_ROPE)


# ------------------------------------------------------------------------------------------------ cases
def listed():
    def decode(name, heads, batch, n_q, groups, prefix, tail_lo, tail_hi, block, tiled, ragged, layout):
        return dict(name=name, op="decode", heads=heads, batch=batch, n_q=n_q, groups=groups, prefix=prefix,
                    tail_lo=tail_lo, tail_hi=tail_hi, block=block, tiled=tiled, ragged=ragged, layout=layout)

    def plan(name, batch, groups, prefix, block, cached_hi, new_lo, new_hi, grow, join, short, layout):
        return dict(name=name, op="plan", batch=batch, groups=groups, prefix=prefix, block=block, cached_hi=cached_hi,
                    new_lo=new_lo, new_hi=new_hi, grow=grow, join=join, short=short, layout=layout)

    def release(name, batch, groups, prefix, block, len_hi, done, layout):
        return dict(name=name, op="release", batch=batch, groups=groups, prefix=prefix, block=block, len_hi=len_hi,
                    done=done, layout=layout)

    return [
        # Two answers drawn from one short prompt, 16 heads: the smallest call, where latency counts.
        decode("decode_h16_b2_p512", 16, 2, 1, 1, 512, 1, 64, 64, True, False, 1),
        # A chat batch under one system prompt, 16 heads (one rank of a head-split model).
        decode("decode_h16_b32_p2048", 16, 32, 1, 1, 2048, 1, 512, 64, True, False, 2),
        # The same at 128 heads and 64 sequences, answers up to 512 tokens behind 4096 shared ones.
        decode("decode_h128_b64_p4096", 128, 64, 1, 1, 4096, 1, 512, 64, True, False, 3),
        # Several prompts in one batch, groups of unequal size, some sequences alone, two query tokens (one drafted),
        # row pool with 128-token blocks.
        decode("decode_h128_b48_groups", 128, 48, 2, 7, 8192, 2, 1024, 128, False, True, 4),
        # Many samples behind one long document: the largest.
        decode("decode_h128_b128_p32768", 128, 128, 1, 1, 32768, 64, 1024, 64, True, False, 5),
        # A decode step: every request grows by one token.
        plan("plan_b64_grow", 64, 1, 4096, 64, 4096, 1, 1, 1.0, 0.0, False, 6),
        # Continuous batching: most requests grow by two tokens, some join behind a shared prompt with their own text.
        plan("plan_b256_mixed", 256, 6, 8192, 64, 8192, 16, 1024, 0.8, 0.15, False, 7),
        # A prompt-heavy step of many requests, with too few free blocks for the last ones: the largest.
        plan("plan_b4096_prompts", 4096, 32, 4096, 16, 2048, 4, 32, 0.3, 0.5, True, 8),
        # A few finished requests.
        release("release_b64", 64, 1, 4096, 64, 8192, 0.1, 9),
        # Half of a large batch is cancelled.
        release("release_b4096", 4096, 32, 4096, 16, 8192, 0.5, 10),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    layout = rng.randrange(1 << 30)
    op = rng.choice(["decode", "decode", "decode", "plan", "release"])
    if op == "decode":
        heads = rng.choice([16, 16, 20, 32, 64, 128, 128])
        n_q = rng.choice([1, 1, 2, 4]) if heads <= 64 else rng.choice([1, 1, 2])
        batch = _log_int(rng, 1, 128)
        block = rng.choice([64, 64, 128])
        groups = rng.choice([1, 1, min(batch, rng.randint(2, 9))])
        prefix = _log_int(rng, 1, 16384 // block) * block
        tail_hi = _log_int(rng, n_q, 1024)
        return dict(op=op, heads=heads, batch=batch, n_q=n_q, groups=groups, prefix=prefix,
                    tail_lo=rng.randint(n_q, tail_hi), tail_hi=tail_hi, block=block, tiled=rng.random() < 0.7,
                    ragged=rng.random() < 0.5, layout=layout)
    batch = _log_int(rng, 1, 4096)
    block = rng.choice([16, 64, 64, 128])
    groups = rng.randint(1, min(batch, 40))
    prefix = _log_int(rng, 1, 4096 // block) * block
    if op == "plan":
        new_lo = _log_int(rng, 1, 16)
        return dict(op=op, batch=batch, groups=groups, prefix=prefix, block=block, cached_hi=_log_int(rng, 1, 2048),
                    new_lo=new_lo, new_hi=new_lo + _log_int(rng, 1, max(2, min(4096, 65536 // batch))),
                    grow=rng.choice([0.0, 0.3, 0.9, 1.0]), join=rng.choice([0.0, 0.1, 0.5]),
                    short=rng.random() < 0.25, layout=layout)
    return dict(op=op, batch=batch, groups=groups, prefix=prefix, block=block, len_hi=_log_int(rng, 1, 8192),
                done=rng.choice([0.02, 0.1, 0.5, 1.0]), layout=layout)


def _groups(case, rng):
    """Offsets of the groups and their prefix lengths (whole blocks).  Ragged groups: unequal sizes, some prefixes
    short or absent."""
    B, G, bs = case["batch"], case["groups"], case["block"]
    cuts = sorted(rng.sample(range(1, B), G - 1)) if G > 1 else []
    offsets = [0] + cuts + [B]
    most = case["prefix"] // bs
    prefixes = [most * bs]
    for _ in range(G - 1):
        prefixes.append((rng.choice([0, 1, rng.randint(0, most), most]) if case.get("ragged", True) else most) * bs)
    rng.shuffle(prefixes)
    return offsets, prefixes


def _decode_shape(case):
    rng = random.Random(case["layout"])
    offsets, prefixes = _groups(case, rng)
    tails = [rng.randint(case["tail_lo"], case["tail_hi"]) for _ in range(case["batch"])]
    return offsets, prefixes, tails


def _plan_shape(case):
    """Per request (own cached tokens behind the prefix, new tokens); own = 0 joins behind its group's prefix."""
    rng = random.Random(case["layout"])
    offsets, prefixes = _groups(case, rng)
    recs = []
    for _ in range(case["batch"]):
        x = rng.random()
        if x < case["grow"]:
            recs.append((rng.randint(1, case["cached_hi"]), rng.choice([1, 1, 2])))
        elif x < case["grow"] + case["join"]:
            recs.append((0, rng.randint(case["new_lo"], case["new_hi"])))
        else:   # a prompt in parts, or a request that waits
            recs.append((rng.randint(1, case["cached_hi"]), rng.choice([0, rng.randint(case["new_lo"], case["new_hi"])])))
    return offsets, prefixes, recs


def _release_shape(case):
    rng = random.Random(case["layout"])
    offsets, prefixes = _groups(case, rng)
    recs = [(rng.randint(0, case["len_hi"]), rng.random() < case["done"]) for _ in range(case["batch"])]
    return offsets, prefixes, recs


def _cdiv(a, b):
    return (a + b - 1) // b


def work(case):
    B, bs = case["batch"], case["block"]
    if case["op"] == "decode":
        offsets, prefixes, tails = _decode_shape(case)
        H, n_q = case["heads"], case["n_q"]
        # Rows of the cache, weights and queries once, outputs once, the block ids of every sequence's own blocks and
        # of each prefix once.
        rows = sum(prefixes) + sum(tails)
        blocks = sum(p // bs for p in prefixes) + sum(_cdiv(t, bs) for t in tails)
        bytes_ = (rows * W * 2 + H * D_C * (D_NOPE + D_V) * 2 + B * n_q * H * (D_NOPE + D_ROPE + D_V) * 2 +
                  4 * (blocks + B + 2 * len(prefixes) + 1))
        # Latent form per (row, key): 2 (576 + 512).  Decompressing a prefix key for one head costs 2 * 512 * 256 once
        # and 2 (192 + 128) per row: counted where it is less (more than 170 query tokens behind one prefix).
        flops = 2 * B * n_q * H * D_C * (D_NOPE + D_V)
        for g, p in enumerate(prefixes):
            nt = (offsets[g + 1] - offsets[g]) * n_q
            latent = nt * 2 * (W + D_C)
            plain = 2 * D_C * (D_NOPE + D_V) + nt * 2 * (D_NOPE + D_ROPE + D_V)
            flops += p * H * min(latent, plain)
        for t in tails:   # causal among the new tokens
            flops += 2 * (W + D_C) * H * sum(t - n_q + j + 1 for j in range(n_q))
        return {"bytes": bytes_, "flops": flops}
    if case["op"] == "plan":
        offsets, prefixes, recs = _plan_shape(case)
        T = sum(n for _, n in recs)
        need = sum(_cdiv(o + n, bs) - _cdiv(o, bs) for o, n in recs)
        joins = sum(o == 0 for o, _ in recs) / B
        copied = joins * sum((offsets[g + 1] - offsets[g]) * (p // bs) for g, p in enumerate(prefixes))
        copied_in = min(copied, sum(p // bs for p in prefixes))
        part = sum(o % bs != 0 and n > 0 for o, n in recs)   # the table entry of a partly filled block
        return {"bytes": int(T * 16 + need * 8 + copied * 4 + copied_in * 4 + part * 4 + B * 16 + 8 * len(prefixes) + 12),
                "flops": int(T + need + 4 * B)}
    _, prefixes, recs = _release_shape(case)
    ids = sum(_cdiv(o, bs) for o, d in recs if d)
    return {"bytes": ids * 8 + B * 12 + 8 * len(prefixes) + 12, "flops": ids + 2 * B}


# ------------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    return {"decode": _prepare_decode, "plan": _prepare_plan, "release": _prepare_release}[case["op"]](case, seed)


def _prepare_decode(case, seed):
    H, B, n_q, bs = case["heads"], case["batch"], case["n_q"], case["block"]
    offsets, prefixes, tails = _decode_shape(case)
    host = random.Random(seed)
    host.shuffle(tails)
    need = sum(p // bs for p in prefixes) + sum(_cdiv(t, bs) for t in tails)
    num_blocks = need + 3
    ids = list(range(num_blocks))
    host.shuffle(ids)
    mb = max(_cdiv(prefixes[g] + tails[b], bs) for g in range(len(prefixes)) for b in range(offsets[g], offsets[g + 1]))
    table = np.full((B, mb), -1, np.int32)
    seqlens, k = [], 0
    for g, p in enumerate(prefixes):
        shared = ids[k:k + p // bs]
        k += p // bs
        for b in range(offsets[g], offsets[g + 1]):
            n = _cdiv(tails[b], bs)
            table[b, :p // bs] = shared
            table[b, p // bs:p // bs + n] = ids[k:k + n]
            k += n
            seqlens.append(p + tails[b])
    gen = _gen(seed)

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(torch.bfloat16)

    rows = randn(num_blocks * bs, W)
    s = dict(case=case, offsets=offsets, prefixes=prefixes, seqlens_host=seqlens, num_blocks=num_blocks, max_blocks=mb,
             max_seqlen=max(seqlens), pool=_to_tiles(rows) if case["tiled"] else rows,
             table=torch.from_numpy(table).cuda(), seqlens=_i32(seqlens), group_offsets=_i32(offsets),
             prefix_lens=_i32(prefixes), q_nope=randn(B, n_q, H, D_NOPE), q_pe=randn(B, n_q, H, D_ROPE),
             w_uk=randn(H, D_C, D_NOPE, scale=D_C ** -0.5), w_uv=randn(H, D_C, D_V, scale=D_C ** -0.5))
    if own:
        import mla_latent_kv_40_b200 as mla
        s["mla"] = mla
        s["dims"] = mla.make_dims(H, D_C, D_ROPE, D_NOPE, D_V, D_MODEL, bs, "bf16",
                                  cache_layout=mla.MLA_CACHE_TILED if case["tiled"] else mla.MLA_CACHE_ROWS)
        s["out"] = torch.empty(B, n_q, H, D_V, dtype=torch.bfloat16, device="cuda")
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["ws"] = mla.alloc_workspace(mla.mla_decode_shared_workspace_size(s["dims"], B, n_q, s["max_seqlen"],
                                                                           len(prefixes)))
    return s


def _to_tiles(rows):
    """Row pool -> pages of 64 tokens, [page][64-dim chunk][token][8 groups of 8 dims], group g of token t at g ^ (t % 8)."""
    x = rows.view(-1, 64, W // 64, 8, 8).permute(0, 2, 1, 3, 4)
    t = torch.arange(64, device=rows.device)
    g = torch.arange(8, device=rows.device)
    src = (g[None, :] ^ (t[:, None] % 8)).view(1, 1, 64, 8, 1).expand(x.shape)
    return torch.gather(x, 3, src).reshape(rows.shape).contiguous()


def _prefix_tables(prefixes, bs, ids, k):
    mpb = max(1, max(p // bs for p in prefixes))
    pt = np.full((len(prefixes), mpb), -1, np.int32)
    for g, p in enumerate(prefixes):
        pt[g, :p // bs] = ids[k:k + p // bs]
        k += p // bs
    return pt, mpb, k


def _prepare_plan(case, seed):
    B, bs = case["batch"], case["block"]
    offsets, prefixes, recs = _plan_shape(case)
    host = random.Random(seed)
    host.shuffle(recs)
    gid = [g for g in range(len(prefixes)) for _ in range(offsets[g], offsets[g + 1])]
    need = sum(_cdiv(o + n, bs) - _cdiv(o, bs) for o, n in recs)
    free = max(0, need * 9 // 10) if case["short"] else need + 7
    held = sum(p // bs for p in prefixes) + sum(_cdiv(o, bs) for o, _ in recs)
    num_blocks = held + need + 7
    ids = np.random.default_rng(seed).permutation(num_blocks).astype(np.int32)
    pt, mpb, k = _prefix_tables(prefixes, bs, ids, 0)
    cached = [prefixes[gid[b]] + recs[b][0] for b in range(B)]
    new = [n for _, n in recs]
    mb = max(prefixes) // bs + max(_cdiv(o + n, bs) for o, n in recs) + 1
    table = np.full((B, mb), -1, np.int32)
    for b in range(B):
        p, o = prefixes[gid[b]] // bs, recs[b][0]
        if o:
            table[b, :p] = pt[gid[b], :p]
            n = _cdiv(o, bs)
            table[b, p:p + n] = ids[k:k + n]
            k += n
    free_list = np.full(num_blocks, -1, np.int32)
    free_list[:free] = ids[k:k + free]
    T = sum(new)
    s = dict(case=case, offsets=offsets, prefixes=prefixes, num_blocks=num_blocks, max_blocks=mb, mpb=mpb, T=T,
             cached=_i32(cached), new=_i32(new), group_offsets=_i32(offsets), prefix_lens=_i32(prefixes),
             prefix_table=torch.from_numpy(pt).cuda(), free_list=torch.from_numpy(free_list).cuda(),
             free_count=_i32([free]), table=torch.from_numpy(table).cuda(), gid=torch.tensor(gid, device="cuda"))
    if own:
        import mla_latent_kv_40_b200 as mla
        s["mla"] = mla
        s["dims"] = mla.make_dims(16, D_C, D_ROPE, D_NOPE, D_V, D_MODEL, bs, "bf16")
        s["out"] = dict(seqlens=_i32([0] * B), cu=_i32([0] * (B + 1)), seq_idx=torch.full((T,), -1, dtype=torch.int32, device="cuda"),
                        pos=torch.full((T,), -1, dtype=torch.int32, device="cuda"),
                        slots=torch.full((T,), -1, dtype=torch.int64, device="cuda"), free_count=_i32([0]),
                        status=_i32([0]))
    return s


def _prepare_release(case, seed):
    B, bs = case["batch"], case["block"]
    offsets, prefixes, recs = _release_shape(case)
    host = random.Random(seed)
    host.shuffle(recs)
    gid = [g for g in range(len(prefixes)) for _ in range(offsets[g], offsets[g + 1])]
    held = sum(p // bs for p in prefixes) + sum(_cdiv(o, bs) for o, _ in recs)
    free = 13   # already free
    num_blocks = held + free
    ids = np.random.default_rng(seed).permutation(num_blocks).astype(np.int32)
    pt, _, k = _prefix_tables(prefixes, bs, ids, 0)
    lens = [prefixes[gid[b]] + recs[b][0] for b in range(B)]
    mb = max(1, max(_cdiv(n, bs) for n in lens))
    table = np.full((B, mb), -1, np.int32)
    for b in range(B):
        p, n = prefixes[gid[b]] // bs, _cdiv(recs[b][0], bs)
        table[b, :p] = pt[gid[b], :p]
        table[b, p:p + n] = ids[k:k + n]
        k += n
    free_list = np.full(num_blocks, -1, np.int32)
    free_list[:free] = ids[k:k + free]
    s = dict(case=case, offsets=offsets, prefixes=prefixes, num_blocks=num_blocks, max_blocks=mb,
             done=_i32([int(d) for _, d in recs]), seqlens=_i32(lens), group_offsets=_i32(offsets),
             prefix_lens=_i32(prefixes), free_list=torch.from_numpy(free_list).cuda(), free_count=_i32([free]),
             table=torch.from_numpy(table).cuda(), gid=torch.tensor(gid, device="cuda"))
    if own:
        import mla_latent_kv_40_b200 as mla
        s["mla"] = mla
        s["dims"] = mla.make_dims(16, D_C, D_ROPE, D_NOPE, D_V, D_MODEL, bs, "bf16")
        s["out"] = dict(seqlens=_i32([0] * B), free_count=_i32([0]), status=_i32([0]))
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    if own:
        return {"decode": _own_decode, "plan": _own_plan, "release": _own_release}[state["case"]["op"]](state)
    return {"decode": _plain_decode, "plan": _plain_plan, "release": _plain_release}[state["case"]["op"]](state)


def _own_decode(s):
    s["mla"].mla_decode_shared(s["dims"], s["q_nope"], s["q_pe"], s["pool"], None if s["case"]["tiled"] else s["pool"][:, D_C:],
                               s["table"], s["max_blocks"], s["num_blocks"], s["seqlens"], s["max_seqlen"],
                               s["group_offsets"], s["prefix_lens"], s["w_uk"], s["w_uv"], s["out"], None, s["ws"],
                               s["status"])
    return s["out"]


def _own_plan(s):
    o = s["out"]
    s["mla"].mla_plan_step(s["dims"], s["cached"], s["new"], s["group_offsets"], s["prefix_lens"], s["prefix_table"],
                           s["free_list"], s["free_count"], s["table"], s["num_blocks"], o["seqlens"], o["cu"],
                           o["seq_idx"], o["pos"], o["slots"], o["free_count"], o["status"])
    return s["table"], o["seqlens"], o["cu"], o["seq_idx"], o["pos"], o["slots"], o["free_count"]


def _own_release(s):
    o = s["out"]
    s["mla"].mla_release_blocks(s["dims"], s["done"], s["seqlens"], s["group_offsets"], s["prefix_lens"], s["table"],
                                s["num_blocks"], s["free_list"], s["free_count"], o["seqlens"], o["free_count"],
                                o["status"])
    return s["free_list"], o["seqlens"], o["free_count"]


def _cache_rows(s, blocks, n_tokens):
    """fp32 rows of the first n_tokens tokens held in `blocks` [..., n] (pool order undone)."""
    bs = s["case"]["block"]
    blocks = blocks.long()
    if s["case"]["tiled"]:
        pages = s["pool"].view(-1, W // 64, 64, 8, 8)
        per = bs // 64
        idx = (blocks[..., None] * per + torch.arange(per, device="cuda")).flatten(-2)
        x = pages[idx]                                             # [..., pages, chunk, token, group, 8]
        t, g = torch.arange(64, device="cuda"), torch.arange(8, device="cuda")
        src = (g[None, :] ^ (t[:, None] % 8)).view(64, 8, 1).expand(x.shape)
        x = torch.gather(x, x.dim() - 2, src).transpose(-3, -4)    # [..., pages, token, chunk, group, 8]
        x = x.reshape(*idx.shape[:-1], idx.shape[-1] * 64, W)
    else:
        x = s["pool"].view(-1, bs, W)[blocks].flatten(-3, -2)
    return x[..., :n_tokens, :].float()


def _rotate(x, pos):
    """RoPE in fp32 with angles formed in 64 bits: pairs (2i, 2i+1), theta_i = base^(-2i/d)."""
    theta = ROPE_BASE ** (-torch.arange(0, D_ROPE, 2, device="cuda", dtype=torch.float64) / D_ROPE)
    ang = pos.double()[..., None] * theta
    c, sn = torch.cos(ang).float()[..., None, :], torch.sin(ang).float()[..., None, :]
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * c - b * sn, a * sn + b * c), -1).flatten(-2)


def _plain_decode(s):
    """Latent form: q_lat = W_UK q_nope; the prefix logits of a group in one product, the tails' in batched ones; one
    softmax over both; o_lat = P C; out = o_lat W_UV."""
    case = s["case"]
    H, B, n_q, bs = case["heads"], case["batch"], case["n_q"], case["block"]
    pos = s["seqlens"].long()[:, None] - n_q + torch.arange(n_q, device="cuda")
    q = torch.cat((torch.einsum("bjhn,hcn->bjhc", s["q_nope"].float(), s["w_uk"].float()),
                   _rotate(s["q_pe"].float(), pos)), -1)
    q = q.reshape(B, n_q * H, W)
    out = []
    for g, p in enumerate(s["prefixes"]):
        b0, b1 = s["offsets"][g], s["offsets"][g + 1]
        tmax = max(s["seqlens_host"][b0:b1]) - p
        nb = _cdiv(tmax, bs)
        shared = _cache_rows(s, s["table"][b0, :p // bs], p)                                  # [p, W]
        tails = _cache_rows(s, s["table"][b0:b1, p // bs:p // bs + nb].clamp(min=0), tmax)    # [n, tmax, W]
        qg = q[b0:b1]
        z_tail = qg @ tails.transpose(1, 2) * SCALE
        key = torch.arange(tmax, device="cuda") + p
        seen = key <= pos[b0:b1, :, None]                                                     # [n, n_q, tmax]
        z_tail = z_tail.view(b1 - b0, n_q, H, tmax).masked_fill(~seen[:, :, None], float("-inf")).flatten(1, 2)
        z_pre = (qg.reshape(-1, W) @ shared.T * SCALE).view(b1 - b0, n_q * H, p)
        m = z_tail.amax(-1) if p == 0 else torch.maximum(z_tail.amax(-1), z_pre.amax(-1))
        e_tail, e_pre = torch.exp(z_tail - m[..., None]), torch.exp(z_pre - m[..., None])
        l = e_tail.sum(-1) + e_pre.sum(-1)
        o = e_tail @ tails[..., :D_C] + (e_pre.flatten(0, 1) @ shared[:, :D_C]).view(b1 - b0, n_q * H, D_C)
        out.append(o / l[..., None])
    o_lat = torch.cat(out).view(B, n_q, H, D_C)
    o = torch.einsum("bjhc,hcv->bjhv", o_lat, s["w_uv"].float())
    return o.to(torch.bfloat16)


def _plain_plan(s):
    bs, B, T = s["case"]["block"], s["case"]["batch"], s["T"]
    mb = s["max_blocks"]
    dev = "cuda"
    cached, new = s["cached"].long(), s["new"].long()
    P = s["prefix_lens"].long()[s["gid"]]
    fc = s["free_count"].long()
    cu = torch.cat((torch.zeros(1, dtype=torch.int64, device=dev), torch.cumsum(new, 0)))
    have = (cached + bs - 1) // bs
    need = (cached + new + bs - 1) // bs - have
    cum = torch.cumsum(need, 0)
    served = (need == 0) | (cum <= fc)
    taken = torch.where(served & (need > 0), cum, 0).amax().view(1)
    seqlens = torch.where(served, cached + new, cached)
    table = torch.cat((s["table"].flatten(), torch.zeros(1, dtype=torch.int32, device=dev)))   # last: writes to drop
    drop = B * mb
    k = torch.arange(s["free_list"].numel(), device=dev)
    b = torch.searchsorted(cum, k, right=True).clamp(max=B - 1)
    at = torch.where(k < taken, b * mb + have[b] + k - (cum[b] - need[b]), drop)
    table[at] = s["free_list"][(fc - 1 - k).clamp(min=0)]
    e = torch.arange(s["mpb"], device=dev)
    join = served & (cached == P) & (P > 0)
    at = torch.where(join[:, None] & (e < P[:, None] // bs), torch.arange(B, device=dev)[:, None] * mb + e, drop)
    table[at] = s["prefix_table"][s["gid"]]
    table = table[:drop].view(B, mb)
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(cu[1:], t, right=True)
    p = cached[b] + t - cu[b]
    ok = served[b]
    slot = table[b, torch.where(ok, p // bs, 0)].long() * bs + p % bs
    i32 = torch.int32
    return (table, seqlens.to(i32), cu.to(i32), torch.where(ok, b, -1).to(i32), torch.where(ok, p, -1).to(i32),
            torch.where(ok, slot, -1), (fc - taken).to(i32))


def _plain_release(s):
    bs = s["case"]["block"]
    lens, done = s["seqlens"].long(), s["done"] != 0
    P = s["prefix_lens"].long()[s["gid"]]
    e = torch.arange(s["max_blocks"], device="cuda")
    mine = (done[:, None] & (e >= P[:, None] // bs) & (e < (lens[:, None] + bs - 1) // bs)).flatten()
    rank = torch.cumsum(mine, 0)
    free_list = torch.cat((s["free_list"], torch.zeros(1, dtype=torch.int32, device="cuda")))   # last: writes to drop
    at = torch.where(mine, s["free_count"].long() + rank - 1, s["free_list"].numel())
    free_list[at] = s["table"].flatten()
    return (free_list[:-1], torch.where(done, 0, s["seqlens"]), s["free_count"] + rank[-1:].to(torch.int32))


# ------------------------------------------------------------------------------------------------ the definition
def exact(case, seed):
    if case["op"] == "decode":
        return _exact_decode(prepare(case, seed))
    return (_exact_plan if case["op"] == "plan" else _exact_release)(prepare(case, seed))


def _exact_decode(s):
    """Per sequence and head: k = [c W_UK | k_pe], v = c W_UV, softmax(scale q k) v over the visible keys, in float64."""
    case = s["case"]
    H, B, n_q, bs = case["heads"], case["batch"], case["n_q"], case["block"]
    f64 = torch.float64
    rows = s["pool"]
    if case["tiled"]:   # the swizzle is its own inverse
        x = rows.view(-1, W // 64, 64, 8, 8)
        t, g = torch.arange(64, device="cuda"), torch.arange(8, device="cuda")
        x = torch.gather(x, 3, (g[None, :] ^ (t[:, None] % 8)).view(1, 1, 64, 8, 1).expand(x.shape))
        rows = x.permute(0, 2, 1, 3, 4).reshape(-1, W)
    freq = ROPE_BASE ** (-2.0 * torch.arange(D_ROPE // 2, device="cuda", dtype=f64) / D_ROPE)
    out = torch.empty(B, n_q, H, D_V, dtype=f64, device="cuda")

    def token_rows(b, lo, hi):
        i = torch.arange(lo, hi, device="cuda")
        return rows[s["table"][b].long()[i // bs] * bs + i % bs].to(f64)

    wk, wv = s["w_uk"].to(f64), s["w_uv"].to(f64)
    for g, p in enumerate(s["prefixes"]):
        b0, b1 = s["offsets"][g], s["offsets"][g + 1]
        pre = token_rows(b0, 0, p)
        own_rows = [token_rows(b, p, s["seqlens_host"][b]) for b in range(b0, b1)]
        cat = torch.cat([pre] + own_rows)
        ends = np.cumsum([p] + [r.shape[0] for r in own_rows])
        for h in range(H):
            K = torch.cat((cat[:, :D_C] @ wk[h], cat[:, D_C:]), 1)
            V = cat[:, :D_C] @ wv[h]
            qs = []
            for b in range(b0, b1):
                z = torch.arange(n_q, device="cuda", dtype=f64) + (s["seqlens_host"][b] - n_q)
                ang = z[:, None] * freq
                x = s["q_pe"][b, :, h].to(f64).view(n_q, D_ROPE // 2, 2)
                rot = torch.stack((x[..., 0] * ang.cos() - x[..., 1] * ang.sin(),
                                   x[..., 0] * ang.sin() + x[..., 1] * ang.cos()), -1).view(n_q, D_ROPE)
                qs.append(torch.cat((s["q_nope"][b, :, h].to(f64), rot), 1))
            zp = torch.cat(qs) @ K[:p].T * SCALE                   # prefix logits of the whole group
            for i, b in enumerate(range(b0, b1)):
                lo, hi = int(ends[i]), int(ends[i + 1])
                zt = qs[i] @ K[lo:hi].T * SCALE
                far = torch.arange(hi - lo, device="cuda")[None] > (hi - lo - n_q + torch.arange(n_q, device="cuda"))[:, None]
                z = torch.cat((zp[i * n_q:(i + 1) * n_q], zt.masked_fill(far, float("-inf"))), 1)
                pr = torch.softmax(z, 1)
                out[b, :, h] = pr[:, :p] @ V[:p] + pr[:, p:] @ V[lo:hi]
    return out


def _exact_plan(s):
    bs, B = s["case"]["block"], s["case"]["batch"]
    cached, new = s["cached"].tolist(), s["new"].tolist()
    gid, prefixes = s["gid"].tolist(), s["prefixes"]
    table, pt, fl = s["table"].cpu().numpy().copy(), s["prefix_table"].cpu().numpy(), s["free_list"].cpu().numpy()
    free = int(s["free_count"].item())
    seqlens, cu = list(cached), [0]
    seq_idx, pos, slots = (np.full(s["T"], -1, np.int64) for _ in range(3))
    top, out_of = free, False
    for b in range(B):
        c, n = cached[b], new[b]
        cu.append(cu[-1] + n)
        have, want = -(-c // bs), -(-(c + n) // bs)
        k = want - have
        if k > 0 and (out_of or k > top):   # served in order: the first that does not fit ends the allocations
            out_of = True
            continue
        for i in range(have, want):
            top -= 1
            table[b, i] = fl[top]
        p = prefixes[gid[b]]
        if p and c == p:
            table[b, :p // bs] = pt[gid[b], :p // bs]
        seqlens[b] = c + n
        z = np.arange(c, c + n)
        seq_idx[cu[-2]:cu[-1]] = b
        pos[cu[-2]:cu[-1]] = z
        slots[cu[-2]:cu[-1]] = table[b, z // bs].astype(np.int64) * bs + z % bs
    i32 = lambda x: torch.from_numpy(np.asarray(x).astype(np.int32)).cuda()   # noqa: E731
    return i32(table), i32(seqlens), i32(cu), i32(seq_idx), i32(pos), torch.from_numpy(slots).cuda(), i32([top])


def _exact_release(s):
    bs = s["case"]["block"]
    lens, done, gid = s["seqlens"].tolist(), s["done"].tolist(), s["gid"].tolist()
    table, fl = s["table"].cpu().numpy(), s["free_list"].cpu().numpy().copy()
    n = int(s["free_count"].item())
    for b, d in enumerate(done):
        if d:
            ids = table[b, s["prefixes"][gid[b]] // bs:-(-lens[b] // bs)]
            fl[n:n + len(ids)] = ids
            n += len(ids)
            lens[b] = 0
    return torch.from_numpy(fl).cuda(), _i32(lens), _i32([n])
