"""Measured cases of the serving operators: prompt attention, and the 8-bit key/value cache with its append,
its attention and its eviction.

`own` false: the operators in plain torch arithmetic (fp32, rounded once at the end). `own` true: the calls a
user makes of the library. Both take what prepare() made; the lengths of a case follow from the case alone,
every value and the order of the cache's blocks from the seed.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------

def listed():
    prompt = dict(op="prompt", causal=True, fused=False, text=0)
    append = dict(op="append")
    attn = dict(op="attn", weights=False)
    evict = dict(op="evict")
    return [
        # a short question with a small model's heads: the latency of one launch
        dict(prompt, name="prompt-short", seqs=1, low=100, high=100, H=8, H_kv=2, d=64),
        # a serving batch of prompts from one token to a long one, q, k and v being slices of one projection
        dict(prompt, name="prompt-packed", seqs=9, low=1, high=2900, H=32, H_kv=8, d=128, fused=True),
        # one long document
        dict(prompt, name="prompt-long", seqs=1, low=16384, high=16384, H=16, H_kv=4, d=128),
        # video tokens (three latent frames of 30 x 52) attending to a text of up to 512 tokens, all to all
        dict(prompt, name="prompt-text", seqs=2, low=4680, high=4680, H=12, H_kv=12, d=128, causal=False, text=512),
        # one token for each of 64 running sequences into the cache
        dict(append, name="append-token", B=64, low=40, high=2048, new=1, ragged=False, H=32, H_kv=8, d=128, block=64),
        # whole prompts into the cache
        dict(append, name="append-prompt", B=6, low=300, high=9001, new=9001, ragged=True, H=32, H_kv=8, d=128, block=64),
        # one short sequence, one token: latency
        dict(attn, name="attn-one-short", B=1, low=300, high=300, new=1, ragged=False, H=8, H_kv=2, d=64, block=32),
        # a full decoding batch of unequal sequences, gathering the weights that eviction goes by
        dict(attn, name="attn-batch", B=64, low=500, high=16000, new=1, ragged=False, H=32, H_kv=8, d=128, block=64,
             weights=True),
        # a few drafted tokens for each sequence, checked in one call; small blocks
        dict(attn, name="attn-drafts", B=16, low=33, high=6000, new=4, ragged=True, H=32, H_kv=8, d=128, block=16,
             weights=True),
        # one very long sequence: the work has to be split over its length
        dict(attn, name="attn-one-long", B=1, low=131072, high=131072, new=1, ragged=False, H=32, H_kv=8, d=128,
             block=128),
        # a small batch brought back to a few hundred tokens
        dict(evict, name="evict-small", B=3, low=200, high=1001, H=8, H_kv=2, d=64, block=32, keep=250, recent=32),
        # a full batch of long sequences brought back to a quarter
        dict(evict, name="evict-large", B=32, low=6000, high=16384, H=32, H_kv=8, d=128, block=64, keep=4096,
             recent=256),
    ]


def _log(rng, low, high):
    return int(round(low * (high / low) ** rng.random()))


def draw(rng):
    op = rng.choice(["prompt", "append", "attn", "attn", "evict"])
    d = rng.choice([64, 128, 128])
    H_kv = rng.choice([1, 2, 3, 4, 8])
    H = H_kv * rng.choice([1, 2, 4, 5, 8])
    block = rng.choice([16, 32, 64, 128])
    low = _log(rng, 1, 3000)
    if op == "prompt":
        seqs = rng.choice([1, 1, 2, 3, 5, 9])
        high = _log(rng, 64, min(8000, 36000 / math.sqrt(seqs * H)))
        if rng.random() < 0.25:
            return dict(op=op, seqs=seqs, low=min(low, high), high=high, H=H, H_kv=H, d=d, causal=False, fused=False,
                        text=_log(rng, 8, 700))
        return dict(op=op, seqs=seqs, low=min(low, high), high=high, H=H, H_kv=H_kv, d=d, causal=rng.random() < 0.85,
                    fused=rng.random() < 0.5, text=0)
    if op == "append":
        B = _log(rng, 1, 64)
        high = _log(rng, 16, 60000 / B)
        new = rng.choice([1, 1, 3, 17, high])
        return dict(op=op, B=B, low=min(low, high), high=high, new=new, ragged=rng.random() < 0.5, H=H, H_kv=H_kv,
                    d=d, block=block)
    if op == "attn":
        B = _log(rng, 1, 64)
        high = _log(rng, 16, 200000 / B)
        new = rng.choice([1, 1, 1, 2, 4, 8])
        return dict(op=op, B=B, low=min(low, high), high=high, new=new, ragged=rng.random() < 0.5, H=H, H_kv=H_kv,
                    d=d, block=block, weights=rng.random() < 0.6)
    B = _log(rng, 1, 32)
    high = _log(rng, 64, 300000 / B)
    keep = max(2, int(high * rng.uniform(0.1, 0.9)))
    return dict(op=op, B=B, low=min(low, high), high=high, H=H, H_kv=H_kv, d=d, block=block, keep=keep,
                recent=int(keep * rng.uniform(0.0, 0.6)))


# ---------------------------------------------------------------------------------------------------------
# sizes that follow from a case
# ---------------------------------------------------------------------------------------------------------

def _lengths(n, low, high):
    """n lengths from `low` to `high`, spread over their logarithm, the largest first."""
    return [high if i == 0 else low if i == 1 else int(round(low * (high / low) ** ((i * 0.6180339887) % 1.0)))
            for i in range(n)]


def _prompt_lengths(c):
    q = _lengths(c["seqs"], c["low"], c["high"])
    return q, ([max(1, c["text"] - 37 * i) for i in range(c["seqs"])] if c["text"] else q)


def _cache_lengths(c):
    """Tokens in the cache after the call, and how many of them are new, for each sequence."""
    total = _lengths(c["B"], c["low"], c["high"])
    new = c.get("new", 0)
    return total, [min(t, 1 + (5 * i + new - 1) % new if c.get("ragged") else new) if new else 0
                   for i, t in enumerate(total)]


def _seen(c, q, k):
    """(query, key) pairs that the mask leaves for a sequence of q queries and k keys."""
    if not c.get("causal", True):
        return q * k
    first = max(0, q - k)                 # queries before the first key
    n = q - first
    return n * (k - q + first + 1) + n * (n - 1) // 2


def work(case):
    c = case
    d, H, H_kv = c["d"], c["H"], c["H_kv"]
    if c["op"] == "prompt":
        q, k = _prompt_lengths(c)
        return {"bytes": 2 * d * (2 * H * sum(q) + 2 * H_kv * sum(k)) + 4 * H * sum(q),
                "flops": 4 * d * H * sum(_seen(c, a, b) for a, b in zip(q, k))}
    total, new = _cache_lengths(c)
    if c["op"] == "append":
        return {"bytes": 2 * sum(new) * H_kv * d * 3, "flops": 2 * sum(new) * H_kv * d}
    if c["op"] == "attn":
        return {"bytes": 2 * sum(total) * H_kv * d + 4 * sum(new) * H * d + (8 * sum(total) * H_kv if c["weights"] else 0),
                "flops": 4 * d * H * sum(_seen({}, a, b) for a, b in zip(new, total))}
    kept = sum(min(t, c["keep"]) for t in total)
    return {"bytes": 4 * sum(total) * H_kv + kept * H_kv * (4 * d + 8), "flops": 0}


# ---------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------

def _offsets(lengths, device):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device=device)


def _fill(shape, sd, gen, device):
    return (torch.randn(shape, generator=gen, device=device) * sd).to(torch.bfloat16)


def _prepare_prompt(c, gen, device):
    nq, nk = _prompt_lengths(c)
    Tq, Tk, H, H_kv, d = sum(nq), sum(nk), c["H"], c["H_kv"], c["d"]
    if c["fused"]:                        # one projection's rows: q heads, k heads, v heads
        rows = _fill((Tq, (H + 2 * H_kv) * d), 1.0, gen, device)
        q, k, v = rows[:, :H * d], rows[:, H * d:(H + H_kv) * d], rows[:, (H + H_kv) * d:]
        q, k, v = q.unflatten(1, (H, d)), k.unflatten(1, (H_kv, d)), v.unflatten(1, (H_kv, d))
    else:
        q, k, v = (_fill((t, h, d), 1.0, gen, device) for t, h in ((Tq, H), (Tk, H_kv), (Tk, H_kv)))
    s = dict(case=c, q=q, k=k, v=v, seq_q=_offsets(nq, device), seq_k=_offsets(nk, device), longest_q=max(nq),
             longest_k=max(nk))
    s["o"] = torch.empty((Tq, H, d), dtype=torch.bfloat16, device=device)
    s["lse"] = torch.empty((Tq, H), dtype=torch.float32, device=device)
    if own:
        from sparse_rank_attention_block_b200 import sda
        s["p"] = sda.prompt_params(n_seq=c["seqs"], rows_q=Tq, rows_k=Tk, H=H, H_kv=H_kv, d=d, causal=c["causal"],
                                   ld_q=q.stride(0), ld_k=k.stride(0), ld_v=v.stride(0))
        s["ws"] = sda.Workspace(s["p"], device=device)
    return s


def _prepare_cache(c, gen, device):
    total, new = _cache_lengths(c)
    B, H, H_kv, d, block = c["B"], c["H"], c["H_kv"], c["d"], c["block"]
    need = [-(-t // block) for t in total]
    keep, recent = c.get("keep", 0), c.get("recent", 0)
    need_dst = [-(-min(t, keep) // block) for t in total] if keep else []
    n_blocks = sum(need) + sum(need_dst) + 1
    order = torch.randperm(n_blocks, generator=gen, device=device).to(torch.int32)

    def table(counts, start):             # rows of block numbers, -1 behind a sequence's last block
        width = max(counts)
        at = _offsets(counts, device).long()
        col = torch.arange(width, device=device)
        inside = col[None, :] < (at[1:] - at[:-1])[:, None]
        where = (start + at[:-1, None] + col[None, :]).clamp_max(n_blocks - 1)
        return torch.where(inside, order[where], -1).to(torch.int32)

    s = dict(case=c, lens=torch.tensor(total, dtype=torch.int32, device=device), table=table(need, 0), block=block)
    # a block's values: normal, each block and head at a scale of its own (a power of two)
    for name in ("k", "v"):
        codes = torch.randn((n_blocks, H_kv, block, d), generator=gen, device=device).mul_(64.0).clamp_(-448, 448)
        s[name + "_codes"] = codes.to(E4M3).view(torch.uint8)
        s[name + "_scale"] = torch.exp2(torch.randint(-7, -4, (n_blocks, H_kv), generator=gen, device=device).float())
        del codes
    T = sum(new)
    if c["op"] != "evict":
        s["seq"] = _offsets(new, device)
        s["longest"] = max(new)
    if c["op"] == "append":
        s["k"], s["v"] = _fill((T, H_kv, d), 1.0, gen, device), _fill((T, H_kv, d), 1.0, gen, device)
        s["w"] = torch.rand((n_blocks, H_kv, block), generator=gen, device=device)
    elif c["op"] == "attn":
        s["q"] = _fill((T, H, d), 1.0, gen, device)
        s["o"] = torch.empty_like(s["q"])
        s["w_in"] = torch.rand((n_blocks, H_kv, block), generator=gen, device=device).mul_(1e-2) if c["weights"] else None
        s["w_out"] = torch.zeros((n_blocks, H_kv, block), device=device) if c["weights"] else None
    else:
        # accumulated weights: heavy-tailed, with equal values among them
        s["w"] = torch.rand((n_blocks, H_kv, block), generator=gen, device=device).pow_(4).mul_(4096).round_().div_(512)
        s["dst_table"] = table(need_dst, sum(need))
        s["kept"] = torch.full((B, H_kv, keep), -1, dtype=torch.int32, device=device)
        s["dst_lens"] = torch.zeros((B,), dtype=torch.int32, device=device)
    if own:
        from sparse_rank_attention_block_b200 import sda
        s["p"] = sda.cache_params(B=B, H=H, H_kv=H_kv, d=d, block=block, n_blocks=n_blocks,
                                  max_blocks=s["table"].shape[1], rows=T, max_new=max(new),
                                  weights=c.get("weights", False), keep=keep, recent=recent)
        s["ws"] = sda.Workspace(s["p"], device=device)
    return s


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device)
    gen.manual_seed(int(seed))
    make = _prepare_prompt if case["op"] == "prompt" else _prepare_cache
    return make(case, gen, device)


# ---------------------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------------------

def _plain_softmax(scores, visible):
    """exp(scores - max) over the visible keys, its sum and the maximum; rows that see nothing: zeros."""
    scores = scores.masked_fill_(~visible, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    e = scores.sub_(top).exp_()
    return e, e.sum(-1, keepdim=True), top


def _plain_prompt(s):
    c = s["case"]
    H, H_kv, d = c["H"], c["H_kv"], c["d"]
    g = H // H_kv
    at_q, at_k = s["seq_q"].long(), s["seq_k"].long()
    n_q, n_k = at_q[1:] - at_q[:-1], at_k[1:] - at_k[:-1]
    dev = at_q.device
    i = torch.arange(s["longest_q"], device=dev)
    j = torch.arange(s["longest_k"], device=dev)
    in_q, in_k = i[None] < n_q[:, None], j[None] < n_k[:, None]
    row_q = torch.where(in_q, at_q[:-1, None] + i[None], 0)
    row_k = torch.where(in_k, at_k[:-1, None] + j[None], 0)
    q = s["q"].float()[row_q].unflatten(2, (H_kv, g)).permute(0, 2, 3, 1, 4)      # [seq, H_kv, g, i, d]
    k = s["k"].float()[row_k].permute(0, 2, 3, 1)[:, :, None]                     # [seq, H_kv, 1, d, j]
    v = s["v"].float()[row_k].permute(0, 2, 1, 3)[:, :, None]
    visible = in_k[:, None, :].expand(-1, i.numel(), -1)
    if c["causal"]:
        visible = visible & (j[None, None, :] <= i[None, :, None] + (n_k - n_q)[:, None, None])
    e, z, top = _plain_softmax(torch.matmul(q, k).mul_(1.0 / math.sqrt(d)), visible[:, None, None])
    o = torch.matmul(e, v) / torch.where(z > 0, z, 1.0)
    lse = (top + torch.log(z)).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[in_q].to(torch.bfloat16)
    return {"o": o, "lse": lse.permute(0, 3, 1, 2).flatten(2, 3)[in_q]}


def _new_rows(s):
    """For each new row: its sequence and its position there."""
    at = s["seq"].long()
    row = torch.arange(s["k" if "k" in s else "q"].shape[0], device=at.device)
    b = torch.searchsorted(at[1:], row, right=True)
    return row, b, s["lens"].long()[b] - (at[b + 1] - row)


def _plain_append(s):
    block = s["block"]
    _, b, pos = _new_rows(s)
    blk, slot = s["table"].long()[b, pos // block], pos % block
    n_new = (s["seq"][1:] - s["seq"][:-1]).long()
    before = s["lens"].long() - n_new                                  # tokens there before the call
    old_rows = (before % block > 0) & (n_new > 0)                      # sequences whose first touched block holds old tokens
    old_blk = s["table"].long()[torch.arange(before.numel(), device=pos.device), before // block * old_rows]
    old_blk = torch.where(old_rows, old_blk, s["k_scale"].shape[0])    # none: a row of its own behind the pool
    for name in ("k", "v"):
        x, scale, codes = s[name].float(), s[name + "_scale"], s[name + "_codes"].view(E4M3)
        top = torch.full((scale.shape[0] + 1, scale.shape[1]), -1.0, device=x.device)
        top.index_reduce_(0, blk, x.abs().amax(-1), "amax")
        m, e = torch.frexp(top)                                        # top = m 2^e, 448 = 0.875 2^9
        want = torch.exp2((e - 9 + (m > 0.875)).clamp(-126, 120).float())
        want = torch.where(top == 0, 2.0 ** -126, want)
        before_scale = torch.cat([scale, torch.zeros_like(scale[:1])])
        has_old = torch.zeros_like(want, dtype=torch.bool)
        has_old[old_blk] = True
        has_old[-1] = False
        after = torch.where(has_old, torch.maximum(before_scale, want), want)
        after = torch.where(top < 0, before_scale, after)              # untouched blocks
        # older tokens of a touched block under its new scale; slots behind the last token stay as they are
        o = old_blk[old_rows]
        ratio = (before_scale[o] / after[o])[:, :, None, None]
        u8 = codes.view(torch.uint8)
        older = torch.arange(block, device=x.device)[None, None, :, None] < (before[old_rows] % block)[:, None, None, None]
        again = (codes[o].float() * ratio).clamp(-448, 448).to(E4M3).view(torch.uint8)
        u8[o] = torch.where(older, again, u8[o])
        u8[blk, :, slot] = (x / after[blk][:, :, None]).clamp(-448, 448).to(E4M3).view(torch.uint8)
        scale.copy_(after[:-1])
    s["w"][blk, :, slot] = 0.0
    return {"k": s["k_codes"].view(E4M3), "v": s["v_codes"].view(E4M3), "k_scale": s["k_scale"],
            "v_scale": s["v_scale"], "w": s["w"]}


def _plain_attn(s):
    c = s["case"]
    H, H_kv, d = c["H"], c["H_kv"], c["d"]
    g = H // H_kv
    table = s["table"].long()
    B, width = table.shape
    dev = table.device
    blk = table.clamp_min(0)
    k = s["k_codes"].view(E4M3)[blk].float() * s["k_scale"][blk][..., None, None]   # [B, width, H_kv, block, d]
    v = s["v_codes"].view(E4M3)[blk].float() * s["v_scale"][blk][..., None, None]
    k = k.permute(0, 2, 4, 1, 3).flatten(3)                                         # [B, H_kv, d, tokens]
    v = v.permute(0, 2, 1, 3, 4).flatten(2, 3)                                      # [B, H_kv, tokens, d]
    _, b, pos = _new_rows(s)
    i = torch.arange(pos.numel(), device=dev) - s["seq"].long()[b]
    q = torch.zeros((B, s["longest"], H, d), device=dev)
    q[b, i] = s["q"].float()
    at = torch.full((B, s["longest"]), -1, dtype=torch.long, device=dev)
    at[b, i] = pos
    q = q.unflatten(2, (H_kv, g)).permute(0, 2, 3, 1, 4).flatten(2, 3)              # [B, H_kv, g * new, d]
    j = torch.arange(k.shape[3], device=dev)
    visible = (j[None, None, :] <= at[:, :, None])[:, None, None].expand(-1, 1, g, -1, -1).flatten(2, 3)
    e, z, _ = _plain_softmax(torch.matmul(q, k).mul_(1.0 / math.sqrt(d)), visible)
    z = torch.where(z > 0, z, 1.0)
    o = (torch.matmul(e, v) / z).unflatten(2, (g, s["longest"])).permute(0, 3, 1, 2, 4).flatten(2, 3)[b, i]
    out = {"o": o.to(torch.bfloat16)}
    if c["weights"]:
        w = e.div_(z).sum(2).unflatten(2, (width, s["block"])).transpose(1, 2)      # [B, width, H_kv, block]
        inside = (j[None] < s["lens"].long()[:, None]).view(B, width, 1, s["block"])
        slots = inside.expand_as(w)
        old = s["w_out"][blk]
        new = torch.where(slots, s["w_in"][blk] + w, old)
        used = table >= 0
        s["w_out"][table[used]] = new[used]
        out["w"] = s["w_out"]
    return out


def _plain_evict(s):
    c = s["case"]
    keep, recent, block, H_kv = c["keep"], c["recent"], s["block"], c["H_kv"]
    table, dst = s["table"].long(), s["dst_table"].long()
    B, width = table.shape
    dev = table.device
    lens = s["lens"].long()
    n = lens.clamp_max(keep)                                                        # tokens that stay
    w = s["w"][table.clamp_min(0)].permute(0, 2, 1, 3).flatten(2)                   # [B, H_kv, tokens]
    j = torch.arange(w.shape[2], device=dev)
    inside = (j[None] < lens[:, None])[:, None]
    last = (j[None] >= (lens - recent)[:, None])[:, None]
    rank = torch.where(inside, torch.where(last, math.inf, w), -math.inf)
    order = torch.sort(rank, dim=2, descending=True, stable=True).indices[:, :, :keep]
    if order.shape[2] < keep:
        order = torch.nn.functional.pad(order, (0, keep - order.shape[2]))
    i = torch.arange(keep, device=dev)
    stays = (i[None] < n[:, None])[:, None].expand(-1, H_kv, -1)
    kept = torch.where(stays, order, w.shape[2]).sort(2).values
    kept = torch.where(stays, kept, -1)
    s["kept"].copy_(kept)
    s["dst_lens"].copy_(n)
    b, h, t = stays.nonzero(as_tuple=True)
    src = kept[b, h, t]
    src_blk, src_slot = table[b, src // block], src % block
    dst_blk, dst_slot = dst[b, t // block], t % block
    for name in ("k", "v"):
        scale, codes = s[name + "_scale"], s[name + "_codes"]
        top = torch.zeros_like(scale)
        top.view(-1).index_reduce_(0, dst_blk * H_kv + h, scale[src_blk, h], "amax")
        fresh = dst[dst >= 0]
        ratio = (scale[src_blk, h] / top[dst_blk, h])[:, None]
        codes[dst_blk, h, dst_slot] = (codes.view(E4M3)[src_blk, h, src_slot].float() * ratio).to(E4M3).view(torch.uint8)
        scale[fresh] = top[fresh]
    s["w"][dst_blk, h, dst_slot] = s["w"][src_blk, h, src_slot]
    return _evicted(s)


def _evicted(s):
    return {"k": s["k_codes"].view(E4M3), "v": s["v_codes"].view(E4M3), "k_scale": s["k_scale"],
            "v_scale": s["v_scale"], "w": s["w"], "kept": s["kept"], "lens": s["dst_lens"]}


# ---------------------------------------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------------------------------------

def _own(s):
    from sparse_rank_attention_block_b200 import sda
    c, ws = s["case"], s["ws"]
    if c["op"] == "prompt":
        sda.sda_prompt_attn_fwd(s["p"], s["q"], s["k"], s["v"], s["seq_q"], s["seq_k"], s["o"], s["lse"], ws.ptr,
                                ws.nbytes)
        return {"o": s["o"], "lse": s["lse"]}
    cache = (s["lens"], s["table"], s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
    if c["op"] == "append":
        sda.sda_cache_append(s["p"], s["k"], s["v"], s["seq"], *cache, s["w"], ws.ptr, ws.nbytes)
        return {"k": s["k_codes"].view(E4M3), "v": s["v_codes"].view(E4M3), "k_scale": s["k_scale"],
                "v_scale": s["v_scale"], "w": s["w"]}
    if c["op"] == "attn":
        sda.sda_cache_attn_fwd(s["p"], s["q"], s["seq"], *cache, s["w_in"], s["w_out"], s["o"], ws.ptr, ws.nbytes)
        return {"o": s["o"], "w": s["w_out"]} if c["weights"] else {"o": s["o"]}
    sda.sda_cache_evict(s["p"], *cache, s["w"], s["dst_table"], s["kept"], s["dst_lens"], ws.ptr, ws.nbytes)
    return _evicted(s)


def run(state):
    if own:
        return _own(state)
    plain = {"prompt": _plain_prompt, "append": _plain_append, "attn": _plain_attn, "evict": _plain_evict}
    return plain[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------------------------
# the definitions in 64 bits, one sequence and key head at a time
# ---------------------------------------------------------------------------------------------------------

def _exact_rows(q, k, v, first, scale):
    """softmax(q k^T scale) v for queries [n, d] whose last visible key is first + row (None: all keys)."""
    a = (q @ k.T) * scale
    if first is not None:
        hidden = torch.arange(k.shape[0], device=a.device)[None] > first[:, None]
        a[hidden] = -math.inf
    lse = torch.logsumexp(a, 1)
    p = torch.exp(a - torch.where(torch.isinf(lse), 0.0, lse)[:, None])
    return p @ v, lse, p


def _e4m3(x):
    """Nearest value of the 8-bit format (4 exponent bits, 3 of the fraction), ties to even, in 64 bits."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp_min(-6).double() - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    H, H_kv, d = c["H"], c["H_kv"], c["d"]
    g, scale = H // H_kv, d ** -0.5
    dev = s["q"].device if "q" in s else s["lens"].device
    if c["op"] == "prompt":
        nq, nk = _prompt_lengths(c)
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
        lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=dev)
        aq = ak = 0
        for a, b in zip(nq, nk):
            first = torch.arange(a, device=dev) + (b - a) if c["causal"] else None
            for h in range(H):
                k, v = (s[n][ak:ak + b, h // g].double() for n in ("k", "v"))
                o[aq:aq + a, h], lse[aq:aq + a, h], _ = _exact_rows(s["q"][aq:aq + a, h].double(), k, v, first, scale)
            aq, ak = aq + a, ak + b
        return {"o": o, "lse": lse}
    total, new = _cache_lengths(c)
    block = c["block"]
    value = {n: s[n + "_codes"].view(E4M3) for n in ("k", "v")}
    if c["op"] == "attn":
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
        w_out = s["w_out"].double() if c["weights"] else None
        at = 0
        for b, (t, n) in enumerate(zip(total, new)):
            blk = s["table"][b, :-(-t // block)].long()
            k, v = ((value[m][blk].double() * s[m + "_scale"][blk].double()[:, :, None, None]).transpose(0, 1)
                    .flatten(1, 2)[:, :t] for m in ("k", "v"))
            first = torch.arange(n, device=dev) + (t - n)
            w = torch.zeros((H_kv, blk.numel() * block), dtype=torch.float64, device=dev)
            for h in range(H):
                o[at:at + n, h], _, p = _exact_rows(s["q"][at:at + n, h].double(), k[h // g], v[h // g], first, scale)
                w[h // g, :t] += p.sum(0)
            if c["weights"]:
                sum_ = s["w_in"][blk].double() + w.view(H_kv, -1, block).transpose(0, 1)
                inside = (torch.arange(blk.numel() * block, device=dev) < t).view(-1, 1, block)
                w_out[blk] = torch.where(inside, sum_, w_out[blk])
            at += n
        return {"o": o, "w": w_out} if c["weights"] else {"o": o}
    out = {"w": s["w"].double()}
    if c["op"] == "append":
        for m in ("k", "v"):
            codes, scales = value[m].double(), s[m + "_scale"].double()
            at = 0
            for b, (t, n) in enumerate(zip(total, new)):
                p = t - n
                while p < t:                                           # one touched block after another
                    i = int(s["table"][b, p // block])
                    lo, hi = p % block, min(block, p % block + t - p)
                    x = s[m][at:at + hi - lo].double().transpose(0, 1)             # [H_kv, tokens, d]
                    top = x.abs().amax((1, 2))
                    want = torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(-126, 120))
                    old = scales[i] if lo else torch.zeros_like(want)
                    now = torch.maximum(old, want)
                    if lo:
                        codes[i, :, :lo] = _e4m3(codes[i, :, :lo] * (old / now)[:, None, None])
                    codes[i, :, lo:hi] = _e4m3(x / now[:, None, None])
                    scales[i] = now
                    if m == "k":
                        out["w"][i, :, lo:hi] = 0
                    at, p = at + hi - lo, p + hi - lo
            out[m], out[m + "_scale"] = codes, scales
        return out
    kept = torch.full((c["B"], H_kv, c["keep"]), -1, dtype=torch.int64, device=dev)
    for m in ("k", "v"):
        out[m], out[m + "_scale"] = value[m].double(), s[m + "_scale"].double()
    for b, t in enumerate(total):
        n = min(t, c["keep"])
        last = min(c["recent"], n)
        blk, dst = s["table"][b, :-(-t // block)].long(), s["dst_table"][b, :-(-n // block)].long()
        for h in range(H_kv):
            w = s["w"][blk, h].flatten()[:t].double()
            older = torch.sort(w[:t - last], descending=True, stable=True).indices[:n - last]
            stay = torch.cat([older.sort().values, torch.arange(t - last, t, device=dev)])
            kept[b, h, :n] = stay
            sb, ss = blk[stay // block], stay % block
            i = torch.arange(n, device=dev)
            out["w"][dst[i // block], h, i % block] = w[stay]
            for m in ("k", "v"):
                sc = s[m + "_scale"][sb, h].double()
                row = value[m][sb, h, ss].double() * sc[:, None]
                top = torch.nn.functional.pad(sc, (0, dst.numel() * block - n)).view(-1, block).amax(1)
                out[m][dst[i // block], h, i % block] = _e4m3(row / top[i // block][:, None])
                out[m + "_scale"][dst, h] = top
    out["kept"], out["lens"] = kept, torch.tensor([min(t, c["keep"]) for t in total], device=dev)
    return out
