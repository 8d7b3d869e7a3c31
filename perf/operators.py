"""Cases that measure the paged-cache operators: the batch plan built on the
GPU (block tables, slots, positions), the writing of new keys and values into
the pages, and attention of new tokens over the pages.

`run` computes them in their plain form (elementary torch operations in 32
bits) where `own` is false, and through the package's public calls where it
is true.  Heads of 128; head counts and lengths are those of the repository's
attention workloads (GQA 64:8, up to 512K keys) and generic ones.
"""
import math
import random
from types import SimpleNamespace

import torch

own = False

D = 128
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
# what a drawn case may cost at most
MOST_KEYS = 16 << 20  # sequences x longest x KV heads
MOST_SCORES = 4 << 30  # sequences x heads x longest chunk x longest length
MOST_FLOPS = 2.0e12


def listed():
    attn = dict(op="attn", mask="CAUSAL", window=0, sinks=0, n_chunk=0, new_lo=1, new_hi=1, pad=0, layout="nhd", type="bf16")
    return [
        # one decode step of a small batch: the scheduler's bookkeeping, all latency
        dict(name="plan_decode_8", op="plan", n_seq=8, ctx_lo=100, ctx_hi=4096, n_chunk=0, new_lo=1, new_hi=1, page=16,
             pad=0, len_seed=1),
        # a full serving batch: 96 prompt chunks among 1024 requests, rows padded to a captured size
        dict(name="plan_mixed_1024", op="plan", n_seq=1024, ctx_lo=1, ctx_hi=32768, n_chunk=96, new_lo=200, new_hi=1000,
             page=64, pad=1500, len_seed=2),
        # the new keys and values of one decode step
        dict(name="write_decode_64", op="write", n_seq=64, ctx_lo=1000, ctx_hi=8192, n_chunk=0, new_lo=1, new_hi=1,
             page=64, pad=0, Hkv=8, layout="nhd", type="bf16", len_seed=3),
        # long prompts written at once, half precision, head-major small pages
        dict(name="write_prompts_16k", op="write", n_seq=5, ctx_lo=0, ctx_hi=900, n_chunk=5, new_lo=2900, new_hi=3900,
             page=16, pad=0, Hkv=8, layout="hnd", type="fp16", len_seed=4),
        # one request generating: the latency of a single token
        dict(attn, name="decode_1x4k", n_seq=1, ctx_lo=4095, ctx_hi=4095, page=64, Hq=64, Hkv=8, len_seed=5),
        # a generating batch of ragged lengths
        dict(attn, name="decode_64_ragged", n_seq=64, ctx_lo=1000, ctx_hi=32767, page=64, Hq=64, Hkv=8, len_seed=6),
        # four very long contexts
        dict(attn, name="decode_4x512k", n_seq=4, ctx_lo=524000, ctx_hi=524287, page=128, Hq=64, Hkv=8, len_seed=7),
        # every head with its own keys, half precision, head-major small pages
        dict(attn, name="decode_mha_fp16", n_seq=32, ctx_lo=2000, ctx_hi=16384, page=16, Hq=16, Hkv=16, layout="hnd",
             type="fp16", len_seed=8),
        # drafts verified five tokens at a time
        dict(attn, name="verify_32x5", n_seq=32, n_chunk=32, new_lo=5, new_hi=5, ctx_lo=1000, ctx_hi=16384, page=32,
             Hq=64, Hkv=8, len_seed=9),
        # a prompt's chunk over what is cached of it: products bound
        dict(attn, name="chunk_2048_at_32k", n_seq=1, n_chunk=1, new_lo=2048, new_hi=2048, ctx_lo=32768, ctx_hi=32768,
             page=64, Hq=64, Hkv=8, len_seed=10),
        # a chunk beside generating requests, sliding window, odd page and group sizes
        dict(attn, name="mixed_window_odd", n_seq=16, n_chunk=1, new_lo=509, new_hi=509, ctx_lo=50, ctx_hi=8191,
             mask="CAUSAL_SLIDING", window=1024, page=48, Hq=24, Hkv=8, len_seed=11),
        # fresh prompts of odd lengths, rows padded to a captured size
        dict(attn, name="prompts_8_ragged", n_seq=8, n_chunk=8, new_lo=101, new_hi=2047, ctx_lo=0, ctx_hi=0, page=64,
             Hq=64, Hkv=8, pad=77, len_seed=12),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["plan", "write", "attn", "attn", "attn", "attn"])
    c = dict(op=op, len_seed=rng.randrange(1 << 30), page=rng.choice([8, 16, 24, 32, 48, 64, 96, 128, 256]), pad=0)
    if op == "plan":
        n = _log(rng, 1, 2048)
        c.update(n_seq=n, ctx_lo=0, ctx_hi=_log(rng, 10, 32768), n_chunk=rng.randrange(0, min(n, 100) + 1), new_lo=1,
                 new_hi=_log(rng, 2, 1000), pad=rng.choice([0, 0, 13, 400]))
        return c
    c.update(layout=rng.choice(["nhd", "hnd"]), type=rng.choice(["bf16", "bf16", "fp16"]))
    if op == "write":
        n = _log(rng, 1, 64)
        c.update(n_seq=n, ctx_lo=0, ctx_hi=_log(rng, 10, 8192), n_chunk=n, new_lo=1, new_hi=_log(rng, 1, 16384 // n),
                 Hkv=rng.choice([1, 2, 4, 7, 8, 16]))
        return c
    Hkv, G = rng.choice([(8, 8), (8, 4), (4, 8), (1, 8), (16, 1), (8, 3), (4, 5), (2, 12), (2, 16), (7, 1), (1, 32)])
    mask = rng.choice(["CAUSAL", "CAUSAL", "CAUSAL", "FULL", "CAUSAL_SLIDING", "GLOBAL_SLIDING"])
    c.update(Hq=Hkv * G, Hkv=Hkv, mask=mask, window=_log(rng, 16, 4096) if "SLIDING" in mask else 0,
             sinks=rng.choice([4, 64]) if mask == "GLOBAL_SLIDING" else 0, pad=rng.choice([0, 0, 0, 5, 130]))
    kind = rng.choice(["decode", "decode", "verify", "chunk", "mixed"])
    n = _log(rng, 1, {"decode": 256, "verify": 64, "chunk": 8, "mixed": 24}[kind])
    new = {"decode": 1, "verify": rng.randrange(2, 9), "chunk": _log(rng, 9, 2048), "mixed": _log(rng, 9, 700)}[kind]
    most = min(MOST_KEYS // (n * Hkv), MOST_SCORES // (n * c["Hq"] * new), int(MOST_FLOPS / (4 * D * c["Hq"] * new * n)))
    c.update(n_seq=n, new_lo=1 if kind == "chunk" else new, new_hi=new,
             n_chunk={"decode": 0, "verify": n, "chunk": n, "mixed": 1 + n // 8}[kind],
             ctx_hi=_log(rng, 1, max(2, min(most, 524288) - new)))
    c["ctx_lo"] = c["ctx_hi"] // rng.choice([1, 4, 50])
    return c


def _lengths(c):
    """(cached, new) of every request; a chunk's request comes first."""
    rng = random.Random(c["len_seed"])
    out = []
    for i in range(c["n_seq"]):
        ctx = _log(rng, c["ctx_lo"] + 1, c["ctx_hi"] + 1) - 1
        out.append((ctx, rng.randint(c["new_lo"], c["new_hi"]) if i < c["n_chunk"] else 1))
    return out


def _pages(c, extra):
    """Lengths, pages of every request (cached and new tokens), the table's width and a count of pages with spares."""
    lens = _lengths(c)
    need = [-(-(a + b) // c["page"]) for a, b in lens]
    return lens, need, max(need) + extra, sum(need) + 8


def prepare(c, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    lens, need, width, n_pages = _pages(c, 3)
    n, page = c["n_seq"], c["page"]
    i32 = dict(dtype=torch.int32, device="cuda")
    s = SimpleNamespace(op=c["op"], page=page, n_pages=n_pages, n_rows=sum(b for _, b in lens) + c["pad"])
    s.ctx = torch.tensor([a for a, _ in lens], **i32)
    s.new = torch.tensor([b for _, b in lens], **i32)
    perm = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    counts = torch.tensor(need, device="cuda")
    first = counts.cumsum(0) - counts
    col = torch.arange(width, device="cuda")
    table = torch.where(col < counts[:, None], perm[(first[:, None] + col).clamp(max=n_pages - 1)], -1)
    if s.op == "plan":
        # the pages of the cached tokens are in the table, the others in the list of free ones, five of it taken
        have = (s.ctx + page - 1) // page
        s.table = torch.where(col < have[:, None], table, -1)
        owned = torch.zeros(n_pages + 1, dtype=torch.bool, device="cuda")
        owned[s.table.long().flatten()] = True  # -1 is the last entry
        spare = perm[~owned[perm.long()]]
        s.free = torch.cat([spare[:5], spare])
        s.taken = torch.tensor([5], **i32)
        return s
    dt = TYPES[c["type"]]
    Hkv = c["Hkv"]
    shape = (n_pages, page, Hkv, D) if c["layout"] == "nhd" else (n_pages, Hkv, page, D)
    s.kc, s.vc = (torch.empty(shape, dtype=dt, device="cuda").normal_(generator=gen) for _ in range(2))
    if c["layout"] == "hnd":
        s.kc, s.vc = s.kc.transpose(1, 2), s.vc.transpose(1, 2)
    q_start = [0]
    for _, b in lens:
        q_start.append(q_start[-1] + b)
    if s.op == "write":
        s.k, s.v = (torch.empty(s.n_rows, Hkv, D, dtype=dt, device="cuda").normal_(generator=gen) for _ in range(2))
        seq = torch.repeat_interleave(torch.arange(n, device="cuda"), s.new.long())
        pos = torch.arange(s.n_rows, device="cuda") - torch.tensor(q_start, device="cuda")[seq] + s.ctx[seq]
        s.slots = (table[seq, pos // page] * page + pos % page).to(torch.int32)
        return s
    s.table = table.to(torch.int32)
    s.q = torch.empty(s.n_rows, c["Hq"], D, dtype=dt, device="cuda").normal_(generator=gen)
    s.q_start = torch.tensor(q_start, **i32)
    s.k_len = s.ctx + s.new
    s.mask = SimpleNamespace(kind=c["mask"], window_left=c["window"], window_right=0, num_global=c["sinks"])
    s.max_q, s.max_k = max(b for _, b in lens), max(a + b for a, b in lens)
    return s


# ------------------------------------------------------------------ the plain forms
def _plan(s):
    n, page = s.ctx.numel(), s.page
    new, ctx = s.new.long(), s.ctx.long()
    q_start = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    have, want = (ctx + page - 1) // page, (ctx + new + page - 1) // page
    taken = (want - have).cumsum(0)
    col = torch.arange(s.table.shape[1], device="cuda")
    at = s.taken + (taken - (want - have))[:, None] + col - have[:, None]
    fresh = (col >= have[:, None]) & (col < want[:, None])
    table = torch.where(fresh, s.free[at.clamp(0, s.free.numel() - 1)], s.table)
    row = torch.arange(s.n_rows, device="cuda")
    seq = (torch.searchsorted(q_start, row, right=True) - 1).clamp(max=n - 1)
    live = row < q_start[-1]
    pos = torch.where(live, row - q_start[seq] + ctx[seq], 0)
    slots = torch.where(live, table[seq, pos // page].long() * page + pos % page, -1)
    state = torch.cat([s.taken + taken[-1:], taken.new_zeros(2), q_start[-1:]])
    i32 = torch.int32
    return {"table": table.to(i32), "q_start": q_start.to(i32), "k_len": (ctx + new).to(i32), "slots": slots.to(i32),
            "positions": pos.to(i32), "state": state.to(i32)}


def _write(s):
    page, at = s.slots.long() // s.page, s.slots.long() % s.page
    s.kc[page, at] = s.k
    s.vc[page, at] = s.v
    return {"k": s.kc, "v": s.vc}


def _attends(mask, i, j, length):
    """Whether the token at position i attends key j of `length` keys."""
    if mask.kind == "FULL":
        ok = j < length
    elif mask.kind == "CAUSAL":
        ok = j <= i
    elif mask.kind == "CAUSAL_SLIDING":
        ok = (j <= i) & (j >= i - mask.window_left)
    else:  # GLOBAL_SLIDING
        g = mask.num_global
        ok = (i < g) | (j < g) | ((j <= i + mask.window_right) & (j >= i - mask.window_left))
    return ok & (j < length)


def _attn(s):
    T, Hq, _ = s.q.shape
    n, Hkv = s.k_len.numel(), s.kc.shape[2]
    q_start, k_len = s.q_start.long(), s.k_len.long()
    new = q_start[1:] - q_start[:-1]
    j = torch.arange(s.max_k, device="cuda")
    page = s.table[:, j // s.page].long().clamp(min=0)
    t = torch.arange(s.max_q, device="cuda")
    q = s.q[(q_start[:-1, None] + t).clamp(max=T - 1)].float() * (1 / math.sqrt(D))  # [n, max_q, Hq, D]
    q = q.view(n, s.max_q, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(n, Hkv, -1, D)
    scores = q @ s.kc[page, j % s.page].float().permute(0, 2, 3, 1)  # [n, Hkv, G * max_q, max_k]
    pos = (k_len - new)[:, None] + t
    ok = _attends(s.mask, pos[:, :, None], j, k_len[:, None, None]) & (t < new[:, None])[:, :, None]
    scores = scores.view(n, Hq, s.max_q, s.max_k).masked_fill_(~ok[:, None], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = p.view(n, Hkv, -1, s.max_k) @ s.vc[page, j % s.page].float().transpose(1, 2)
    o = o.view(n, Hq, s.max_q, D) / total.clamp(min=1e-30)
    lse = (top + total.log()).squeeze(-1)
    row = torch.arange(T, device="cuda")
    seq = (torch.searchsorted(q_start, row, right=True) - 1).clamp(max=n - 1)
    live, at = row < q_start[-1], (row - q_start[seq]).clamp(max=s.max_q - 1)
    o = torch.where(live[:, None, None], o[seq, :, at], 0)
    lse = torch.where(live[:, None], lse[seq, :, at], -math.inf)
    return {"o": o.to(s.q.dtype), "lse": lse.t().contiguous()}


def run(s):
    if own:
        import long_context_masked_attention_gb300 as lca

        if s.op == "plan":
            p = lca.paged_plan(s.ctx, s.new, s.free, s.taken, s.table, s.page, s.n_pages, s.n_rows)
            return {"table": s.table, "q_start": p.q_start, "k_len": p.k_len, "slots": p.slots,
                    "positions": p.positions, "state": p.state}
        if s.op == "write":
            lca.paged_write(s.k, s.v, s.kc, s.vc, s.slots)
            return {"k": s.kc, "v": s.vc}
        o, lse = lca.attn_paged(s.q, s.kc, s.vc, s.table, s.q_start, s.k_len, s.mask, max_q_len=s.max_q)
        return {"o": o, "lse": lse}
    return {"plan": _plan, "write": _write, "attn": _attn}[s.op](s)


def _cells(c):
    """Attended (token, key) pairs and keys that some token of their request attends."""
    cells = keys = 0
    for ctx, new in _lengths(c):
        length, w, g = ctx + new, c["window"], c["sinks"]
        if c["mask"] == "FULL":
            cells, keys = cells + new * length, keys + length
        elif c["mask"] == "CAUSAL":
            cells, keys = cells + new * ctx + new * (new + 1) // 2, keys + length
        elif c["mask"] == "CAUSAL_SLIDING":
            cells += sum(min(i, w) + 1 for i in range(ctx, length))
            keys += length - max(0, ctx - w)
        else:
            for i in range(ctx, length):
                cells += length if i < g else min(g, length) + max(0, i + 1 - max(g, i - w))
            keys += length if ctx < g else min(g, length) + max(0, length - max(g, ctx - w))
    return cells, keys


def work(c):
    lens = _lengths(c)
    rows = sum(b for _, b in lens) + c["pad"]
    if c["op"] == "plan":
        n, page = c["n_seq"], c["page"]
        fresh = sum(-(-(a + b) // page) - -(-a // page) for a, b in lens)
        # lengths read, row starts and key lengths written; pages read and entered; slots and positions written
        return {"bytes": 4 * (4 * n + 1 + 2 * fresh + 2 * rows + 5), "flops": 0}
    if c["op"] == "write":
        return {"bytes": rows * (4 + 2 * 2 * 2 * c["Hkv"] * D), "flops": 0}
    cells, keys = _cells(c)
    kv = 2 * keys * c["Hkv"] * D * 2
    return {"bytes": kv + rows * c["Hq"] * (2 * 2 * D + 4) + 4 * (keys // c["page"] + 2 * c["n_seq"] + 1),
            "flops": 4 * D * c["Hq"] * cells}


def exact(c, seed):
    """softmax(q k' / sqrt(d)) v and its log-sum-exp in 64 bits, request by request and head by head."""
    if c["op"] != "attn":
        return None
    s = prepare(c, seed)
    Hq, Hkv, G = c["Hq"], c["Hkv"], c["Hq"] // c["Hkv"]
    o = torch.zeros(s.n_rows, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((Hq, s.n_rows), -math.inf, dtype=torch.float64, device="cuda")
    r0 = 0
    for i, (ctx, new) in enumerate(_lengths(c)):
        length = ctx + new
        n_pages = -(-length // c["page"])
        pages = s.table[i, :n_pages].long()
        qi = torch.arange(ctx, length, device="cuda")[:, None]
        kj = torch.arange(length, device="cuda")[None]
        w, g = c["window"], c["sinks"]
        hidden = {"FULL": lambda: kj < 0, "CAUSAL": lambda: kj > qi, "CAUSAL_SLIDING": lambda: (kj > qi) | (kj < qi - w),
                  "GLOBAL_SLIDING": lambda: (qi >= g) & (kj >= g) & ((kj > qi) | (kj < qi - w))}[c["mask"]]()
        for h in range(Hkv):
            keys = s.kc[pages, :, h].reshape(-1, D)[:length].double()
            values = s.vc[pages, :, h].reshape(-1, D)[:length].double()
            for head in range(h * G, h * G + G):
                x = s.q[r0:r0 + new, head].double() @ keys.T / math.sqrt(D)
                x.masked_fill_(hidden, -math.inf)
                z = torch.logsumexp(x, 1)
                lse[head, r0:r0 + new] = z
                o[r0:r0 + new, head] = x.sub_(z[:, None]).exp_() @ values
        r0 += new
    return {"o": o, "lse": lse}
