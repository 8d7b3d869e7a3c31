"""Cases that measure rotary positions and the 8-bit paged cache: rotating
queries and keys (and their gradients back), quantising new keys and values as
they are written into the pages, reading pages back as 16-bit values, and
attention of new tokens over the 8-bit pages.

`run` computes them in their plain form (elementary torch operations in 32
bits, angles in 64) where `own` is false, and through the package's public
calls where it is true.  Heads of 128; head counts and lengths are those of the
repository's attention workloads (GQA 64:8, up to 512K keys) and generic ones.

A row of 128 values is kept as e4m3 values times 2^(b - 127): b is a byte per
token and head, the smallest for which the row's largest magnitude is at most
448 2^(b - 127), within 2^-48 to 2^48.
"""
import math
import random
from types import SimpleNamespace

import numpy as np
import torch

own = False

D = 128
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn
LOWEST, HIGHEST = -48, 48  # exponents of a row's factor
# what a drawn case may cost at most
MOST_KEYS = 16 << 20  # sequences x longest x KV heads
MOST_SCORES = 4 << 30  # sequences x heads x longest chunk x longest length
MOST_FLOPS = 2.0e12
MOST_VALUES = 300 << 20  # rows x heads x 128


def listed():
    rope = dict(op="rope", back=False, rot=128, interleaved=False, base=10000.0, factor=1.0, len_seed=0)
    attn = dict(op="attn", mask="CAUSAL", window=0, sinks=0, n_chunk=0, new_lo=1, new_hi=1, pad=0, layout="nhd", type="bf16")
    return [
        # one decode step: the new tokens' queries and keys, a launch's latency
        dict(rope, name="rope_decode_64", T=64, Hq=64, Hkv=8, far=32768, type="bf16"),
        # a packed training batch's forward, documents of a long-context run
        dict(rope, name="rope_train_32k", T=32768, Hq=64, Hkv=8, far=32768, type="bf16", base=500000.0),
        # the way back in half precision: pairs side by side, half of each head, a scaled table, far positions
        dict(rope, name="rope_bwd_partial", back=True, T=8191, Hq=24, Hkv=8, far=524288, type="fp16", rot=64,
             interleaved=True, factor=16.0),
        # the new keys and values of one decode step
        dict(name="write_decode_64", op="write", n_seq=64, ctx_lo=1000, ctx_hi=8192, n_chunk=0, new_lo=1, new_hi=1,
             page=64, pad=0, Hkv=8, layout="nhd", type="bf16", len_seed=3),
        # long prompts written at once, half precision, head-major small pages, rows padded to a captured size
        dict(name="write_prompts_16k", op="write", n_seq=5, ctx_lo=0, ctx_hi=900, n_chunk=5, new_lo=2900, new_hi=3900,
             page=16, pad=300, Hkv=8, layout="hnd", type="fp16", len_seed=4),
        # a short request's pages read back
        dict(name="read_1k", op="read", n=16, page=64, Hkv=8, layout="nhd", type="bf16"),
        # the cached part of a long prompt read back
        dict(name="read_128k", op="read", n=1365, page=96, Hkv=8, layout="hnd", type="bf16"),
        # one request generating: the latency of a single token
        dict(attn, name="decode_1x4k", n_seq=1, ctx_lo=4095, ctx_hi=4095, page=64, Hq=64, Hkv=8, len_seed=5),
        # a generating batch of ragged lengths
        dict(attn, name="decode_64_ragged", n_seq=64, ctx_lo=1000, ctx_hi=32767, page=64, Hq=64, Hkv=8, len_seed=6),
        # every head with its own keys, half precision, head-major small pages
        dict(attn, name="decode_mha_fp16", n_seq=32, ctx_lo=2000, ctx_hi=16384, page=16, Hq=16, Hkv=16, layout="hnd",
             type="fp16", len_seed=8),
        # drafts verified five tokens at a time
        dict(attn, name="verify_32x5", n_seq=32, n_chunk=32, new_lo=5, new_hi=5, ctx_lo=1000, ctx_hi=16384, page=32,
             Hq=64, Hkv=8, len_seed=9),
        # a prompt's chunk over what is cached of it: products bound
        dict(attn, name="chunk_2048_at_32k", n_seq=1, n_chunk=1, new_lo=2048, new_hi=2048, ctx_lo=32768, ctx_hi=32768,
             page=64, Hq=64, Hkv=8, len_seed=10),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "write", "read", "attn", "attn", "attn", "attn"])
    c = dict(op=op, type=rng.choice(["bf16", "bf16", "fp16"]))
    if op == "rope":
        Hkv, G = rng.choice([(8, 8), (8, 4), (1, 8), (16, 1), (8, 3), (7, 1), (2, 12), (4, 5)])
        T = _log(rng, 1, min(65536, MOST_VALUES // (D * Hkv * (G + 1))))
        c.update(T=T, Hq=Hkv * G, Hkv=Hkv, rot=rng.choice([128, 128, 128, 64, 32, 96, 20, 2]),
                 interleaved=rng.choice([False, False, True]), back=rng.choice([False, True]),
                 base=rng.choice([10000.0, 500000.0, 1e6]), factor=rng.choice([1.0, 1.0, 8.0, 40.0]),
                 far=_log(rng, 100, 1 << 20), len_seed=rng.randrange(1 << 30))
        return c
    c.update(page=rng.choice([8, 16, 24, 32, 48, 64, 96, 128, 256]), layout=rng.choice(["nhd", "hnd"]))
    if op == "read":
        Hkv = rng.choice([1, 2, 4, 7, 8, 16])
        c.update(n=_log(rng, 1, max(2, MOST_VALUES // (2 * D * Hkv * c["page"]))), Hkv=Hkv)
        return c
    c.update(len_seed=rng.randrange(1 << 30), pad=0)
    if op == "write":
        n = _log(rng, 1, 64)
        c.update(n_seq=n, ctx_lo=0, ctx_hi=_log(rng, 10, 8192), n_chunk=n, new_lo=1, new_hi=_log(rng, 1, 16384 // n),
                 Hkv=rng.choice([1, 2, 4, 7, 8, 16]), pad=rng.choice([0, 0, 13, 400]))
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


def _frequencies(c):
    """Radians per position of each pair, and the factor of a table for longer contexts: slow pairs are stretched by
    `factor`, fast ones kept, those between blended by how often they turn in 4096 positions (32 to 1 turns)."""
    rot, base, factor = c["rot"], c["base"], c["factor"]
    inv = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if factor == 1.0:
        return inv, 1.0
    low, high = (rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0))
    low, high = max(math.floor(low), 0), min(math.ceil(high), rot - 1)
    keep = 1 - np.clip((np.arange(rot // 2) - low) / max(high - low, 1e-3), 0, 1)
    return inv / factor * (1 - keep) + inv * keep, 0.1 * math.log(factor) + 1.0


def _two_to(b):
    """2^(b - 127) of bytes 1 to 254."""
    return (b.to(torch.int32) << 23).view(torch.float32)


def _quantise(x):
    """[.., 128] values -> their e4m3 values and the byte of each row's factor."""
    x = x.float()
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)  # top = m 2^e, m in [1/2, 1); 448 = 7/8 2^9
    e = torch.where(top > 0, torch.where(m <= 0.875, e - 9, e - 8), LOWEST).clamp(LOWEST, HIGHEST)
    y = (x * _two_to(127 - e)[..., None]).clamp(-448.0, 448.0)
    return y.to(E4M3), (e + 127).to(torch.uint8)


def _cache(gen, n_pages, page, Hkv, layout, filled):
    """Pages of e4m3 values [n_pages, page, Hkv, 128] (views of either order) and bytes [n_pages, Hkv, page]; rows
    differ in size, as keys and values do."""
    shape = (n_pages, page, Hkv, D) if layout == "nhd" else (n_pages, Hkv, page, D)
    if not filled:
        c, b = torch.zeros(shape, dtype=torch.uint8, device="cuda").view(E4M3), torch.zeros(n_pages, Hkv, page, dtype=torch.uint8, device="cuda")
    else:
        x = torch.empty(shape, device="cuda").normal_(generator=gen)
        x *= torch.empty(shape[:3], device="cuda").normal_(generator=gen).exp2_()[..., None]
        c, b = _quantise(x)
        b = (b.transpose(1, 2) if layout == "nhd" else b).contiguous()
    return (c if layout == "nhd" else c.transpose(1, 2)), b


def prepare(c, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    dt = TYPES[c["type"]]
    i32 = dict(dtype=torch.int32, device="cuda")
    Hkv = c["Hkv"]
    s = SimpleNamespace(op=c["op"], dt=dt)
    if s.op == "rope":
        # queries and keys as parts of one projection's rows; positions of documents packed one after another
        T, Hq = c["T"], c["Hq"]
        rows = torch.empty(T, Hq + 2 * Hkv, D, dtype=dt, device="cuda").normal_(generator=gen)
        s.q, s.k = rows[:, :Hq], rows[:, Hq:Hq + Hkv]
        if c["back"]:  # gradients come whole
            s.q, s.k = s.q.contiguous(), s.k.contiguous()
        n_doc = 1 + T // 4096
        start = torch.randint(0, c["far"], (n_doc,), generator=gen, device="cuda")
        at = torch.arange(T, device="cuda")
        s.positions = ((start[at % n_doc if T < 4096 else at // 4096] + at) % c["far"]).to(torch.int32)
        inv, scale = _frequencies(c)
        s.freqs = SimpleNamespace(inv_freq=inv, scale=scale)
        s.inv = torch.tensor(inv, device="cuda")
        s.rot, s.interleaved, s.back = c["rot"], c["interleaved"], c["back"]
        return s
    page = s.page = c["page"]
    if s.op == "read":
        # every second page of the cache is one of those asked for
        n_pages = 2 * c["n"] + 1
        s.kc, s.ks = _cache(gen, n_pages, page, Hkv, c["layout"], True)
        s.vc, s.vs = _cache(gen, n_pages, page, Hkv, c["layout"], True)
        s.pages = torch.randperm(n_pages, generator=gen, device="cuda")[:c["n"]].to(torch.int32)
        s.k, s.v = (torch.zeros(c["n"], page, Hkv, D, dtype=dt, device="cuda") for _ in range(2))
        return s
    lens = _lengths(c)
    need = [-(-(a + b) // page) for a, b in lens]
    width, n_pages, n = max(need) + 3, sum(need) + 8, c["n_seq"]
    n_rows = sum(b for _, b in lens) + c["pad"]
    ctx, new = torch.tensor([a for a, _ in lens], **i32), torch.tensor([b for _, b in lens], **i32)
    perm = torch.randperm(n_pages, generator=gen, device="cuda")
    counts = torch.tensor(need, device="cuda")
    first = counts.cumsum(0) - counts
    col = torch.arange(width, device="cuda")
    table = torch.where(col < counts[:, None], perm[(first[:, None] + col).clamp(max=n_pages - 1)], -1)
    s.kc, s.ks = _cache(gen, n_pages, page, Hkv, c["layout"], s.op == "attn")
    s.vc, s.vs = _cache(gen, n_pages, page, Hkv, c["layout"], s.op == "attn")
    q_start = [0]
    for _, b in lens:
        q_start.append(q_start[-1] + b)
    if s.op == "write":
        s.k, s.v = (torch.empty(n_rows, Hkv, D, dtype=dt, device="cuda").normal_(generator=gen) for _ in range(2))
        seq = torch.repeat_interleave(torch.arange(n, device="cuda"), new.long())
        pos = torch.arange(q_start[-1], device="cuda") - torch.tensor(q_start, device="cuda")[seq] + ctx[seq]
        slots = table[seq, pos // page] * page + pos % page
        s.slots = torch.cat([slots, slots.new_full((c["pad"],), -1)]).to(torch.int32)
        return s
    s.table = table.to(torch.int32)
    s.q = torch.empty(n_rows, c["Hq"], D, dtype=dt, device="cuda").normal_(generator=gen)
    s.q_start = torch.tensor(q_start, **i32)
    s.k_len = ctx + new
    s.mask = SimpleNamespace(kind=c["mask"], window_left=c["window"], window_right=0, num_global=c["sinks"])
    s.max_q, s.max_k = max(b for _, b in lens), max(a + b for a, b in lens)
    return s


# ------------------------------------------------------------------ the plain forms
def _rotate(s, x):
    """The pairs of x turned by position times frequency, or back."""
    angle = s.positions[:, None].double() * s.inv  # far positions lose their angle in 32 bits
    cos, sin = ((f(angle) * s.freqs.scale).float()[:, None] for f in (torch.cos, torch.sin))
    if s.back:
        sin = -sin
    h = s.rot // 2
    y = x.float()
    a, b = (y[..., 0:s.rot:2], y[..., 1:s.rot:2]) if s.interleaved else (y[..., :h], y[..., h:s.rot])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, v], -1).flatten(-2) if s.interleaved else torch.cat([u, v], -1)
    return torch.cat([turned, y[..., s.rot:]], -1).to(x.dtype)


def _write(s):
    """Rows whose slot is -1 are left out."""
    live = (s.slots >= 0).nonzero().flatten()
    at = s.slots[live].long()
    page, at = at // s.page, at % s.page
    for x, cache, factors in ((s.k, s.kc, s.ks), (s.v, s.vc, s.vs)):
        y, b = _quantise(x[live])
        cache.view(torch.uint8)[page, at] = y.view(torch.uint8)
        factors[page, :, at] = b
    return {"k": s.kc, "v": s.vc, "k_scale": s.ks, "v_scale": s.vs}


def _values(cache, factors, page, at):
    """The values that tokens `at` of pages `page` stand for: [.., Hkv, 128] in 32 bits."""
    return cache.view(torch.uint8)[page, at].view(E4M3).float() * _two_to(factors[page, :, at])[..., None]


def _read(s):
    p, at = s.pages.long()[:, None], torch.arange(s.page, device="cuda")
    s.k.copy_(_values(s.kc, s.ks, p, at))
    s.v.copy_(_values(s.vc, s.vs, p, at))
    return {"k": s.k, "v": s.v}


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
    page, at = s.table[:, j // s.page].long().clamp(min=0), (j % s.page).expand(n, -1)
    t = torch.arange(s.max_q, device="cuda")
    q = s.q[(q_start[:-1, None] + t).clamp(max=T - 1)].float() * (1 / math.sqrt(D))  # [n, max_q, Hq, D]
    q = q.view(n, s.max_q, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(n, Hkv, -1, D)
    scores = q @ _values(s.kc, s.ks, page, at).permute(0, 2, 3, 1)  # [n, Hkv, G * max_q, max_k]
    pos = (k_len - new)[:, None] + t
    ok = _attends(s.mask, pos[:, :, None], j, k_len[:, None, None]) & (t < new[:, None])[:, :, None]
    scores = scores.view(n, Hq, s.max_q, s.max_k).masked_fill_(~ok[:, None], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = p.view(n, Hkv, -1, s.max_k) @ _values(s.vc, s.vs, page, at).transpose(1, 2)
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

        if s.op == "rope":
            turn = lca.rope_bwd if s.back else lca.rope
            q, k = turn(s.q, s.k, s.positions, s.freqs, interleaved=s.interleaved)
            return {"q": q, "k": k}
        if s.op == "write":
            lca.paged_write_fp8(s.k, s.v, s.kc, s.vc, s.ks, s.vs, s.slots)
            return {"k": s.kc, "v": s.vc, "k_scale": s.ks, "v_scale": s.vs}
        if s.op == "read":
            k, v = lca.paged_read_fp8(s.kc, s.vc, s.ks, s.vs, s.pages, k_out=s.k, v_out=s.v)
            return {"k": k, "v": v}
        o, lse = lca.attn_paged_fp8(s.q, s.kc, s.vc, s.ks, s.vs, s.table, s.q_start, s.k_len, s.mask,
                                    max_q_len=s.max_q)
        return {"o": o, "lse": lse}
    if s.op == "rope":
        return {"q": _rotate(s, s.q), "k": _rotate(s, s.k)}
    return {"write": _write, "read": _read, "attn": _attn}[s.op](s)


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
    Hkv = c["Hkv"]
    if c["op"] == "rope":
        # rows read and written, a position each; two products and a sum for each value that turns
        heads = c["T"] * (c["Hq"] + Hkv)
        return {"bytes": heads * D * 4 + 4 * c["T"], "flops": 3 * heads * c["rot"]}
    if c["op"] == "read":  # K and V: values and a byte a row read, 16-bit values written
        return {"bytes": c["n"] * (4 + c["page"] * Hkv * 2 * (D + 1 + 2 * D)), "flops": 0}
    lens = _lengths(c)
    live = sum(b for _, b in lens)
    rows = live + c["pad"]
    if c["op"] == "write":
        return {"bytes": 4 * rows + live * Hkv * 2 * (2 * D + D + 1), "flops": 0}
    cells, keys = _cells(c)
    kv = 2 * keys * Hkv * (D + 1)
    return {"bytes": kv + rows * c["Hq"] * (2 * 2 * D + 4) + 4 * (keys // c["page"] + 2 * c["n_seq"] + 1),
            "flops": 4 * D * c["Hq"] * cells}


# ------------------------------------------------------------------ in 64 bits
def _exact_two_to(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_values(cache, factors):
    """[page, token, head, 128] values of whole pages."""
    return cache.to(torch.float64) * _exact_two_to(factors.transpose(1, 2).to(torch.int64) - 127)[..., None]


def _exact_rope(c, s):
    out = {}
    angle = s.positions.double()[:, None] * torch.tensor(_frequencies(c)[0], device="cuda")
    turn = torch.polar(torch.full_like(angle, _frequencies(c)[1]), -angle if c["back"] else angle)[:, None]
    for name, x in (("q", s.q), ("k", s.k)):
        y = x.double()
        part = y[..., :c["rot"]]
        z = part.unflatten(-1, (-1, 2)) if c["interleaved"] else part.unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
        y[..., :c["rot"]] = (z if c["interleaved"] else z.transpose(-1, -2)).flatten(-2)
        out[name] = y
    return out


def _exact_write(c, s):
    """Each value is the multiple of 2^-3 of its binade (2^-9 below 2^-6) nearest to x over the row's factor, the
    even one of two."""
    out = {}
    for name, x, cache in (("k", s.k, s.kc), ("v", s.v, s.vc)):
        x = x.double()
        top = x.abs().amax(-1, keepdim=True)
        e = torch.zeros_like(top, dtype=torch.int64) + LOWEST
        for k in range(LOWEST, HIGHEST):
            e += top > 448 * 2.0 ** k
        y = x / _exact_two_to(e)
        binade = (y.abs().clamp(min=2.0 ** -6).view(torch.int64) >> 52) - 1023
        step = _exact_two_to(binade - 3)
        y = (torch.round(y / step) * step).clamp(-448, 448)
        whole = cache.to(torch.float64)
        flat = whole.reshape(-1, *whole.shape[2:])
        live = s.slots >= 0
        flat[s.slots[live].long()] = y[live]
        out[name] = flat.view(whole.shape)
    return {**out, "k_scale": None, "v_scale": None}


def exact(c, seed):
    """The definitions in 64 bits; attention request by request and head by head."""
    s = prepare(c, seed)
    if c["op"] == "rope":
        return _exact_rope(c, s)
    if c["op"] == "write":
        return _exact_write(c, s)
    if c["op"] == "read":
        return {"k": _exact_values(s.kc[s.pages.long()], s.ks[s.pages.long()]),
                "v": _exact_values(s.vc[s.pages.long()], s.vs[s.pages.long()])}
    Hq, Hkv, G = c["Hq"], c["Hkv"], c["Hq"] // c["Hkv"]
    n_rows = s.q.shape[0]
    o = torch.zeros(n_rows, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((Hq, n_rows), -math.inf, dtype=torch.float64, device="cuda")
    r0 = 0
    for i, (ctx, new) in enumerate(_lengths(c)):
        length = ctx + new
        pages = s.table[i, :-(-length // c["page"])].long()
        qi = torch.arange(ctx, length, device="cuda")[:, None]
        kj = torch.arange(length, device="cuda")[None]
        w, g = c["window"], c["sinks"]
        hidden = {"FULL": lambda: kj < 0, "CAUSAL": lambda: kj > qi, "CAUSAL_SLIDING": lambda: (kj > qi) | (kj < qi - w),
                  "GLOBAL_SLIDING": lambda: (qi >= g) & (kj >= g) & ((kj > qi) | (kj < qi - w))}[c["mask"]]()
        for h in range(Hkv):
            keys, values = (_exact_values(x[:, :, h:h + 1].view(torch.uint8)[pages].view(E4M3), f[pages, h:h + 1]).reshape(-1, D)[:length]
                            for x, f in ((s.kc, s.ks), (s.vc, s.vs)))
            for head in range(h * G, h * G + G):
                x = s.q[r0:r0 + new, head].double() @ keys.T / math.sqrt(D)
                x.masked_fill_(hidden, -math.inf)
                z = torch.logsumexp(x, 1)
                lse[head, r0:r0 + new] = z
                o[r0:r0 + new, head] = x.sub_(z[:, None]).exp_() @ values
        r0 += new
    return {"o": o, "lse": lse}
