"""The paged-cache operators on the GPU: the plan against a plain loop, the
writes exactly, attention against the fp64 oracle within bounds derived from
the roundings (tests/paged_util.py), and the three together."""
from __future__ import annotations

import numpy as np
import pytest

from gen import MaskSpec, Segment
from tests.paged_util import MASKS, Paged, check, lay_out, make, reference

pytestmark = pytest.mark.gpu
CAUSAL = MaskSpec("CAUSAL")


# ------------------------------------------------------------------ plan
def loop_plan(ctx, new, free, taken, table, page, n_pages, n_rows):
    table = table.copy()
    room = table.shape[1] * page
    used, row, bad = min(max(taken, 0), len(free)), 0, 0
    short = 0
    q_start, k_len = [0], []
    slots, pos = np.full(n_rows, -1), np.zeros(n_rows, dtype=np.int64)
    for i, (c0, w0) in enumerate(zip(ctx.tolist(), new.tolist())):
        c, w = min(max(c0, 0), room), max(w0, 0)
        total = min(c + w, room)
        wrong = c0 < 0 or w0 < 0 or c0 > room or c + w > room or row + w > n_rows
        for e in range(-(-c // page), -(-total // page)):
            if used < len(free):
                p = free[used]
                used += 1
            else:
                p, short = -1, short + 1
            table[i, e] = p if 0 <= p < n_pages else -1
        for t in range(w):
            if row + t >= n_rows:
                break
            pos[row + t] = c + t
            if c + t < room and 0 <= table[i, (c + t) // page] < n_pages:
                slots[row + t] = table[i, (c + t) // page] * page + (c + t) % page
        row += w
        bad += wrong
        q_start.append(min(row, n_rows))
        k_len.append(total)
    return table, q_start, k_len, slots, pos, [used, short, bad, min(row, n_rows)]


def run_plan(lca, ctx, new, free, taken, table, page, n_pages, n_rows):
    import torch

    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    t = i32(table)
    p = lca.paged_plan(i32(ctx), i32(new), i32(free), i32([taken]), t, page, n_pages, n_rows)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (t, p.q_start, p.k_len, p.slots, p.positions, p.state)]


def same_plan(got, want):
    for name, g, w in zip(("table", "q_start", "k_len", "slots", "positions", "state"), got, want):
        np.testing.assert_array_equal(g, np.asarray(w), err_msg=name)


@pytest.mark.parametrize("n,page,most_new,pad,seed", [
    (1, 16, 1, 0, 0), (1, 8, 5000, 3, 1), (7, 16, 1, 0, 2), (33, 24, 40, 7, 3), (1024, 16, 3, 0, 4), (1025, 64, 30, 9000, 5),
    (2500, 32, 12, 1, 6), (0, 16, 1, 5, 7), (300, 8, 0, 0, 8),
])
def test_plan(lca, n, page, most_new, pad, seed):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, 300, n)
    new = rng.integers(0, most_new + 1, n)
    width = int(max([0, *(ctx + new)])) // page + 2
    have = -(-ctx // page)
    n_pages = int((-(-(ctx + new) // page)).sum()) + 20
    perm = rng.permutation(n_pages)
    table = np.full((n, width), -1)
    at = 0
    for i in range(n):
        table[i, :have[i]] = perm[at:at + have[i]]
        at += have[i]
    free = np.concatenate([perm[:4], perm[at:]])
    args = (ctx, new, free, 4, table, page, n_pages, int(new.sum()) + pad)
    want = loop_plan(*args)
    assert want[-1][1] == want[-1][2] == 0
    same_plan(run_plan(lca, *args), want)


@pytest.mark.parametrize("over", [
    dict(n_free=3), dict(n_free=0), dict(taken=-5), dict(taken=1 << 30), dict(rows=5), dict(rows=0), dict(width=2),
    dict(bad_ctx=True), dict(bad_free=True), dict(bad_table=True),
], ids=str)
def test_plan_answers_what_cannot_be_served(lca, over):
    """Too few pages, rows or table entries, negative lengths, entries that
    are no pages: -1 in their place and the counts in state."""
    ctx, new = np.array([3, 16, 0, 40, 7]), np.array([2, 20, 5, 0, 30])
    if "bad_ctx" in over:
        ctx, new = np.array([3, -16, 2**31 - 1, 40, 7]), np.array([2, 20, 5, -2**31, 30])
    width, n_pages = over.get("width", 4), 30
    table = np.full((5, width), -1)
    at = 0
    for i in range(5):
        for e in range(min(width, max(0, -(-int(ctx[i]) // 16)))):
            table[i, e], at = at, at + 1
    if "bad_table" in over:
        table[0, 0], table[4, 0] = 30, -7
    free = np.arange(12, 12 + over.get("n_free", 9))
    if "bad_free" in over:
        free[1], free[2] = 30, -4
    args = (ctx, new, free, over.get("taken", 0), table, 16, n_pages, over.get("rows", 60))
    same_plan(run_plan(lca, *args), loop_plan(*args))


def test_plan_can_be_repeated_and_refuses_aliases(lca):
    import torch

    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ctx, new, free, taken = i32(5, 16), i32(20, 1), i32(4, 3, 2, 1, 0), i32(0)
    table = torch.full((2, 6), -1, dtype=torch.int32, device="cuda")
    table[:, 0] = i32(7, 8)
    wide = table.clone()
    a = lca.paged_plan(ctx, new, free, taken, table[:, :4], 16, 9, 21)
    first = table.clone()
    b = lca.paged_plan(ctx, new, free, taken, table[:, :4], 16, 9, 21)
    assert torch.equal(first, table) and torch.equal(a.slots, b.slots) and torch.equal(a.state, b.state)
    assert table.tolist() == [[7, 4, -1, -1, -1, -1], [8, 3, -1, -1, -1, -1]]
    assert torch.equal(wide[:, 4:], table[:, 4:])
    c = lca.paged_plan(a.k_len, i32(8, 0), free, a.state[:1], table[:, :4], 16, 9, 8)
    assert c.state.tolist() == [3, 0, 0, 8] and c.slots.tolist() == [4 * 16 + 9 + t for t in range(7)] + [2 * 16]
    for kw in (dict(k_len=ctx), dict(state=torch.cat([taken, i32(0, 0, 0)])), dict(q_start=free[:3])):
        if "state" in kw:
            with pytest.raises(lca.LcaError, match="INVALID"):
                lca.paged_plan(ctx, new, free, kw["state"][:1], table, 16, 9, 21, **kw)
        else:
            with pytest.raises(lca.LcaError, match="INVALID"):
                lca.paged_plan(ctx, new, free, taken, table, 16, 9, 21, **kw)


# ------------------------------------------------------------------ write
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "kv"])
@pytest.mark.parametrize("T,Hkv,page", [(1, 1, 8), (64, 8, 16), (133, 3, 24), (2000, 2, 256), (0, 2, 8)])
def test_write(lca, T, Hkv, page, layout, dtype):
    import torch

    g = torch.Generator().manual_seed(T + Hkv)
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    n_pages = T // page + 3
    lk, lv = (torch.randn(n_pages, page, Hkv, 128, generator=g).to(dt) for _ in range(2))
    kc, vc = lay_out(lk, lv, layout, "cuda")
    slots = torch.randperm(n_pages * page, generator=g)[:T].to(torch.int32)
    slots[::5] = -1
    slots[1::7] = n_pages * page + 3  # outside: skipped
    # rows as parts of a wider projection
    qkv = torch.randn(T, 3 * Hkv, 128, generator=g).to(dt)
    k, v = qkv[:, Hkv:2 * Hkv], qkv[:, 2 * Hkv:]
    dev = qkv.cuda()
    lca.paged_write(dev[:, Hkv:2 * Hkv], dev[:, 2 * Hkv:], kc, vc, slots.cuda())
    ok = ((slots >= 0) & (slots < n_pages * page)).nonzero().flatten()
    at = slots[ok].long()
    lk[at // page, at % page] = k[ok]
    lv[at // page, at % page] = v[ok]
    assert torch.equal(kc.cpu().contiguous().view(torch.int16), lk.view(torch.int16))
    assert torch.equal(vc.cpu().contiguous().view(torch.int16), lv.view(torch.int16))


def test_write_of_one_slot_twice_stores_rows_of_the_call(lca):
    import torch

    kc, vc = (torch.zeros(4, 8, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k = torch.ones(6, 2, 128, dtype=torch.bfloat16, device="cuda") * torch.arange(1, 7, device="cuda")[:, None, None]
    lca.paged_write(k, k, kc, vc, torch.tensor([3, 9, 3, 3, 11, 9], dtype=torch.int32, device="cuda"))
    flat = kc.view(32, 256).float()
    assert bool(torch.isin(flat[3], torch.tensor([1.0, 3.0, 4.0], device="cuda")).all())
    assert bool(torch.isin(flat[9], torch.tensor([2.0, 6.0], device="cuda")).all()) and bool((flat[11] == 5).all())
    assert float(flat.sum(1)[[0, 1, 2, 4, 5, 6, 7, 8, 10, 12]].abs().max()) == 0


def test_write_from_the_cache_itself_is_refused(lca):
    """Rows that are read while others are written would be either."""
    import torch

    kc, vc = (torch.arange(4 * 8 * 2 * 128, device="cuda").view(4, 8, 2, 128).to(torch.bfloat16) for _ in range(2))
    before = kc.clone(), vc.clone()
    k = torch.zeros(6, 2, 128, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(6, dtype=torch.int32, device="cuda")
    rows = kc.view(32, 2, 128)
    inside = vc.view(-1)[:512].view(torch.int32)[:6]
    for args in ((rows[8:14], k, slots), (k, rows[26:], slots), (k, vc.view(32, 2, 128)[3:9], slots), (k, k, inside)):
        with pytest.raises(lca.LcaError, match="INVALID"):
            lca.paged_write(args[0], args[1], kc, vc, args[2])
    assert torch.equal(kc, before[0]) and torch.equal(vc, before[1])


# ------------------------------------------------------------------ attention
def attend(lca, p: Paged, **kw):
    import torch

    need = lca.attn_paged_workspace_size(p.q, p.kc, p.vc, p.table, p.prob.mask)
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")  # nothing may depend on what it held
    o = torch.full(p.q.shape, 7.0, dtype=p.q.dtype, device="cuda")
    lse = torch.full((p.prob.Hq, p.prob.Tq), 7.0, device="cuda")
    lca.attn_paged(p.q, p.kc, p.vc, p.table, p.q_start, p.k_len, p.prob.mask, p.prob.scale, out=o, lse=lse, workspace=ws,
                   **kw)
    torch.cuda.synchronize()
    return o, lse, lca.read_status(ws)


DECODE = [(0, 1), (7, 1), (126, 1), (127, 1), (128, 1), (1000, 1), (31, 1)]
CHUNKS = [(0, 1), (0, 130), (300, 257), (0, 0), (64, 64), (5, 0), (1, 2), (511, 17)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (16, 2), (3, 3), (12, 4), (10, 2), (32, 1), (24, 1), (40, 1)])
def test_decode(lca, Hq, Hkv, dtype):
    p = make(DECODE, 16, Hq, Hkv, CAUSAL, dtype, pad=2, seed=Hq, device="cuda")
    ref = reference(p)
    for hint in (0, 1, 300):
        o, lse, st = attend(lca, p, max_q_len=hint)
        check(o, lse, p, ref, what=f"max_q_len={hint}")
        assert st == (0, 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (2, 2), (6, 2), (5, 1), (16, 1), (48, 1), (14, 2)])
def test_chunks(lca, Hq, Hkv, dtype):
    p = make(CHUNKS, 32, Hq, Hkv, CAUSAL, dtype, pad=3, seed=Hq, device="cuda")
    ref = reference(p)
    for hint in (0, 257):
        o, lse, st = attend(lca, p, max_q_len=hint)
        check(o, lse, p, ref, what=f"max_q_len={hint}")
        assert st == (0, 0)


@pytest.mark.parametrize("layout", ["nhd", "hnd", "kv"])
@pytest.mark.parametrize("page", [8, 16, 24, 40, 48, 64, 128, 136, 256, 1024])
def test_pages_and_layouts(lca, page, layout):
    """Pages that end inside a tile, at it and past it; the cache holds NaN
    wherever no request's token lies."""
    p = make([(0, 1), (250, 3), (129, 140), (page, 1), (2 * page - 1, 2)], page, 8, 2, CAUSAL, "fp16", layout, seed=page,
             device="cuda")
    o, lse, st = attend(lca, p)
    check(o, lse, p)
    assert st == (0, 0)


@pytest.mark.parametrize("mask", MASKS, ids=lambda m: f"{m.kind}{m.window_left or ''}")
@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (3, 1)])
def test_masks(lca, mask, Hq, Hkv):
    """Every family; in the last two requests the cache holds fewer keys than
    there are new tokens, so that causal rows before the first key are empty."""
    p = make([(0, 1), (600, 1), (99, 1), (0, 200), (333, 100), (150, 5)], 16, Hq, Hkv, mask, seed=3, device="cuda")
    o, lse, st = attend(lca, p)
    check(o, lse, p, what=mask.kind)
    assert st == (0, 0)


@pytest.mark.parametrize("mask", [CAUSAL, MASKS[4], MASKS[7], MASKS[8]], ids=lambda m: m.kind)
def test_rows_that_attend_nothing(lca, mask):
    """More new tokens than keys: the first of them have no key at or before them."""
    import torch

    p = make([(0, 40), (0, 9), (0, 300)], 16, 8, 2, mask, seed=9, device="cuda")
    p.k_len = torch.tensor([11, 0, 7], dtype=torch.int32, device="cuda")
    segs = p.prob.segments
    for s, n in zip(segs, (11, 0, 7)):
        s.k_len = n
    ref = reference(p)
    assert np.isneginf(ref[1]).any()
    o, lse, st = attend(lca, p)
    check(o, lse, p, ref)
    assert st == (0, 0)


@pytest.mark.parametrize("mask", [CAUSAL, MaskSpec("CAUSAL_SLIDING", window_left=100), MaskSpec("FULL"),
                                  MaskSpec("GLOBAL_SLIDING", window_left=300, window_right=0, num_global=10)],
                         ids=lambda m: m.kind)
@pytest.mark.parametrize("new", [1, 2, 20, 200])
def test_long_contexts_split_over_keys(lca, mask, new):
    """One request with far more keys than rows, and a batch of uneven ones."""
    p = make([(6000, new)], 64, 8, 1, mask, seed=new, device="cuda")
    check(*attend(lca, p)[:2], p)
    p = make([(3000, new), (1, 1), (0, 1), (2500, 1), (17, new)], 64, 4, 2, mask, "fp16", seed=new, device="cuda")
    check(*attend(lca, p)[:2], p)


@pytest.mark.parametrize("value", ["inf", "-inf", "nan", "65504"])
@pytest.mark.parametrize("new", [1, 3, 150])
def test_hidden_keys_reach_nothing(lca, value, new):
    """Keys in the pages before a sliding window, and all slots no request
    owns, hold infinities, NaN or the type's largest value; the results are
    those of a cache that holds zeros there, bit for bit."""
    import torch

    mask = MaskSpec("CAUSAL_SLIDING", window_left=77)
    outs = []
    for fill in (float(value), 0.0):
        p = make([(400, new), (9, new), (128, new)], 16, 8, 2, mask, "fp16", fill=fill, seed=5, device="cuda")
        hidden = 400 - 77  # no new token of request 0 sees a key before this
        for j in range(hidden):
            page, at = int(p.table[0, j // 16]), j % 16
            p.kc[page, at] = fill
            p.vc[page, at] = fill
        outs.append(attend(lca, p))
    (o, lse, st), (o0, lse0, _) = outs
    assert st == (0, 0)
    assert torch.equal(o, o0) and torch.equal(lse, lse0)
    check(o, lse, p)


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_later_tokens_infinities_reach_no_earlier_row(lca, value):
    """A new token whose key or value is not finite is hidden from the rows
    before it: those rows keep their results."""
    import torch

    for lens, bad in (([(50, 9)], 55), ([(0, 300)], 200), ([(1000, 40)], 1001), ([(130, 2)], 131)):
        p = make(lens, 16, 8, 2, CAUSAL, seed=6, device="cuda")
        ref = attend(lca, p)
        page, at = int(p.table[0, bad // 16]), bad % 16
        p.vc[page, at, :, ::3] = value
        p.kc[page, at, :, 5] = value
        o, lse, _ = attend(lca, p)
        first = bad - lens[0][0]  # the row of the token itself
        assert bool(torch.isfinite(o[:first]).all())
        p.prob.segments[0].q_len = first
        check(o[:first], lse[:, :first], cut(p, first))
        assert not bool(torch.isfinite(o[first:]).all()) and torch.equal(ref[0][:0], o[:0])


def cut(p, rows):
    p.q = p.q[:rows]
    p.prob.Tq = rows
    s = p.prob.segments[0]
    new_keys = p.k.shape[0] - p.prob.extra.setdefault("tail", 0)
    s.k_len = int(p.k_len[0]) - (int(p.q_start[1]) - rows)
    assert s.k_len <= new_keys
    return p


def test_infinities_among_a_long_contexts_last_keys(lca):
    """The rows before such a token are found again without it, in time."""
    for lens, bad in (([(60000, 40)], 60030), ([(40000, 300)], 40100)):
        p = make(lens, 64, 4, 1, CAUSAL, "fp16", seed=16, device="cuda")
        page, at = int(p.table[0, bad // 64]), bad % 64
        p.vc[page, at, 0, 7] = float("inf")
        o, lse, st = attend(lca, p)
        assert st == (0, 0)
        first = bad - lens[0][0]
        p.prob.segments[0].q_len = first
        check(o[:first], lse[:, :first], cut(p, first))
        assert bool((o[first:, :, 7] == float("inf")).all()) and bool(o[first:, :, :7].isfinite().all())


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("lens,bads", [
    ([(0, 100)], [3, 60]),                         # the only tile of its items
    ([(0, 9), (3, 15), (500, 11)], [4, 6, 505]),   # narrow items, one after another
    ([(0, 700)], list(range(5, 700, 64))),         # every item, several tiles each
    ([(1000, 300), (5, 260), (2, 13)], [1000, 1130, 1299, 100, 8]),
    ([(126, 14), (254, 14)], [127, 128, 255, 256]),  # two tiles of a narrow item in turn
], ids=str)
def test_several_tiles_with_infinities(lca, lens, bads, value):
    """Every row equals the one that a cache without the infinities that it
    does not attend gives; those that attend one have it in that column only."""
    import torch

    p = make(lens, 16, 8, 2, CAUSAL, seed=len(bads), device="cuda")
    ref = reference(p)
    o0, lse0, _ = attend(lca, p)
    check(o0, lse0, p, ref)
    hit = torch.zeros(p.q.shape[0], dtype=torch.bool)
    row = 0
    for i, (ctx, new) in enumerate(lens):
        mine = [b for b in bads if ctx <= b < ctx + new]
        for b in mine:
            p.vc[int(p.table[i, b // 16]), b % 16, :, 77] = value
        if mine:
            hit[row + min(mine) - ctx:row + new] = True
        row += new
    assert bool(hit.any()) and not bool(hit.all())
    for _ in range(3):
        o, lse, st = attend(lca, p)
        assert st == (0, 0)
        hid = hit.nonzero().flatten().cuda()
        assert not bool(o[hid][:, :, 77].isfinite().any())
        o[hid, :, 77] = o0[hid, :, 77]  # all else within its bound
        check(o, lse, p, ref)


@pytest.mark.parametrize("mask", MASKS, ids=lambda m: f"{m.kind}{m.window_left or ''}")
@pytest.mark.parametrize("Hq", [8, 3])
def test_infinities_reach_the_rows_that_attend_them(lca, mask, Hq):
    """Under every family: a column of the values of a few keys holds infinities;
    it is not finite in the rows that attend one of them, all else as without."""
    import torch

    from oracle.masks import segment_mask

    lens = [(600, 1), (0, 200), (333, 100), (150, 5), (1000, 300)]
    p = make(lens, 16, Hq, 1, mask, seed=Hq, device="cuda")
    ref = reference(p)
    o0, lse0, _ = attend(lca, p)
    check(o0, lse0, p, ref, what=mask.kind)
    hit = torch.zeros(p.q.shape[0], dtype=torch.bool)
    for i, seg in enumerate(p.prob.segments):
        bads = [2, 64, 65, 127, seg.k_len // 2, seg.k_len - 3, seg.k_len - 60]
        bads = [b for b in bads if 0 <= b < seg.k_len]
        for b in bads:
            p.vc[int(p.table[i, b // 16]), b % 16, :, 77] = float("inf")
        hit[seg.q_off:seg.q_off + seg.q_len] = torch.from_numpy(segment_mask(mask, i, seg)[:, bads].any(1))
    for _ in range(2):
        o, lse, st = attend(lca, p)
        assert st == (0, 0) and torch.equal(lse, lse0)
        assert not bool(o[hit.cuda()][:, :, 77].isfinite().any()), mask.kind
        o[hit.cuda(), :, 77] = o0[hit.cuda(), :, 77]
        check(o, lse, p, ref, what=mask.kind)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("new", [1, 3, 300])
def test_an_infinity_of_small_weight_is_not_lost(lca, new, dtype):
    """A context in pieces, whose first keys have some 2^-260 of the last ones'
    weight: an infinity or NaN among their values still reaches every row that
    attends it, as a weight is never zero."""
    import torch

    ctx, hit = 16000, 100
    p = make([(ctx, new), (20, 1)], 64, 8, 1, CAUSAL, dtype, seed=new, device="cuda")
    p.q.fill_(8.0)
    for j in range(0, ctx + new, 64):
        p.kc[int(p.table[0, j // 64])] = -1.0 if j < ctx // 2 else 1.0
    o0, lse0, _ = attend(lca, p)
    assert bool(o0.isfinite().all())
    for value in (float("inf"), float("nan")):
        p.vc[int(p.table[0, hit // 64]), hit % 64, 0, 77] = value
        o, lse, st = attend(lca, p)
        assert st == (0, 0) and torch.equal(lse, lse0)
        assert not bool(o[:new, :, 77].isfinite().any())
        o[:new, :, 77] = o0[:new, :, 77]
        assert torch.equal(o, o0)


def test_infinities_among_a_very_long_contexts_last_keys(lca):
    """Pieces of hundreds of thousands of keys, with one value that is not
    finite: what it costs goes by its tile, not by the piece."""
    import torch

    ctx, new, page, Hkv = 786432, 2048, 64, 8
    n = (ctx + new) // page
    g = torch.Generator(device="cuda").manual_seed(3)
    kc, vc = (torch.rand(n, page, Hkv, 128, device="cuda", generator=g, dtype=torch.bfloat16) - 0.5 for _ in range(2))
    q = torch.rand(new, 8 * Hkv, 128, device="cuda", generator=g, dtype=torch.bfloat16) - 0.5
    table = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    q_start, k_len = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, new], [ctx + new]))
    ws = torch.empty(lca.attn_paged_workspace_size(q, kc, vc, table, CAUSAL), dtype=torch.uint8, device="cuda")
    call = lambda: lca.attn_paged(q, kc, vc, table, q_start, k_len, CAUSAL, workspace=ws)  # noqa: E731
    o0, lse0 = call()
    bad = ctx + 1000
    vc[bad // page, bad % page, :, 9] = float("inf")
    o, lse = call()
    assert lca.read_status(ws) == (0, 0)
    assert torch.equal(lse, lse0)  # no score changed
    assert bool((o[1000:, :, 9] == float("inf")).all()) and bool(o[:1000].isfinite().all())
    o[1000:, :, 9] = o0[1000:, :, 9]
    # both are roundings of sums whose weights are off by 2^-8 at most, |v| <= 1/2
    assert float((o.float() - o0.float()).abs().max()) <= 2 * (2.0**-8 * 0.5 + 2.0**-8 * 0.5)


@pytest.mark.parametrize("new", [1, 3, 90])
def test_pages_between_sinks_and_window_may_be_gone(lca, new):
    """GLOBAL_SLIDING over a long context: the table has no entry, and the
    cache NaN, between the first keys and the window of the first new token."""
    mask = MaskSpec("GLOBAL_SLIDING", window_left=200, window_right=0, num_global=20)
    p = make([(3000, new), (900, new)], 16, 8, 2, mask, seed=new, device="cuda")
    ref = reference(p)
    for i, ctx in enumerate((3000, 900)):
        for e in range(2, (ctx - 200) // 16):
            page = int(p.table[i, e])
            p.kc[page] = float("nan")
            p.vc[page] = float("nan")
            p.table[i, e] = -1
    o, lse, st = attend(lca, p)
    assert st == (0, 0)
    check(o, lse, p, ref)


@pytest.mark.parametrize("Hq", [64, 100, 128, 136, 260])
def test_many_heads_of_one_group(lca, Hq):
    """More heads than rows of a tile among them."""
    p = make([(200, 1), (0, 5), (130, 3)], 16, Hq, 1, CAUSAL, seed=Hq, device="cuda")
    o, lse, st = attend(lca, p)
    check(o, lse, p)
    assert st == (0, 0)


def test_many_requests(lca):
    """More requests than are placed at once, some without new tokens, some
    with no keys, short and long ones mixed."""
    rng = np.random.default_rng(5)
    lens = [(int(rng.integers(0, 260)), int(rng.choice([0, 1, 1, 1, 2, 5, 40]))) for _ in range(1100)]
    p = make(lens, 8, 4, 1, CAUSAL, "fp16", pad=9, seed=17, device="cuda")
    ref = reference(p)
    for hint in (0, 40):
        o, lse, st = attend(lca, p, max_q_len=hint)
        check(o, lse, p, ref)
        assert st == (0, 0)


def test_long_lines_are_claimed(lca):
    """Enough keys that the last part of the work is claimed by the CTAs that
    are done first; the results do not depend on who was."""
    import torch

    p = make([(90000, 1), (70000, 1), (52000, 1), (3, 1)], 128, 16, 16, CAUSAL, seed=18, device="cuda")
    o, lse, st = attend(lca, p)
    assert st == (0, 0)
    check(o, lse, p)
    for _ in range(4):
        o2, lse2, _ = attend(lca, p)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_pages_far_apart(lca):
    """Pages more than 2^31 elements apart, read and written."""
    import torch

    far = (1 << 31) + 64
    buf = torch.empty(3 * far + 4096, dtype=torch.bfloat16, device="cuda")
    for new in (1, 60):
        p = make([(20, new)], 32, 8, 2, CAUSAL, seed=new, device="cuda")
        n = p.kc.shape[0]
        assert n <= 6
        keep = [int(x) for x in p.table[0] if x >= 0]
        view = lambda at: buf.as_strided((3, 32, 2, 128), (far, 256, 128, 1), at)  # noqa: E731
        kc, vc = view(0), view(64 * 256)
        table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
        for i, page in enumerate(keep):
            kc[table[0, i]] = p.kc[page]
            vc[table[0, i]] = p.vc[page]
        p.kc, p.vc, p.table = kc, vc, table
        o, lse, st = attend(lca, p)
        assert st == (0, 0)
        check(o, lse, p)
        # the new tokens' rows again through the write
        slots = torch.tensor([int(table[0, j // 32]) * 32 + j % 32 for j in range(20, 20 + new)], dtype=torch.int32)
        before = [kc[int(s) // 32, int(s) % 32].clone() for s in slots]
        for s in slots:
            kc[int(s) // 32, int(s) % 32] = 0
        lca.paged_write(p.k[20:].cuda(), p.v[20:].cuda(), kc, vc, slots.cuda())
        assert all(torch.equal(b, kc[int(s) // 32, int(s) % 32]) for b, s in zip(before, slots))


@pytest.mark.parametrize("order", [(0, 1, 2), (1, 0, 2), (2, 0, 1), (1, 2, 0), (0, 2, 1), (2, 1, 0)], ids=str)
def test_any_order_of_the_axes(lca, order):
    """The cache's axes (page, token, head) in every order in memory."""
    p = make([(40, 1), (10, 90), (70, 4)], 24, 6, 2, CAUSAL, "fp16", seed=3, device="cuda")
    back = [order.index(i) for i in range(3)] + [3]
    p.kc, p.vc = (x.permute(*order, 3).contiguous().permute(*back) for x in (p.kc, p.vc))
    o, lse, st = attend(lca, p)
    check(o, lse, p)
    assert st == (0, 0)


def test_narrow_items_among_wide_ones_repeat(lca):
    """Items of one sub-tile between items of two, many times over."""
    import torch

    p = make(CHUNKS * 3, 32, 8, 1, CAUSAL, "fp16", seed=8, device="cuda")
    ref = reference(p)
    a = attend(lca, p)
    check(a[0], a[1], p, ref)
    for _ in range(60):
        b = attend(lca, p)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_narrow_items_never_wait_in_vain(lca):
    """Many calls of nothing but narrow items with long and short pieces: no
    wait runs out (a wait that could miss its phase did so once in some
    thousand items)."""
    import torch

    p = make([(int(c), 5) for c in np.linspace(200, 5000, 24)], 32, 16, 2, CAUSAL, seed=21, device="cuda")
    need = lca.attn_paged_workspace_size(p.q, p.kc, p.vc, p.table, CAUSAL)
    first = None
    for _ in range(6):
        spaces = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(50)]
        outs = [lca.attn_paged(p.q, p.kc, p.vc, p.table, p.q_start, p.k_len, CAUSAL, workspace=w) for w in spaces]
        torch.cuda.synchronize()
        first = first or outs[0]
        for w, (o, lse) in zip(spaces, outs):
            assert lca.read_status(w) == (0, 0)
            assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    check(first[0], first[1], p)


def test_overlapping_outputs_are_refused(lca):
    import torch

    p = make([(40, 3)], 16, 8, 8, CAUSAL, seed=2, device="cuda")
    call = lambda **kw: lca.attn_paged(p.q, p.kc, p.vc, p.table, p.q_start, p.k_len, CAUSAL, **kw)  # noqa: E731
    o, lse = call()
    flat = torch.empty(4096, dtype=torch.float32, device="cuda")
    for kw in (dict(out=p.q), dict(out=p.kc[0, :3]), dict(out=flat[:1536].view(torch.bfloat16).view(3, 8, 128), lse=flat[1000:1024].view(8, 3))):
        with pytest.raises(lca.LcaError, match="INVALID"):
            call(**kw)


@pytest.mark.parametrize("rows", [0, 3])
def test_a_workspace_inside_an_input_is_refused(lca, rows):
    """Whatever the batch: one without rows writes its workspace too."""
    import torch

    p = make([(40, 3)], 16, 8, 8, CAUSAL, seed=2, device="cuda")
    q, starts = p.q[:rows], torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    need = lca.attn_paged_workspace_size(p.q, p.kc, p.vc, p.table, CAUSAL)
    buf = torch.zeros(need + 4096, dtype=torch.uint8, device="cuda")
    ints = buf[1024:].view(torch.int32)
    kc = buf[:need // 4096 // 16 * 4096 * 16].view(torch.bfloat16).view(-1, 16, 8, 128)
    assert kc.numel() * 2 >= need - 65536
    kw = dict(q_start=starts, k_len=p.k_len, block_table=p.table, k_cache=p.kc, v_cache=p.vc)
    for over in (dict(k_cache=kc, v_cache=kc), dict(q_start=ints[:2]), dict(k_len=ints[:1]), dict(ctx_len=ints[:1]),
                 dict(block_table=ints[:8].view(1, 8))):
        with pytest.raises(lca.LcaError, match="INVALID"):
            lca.attn_paged(q, mask=CAUSAL, workspace=buf[:need], **{**kw, **over})
    assert not bool(buf.any())
    lca.attn_paged(q, mask=CAUSAL, workspace=buf[:need], **kw)
    assert lca.read_status(buf) == (0, 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_large_scores_and_an_explicit_scale(lca, dtype):
    """Scores of some hundreds (one key takes all), and a scale of the user's own."""
    import torch

    p = make([(500, 1), (100, 60)], 16, 8, 2, CAUSAL, dtype, seed=8, q_scale=100.0, device="cuda")
    o, lse, _ = attend(lca, p)
    assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(lse).all())
    check(o, lse, p)
    p = make([(500, 1), (100, 60)], 16, 8, 2, CAUSAL, dtype, seed=8, device="cuda")
    p.prob.scale = 0.3
    check(*attend(lca, p)[:2], p)


@pytest.mark.parametrize("lens", [[(300, 1), (20, 1)], [(300, 200), (20, 1)]], ids=str)
def test_bad_pages_and_lengths_are_reported(lca, lens):
    """Table entries that are no pages read as zeros; lengths that the
    tensors do not hold are clamped; each sets the status."""
    import torch

    p = make(lens, 16, 8, 2, CAUSAL, seed=4, device="cuda")
    assert attend(lca, p)[2] == (0, 0)
    for bad in (-1, p.kc.shape[0], 2**31 - 1, -2**31):
        q = make(lens, 16, 8, 2, CAUSAL, seed=4, device="cuda")
        q.table[0, 3] = bad
        o, lse, st = attend(lca, q)
        assert st[0] == 6
        q.k[48:64] = 0
        q.v[48:64] = 0
        check(o, lse, q)
    # an entry behind the last key, or before the window, is not needed
    q = make(lens, 16, 8, 2, MaskSpec("CAUSAL_SLIDING", window_left=30), seed=4, device="cuda")
    q.table[0, 0] = 1 << 20
    q.table[1, -1] = -9
    o, lse, st = attend(lca, q)
    assert st == (0, 0)
    check(o, lse, q)
    room = p.table.shape[1] * 16
    for name, i, x in (("k_len", 0, -4), ("k_len", 1, room + 1), ("k_len", 0, 2**31 - 1), ("q_start", 2, 2**31 - 1),
                       ("q_start", 1, -3), ("q_start", 0, -2**31), ("q_start", 1, 10**6)):
        q = make(lens, 16, 8, 2, CAUSAL, fill=0.0, seed=4, device="cuda")
        getattr(q, name)[i] = x
        assert attend(lca, q)[2][0] == 6, (name, i, x)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_a_bad_request_spoils_no_other(lca, dtype):
    """A page or a length that cannot be used, in one request of a batch whose
    items take longer than a wait's first polls: the call goes on, and every
    row is, bit for bit, that of a call with zeros in the page's place, or with
    the length that the bad one is clamped to."""
    import torch

    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    g = torch.Generator(device="cuda").manual_seed(5)
    page, Hkv, G = 64, 8, 8
    lens = [(300, 5)] + [(30000 + 17 * i, 5) if i % 2 else (200, 20) for i in range(24)] + [
        (120000, 5), (110000, 300), (900, 1), (30000, 300), (300, 40), (64000, 1)]
    n = len(lens)
    need = [-(-(c + w) // page) for c, w in lens]
    n_pages = sum(need) + 1
    kc, vc = (torch.randn(n_pages, page, Hkv, 128, device="cuda", generator=g).to(dt) for _ in range(2))
    table = torch.full((n, max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = torch.arange(at, at + m, dtype=torch.int32, device="cuda")
        at += m
    kc[at], vc[at] = 0, 0  # the last page
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q_start, k_len = i32(np.cumsum([0] + [w for _, w in lens])), i32([c + w for c, w in lens])
    q = torch.randn(int(q_start[-1]), Hkv * G, 128, device="cuda", generator=g).to(dt)
    ws = torch.full((lca.attn_paged_workspace_size(q, kc, vc, table, CAUSAL),), 0xA5, dtype=torch.uint8, device="cuda")

    def call(table, k_len):
        o, lse = torch.full_like(q, 7.0), torch.full((Hkv * G, q.shape[0]), 7.0, device="cuda")
        lca.attn_paged(q, kc, vc, table, q_start, k_len, CAUSAL, out=o, lse=lse, workspace=ws)
        return o, lse, lca.read_status(ws)[0]

    def put(t, *at, value):
        t = t.clone()
        t[at] = value
        return t

    for who in (0, n - 2, n - 1):  # served by the kernel for many rows, and by the one for few
        want = call(put(table, who, 3, value=at), k_len)
        bad = call(put(table, who, 3, value=-1), k_len)
        assert want[2] == 0 and bad[2] == 6
        assert torch.equal(want[0], bad[0]) and torch.equal(want[1], bad[1])
    want, bad = call(table, put(k_len, 0, value=0)), call(table, put(k_len, 0, value=-5))
    assert want[2] == 0 and bad[2] == 6
    assert torch.equal(want[0], bad[0]) and torch.equal(want[1], bad[1])


def test_q_rows_of_a_wider_projection_and_no_requests(lca):
    import torch

    p = make([(40, 3), (0, 70)], 16, 8, 2, CAUSAL, seed=2, device="cuda")
    ref = reference(p)
    wide = torch.randn(p.q.shape[0], 13, 128, device="cuda").to(p.q.dtype)
    wide[:, 3:11] = p.q
    o, lse = lca.attn_paged(wide[:, 3:11], p.kc, p.vc, p.table, p.q_start, p.k_len, CAUSAL)
    check(o, lse, p, ref)
    q = p.q[:5].contiguous()
    o, lse = lca.attn_paged(q, p.kc, p.vc, p.table[:0], p.q_start[:1], p.k_len[:0], CAUSAL)
    assert float(o.abs().max()) == 0 and bool(torch.isneginf(lse).all())
    o, lse = lca.attn_paged(q[:0], p.kc, p.vc, p.table, p.q_start * 0, p.k_len, CAUSAL)
    assert o.shape == (0, 8, 128) and lse.shape == (8, 0)
    o, lse = lca.attn_paged(q, p.kc[:0], p.vc[:0], p.table[:, :0], p.q_start * 0, p.k_len * 0, CAUSAL)
    assert float(o.abs().max()) == 0 and bool(torch.isneginf(lse).all())


def test_results_repeat_bit_for_bit(lca):
    import torch

    p = make([(3000, 1), (100, 1), (2000, 40), (0, 300)], 16, 16, 2, CAUSAL, seed=12, device="cuda")
    a = attend(lca, p)
    for _ in range(5):
        b = attend(lca, p)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_streams_with_a_workspace_each(lca):
    import torch

    ps = [make([(900 + 50 * i, 1), (30, 80)], 16, 8, 2, CAUSAL, seed=20 + i, device="cuda") for i in range(2)]
    refs = [reference(p) for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        outs = [lca.attn_paged(p.q, p.kc, p.vc, p.table, p.q_start, p.k_len, CAUSAL, stream=s)
                for p, s in zip(ps, streams)]
    torch.cuda.synchronize()
    for p, r, (o, lse) in zip(ps, refs, outs):
        check(o, lse, p, r)


# ------------------------------------------------------------------ together
def test_a_captured_step_serves_later_batches(lca):
    """Plan, write and attention captured once; the replays see other lengths,
    pages and values, among them batches with fewer rows than the captured one."""
    import torch

    g = torch.Generator().manual_seed(3)
    n, page, Hq, Hkv, rows, n_pages, width = 4, 16, 8, 2, 40, 64, 12
    dev = dict(device="cuda")
    ctx, new = (torch.zeros(n, dtype=torch.int32, **dev) for _ in range(2))
    taken = torch.zeros(1, dtype=torch.int32, **dev)
    free = torch.randperm(n_pages, generator=g).to(torch.int32).cuda()
    table = torch.full((n, width), -1, dtype=torch.int32, **dev)
    kc, vc = (torch.full((n_pages, page, Hkv, 128), float("nan"), dtype=torch.bfloat16, **dev) for _ in range(2))
    q, k, v = (torch.zeros(rows, h, 128, dtype=torch.bfloat16, **dev) for h in (Hq, Hkv, Hkv))

    def step():
        plan = lca.paged_plan(ctx, new, free, taken, table, page, n_pages, rows)
        lca.paged_write(k, v, kc, vc, plan.slots)
        return plan, lca.attn_paged(q, kc, vc, table, plan.q_start, plan.k_len, CAUSAL)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan, (o, lse) = step()
    have = [0] * n
    hist = [([], []) for _ in range(n)]
    for news in ([5, 0, 17, 1], [1, 1, 1, 1], [0, 30, 1, 9], [1, 1, 1, 1], [0, 0, 0, 0], [16, 3, 1, 20]):
        ctx.copy_(torch.tensor(have, dtype=torch.int32))
        new.copy_(torch.tensor(news, dtype=torch.int32))
        total = sum(news)
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        assert plan.state.tolist()[1:] == [0, 0, total]
        taken.copy_(plan.state[:1])
        at, ks, vs, segs, kat = 0, [], [], [], 0
        for i, w in enumerate(news):
            hist[i][0].append(k[at:at + w].cpu())
            hist[i][1].append(v[at:at + w].cpu())
            have[i] += w
            ks.append(torch.cat(hist[i][0]))
            vs.append(torch.cat(hist[i][1]))
            segs.append(Segment(at, w, kat, have[i]))
            at, kat = at + w, kat + have[i]
        p = make([(0, 1)], 16, Hq, Hkv, CAUSAL)
        p.q, p.k, p.v = q, torch.cat(ks), torch.cat(vs)
        p.prob.Tq, p.prob.Tk, p.prob.segments = rows, kat, segs
        check(o, lse, p, what=str(news))


def test_agrees_with_the_packed_forward_and_merges(lca):
    """A prompt through attn_fwd and through the cache; and a shared prefix in
    one call, the rest in another, merged, against one call over both."""
    import torch

    p = make([(0, 333), (0, 190)], 32, 16, 4, CAUSAL, seed=14, device="cuda")
    o, lse, _ = attend(lca, p)
    check(o, lse, p)
    o2, lse2 = lca.attn_fwd(p.q, p.k.cuda(), p.v.cuda(), p.prob.segments, CAUSAL)
    ref = reference(p)
    check(o2, lse2, p, ref)
    # tokens 96.. of request 0 over its first 96 keys (FULL) and over the rest (CAUSAL)
    q, T = p.q[96:333], 333 - 96
    qs = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    kl = lambda n: torch.tensor([n], dtype=torch.int32, device="cuda")  # noqa: E731
    a = lca.attn_paged(q, p.kc, p.vc, p.table[:1], qs, kl(96), MaskSpec("FULL"))
    b = lca.attn_paged(q, p.kc, p.vc, p.table[:1, 3:], qs, kl(T), CAUSAL)
    o3, lse3 = lca.attn_merge([a[0], b[0]], [a[1], b[1]])
    # each part is rounded to bf16 once more before the merge: twice the one call's bound
    assert bool(((o3.double().cpu() - torch.from_numpy(ref[0][96:333])).abs() <= 2 * torch.from_numpy(ref[2][96:333]) + 2.0 ** -8 * torch.from_numpy(ref[0][96:333]).abs() + 2.0 ** -7).all())
    assert bool(((lse3.double().cpu() - torch.from_numpy(ref[1][:, 96:333])).abs() <= 1e-4).all())


FITS_NOT = {
    # (cached, new) per request, rows of the packed batch, entries of a table row
    "rows": ([(30, 3), (100, 40), (5, 7), (64, 1)], 20, 12),
    "table": ([(60, 8), (10, 20), (64, 5), (3, 70), (63, 2), (0, 64), (50, 1)], 175, 4),
    "both": ([(0, 70), (62, 3), (1, 2), (40, 300)], 200, 4),
    "long": ([(1500, 700), (2000, 90), (2047, 1), (2048, 1), (1990, 300)], 900, 128),
}


@pytest.mark.parametrize("mask", MASKS, ids=lambda m: f"{m.kind}{m.window_left or ''}")
@pytest.mark.parametrize("case", FITS_NOT)
def test_a_batch_that_does_not_fit_keeps_its_positions(lca, case, mask):
    """Plan, write and attention of requests that the packed rows or the
    tables have no room for: the rows with a slot are attended at the plan's
    positions, to keys that were written (all else in the cache is NaN); the
    others get 0 and -inf."""
    import torch

    lens, rows, width = FITS_NOT[case]
    page, Hq, Hkv, n = 16, 8, 2, len(lens)
    room, g = width * page, torch.Generator().manual_seed(len(case))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    n_pages = sum(-(-c // page) for c, _ in lens) + sum(-(-w // page) + 1 for _, w in lens)
    perm = torch.randperm(n_pages, generator=g).to(torch.int32)
    table, at = torch.full((n, width), -1, dtype=torch.int32), 0
    kc, vc = (torch.full((n_pages, page, Hkv, 128), float("nan"), dtype=torch.bfloat16) for _ in range(2))
    old = [[torch.randn(c, Hkv, 128, generator=g).to(torch.bfloat16) for _ in range(2)] for c, _ in lens]
    for i, (c, _) in enumerate(lens):
        m, j = -(-c // page), torch.arange(c)
        table[i, :m] = perm[at:at + m]
        at += m
        for cache, x in zip((kc, vc), old[i]):
            cache[table[i].long()[j // page], j % page] = x
    q, k, v = (torch.randn(rows, h, 128, generator=g).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    kc, vc, table, qd = kc.cuda(), vc.cuda(), table.cuda(), q.cuda()
    ctx = i32([c for c, _ in lens])
    plan = lca.paged_plan(ctx, i32([w for _, w in lens]), perm[at:].cuda(), i32([0]), table, page, n_pages, rows)
    lca.paged_write(k.cuda(), v.cuda(), kc, vc, plan.slots)
    assert int(plan.state[1]) == 0 and int(plan.state[2]) > 0
    segs, ks, vs, kat, row, behind = [], [], [], 0, 0, False
    for i, (c, w) in enumerate(lens):
        have = min(row + w, rows) - min(row, rows)  # its rows in the batch
        served = min(have, room - c)
        behind |= served < have
        segs.append(Segment(min(row, rows), served, kat, c + served))
        ks += [old[i][0], k[row:row + served]]
        vs += [old[i][1], v[row:row + served]]
        assert plan.positions[row:row + served].tolist() == list(range(c, c + served))
        assert (plan.slots[row:row + have] >= 0).tolist() == [t < served for t in range(have)]
        kat, row = kat + c + served, row + w
    p = make([(0, 1)], 16, Hq, Hkv, mask)
    p.q, p.kc, p.vc, p.table, p.q_start, p.k_len = qd, kc, vc, table, plan.q_start, plan.k_len
    p.k, p.v = torch.cat(ks), torch.cat(vs)
    p.prob.Tq, p.prob.Tk, p.prob.segments = rows, kat, segs
    ref = reference(p)
    for hint in (0, 700):
        o, lse, st = attend(lca, p, ctx_len=ctx, max_q_len=hint)
        assert st[0] == (6 if behind else 0)
        check(o, lse, p, ref, what=f"{case}, max_q_len={hint}")


@pytest.mark.parametrize("lens", [DECODE, CHUNKS, [(3000, 1), (100, 1), (2000, 40), (0, 300)]], ids=["decode", "chunks", "mixed"])
def test_cached_lengths_change_nothing_in_a_batch_that_fits(lca, lens):
    import torch

    p = make(lens, 16, 8, 2, CAUSAL, pad=3, seed=4, device="cuda")
    ctx = torch.tensor([c for c, _ in lens], dtype=torch.int32, device="cuda")
    a, b = attend(lca, p), attend(lca, p, ctx_len=ctx)
    assert a[2] == b[2] == (0, 0) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    o, lse = lca.attn_paged(p.q, p.kc, p.vc, p.table, p.q_start, p.k_len, CAUSAL, ctx_len=ctx, stream=s)
    s.synchronize()
    assert torch.equal(a[0], o) and torch.equal(a[1], lse)
    for i, x in ((0, -3), (1, p.table.shape[1] * 16 + 1), (2, 2**31 - 1), (0, -2**31)):
        bad = ctx.clone()
        bad[i] = x
        assert attend(lca, p, ctx_len=bad)[2] == (6, 52)
    for bad in (ctx.long(), ctx[1:], ctx.cpu(), torch.stack([ctx, ctx], 1)[:, 0]):
        with pytest.raises(ValueError, match="ctx_len"):
            lca.attn_paged(p.q, p.kc, p.vc, p.table, p.q_start, p.k_len, CAUSAL, ctx_len=bad)
    out = torch.empty(p.q.shape, dtype=p.q.dtype, device="cuda")
    inside = out.view(-1).view(torch.int32)[:len(lens)]
    with pytest.raises(lca.LcaError, match="INVALID"):
        lca.attn_paged(p.q, p.kc, p.vc, p.table, p.q_start, p.k_len, CAUSAL, ctx_len=inside, out=out)


@pytest.mark.parametrize("split", [32, 96, 320])
def test_merged_parts_are_off_by_their_roundings(lca, split):
    """A prefix of the keys in one call (FULL), the rest in another (CAUSAL),
    merged.  With w_p = exp(L_p - L) the merged row is sum_p w_p O_p, so it is
    off by no more than
      sum_p w_p (bound of O_p + |O_p| d_p)   d_p: how far log w_p may be off
      + u |O|                                its own rounding
    where L is off by the largest bound of the L_p, and d_p by that and L_p's
    own, each and every exp, log, product and sum in fp32 adding no more than
    16 e (1 + |L|); (1 + 2^-6) covers products of two such errors."""
    import torch

    p = make([(0, 333)], 32, 16, 4, CAUSAL, seed=14, device="cuda")
    q, T = p.q[split:], 333 - split
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    args = p.kc, p.vc
    a = lca.attn_paged(q, *args, p.table, i32(0, T), i32(split), MaskSpec("FULL"))
    b = lca.attn_paged(q, *args, p.table[:, split // 32:], i32(0, T), i32(T), CAUSAL)
    o, lse = lca.attn_merge([a[0], b[0]], [a[1], b[1]])
    ref = reference(p)
    O, L = ref[0][split:], ref[1][:, split:]
    p.q, p.prob.Tq = q, T
    refs = []
    for mask, seg, part in ((MaskSpec("FULL"), Segment(0, T, 0, split), a), (CAUSAL, Segment(0, T, split, T), b)):
        p.prob.mask, p.prob.segments = mask, [seg]
        refs.append(reference(p))
        check(*part, p, refs[-1])
    e, u = 2.0 ** -24, 2.0 ** -8
    few = 16 * e * (1 + np.abs(L))
    off_l = np.maximum(refs[0][3], refs[1][3]) + few
    tol = u * np.abs(O)
    for Op, Lp, to, tl in refs:
        w, d = np.exp(Lp - L).T[:, :, None], (tl + off_l + few).T[:, :, None]
        tol = tol + w * (to + np.abs(Op) * d)
    check(o, lse, p, (O, L, tol * (1 + 2.0 ** -6), off_l))


def test_a_captured_step_serves_batches_that_do_not_fit(lca):
    """One graph of plan, write and attention with the cached lengths; its
    replays see batches that fit, that outgrow the packed rows and that outgrow
    the tables, and give the bits of eager calls."""
    import torch

    g = torch.Generator().manual_seed(9)
    n, page, Hq, Hkv, rows, width = 5, 16, 8, 2, 300, 6
    n_pages = n * width + 40
    ctx, new = (torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(2))
    taken = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.arange(n * width, dtype=torch.int32, device="cuda").view(n, width)
    free = torch.arange(n * width, n_pages, dtype=torch.int32, device="cuda")
    kc, vc = (torch.randn(n_pages, page, Hkv, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q, k, v = (torch.randn(rows, h, 128, generator=g).to(torch.bfloat16).cuda() for h in (Hq, Hkv, Hkv))
    first = [t.clone() for t in (table, kc, vc)]

    def step():
        for t, x in zip((table, kc, vc), first):
            t.copy_(x)
        plan = lca.paged_plan(ctx, new, free, taken, table, page, n_pages, rows)
        lca.paged_write(k, v, kc, vc, plan.slots)
        return *lca.attn_paged(q, kc, vc, table, plan.q_start, plan.k_len, CAUSAL, ctx_len=ctx), plan.state

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for ctxs, news in (([10, 0, 30, 5, 90], [3, 60, 1, 0, 6]), ([0, 0, 50, 9, 3], [90, 90, 40, 80, 9]),
                       ([90, 96, 40, 95, 0], [7, 2, 70, 1, 96]), ([60] * 5, [80] * 5)):
        ctx.copy_(torch.tensor(ctxs, dtype=torch.int32))
        new.copy_(torch.tensor(news, dtype=torch.int32))
        for t in outs:
            t.fill_(7)
        graph.replay()
        got = [t.clone() for t in outs]
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and bool(want[0].isfinite().all())
        row = 0
        for c, w in zip(ctxs, news):  # a request's rows behind the table's end, and no others, are empty
            have = min(row + w, rows) - min(row, rows)
            empty = want[1][0, row:row + have].isneginf().tolist()
            assert empty == [c + t >= width * page for t in range(have)]
            row += w
