"""The 8-bit paged cache on the GPU: writes and reads exactly, attention
against the fp64 oracle over the values that the cache stands for, within bounds
derived from the roundings (tests/paged8_util.py), and all of a step together."""
from __future__ import annotations

import numpy as np
import pytest

from gen import MaskSpec, Segment
from tests.paged8_util import check8, lay_out8, make8, quantise, reference8, to_bits
from tests.paged_util import MASKS

pytestmark = pytest.mark.gpu
CAUSAL = MaskSpec("CAUSAL")
TYPES = ["bf16", "fp16"]


def torch_type(name):
    import torch

    return {"bf16": torch.bfloat16, "fp16": torch.float16}[name]


def random_cache(n_pages, page, Hkv, layout, g):
    """Any bytes at all, on the CPU and laid out on the device."""
    import torch

    parts = [torch.randint(0, 256, (n_pages, page, Hkv, 128), generator=g).to(torch.uint8) for _ in range(2)]
    parts += [torch.randint(0, 256, (n_pages, Hkv, page), generator=g).to(torch.uint8) for _ in range(2)]
    return parts, lay_out8(*parts, layout, "cuda")


# ------------------------------------------------------------------ write
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("layout", ["nhd", "hnd", "kv"])
@pytest.mark.parametrize("T,Hkv,page", [(1, 1, 8), (64, 8, 16), (133, 3, 24), (2000, 2, 256), (0, 2, 8)])
def test_write(lca, T, Hkv, page, layout, dtype):
    """Values and factors bit for bit, rows of many sizes; skipped rows and all else in the cache as it was."""
    import torch

    g = torch.Generator().manual_seed(T + Hkv)
    n_pages = T // page + 3
    parts, dev = random_cache(n_pages, page, Hkv, layout, g)
    slots = torch.randperm(n_pages * page, generator=g)[:T].to(torch.int32)
    slots[::5] = -1
    slots[1::7] = n_pages * page + 3
    x = torch.randn(T, 3 * Hkv, 128, generator=g) * torch.randint(-9, 9, (T, 3 * Hkv, 1), generator=g).float().exp2()
    x = x.to(torch_type(dtype))
    qkv = x.cuda()
    lca.paged_write_fp8(qkv[:, Hkv:2 * Hkv], qkv[:, 2 * Hkv:], *dev, slots.cuda())
    ok = ((slots >= 0) & (slots < n_pages * page)).nonzero().flatten()
    at = slots[ok].long()
    for rows, c, s in ((x[:, Hkv:2 * Hkv], parts[0], parts[2]), (x[:, 2 * Hkv:], parts[1], parts[3])):
        y, e = quantise(rows[ok].double().numpy())
        c[at // page, at % page] = to_bits(y).view(torch.uint8)
        s[at // page, :, at % page] = torch.from_numpy(e + 127).to(torch.uint8)
    for got, want in zip(dev, parts):
        assert torch.equal(got.view(torch.uint8).cpu(), want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hkv", [5, 8])
@pytest.mark.parametrize("T,extra,first", [(16001, 0, 0), (16001, 8, 8), (37, 8, 0), (37, 16, 8)])
def test_write_of_many_rows_and_of_rows_off_32_bytes(lca, T, extra, first, Hkv, dtype):
    """So many rows that threads take two heads each; rows that start on 16 bytes only; an infinity among them."""
    import torch

    g = torch.Generator().manual_seed(T + extra + Hkv)
    page, W = 16, Hkv * 128
    n_pages = T // page + 2
    x = torch.randn(T, 2 * W + extra + first, generator=g) * torch.randint(-9, 9, (T, 1), generator=g).float().exp2()
    x[T // 2, first + 130] = float("inf")
    x = x.to(torch_type(dtype))
    slots = torch.randperm(n_pages * page, generator=g)[:T].to(torch.int32)
    slots[3::11] = -1
    parts, dev = random_cache(n_pages, page, Hkv, "hnd", g)
    d = x.cuda()
    k, v = (t.unflatten(1, (Hkv, 128)) for t in (d[:, first:first + W], d[:, first + W:first + 2 * W]))
    lca.paged_write_fp8(k, v, *dev, slots.cuda())
    ok = (slots >= 0).nonzero().flatten()
    at = slots[ok].long()
    for rows, c, s in ((k.cpu(), parts[0], parts[2]), (v.cpu(), parts[1], parts[3])):
        y, e = quantise(rows[ok].double().numpy())
        c[at // page, at % page] = to_bits(y).view(torch.uint8)
        s[at // page, :, at % page] = torch.from_numpy(e + 127).to(torch.uint8)
    for got, want in zip(dev, parts):
        got, want = got.view(torch.uint8).cpu(), want
        nan = (want & 0x7F == 0x7F) & (got & 0x7F == 0x7F) if got.dim() == 4 else torch.zeros_like(want, dtype=torch.bool)
        assert bool(((got == want) | nan).all())  # a NaN's sign is free


@pytest.mark.parametrize("dtype", TYPES)
def test_write_of_edges(lca, dtype):
    """Rows of zeros, of one value, of the type's largest and smallest, of values that lie between two e4m3 ones, and
    rows with infinities and NaN, which are NaN and do not raise the factor."""
    import torch

    dt = torch_type(dtype)
    big = torch.finfo(dt).max
    rows = [[0.0], [-0.0, 0.0], [448.0, 1.0], [449.0, 1.0], [450.0, -3.0], [big, 1.0], [-big, big / 2], [torch.finfo(dt).tiny, 0.0],
            [1e-7, -3e-8], [float("inf"), 2.0, -1.0], [float("-inf"), float("nan"), 0.3], [float("nan")], [240.0, 17.0, 18.0, 19.0, -17.0],
            [448.0, 2.0 ** -6, 2.0 ** -7, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11, -5 * 2.0 ** -10],
            [1.75, 1.0625, 1.1875], [1.76, 1.0625], [2.0 ** -14] * 128, [65504.0], [1e-30], [2.0 ** 60, -1.0], [3e38]]
    x = torch.zeros(len(rows), 1, 128, dtype=dt)
    for i, r in enumerate(rows):
        x[i, 0, :len(r)] = torch.tensor(r).to(dt)
    n = len(rows)
    kc = torch.zeros(4, 8, 1, 128, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    vc, ks, vs = torch.zeros_like(kc), torch.zeros(4, 1, 8, dtype=torch.uint8, device="cuda"), torch.zeros(4, 1, 8, dtype=torch.uint8, device="cuda")
    d = x.cuda()
    lca.paged_write_fp8(d, d.flip(0).contiguous(), kc, vc, ks, vs, torch.arange(n, dtype=torch.int32, device="cuda"))
    y, e = quantise(x.double().numpy())
    for c, s, flip in ((kc, ks, False), (vc, vs, True)):
        got = c.float().cpu().view(32, 1, 128)[:n].double().numpy()
        exps = s.cpu().view(32)[:n].numpy().astype(int) - 127
        want, we = (y[::-1], e[::-1]) if flip else (y, e)
        assert np.array_equal(exps, we[:, 0])
        assert np.array_equal(got, want, equal_nan=True)
    b, want = kc.view(torch.uint8).cpu().view(32, 128)[:n], to_bits(y).view(torch.uint8)[:, 0]
    same = b == want
    assert bool((same | torch.from_numpy(np.isnan(y[:, 0]))).all())  # zeros keep their signs


def test_write_from_the_cache_itself_is_refused(lca):
    import torch

    kc, vc = (torch.zeros(4, 8, 2, 128, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.zeros(1024, dtype=torch.uint8, device="cuda")[:64].view(4, 2, 8) for _ in range(2))
    k = torch.zeros(6, 2, 128, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(6, dtype=torch.int32, device="cuda")
    rows = kc.view(torch.bfloat16).view(16, 2, 128)
    scale_rows = vs.view(-1).view(torch.int32)[4:10]
    for a, b, s in ((rows[8:14], k, slots), (k, rows[10:], slots), (k, k, vc.view(torch.uint8).view(-1)[:24].view(torch.int32)), (k, k, scale_rows)):
        with pytest.raises(lca.LcaError, match="INVALID"):
            lca.paged_write_fp8(a, b, kc, vc, ks, vs, s)
    assert not bool(kc.view(torch.uint8).any())
    for bad in (dict(k=k.float()), dict(v=k.half()), dict(v=k[:5]), dict(slots=slots.long()), dict(k_cache=kc.view(torch.uint8)),
                dict(k_scale=ks.float()), dict(v_scale=vs.transpose(1, 2)), dict(k_cache=kc[:3]), dict(k_cache=kc.transpose(2, 3))):
        args = dict(dict(k=k, v=k, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, slots=slots), **bad)
        with pytest.raises((ValueError, TypeError)):
            lca.paged_write_fp8(**args)


# ------------------------------------------------------------------ read
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("layout", ["nhd", "hnd", "kv"])
@pytest.mark.parametrize("n,Hkv,page", [(1, 1, 8), (5, 8, 16), (40, 3, 24), (7, 2, 256), (0, 2, 8)])
def test_read(lca, n, Hkv, page, layout, dtype):
    """Any bytes: every value bit for bit (bytes of factors past the range count as its ends, fp16 ends at 65504); pages
    in any order and more than once; entries that are none leave what was there."""
    import torch

    g = torch.Generator().manual_seed(n + page)
    (lk, lv, lks, lvs), dev = random_cache(n + 2, page, Hkv, layout, g)
    pages = torch.randint(0, n + 2, (n,), generator=g).to(torch.int32)
    pages[::4] = torch.tensor([-1, n + 2, 2**31 - 1, -2**31] * n, dtype=torch.int32)[:len(pages[::4])]
    dt = torch_type(dtype)
    outs = [torch.full((n, page, Hkv, 128), 7.0, dtype=dt, device="cuda") for _ in range(2)]
    if layout == "hnd":
        outs = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in outs]
    got = lca.paged_read_fp8(*dev, pages.cuda(), k_out=outs[0], v_out=outs[1])
    assert got[0] is outs[0]
    made = lca.paged_read_fp8(*dev, pages.cuda(), dtype=dt)
    ok = (pages >= 0) & (pages < n + 2)
    for c, s, x, y in ((lk, lks, got[0], made[0]), (lv, lvs, got[1], made[1])):
        at = pages[ok].long()
        e = s[at].transpose(1, 2).double().clamp(79, 175) - 127
        want = c[at].view(torch.float8_e4m3fn).double() * 2.0 ** e[..., None]
        want = want.clamp(-65504, 65504) if dtype == "fp16" else want  # NaN stays
        want = want.to(dt)
        for z, rest in ((x, 7.0), (y, 0.0)):
            assert torch.equal(torch.nan_to_num(z.cpu()[ok].double(), nan=3e300), torch.nan_to_num(want.double(), nan=3e300))
            assert bool((z.cpu()[~ok] == rest).all())


@pytest.mark.parametrize("first", [0, 8])
@pytest.mark.parametrize("layout,dtype", [("nhd", "bf16"), ("hnd", "fp16")])
def test_read_of_many_pages(lca, layout, dtype, first):
    """So many rows that threads take four each, pages of a number of rows that 128 does not divide; results that
    start on 16 bytes only; nothing written beside them."""
    import torch

    n, page, Hkv = 90, 200, 9
    g = torch.Generator().manual_seed(first + 1)
    (lk, lv, lks, lvs), dev = random_cache(50, page, Hkv, layout, g)
    pages = torch.randint(-1, 51, (n,), generator=g).to(torch.int32)
    dt, size = torch_type(dtype), n * page * Hkv * 128
    flat = [torch.full((size + 16,), 7.0, dtype=dt, device="cuda") for _ in range(2)]
    outs = [x[first:first + size].view(n, page, Hkv, 128) for x in flat]
    lca.paged_read_fp8(*dev, pages.cuda(), k_out=outs[0], v_out=outs[1])
    ok = (pages >= 0) & (pages < 50)
    for c, s, x, f in ((lk, lks, outs[0], flat[0]), (lv, lvs, outs[1], flat[1])):
        e = s.transpose(1, 2).float().clamp(79, 175) - 127
        want = c.view(torch.float8_e4m3fn).float() * e.exp2()[..., None]
        want = (want.clamp(-65504, 65504) if dtype == "fp16" else want).to(dt)[pages[ok].long()]
        assert torch.equal(torch.nan_to_num(x.cpu()[ok].float(), nan=3e30), torch.nan_to_num(want.float(), nan=3e30))
        assert bool((x.cpu()[~ok] == 7).all()) and bool((f[:first] == 7).all()) and bool((f[first + size:] == 7).all())


def test_reads_that_overlap_or_do_not_fit_are_refused(lca):
    import torch

    g = torch.Generator().manual_seed(1)
    _, (kc, vc, ks, vs) = random_cache(16, 8, 2, "nhd", g)
    pages = torch.arange(4, dtype=torch.int32, device="cuda")
    o = lambda n=4: torch.zeros(n, 8, 2, 128, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    inside = kc.view(torch.bfloat16).view(-1)[:8192].view(4, 8, 2, 128)
    out = o()
    for kw in (dict(k_out=inside, v_out=o()), dict(k_out=o(), v_out=inside), dict(k_out=out, v_out=o(), pages=out.view(-1).view(torch.int32)[:4])):
        with pytest.raises(lca.LcaError, match="INVALID"):
            lca.paged_read_fp8(kc, vc, ks, vs, kw.pop("pages", pages), **kw)
    for kw in (dict(k_out=o()), dict(k_out=o(5), v_out=o(5)), dict(k_out=o(), v_out=o(), dtype=torch.float16), dict(dtype=torch.float32),
               dict(k_out=o().float(), v_out=o().float()), dict(k_out=o().cpu(), v_out=o().cpu())):
        with pytest.raises((ValueError, TypeError)):
            lca.paged_read_fp8(kc, vc, ks, vs, pages, **kw)
    for bad in (pages.long(), pages.cpu(), [0, 1]):
        with pytest.raises((ValueError, TypeError), match="pages"):
            lca.paged_read_fp8(kc, vc, ks, vs, bad)


# ------------------------------------------------------------------ attention
def attend(lca, p, **kw):
    import torch

    need = lca.attn_paged_fp8_workspace_size(p.q, p.kc, p.vc, p.ks, p.vs, p.table, p.prob.mask)
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")  # nothing may depend on what it held
    o = torch.full(p.q.shape, 7.0, dtype=p.q.dtype, device="cuda")
    lse = torch.full((p.prob.Hq, p.prob.Tq), 7.0, device="cuda")
    lca.attn_paged_fp8(p.q, p.kc, p.vc, p.ks, p.vs, p.table, p.q_start, p.k_len, p.prob.mask, p.prob.scale, out=o, lse=lse,
                       workspace=ws, **kw)
    torch.cuda.synchronize()
    return o, lse, lca.read_status(ws)


DECODE = [(0, 1), (7, 1), (126, 1), (127, 1), (128, 1), (1000, 1), (31, 1)]
CHUNKS = [(0, 1), (0, 130), (300, 257), (0, 0), (64, 64), (5, 0), (1, 2), (511, 17)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (16, 2), (3, 3), (12, 4), (10, 2), (32, 1), (24, 1), (40, 1)])
def test_decode(lca, Hq, Hkv, dtype):
    p = make8(DECODE, 16, Hq, Hkv, CAUSAL, dtype, pad=2, seed=Hq, device="cuda")
    ref = reference8(p)
    for hint in (0, 1, 300):
        o, lse, st = attend(lca, p, max_q_len=hint)
        check8(o, lse, p, ref, what=f"max_q_len={hint}")
        assert st == (0, 0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (2, 2), (6, 2), (5, 1), (16, 1), (48, 1), (14, 2)])
def test_chunks(lca, Hq, Hkv, dtype):
    p = make8(CHUNKS, 32, Hq, Hkv, CAUSAL, dtype, pad=3, seed=Hq, device="cuda")
    ref = reference8(p)
    for hint in (0, 257):
        o, lse, st = attend(lca, p, max_q_len=hint)
        check8(o, lse, p, ref, what=f"max_q_len={hint}")
        assert st == (0, 0)


@pytest.mark.parametrize("layout", ["nhd", "hnd", "kv"])
@pytest.mark.parametrize("page", [8, 16, 24, 40, 48, 64, 128, 136, 256, 1024])
def test_pages_and_layouts(lca, page, layout):
    """Pages that end inside a tile, at it and past it; NaN wherever no request's token lies."""
    p = make8([(0, 1), (250, 3), (129, 140), (page, 1), (2 * page - 1, 2)], page, 8, 2, CAUSAL, "fp16", layout, seed=page,
              device="cuda")
    o, lse, st = attend(lca, p)
    check8(o, lse, p)
    assert st == (0, 0)


@pytest.mark.parametrize("mask", MASKS, ids=lambda m: f"{m.kind}{m.window_left or ''}")
@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (3, 1)])
def test_masks(lca, mask, Hq, Hkv):
    p = make8([(0, 1), (600, 1), (99, 1), (0, 200), (333, 100), (150, 5)], 16, Hq, Hkv, mask, seed=3, device="cuda")
    o, lse, st = attend(lca, p)
    check8(o, lse, p, what=mask.kind)
    assert st == (0, 0)


@pytest.mark.parametrize("mask", [CAUSAL, MASKS[4], MASKS[7], MASKS[8]], ids=lambda m: m.kind)
def test_rows_that_attend_nothing(lca, mask):
    import torch

    p = make8([(0, 40), (0, 9), (0, 300)], 16, 8, 2, mask, seed=9, device="cuda")
    p.k_len = torch.tensor([11, 0, 7], dtype=torch.int32, device="cuda")
    for s, n in zip(p.prob.segments, (11, 0, 7)):
        s.k_len = n
    ref = reference8(p)
    assert np.isneginf(ref[1]).any()
    o, lse, st = attend(lca, p)
    check8(o, lse, p, ref)
    assert st == (0, 0)


@pytest.mark.parametrize("mask", [CAUSAL, MaskSpec("CAUSAL_SLIDING", window_left=100), MaskSpec("FULL"),
                                  MaskSpec("GLOBAL_SLIDING", window_left=300, window_right=0, num_global=10)],
                         ids=lambda m: m.kind)
@pytest.mark.parametrize("new", [1, 2, 20, 200])
def test_long_contexts_split_over_keys(lca, mask, new):
    p = make8([(6000, new)], 64, 8, 1, mask, seed=new, device="cuda")
    check8(*attend(lca, p)[:2], p)
    p = make8([(3000, new), (1, 1), (0, 1), (2500, 1), (17, new)], 64, 4, 2, mask, "fp16", seed=new, device="cuda")
    check8(*attend(lca, p)[:2], p)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new", [1, 3, 40])
def test_factors_of_every_size(lca, new, dtype):
    """Rows of values between 2^-48 and 2^48 times the others, zeros among them, in every order of sizes: what a key
    weighs does not depend on its values, and every row is right on the scale of its own sum.  (Their sums span 96
    binades; fp16's o is kept in range by the smaller half.)"""
    import torch

    lens = [(700, new), (90, new)]
    p = make8(lens, 16, 8, 2, CAUSAL, dtype, seed=new, device="cuda")
    g = torch.Generator().manual_seed(new)
    lo, hi = (-48, 48) if dtype == "bf16" else (-48, 6)
    at = 0
    for i, (c, w) in enumerate(lens):
        m = c + w
        e = torch.randint(lo, hi + 1, (m, 2), generator=g)
        if i == 1:
            e = e.sort(0)[0]
        j = torch.arange(m)
        pages = p.table[i].cpu().long()[j // 16]
        old = (p.vs.cpu()[pages, :, j % 16].to(torch.int64) - 127)
        p.v[at:at + m] *= 2.0 ** (e - old).double()[..., None].float()
        vs = p.vs.cpu()
        vs[pages, :, j % 16] = (e + 127).to(torch.uint8)
        p.vs = vs.cuda()
        at += m
    o, lse, st = attend(lca, p)
    assert st == (0, 0)
    check8(o, lse, p)


def test_keys_of_every_size(lca):
    """Keys' factors over their whole range: scores of 2^44 among others, one key takes all."""
    import torch

    p = make8([(300, 1), (50, 30)], 16, 8, 2, CAUSAL, seed=3, device="cuda")
    g = torch.Generator().manual_seed(5)
    for hi in (-20, 20):
        at = 0
        ks = p.ks.cpu()
        for i, m in enumerate(p.k_len.tolist()):
            j = torch.arange(m)
            pages = p.table[i].cpu().long()[j // 16]
            e = torch.randint(-48, hi, (m, 2), generator=g)
            old = ks[pages, :, j % 16].to(torch.int64) - 127
            p.k[at:at + m] *= 2.0 ** (e - old).double()[..., None].float()
            ks[pages, :, j % 16] = (e + 127).to(torch.uint8)
            at += m
        p.ks = ks.cuda()
        o, lse, st = attend(lca, p)
        assert st == (0, 0) and bool(o.isfinite().all())
        if hi < 0:  # beyond, a score's rounding is more than 1 and the bound says nothing
            check8(o, lse, p)


@pytest.mark.parametrize("size", [1e-30, 1e-5, 1e4, 1e30])
def test_queries_of_every_size(lca, size):
    """Queries of any size bf16 has, beside ones of another: each row keeps its own scale."""
    import torch

    p = make8([(200, 2), (40, 20)], 16, 8, 2, CAUSAL, seed=3, device="cuda")
    p.q[::2] = (p.q[::2].double() * size).to(p.q.dtype)
    if size > 1:
        p.prob.scale = 1.0 / size
    o, lse, st = attend(lca, p)
    assert st == (0, 0)
    check8(o, lse, p)


@pytest.mark.parametrize("byte", [0x7F, 0xFF, 0x7E, 0x00])
@pytest.mark.parametrize("new", [1, 3, 150])
def test_hidden_keys_reach_nothing(lca, byte, new):
    """Keys in the pages before a sliding window, and all slots no request owns, hold NaN or the largest value and any
    factor; the results are those of a cache that holds zeros there, bit for bit."""
    import torch

    mask = MaskSpec("CAUSAL_SLIDING", window_left=77)
    outs = []
    for fill, factor in ((byte, 0xFF if byte else 0), (0, 127)):
        p = make8([(400, new), (9, new), (128, new)], 16, 8, 2, mask, "fp16", fill=fill, fill_scale=factor, seed=5, device="cuda")
        for j in range(400 - 77):  # no new token of request 0 sees a key before this
            page, at = int(p.table[0, j // 16]), j % 16
            p.kc.view(torch.uint8)[page, at] = fill
            p.vc.view(torch.uint8)[page, at] = fill
            p.ks[page, :, at] = factor
            p.vs[page, :, at] = factor
        outs.append(attend(lca, p))
    (o, lse, st), (o0, lse0, _) = outs
    assert st == (0, 0)
    assert torch.equal(o, o0) and torch.equal(lse, lse0)
    check8(o, lse, p)


@pytest.mark.parametrize("mask", MASKS, ids=lambda m: f"{m.kind}{m.window_left or ''}")
@pytest.mark.parametrize("Hq", [8, 3])
def test_nan_reaches_the_rows_that_attend_it(lca, mask, Hq):
    """Under every family: a column of the values of a few keys is NaN; it is NaN in the rows that attend one of them,
    all else as without."""
    import torch

    from oracle.masks import segment_mask

    lens = [(600, 1), (0, 200), (333, 100), (150, 5), (1000, 300), (70, 2)]
    p = make8(lens, 16, Hq, 1, mask, seed=Hq, device="cuda")
    ref = reference8(p)
    o0, lse0, _ = attend(lca, p)
    check8(o0, lse0, p, ref, what=mask.kind)
    hit = torch.zeros(p.q.shape[0], dtype=torch.bool)
    for i, seg in enumerate(p.prob.segments):
        bads = [2, 64, 65, 127, seg.k_len // 2, seg.k_len - 1, seg.k_len - 3, seg.k_len - 60]
        bads = [b for b in bads if 0 <= b < seg.k_len]
        for b in bads:
            p.vc.view(torch.uint8)[int(p.table[i, b // 16]), b % 16, :, 77] = 0xFF if b % 2 else 0x7F
        hit[seg.q_off:seg.q_off + seg.q_len] = torch.from_numpy(segment_mask(mask, i, seg)[:, bads].any(1))
    for _ in range(2):
        o, lse, st = attend(lca, p)
        assert st == (0, 0) and torch.equal(lse, lse0)
        assert bool(o[hit.cuda()][:, :, 77].isnan().all()), mask.kind
        o[hit.cuda(), :, 77] = o0[hit.cuda(), :, 77]
        check8(o, lse, p, ref, what=mask.kind)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new", [1, 3, 300])
def test_nan_of_small_weight_is_not_lost(lca, new, dtype):
    """A context in pieces, whose first keys have a vanishing share of the last ones' weight."""
    import torch

    ctx, hit = 16000, 100
    p = make8([(ctx, new), (20, 1)], 64, 8, 1, CAUSAL, dtype, seed=new, device="cuda")
    p.q.fill_(8.0)
    one = torch.tensor([1.0, -1.0]).to(torch.float8_e4m3fn).view(torch.uint8).tolist()
    for j in range(0, ctx + new, 64):
        page = int(p.table[0, j // 64])
        p.kc.view(torch.uint8)[page] = one[j < ctx // 2]
        p.ks[page] = 127
    o0, lse0, _ = attend(lca, p)
    assert bool(o0.isfinite().all())
    p.vc.view(torch.uint8)[int(p.table[0, hit // 64]), hit % 64, 0, 77] = 0x7F
    o, lse, st = attend(lca, p)
    assert st == (0, 0) and torch.equal(lse, lse0)
    assert bool(o[:new, :, 77].isnan().all())
    o[:new, :, 77] = o0[:new, :, 77]
    assert torch.equal(o, o0)


@pytest.mark.parametrize("new", [1, 3, 90])
def test_pages_between_sinks_and_window_may_be_gone(lca, new):
    import torch

    mask = MaskSpec("GLOBAL_SLIDING", window_left=200, window_right=0, num_global=20)
    p = make8([(3000, new), (900, new)], 16, 8, 2, mask, seed=new, device="cuda")
    ref = reference8(p)
    for i, ctx in enumerate((3000, 900)):
        for e in range(2, (ctx - 200) // 16):
            page = int(p.table[i, e])
            for t in (p.kc, p.vc):
                t.view(torch.uint8)[page] = 0x7F
            p.table[i, e] = -1
    o, lse, st = attend(lca, p)
    assert st == (0, 0)
    check8(o, lse, p, ref)


@pytest.mark.parametrize("Hq", [64, 100, 128, 136, 260])
def test_many_heads_of_one_group(lca, Hq):
    p = make8([(200, 1), (0, 5), (130, 3)], 16, Hq, 1, CAUSAL, seed=Hq, device="cuda")
    o, lse, st = attend(lca, p)
    check8(o, lse, p)
    assert st == (0, 0)


def test_many_requests(lca):
    rng = np.random.default_rng(5)
    lens = [(int(rng.integers(0, 260)), int(rng.choice([0, 1, 1, 1, 2, 5, 40]))) for _ in range(1100)]
    p = make8(lens, 8, 4, 1, CAUSAL, "fp16", pad=9, seed=17, device="cuda")
    ref = reference8(p)
    for hint in (0, 40):
        o, lse, st = attend(lca, p, max_q_len=hint)
        check8(o, lse, p, ref)
        assert st == (0, 0)


def test_long_lines_are_claimed(lca):
    """Enough keys that the last part of the work is claimed; the results do not depend on who claims it."""
    import torch

    p = make8([(90000, 1), (70000, 1), (52000, 1), (3, 1)], 128, 16, 16, CAUSAL, seed=18, device="cuda")
    o, lse, st = attend(lca, p)
    assert st == (0, 0)
    check8(o, lse, p)
    for _ in range(4):
        o2, lse2, _ = attend(lca, p)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_pages_far_apart(lca):
    """Pages and factors more than 2^31 bytes apart, written, read back and attended."""
    import torch

    far = (1 << 31) + 64
    buf = torch.zeros(3 * far + (1 << 16), dtype=torch.uint8, device="cuda")
    for new in (1, 60):
        p = make8([(20, new)], 32, 8, 2, CAUSAL, seed=new, device="cuda")
        keep = [int(x) for x in p.table[0] if x >= 0]
        view = lambda at: buf.as_strided((3, 32, 2, 128), (far, 256, 128, 1), at).view(torch.float8_e4m3fn)  # noqa: E731
        views = lambda at: buf.as_strided((3, 2, 32), (far, 32, 1), at)  # noqa: E731
        kc, vc, ks, vs = view(0), view(32 * 256), views(64 * 256), views(64 * 256 + 64)
        table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
        for i, page in enumerate(keep):
            for to, of in ((kc, p.kc), (vc, p.vc)):
                to.view(torch.uint8)[table[0, i]] = of.view(torch.uint8)[page]
            ks[table[0, i]], vs[table[0, i]] = p.ks[page], p.vs[page]
        first = [x.view(torch.uint8).clone() for x in (kc, vc, ks, vs)]
        p.kc, p.vc, p.ks, p.vs, p.table = kc, vc, ks, vs, table
        o, lse, st = attend(lca, p)
        assert st == (0, 0)
        check8(o, lse, p)
        slots = torch.tensor([int(table[0, j // 32]) * 32 + j % 32 for j in range(20, 20 + new)], dtype=torch.int32)
        for s in slots:
            for c, f in ((kc, ks), (vc, vs)):
                c.view(torch.uint8)[int(s) // 32, int(s) % 32] = 1
                f[int(s) // 32, :, int(s) % 32] = 1
        # the new rows again through the write: the same values (a row whose largest was rounded to 224 of its factor gets
        # half of it and twice the e4m3 values), and all else as it was
        lca.paged_write_fp8(p.k[20:].to(torch.bfloat16).cuda(), p.v[20:].to(torch.bfloat16).cuda(), kc, vc, ks, vs, slots.cuda())
        old = torch.ones(3, 32, dtype=torch.bool, device="cuda")
        old.view(-1)[slots.long().cuda()] = False
        for now, was in zip((kc, vc, ks, vs), first):
            now, was = (x.view(torch.uint8) if x.dim() == 4 else x.transpose(1, 2) for x in (now, was))
            assert torch.equal(now[old], was[old])
        a, b = lca.paged_read_fp8(kc, vc, ks, vs, table[0])
        flat = a.view(96, 2, 128)[:20 + new].cpu(), b.view(96, 2, 128)[:20 + new].cpu()
        assert torch.equal(flat[0].float(), p.k) and torch.equal(flat[1].float(), p.v)


@pytest.mark.parametrize("order", [(0, 1, 2), (1, 0, 2), (2, 0, 1), (1, 2, 0), (0, 2, 1), (2, 1, 0)], ids=str)
def test_any_order_of_the_axes(lca, order):
    import torch

    p = make8([(40, 1), (10, 90), (70, 4)], 24, 6, 2, CAUSAL, "fp16", seed=3, device="cuda")
    back = [order.index(i) for i in range(3)] + [3]
    p.kc, p.vc = (x.view(torch.uint8).permute(*order, 3).contiguous().permute(*back).view(torch.float8_e4m3fn) for x in (p.kc, p.vc))
    p.ks, p.vs = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (p.ks, p.vs))
    o, lse, st = attend(lca, p)
    check8(o, lse, p)
    assert st == (0, 0)


def test_narrow_items_among_wide_ones_repeat(lca):
    import torch

    p = make8(CHUNKS * 3, 32, 8, 1, CAUSAL, "fp16", seed=8, device="cuda")
    ref = reference8(p)
    a = attend(lca, p)
    check8(a[0], a[1], p, ref)
    for _ in range(60):
        b = attend(lca, p)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_waits_never_end_in_vain(lca):
    """Many calls with long and short pieces of narrow items, and of wide ones: no wait runs out."""
    import torch

    for lens in ([(int(c), 5) for c in np.linspace(200, 5000, 24)], [(int(c), 70) for c in np.linspace(0, 3000, 12)]):
        p = make8(lens, 32, 16, 2, CAUSAL, seed=21, device="cuda")
        need = lca.attn_paged_fp8_workspace_size(p.q, p.kc, p.vc, p.ks, p.vs, p.table, CAUSAL)
        first = None
        for _ in range(4):
            spaces = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(40)]
            outs = [lca.attn_paged_fp8(p.q, p.kc, p.vc, p.ks, p.vs, p.table, p.q_start, p.k_len, CAUSAL, workspace=w) for w in spaces]
            torch.cuda.synchronize()
            first = first or outs[0]
            for w, (o, lse) in zip(spaces, outs):
                assert lca.read_status(w) == (0, 0)
                assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
        check8(first[0], first[1], p)


def test_overlapping_memory_is_refused(lca):
    import torch

    p = make8([(40, 3)], 16, 8, 8, CAUSAL, seed=2, device="cuda")
    call = lambda **kw: lca.attn_paged_fp8(**{**dict(q=p.q, k_cache=p.kc, v_cache=p.vc, k_scale=p.ks, v_scale=p.vs, block_table=p.table,  # noqa: E731
                                                     q_start=p.q_start, k_len=p.k_len, mask=CAUSAL), **kw})
    o, lse = call()
    flat = torch.empty(4096, dtype=torch.float32, device="cuda")
    need = lca.attn_paged_fp8_workspace_size(p.q, p.kc, p.vc, p.ks, p.vs, p.table, CAUSAL)
    buf = torch.zeros(need + 4096, dtype=torch.uint8, device="cuda")
    n = p.kc.shape[0]
    kc = buf[:p.kc.numel()].view(torch.float8_e4m3fn).view(p.kc.shape)
    ks = buf[1024:1024 + p.ks.numel()].view(p.ks.shape)
    for kw in (dict(out=p.q), dict(out=p.kc.view(torch.bfloat16).view(-1)[:3 * 8 * 128].view(3, 8, 128)),
               dict(out=flat[:1536].view(torch.bfloat16).view(3, 8, 128), lse=flat[1000:1024].view(8, 3)),
               dict(k_cache=kc, workspace=buf[:need]), dict(v_cache=kc, workspace=buf[:need]), dict(k_scale=ks, workspace=buf[:need]),
               dict(v_scale=ks, workspace=buf[:need]), dict(v_scale=flat.view(torch.uint8)[:p.ks.numel()].view(p.ks.shape), lse=flat[8:32].view(8, 3))):
        with pytest.raises(lca.LcaError, match="INVALID"):
            call(**kw)
    assert n > 0 and not bool(buf.any())
    for bad in (dict(q=p.q.float()), dict(q=p.q.cpu()), dict(k_scale=p.ks[:-1]), dict(v_scale=p.vs.float()), dict(k_cache=p.kc.view(torch.uint8)),
                dict(block_table=p.table.long()), dict(k_len=p.k_len[:0]), dict(out=o.half()), dict(q=p.q[:, :, :64])):
        with pytest.raises((ValueError, TypeError)):
            call(**bad)


@pytest.mark.parametrize("dtype", TYPES)
def test_large_scores_and_an_explicit_scale(lca, dtype):
    import torch

    p = make8([(500, 1), (100, 60)], 16, 8, 2, CAUSAL, dtype, seed=8, q_scale=100.0, device="cuda")
    o, lse, _ = attend(lca, p)
    assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(lse).all())
    check8(o, lse, p)
    p = make8([(500, 1), (100, 60)], 16, 8, 2, CAUSAL, dtype, seed=8, device="cuda")
    p.prob.scale = 0.3
    check8(*attend(lca, p)[:2], p)


@pytest.mark.parametrize("lens", [[(300, 1), (20, 1)], [(300, 200), (20, 1)]], ids=str)
def test_bad_pages_and_lengths_are_reported(lca, lens):
    p = make8(lens, 16, 8, 2, CAUSAL, seed=4, device="cuda")
    assert attend(lca, p)[2] == (0, 0)
    for bad in (-1, p.kc.shape[0], 2**31 - 1, -2**31):
        q = make8(lens, 16, 8, 2, CAUSAL, seed=4, device="cuda")
        q.table[0, 3] = bad
        o, lse, st = attend(lca, q)
        assert st[0] == 6
        q.k[48:64] = 0
        q.v[48:64] = 0
        check8(o, lse, q)
    q = make8(lens, 16, 8, 2, MaskSpec("CAUSAL_SLIDING", window_left=30), seed=4, device="cuda")
    q.table[0, 0] = 1 << 20
    q.table[1, -1] = -9
    o, lse, st = attend(lca, q)
    assert st == (0, 0)
    check8(o, lse, q)
    room = p.table.shape[1] * 16
    for name, i, x in (("k_len", 0, -4), ("k_len", 1, room + 1), ("k_len", 0, 2**31 - 1), ("q_start", 2, 2**31 - 1),
                       ("q_start", 1, -3), ("q_start", 0, -2**31), ("q_start", 1, 10**6)):
        q = make8(lens, 16, 8, 2, CAUSAL, fill=0, fill_scale=0, seed=4, device="cuda")
        getattr(q, name)[i] = x
        assert attend(lca, q)[2][0] == 6, (name, i, x)


def test_q_rows_of_a_wider_projection_and_no_requests(lca):
    import torch

    p = make8([(40, 3), (0, 70)], 16, 8, 2, CAUSAL, seed=2, device="cuda")
    ref = reference8(p)
    wide = torch.randn(p.q.shape[0], 13, 128, device="cuda").to(p.q.dtype)
    wide[:, 3:11] = p.q
    call = lambda q, table, qs, kl, cut=None: lca.attn_paged_fp8(q, p.kc[:cut], p.vc[:cut], p.ks[:cut], p.vs[:cut], table, qs, kl, CAUSAL)  # noqa: E731
    o, lse = call(wide[:, 3:11], p.table, p.q_start, p.k_len)
    check8(o, lse, p, ref)
    q = p.q[:5].contiguous()
    o, lse = call(q, p.table[:0], p.q_start[:1], p.k_len[:0])
    assert float(o.abs().max()) == 0 and bool(torch.isneginf(lse).all())
    o, lse = call(q[:0], p.table, p.q_start * 0, p.k_len)
    assert o.shape == (0, 8, 128) and lse.shape == (8, 0)
    o, lse = call(q, p.table[:, :0], p.q_start * 0, p.k_len * 0, 0)
    assert float(o.abs().max()) == 0 and bool(torch.isneginf(lse).all())


def test_results_repeat_bit_for_bit(lca):
    import torch

    p = make8([(3000, 1), (100, 1), (2000, 40), (0, 300)], 16, 16, 2, CAUSAL, seed=12, device="cuda")
    a = attend(lca, p)
    for _ in range(5):
        b = attend(lca, p)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("lens", [DECODE, CHUNKS, [(3000, 1), (100, 1), (2000, 40), (0, 300)]], ids=["decode", "chunks", "mixed"])
def test_cached_lengths_change_nothing_in_a_batch_that_fits(lca, lens):
    import torch

    p = make8(lens, 16, 8, 2, CAUSAL, pad=3, seed=4, device="cuda")
    ctx = torch.tensor([c for c, _ in lens], dtype=torch.int32, device="cuda")
    a, b = attend(lca, p), attend(lca, p, ctx_len=ctx)
    assert a[2] == b[2] == (0, 0) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    bad = ctx.clone()
    bad[0] = -3
    assert attend(lca, p, ctx_len=bad)[2] == (6, 52)


def test_two_streams_with_a_workspace_each(lca):
    import torch

    ps = [make8([(900 + 50 * i, 1), (30, 80)], 16, 8, 2, CAUSAL, seed=20 + i, device="cuda") for i in range(2)]
    refs = [reference8(p) for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        outs = [lca.attn_paged_fp8(p.q, p.kc, p.vc, p.ks, p.vs, p.table, p.q_start, p.k_len, CAUSAL, stream=s) for p, s in zip(ps, streams)]
    torch.cuda.synchronize()
    for p, r, (o, lse) in zip(ps, refs, outs):
        check8(o, lse, p, r)


# ------------------------------------------------------------------ together
def test_a_cache_read_back_gives_what_the_8_bit_one_gives(lca):
    """Attention over the 8-bit pages, over their 16-bit copy, and the packed forward over its rows: the same values, so
    each within its own bound of the same reference."""
    import torch

    p = make8([(400, 1), (100, 130), (0, 60)], 32, 8, 2, CAUSAL, seed=14, device="cuda")
    ref = reference8(p)
    o, lse, _ = attend(lca, p)
    check8(o, lse, p, ref)
    pages = p.table.flatten()
    k, v = lca.paged_read_fp8(p.kc, p.vc, p.ks, p.vs, pages)
    table = torch.arange(pages.numel(), dtype=torch.int32, device="cuda").view(p.table.shape)
    o2, lse2 = lca.attn_paged(p.q, k, v, table, p.q_start, p.k_len, CAUSAL)
    check8(o2, lse2, p, ref)
    width = p.table.shape[1] * 32
    segs = [Segment(s.q_off, s.q_len, i * width, s.k_len) for i, s in enumerate(p.prob.segments)]
    # the packed forward multiplies what lies behind a segment's last key by 0: no NaN of unwritten slots may lie there
    k, v = k.nan_to_num_(0.0), v.nan_to_num_(0.0)
    o3, lse3 = lca.attn_fwd(p.q, k.view(-1, 2, 128), v.view(-1, 2, 128), segs, CAUSAL)
    check8(o3, lse3, p, ref)


@pytest.mark.parametrize("dtype,interleaved", [("bf16", False), ("fp16", True)])
def test_a_captured_step_serves_later_batches(lca, dtype, interleaved):
    """Plan, rotary positions, quantising write and attention captured once; the replays see other lengths, pages and
    values, and their results are those of the oracle over the rotated, quantised history."""
    import torch

    g = torch.Generator().manual_seed(3)
    dt = torch_type(dtype)
    n, page, Hq, Hkv, rows, n_pages, width = 4, 16, 8, 2, 40, 64, 12
    ctx, new = (torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(2))
    taken = torch.zeros(1, dtype=torch.int32, device="cuda")
    free = torch.randperm(n_pages, generator=g).to(torch.int32).cuda()
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    kc, vc = (torch.full((n_pages, page, Hkv, 128), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.full((n_pages, Hkv, page), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2))
    qkv = torch.zeros(rows, Hq + 2 * Hkv, 128, dtype=dt, device="cuda")
    f = lca.rope_frequencies(64, 1000.0)

    def step():
        plan = lca.paged_plan(ctx, new, free, taken, table, page, n_pages, rows)
        q, k = lca.rope(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], plan.positions, f, interleaved=interleaved)
        lca.paged_write_fp8(k, qkv[:, Hq + Hkv:], kc, vc, ks, vs, plan.slots)
        return plan, q, k, lca.attn_paged_fp8(q, kc, vc, ks, vs, table, plan.q_start, plan.k_len, CAUSAL)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan, q, k, (o, lse) = step()
    have = [0] * n
    hist = [([], []) for _ in range(n)]
    for news in ([5, 0, 17, 1], [1, 1, 1, 1], [0, 30, 1, 9], [1, 1, 1, 1], [0, 0, 0, 0], [16, 3, 1, 20]):
        ctx.copy_(torch.tensor(have, dtype=torch.int32))
        new.copy_(torch.tensor(news, dtype=torch.int32))
        total = sum(news)
        qkv.copy_(torch.randn(qkv.shape, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        assert plan.state.tolist()[1:] == [0, 0, total]
        taken.copy_(plan.state[:1])
        at, kk, vv, segs, kat = 0, [], [], [], 0
        for i, w in enumerate(news):
            for h, x in ((hist[i][0], k), (hist[i][1], qkv[:, Hq + Hkv:])):
                y, e = quantise(x[at:at + w].double().cpu().numpy())
                h.append(torch.from_numpy(y * 2.0 ** e[..., None]).float())
            have[i] += w
            kk.append(torch.cat(hist[i][0]))
            vv.append(torch.cat(hist[i][1]))
            segs.append(Segment(at, w, kat, have[i]))
            at, kat = at + w, kat + have[i]
        p = make8([(0, 1)], 16, Hq, Hkv, CAUSAL, dtype)
        p.q, p.k, p.v = q, torch.cat(kk), torch.cat(vv)
        p.prob.Tq, p.prob.Tk, p.prob.segments = rows, kat, segs
        check8(o, lse, p, what=str(news))


@pytest.mark.parametrize("mask", MASKS, ids=lambda m: f"{m.kind}{m.window_left or ''}")
@pytest.mark.parametrize("case", ["rows", "table", "both", "long"])
def test_a_batch_that_does_not_fit_keeps_its_positions(lca, case, mask):
    """As in the 16-bit cache's test: rows with a slot are attended at the plan's positions, to keys that were written."""
    import torch

    from tests.test_paged_gpu import FITS_NOT

    lens, rows, width = FITS_NOT[case]
    page, Hq, Hkv, n = 16, 8, 2, len(lens)
    room, g = width * page, torch.Generator().manual_seed(len(case))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    n_pages = sum(-(-c // page) for c, _ in lens) + sum(-(-w // page) + 1 for _, w in lens)
    perm = torch.randperm(n_pages, generator=g).to(torch.int32)
    table, at = torch.full((n, width), -1, dtype=torch.int32), 0
    kc, vc = (torch.full((n_pages, page, Hkv, 128), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.full((n_pages, Hkv, page), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2))
    old = [[torch.randn(c, Hkv, 128, generator=g).to(torch.bfloat16) for _ in range(2)] for c, _ in lens]
    for i, (c, _) in enumerate(lens):
        m, j = -(-c // page), torch.arange(c)
        table[i, :m] = perm[at:at + m]
        at += m
        slots = (table[i].long()[j // page] * page + j % page).to(torch.int32)
        lca.paged_write_fp8(old[i][0].cuda(), old[i][1].cuda(), kc, vc, ks, vs, slots.cuda())
    q, k, v = (torch.randn(rows, h, 128, generator=g).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    table, qd, ctx = table.cuda(), q.cuda(), i32([c for c, _ in lens])
    plan = lca.paged_plan(ctx, i32([w for _, w in lens]), perm[at:].cuda(), i32([0]), table, page, n_pages, rows)
    lca.paged_write_fp8(k.cuda(), v.cuda(), kc, vc, ks, vs, plan.slots)
    segs, kk, vv, kat, row, behind = [], [], [], 0, 0, False
    for i, (c, w) in enumerate(lens):
        have = min(row + w, rows) - min(row, rows)
        served = min(have, room - c)
        behind |= served < have
        segs.append(Segment(min(row, rows), served, kat, c + served))
        kk += [old[i][0], k[row:row + served]]
        vv += [old[i][1], v[row:row + served]]
        kat, row = kat + c + served, row + w
    p = make8([(0, 1)], 16, Hq, Hkv, mask)
    p.q, p.kc, p.vc, p.ks, p.vs, p.table, p.q_start, p.k_len = qd, kc, vc, ks, vs, table, plan.q_start, plan.k_len
    for name, parts in (("k", kk), ("v", vv)):
        y, e = quantise(torch.cat(parts).double().numpy())
        setattr(p, name, torch.from_numpy(y * 2.0 ** e[..., None]).float())
    p.prob.Tq, p.prob.Tk, p.prob.segments = rows, kat, segs
    ref = reference8(p)
    for hint in (0, 700):
        o, lse, st = attend(lca, p, ctx_len=ctx, max_q_len=hint)
        assert st[0] == (6 if behind else 0)
        check8(o, lse, p, ref, what=f"{case}, max_q_len={hint}")


# ------------------------------------------------------------------ prompts of so many rows that the pages are copied first
LONG = [(300, 1100), (0, 1200), (700, 1), (1025, 900)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("layout,page", [("nhd", 16), ("hnd", 64), ("kv", 24), ("nhd", 256)])
def test_long_prompts(lca, layout, page, dtype):
    """6 heads of a group, so that the four requests have more than 4096 rows on average; beside them padding rows, and
    NaN wherever no request's token lies."""
    p = make8(LONG, page, 12, 2, CAUSAL, dtype, layout, pad=7, seed=page, device="cuda")
    ref = reference8(p)
    sizes = [lca.attn_paged_fp8_workspace_size(p.q, p.kc, p.vc, p.ks, p.vs, p.table, CAUSAL, max_q_len=h) for h in (0, 1200, 500, 1)]
    assert sizes[0] == max(sizes)  # a workspace for an unknown longest request serves every hint
    for kw in (dict(), dict(max_q_len=1200)):
        o, lse, st = attend(lca, p, **kw)
        check8(o, lse, p, ref)
        assert st == (0, 0)


def test_long_prompts_over_tables_and_pages_of_several_widths(lca):
    """Calls of the same rows whose workspaces differ, none of them given: wider tables, larger pages, a larger cache."""
    for page, more in ((16, 0), (16, 40), (64, 0), (16, 200), (64, 30)):
        import torch

        p = make8([(300, 600)], page, 8, 1, CAUSAL, seed=9, device="cuda")
        p.table = torch.nn.functional.pad(p.table, (0, more), value=-1)
        o, lse = lca.attn_paged_fp8(p.q, p.kc, p.vc, p.ks, p.vs, p.table, p.q_start, p.k_len, CAUSAL)
        check8(o, lse, p, what=f"{page}, {more}")


@pytest.mark.parametrize("mask", MASKS, ids=lambda m: f"{m.kind}{m.window_left or ''}")
def test_masks_of_long_prompts(lca, mask):
    p = make8([(300, 600), (0, 700)], 16, 8, 1, mask, seed=5, device="cuda")
    o, lse, st = attend(lca, p)
    check8(o, lse, p, what=mask.kind)
    assert st == (0, 0)


def test_long_prompts_with_pages_gone_or_bad(lca):
    """Pages before a window are gone and hold NaN; entries that are no page read as zeros and are reported, ones that
    no row needs are not; the next call on the same workspace sees nothing of them."""
    import torch

    mask = MaskSpec("CAUSAL_SLIDING", window_left=100)
    p = make8([(900, 600), (0, 520)], 16, 8, 1, mask, seed=6, device="cuda")
    ref = reference8(p)
    for e in range((900 - 100) // 16):
        for t in (p.kc, p.vc):
            t.view(torch.uint8)[int(p.table[0, e])] = 0x7F
        p.table[0, e] = -1 if e % 2 else 1 << 30
    o, lse, st = attend(lca, p)
    assert st == (0, 0)
    check8(o, lse, p, ref)
    q = make8([(900, 600), (0, 520)], 16, 8, 1, CAUSAL, seed=6, device="cuda")
    good = q.table.clone()
    q.table[0, 5] = q.kc.shape[0]
    o, lse, st = attend(lca, q)
    assert st[0] == 6
    k, v = q.k.clone(), q.v.clone()
    q.k[80:96] = 0
    q.v[80:96] = 0
    check8(o, lse, q)
    q.table, q.k, q.v = good, k, v
    o, lse, st = attend(lca, q)
    assert st == (0, 0)
    check8(o, lse, q)


def test_nan_in_long_prompts_and_lengths_that_do_not_fit(lca):
    """A NaN reaches the rows that attend it, in its column; cached lengths place the rows of a request that the tables
    have no room for; a bad length is clamped and reported."""
    import torch

    p = make8([(40, 1100)], 32, 8, 2, CAUSAL, seed=8, device="cuda")
    ref = reference8(p)
    o0, lse0, _ = attend(lca, p)
    check8(o0, lse0, p, ref)
    p.vc.view(torch.uint8)[int(p.table[0, 500 // 32]), 500 % 32, 0, 9] = 0x7F
    o, lse, st = attend(lca, p)
    assert st == (0, 0) and torch.equal(lse, lse0)
    assert bool(o[460:, :4, 9].isnan().all())
    o[460:, :4, 9] = o0[460:, :4, 9]
    check8(o, lse, p, ref)
    p = make8([(40, 1100)], 32, 8, 2, CAUSAL, seed=8, device="cuda")
    ctx = torch.tensor([40], dtype=torch.int32, device="cuda")
    room = 30 * 32
    p.table = p.table[:, :30].contiguous()
    p.k_len[0] = room
    o, lse, st = attend(lca, p, ctx_len=ctx)
    assert st[0] == 6
    assert bool(torch.isneginf(lse[:, room - 40:]).all()) and float(o[room - 40:].abs().max()) == 0
    p.prob.segments[0].q_len, p.prob.segments[0].k_len = room - 40, room
    check8(o, lse, p)
    p.k_len[0] = -1
    assert attend(lca, p)[2][0] == 6


def test_a_captured_long_prompt(lca):
    """One graph; its replays see other pages, lengths and queries."""
    import torch

    ps = [make8([(c, n)], 16, 8, 1, CAUSAL, seed=30 + c, device="cuda") for c, n in ((100, 700), (428, 400), (0, 800))]
    n = max(p.kc.shape[0] for p in ps)
    kc, vc = (torch.zeros(n, 16, 1, 128, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.zeros(n, 1, 16, dtype=torch.uint8, device="cuda") for _ in range(2))
    table = torch.full((1, max(p.table.shape[1] for p in ps)), -1, dtype=torch.int32, device="cuda")
    q = torch.zeros(800, 8, 128, dtype=torch.bfloat16, device="cuda")
    qs, kl = (torch.zeros(m, dtype=torch.int32, device="cuda") for m in (2, 1))

    def step():
        return lca.attn_paged_fp8(q, kc, vc, ks, vs, table, qs, kl, CAUSAL)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step()
    for p in ps:
        m, T = p.kc.shape[0], p.q.shape[0]
        for to, of in ((kc, p.kc), (vc, p.vc)):
            to.view(torch.uint8)[:m] = of.view(torch.uint8)
        ks[:m], vs[:m] = p.ks, p.vs
        table.fill_(-1)
        table[:, :p.table.shape[1]] = p.table
        q.zero_()
        q[:T] = p.q
        qs.copy_(p.q_start), kl.copy_(p.k_len)
        graph.replay()
        torch.cuda.synchronize()
        check8(o[:T], lse[:, :T], p)
        assert float(o[T:].abs().sum()) == 0 and bool(torch.isneginf(lse[:, T:]).all())


def test_a_long_prompt_with_a_window_copies_what_it_needs(lca):
    """500K cached tokens, most of them before the window, whose entries of the table are no page."""
    import torch

    page, Hkv, ctx, new = 64, 1, 500000, 600
    mask = MaskSpec("CAUSAL_SLIDING", window_left=1000)
    p = make8([(1400, new)], page, 8, Hkv, mask, seed=7, device="cuda")
    ref = reference8(p)
    o, lse, _ = attend(lca, p)
    check8(o, lse, p, ref)
    gone = (ctx - ctx % page - 1400 + 1400 % page) // page  # whole pages put before the request
    table = torch.full((1, gone + p.table.shape[1]), -1, dtype=torch.int32, device="cuda")
    table[:, gone:] = p.table
    p.table, p.k_len = table, p.k_len + gone * page
    o, lse, st = attend(lca, p)  # tiles of 128 keys may begin elsewhere, so other bits, within the same bounds
    assert st == (0, 0)
    check8(o, lse, p, ref)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hq,Hkv,new", [(8, 1, 1), (8, 2, 3), (8, 1, 2), (8, 1, 3), (12, 2, 4), (8, 1, 4), (3, 1, 7), (1, 1, 31), (32, 1, 1),
                                        (5, 1, 5), (28, 4, 4)])
def test_tiles_of_every_size(lca, Hq, Hkv, new, dtype):
    """Drafts of up to 32 rows per KV head, which one kernel serves in tiles of 8 to 32, beside shorter requests, and
    with hints that are larger than needed."""
    lens = [(700, new), (0, new), (33, 1), (5, 0), (1290, new), (64, max(1, new - 1))]
    for mask in (CAUSAL, MaskSpec("CAUSAL_SLIDING", window_left=50), MaskSpec("GLOBAL_SLIDING", window_left=70, window_right=0, num_global=5)):
        p = make8(lens, 24, Hq, Hkv, mask, dtype, pad=3, seed=new, device="cuda")
        ref = reference8(p)
        for hint in (new, 0, 400):
            o, lse, st = attend(lca, p, max_q_len=hint)
            check8(o, lse, p, ref, what=f"{mask.kind}, max_q_len={hint}")
            assert st == (0, 0)


@pytest.mark.parametrize("new", [2, 3, 4])
def test_nan_in_drafts(lca, new):
    """Every tile size: a NaN in the values of the drafts' own keys reaches the rows at and after it."""
    import torch

    p = make8([(600, new), (30, new)], 16, 8, 1, CAUSAL, seed=new, device="cuda")
    o0, lse0, _ = attend(lca, p, max_q_len=new)
    check8(o0, lse0, p)
    for i, c in enumerate((600, 30)):
        j = c + 1
        p.vc.view(torch.uint8)[int(p.table[i, j // 16]), j % 16, 0, 40] = 0xFF
    o, lse, st = attend(lca, p, max_q_len=new)
    assert st == (0, 0) and torch.equal(lse, lse0)
    hit = torch.tensor([t >= 1 for _ in range(2) for t in range(new)], device="cuda")
    assert bool(o[hit][:, :, 40].isnan().all()) and bool(o[~hit].isfinite().all())
    o[hit, :, 40] = o0[hit, :, 40]
    assert torch.equal(o, o0)
