"""Attention over the 8-bit paged cache where rows' factors differ far more than rows of one model's keys and values
do: every row of a result against the fp64 definition, within a bound of that row's own weights, so that a row of small
sums beside keys of large factors is tested as closely as any other."""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np
import pytest

from gen import MaskSpec
from tests.paged8_util import D, lay_out8, quantise, to_bits

SCALE = 1 / np.sqrt(D)
E32 = 2.0 ** -24
FAR = 1 << 29  # a window that hides nothing


@dataclass
class Batch:
    lens: list    # (cached tokens, new tokens) of each request
    Hq: int
    Hkv: int
    k8: list      # per request [n, Hkv, 128] e4m3 values, and the exponents of their rows' factors [n, Hkv]
    ke: list
    v8: list
    ve: list
    q: object     # [T, Hq, 128], a tensor of its type
    window: int = FAR

    @property
    def mask(self):
        return MaskSpec("CAUSAL") if self.window == FAR else MaskSpec("CAUSAL_SLIDING", window_left=self.window, window_right=0)


def make(lens, Hq, Hkv, dtype, seed, window=FAR):
    import torch

    g = np.random.default_rng(seed)
    parts = [[quantise(g.standard_normal((c + w, Hkv, D))) for c, w in lens] for _ in range(2)]
    (k8, ke), (v8, ve) = ([[x[i] for x in part] for i in (0, 1)] for part in parts)
    q = torch.from_numpy(g.standard_normal((sum(w for _, w in lens), Hq, D)))
    return Batch(lens, Hq, Hkv, k8, ke, v8, ve, q.to({"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]), window)


def on_gpu(b, page, layout="nhd", extra=0, seed=0):
    """The batch's cache, its pages in a shuffled order, and its tables; `extra` more entries to each table's row."""
    import torch

    g = torch.Generator().manual_seed(seed)
    need = [-(-(c + w) // page) for c, w in b.lens]
    n_pages = sum(need) + 2
    perm = torch.randperm(n_pages, generator=g)
    table = torch.full((len(need), max(need) + 1 + extra), -1, dtype=torch.int32)
    parts = [torch.full((n_pages, page, b.Hkv, D), 0x7F, dtype=torch.uint8) for _ in range(2)]
    parts += [torch.full((n_pages, b.Hkv, page), 0xFF, dtype=torch.uint8) for _ in range(2)]
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n].to(torch.int32)
        at += n
        j = torch.arange(sum(b.lens[i]))
        pages = table[i].long()[j // page]
        for to, f, x, e in ((parts[0], parts[2], b.k8[i], b.ke[i]), (parts[1], parts[3], b.v8[i], b.ve[i])):
            to[pages, j % page] = to_bits(x).view(torch.uint8)
            f[pages, :, j % page] = torch.from_numpy(e + 127).to(torch.uint8)
    q_start = np.cumsum([0] + [w for _, w in b.lens])
    i32 = lambda x: torch.tensor([int(y) for y in x], dtype=torch.int32, device="cuda")  # noqa: E731
    return (b.q.cuda(), *lay_out8(*parts, layout, "cuda"), table.cuda(), i32(q_start), i32(c + w for c, w in b.lens))


def bounds(b, copied=False):
    """(O, LSE, how far each element of O and LSE may be off), from the definition in 64 bits.

    A score is off by at most d_j = 130 e |q| |k_j| scale + 3 e (34 + |s_j|), e = 2^-24: its products and their sum, and
    the two roundings of score plus exponent (at most 48 ln 2 = 34).  A weight is w_j = 1 / (1 + sum of the others' e^(s_i
    - s_j)), so it lies between the values that it has with its own score off one way and all others the other way.
    Weights are rounded to 11 bits, or to the type's in the kernel over a copy of the pages, and the sums of n terms in
    32 bits cost (n + 16) e.  A weight in fp16 may also be off by 2^-25 however small it is (bf16 has the exponents of 32
    bits); the unit is at most twice the largest w_j 2^ev_j (the header's border of 2^-24), a term's value at most |v8_j|
    in it.
    O's own rounding: half a step, in fp16 at least 2^-25."""
    import torch

    u = torch.finfo(b.q.dtype).eps / 2
    u_w = u if copied else 2.0 ** -11
    q = b.q.double().numpy()
    T, G = q.shape[0], b.Hq // b.Hkv
    O, tol_o = np.zeros((T, b.Hq, D)), np.zeros((T, b.Hq, D))
    L, tol_l = np.zeros((b.Hq, T)), np.zeros((b.Hq, T))
    at = 0
    for i, (ctx, new) in enumerate(b.lens):
        r = slice(at, at + new)
        pos, j = np.arange(ctx, ctx + new)[:, None], np.arange(ctx + new)[None]
        seen = (j <= pos) & (j >= pos - b.window)
        n = seen.sum(1)[:, None]
        for h in range(b.Hkv):
            f = 2.0 ** b.ve[i][:, h]
            k, v8 = b.k8[i][:, h] * 2.0 ** b.ke[i][:, h, None], b.v8[i][:, h]
            v, kn = v8 * f[:, None], np.linalg.norm(k, axis=1)
            for head in range(h * G, h * G + G):
                x = q[r, head]
                s = x @ k.T * SCALE
                d = 130 * E32 * np.linalg.norm(x, axis=1)[:, None] * kn * SCALE + 3 * E32 * (34 + np.abs(s))
                s, lo, hi = (np.where(seen, y, -np.inf) for y in (s, s - d, s + d))

                def total(y):
                    m = y.max(1, keepdims=True)
                    return m + np.log(np.exp(y - m).sum(1, keepdims=True))

                def others(y):  # log of the sum of the others' e^y
                    t = total(y)
                    with np.errstate(divide="ignore"):
                        return t + np.log1p(-np.minimum(np.exp(y - t), 1.0))

                def share(own, rest):
                    return 1 / (1 + np.exp(np.clip(np.where(seen, rest - own, np.inf), -745, 700)))

                lse = total(s)
                w = np.where(seen, np.exp(s - lse), 0)
                off = np.where(seen, np.maximum(share(hi, others(lo)) - w, w - share(lo, others(hi))), 0)
                O[r, head] = w @ v
                L[head, r] = lse[:, 0]
                err = (off + w * (u_w + 2 * (n + 16) * E32)) @ np.abs(v)
                if not copied:
                    err += 2.0 ** -24 * (w * f).max(1, keepdims=True) * (seen @ np.abs(v8))
                tol_o[r, head] = u * np.abs(O[r, head]) + err * (1 + u) + (2.0 ** -25 if u == 2.0 ** -11 else 1e-38)
                tol_l[head, r] = np.maximum(total(hi) - lse, lse - total(lo))[:, 0] + n[:, 0] * E32 + 16 * E32 + \
                    4 * E32 * (2 * np.abs(lse[:, 0]) + 68)
        at += new
    return O, L, tol_o, tol_l


def close(o, lse, ref, what=""):
    O, L, tol_o, tol_l = ref
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    for name, x, X, tol in (("o", o, O, tol_o), ("lse", lse, L, tol_l)):
        bad = ~(np.abs(x - X) <= tol)
        at = np.argwhere(bad)[0] if bad.any() else None
        assert at is None, f"{what} {name}: {bad.sum()} of {bad.size}, first at {at}: {x[tuple(at)]}, expected {X[tuple(at)]} +- {tol[tuple(at)]}"


def attend(lca, b, page, layout="nhd", **kw):
    import torch

    q, kc, vc, ks, vs, table, q_start, k_len = on_gpu(b, page, layout, kw.pop("extra", 0))
    need = lca.attn_paged_fp8_workspace_size(q, kc, vc, ks, vs, table, b.mask)
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")
    o, lse = lca.attn_paged_fp8(q, kc, vc, ks, vs, table, q_start, k_len, b.mask, workspace=ws, **kw)
    torch.cuda.synchronize()
    assert lca.read_status(ws) == (0, 0)
    return o, lse


# ------------------------------------------------------------------ batches
# requests of few and of many rows; prompts whose pages are copied first (bf16 queries)
DIRECT = [(300, 40), (90, 3), (500, 75)]
COPIED = [(300, 260), (0, 320)]
KINDS = {"direct": (DIRECT, 8, 2), "copied": (COPIED, 8, 1)}
CASES = [(kind, dtype) for kind in KINDS for dtype in ("bf16", "fp16")]


def values_hidden(b, by):
    """Values 2^by times the others' in keys that the requests' first new tokens do not attend."""
    for (c, w), e in zip(b.lens, b.ve):
        e[c + w // 2] += by
        if c > 100:
            e[c + w - 1, 0] += by


def values_negligible(b, by):
    """Values 2^by times the others' in early keys that all rows attend with a weight of about e^-100 and less."""
    b.q[..., 0] = 20.0
    for (c, w), k8, ke, ve in zip(b.lens, b.k8, b.ke, b.ve):
        if c > 20:
            j = [5, 17]
            k8[j, :, 0], ke[j] = -448, -3
            ve[j] += by


def values_descending(b, by):
    """From 2^by times the last keys' down, under a window: what a row attends is smaller than all before."""
    for (c, w), ve in zip(b.lens, b.ve):
        ve += np.linspace(by, 0, c + w).astype(ve.dtype)[:, None]


def values_any(b, by):
    g = np.random.default_rng(by)
    for ve in b.ve:
        ve[:] = g.integers(-by // 2, by // 2 + 1, ve.shape)


VALUES = {"hidden": (values_hidden, FAR), "negligible": (values_negligible, FAR), "descending": (values_descending, 30),
          "any": (values_any, FAR), "any_window": (values_any, 3)}


def keys_hidden(b, by):
    """Keys 2^by times the others in places that the requests' first new tokens do not attend."""
    for (c, w), e in zip(b.lens, b.ke):
        e[c + w // 2] += by


def keys_against(b, by):
    """Keys 2^by times the others whose scores are far below all others, so that they weigh nothing."""
    b.q[..., 0] = 1.0
    for (c, w), k8, ke in zip(b.lens, b.k8, b.ke):
        if c > 20:
            k8[[3, 150 % c]] = 0
            k8[[3, 150 % c], :, 0] = -448
            ke[[3, 150 % c]] = by - 8


def keys_any(b, by):
    """Factors of every size below the others' own."""
    g = np.random.default_rng(by)
    for ke in b.ke:
        ke[:] = g.integers(-by - 6, -6, ke.shape)


def keys_that_take_all(b, by):
    """One key of a score of about 2^by for some rows and about -2^by for others."""
    for (c, w), ke in zip(b.lens, b.ke):
        ke[c // 2] += by


def keys_all_large(b, by):
    for ke in b.ke:
        ke += by


KEYS = {"all_large": keys_all_large, "hidden": keys_hidden, "against": keys_against, "any": keys_any, "take_all": keys_that_take_all}


def batch(kind, dtype, change, by, window=FAR, seed=1):
    lens, Hq, Hkv = KINDS[kind]
    b = make(lens, Hq, Hkv, dtype, seed, window)
    change(b, by)
    if dtype == "fp16":  # o stays in range
        for ve in b.ve:
            ve -= max(ve.max() - 5, 0)
    return b


# ------------------------------------------------------------------ the bound itself
@pytest.mark.parametrize("name,by", [("hidden", 40), ("negligible", 40), ("descending", 40), ("any", 80), ("any_window", 80)])
def test_the_bound_refuses_a_row_of_zeros(name, by):
    """Every row's bound is small beside the row itself: an o of zeros is outside it, and so is one made without the
    keys of small factors, unless every row attends large ones."""
    change, window = VALUES[name]
    b = batch("direct", "bf16", change, by, window)
    O, L, tol_o, tol_l = bounds(b)
    assert (tol_o.max(-1) < 0.2 * np.abs(O).max(-1)).all()
    assert (np.abs(O) > tol_o).any(-1).all()
    if name == "any":
        return
    for i in range(len(b.lens)):  # what lies 2^31 below the largest factor goes
        b.v8[i] *= (b.ve[i] > b.ve[i].max() - 31)[..., None]
    wrong = bounds(b)[0]
    assert (np.abs(wrong - O) > tol_o).any()


@pytest.mark.parametrize("name", list(KEYS))
def test_the_bound_of_scores(name):
    b = batch("direct", "bf16", KEYS[name], 30)
    O, L, tol_o, tol_l = bounds(b)
    fine = tol_o.max(-1) < 0.2 * np.abs(O).max(-1)
    assert fine.mean() > 0.98  # a row of two huge scores that are nearly equal has no bound
    assert fine[(np.abs(L.T) < 100)].all()


# ------------------------------------------------------------------ values
@pytest.mark.gpu
@pytest.mark.parametrize("kind,dtype", CASES)
@pytest.mark.parametrize("by", [6, 9, 14, 24, 33, 45])
@pytest.mark.parametrize("name", list(VALUES))
def test_values_of_far_sizes(lca, name, by, kind, dtype):
    change, window = VALUES[name]
    b = batch(kind, dtype, change, 2 * by if "any" in name else by, window)
    ref = bounds(b, (kind, dtype) == ("copied", "bf16"))
    for page, layout in ((16, "nhd"), (64, "hnd")):
        close(*attend(lca, b, page, layout), ref, f"{name}, pages of {page}")


@pytest.mark.gpu
@pytest.mark.parametrize("kind,dtype", CASES)
@pytest.mark.parametrize("by", [6, 20, 26, 40])
@pytest.mark.parametrize("name", list(KEYS))
def test_keys_of_far_sizes(lca, name, by, kind, dtype):
    b = batch(kind, dtype, KEYS[name], by)
    ref = bounds(b, (kind, dtype) == ("copied", "bf16"))
    for page, layout in ((16, "nhd"), (64, "hnd")):
        close(*attend(lca, b, page, layout), ref, f"{name}, pages of {page}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,by,q_by", [("bf16", 6, 0), ("bf16", 26, 0), ("bf16", 40, 0), ("fp16", 6, 0), ("fp16", 13, 7), ("fp16", 13, 12)])
def test_large_scores_over_the_cache_read_back(lca, dtype, by, q_by):
    """The same through lca_attn_paged over a 16-bit cache of the same values: prompts, whose kernel is shared."""
    import torch

    b = make([(300, 40), (500, 75)], 8, 2, dtype, 3)
    keys_all_large(b, by)
    b.q *= 2.0 ** q_by
    q, kc, vc, ks, vs, table, q_start, k_len = on_gpu(b, 16)
    k, v = lca.paged_read_fp8(kc, vc, ks, vs, torch.arange(kc.shape[0], dtype=torch.int32, device="cuda"), dtype=b.q.dtype)
    close(*lca.attn_paged(q, k, v, table, q_start, k_len, b.mask), bounds(b, copied=dtype == "bf16"))


@pytest.mark.gpu
@pytest.mark.parametrize("by", [0, 26])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_many_requests_without_keys_beside_one_with(lca, dtype, by):
    """Rows of requests that hold no keys, more blocks of them than CTAs, before, between and behind one that does."""
    import torch

    lens = [(0, 300)] * 40 + [(200, 70)] + [(0, 260)] * 40 + [(500, 33)] + [(0, 300)] * 5
    b = make(lens, 8, 2, dtype, 4)
    keys_all_large(b, by)
    q, kc, vc, ks, vs, table, q_start, k_len = on_gpu(b, 16)
    held = torch.tensor([c > 0 for c, _ in lens], device="cuda")
    o, lse = lca.attn_paged_fp8(q, kc, vc, ks, vs, table, q_start, torch.where(held, k_len, 0).to(torch.int32), b.mask)
    kept = held.repeat_interleave(torch.tensor([w for _, w in lens], device="cuda"))
    assert not bool(o[~kept].any()) and bool(torch.isneginf(lse[:, ~kept]).all())
    some = [i for i, (c, _) in enumerate(lens) if c > 0]
    part = Batch([lens[i] for i in some], 8, 2, *([x[i] for i in some] for x in (b.k8, b.ke, b.v8, b.ve)), b.q[kept.cpu()])
    close(o[kept], lse[:, kept], bounds(part))


@pytest.mark.gpu
def test_a_request_gets_the_same_alone_and_in_a_prompt_of_many_rows(lca):
    """fp16 queries and keys that would pass 65504 as fp16 values: a few tokens alone, in a call that takes the kernel
    for few rows, and as the last ones of a long prompt."""
    import torch

    b = make([(0, 500)], 8, 1, "fp16", 6)
    b.k8[0][:, :, 64:] = 0
    b.ke[0][::7] += 18
    b.q[..., :64] *= 2.0 ** -14
    ref = bounds(b)
    o, lse = attend(lca, b, 16)
    close(o, lse, ref)
    few = Batch([(497, 3)], 8, 1, b.k8, b.ke, b.v8, b.ve, b.q[497:])
    o3, lse3 = attend(lca, few, 16, max_q_len=3)
    close(o3, lse3, tuple(x[497:] if i in (0, 2) else x[:, 497:] for i, x in enumerate(ref)))


@pytest.mark.gpu
def test_prompts_of_wider_groups_are_not_copied(lca):
    """136 query heads of a KV head have no use for a copy of the pages: no workspace for one, and the results."""
    import torch

    b = make([(40, 30)], 136, 1, "bf16", 7)
    close(*attend(lca, b, 16), bounds(b))
    _, kc, vc, ks, vs, table, _, _ = on_gpu(b, 16, extra=1 << 14)
    narrow, wide = (lca.attn_paged_fp8_workspace_size(b.q.cuda(), kc, vc, ks, vs, t, b.mask) for t in (table[:, :8].contiguous(), table))
    assert narrow == wide


@pytest.mark.gpu
@pytest.mark.parametrize("name,by", [("all_large", 26), ("all_large", 40), ("hidden", 40), ("any", 40)])
def test_few_rows_beside_prompts_whose_pages_are_copied(lca, name, by):
    """Single tokens and drafts in the batch of such prompts: as exact as they are without it."""
    b = make([(300, 500), (200, 1), (0, 520), (60, 2)], 8, 1, "bf16", 2)
    KEYS[name](b, by)
    o, lse = attend(lca, b, 16)
    ref = bounds(b, copied=True)
    close(o, lse, ref)
    few = [500, 1021, 1022]
    near = bounds(b)
    close(o[few], lse[:, few], tuple(x[few] if i in (0, 2) else x[:, few] for i, x in enumerate(near)))


# ------------------------------------------------------------------ far factors and everything else
@pytest.mark.gpu
@pytest.mark.parametrize("name,by", [("hidden", 45), ("negligible", 33), ("descending", 45), ("any", 90), ("any_window", 60)])
def test_values_of_far_sizes_split_over_keys(lca, name, by):
    """Items that several CTAs share, whose sums are joined."""
    change, window = VALUES[name]
    b = make([(5000, 40), (1000, 130), (0, 33)], 8, 2, "bf16", 5, window)
    change(b, by)
    close(*attend(lca, b, 64), bounds(b))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("by,col", [(0, 40), (0, 41), (0, 42), (0, 43), (40, 0), (40, 127)])
def test_nan_beside_far_sizes(lca, by, col, dtype):
    """A NaN in a key, or in its values, whose factors are 2^by times the others': the rows that do not attend it are
    those of the batch without it, bit for bit; those that do are NaN, in its column if it is in the values."""
    import torch

    b = make([(300, 60), (40, 200)], 8, 2, dtype, 8)
    values_hidden(b, by)
    if dtype == "fp16":
        for ve in b.ve:
            ve -= max(ve.max() - 5, 0)
    at = [330, 140]  # hidden from the requests' first new tokens: 30 of 60, 100 of 200
    q, kc, vc, ks, vs, table, q_start, k_len = on_gpu(b, 16)
    call = lambda: lca.attn_paged_fp8(q, kc, vc, ks, vs, table, q_start, k_len, b.mask)  # noqa: E731
    o0, lse0 = call()
    seen = torch.cat([torch.arange(60) >= 30, torch.arange(200) >= 100]).cuda()
    for c, cols in ((vc, [col]), (kc, slice(None))):
        old = c.view(torch.uint8).clone()
        for i, j in enumerate(at):
            c.view(torch.uint8)[int(table[i, j // 16]), j % 16, 1, col] = 0x7F
        o, lse = call()
        assert torch.equal(o[~seen], o0[~seen]) and torch.equal(lse[:, ~seen], lse0[:, ~seen])
        assert torch.equal(o[:, :4], o0[:, :4])  # the other KV head's
        assert bool(o[seen][:, 4:, cols].isnan().all())
        if cols != slice(None):
            rest = [x for x in range(D) if x != col]
            assert torch.equal(o[:, :, rest], o0[:, :, rest]) and torch.equal(lse, lse0)
        c.view(torch.uint8)[:] = old
