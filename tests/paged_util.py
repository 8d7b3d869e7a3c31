"""Paged caches for the tests: requests' keys and values scattered over pages
in a shuffled order, everything else in the cache filled with a given value,
and the same batch as packed segments for the fp64 oracle."""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

import oracle
from gen import MaskSpec, Problem, Segment

D = 128


@dataclass
class Paged:
    q: object
    kc: object
    vc: object
    table: object
    q_start: object
    k_len: object
    k: object  # packed keys, request after request [sum k_len, Hkv, 128]
    v: object
    prob: object


def make(lens, page, Hq, Hkv, mask, dtype="bf16", layout="nhd", fill=float("nan"), pad=0, seed=1, q_scale=1.0,
         device="cpu"):
    """lens: (cached tokens, new tokens) per request.  fill: what the rest of
    the cache holds.  pad: rows of q behind the last request."""
    import torch

    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    g = torch.Generator().manual_seed(seed)
    n = len(lens)
    k_len = [c + w for c, w in lens]
    q_start = np.concatenate([[0], np.cumsum([w for _, w in lens])]).astype(np.int64)
    T = int(q_start[-1]) + pad
    need = [-(-x // page) for x in k_len]
    n_pages, width = sum(need) + 3, max(need + [0]) + 2
    perm = torch.randperm(n_pages, generator=g)
    table = torch.full((n, width), -1, dtype=torch.int32)
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = perm[at:at + m].to(torch.int32)
        at += m
    k, v = (torch.randn(sum(k_len), Hkv, D, generator=g).to(dt) for _ in range(2))
    q = (torch.randn(T, Hq, D, generator=g) * q_scale).to(dt)
    # logical caches [n_pages, page, Hkv, D], then laid out
    lk, lv = (torch.full((n_pages, page, Hkv, D), fill, dtype=dt) for _ in range(2))
    at = 0
    for i, m in enumerate(k_len):
        j = torch.arange(m)
        pages = table[i].long()[j // page]
        lk[pages, j % page] = k[at:at + m]
        lv[pages, j % page] = v[at:at + m]
        at += m
    kc, vc = lay_out(lk, lv, layout, device)
    segs, at = [], 0
    for i, m in enumerate(k_len):
        segs.append(Segment(int(q_start[i]), lens[i][1], at, m))
        at += m
    prob = Problem("paged", T, sum(k_len), Hq, Hkv, D, segs, mask, seed)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=device)  # noqa: E731
    return Paged(q.to(device), kc, vc, table.to(device), i32([int(x) for x in q_start]), i32(k_len), k, v, prob)


def lay_out(lk, lv, layout, device):
    """nhd / hnd: one array each; kv: K and V in one array, [page][K, V][token][head]."""
    import torch

    if layout == "nhd":
        return lk.to(device), lv.to(device)
    if layout == "hnd":
        return tuple(x.transpose(1, 2).contiguous().to(device).transpose(1, 2) for x in (lk, lv))
    both = torch.stack([lk, lv], 1).to(device)
    return both[:, 0], both[:, 1]


def reference(p: Paged):
    """O, LSE in fp64, and the elementwise bounds of what a kernel may be off.

    With u the half step of the type (2^-8 bf16, 2^-11 fp16, relative to the
    value), e = 2^-24 that of fp32, A = sum_j p_j |v_j| and B >= every
    scale * sum_c |q_c k_c| of the row:
      scores    130 e B                      (128 products summed in any order, scaled)
      O         u |O| for its own rounding, and A times u (p is rounded to the
                type before the products) plus twice (the numerator's and the
                denominator's) 130 e B + (n + 16) e (n terms summed, exp2)
      LSE       130 e B + (n + 16) e + 4 e |LSE|
    A row that attends nothing has 0 and -inf exactly."""
    import torch

    O, L = oracle.attention_forward(p.prob, p.q, p.k, p.v)
    A, _ = oracle.attention_forward(p.prob, p.q, p.k, p.v.float().abs())
    u = torch.finfo(p.q.dtype).eps / 2
    e = 2.0 ** -24
    qn = p.q.float().cpu().norm(dim=-1).double().numpy()  # [T, Hq]
    G = p.prob.Hq // p.prob.Hkv
    tol_o, tol_l = np.zeros_like(O), np.zeros_like(L)
    for s in p.prob.segments:
        r = slice(s.q_off, s.q_off + s.q_len)
        if s.q_len == 0 or s.k_len == 0:
            continue
        kn = p.k[s.k_off:s.k_off + s.k_len].float().norm(dim=-1).amax(0).double().numpy().repeat(G)  # [Hq]
        sc = 130 * e * qn[r] * kn * p.prob.softmax_scale
        n = (s.k_len + 16) * e
        tol_o[r] = u * np.abs(O[r]) + A[r] * (u + 2 * (sc + n))[:, :, None] * (1 + u) + 1e-30
        fin = np.isfinite(L[:, r])
        tol_l[:, r] = np.where(fin, sc.T + n + 4 * e * np.abs(np.where(fin, L[:, r], 0)), 0)
    return O, L, tol_o, tol_l


def check(o, lse, p: Paged, ref=None, what=""):
    import torch

    O, L, tol_o, tol_l = ref or reference(p)
    assert o.dtype == p.q.dtype and lse.dtype == torch.float32
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(o).all(), f"{what}: {np.argwhere(~np.isfinite(o))[:4]} not finite"
    assert np.array_equal(np.isneginf(lse), np.isneginf(L)), f"{what}: rows without keys differ"
    fin = np.isfinite(L)
    off = np.abs(np.where(fin, lse, 0) - np.where(fin, L, 0)) - tol_l
    assert off.max(initial=-1) <= 0, f"{what}: LSE off by {off.max():.3g} past its bound at {np.unravel_index(off.argmax(), off.shape)}"
    off = np.abs(o - O) - tol_o
    assert off.max(initial=-1) <= 0, f"{what}: O off by {off.max():.3g} past its bound at {np.unravel_index(off.argmax(), off.shape)}"


MASKS = [
    MaskSpec("CAUSAL"), MaskSpec("FULL"), MaskSpec("DOC"), MaskSpec("CAUSAL_DOC"),
    MaskSpec("SLIDING", window_left=40, window_right=9), MaskSpec("CAUSAL_SLIDING", window_left=0),
    MaskSpec("CAUSAL_SLIDING", window_left=150), MaskSpec("GLOBAL_SLIDING", window_left=70, window_right=0, num_global=5),
    MaskSpec("CAUSAL_BLOCKWISE", block=100), MaskSpec("PREFIX_LM_CAUSAL", prefix_len=90),
    MaskSpec("BLOCK_CAUSAL_DOC", block=50),
]
