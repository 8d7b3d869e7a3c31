"""8-bit paged caches for the tests: the requests of paged_util with their keys
and values quantised by a plain loop in doubles, and what a kernel's results may be off."""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

import oracle
from tests import paged_util
from tests.paged_util import D, Paged

LOW, HIGH = -48, 48  # exponents of a row's factor


def quantise(x):
    """[.., 128] numbers -> (e4m3 values as doubles, exponents of the rows' factors): the smallest e with
    448 2^e >= the largest finite magnitude, values rounded to the nearest multiple of 2^-3 of their binade (2^-9
    below 2^-6), even ones of two; infinities and NaN become NaN."""
    x = np.asarray(x, dtype=np.float64)
    fin = np.isfinite(x)
    top = np.abs(np.where(fin, x, 0)).max(-1)
    e = np.full(top.shape, LOW)
    for k in range(LOW, HIGH):
        e += top > 448 * 2.0 ** k
    y = np.where(fin, x, 0) / 2.0 ** e[..., None]
    binade = np.frexp(np.maximum(np.abs(y), 2.0 ** -6))[1] - 1
    step = 2.0 ** (binade - 3.0)
    return np.where(fin, np.clip(np.rint(y / step) * step, -448, 448), np.nan), e


def to_bits(y):
    """e4m3 values as float8 tensors, by torch's own table of them."""
    import torch

    return torch.from_numpy(np.ascontiguousarray(y)).float().to(torch.float8_e4m3fn)


@dataclass
class Paged8(Paged):
    ks: object = None
    vs: object = None


def lay_out8(lk, lv, lks, lvs, layout, device):
    """Values [n_pages, page, Hkv, D] (uint8) and bytes [n_pages, Hkv, page] on the device: nhd, hnd, or kv: all of a
    page in one row of bytes, K, V, and their factors behind them."""
    import torch

    e4 = torch.float8_e4m3fn
    if layout == "nhd":
        return tuple(x.to(device).view(e4) for x in (lk, lv)) + tuple(x.to(device) for x in (lks, lvs))
    if layout == "hnd":
        kc, vc = (x.transpose(1, 2).contiguous().to(device).transpose(1, 2).view(e4) for x in (lk, lv))
        return kc, vc, lks.to(device), lvs.to(device)
    n, page, H, _ = lk.shape
    m, f = page * H * D, H * page
    blob = torch.cat([lk.reshape(n, -1), lv.reshape(n, -1), lks.reshape(n, -1), lvs.reshape(n, -1)], 1)
    pad = -blob.shape[1] % 16
    blob = torch.cat([blob, blob.new_zeros(n, pad)], 1).to(device)
    row = blob.shape[1]
    kc, vc = (blob.as_strided((n, page, H, D), (row, H * D, D, 1), at).view(e4) for at in (0, m))
    ks, vs = (blob.as_strided((n, H, page), (row, page, 1), at) for at in (2 * m, 2 * m + f))
    return kc, vc, ks, vs


def make8(lens, page, Hq, Hkv, mask, dtype="bf16", layout="nhd", fill=0x7F, fill_scale=0xFF, pad=0, seed=1, q_scale=1.0,
          kv_scale=1.0, device="cpu") -> Paged8:
    """As paged_util.make.  fill, fill_scale: bytes of the rest of the cache and of its factors (0x7F is NaN).  Rows
    differ in size by powers of two."""
    import torch

    p = paged_util.make(lens, page, Hq, Hkv, mask, dtype, "nhd", 0.0, pad, seed, q_scale)
    n_pages = p.kc.shape[0]
    lk, lv = (torch.full((n_pages, page, Hkv, D), fill, dtype=torch.uint8) for _ in range(2))
    lks, lvs = (torch.full((n_pages, Hkv, page), fill_scale, dtype=torch.uint8) for _ in range(2))
    g = torch.Generator().manual_seed(seed + 1000)
    packed = []
    for x, c, s in ((p.k, lk, lks), (p.v, lv, lvs)):
        x = x.double() * kv_scale * torch.randint(-3, 3, (*x.shape[:2], 1), generator=g).double().exp2()
        y, e = quantise(x.numpy())
        packed.append(torch.from_numpy(y * 2.0 ** e[..., None]).float())
        bits, e, at = to_bits(y).view(torch.uint8), torch.from_numpy(e + 127).to(torch.uint8), 0
        for i, (ctx, new) in enumerate(lens):
            j = torch.arange(ctx + new)
            pages = p.table[i].long()[j // page]
            c[pages, j % page] = bits[at:at + len(j)]
            s[pages, :, j % page] = e[at:at + len(j)]
            at += len(j)
    kc, vc, ks, vs = lay_out8(lk, lv, lks, lvs, layout, device)
    return Paged8(p.q.to(device), kc, vc, p.table.to(device), p.q_start.to(device), p.k_len.to(device), *packed, p.prob, ks, vs)


def reference8(p: Paged8):
    """paged_util.reference over the values that the cache stands for, with what differs in the 8-bit kernels.  In
    natural units and beside that reference's bounds:
      scores    q's 16-bit form is exact but for values below 2^-28 of the row's largest, which lose 2^-39 of it:
                inside the 130 e B that cover the products (e = 2^-24); a key's score plus its factor's exponent (at
                most 48 ln 2 = 34) is rounded twice and the maximum is taken off: 3 e (34 + |s|), |s| <= B
      weights   are rounded to 2^-11 or the type's u, whichever is more in the kernel that serves the row, and lose
                2^-37 of the largest weight: times 448 2^ev and against a sum that has the largest key's weight (its
                row's largest value at least 224 2^ev, or a row of zeros), 2^-36 of the largest |v| for each key
      O         in fp16 a result below 2^-14 is rounded to a multiple of 2^-24, off by 2^-25 however small it is, so u |O|
                alone does not hold its own rounding
      LSE       the maximum and the logarithm of the sum, each at most |LSE| + 34 + B, cancel: 4 e of both"""
    import torch

    O, L = oracle.attention_forward(p.prob, p.q, p.k, p.v)
    A, _ = oracle.attention_forward(p.prob, p.q, p.k, p.v.abs())
    u = torch.finfo(p.q.dtype).eps / 2
    e = 2.0 ** -24
    qn = p.q.float().cpu().norm(dim=-1).double().numpy()
    G = p.prob.Hq // p.prob.Hkv
    tol_o, tol_l = np.zeros_like(O), np.zeros_like(L)
    for s in p.prob.segments:
        r = slice(s.q_off, s.q_off + s.q_len)
        if s.q_len == 0 or s.k_len == 0:
            continue
        ks = slice(s.k_off, s.k_off + s.k_len)
        kn = p.k[ks].norm(dim=-1).amax(0).double().numpy().repeat(G)
        vm = p.v[ks].abs().amax(-1).amax(0).double().numpy().repeat(G)  # [Hq]
        B = qn[r] * kn * p.prob.softmax_scale
        sc = 130 * e * B + 3 * e * (34 + B)
        n = (s.k_len + 16) * e
        tol_o[r] = u * np.abs(O[r]) + A[r] * (u + 2 * (sc + n))[:, :, None] * (1 + u) + (s.k_len * 2.0 ** -36 * vm)[None, :, None] + (2.0 ** -25 if u == 2.0 ** -11 else 1e-30)
        fin = np.isfinite(L[:, r])
        tol_l[:, r] = np.where(fin, sc.T + n + 4 * e * (2 * np.abs(np.where(fin, L[:, r], 0)) + 68 + 2 * B.T), 0)
    return O, L, tol_o, tol_l


def check8(o, lse, p, ref=None, what=""):
    paged_util.check(o, lse, p, ref or reference8(p), what)
