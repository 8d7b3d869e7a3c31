"""The 8-bit paged cache without a GPU: refusals come before any launch (the
pointers are made up), and the tests' own quantisation against torch's e4m3."""
from __future__ import annotations

import ctypes as C
import os

import numpy as np
import pytest
import torch

import long_context_masked_attention_gb300 as lib
from gen import MaskSpec
from long_context_masked_attention_gb300 import binding as B
from tests.paged8_util import make8, quantise, reference8, to_bits

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
FAKE = 0x100000


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.LIB_PATH):
        lib.build()
    return lib.load()


def cache(**kw):
    c = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, n_pages=16, page_size=16, Hkv=2, d=128, page_stride=16 * 256,
             token_stride=256, head_stride=128, scale_page_stride=32, scale_head_stride=16)
    c.update(kw)
    return B.PagedCacheFp8_t(*c.values())


def out(**kw):
    c = dict(k=FAKE, v=FAKE, n_pages=16, page_size=16, Hkv=2, d=128, dtype=0, page_stride=16 * 256, token_stride=256,
             head_stride=128)
    c.update(kw)
    return B.PagedCache_t(*c.values())


def shape(**kw):
    s = dict(Tq=4, Hq=8, n_seq=2, max_pages=5, table_stride=5, q_stride=1024, max_q_len=0, scale=0.0)
    s.update(kw)
    return B.PagedShape_t(*s.values())


def write(L, ca, k=FAKE, v=FAKE, ks=256, vs=256, dtype=0, slots=FAKE, n=3):
    return L.lca_paged_write_fp8(k, v, ks, vs, dtype, slots, n, C.byref(ca) if ca else None, None)


def read(L, ca, o, pages=FAKE, n=4):
    return L.lca_paged_read_fp8(C.byref(ca) if ca else None, pages, n, C.byref(o) if o else None, None)


def attn(L, sh, ca, mask=MaskSpec("CAUSAL"), dtype=0, ws=0x100000, ws_bytes=1 << 40):
    md = B._paged_mask(mask)
    return L.lca_attn_paged_fp8(FAKE, dtype, C.byref(ca) if ca else None, FAKE, FAKE, FAKE, FAKE, FAKE, C.byref(sh),
                                C.byref(md), ws, ws_bytes, None)


def size(L, sh, ca, mask=MaskSpec("CAUSAL")):
    n = C.c_size_t(0)
    md = B._paged_mask(mask)
    return L.lca_attn_paged_fp8_workspace_size(C.byref(sh), C.byref(ca), C.byref(md), C.byref(n)), n.value


BAD_CACHE = [
    (dict(n_pages=-1), INVALID), (dict(page_size=0), INVALID), (dict(Hkv=0), INVALID), (dict(d=64), UNSUPPORTED),
    (dict(page_size=20), UNSUPPORTED), (dict(n_pages=1 << 28), UNSUPPORTED), (dict(page_stride=0), INVALID),
    (dict(token_stride=264), INVALID), (dict(head_stride=-128), INVALID), (dict(page_stride=1 << 39), INVALID),
    (dict(scale_page_stride=0), INVALID), (dict(scale_page_stride=36), INVALID), (dict(scale_head_stride=12), INVALID),
    (dict(scale_head_stride=-16), INVALID), (dict(scale_page_stride=1 << 39), INVALID),
    (dict(n_pages=100000, scale_page_stride=1 << 38), INVALID), (dict(Hkv=1 << 20, head_stride=1 << 38), INVALID),
    (dict(Hkv=1 << 24), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", BAD_CACHE, ids=str)
def test_bad_caches_are_refused(L, kw, code):
    ca, before = cache(**kw), L.lca_launch_count()
    assert write(L, ca) == code
    assert read(L, ca, out()) == code
    assert attn(L, shape(), ca) == code
    assert size(L, shape(), ca)[0] == code
    assert L.lca_launch_count() == before


@pytest.mark.parametrize("kw", [dict(ks=248), dict(vs=252), dict(ks=1 << 39), dict(dtype=2), dict(dtype=-1), dict(n=-1),
                                dict(k=None), dict(v=FAKE + 8), dict(slots=None), dict(slots=FAKE + 2), dict()], ids=str)
def test_bad_writes_are_refused(L, kw):
    assert write(L, cache(), **kw) == INVALID  # the last: memory that CUDA does not know


def test_bad_reads_are_refused(L):
    for o in (out(page_size=32), out(Hkv=4), out(n_pages=3), out(dtype=2), out(token_stride=260), out(), None):
        assert read(L, cache(), o) == INVALID
    assert read(L, cache(), out(d=64)) == UNSUPPORTED
    assert read(L, cache(), out(), n=-1) == INVALID and read(L, None, out()) == INVALID
    assert read(L, cache(), out(), pages=FAKE + 1) == INVALID


def test_nothing_to_do(L):
    assert write(L, cache(), n=0) == 0
    assert read(L, cache(), out(), n=0) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(Tq=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hq=7), INVALID), (dict(n_seq=-1), INVALID),
    (dict(max_pages=-1), INVALID), (dict(table_stride=4), INVALID), (dict(q_stride=1016), INVALID),
    (dict(q_stride=1028), INVALID), (dict(max_q_len=-1), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=3e38), INVALID), (dict(max_pages=1 << 26, table_stride=1 << 26), UNSUPPORTED),
    (dict(Tq=1 << 30), UNSUPPORTED), (dict(n_seq=1 << 30), UNSUPPORTED),
    (dict(Tq=1, Hq=1 << 24, q_stride=1 << 31), UNSUPPORTED),
], ids=str)
def test_bad_shapes_are_refused(L, kw, code):
    assert attn(L, shape(**kw), cache()) == code
    assert size(L, shape(**kw), cache())[0] == code


def test_masks_types_and_workspaces(L):
    for kind in ("SHARED_QUESTION", "PREFIX_LM_DOC", "BLOCK_SPARSE_UNIFORM", "BLOCK_SPARSE_VARIABLE", "FLASHMASK"):
        assert attn(L, shape(), cache(), MaskSpec(kind)) == UNSUPPORTED
    assert attn(L, shape(), cache(), MaskSpec("SLIDING", window_left=-1)) == INVALID
    assert attn(L, shape(), cache(), dtype=2) == INVALID and attn(L, shape(), None) == INVALID
    code, need = size(L, shape(), cache())
    assert code == 0 and need > 0
    assert attn(L, shape(), cache(), ws_bytes=need - 1) == WORKSPACE
    assert attn(L, shape(), cache(), ws=0x100010) == WORKSPACE and attn(L, shape(), cache(), ws=None) == WORKSPACE


def test_the_binding_turns_away_what_it_cannot_pass(L):
    meta = torch.device("meta")
    kc = torch.empty(4, 16, 2, 128, dtype=torch.float8_e4m3fn)
    ks = torch.empty(4, 2, 16, dtype=torch.uint8)
    k, slots = torch.empty(3, 2, 128, dtype=torch.bfloat16), torch.empty(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        lib.paged_write_fp8(k, k, kc, kc, ks, ks, slots)
    with pytest.raises(TypeError, match="k_cache"):
        lib.paged_write_fp8(k, k, None, kc, ks, ks, slots)
    with pytest.raises(ValueError, match="CUDA"):
        lib.paged_read_fp8(kc.to(meta), kc.to(meta), ks.to(meta), ks.to(meta), slots)
    with pytest.raises(ValueError, match="CUDA"):
        lib.attn_paged_fp8(k, kc, kc, ks, ks, slots[None], slots, slots, MaskSpec("CAUSAL"))


def test_the_plain_quantisation_is_torchs():
    """Every bf16 value of a few binades, and halves between e4m3 values, as torch rounds them."""
    x = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = x[torch.isfinite(x) & (x.abs() <= 448) & (x.abs() > 2.0 ** -20)]
    x = torch.cat([x, torch.zeros(-len(x) % 127, dtype=x.dtype)]).view(-1, 127)
    x = torch.cat([x, torch.full((len(x), 1), 448.0, dtype=x.dtype)], 1).float()  # every row's factor is 1
    y, e = quantise(x.numpy())
    assert (e == 0).all()
    assert np.array_equal(y, x.to(torch.float8_e4m3fn).double().numpy())
    assert torch.equal(to_bits(y).double(), torch.from_numpy(y))
    y, e = quantise(np.array([[448.0, 1.0], [448.1, 1.0], [0.0, 0.0], [1e30, 1.0], [1e-30, 0.0], [np.inf, 3.5], [224.0, 0], [225.0, 0]]))
    assert e.tolist() == [0, 1, -48, 48, -48, -7, -1, 0]
    assert y[3, 0] == 448 and np.isnan(y[5, 0]) and y[5, 1] == 448


def test_the_oracle_batch_is_what_its_cache_says():
    p = make8([(20, 3), (0, 9)], 16, 4, 2, MaskSpec("CAUSAL"), layout="kv", seed=3)
    e = (p.ks.to(torch.int32) - 127).transpose(1, 2)
    at = 0
    for i, n in enumerate(p.k_len.tolist()):
        j = torch.arange(n)
        pages = p.table[i].long()[j // 16]
        got = p.kc.float()[pages, j % 16].double() * 2.0 ** e[pages, j % 16].double()[..., None]
        assert torch.equal(got, p.k[at:at + n].double())
        at += n
    O, _, tol, _ = reference8(p)
    assert np.isfinite(O).all() and (tol > 0).all() and np.median(tol / np.abs(O).mean()) < 0.02
