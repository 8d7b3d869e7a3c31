"""The paged-cache entry points without a GPU: every refusal comes before any
launch (all pointers below are made up), workspaces are sized on the host, and
the binding turns away tensors that the library would misread."""
from __future__ import annotations

import ctypes as C
import os

import numpy as np
import pytest
import torch

import long_context_masked_attention_gb300 as lib
from gen import MaskSpec
from long_context_masked_attention_gb300 import binding as B

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
FAKE = 0x100000


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.LIB_PATH):
        lib.build()
    return lib.load()


def cache(**kw):
    c = dict(k=FAKE, v=FAKE, n_pages=16, page_size=16, Hkv=2, d=128, dtype=0, page_stride=16 * 256, token_stride=256,
             head_stride=128)
    c.update(kw)
    return B.PagedCache_t(*c.values())


def shape(**kw):
    s = dict(Tq=4, Hq=8, n_seq=2, max_pages=5, table_stride=5, q_stride=1024, max_q_len=0, scale=0.0)
    s.update(kw)
    return B.PagedShape_t(*s.values())


def size(L, sh, ca, mask=MaskSpec("CAUSAL")):
    n = C.c_size_t(0)
    md = B._paged_mask(mask)
    return L.lca_attn_paged_workspace_size(C.byref(sh), C.byref(ca), C.byref(md), C.byref(n)), n.value


def attn(L, sh, ca, mask=MaskSpec("CAUSAL"), ws=0x100000, ws_bytes=1 << 40):
    md = B._paged_mask(mask)
    return L.lca_attn_paged(FAKE, C.byref(ca), FAKE, FAKE, FAKE, FAKE, FAKE, C.byref(sh), C.byref(md), ws, ws_bytes, None)


BAD_CACHE = [
    (dict(dtype=2), INVALID), (dict(n_pages=-1), INVALID), (dict(page_size=0), INVALID), (dict(Hkv=0), INVALID),
    (dict(d=64), UNSUPPORTED), (dict(page_size=20), UNSUPPORTED), (dict(n_pages=1 << 28), UNSUPPORTED),
    (dict(page_stride=0), INVALID), (dict(token_stride=130), INVALID), (dict(head_stride=-128), INVALID),
    (dict(page_stride=1 << 39), INVALID),
]
BAD_SHAPE = [
    (dict(Tq=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hq=7), INVALID), (dict(n_seq=-1), INVALID),
    (dict(max_pages=-1), INVALID), (dict(max_q_len=-1), INVALID), (dict(table_stride=4), INVALID),
    (dict(q_stride=1016), INVALID), (dict(q_stride=1025), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(max_pages=1 << 27, table_stride=1 << 27), UNSUPPORTED), (dict(Tq=1 << 30), UNSUPPORTED),
    (dict(Tq=1 << 29), UNSUPPORTED),
]
BAD_MASK = [
    (MaskSpec("SLIDING", window_left=-1), INVALID), (MaskSpec("CAUSAL_SLIDING", window_right=-1), INVALID),
    (MaskSpec("GLOBAL_SLIDING", num_global=-1), INVALID), (MaskSpec("PREFIX_LM_CAUSAL", prefix_len=-2), INVALID),
    (MaskSpec("CAUSAL_BLOCKWISE", block=0), INVALID), (MaskSpec("BLOCK_CAUSAL_DOC", block=-3), INVALID),
    (MaskSpec(99), INVALID), (MaskSpec(-1), INVALID), (MaskSpec("SHARED_QUESTION"), UNSUPPORTED),
    (MaskSpec("PREFIX_LM_DOC"), UNSUPPORTED), (MaskSpec("BLOCK_SPARSE_UNIFORM"), UNSUPPORTED),
    (MaskSpec("BLOCK_SPARSE_VARIABLE"), UNSUPPORTED), (MaskSpec("FLASHMASK"), UNSUPPORTED),
]


@pytest.mark.parametrize("over,code", BAD_CACHE, ids=str)
def test_bad_cache_refused(L, over, code):
    assert size(L, shape(), cache(**over))[0] == code
    assert attn(L, shape(), cache(**over)) == code
    ca = cache(**over)
    assert L.lca_paged_write(FAKE, FAKE, 256, 256, FAKE, 4, C.byref(ca), None) == code


@pytest.mark.parametrize("over,code", BAD_SHAPE, ids=str)
def test_bad_shape_refused(L, over, code):
    assert size(L, shape(**over), cache())[0] == code
    assert attn(L, shape(**over), cache()) == code


@pytest.mark.parametrize("mask,code", BAD_MASK, ids=str)
def test_bad_mask_refused(L, mask, code):
    assert size(L, shape(), cache(), mask)[0] == code
    assert attn(L, shape(), cache(), mask) == code


def test_workspace(L):
    code, n = size(L, shape(), cache())
    assert code == 0 and n > 0 and n % 256 == 0
    assert size(L, shape(Tq=0, n_seq=0, max_pages=0, table_stride=0), cache(n_pages=0))[0] == 0
    assert attn(L, shape(), cache(), ws_bytes=n - 1) == WORKSPACE
    assert attn(L, shape(), cache(), ws=0x100010) == WORKSPACE
    assert attn(L, shape(), cache(), ws=None) == WORKSPACE
    assert L.lca_attn_paged_workspace_size(None, None, None, None) == INVALID


def test_workspace_size_grows_no_faster_than_the_batch(L):
    """A long context or a large batch does not need a workspace of its own size."""
    a = size(L, shape(Tq=1, n_seq=1), cache())[1]
    b = size(L, shape(Tq=1, n_seq=1, max_pages=1 << 20, table_stride=1 << 20), cache())[1]
    assert b == a
    assert size(L, shape(Tq=4096, n_seq=4096, Hq=64, q_stride=8192), cache(Hkv=8))[1] < 512 << 20


def plan(L, **kw):
    a = dict(ctx=FAKE, new=FAKE, n=2, free=FAKE, n_free=3, taken=FAKE, table=FAKE, stride=5, width=5, page=16, pages=9,
             rows=4, q_start=FAKE, k_len=FAKE, slots=FAKE, positions=FAKE, state=FAKE)
    a.update(kw)
    return L.lca_paged_plan(*a.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(n=-1), INVALID), (dict(n_free=-1), INVALID), (dict(width=-1), INVALID), (dict(page=0), INVALID),
    (dict(pages=-1), INVALID), (dict(rows=-1), INVALID), (dict(stride=4), INVALID),
    (dict(pages=1 << 28), UNSUPPORTED), (dict(width=1 << 28, stride=1 << 28), UNSUPPORTED),
    (dict(n=0x7FFFFFFF), UNSUPPORTED), (dict(ctx=None), INVALID), (dict(state=None), INVALID),
    (dict(slots=FAKE + 2), INVALID),
], ids=str)
def test_plan_refusals(L, over, code):
    assert plan(L, **over) == code


def test_unknown_memory_refused(L):
    """Pointers that CUDA does not know are refused, not read."""
    assert plan(L) == INVALID
    ca = cache()
    assert L.lca_paged_write(FAKE, FAKE, 256, 256, FAKE, 4, C.byref(ca), None) == INVALID
    assert L.lca_paged_write(FAKE, FAKE, 248, 256, FAKE, 4, C.byref(ca), None) == INVALID
    assert L.lca_paged_write(FAKE, FAKE, 256, 260, FAKE, 4, C.byref(ca), None) == INVALID
    assert L.lca_paged_write(FAKE, FAKE, 256, 256, FAKE, -1, C.byref(ca), None) == INVALID
    assert L.lca_paged_write(None, None, 256, 256, None, 0, C.byref(ca), None) == 0  # nothing to write


def test_binding_turns_away_unsuitable_tensors():
    bf = torch.bfloat16
    kc = torch.zeros(4, 16, 2, 128, dtype=bf)
    q, t = torch.zeros(3, 8, 128, dtype=bf), torch.zeros(2, 4, dtype=torch.int32)
    s = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        lib.attn_paged(q, kc, kc, t, s, s[:2], MaskSpec("CAUSAL"))
    with pytest.raises(ValueError, match="CUDA"):
        lib.paged_write(q[:, :2], q[:, :2], kc, kc, s)
    with pytest.raises(ValueError, match="CUDA"):
        lib.paged_plan(s, s, s, s[:1], t, 16, 4, 3)
    with pytest.raises(TypeError):
        lib.attn_paged(q, np.zeros((4, 16, 2, 128)), kc, t, s, s[:2], MaskSpec("CAUSAL"))
    with pytest.raises(TypeError):
        lib.paged_plan([1], s, s, s[:1], t, 16, 4, 3)
    # the checks themselves, on metadata alone
    meta = torch.device("meta")
    x = torch.empty(3, 8, 128, dtype=bf, device=meta)
    assert B._rows(x, "q", 8, 128, bf, meta) == 1024
    assert B._rows(torch.empty(3, 20, 128, dtype=bf, device=meta)[:, 8:16], "q", 8, 128, bf, meta) == 20 * 128
    for bad in (x.transpose(0, 1), x[:, ::2], x[..., :64], x[0]):
        with pytest.raises(ValueError):
            B._rows(bad, "q", None, 128, bf, meta)
    with pytest.raises(ValueError, match="dtype"):
        B._rows(x, "q", 8, 128, torch.float16, meta)
    tab = torch.empty(2, 9, dtype=torch.int32, device=meta)
    assert B._table(tab[:, :4], 2, meta)[1:] == (4, 9)
    for bad in (tab.t(), tab[:, ::2], tab.expand(2, 9)[:1].expand(2, 9), tab.long()):
        with pytest.raises(ValueError):
            B._table(bad, 2, meta)


@pytest.mark.parametrize("current", [0, 1])
def test_calls_run_on_the_tensors_device(monkeypatch, current):
    """The library is called with the tensors' device current and that
    device's stream, whichever device the caller had selected."""
    log = []
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 1000 + i, raising=False)

    class On:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            log.append(("enter", self.device.index))

        def __exit__(self, *a):
            log.append(("exit", self.device.index))

    monkeypatch.setattr(torch.cuda, "device", On)

    def fn(*args):
        log.append(args)
        return 0

    B._call(fn, "f", torch.device("cuda", 1), None, 5, 6)
    assert log == ([(5, 6, 1001)] if current == 1 else [("enter", 1), (5, 6, 1001), ("exit", 1)])
    with pytest.raises(lib.LcaError, match="INVALID"):
        B._call(lambda *a: 1, "f", torch.device("cuda", 1), None)


def test_workspace_sizes_of_shapes_that_need_no_tiles_of_many_rows(L):
    """One new token per request, a group too wide for a tile, no pages, or
    pages closer together than their tokens: no room for sums of many rows."""
    many = size(L, shape(Tq=40), cache())[1]
    few = size(L, shape(Tq=40, max_q_len=1), cache())[1]
    assert few < many
    assert size(L, shape(Tq=40, Hq=512, q_stride=512 * 128), cache())[1] == few
    assert size(L, shape(Tq=40), cache(n_pages=0))[1] == few
    assert size(L, shape(Tq=40), cache(page_stride=128, token_stride=4096))[1] == few
    assert size(L, shape(Tq=40), cache(n_pages=1, page_stride=128, token_stride=4096))[1] == many


@pytest.mark.parametrize("over", [dict(page_stride=1 << 38, n_pages=1 << 20), dict(token_stride=1 << 38, page_size=1 << 20),
                                  dict(head_stride=1 << 38, Hkv=1 << 20)], ids=str)
def test_a_cache_longer_than_any_memory_is_refused(L, over):
    """Its last byte's address does not fit 64 bits, nor do the checks for overlaps."""
    ca = cache(**over)
    assert size(L, shape(Hq=ca.Hkv, q_stride=ca.Hkv * 128), ca)[0] == INVALID
    assert size(L, shape(Hq=8), cache(page_stride=1 << 38, n_pages=3))[0] == 0  # long, but possible


@pytest.mark.parametrize("over,code", [
    (dict(n_seq=4, table_stride=1 << 62), INVALID), (dict(n_seq=1 << 20, table_stride=1 << 40), INVALID),
    (dict(Tq=1 << 20, q_stride=1 << 38), INVALID), (dict(scale=3e38), INVALID), (dict(n_seq=1 << 30), UNSUPPORTED),
    (dict(n_seq=0x7FFFFFFF), UNSUPPORTED), (dict(n_seq=1, table_stride=1 << 62), 0),
], ids=str)
def test_shapes_past_64_bits_are_refused(L, over, code):
    assert size(L, shape(**over), cache())[0] == code


@pytest.mark.parametrize("over,code", [
    (dict(stride=1 << 62, n=4), INVALID), (dict(stride=1 << 40, n=1 << 20), INVALID), (dict(n=1 << 30), UNSUPPORTED),
    (dict(n=0x7FFFFC10), UNSUPPORTED),
], ids=str)
def test_plans_past_64_bits_are_refused(L, over, code):
    assert plan(L, **over) == code


def test_numbers_past_32_bits_are_not_cut(monkeypatch):
    """ctypes would keep the low 32 bits: a page size of 2^32 + 16 as one of 16."""
    s, t = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 4, dtype=torch.int32)
    monkeypatch.setattr(B, "_ptr", lambda *a: FAKE)
    called = []
    monkeypatch.setattr(B, "_call", lambda *a: called.append(a))
    monkeypatch.setattr(B, "_side_stream", lambda *a: None)
    outs = dict(q_start=s, k_len=s, slots=s, positions=s, state=s)
    for page, pages, rows, name in (((1 << 32) + 16, 4, 3, "page_size"), (16, (1 << 32) + 4, 3, "n_pages"),
                                    (16, 4, (1 << 32) + 3, "n_rows"), (-(1 << 32) + 16, 4, 3, "page_size")):
        with pytest.raises(ValueError, match=name):
            lib.paged_plan(s, s, s, s[:1], t, page, pages, rows, **outs)
    assert not called
    lib.paged_plan(s, s, s, s[:1], t, 16, 4, 3, **outs)
    assert len(called) == 1


@pytest.mark.parametrize("kind", ["SLIDING", "CAUSAL_SLIDING", "GLOBAL_SLIDING", "PREFIX_LM_CAUSAL", "CAUSAL_BLOCKWISE"])
@pytest.mark.parametrize("value", [1 << 31, 1 << 32, (1 << 40) + 16, -(1 << 32) + 16])
def test_distances_past_32_bits_are_refused(kind, value):
    """A window of 2^32 meant as no limit would be one of 0, a block of 2^32 + 16 one of 16."""
    for name in ("window_left", "window_right", "num_global", "prefix_len", "block"):
        with pytest.raises(ValueError, match=name):
            B._paged_mask(MaskSpec(kind, **{name: value}))
        assert getattr(B._paged_mask(MaskSpec(kind, **{name: 0x7FFFFFFF})), name) == 0x7FFFFFFF


def test_tensors_past_32_bits_are_refused():
    meta = torch.device("meta")
    with pytest.raises(ValueError, match="kind"):
        B._paged_mask(MaskSpec((1 << 32) + 1))  # CAUSAL is 1
    with pytest.raises(ValueError, match="entries"):
        B._table(torch.empty(1, (1 << 32) + 4, dtype=torch.int32, device=meta), 1, meta)
    s, long = torch.empty(1, dtype=torch.int32, device=meta), torch.empty((1 << 32) + 1, dtype=torch.int32, device=meta)
    t = torch.empty(1, 4, dtype=torch.int32, device=meta)
    for args in ((long, s, s), (s, s, long)):
        with pytest.raises(ValueError, match="entries"):
            lib.paged_plan(*args, s, t, 16, 4, 3)


def test_a_longest_request_past_32_bits_is_refused():
    meta = torch.device("meta")
    q = torch.empty(3, 8, 128, dtype=torch.bfloat16, device=meta)
    kc = torch.empty(4, 16, 2, 128, dtype=torch.bfloat16, device=meta)
    table = torch.empty(2, 4, dtype=torch.int32, device=meta)

    def shape(max_q_len):
        return B._paged_shape(q, cache(), kc, table, 0.0, max_q_len)[0].max_q_len

    assert shape(3) == 3
    for n in (1 << 31, (1 << 32) + 1, -(1 << 32)):
        with pytest.raises(ValueError, match="max_q_len"):
            shape(n)
