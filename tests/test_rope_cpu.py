"""Rotary positions without a GPU: tables of frequencies against their formulas,
and refusals, all of which come before any launch (the pointers are made up)."""
from __future__ import annotations

import ctypes as C
import math
import os

import numpy as np
import pytest
import torch

import long_context_masked_attention_gb300 as lib
from long_context_masked_attention_gb300 import binding as B

INVALID, UNSUPPORTED = 1, 2
FAKE = 0x100000


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.LIB_PATH):
        lib.build()
    return lib.load()


# A frequency is a power, a blend of it and its quotient, in doubles: pow is off by
# at most 2^-50 of its result with an exponent of at most 1, each of the other
# steps by 2^-53.
FREQ_TOL = 2.0 ** -48


@pytest.mark.parametrize("rot", [2, 4, 20, 64, 96, 128])
@pytest.mark.parametrize("base", [10000.0, 500000.0, 1.5])
def test_plain_linear_and_ntk(L, rot, base):
    i = np.arange(rot // 2, dtype=np.float64)
    w = np.array([math.exp(-2 * k / rot * math.log(base)) for k in i])
    tol = 2.0 ** -47  # exp of a logarithm of up to 14: 14 2^-53 more
    f = lib.rope_frequencies(rot, base)
    assert f.inv_freq.shape == (rot // 2,) and f.scale == 1.0
    np.testing.assert_allclose(f.inv_freq, w, rtol=tol)
    np.testing.assert_allclose(lib.rope_frequencies(rot, base, "LINEAR", factor=8).inv_freq, w / 8, rtol=tol)
    assert np.array_equal(lib.rope_frequencies(rot, base, "LINEAR").inv_freq, f.inv_freq)
    if rot > 2:
        g = lib.rope_frequencies(rot, base, "NTK", factor=4.0).inv_freq
        np.testing.assert_allclose(g[0], 1.0, rtol=tol)  # the fastest pair keeps its frequency
        np.testing.assert_allclose(g[-1], w[-1] / 4, rtol=2 * tol)  # the slowest is stretched by the factor


@pytest.mark.parametrize("kind,kw", [("YARN", dict(fast=32.0, slow=1.0)), ("YARN", dict(fast=8.0, slow=0.5)),
                                     ("BANDS", dict(fast=4.0, slow=1.0)), ("BANDS", dict(fast=64.0, slow=2.0))])
@pytest.mark.parametrize("rot,base,L0,factor", [(128, 10000.0, 4096, 16.0), (64, 500000.0, 8192, 8.0), (96, 1e6, 100, 2.5),
                                                (32, 10000.0, 1, 3.0)])
def test_blended_tables(L, kind, kw, rot, base, L0, factor):
    f = lib.rope_frequencies(rot, base, kind, factor, L0, **kw)
    low = rot * math.log(L0 / (kw["fast"] * 2 * math.pi)) / (2 * math.log(base))
    high = rot * math.log(L0 / (kw["slow"] * 2 * math.pi)) / (2 * math.log(base))
    for i in range(rot // 2):
        w = base ** (-2 * i / rot)
        if kind == "YARN":
            a, b = max(math.floor(low), 0), min(math.ceil(high), rot - 1)
            stretch = min(max((i - a) / max(b - a, 1e-3), 0.0), 1.0)
        else:
            turns = L0 * w / (2 * math.pi)
            stretch = 1 - min(max((turns - kw["slow"]) / (kw["fast"] - kw["slow"]), 0.0), 1.0)
        want = w * (1 - stretch) + w / factor * stretch
        assert abs(f.inv_freq[i] - want) <= 2.0 ** -45 * w, i
        assert w / factor * (1 - 2.0 ** -45) <= f.inv_freq[i] <= w * (1 + 2.0 ** -45)
    assert f.scale == np.float32(0.1 * math.log(factor) + 1 if kind == "YARN" else 1.0)
    one = lib.rope_frequencies(rot, base, kind, 1.0, L0, **kw)
    assert one.scale == 1.0
    np.testing.assert_allclose(one.inv_freq, lib.rope_frequencies(rot, base).inv_freq, rtol=FREQ_TOL)


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=130), dict(rot_dim=-2), dict(base=1.0), dict(base=float("nan")),
    dict(base=float("inf")), dict(factor=0.5), dict(factor=float("nan")), dict(scaling=5), dict(scaling=-1),
    dict(scaling="YARN"), dict(scaling="BANDS", original_len=-1), dict(scaling="YARN", original_len=100, slow=0.0),
    dict(scaling="BANDS", original_len=100, fast=1.0, slow=1.0), dict(scaling="YARN", original_len=100, fast=float("inf")),
    dict(scaling="NTK", rot_dim=2, factor=2.0), dict(scaling="NTK", rot_dim=4, base=1e300, factor=1e10),
], ids=str)
def test_bad_tables_are_refused(L, kw):
    with pytest.raises(lib.LcaError, match="INVALID"):
        lib.rope_frequencies(**kw)


def rows(**kw):
    r = dict(x=FAKE, y=FAKE + 0x100000, heads=4, x_stride=512, y_stride=512)
    r.update(kw)
    return B.RopeRows_t(*r.values())


def call(L, q=None, k=None, positions=FAKE + 0x800000, n_rows=8, d=128, dtype=0, inv=(1.0, 0.5), rot=None, scale=1.0, null=False):
    arr = np.array(inv, dtype=np.float64)
    desc = B.RopeDesc_t(rot if rot is not None else 2 * arr.size, 0, None if null else arr.ctypes.data, scale)
    ref = [C.byref(x) if x is not None else None for x in (q, k)]
    return L.lca_rope(*ref, positions, n_rows, d, dtype, C.byref(desc), 0, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n_rows=-1), INVALID), (dict(d=64), UNSUPPORTED), (dict(dtype=2), INVALID), (dict(rot=3), INVALID),
    (dict(rot=0), INVALID), (dict(rot=130), INVALID), (dict(null=True), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(inv=(1.0, -0.1)), INVALID),
    (dict(inv=(float("nan"), 1.0)), INVALID), (dict(inv=(1.0, 2.0 ** 21)), INVALID), (dict(inv=(float("inf"),)), INVALID),
    (dict(q=rows(heads=-1)), INVALID), (dict(q=rows(x_stride=504)), INVALID), (dict(q=rows(y_stride=516)), INVALID),
    (dict(q=rows(x_stride=1 << 39)), INVALID), (dict(k=rows(x_stride=1 << 38), n_rows=1 << 30), INVALID),
    (dict(q=rows(heads=1 << 24, x_stride=1 << 31, y_stride=1 << 31)), UNSUPPORTED),
    (dict(q=rows(heads=1 << 29, x_stride=1 << 36, y_stride=1 << 36), k=rows(heads=1 << 29, x_stride=1 << 36, y_stride=1 << 36)), UNSUPPORTED),
    # pointers that CUDA does not know, misaligned ones, none
    (dict(), INVALID), (dict(q=rows(x=FAKE + 8)), INVALID), (dict(q=rows(y=None)), INVALID), (dict(positions=None), INVALID),
], ids=str)
def test_bad_calls_are_refused_before_anything_runs(L, kw, code):
    kw = {"q": rows(), **kw}
    before = L.lca_launch_count()
    assert call(L, **kw) == code
    assert L.lca_launch_count() == before


def test_no_rows_and_no_heads_are_nothing_to_do(L):
    assert call(L, q=rows(), n_rows=0) == 0
    assert call(L) == 0
    assert call(L, q=rows(heads=0, x=None, y=None)) == 0


def test_the_binding_turns_away_what_it_cannot_pass(L):
    f = lib.RopeFreqs(np.ones(64))
    q, pos = torch.zeros(3, 4, 128, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        lib.rope(q, None, pos, f)
    for x in (None, 5):
        with pytest.raises(TypeError):
            lib.rope(x, x, pos, f)
    meta = torch.device("meta")
    with pytest.raises(ValueError, match="CUDA"):
        lib.rope(None, q.to(meta), pos.to(meta), f)
