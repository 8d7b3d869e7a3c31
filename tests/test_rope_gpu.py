"""Rotary positions on the GPU against their formula in 64 bits, forward and back."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
from gen import MaskSpec, Segment
from tests.paged_util import make

pytestmark = pytest.mark.gpu


def formula(x, positions, inv, scale, interleaved, back):
    """The turned rows in doubles, angles in the longest floats there are (a position of 2^31 costs a double 2^-22),
    and what a kernel's values may be off: with u the half step of the type and a, b a pair's magnitudes,
      u |y|                    its own rounding
      (|a| + |b|) scale 5e-7   cos and sin: the angle's fraction of half a turn is one fp32 rounding off (2^-25 pi, and
                               2 pi 2^-32 for what is cut), they are one step off (2^-23), their product with scale
                               half a step, and so are the two roundings of a pair's sum
      2^-25                    fp16's smallest numbers."""
    import torch

    inv = np.asarray(inv, dtype=np.longdouble)
    turn = np.longdouble("6.283185307179586476925286766559005768")
    angle = np.fmod(np.asarray(positions, dtype=np.longdouble)[:, None] * inv, turn).astype(np.float64)
    cos, sin = (scale * f(angle)[:, None] for f in (np.cos, np.sin))
    if back:
        sin = -sin
    h = len(inv)
    y = x.double().cpu().numpy()
    at = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    a, b = y[..., at[0]], y[..., at[1]]
    out, tol = y.copy(), np.zeros_like(y)
    out[..., at[0]], out[..., at[1]] = a * cos - b * sin, b * cos + a * sin
    u = torch.finfo(x.dtype).eps / 2
    for s in at:
        tol[..., s] = u * np.abs(out[..., s]) + (np.abs(a) + np.abs(b)) * scale * 5e-7 * (1 + u) + 2.0 ** -25
    return out, tol


def check(got, x, positions, f, interleaved, back, what=""):
    out, tol = formula(x, positions, f.inv_freq, f.scale, interleaved, back)
    assert got.dtype == x.dtype and got.shape == x.shape
    off = np.abs(got.double().cpu().numpy() - out) - tol
    assert off.max(initial=-1) <= 0, f"{what}: off by {off.max():.3g} past its bound at {np.unravel_index(off.argmax(), off.shape)}"


def inputs(T, Hq, Hkv, dtype, seed=0, far=4096):
    import torch

    g = torch.Generator().manual_seed(seed)
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    q, k = (torch.randn(T, h, 128, generator=g).to(dt).cuda() for h in (Hq, Hkv))
    pos = torch.randint(0, far, (T,), generator=g).to(torch.int32)
    return q, k, pos


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [128, 64, 32, 16, 96, 40, 24, 20, 12, 6, 2, 126])
def test_layouts_and_parts_of_the_head(lca, rot, interleaved, dtype):
    """Units of 8, 4, 2 and 1 values; what does not turn is copied bit for bit."""
    import torch

    q, k, pos = inputs(37, 6, 2, dtype, seed=rot)
    k[3, 1, 100:] = float("nan")  # not a number, and copied where it does not turn
    f = lca.rope_frequencies(rot, 500.0)
    for back, turn in ((False, lca.rope), (True, lca.rope_bwd)):
        a, b = turn(q, k, pos.cuda(), f, interleaved=interleaved)
        check(a, q, pos, f, interleaved, back, "q")
        keep = torch.ones(37, dtype=torch.bool)
        keep[3] = False
        check(b[keep], k[keep], pos[keep], f, interleaved, back, "k")
        assert torch.equal(a[..., rot:].view(torch.int16), q[..., rot:].view(torch.int16))
        assert torch.equal(b[..., rot:].view(torch.int16), k[..., rot:].view(torch.int16))


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (1, 64, 8), (2, 7, 7), (3, 5, 0), (5, 0, 3), (64, 64, 8), (4097, 8, 1), (700, 33, 11),
                                      (20000, 1, 1), (0, 4, 2)])
def test_sizes(lca, T, Hq, Hkv):
    q, k, pos = inputs(T, Hq, Hkv, "bf16", seed=T)
    f = lca.rope_frequencies()
    a, b = lca.rope(q if Hq else None, k if Hkv else None, pos.cuda(), f)
    for got, x in ((a, q), (b, k)):
        if x.shape[1]:
            check(got, x, pos, f, False, False)
        else:
            assert got is None


@pytest.mark.parametrize("back", [False, True])
def test_far_positions_keep_their_angles(lca, back):
    """Up to 2^31 - 1 and down to -2^31, with frequencies up to 2^20; scaled tables; a factor of the values."""
    import torch

    edge = [0, 1, -1, 524287, 524288, (1 << 20) + 1, (1 << 24) + 1, (1 << 31) - 1, -(1 << 31), 123456789, -7654321]
    q, k, _ = inputs(len(edge), 3, 2, "fp16", seed=5)
    pos = torch.tensor(edge, dtype=torch.int32)
    for f in (lca.rope_frequencies(), lca.rope_frequencies(128, 5e5, "YARN", 40.0, 4096), lca.rope_frequencies(64, 1e6, "BANDS", 8.0, 8192),
              lca.RopeFreqs(np.linspace(0, 3.0, 64), 0.37), lca.RopeFreqs(np.array([2.0 ** 20, 1048575.3, np.pi, 2 * np.pi, 0.0]))):
        a, b = (lca.rope_bwd if back else lca.rope)(q, k, pos.cuda(), f)
        check(a, q, pos, f, False, back)
        check(b, k, pos, f, False, back)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [128, 64, 20])
def test_rows_of_a_projection_and_in_place(lca, rot, interleaved):
    """q and k as parts of wider rows, turned into rows of another width and in place; what lies beside them stays."""
    import torch

    T, Hq, Hkv = 50, 6, 2
    g = torch.Generator().manual_seed(rot)
    wide = torch.randn(T, Hq + 2 * Hkv + 1, 128, generator=g).to(torch.bfloat16).cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 3
    f = lca.rope_frequencies(rot)
    q, k = wide[:, 1:1 + Hq], wide[:, 1 + Hq:1 + Hq + Hkv]
    a, b = lca.rope(q, k, pos, f, interleaved=interleaved)
    check(a, q, pos.cpu(), f, interleaved, False)
    check(b, k, pos.cpu(), f, interleaved, False)
    to = torch.full((T, Hq + Hkv + 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    x, y = lca.rope(q, k, pos, f, interleaved=interleaved, q_out=to[:, 1:1 + Hq], k_out=to[:, 1 + Hq:-1])
    assert torch.equal(x, a) and torch.equal(y, b) and bool((to[:, 0] == 7).all()) and bool((to[:, -1] == 7).all())
    before = wide.clone()
    x, y = lca.rope(q, k, pos, f, interleaved=interleaved, q_out=q, k_out=k)
    assert x is q and torch.equal(q, a) and torch.equal(k, b)
    assert torch.equal(wide[:, 0], before[:, 0]) and torch.equal(wide[:, 1 + Hq + Hkv:], before[:, 1 + Hq + Hkv:])
    x, _ = lca.rope(before[:, :Hq], None, pos, f, interleaved=interleaved)
    check(x, before[:, :Hq], pos.cpu(), f, interleaved, False)


def test_overlaps_and_other_tensors_are_refused(lca):
    import torch

    q, k, pos = inputs(8, 4, 2, "bf16")
    pos, f = pos.cuda(), lca.rope_frequencies()
    flat = torch.zeros(1 << 16, dtype=torch.bfloat16, device="cuda")
    at = lambda o, h, s=None: flat[o:].as_strided((8, h, 128), (s or h * 128, 128, 1))  # noqa: E731
    for kw in (dict(q=at(0, 4), q_out=at(128, 4)), dict(q=at(0, 4), k=at(1024, 2)  , q_out=at(2048, 4)), dict(q=at(0, 4), k=k, k_out=at(512, 2), q_out=at(0, 4)),
               dict(q=at(0, 4, 1024), q_out=at(0, 4, 512)), dict(q=at(0, 4, 768), k=at(384, 2, 768), q_out=at(0, 4, 768)),
               dict(q=q, q_out=at(0, 4), k=k, k_out=at(4000, 2))):
        with pytest.raises(lca.LcaError, match="INVALID"):
            lca.rope(kw.pop("q"), kw.pop("k", None), pos, f, **kw)
    inside = flat[:4096].view(torch.int32)[:8]
    with pytest.raises(lca.LcaError, match="INVALID"):
        lca.rope(q, None, inside, f, q_out=at(0, 4))
    assert not bool(flat.any())
    for bad in (dict(q=q.float()), dict(q=q[..., :64]), dict(q=q[:7]), dict(k=k.half()), dict(k=k.cpu()), dict(k=k.transpose(1, 2)),
                dict(q_out=q[:, :3]), dict(q_out=q.half()), dict(k=None, k_out=k)):
        args = dict(dict(q=q, k=k), **bad)
        with pytest.raises((ValueError, TypeError)):
            lca.rope(args.pop("q"), args.pop("k"), pos, f, **args)
    for bad in (pos.long(), pos[:5], pos.cpu(), torch.stack([pos, pos], 1)[:, 0]):
        with pytest.raises(ValueError, match="positions"):
            lca.rope(q, k, bad, f)
    for bad in (np.ones((2, 32)),):
        with pytest.raises(ValueError, match="inv_freq"):
            lca.rope(q, k, pos, lca.RopeFreqs(bad))
    for bad in (np.ones(65), np.ones(0), -np.ones(3)):
        with pytest.raises(lca.LcaError, match="INVALID"):
            lca.rope(q, k, pos, lca.RopeFreqs(bad))


def test_the_way_back_is_the_gradient(lca):
    """f(x) = sum g rope(x) is linear, so its difference in a direction d is sum d rope_bwd(g), whatever the step; the
    sums of both sides in doubles, each off by the bounds of its values."""
    import torch

    g = torch.Generator().manual_seed(2)
    for rot, inter in ((128, False), (64, True), (20, False)):
        f = lca.rope_frequencies(rot, 1000.0, "YARN", 4.0, 512)
        x, grad, d = (torch.randn(40, 3, 128, generator=g).to(torch.float16).cuda() for _ in range(3))
        pos = torch.randint(0, 9000, (40,), generator=g).to(torch.int32)
        dx = lca.rope_bwd(grad, None, pos.cuda(), f, interleaved=inter)[0]
        hi, lo = (x.double() + 2 * d.double()).half(), (x.double() - 2 * d.double()).half()  # the step that was taken
        step = (hi.double() - lo.double())
        y1, y0 = (lca.rope(t, None, pos.cuda(), f, interleaved=inter)[0] for t in (hi, lo))
        left = float((grad.double() * (y1.double() - y0.double())).sum())
        right = float((step * dx.double()).sum())
        tol = 0.0
        for t, w in ((hi, grad), (lo, grad)):
            tol += float((formula(t, pos, f.inv_freq, f.scale, inter, False)[1] * w.double().abs().cpu().numpy()).sum())
        tol += float((formula(grad, pos, f.inv_freq, f.scale, inter, True)[1] * step.abs().cpu().numpy()).sum())
        assert abs(left - right) <= tol and abs(right) > 0


def test_scores_depend_on_distances(lca):
    """q at p + s and k at p' + s have the product that they have at p and p'."""
    import torch

    q, k, _ = inputs(1, 4, 4, "fp16", seed=7)
    f = lca.rope_frequencies()
    want = None
    for s in (0, 1000, 500000):
        a = lca.rope(q, None, torch.tensor([17 + s], dtype=torch.int32, device="cuda"), f)[0]
        b = lca.rope(None, k, torch.tensor([5 + s], dtype=torch.int32, device="cuda"), f)[1]
        got = (a.double() * b.double()).sum(-1)
        want = got if want is None else want
        # 128 products, each factor rounded to 2^-11 of itself: |a b| 2^-10 a side, and 5e-7 of both for cos and sin
        tol = 2 * ((a.double() * b.double()).abs().sum(-1) * 2.0 ** -10 + a.double().norm(dim=-1) * b.double().norm(dim=-1) * 2e-6 + 1e-6)
        assert bool(((got - want).abs() <= tol).all())


def test_streams_and_a_captured_call(lca):
    """A call on another stream, and one captured and replayed with other rows and positions."""
    import torch

    q, k, pos = inputs(300, 8, 2, "bf16", seed=1)
    pos, f = pos.cuda(), lca.rope_frequencies(64)
    want = lca.rope(q, k, pos, f)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        got = lca.rope(q, k, pos, f, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = lca.rope(q, k, pos, f)
    for seed in (3, 4):
        a, b, p = inputs(300, 8, 2, "bf16", seed=seed)
        q.copy_(a), k.copy_(b), pos.copy_(p)
        graph.replay()
        want = lca.rope(q, k, pos, f)
        assert all(torch.equal(x, y) for x, y in zip(outs, want))


@pytest.mark.parametrize("rot,interleaved", [(128, False), (64, True)])
def test_a_training_step(lca, rot, interleaved):
    """rope, attention, its backward, and the gradients back through rope, against the fp64 oracle of all of it.
    With u = 2^-8 the rotated rows and their gradients are rounded once more than the oracle's; the bar is the one of the
    attention backward's own tests (2e-2 of the norm), and u more for each of the three roundings."""
    import torch

    segs = [Segment(0, 200, 0, 200), Segment(200, 77, 200, 77)]
    g = torch.Generator().manual_seed(4)
    q, do = (torch.randn(277, 4, 128, generator=g).to(torch.bfloat16) for _ in range(2))
    k, v = (torch.randn(277, 2, 128, generator=g).to(torch.bfloat16) for _ in range(2))
    pos = torch.cat([torch.arange(200), torch.arange(77)]).to(torch.int32)
    f = lca.rope_frequencies(rot)
    mask = MaskSpec("CAUSAL_DOC")
    qr, kr = lca.rope(q.cuda(), k.cuda(), pos.cuda(), f, interleaved=interleaved)
    o, lse = lca.attn_fwd(qr, kr, v.cuda(), segs, mask)
    dqr, dkr, dv = lca.attn_bwd(do.cuda(), qr, kr, v.cuda(), o, lse, segs, mask)
    dq, dk = lca.rope_bwd(dqr, dkr, pos.cuda(), f, interleaved=interleaved)
    p = make([(0, 1)], 16, 4, 2, mask)
    p.prob.Tq = p.prob.Tk = 277
    p.prob.segments = segs
    Q, K = (torch.from_numpy(formula(x, pos, f.inv_freq, f.scale, interleaved, False)[0]) for x in (q, k))
    dQ, dK, dV = oracle.attention_backward(p.prob, Q, K, v, do)
    want = [formula(torch.from_numpy(x), pos, f.inv_freq, f.scale, interleaved, True)[0] for x in (dQ, dK)] + [dV]
    for got, ref, name in zip((dq, dk, dv), want, ("dq", "dk", "dv")):
        rel = np.linalg.norm(got.double().cpu().numpy() - ref) / np.linalg.norm(ref)
        assert rel <= 2e-2 + 3 * 2.0 ** -8, (name, rel)
