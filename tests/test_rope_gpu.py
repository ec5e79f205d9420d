"""GPU parity of head norm + rotary positions and its gradient
(nle_qk_norm_rope_fwd / _bwd) against the fp64 definition.

Tolerances, derived: one rounding to bf16 of the value (2^-8 of it), plus fp32
arithmetic.  A forward value is a sum of two products of three fp32 factors,
each with a few roundings (r, cos, sin: at most 4 ulp each), so its fp32 error
is below 16 * 2^-24 (|z_a| + |z_b|) c.  A gradient is r (g - n m): below 64 *
2^-24 of r (|g| + |n| mean|g n|), where |g| counts both members of its pair.
A weight gradient adds N terms of relative error below 32 * 2^-24 each in fp32
chains of at most N additions: below (N + 32) 2^-24 sum|terms|."""
import numpy as np
import pytest
import torch

from chunked_block_self_b200 import workloads as wl
from oracle import rope

pytestmark = pytest.mark.gpu

EPS32 = 2.0 ** -24
BF16 = 2.0 ** -8


def _nle():
    from chunked_block_self_b200 import nle
    return nle


def _freq(rot, base=10000.0):
    return base ** (-2.0 * np.arange(rot // 2) / rot)


def _draw(lengths, qh, kh, seed, norm=True, factor=1.0):
    rng = np.random.default_rng(seed)
    t = int(np.sum(lengths))
    x = dict(cu=wl.cu_seqlens(lengths), t=t)
    for n, h in (("q", qh), ("k", kh), ("dq", qh), ("dk", kh)):
        x[n] = wl.bf16_normal(rng, (t, h, 64), factor)
    for n in ("wq", "wk"):
        x[n] = torch.from_numpy(1.0 + 0.3 * rng.standard_normal(64)).to(torch.bfloat16) if norm else None
    return x


def _np(t):
    return None if t is None else t.detach().float().cpu().double().numpy()


def _partner_abs(z, rot, inter):
    """|z_a| + |z_b| at both members of a pair, |z| elsewhere."""
    a = np.abs(z)
    out = a.copy()
    m = rot // 2
    i = np.arange(m)
    p, q = (2 * i, 2 * i + 1) if inter else (i, i + m)
    out[..., p] = out[..., q] = a[..., p] + a[..., q]
    return out


def _check_fwd(got, x, w, pos, f, eps=1e-6, inter=False, scale=1.0):
    ref = rope.norm_rope(_np(x), _np(w), pos, f, eps, inter, scale)
    z, _, _ = rope.norm(_np(x), _np(w), eps)
    tol = BF16 * np.abs(ref) + 16 * EPS32 * max(scale, 1.0) * _partner_abs(z, 2 * len(f), inter) * (1 + BF16) + 1e-38
    bad = ~(np.abs(_np(got) - ref) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:3], np.abs(_np(got) - ref)[bad][:3], tol[bad][:3])


def _check_bwd(got, got_dw, dy, x, w, pos, f, eps=1e-6, inter=False, scale=1.0):
    dx, dw, dz = rope.norm_rope_bwd(_np(dy), _np(x), _np(w), pos, f, eps, inter, scale)
    big = _partner_abs(_np(dy), 2 * len(f), inter) * max(scale, 1.0)   # bounds |dz| before cancellation
    if w is None:
        tol = BF16 * np.abs(dx) + 16 * EPS32 * big * (1 + BF16)
    else:
        _, n, r = rope.norm(_np(x), _np(w), eps)
        g = big * np.abs(_np(w))
        tol = BF16 * np.abs(dx) + 64 * EPS32 * r * (g + np.abs(n) * (g * np.abs(n)).mean(-1, keepdims=True)) * (1 + BF16)
        rows = dx.shape[0] * dx.shape[1]
        tol_w = (rows + 32) * EPS32 * (big * np.abs(n)).sum((0, 1))
        assert (np.abs(_np(got_dw) - dw) <= tol_w).all(), (np.abs(_np(got_dw) - dw) / tol_w).max()
    bad = ~(np.abs(_np(got) - dx) <= tol + 1e-38)
    assert not bad.any(), (np.argwhere(bad)[:3], np.abs(_np(got) - dx)[bad][:3], tol[bad][:3])


def _dev(x, dev):
    return {n: (torch.from_numpy(v) if isinstance(v, np.ndarray) else v).to(dev)
            if isinstance(v, (np.ndarray, torch.Tensor)) else v for n, v in x.items()}


CASES = [
    # lengths, q heads, k heads, rot, interleaved, norm, scale
    ([1], 1, 1, 64, False, True, 1.0),
    ([1, 1, 1], 3, 2, 64, True, True, 1.0),
    ([7], 8, 8, 64, False, False, 1.0),
    ([9, 0, 15, 0], 5, 1, 32, False, True, 1.5),
    ([31, 2, 33], 16, 4, 32, True, True, 1.0),
    ([40, 41], 17, 17, 48, False, True, 0.75),
    ([64, 3], 2, 33, 16, True, False, 1.25),
    ([100], 4, 0, 64, False, True, 1.0),
    ([100], 0, 4, 16, False, True, 1.0),
    ([50, 27], 6, 3, 0, False, True, 1.0),
]


@pytest.mark.parametrize("lengths,qh,kh,rot,inter,norm,scale", CASES)
def test_forward_and_gradient(lengths, qh, kh, rot, inter, norm, scale, cuda_device):
    nle = _nle()
    x = _draw(lengths, qh, kh, 17 + sum(lengths) + rot, norm)
    d = _dev(x, cuda_device)
    f = _freq(rot) if rot else np.zeros(0)
    ft = torch.from_numpy(f).to(cuda_device) if rot else None
    q, k, dq, dk = (d[n] if h else None for n, h in (("q", qh), ("k", kh), ("dq", qh), ("dk", kh)))
    wq, wk = (d["wq"] if qh else None), (d["wk"] if kh else None)
    qo, ko = nle.qk_norm_rope(q, k, d["cu"], ft, wq, wk, interleaved=inter, rot_scale=scale)
    gq, gk, gwq, gwk = nle.qk_norm_rope_bwd(dq, dk, d["cu"], ft, q, k, wq, wk, interleaved=inter, rot_scale=scale)
    pos = rope.positions(x["cu"])
    for y, g, gw, n, h in ((qo, gq, gwq, "q", qh), (ko, gk, gwk, "k", kh)):
        if h == 0:
            assert y is None and g is None and gw is None
            continue
        _check_fwd(y, x[n], x["w" + n], pos, f, inter=inter, scale=scale)
        _check_bwd(g, gw, x["d" + n], x[n], x["w" + n], pos, f, inter=inter, scale=scale)
        assert (gw is not None) == norm


@pytest.mark.parametrize("inter", [False, True])
def test_batch_large_enough_for_every_launch_form(inter, cuda_device):
    """More frames than eight per warp slot of the GPU, so the forward takes
    four frames per warp and the gradient's CTAs several units each."""
    nle = _nle()
    lengths = [4001, 1, 2999, 3500, 17]
    x = _draw(lengths, 2, 1, 5)
    d = _dev(x, cuda_device)
    f = _freq(64)
    ft = torch.from_numpy(f).to(cuda_device)
    qo, ko = nle.qk_norm_rope(d["q"], d["k"], d["cu"], ft, d["wq"], d["wk"], interleaved=inter)
    gq, gk, gwq, gwk = nle.qk_norm_rope_bwd(d["dq"], d["dk"], d["cu"], ft, d["q"], d["k"], d["wq"], d["wk"],
                                            interleaved=inter)
    pos = rope.positions(x["cu"])
    _check_fwd(qo, x["q"], x["wq"], pos, f, inter=inter)
    _check_fwd(ko, x["k"], x["wk"], pos, f, inter=inter)
    _check_bwd(gq, gwq, x["dq"], x["q"], x["wq"], pos, f, inter=inter)
    _check_bwd(gk, gwk, x["dk"], x["k"], x["wk"], pos, f, inter=inter)


def test_many_utterances(cuda_device):
    """More utterances than one step of the plan walk covers, many empty."""
    nle = _nle()
    rng = np.random.default_rng(8)
    lengths = rng.integers(0, 12, 700)
    x = _draw(lengths, 1, 1, 9)
    d = _dev(x, cuda_device)
    f = _freq(64)
    ft = torch.from_numpy(f).to(cuda_device)
    qo, _ = nle.qk_norm_rope(d["q"], d["k"], d["cu"], ft, d["wq"], d["wk"])
    gq, _, gwq, _ = nle.qk_norm_rope_bwd(d["dq"], d["dk"], d["cu"], ft, d["q"], d["k"], d["wq"], d["wk"])
    pos = rope.positions(x["cu"])
    _check_fwd(qo, x["q"], x["wq"], pos, f)
    _check_bwd(gq, gwq, x["dq"], x["q"], x["wq"], pos, f)


@pytest.mark.parametrize("with_cu", [False, True])
def test_explicit_far_positions(with_cu, cuda_device):
    """Positions up to 2^31 - 1 and negative: the angle is formed in fp64, so
    the only error left is that of the definition's own fp64 angle."""
    nle = _nle()
    x = _draw([23, 20], 3, 2, 6)
    d = _dev(x, cuda_device)
    f = _freq(64)
    rng = np.random.default_rng(2)
    pos = rng.integers(-(1 << 20), 1 << 20, 43)
    pos[:4] = [2**31 - 1, -2**31, 0, 180000]
    pt = torch.from_numpy(pos.astype(np.int32)).to(cuda_device)
    qo, ko = nle.qk_norm_rope(d["q"], d["k"], d["cu"] if with_cu else None, torch.from_numpy(f).to(cuda_device),
                              d["wq"], d["wk"], positions=pt)
    # |t| up to 2^31: the roundings of the two sides (1 / (2 pi), the frequency in turns and both products:
    # four of 2^-53 each) move the angle by up to 4 * 2^-53 * 2^31 = 2^-20
    for y, n in ((qo, "q"), (ko, "k")):
        ref = rope.norm_rope(_np(x[n]), _np(x["w" + n]), pos, f)
        z, _, _ = rope.norm(_np(x[n]), _np(x["w" + n]), 1e-6)
        tol = BF16 * np.abs(ref) + (16 * EPS32 + 2.0 ** -20) * _partner_abs(z, 64, False) * (1 + BF16)
        assert (np.abs(_np(y) - ref) <= tol).all()


def test_strided_views_in_place_and_rows_outside(cuda_device):
    """q and k inside one projection buffer with v; written in place; frames
    before the first and behind the last utterance, v and nothing else stay."""
    nle = _nle()
    rng = np.random.default_rng(4)
    t, qh, kh = 90, 4, 2
    buf = wl.bf16_normal(rng, (t, qh + 2 * kh, 64)).to(cuda_device)
    buf[70:] = float("nan")
    buf[:5] = float("inf")
    was = buf.clone()
    q, k = buf[:, :qh], buf[:, qh:qh + kh]
    cu = torch.tensor([5, 30, 70], dtype=torch.int32, device=cuda_device)
    w = torch.from_numpy(1 + 0.2 * rng.standard_normal((2, 64))).to(torch.bfloat16).to(cuda_device)
    f = _freq(32)
    ft = torch.from_numpy(f).to(cuda_device)
    fresh = nle.qk_norm_rope(q[5:70], k[5:70], cu - 5, ft, w[0], w[1])
    out = nle.qk_norm_rope(q, k, cu, ft, w[0], w[1], out=(q, k))
    assert out[0] is q
    assert torch.equal(q[5:70], fresh[0]) and torch.equal(k[5:70], fresh[1])
    assert torch.equal(buf[:, qh + kh:].view(torch.int16), was[:, qh + kh:].view(torch.int16))
    assert torch.equal(buf[70:].view(torch.int16), was[70:].view(torch.int16))
    assert torch.equal(buf[:5].view(torch.int16), was[:5].view(torch.int16))
    pos = rope.positions([0, 25, 65])
    _check_fwd(fresh[0], was[5:70, :qh], w[0], pos, f)
    # gradient, from views, in place over the incoming gradient
    g = wl.bf16_normal(rng, (t, qh + kh, 64)).to(cuda_device)
    g[70:] = float("nan")
    g0 = g.clone()
    dq, dk = g[:, :qh], g[:, qh:]
    _, _, dwq, dwk = nle.qk_norm_rope_bwd(dq, dk, cu, ft, was[:, :qh], was[:, qh:qh + kh], w[0], w[1], out=(dq, dk))
    _check_bwd(dq[5:70], dwq, g0[5:70, :qh], was[5:70, :qh], w[0], pos, f)
    _check_bwd(dk[5:70], dwk, g0[5:70, qh:], was[5:70, qh:qh + kh], w[1], pos, f)
    assert torch.equal(g[70:].view(torch.int16), g0[70:].view(torch.int16))


def test_unrotated_part_passes_infinities(cuda_device):
    """Without norm, elements past rot_dim are copied bit for bit: an infinity
    there stays one and reaches no other element."""
    nle = _nle()
    for inter in (False, True):
        x = _draw([6], 2, 1, 12, norm=False)
        x["q"][2, 1, 40] = float("inf")
        x["q"][3, 0, 41] = float("nan")
        d = _dev(x, cuda_device)
        qo, _ = nle.qk_norm_rope(d["q"], d["k"], d["cu"], torch.from_numpy(_freq(32)).to(cuda_device),
                                 interleaved=inter)
        assert torch.equal(qo[..., 32:].cpu().view(torch.int16), x["q"][..., 32:].contiguous().view(torch.int16))
        assert torch.isfinite(qo[..., :32].float()).all()


def test_zero_rows_and_eps(cuda_device):
    """An all-zero row has r = 1 / sqrt(eps): its output is zero and its
    gradient that of the formula."""
    nle = _nle()
    x = _draw([5], 2, 2, 13)
    x["q"][1] = 0
    d = _dev(x, cuda_device)
    f = _freq(64)
    ft = torch.from_numpy(f).to(cuda_device)
    qo, _ = nle.qk_norm_rope(d["q"], d["k"], d["cu"], ft, d["wq"], d["wk"], eps=1e-3)
    assert (qo[1] == 0).all()
    gq, _, gwq, _ = nle.qk_norm_rope_bwd(d["dq"], d["dk"], d["cu"], ft, d["q"], d["k"], d["wq"], d["wk"], eps=1e-3)
    pos = rope.positions(x["cu"])
    _check_fwd(qo, x["q"], x["wq"], pos, f, eps=1e-3)
    _check_bwd(gq, gwq, x["dq"], x["q"], x["wq"], pos, f, eps=1e-3)


def test_gradient_is_repeatable_and_empty_batches(cuda_device):
    nle = _nle()
    x = _draw([3000, 1234], 4, 4, 14)
    d = _dev(x, cuda_device)
    ft = torch.from_numpy(_freq(64)).to(cuda_device)
    runs = [nle.qk_norm_rope_bwd(d["dq"], d["dk"], d["cu"], ft, d["q"], d["k"], d["wq"], d["wk"]) for _ in range(3)]
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))
    # empty utterances only: nothing written, weight gradients are empty sums
    cu0 = torch.zeros(4, dtype=torch.int32, device=cuda_device)
    keep = (torch.full_like(d["q"], 3.0), torch.full_like(d["k"], 3.0))
    _, _, dwq, dwk = nle.qk_norm_rope_bwd(d["dq"], d["dk"], cu0, ft, d["q"], d["k"], d["wq"], d["wk"], out=keep)
    assert (dwq == 0).all() and (dwk == 0).all() and (keep[0] == 3).all()
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=cuda_device)
    qo, ko = nle.qk_norm_rope(e, e, cu0, ft, d["wq"], d["wk"])
    assert qo.shape == (0, 4, 64)
    _, _, dwq, _ = nle.qk_norm_rope_bwd(e, e, cu0, ft, e, e, d["wq"], d["wk"])
    assert (dwq == 0).all()


def test_invalid_offsets_are_skipped_and_reported(cuda_device):
    nle = _nle()
    x = _draw([40, 20], 2, 2, 15)
    d = _dev(x, cuda_device)
    ft = torch.from_numpy(_freq(64)).to(cuda_device)
    for bwd in (False, True):
        status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
        bad = torch.tensor([0, 40, 900], dtype=torch.int32, device=cuda_device)
        out = (torch.full_like(d["q"], 9.0), torch.full_like(d["k"], 9.0))
        if bwd:
            nle.qk_norm_rope_bwd(d["dq"], d["dk"], bad, ft, d["q"], d["k"], d["wq"], d["wk"], out=out,
                                 dev_status=status)
        else:
            nle.qk_norm_rope(d["q"], d["k"], bad, ft, d["wq"], d["wk"], out=out, dev_status=status)
        assert int(status.item()) == nle.NLE_ERR_INVALID_ARG
        assert (out[0][40:] == 9.0).all() and not (out[0][:40] == 9.0).all()


def test_other_stream_and_graph_replay(cuda_device):
    """On a side stream, and captured and replayed on new values, the results
    are those of a plain call, bit for bit."""
    nle = _nle()
    x = _draw([300, 41], 4, 2, 16)
    d = _dev(x, cuda_device)
    ft = torch.from_numpy(_freq(64)).to(cuda_device)

    def both():
        return (*nle.qk_norm_rope(d["q"], d["k"], d["cu"], ft, d["wq"], d["wk"]),
                *nle.qk_norm_rope_bwd(d["dq"], d["dk"], d["cu"], ft, d["q"], d["k"], d["wq"], d["wk"]))

    ref = [t.clone() for t in both()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (*nle.qk_norm_rope(d["q"], d["k"], d["cu"], ft, d["wq"], d["wk"], stream=side),
           *nle.qk_norm_rope_bwd(d["dq"], d["dk"], d["cu"], ft, d["q"], d["k"], d["wq"], d["wk"],
                                 stream=side.cuda_stream))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = both()
    d["q"].mul_(2), d["dk"].mul_(-1)
    want = [t.clone() for t in both()]
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, want))
    assert not torch.equal(want[0], ref[0]) or not torch.equal(want[3], ref[3])


def test_offsets_past_32_bits(cuda_device):
    """Frames so far apart that element offsets pass 2^31: the bits of the
    dense call, forward and gradient (2.2e9 elements of bf16, 4.4 GB)."""
    nle = _nle()
    x = _draw([300, 33], 2, 1, 21)
    d = _dev(x, cuda_device)
    ft = torch.from_numpy(_freq(64)).to(cuda_device)
    ref = (*nle.qk_norm_rope(d["q"], d["k"], d["cu"], ft, d["wq"], d["wk"]),
           *nle.qk_norm_rope_bwd(d["dq"], d["dk"], d["cu"], ft, d["q"], d["k"], d["wq"], d["wk"]))
    stride = 6_600_000
    wide = torch.empty(333 * stride, dtype=torch.bfloat16, device=cuda_device)
    q, k, dq, dk = (wide.as_strided((333, h, 64), (stride, 64, 1), o * 64) for h, o in ((2, 0), (1, 2), (2, 3), (1, 5)))
    for v, n in ((q, "q"), (k, "k"), (dq, "dq"), (dk, "dk")):
        v.copy_(d[n])
    _, _, gwq, gwk = nle.qk_norm_rope_bwd(dq, dk, d["cu"], ft, q, k, d["wq"], d["wk"], out=(dq, dk))
    nle.qk_norm_rope(q, k, d["cu"], ft, d["wq"], d["wk"], out=(q, k))
    assert all(torch.equal(a, b) for a, b in zip((q, k, dq, dk, gwq, gwk), ref))


def test_heads_beyond_one_batch(cuda_device):
    """More heads than a lane keeps in flight at once (16), not multiples of four."""
    nle = _nle()
    for inter in (False, True):
        x = _draw([11], 37, 21, 22)
        d = _dev(x, cuda_device)
        f = _freq(48)
        ft = torch.from_numpy(f).to(cuda_device)
        qo, ko = nle.qk_norm_rope(d["q"], d["k"], d["cu"], ft, d["wq"], d["wk"], interleaved=inter)
        gq, gk, gwq, gwk = nle.qk_norm_rope_bwd(d["dq"], d["dk"], d["cu"], ft, d["q"], d["k"], d["wq"], d["wk"],
                                                interleaved=inter)
        pos = rope.positions(x["cu"])
        _check_fwd(qo, x["q"], x["wq"], pos, f, inter=inter)
        _check_fwd(ko, x["k"], x["wk"], pos, f, inter=inter)
        _check_bwd(gq, gwq, x["dq"], x["q"], x["wq"], pos, f, inter=inter)
        _check_bwd(gk, gwk, x["dk"], x["k"], x["wk"], pos, f, inter=inter)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("heads", [1, 3, 5, 17])
def test_gradient_without_eps(heads, inter, cuda_device):
    """eps = 0 and head counts that are no multiples of four: a lane without a
    head has a zero row, whose r is infinite, and must add nothing to the
    weights' gradients."""
    nle = _nle()
    x = _draw([21, 2], heads, 2, 23 + heads)
    d = _dev(x, cuda_device)
    f = _freq(32)
    ft = torch.from_numpy(f).to(cuda_device)
    qo, ko = nle.qk_norm_rope(d["q"], d["k"], d["cu"], ft, d["wq"], d["wk"], eps=0.0, interleaved=inter)
    gq, gk, gwq, gwk = nle.qk_norm_rope_bwd(d["dq"], d["dk"], d["cu"], ft, d["q"], d["k"], d["wq"], d["wk"], eps=0.0,
                                            interleaved=inter)
    pos = rope.positions(x["cu"])
    for y, g, gw, n in ((qo, gq, gwq, "q"), (ko, gk, gwk, "k")):
        _check_fwd(y, x[n], x["w" + n], pos, f, eps=0.0, inter=inter)
        _check_bwd(g, gw, x["d" + n], x[n], x["w" + n], pos, f, eps=0.0, inter=inter)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [0, 16, 32, 48])
def test_norm_of_rows_with_infinities_past_the_rotation(rot, inter, cuda_device):
    """An infinity makes the row's r zero: the element itself becomes NaN
    (Inf * 0) and every other one zero, its neighbour too where pairs are
    neighbours.  A NaN among the weights past rot_dim reaches its own element
    of every row and no other."""
    nle = _nle()
    x = _draw([9], 2, 3, 31 + rot)
    x["q"][2, 1, 50] = float("inf")
    x["q"][3, 0, 51] = -float("inf")
    d = _dev(x, cuda_device)
    ft = torch.from_numpy(_freq(rot)).to(cuda_device) if rot else None
    bad = d["wk"].clone()
    bad[53] = float("nan")
    _, want = nle.qk_norm_rope(d["q"], d["k"], d["cu"], ft, d["wq"], d["wk"], interleaved=inter)
    qo, ko = nle.qk_norm_rope(d["q"], d["k"], d["cu"], ft, d["wq"], bad, interleaved=inter)
    for f, h, e in ((2, 1, 50), (3, 0, 51)):
        row = qo[f, h].clone()
        assert torch.isnan(row[e])
        row[e] = 0
        assert (row == 0).all(), torch.nonzero(row != 0).flatten().tolist()
    assert torch.isnan(ko[..., 53]).all()
    keep = [e for e in range(64) if e != 53]
    assert torch.equal(ko[..., keep], want[..., keep])


def test_gradient_over_its_inputs_and_refused_overlaps(cuda_device):
    """dq and dk may be written over q and k; an output that begins at another
    output or at the other tensor is refused."""
    nle = _nle()
    x = _draw([70, 13], 37, 3, 41)
    d = _dev(x, cuda_device)
    ft = torch.from_numpy(_freq(64)).to(cuda_device)
    rest = (d["cu"], ft)
    ref = nle.qk_norm_rope_bwd(d["dq"], d["dk"], *rest, d["q"], d["k"], d["wq"], d["wk"])
    q, k = d["q"].clone(), d["k"].clone()
    got = nle.qk_norm_rope_bwd(d["dq"], d["dk"], *rest, q, k, d["wq"], d["wk"], out=(q, k))
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    # three heads each, so that either tensor's shape fits
    a, b, c = d["k"], d["dk"], torch.empty_like(d["k"])
    for out in ((c, c), (b, c), (c, a), (b, a)):
        with pytest.raises(nle.NLEError):
            nle.qk_norm_rope(a, b, *rest, d["wq"], d["wk"], out=out)
    for out in ((c, c), (b, c), (c, a)):
        with pytest.raises(nle.NLEError):
            nle.qk_norm_rope_bwd(a, b, *rest, torch.empty_like(a), torch.empty_like(a), d["wq"], d["wk"], out=out)


def _check_dw(got, dy, x, w, pos, f, units, frames, heads, inter, dev):
    """The weights' gradient against the definition, under the bound of the
    kernel's own chain: a CTA's warp adds a frame of each of its units of 8
    frames, ceil(heads / 4) terms a lane, then 2 steps of a shuffle and the
    CTA's 8 warps in fp32 (the CTAs in fp64, rounded once); a term's own error
    is below 32 * 2^-24."""
    grid = min(frames // 8 + 5, 2 * torch.cuda.get_device_properties(dev).multi_processor_count, 2048)
    chain = -(-units // grid) * -(-heads // 4) + 2 + 8 + 1 + 32
    _, dw, _ = rope.norm_rope_bwd(_np(dy), _np(x), _np(w), pos, f, 1e-6, inter)
    _, n, _ = rope.norm(_np(x), _np(w), 1e-6)
    tol = chain * EPS32 * (1 + 2.0 ** -10) * (_partner_abs(_np(dy), 2 * len(f), inter) * np.abs(n)).sum((0, 1))
    assert (np.abs(_np(got) - dw) <= tol + 1e-38).all(), (np.abs(_np(got) - dw) / tol).max()


@pytest.mark.parametrize("inter", [False, True])
def test_weight_gradient_of_every_unit(inter, cuda_device):
    """A batch whose persistent CTAs take several units of frames each: dw
    under the bound of the kernel's chain, far below one frame's share; and with
    a gradient in one unit alone (of every round of the CTAs, and the last one,
    of one frame) dw is that unit's."""
    nle = _nle()
    lengths = [4001, 1, 2999, 3500, 17]
    x = _draw(lengths, 2, 1, 5)
    d = _dev(x, cuda_device)
    f = _freq(64)
    ft = torch.from_numpy(f).to(cuda_device)
    pos = rope.positions(x["cu"])
    starts = [(int(a) + s, min(8, int(b - a) - s)) for a, b in zip(x["cu"][:-1], x["cu"][1:]) for s in range(0, b - a, 8)]
    run = lambda dq, dk: nle.qk_norm_rope_bwd(dq, dk, d["cu"], ft, d["q"], d["k"], d["wq"], d["wk"],   # noqa: E731
                                              interleaved=inter)
    _, _, gwq, gwk = run(d["dq"], d["dk"])
    _check_dw(gwq, x["dq"], x["q"], x["wq"], pos, f, len(starts), x["t"], 2, inter, cuda_device)
    _check_dw(gwk, x["dk"], x["k"], x["wk"], pos, f, len(starts), x["t"], 1, inter, cuda_device)
    grid = 2 * torch.cuda.get_device_properties(cuda_device).multi_processor_count
    assert len(starts) > 2 * grid
    for u in [0, *range(7, len(starts), grid), 500, 501, len(starts) - 1]:
        a, n = starts[u]
        rows = slice(a, a + n)
        only = [torch.zeros_like(d[m]) for m in ("dq", "dk")]
        for o, m in zip(only, ("dq", "dk")):
            o[rows] = d[m][rows]
        gq, gk, gwq, gwk = run(*only)
        for g, gw, m, heads in ((gq, gwq, "q", 2), (gk, gwk, "k", 1)):
            _check_dw(gw, x["d" + m][rows], x[m][rows], x["w" + m], pos[rows], f, 1, 8, heads, inter, cuda_device)
            assert (gw != 0).all() and (g[rows] != 0).any()
            g[rows] = 0
            assert (g == 0).all()
