"""Pins of the fp64 definition of head norm + rotary positions, the frequency
helper, and the entry points' host-side refusals (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

from chunked_block_self_b200 import nle
from oracle import rope


def _freq(rot, base=10000.0):
    return base ** (-2.0 * np.arange(rot // 2) / rot)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [16, 64])
def test_rotation_is_relative_and_keeps_length(inter, rot):
    """<R(m) q, R(n) k> depends on m - n only; a rotation keeps the norm;
    position 0 is the identity; elements past rot_dim never move."""
    rng = np.random.default_rng(3)
    q, k = rng.standard_normal((2, 64))
    f = _freq(rot)
    a = rope.rotation(7, f, inter) @ q @ (rope.rotation(3, f, inter) @ k)
    b = rope.rotation(104, f, inter) @ q @ (rope.rotation(100, f, inter) @ k)
    assert abs(a - b) < 1e-11
    y = rope.rotation(55, f, inter) @ q
    assert abs(np.linalg.norm(y) - np.linalg.norm(q)) < 1e-12
    assert np.array_equal(y[rot:], q[rot:])
    assert np.array_equal(rope.rotation(0, f, inter), np.eye(64))


def test_rotation_closed_form():
    """One pair turned by a quarter: (1, 0) becomes (0, 1), in both layouts."""
    f = np.array([np.pi / 2] + [0.0] * 7)
    x = np.zeros((1, 1, 64))
    x[0, 0, 0] = 1.0
    y = rope.norm_rope(x, None, [1], f)
    assert abs(y[0, 0, 8] - 1.0) < 1e-15 and abs(y[0, 0, 0]) < 1e-15
    y = rope.norm_rope(x, None, [1], f, interleaved=True)
    assert abs(y[0, 0, 1] - 1.0) < 1e-15 and abs(y[0, 0, 0]) < 1e-15


@pytest.mark.parametrize("inter,scale,norm", [(False, 1.0, True), (True, 1.25, True), (False, 1.1, False)])
def test_gradient_against_differences(inter, scale, norm):
    """dx and dw against central differences of sum(y * dy).  The difference
    quotient's truncation error is of order h^2 and its rounding error of order
    1e-16 / h: with h = 1e-5 both stay below 1e-8 for values of order 1."""
    rng = np.random.default_rng(11)
    x, dy = rng.standard_normal((2, 3, 2, 64))
    w = 1.0 + 0.3 * rng.standard_normal(64) if norm else None
    f, pos, h = _freq(32), [0, 5, 1000], 1e-5
    run = lambda xx, ww: (rope.norm_rope(xx, ww, pos, f, 1e-3, inter, scale) * dy).sum()   # noqa: E731
    dx, dw, _ = rope.norm_rope_bwd(dy, x, w, pos, f, 1e-3, inter, scale)
    for i in [(0, 0, 0), (1, 1, 17), (2, 0, 31), (2, 1, 63)]:
        e = np.zeros_like(x)
        e[i] = h
        assert abs((run(x + e, w) - run(x - e, w)) / (2 * h) - dx[i]) < 1e-7
    if norm:
        for i in (0, 16, 40, 63):
            e = np.zeros(64)
            e[i] = h
            assert abs((run(x, w + e) - run(x, w - e)) / (2 * h) - dw[i]) < 1e-7


def test_inv_freq_plain_and_stretched():
    f, s = nle.rope_inv_freq(32, 10000.0, device="cpu")
    assert f.dtype == torch.float64 and s == 1.0
    np.testing.assert_allclose(f.numpy(), _freq(32), rtol=1e-15)
    g, _ = nle.rope_inv_freq(32, 10000.0, device="cpu", linear=4.0)
    np.testing.assert_allclose(g.numpy(), _freq(32) / 4, rtol=1e-15)
    g, _ = nle.rope_inv_freq(32, 10000.0, device="cpu", ntk=8.0)
    assert g[0] == 1.0
    np.testing.assert_allclose(g[-1].item(), f[-1].item() / 8, rtol=1e-12)   # the lowest frequency, stretched by 8
    g, s = nle.rope_inv_freq(64, 10000.0, device="cpu", yarn=4.0, yarn_frames=2048)
    ref = _freq(64)
    assert g[0].item() == ref[0]
    np.testing.assert_allclose(g[-1].item(), ref[-1] / 4, rtol=1e-15)
    ratio = g.numpy() / ref
    assert (np.diff(ratio) <= 1e-15).all() and abs(s - (0.1 * np.log(4.0) + 1.0)) < 1e-15
    # frequencies on either side of the ramp turn more / fewer times than the two limits
    turns = 2048 * ref / (2 * np.pi)
    assert (turns[ratio < 0.2501] < 1.5).all() and (turns[ratio > 0.9999] > 20).all()


@pytest.mark.parametrize("kw", [dict(rot_dim=3), dict(rot_dim=0), dict(base=1.0), dict(linear=0.5),
                                dict(linear=2.0, ntk=2.0), dict(yarn=2.0), dict(yarn=2.0, yarn_frames=100,
                                                                             yarn_beta=(1.0, 2.0))])
def test_inv_freq_refusals(kw):
    with pytest.raises(ValueError):
        nle.rope_inv_freq(device="cpu", **kw)


def _plan(**kw):
    a = dict(cu_seqlens=16, positions=None, q_weight=16, k_weight=16, inv_freq=16, dev_status=None, total_frames=400,
             n_seq=1, q_heads=8, k_heads=8, d_head=64, rot_dim=64, interleaved=0, eps=1e-6, rot_scale=1.0)
    a.update(kw)
    return nle.RopePlan(*[a[n] for n, _ in nle.RopePlan._fields_])


def _fwd(plan=None, q=16, k=16, qo=16, ko=16, qs=0, ks=0, **kw):
    p = _plan(**kw) if plan is None else plan
    return nle._lib.nle_qk_norm_rope_fwd(ctypes.byref(p), q, qs, k, ks, qo, 0, ko, 0, None)


def _bwd(dq=16, dk=16, q=16, k=16, oq=16, ok=16, work=16, qs=0, **kw):
    p = _plan(**kw)
    return nle._lib.nle_qk_norm_rope_bwd(ctypes.byref(p), dq, 0, dk, 0, q, qs, k, 0, oq, 0, ok, 0, None, None, work,
                                         None)


@pytest.mark.parametrize("f", [_fwd, _bwd])
def test_host_refusals(f):
    inv, uns, mis = nle.NLE_ERR_INVALID_ARG, nle.NLE_ERR_UNSUPPORTED, nle.NLE_ERR_MISALIGNED
    for kw, want in [(dict(d_head=128), uns), (dict(rot_dim=72), uns), (dict(rot_dim=24), uns), (dict(rot_dim=-16), inv),
                     (dict(n_seq=-1), inv), (dict(total_frames=-1), inv), (dict(total_frames=1 << 31), uns),
                     (dict(q_heads=-1), inv), (dict(q_heads=0, k_heads=0), inv), (dict(eps=-1.0), inv),
                     (dict(eps=float("nan")), inv), (dict(interleaved=2), inv), (dict(inv_freq=None), inv),
                     (dict(cu_seqlens=None), inv), (dict(q_weight=None), inv), (dict(k_weight=None), inv),
                     (dict(q_weight=8), mis), (dict(q=None), inv), (dict(k=None), inv), (dict(q=8), mis),
                     (dict(qs=8 * 64 - 8), inv), (dict(qs=8 * 64 + 4), mis), (dict(qs=1 << 41), inv),
                     (dict(cu_seqlens=18), mis), (dict(positions=18), mis), (dict(inv_freq=20), mis)]:
        assert f(**kw) == want, kw
    # nothing to do: no pointer is looked at
    assert f(n_seq=0, q=None) == nle.NLE_OK
    if f is _fwd:
        assert f(total_frames=0, q=None) == nle.NLE_OK
        assert f(qo=None) == inv and f(ko=24) == mis
        assert f(qs=9 * 64) == inv   # in place with another stride
        assert nle._lib.nle_qk_norm_rope_fwd(None, 16, 0, 16, 0, 16, 0, 16, 0, None) == inv
    else:
        assert f(dq=None) == inv and f(oq=None) == inv and f(work=None) == inv and f(work=24) == mis


def test_binding_refusals():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(TypeError):
        nle.qk_norm_rope(x, x, cu, None)
    with pytest.raises(ValueError):
        nle.qk_norm_rope(None, None, cu, None)
    with pytest.raises(ValueError):
        nle.qk_norm_rope_bwd(None, None, cu, None)


_NAMES = ("q", "k", "q_weight", "k_weight", "inv_freq", "cu_seqlens", "positions", "dev_status")
_FWD_OUT = ("q_out", "k_out")
_BWD_OUT = ("dq_out", "dk_out", "dq", "dk", "dq_weight", "dk_weight", "workspace")   # and the gradients read


def _distinct(outputs, **kw):
    """A call's buffers at addresses of their own (plan fields among them)."""
    a = {n: 4096 * (i + 1) for i, n in enumerate(_NAMES + outputs)}
    a.update(kw)
    return a, _plan(**{n: a[n] for n in _NAMES[2:]})


def _fwd_at(**kw):
    a, p = _distinct(_FWD_OUT, **kw)
    return nle._lib.nle_qk_norm_rope_fwd(ctypes.byref(p), a["q"], a.get("qs", 0), a["k"], 0, a["q_out"],
                                         a.get("qos", 0), a["k_out"], 0, None)


def _bwd_at(**kw):
    a, p = _distinct(_BWD_OUT, **kw)
    return nle._lib.nle_qk_norm_rope_bwd(ctypes.byref(p), a["dq_out"], 0, a["dk_out"], 0, a["q"], a.get("qs", 0),
                                         a["k"], 0, a["dq"], a.get("qos", 0), a["dk"], 0, a["dq_weight"],
                                         a["dk_weight"], a["workspace"], None)


@pytest.mark.parametrize("f,written,own", [
    (_fwd_at, ("q_out", "k_out"), {("q_out", "q"), ("k_out", "k")}),
    (_bwd_at, ("dq", "dk", "dq_weight", "dk_weight", "workspace"),
     {("dq", "dq_out"), ("dq", "q"), ("dk", "dk_out"), ("dk", "k")})])
def test_outputs_that_begin_at_another_buffer(f, written, own):
    """Refused wherever an output begins at another output or at any buffer that
    is read, but its own tensor's source at the same stride; without them the
    call gets as far as the device (no status of the argument checks)."""
    checks = (nle.NLE_ERR_INVALID_ARG, nle.NLE_ERR_MISALIGNED)
    a, _ = _distinct(_FWD_OUT if f is _fwd_at else _BWD_OUT)
    if not torch.cuda.is_available():   # with a device a good call would launch on these addresses
        assert f() not in checks
        for n, m in own:
            assert f(**{n: a[m]}) not in checks, (n, m)
    for n in written:
        for m in a:
            if m != n and (n, m) not in own:
                assert f(**{n: a[m]}) == nle.NLE_ERR_INVALID_ARG, (n, m)
    # its own source, frames apart by another stride
    n, m = ("q_out", "q") if f is _fwd_at else ("dq", "q")
    assert f(**{n: a[m], "qs": 9 * 64}) == nle.NLE_ERR_INVALID_ARG
    assert f(**{n: a[m], "qos": 9 * 64}) == nle.NLE_ERR_INVALID_ARG


@pytest.mark.parametrize("f,names", [(_fwd_at, ("dev_status",)), (_bwd_at, ("dq_weight", "dk_weight", "dev_status"))])
def test_pointers_off_their_alignment(f, names):
    for n in names:
        assert f(**{n: (1 << 20) + 2}) == nle.NLE_ERR_MISALIGNED, n
