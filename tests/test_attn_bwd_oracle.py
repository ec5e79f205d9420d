"""Pins of the fp64 attention gradient (against the C oracle's forward and
central differences), and the host-side refusals of the training entry points
(no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from chunked_block_self_b200 import nle
from chunked_block_self_b200 import workloads as wl
from oracle import attn_bwd


def _np(t):
    return t.float().double().numpy()


def test_segments():
    assert attn_bwd.segments([0, 5, 5, 12], 4) == [(0, 4), (4, 1), (5, 4), (9, 3)]
    assert attn_bwd.segments([2, 5, 5, 12]) == [(2, 3), (5, 7)]


@pytest.mark.parametrize("block", [0, 7])
def test_forward_matches_the_c_oracle(block):
    x = wl.block_inputs(lengths=[9, 0, 21, 1], heads=2, seed=3)
    segs = attn_bwd.segments(x["cu"], block)
    out, lse = attn_bwd.forward(_np(x["q"]), _np(x["k"]), _np(x["v"]), segs)
    ref = oracle.block_attn(x["q"], x["k"], x["v"], x["cu"], block_frames=block or 64)
    np.testing.assert_allclose(out, ref, atol=1e-13)
    # lse: probabilities of a row sum to one
    a, n = segs[-2]
    s = np.einsum("id,jd->ij", _np(x["q"])[a:a + n, 1], _np(x["k"])[a:a + n, 1]) / 8
    np.testing.assert_allclose(np.exp(s - lse[1, a:a + n, None]).sum(-1), 1.0, atol=1e-13)


@pytest.mark.parametrize("block,scale", [(0, 0.125), (5, 0.3)])
def test_gradient_against_differences(block, scale):
    """Central differences of sum(out * dout) with h = 1e-5: truncation of
    order h^2 and rounding of order 1e-16 / h, both below 1e-8 for values of
    order 1."""
    rng = np.random.default_rng(5)
    q, k, v, dout = rng.standard_normal((4, 14, 2, 64))
    segs = attn_bwd.segments([0, 6, 14], block)
    out, _ = attn_bwd.forward(q, k, v, segs, scale)
    grads = attn_bwd.backward(dout, q, k, v, out, segs, scale)
    h = 1e-5
    for which in range(3):
        for i in [(0, 0, 0), (5, 1, 63), (7, 0, 31), (13, 1, 5)]:
            args = [q.copy(), k.copy(), v.copy()]
            args[which][i] += h
            up = (attn_bwd.forward(*args, segs, scale)[0] * dout).sum()
            args[which][i] -= 2 * h
            dn = (attn_bwd.forward(*args, segs, scale)[0] * dout).sum()
            assert abs((up - dn) / (2 * h) - grads[which][i]) < 1e-7


def test_gradient_closed_forms():
    """One frame alone: dV = dout, dQ = dK = 0.  Equal keys: P = 1/n, so
    dV is the mean of dout over the segment and dQ = 0."""
    rng = np.random.default_rng(6)
    q, k, v, dout = rng.standard_normal((4, 1, 1, 64))
    dq, dk, dv = attn_bwd.backward(dout, q, k, v, v, [(0, 1)])
    assert np.abs(dq).max() < 1e-13 and np.abs(dk).max() < 1e-13 and np.array_equal(dv, dout)
    q, k, v, dout = rng.standard_normal((4, 6, 1, 64))
    k[:] = k[0]
    out, _ = attn_bwd.forward(q, k, v, [(0, 6)])
    dq, _, dv = attn_bwd.backward(dout, q, k, v, out, [(0, 6)])
    assert np.abs(dq).max() < 1e-13
    np.testing.assert_allclose(dv, np.broadcast_to(dout.mean(0, keepdims=True), dv.shape), atol=1e-14)


# ------------------------------------------------------------------ refusals
def _args(**kw):
    a = dict(q=16, k=16, v=16, out=16, dout=16, lse=16, dq=16, dk=16, dv=16, cu_seqlens=16, workspace=16,
             dev_status=None, total_frames=400, row_stride_qkv=0, row_stride_dqkv=0, wait_limit_ns=0, n_seq=1, heads=8,
             d_head=64, flags=0, softmax_scale=0.0)
    a.update(kw)
    return nle.AttnBwdArgs(*[a[n] for n, _ in nle.AttnBwdArgs._fields_])


def _block(block=200, **kw):
    return nle._lib.nle_block_attn_bwd(ctypes.byref(_args(**kw)), block, None)


def _varlen(**kw):
    return nle._lib.nle_varlen_attn_bwd(ctypes.byref(_args(**kw)), None)


@pytest.mark.parametrize("f", [_block, _varlen])
def test_backward_host_refusals(f):
    inv, uns, mis = nle.NLE_ERR_INVALID_ARG, nle.NLE_ERR_UNSUPPORTED, nle.NLE_ERR_MISALIGNED
    for kw, want in [(dict(n_seq=-1), inv), (dict(total_frames=-1), inv), (dict(heads=0), inv), (dict(d_head=32), uns),
                     (dict(total_frames=1 << 31), uns), (dict(wait_limit_ns=-1), inv),
                     (dict(row_stride_qkv=8 * 64 - 8), inv), (dict(row_stride_qkv=8 * 64 + 4), mis),
                     (dict(row_stride_dqkv=8 * 64 - 8), inv), (dict(row_stride_dqkv=8 * 64 + 4), mis),
                     (dict(row_stride_qkv=1 << 39), inv), (dict(total_frames=2**31 - 1, heads=64), uns)]:
        assert f(**kw) == want, kw
    for n in ("q", "k", "v", "out", "dout", "dq", "dk", "dv", "lse", "cu_seqlens", "workspace"):
        assert f(**{n: None}) == inv, n
    for n in ("q", "k", "v", "out", "dout", "dq", "dk", "dv"):
        assert f(**{n: 24}) == mis, n
    for n in ("lse", "cu_seqlens", "workspace"):
        assert f(**{n: 18}) == mis, n
    assert f(n_seq=0, q=None) == nle.NLE_OK and f(total_frames=0, q=None) == nle.NLE_OK


@pytest.mark.parametrize("f", [_block, _varlen])
def test_outputs_that_begin_at_another_buffer(f):
    """Only outputs that begin at an input, at another output or at the
    workspace are refused; without them the call gets as far as the device."""
    names = ("q", "k", "v", "out", "dout", "lse", "cu_seqlens", "dq", "dk", "dv", "workspace")
    a = {n: 1024 * (i + 1) for i, n in enumerate(names)}
    for n in ("dq", "dk", "dv", "workspace"):
        for m in names:
            if m != n:
                assert f(**dict(a, **{n: a[m]})) == nle.NLE_ERR_INVALID_ARG, (n, m)


def test_block_and_forward_host_refusals():
    assert _block(0) == nle.NLE_ERR_INVALID_ARG and _block(-1) == nle.NLE_ERR_INVALID_ARG
    assert _block(257) == nle.NLE_ERR_UNSUPPORTED
    assert nle._lib.nle_block_attn_bwd(None, 200, None) == nle.NLE_ERR_INVALID_ARG
    assert nle._lib.nle_varlen_attn_bwd(None, None) == nle.NLE_ERR_INVALID_ARG
    f = nle._lib.nle_block_attn_fwd_lse
    assert f(16, 16, 16, 16, None, 16, 1, 400, 8, 64, 200, 0.0, 0, None, 0, 0, None) == nle.NLE_ERR_INVALID_ARG
    assert f(16, 16, 16, 16, 16, 16, 1, 400, 8, 32, 200, 0.0, 0, None, 0, 0, None) == nle.NLE_ERR_UNSUPPORTED
    assert f(16, 16, 16, 16, None, 16, 0, 400, 8, 64, 200, 0.0, 0, None, 0, 0, None) == nle.NLE_OK
    assert f(16, 16, 16, 16, 18, 16, 1, 400, 8, 64, 200, 0.0, 0, None, 0, 0, None) == nle.NLE_ERR_MISALIGNED
    f = nle._lib.nle_varlen_attn_fwd_lse
    assert f(16, 16, 16, 16, None, 16, 1, 400, 8, 64, 0.0, 0, None, 0, 0, None) == nle.NLE_ERR_INVALID_ARG
    assert f(16, 16, 16, 24, 16, 16, 1, 400, 8, 64, 0.0, 0, None, 0, 0, None) == nle.NLE_ERR_MISALIGNED
    assert f(16, 16, 16, 16, 18, 16, 1, 400, 8, 64, 0.0, 0, None, 0, 0, None) == nle.NLE_ERR_MISALIGNED


def test_binding_rejects_cpu_tensors():
    x = torch.zeros(4, 1, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    lse = torch.zeros(1, 4)
    for f in (nle.block_attn_lse, nle.varlen_attn_lse):
        with pytest.raises(TypeError):
            f(x, x, x, cu)
    for f in (nle.block_attn_bwd, nle.varlen_attn_bwd):
        with pytest.raises(TypeError):
            f(x, x, x, x, x, lse, cu)


def test_status_off_its_alignment():
    """dev_status is written by an atomic: 4-byte aligned, as the other small buffers."""
    a = {n: 1024 * (i + 1) for i, n in enumerate(("q", "k", "v", "out", "dout", "lse", "cu_seqlens", "dq", "dk", "dv",
                                                  "workspace"))}
    for f in (_block, _varlen):
        assert f(**a, dev_status=18) == nle.NLE_ERR_MISALIGNED
    f = nle._lib.nle_block_attn_fwd_lse
    assert f(16, 16, 16, 48, 64, 16, 1, 400, 8, 64, 200, 0.0, 0, 18, 0, 0, None) == nle.NLE_ERR_MISALIGNED
    f = nle._lib.nle_varlen_attn_fwd_lse
    assert f(16, 16, 16, 48, 64, 16, 1, 400, 8, 64, 0.0, 0, 18, 0, 0, None) == nle.NLE_ERR_MISALIGNED


def test_binding_names_missing_offsets():
    with pytest.raises(TypeError, match="cu_seqlens must be a CUDA tensor"):
        nle._n_seq(None, 0)


@pytest.mark.parametrize("block", [200, None])
def test_forward_outputs_that_begin_at_another_buffer(block):
    """The forwards that keep the log-sum-exp: out and lse begin at no input and not at each other."""
    names = ("q", "k", "v", "out", "lse", "cu_seqlens", "dev_status")

    def f(**kw):
        a = dict({n: 1024 * (i + 1) for i, n in enumerate(names)}, **kw)
        head = [a[n] for n in names[:6]] + [1, 400, 8, 64]
        tail = [0.0, 0, a["dev_status"], 0, 0, None]
        if block:
            return nle._lib.nle_block_attn_fwd_lse(*head, block, *tail)
        return nle._lib.nle_varlen_attn_fwd_lse(*head, *tail)

    for n in ("out", "lse"):
        for i, m in enumerate(names):
            if m != n:
                assert f(**{n: 1024 * (i + 1)}) == nle.NLE_ERR_INVALID_ARG, (n, m)
