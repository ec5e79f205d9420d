"""GPU parity of the training forms of block and full-utterance attention
(nle_*_fwd_lse, nle_*_bwd) against the fp64 definition.

Tolerances are elementwise bounds from the kernel's arithmetic
(oracle/attn_bwd.py): P and dS are each rounded once to bf16 (2^-8 of a term),
P's exponent carries the fp32 error of a 64-term product (64 * 2^-24 of the
sum of absolute products, below 2^-12 of P for the inputs here), D and delta
that of theirs, and the result is rounded once more (2^-8).  lse: the fp32
error of its largest scores, of a sum of T terms and of the logarithm."""
import numpy as np
import pytest
import torch

from chunked_block_self_b200 import workloads as wl
from oracle import attn_bwd, rope

pytestmark = pytest.mark.gpu


# (block length, 0: whole utterances; work split: 2 whole blocks on chip, 4 tiles)
MODES = [(0, 0), (200, 2), (200, 4), (70, 2), (70, 4)]


def _nle():
    from chunked_block_self_b200 import nle
    return nle


def _np(t):
    return t.detach().float().cpu().double().numpy()


def _inputs(lengths, heads, seed, factor=1.0, dev="cuda"):
    x = wl.block_inputs(lengths=lengths, heads=heads, seed=seed, factor=factor)
    x["dout"] = wl.bf16_normal(np.random.default_rng(seed + 1), (x["total"], heads, 64))
    for n in ("q", "k", "v", "dout"):
        x[n] = x[n].to(dev)
    x["cud"] = torch.from_numpy(x["cu"]).to(dev)
    return x


def _fwd(x, block, **kw):
    nle = _nle()
    if block:
        return nle.block_attn_lse(x["q"], x["k"], x["v"], x["cud"], block, **kw)
    return nle.varlen_attn_lse(x["q"], x["k"], x["v"], x["cud"], **kw)


def _bwd(x, block, out, lse, **kw):
    nle = _nle()
    if block:
        return nle.block_attn_bwd(x["dout"], x["q"], x["k"], x["v"], out, lse, x["cud"], block, **kw)
    return nle.varlen_attn_bwd(x["dout"], x["q"], x["k"], x["v"], out, lse, x["cud"], **kw)


def _check_lse(lse, x, segs, scale=0.125):
    q, k = _np(x["q"]), _np(x["k"])
    _, ref = attn_bwd.forward(q, k, np.zeros_like(q), segs, scale)
    covered = np.zeros(len(q), bool)
    longest = 1
    for a, n in segs:
        covered[a:a + n] = True
        longest = max(longest, n)
    big = np.sqrt((q[covered] ** 2).sum(-1).max() * (k[covered] ** 2).sum(-1).max()) * scale
    tol = 64 * 2.0 ** -24 * big + longest * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * np.abs(ref)
    err = np.abs(lse.cpu().double().numpy() - ref)
    assert (err[:, covered] <= tol[:, covered]).all(), err[:, covered].max()


def _check_grads(grads, x, out, segs, scale=0.125, rows=None):
    ref = attn_bwd.backward(_np(x["dout"]), _np(x["q"]), _np(x["k"]), _np(x["v"]), _np(out), segs, scale, bounds=True)
    for got, want, tol, name in zip(grads, ref[:3], ref[3:], ("dq", "dk", "dv")):
        got = _np(got)
        keep = slice(None) if rows is None else rows
        bad = ~(np.abs(got[keep] - want[keep]) <= tol[keep] + 1e-30)
        assert not bad.any(), (name, np.argwhere(bad)[:4], np.abs(got[keep] - want[keep])[bad][:4],
                               tol[keep][bad][:4], want[keep][bad][:4])


@pytest.mark.parametrize("flags", [2, 4])   # whole blocks, tiles
@pytest.mark.parametrize("block", [1, 2, 15, 16, 17, 48, 63, 64, 65, 97, 127, 128, 129, 143, 192, 200, 208, 255, 256])
def test_block_gradient(block, flags, cuda_device):
    """Block lengths around every tile and MMA granule; utterances of one frame,
    shorter than, equal to and just past whole blocks; both work splits."""
    lengths = [1, block, 2 * block + 1, 0, max(1, block - 1), 3 * block + block // 2]
    x = _inputs(lengths, 3, 100 + block)
    out, lse = _fwd(x, block)
    segs = attn_bwd.segments(x["cu"], block)
    _check_lse(lse, x, segs)
    _check_grads(_bwd(x, block, out, lse, flags=flags), x, out, segs)


@pytest.mark.parametrize("lengths", [
    [1], [2], [15], [16], [17], [63], [64], [65], [127], [128], [129], [191], [192], [193], [255], [256], [257],
    [384], [385], [0, 5, 0, 333, 1, 0], [600, 1, 129, 256, 40],
])
def test_full_gradient(lengths, cuda_device):
    x = _inputs(lengths, 3, 7 + sum(lengths))
    out, lse = _fwd(x, 0)
    segs = attn_bwd.segments(x["cu"])
    _check_lse(lse, x, segs)
    _check_grads(_bwd(x, 0, out, lse), x, out, segs)


def test_long_utterances_full_gradient(cuda_device):
    x = _inputs([2011, 700, 3], 2, 91)
    out, lse = _fwd(x, 0)
    segs = attn_bwd.segments(x["cu"])
    _check_lse(lse, x, segs)
    _check_grads(_bwd(x, 0, out, lse), x, out, segs)


@pytest.mark.parametrize("block", [0, 200])
def test_forward_output_is_that_of_the_inference_form(block, cuda_device):
    nle = _nle()
    x = _inputs([700, 45, 1200], 4, 21)
    out, _ = _fwd(x, block)
    ref = nle.block_attn(x["q"], x["k"], x["v"], x["cud"], block) if block else \
        nle.varlen_attn(x["q"], x["k"], x["v"], x["cud"])
    assert torch.equal(out, ref)


@pytest.mark.parametrize("cfg,block", [(4, 200), (3, 0)])
def test_workload_gradients_sampled_segments(cfg, block, cuda_device):
    """The batch-128 and long-clip workloads at full size: whole (segment,
    head) pairs against the definition, everything finite, and the same bits
    on a second call."""
    x = wl.block_inputs(cfg)
    x["dout"] = wl.bf16_normal(np.random.default_rng(cfg), (x["total"], x["heads"], 64))
    for n in ("q", "k", "v", "dout"):
        x[n] = x[n].to(cuda_device)
    x["cud"] = torch.from_numpy(x["cu"]).to(cuda_device)
    out, lse = _fwd(x, block)
    grads = _bwd(x, block, out, lse)
    again = _bwd(x, block, out, lse)
    for a, b in zip(grads, again):
        assert torch.isfinite(a.float()).all() and torch.equal(a, b)
    segs = attn_bwd.segments(x["cu"], block)
    rng = np.random.default_rng(1)
    picks = [(segs[0], 0), (segs[-1], x["heads"] - 1)]
    picks += [(segs[int(i)], int(rng.integers(x["heads"]))) for i in rng.integers(0, len(segs), 30 if block else 2)]
    for (a, n), h in picks:
        y = {m: x[m][a:a + n, h:h + 1] for m in ("q", "k", "v", "dout")}
        _check_grads([g[a:a + n, h:h + 1] for g in grads], y, out[a:a + n, h:h + 1], [(0, n)])


@pytest.mark.parametrize("block,flags", MODES)
def test_gradient_locality_bit_exact(block, flags, cuda_device):
    """Poisoning every frame outside utterance 1 (Inf and NaN in q, k, v, dout,
    out and lse of its neighbours) leaves its gradients bit for bit."""
    x = _inputs([300, 450, 77], 2, 92)
    out, lse = _fwd(x, block)
    ref = _bwd(x, block, out, lse, flags=flags)
    y = dict(x)
    for n in ("q", "k", "v", "dout"):
        y[n] = x[n].clone()
        y[n][:300] = float("inf") if n in "qv" else float("nan")
        y[n][750:] = float("nan") if n in "qv" else float("inf")
    out2, lse2 = out.clone(), lse.clone()
    out2[:300] = float("nan")
    out2[750:] = float("inf")
    lse2[:, :300] = float("nan")
    lse2[:, 750:] = -float("inf")
    got = _bwd(y, block, out2, lse2, flags=flags)
    for a, b in zip(got, ref):
        assert torch.equal(a[300:750], b[300:750])


@pytest.mark.parametrize("block,flags", MODES)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_extreme_scores(block, flags, sign, cuda_device):
    """Scores of about +-200 in every valid place: exp of the masked places'
    score 0 relative to the row would overflow (-200) or vanish (+200)."""
    x = _inputs([137, 350], 2, 33, factor=0.05)
    x["q"] = (x["q"].float() + 5.0).to(torch.bfloat16)
    x["k"] = (x["k"].float() + sign * 5.0).to(torch.bfloat16)
    out, lse = _fwd(x, block)
    segs = attn_bwd.segments(x["cu"], block)
    _check_lse(lse, x, segs)
    assert (lse.abs() > 150).all()
    ref = attn_bwd.backward(*(_np(x[n]) for n in ("dout", "q", "k", "v")), _np(out), segs, bounds=True,
                            # the exponent's error: 64 * 2^-24 * 200 of P, below 2^-10
                            rel=2.0 ** -8 + 2.0 ** -10)
    for got, want, tol in zip(_bwd(x, block, out, lse, flags=flags), ref[:3], ref[3:]):
        assert (np.abs(_np(got) - want) <= tol + 1e-30).all()


@pytest.mark.parametrize("block,flags", [(0, 0), (100, 4), (150, 2), (150, 4)])
def test_peaked_rows(block, flags, cuda_device):
    """A few keys dominate: probabilities near one and near zero."""
    x = _inputs([260, 333], 2, 34)
    k = x["k"].float()
    k[[5, 140, 141, 300, 590]] *= 6.0
    x["k"] = k.to(torch.bfloat16)
    out, lse = _fwd(x, block)
    segs = attn_bwd.segments(x["cu"], block)
    _check_lse(lse, x, segs)
    _check_grads(_bwd(x, block, out, lse, flags=flags), x, out, segs)


@pytest.mark.parametrize("block,flags", [(0, 0), (60, 4), (130, 2)])
def test_projection_buffer_views_and_scale(block, flags, cuda_device):
    """q, k, v inside one projection buffer, the gradients inside another, an
    explicit scale; rows of no utterance and the rest of the buffers stay."""
    x = _inputs([133, 45], 4, 95)
    t = 20 + 178 + 9
    buf = torch.full((t, 4, 4, 64), float("nan"), dtype=torch.bfloat16, device=cuda_device)
    for i, n in enumerate(("q", "k", "v")):
        buf[20:198, i] = x[n]
    dout = torch.full((t, 4, 64), float("nan"), dtype=torch.bfloat16, device=cuda_device)
    dout[20:198] = x["dout"]
    y = dict(q=buf[:, 0], k=buf[:, 1], v=buf[:, 2], dout=dout, cud=x["cud"] + 20)
    out, lse = _fwd(y, block, softmax_scale=0.3)
    grads = torch.full((t, 3, 5, 64), 7.0, dtype=torch.bfloat16, device=cuda_device)
    views = (grads[:, 0, :4], grads[:, 1, :4], grads[:, 2, :4])
    got = _bwd(y, block, out, lse, softmax_scale=0.3, grads=views, flags=flags)
    assert all(a is b for a, b in zip(got, views))
    segs = attn_bwd.segments(x["cu"], block)
    _check_grads([g[20:198] for g in got], x, out[20:198], segs, scale=0.3)
    assert (grads[:20] == 7).all() and (grads[198:] == 7).all() and (grads[:, :, 4] == 7).all()


@pytest.mark.parametrize("block,flags", MODES[:3])
def test_empty_and_invalid_offsets(block, flags, cuda_device):
    nle = _nle()
    x = _inputs([300, 100], 2, 96)
    out, lse = _fwd(x, block)
    for cu in (torch.zeros(3, dtype=torch.int32, device=cuda_device),
               torch.zeros(1, dtype=torch.int32, device=cuda_device)):
        grads = tuple(torch.full_like(x["q"], 5.0) for _ in range(3))
        _bwd(dict(x, cud=cu), block, out, lse, grads=grads, flags=flags)
        assert all((g == 5).all() for g in grads)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    grads = tuple(torch.full_like(x["q"], 5.0) for _ in range(3))
    bad = torch.tensor([0, 300, 900], dtype=torch.int32, device=cuda_device)   # beyond total
    _bwd(dict(x, cud=bad), block, out, lse, grads=grads, dev_status=status, flags=flags)
    assert int(status.item()) == nle.NLE_ERR_INVALID_ARG
    ref = _bwd(x, block, out, lse, flags=flags)
    for g, r in zip(grads, ref):
        assert torch.equal(g[:300], r[:300]) and (g[300:] == 5).all()
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=cuda_device)
    z = dict(q=e, k=e, v=e, dout=e, cud=torch.zeros(2, dtype=torch.int32, device=cuda_device))
    eo, el = _fwd(z, block)
    assert all(g.shape == (0, 2, 64) for g in _bwd(z, block, eo, el, flags=flags))


@pytest.mark.parametrize("block,flags", MODES[:3])
def test_timeout_path_reports_and_recovers(block, flags, cuda_device):
    nle = _nle()
    x = _inputs([600, 300], 2, 97)
    out, lse = _fwd(x, block)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    _bwd(x, block, out, lse, dev_status=status, flags=flags | nle.NLE_FLAG_TEST_SKIP_FIRST_LOAD,
         wait_limit_ns=2_000_000)
    torch.cuda.synchronize()
    assert int(status.item()) == nle.NLE_ERR_TIMEOUT
    _check_grads(_bwd(x, block, out, lse, flags=flags), x, out, attn_bwd.segments(x["cu"], block))


@pytest.mark.parametrize("block,flags", MODES[:3])
def test_streams_and_graphs(block, flags, cuda_device):
    """On a side stream; two captured graphs replayed in turn, each with its
    own scratch, on new values: the bits of plain calls."""
    x = _inputs([300, 741], 2, 98)
    out, lse = _fwd(x, block)
    ref = [g.clone() for g in _bwd(x, block, out, lse, flags=flags)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, l2 = _fwd(x, block, stream=side)
    got = _bwd(x, block, o2, l2, stream=side, flags=flags)
    side.synchronize()
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    graphs, held = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, l = _fwd(x, block)
            held.append(_bwd(x, block, o, l, flags=flags))
        graphs.append(g)
    x["v"].mul_(2)
    x["dout"].mul_(-0.5)
    out, lse = _fwd(x, block)
    want = [g.clone() for g in _bwd(x, block, out, lse, flags=flags)]
    for i in (0, 1, 0):
        graphs[i].replay()
    torch.cuda.synchronize()
    for h in held:
        assert all(torch.equal(a, b) for a, b in zip(h, want))


@pytest.mark.parametrize("seed", range(6))
def test_random_batches(seed, cuda_device):
    """Random batches and block lengths (many items a CTA, one-frame blocks next
    to full ones): every gradient against the definition, both splits."""
    rng = np.random.default_rng(1000 + seed)
    block = int(rng.integers(1, 257)) if seed % 2 else int(rng.integers(129, 257))
    lengths = rng.integers(0, 3 * block, 90)
    x = _inputs(lengths, 4, 2000 + seed)
    out, lse = _fwd(x, block)
    segs = attn_bwd.segments(x["cu"], block)
    _check_grads(_bwd(x, block, out, lse, flags=2), x, out, segs)
    _check_grads(_bwd(x, block, out, lse, flags=4), x, out, segs)


def test_random_utterances(cuda_device):
    """Many short utterances: items of one tile, so that one elementwise stream
    of a CTA often has none."""
    x = _inputs(np.random.default_rng(5).integers(0, 150, 120), 5, 3000)
    out, lse = _fwd(x, 0)
    _check_grads(_bwd(x, 0, out, lse), x, out, attn_bwd.segments(x["cu"]))


@pytest.mark.parametrize("block,flags", [(0, 0), (150, 2), (150, 4)])
def test_offsets_past_32_bits(block, flags, cuda_device):
    """Frames so far apart that element offsets pass 2^31 and byte offsets
    2^32: the bits of the dense call (2.2e9 elements of bf16, 4.4 GB a buffer)."""
    x = _inputs([300, 33], 2, 77)
    out, lse = _fwd(x, block)
    ref = _bwd(x, block, out, lse, flags=flags)
    stride = 6_600_000
    wide = torch.empty(333 * stride, dtype=torch.bfloat16, device=cuda_device)
    grads = torch.empty(333 * stride, dtype=torch.bfloat16, device=cuda_device)
    views = [wide.as_strided((333, 2, 64), (stride, 64, 1), i * 128) for i in range(3)]
    for v, n in zip(views, "qkv"):
        v.copy_(x[n])
    gviews = [grads.as_strided((333, 2, 64), (stride, 64, 1), i * 128) for i in range(3)]
    y = dict(x, q=views[0], k=views[1], v=views[2])
    o2, l2 = _fwd(y, block)
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    got = _bwd(y, block, o2, l2, grads=gviews, flags=flags)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_two_calls_at_once(cuda_device):
    """Two gradients on two streams, interleaved: each has its own scratch."""
    x, y = _inputs([900, 411], 3, 78), _inputs([511, 77, 640], 3, 79)
    fx, fy = _fwd(x, 0), _fwd(y, 200)
    rx, ry = _bwd(x, 0, *fx), _bwd(y, 200, *fy)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        gx = _bwd(x, 0, *fx, stream=s1)
        gy = _bwd(y, 200, *fy, stream=s2)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(gx + gy, rx + ry))


def test_refused_tensors(cuda_device):
    nle = _nle()
    x = _inputs([50], 2, 99)
    out, lse = _fwd(x, 0)
    one = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device=cuda_device)
    with pytest.raises(ValueError):       # an expanded gradient
        nle.varlen_attn_bwd(one.expand(50, 2, 64), x["q"], x["k"], x["v"], out, lse, x["cud"])
    with pytest.raises(ValueError):       # expanded keys
        nle.varlen_attn_lse(x["q"], one.expand(50, 2, 64), x["v"], x["cud"])
    with pytest.raises(ValueError):
        nle.varlen_attn_bwd(x["dout"], x["q"], x["k"], x["v"], out, lse[:, :-1], x["cud"])
    with pytest.raises(TypeError):
        nle.varlen_attn_bwd(x["dout"].float(), x["q"], x["k"], x["v"], out, lse, x["cud"])
    with pytest.raises(ValueError):
        nle.varlen_attn_lse(x["q"].transpose(1, 2), x["k"], x["v"], x["cud"])
    with pytest.raises(nle.NLEError):
        nle.block_attn_bwd(x["dout"], x["q"], x["k"], x["v"], out, lse, x["cud"], 257)


@pytest.mark.parametrize("block", [0, 50])
def test_layer_chain_forward_and_gradient(block, cuda_device):
    """As a layer trains: head norm + rotation, attention, and back.  Every
    intermediate is rounded to bf16 (q', k', out, dq', dk': 2^-8 each at most,
    spread over sums), so against one fp64 chain without roundings each result
    stays within 2 % in relative L2 norm (five roundings, each at most 2^-8)."""
    nle = _nle()
    lengths, heads = [160, 1, 75], 3
    x = _inputs(lengths, heads, 55)
    rng = np.random.default_rng(2)
    wq, wk = (torch.from_numpy(1 + 0.2 * rng.standard_normal(64)).to(torch.bfloat16) for _ in range(2))
    f, _ = nle.rope_inv_freq(64, 10000.0, device=cuda_device)
    dq_w, dk_w = wq.to(cuda_device), wk.to(cuda_device)
    qr, kr = nle.qk_norm_rope(x["q"], x["k"], x["cud"], f, dq_w, dk_w)
    y = dict(x, q=qr, k=kr)
    out, lse = _fwd(y, block)
    dqr, dkr, dv = _bwd(y, block, out, lse)
    dq, dk, gwq, gwk = nle.qk_norm_rope_bwd(dqr, dkr, x["cud"], f, x["q"], x["k"], dq_w, dk_w)
    pos, fr = rope.positions(x["cu"]), f.cpu().numpy()
    q64, k64, v64, do64 = (_np(x[n]) for n in ("q", "k", "v", "dout"))
    rq, rk = rope.norm_rope(q64, _np(wq), pos, fr), rope.norm_rope(k64, _np(wk), pos, fr)
    segs = attn_bwd.segments(x["cu"], block)
    o64, _ = attn_bwd.forward(rq, rk, v64, segs)
    g = attn_bwd.backward(do64, rq, rk, v64, o64, segs)
    rdq, rwq, _ = rope.norm_rope_bwd(g[0], q64, _np(wq), pos, fr)
    rdk, rwk, _ = rope.norm_rope_bwd(g[1], k64, _np(wk), pos, fr)
    for got, want in ((out, o64), (dq, rdq), (dk, rdk), (dv, g[2]), (gwq, rwq), (gwk, rwk)):
        assert np.linalg.norm(_np(got) - want) <= 5 * 2.0 ** -8 * np.linalg.norm(want)


@pytest.mark.parametrize("f", ["block_attn", "varlen_attn"])
def test_missing_tensors_are_named(f, cuda_device):
    nle = _nle()
    x = _inputs([30], 2, 98)
    fwd, bwd = getattr(nle, f + "_lse"), getattr(nle, f + "_bwd")
    out, lse = fwd(x["q"], x["k"], x["v"], x["cud"])
    with pytest.raises(TypeError, match="cu_seqlens"):
        fwd(x["q"], x["k"], x["v"], None)
    args = dict(dout=x["dout"], q=x["q"], k=x["k"], v=x["v"], out=out, lse=lse, cu_seqlens=x["cud"])
    for n in args:
        with pytest.raises(TypeError, match=n):
            bwd(**dict(args, **{n: None}))
