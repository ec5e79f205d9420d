"""Cases of the operators that train the attention layers.

Four operators over packed utterances (``cu`` offsets, rows = frames, heads of 64):

* ``rope``      per-head RMS norm of queries and keys (optional) and the rotary
                position rotation in one pass;
* ``rope_bwd``  its gradient: of q and k, and of the two norm weights;
* ``block_bwd`` gradient of block attention (every frame attends to its own block);
* ``full_bwd``  gradient of attention inside whole utterances.

``run`` computes an operator either in its plain form (elementary torch operations in
32 bits, positions' angles in 64) or, with ``own``, through the package's entry points.
Utterance lengths follow from a case alone; the values from the seed.
"""
import math
import random

import torch

own = False

D = 64            # head width of every attention operator of the package
ROPE_BASE = 10000.0


# ------------------------------------------------------------------ cases
def _case(name, op, n_seq, t_min, t_max, heads, **kw):
    c = {"name": name, "op": op, "n_seq": n_seq, "t_min": t_min, "t_max": t_max, "heads": heads, "len_seed": 7}
    if op.startswith("rope"):
        c.update(kv_heads=heads, rot_dim=64, interleaved=False, norm=True, far=0, stretch=1.0)
    if op == "block_bwd":
        c.update(block=200)
    c.update(fused=False)
    c.update(kw)
    return c


def listed():
    return [
        # one 8 s utterance: a single small call, all latency; rotation alone
        _case("rope one utterance", "rope", 1, 400, 400, 8, norm=False),
        # the batch-128 throughput setting: 2-16 s utterances
        _case("rope batch-128", "rope", 128, 100, 800, 16),
        # 39-94 s clips cut out of hour-long recordings (explicit far positions),
        # stretched frequencies, half of each head rotated, interleaved pairs
        _case("rope long clips far", "rope", 16, 1950, 4700, 16, rot_dim=32, interleaved=True, far=180000, stretch=4.0),
        # gradient of a single 16 s bucket
        _case("rope_bwd bucket", "rope_bwd", 1, 800, 800, 16),
        _case("rope_bwd batch-128", "rope_bwd", 128, 100, 800, 16),
        # grouped key heads out of one projection buffer, rotation alone
        _case("rope_bwd grouped", "rope_bwd", 16, 1950, 4700, 16, kv_heads=4, norm=False, interleaved=True, fused=True),
        # one 8 s utterance: two blocks, eight heads
        _case("block_bwd one utterance", "block_bwd", 1, 400, 400, 8),
        _case("block_bwd batch-128", "block_bwd", 128, 100, 800, 16),
        # short odd utterances in short odd blocks, operands inside one projection buffer
        _case("block_bwd ragged", "block_bwd", 37, 1, 333, 3, block=97, fused=True),
        # the 16 s bucket attended as a whole
        _case("full_bwd bucket", "full_bwd", 1, 800, 800, 16),
        _case("full_bwd ragged", "full_bwd", 40, 1, 701, 5, fused=True),
        # 39-94 s clips, full attention inside each
        _case("full_bwd long clips", "full_bwd", 16, 1950, 4700, 16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "block_bwd", "full_bwd"])
    heads = rng.randint(1, 16)
    # frames of the batch first, then how they split into utterances
    top = 30000 if op == "full_bwd" else 56000
    # (a segment of one frame alone has no gradient but rounding noise in q and k:
    # such segments come beside longer ones, in the listed ragged cases)
    shortest = 1 if op.startswith("rope") else 2
    t_max = _log_int(rng, shortest, 4700)
    n_seq = _log_int(rng, 1, max(1, min(160, top // t_max)))
    t_min = rng.randint(shortest, t_max)
    kw = {"fused": rng.random() < 0.5}
    if op.startswith("rope"):
        kw.update(kv_heads=rng.randint(1, heads), rot_dim=rng.choice([16, 32, 48, 64]), interleaved=rng.random() < 0.5,
                  norm=rng.random() < 0.7, far=rng.choice([0, 1000, 180000]), stretch=rng.choice([1.0, 2.0, 8.0]))
    if op == "block_bwd":
        kw.update(block=rng.randint(2, 256))
    c = _case("", op, n_seq, t_min, t_max, heads, len_seed=rng.randrange(1 << 20), **kw)
    del c["name"]
    return c


def _lengths(case):
    r = random.Random(case["len_seed"])
    return [r.randint(case["t_min"], case["t_max"]) for _ in range(case["n_seq"])]


def _segments(case):
    """(first frame, frames) of every block (block_bwd) or utterance (full_bwd)."""
    segs, start = [], 0
    for t in _lengths(case):
        step = case.get("block", t)
        segs += [(start + a, min(step, t - a)) for a in range(0, t, step)]
        start += t
    return segs


# ------------------------------------------------------------------ inputs
def _normal(g, shape, factor=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * factor).to(torch.bfloat16)


def _projected(g, case, total, heads, factor=1.0):
    """bf16 [total, h, 64] for each h of heads: views of one buffer where the case has a fused projection."""
    if not case["fused"]:
        return [_normal(g, (total, h, D), factor) for h in heads]
    buf = _normal(g, (total, sum(heads), D), factor)
    return list(buf.split(heads, dim=1))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    lengths = _lengths(case)
    total = sum(lengths)
    offsets = [0]
    for t in lengths:
        offsets.append(offsets[-1] + t)
    s = {"op": case["op"], "cu": torch.tensor(offsets, dtype=torch.int32, device="cuda")}
    if case["op"].startswith("rope"):
        q_heads, k_heads = case["heads"], case["kv_heads"]
        s["q"], s["k"] = _projected(g, case, total, [q_heads, k_heads])
        half = case["rot_dim"] // 2
        # frequencies of stretched positions, kept in 64 bits by the program
        s["inv_freq"] = (ROPE_BASE ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)) / case["stretch"]
        s["interleaved"] = case["interleaved"]
        s["w_q"] = s["w_k"] = None
        if case["norm"]:
            s["w_q"], s["w_k"] = ((1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2))
        frames = torch.arange(total, device="cuda")
        inside = frames - s["cu"][torch.searchsorted(s["cu"], frames.int(), right=True) - 1]
        s["positions"] = (inside + case["far"]).int() if case["far"] else None
        s["inside"] = inside   # position of each frame in its utterance, for the plain form
        if case["op"] == "rope_bwd":
            s["dq"], s["dk"] = _projected(g, case, total, [q_heads, k_heads], 0.02)
        return s
    heads = case["heads"]
    s["q"], s["k"], s["v"] = _projected(g, case, total, [heads] * 3)
    s["dout"] = _normal(g, (total, heads, D), 0.02)
    segs = _segments(case)
    longest = max(n for _, n in segs)
    first = torch.tensor([a for a, _ in segs], device="cuda")[:, None]
    count = torch.tensor([n for _, n in segs], device="cuda")[:, None]
    lane = torch.arange(longest, device="cuda")[None]
    s["block"] = case.get("block", 0)
    s["valid"] = lane < count                                  # [segments, longest]
    s["rows"] = torch.where(s["valid"], first + lane, first)   # frame of each place
    # what the forward pass kept for the backward one
    p = _scores(s)
    p.masked_fill_(~s["valid"][:, None, None, :], -math.inf)
    lse = torch.logsumexp(p, dim=-1)
    p.sub_(lse[..., None]).exp_()
    out = torch.matmul(p, _padded(s, "v"))
    s["out"] = _unpadded(s, out)
    s["lse"] = torch.empty(heads, total, device="cuda")
    s["lse"][:, s["rows"][s["valid"]]] = lse.permute(1, 0, 2)[:, s["valid"]]
    return s


# ------------------------------------------------------------------ plain forms
def _angles(s):
    pos = s["inside"] if s["positions"] is None else s["positions"]
    a = pos.double()[:, None] * s["inv_freq"]
    return a.cos().float()[:, None], a.sin().float()[:, None]   # [frames, 1, rot_dim / 2]


def _pairs(s, x):
    """The two members of every rotated pair, and what is not rotated."""
    half = s["inv_freq"].numel()
    if s["interleaved"]:
        return x[..., 0:2 * half:2], x[..., 1:2 * half:2], x[..., 2 * half:]
    return x[..., :half], x[..., half:2 * half], x[..., 2 * half:]


def _joined(s, a, b, rest):
    ab = torch.stack([a, b], dim=-1).flatten(-2) if s["interleaved"] else torch.cat([a, b], dim=-1)
    return torch.cat([ab, rest], dim=-1)


def _rotated(s, x, back):
    cos, sin = _angles(s)
    if back:
        sin = -sin
    a, b, rest = _pairs(s, x)
    return _joined(s, a * cos - b * sin, b * cos + a * sin, rest)


def _rope_plain(s, x, w):
    z = x.float()
    if w is not None:
        z = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    return _rotated(s, z, False).to(torch.bfloat16)


def _rope_bwd_plain(s, dy, x, w):
    dz = _rotated(s, dy.float(), True)
    if w is None:
        return dz.to(torch.bfloat16), None
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    n = x * r
    g = dz * w.float()
    dx = r * (g - n * (g * n).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), (dz * n).sum((0, 1), dtype=torch.float64).float()


def _padded(s, name):
    """[segments, heads, longest, 64] in 32 bits, places past a segment's end zero."""
    x = s[name].float()[s["rows"]].masked_fill_(~s["valid"][..., None, None], 0.0)
    return x.permute(0, 2, 1, 3)


def _unpadded(s, x):
    out = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    out[s["rows"][s["valid"]]] = x.permute(0, 2, 1, 3)[s["valid"]].to(torch.bfloat16)
    return out


def _scores(s):
    return torch.matmul(_padded(s, "q") * (1.0 / math.sqrt(D)), _padded(s, "k").transpose(-1, -2))


def _attention_bwd_plain(s):
    scale = 1.0 / math.sqrt(D)
    do, pad = _padded(s, "dout"), ~s["valid"]
    lse = s["lse"][:, s["rows"]].permute(1, 0, 2)[..., None]
    p = _scores(s).sub_(lse).exp_()
    p.masked_fill_(pad[:, None, None, :], 0.0).masked_fill_(pad[:, None, :, None], 0.0)
    dv = torch.matmul(p.transpose(-1, -2), do)
    delta = (do * _padded(s, "out")).sum(-1, keepdim=True)
    ds = torch.matmul(do, _padded(s, "v").transpose(-1, -2)).sub_(delta).mul_(p)
    del p
    dq = torch.matmul(ds, _padded(s, "k")) * scale
    dk = torch.matmul(ds.transpose(-1, -2), _padded(s, "q")) * scale
    return [_unpadded(s, x) for x in (dq, dk, dv)]


def run(s):
    op = s["op"]
    if own:
        from chunked_block_self_b200 import nle
        if op == "rope":
            return nle.qk_norm_rope(s["q"], s["k"], s["cu"], s["inv_freq"], s["w_q"], s["w_k"],
                                    interleaved=s["interleaved"], positions=s["positions"])
        if op == "rope_bwd":
            dq, dk, dw_q, dw_k = nle.qk_norm_rope_bwd(s["dq"], s["dk"], s["cu"], s["inv_freq"], s["q"], s["k"],
                                                      s["w_q"], s["w_k"], interleaved=s["interleaved"],
                                                      positions=s["positions"])
            return dq, dk, dw_q, dw_k
        if op == "block_bwd":
            return nle.block_attn_bwd(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["cu"],
                                      block_frames=s["block"])
        return nle.varlen_attn_bwd(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["cu"])
    if op == "rope":
        return _rope_plain(s, s["q"], s["w_q"]), _rope_plain(s, s["k"], s["w_k"])
    if op == "rope_bwd":
        dq, dw_q = _rope_bwd_plain(s, s["dq"], s["q"], s["w_q"])
        dk, dw_k = _rope_bwd_plain(s, s["dk"], s["k"], s["w_k"])
        return dq, dk, dw_q, dw_k
    return tuple(_attention_bwd_plain(s))


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    total = sum(_lengths(case))
    if case["op"].startswith("rope"):
        rows = total * (case["heads"] + case["kv_heads"])
        back = case["op"] == "rope_bwd"
        tensors = 2 + (1 if back and case["norm"] else 0)   # the gradient needs x itself only for the norm
        small = 4 * total * (1 if case["far"] else 0) + 8 * case["rot_dim"] // 2 + 4 * (case["n_seq"] + 1)
        if case["norm"]:
            small += 2 * D * (6 if back else 2)
        per_row = 3 * case["rot_dim"] + ((10 if back else 5) * D if case["norm"] else 0)
        return {"bytes": tensors * rows * D * 2 + small, "flops": rows * per_row}
    pairs = sum(n * n for _, n in _segments(case))
    heads = case["heads"]
    # read q, k, v, out, dout and lse; write dq, dk, dv; five products of 2 * 64 each per (query, key) pair
    return {"bytes": total * heads * (8 * D * 2 + 4) + 4 * (case["n_seq"] + 1), "flops": 10 * D * pairs * heads}


# ------------------------------------------------------------------ the definitions, in 64 bits
def _exact_rope(case, s, back):
    total = s["q"].shape[0]
    start = torch.zeros(total, dtype=torch.float64, device="cuda")
    lengths = _lengths(case)
    at = 0
    for t in lengths:
        start[at:at + t] = at
        at += t
    pos = torch.arange(total, dtype=torch.float64, device="cuda") - start + case["far"]
    m = case["rot_dim"] // 2
    turn = torch.polar(torch.ones(total, m, dtype=torch.float64, device="cuda"), torch.outer(pos, s["inv_freq"]))
    if back:
        turn = turn.conj()
    i = torch.arange(m, device="cuda")
    re, im = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + m)

    def rotate(z):
        z = z.clone()
        c = torch.complex(z[..., re], z[..., im]) * turn[:, None]
        z[..., re], z[..., im] = c.real, c.imag
        return z

    outs, weights = [], []
    for name, wname in (("q", "w_q"), ("k", "w_k")):
        x, w = s[name].double(), s[wname]
        rms = None if w is None else ((x * x).sum(-1, keepdim=True) / D + 1e-6).sqrt()
        if not back:
            outs.append(rotate(x if w is None else w.double() * x / rms))
            continue
        dz = rotate(s["d" + name].double())
        if w is None:
            outs.append(dz)
            weights.append(None)
            continue
        gx = (dz * w.double() * x).sum(-1, keepdim=True)
        outs.append(dz * w.double() / rms - x * gx / (D * rms ** 3))
        weights.append((dz * x / rms).flatten(0, 1).sum(0))
    return tuple(outs + weights) if back else tuple(outs)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("rope"):
        return _exact_rope(case, s, case["op"] == "rope_bwd")
    grads = [torch.empty(s["q"].shape, dtype=torch.float64, device="cuda") for _ in range(3)]
    for a, n in _segments(case):
        q, k, v, do, o = (s[x][a:a + n].double().transpose(0, 1) for x in ("q", "k", "v", "dout", "out"))
        p = torch.einsum("hid,hjd->hij", q, k).div_(math.sqrt(D)).sub_(s["lse"][:, a:a + n].double()[..., None]).exp_()
        dv = torch.einsum("hij,hid->hjd", p, do)
        p.mul_(torch.einsum("hid,hjd->hij", do, v) - torch.einsum("hid,hid->hi", do, o)[..., None]).div_(math.sqrt(D))
        for to, x in zip(grads, (torch.einsum("hij,hjd->hid", p, k), torch.einsum("hij,hid->hjd", p, q), dv)):
            to[a:a + n] = x.transpose(0, 1)
    return tuple(grads)
