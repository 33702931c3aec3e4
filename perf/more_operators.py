"""Measured cases of the operators over serialised voxel rows: windowed attention, gated scan, layer norm and dropout.

``own`` is False: ``run`` computes an operator from elementary torch operations in 32 bits, rounded once at the end.
``own`` is True: ``run`` makes the calls of ``sparse_submanifold_convolution_amd`` that a program makes.  Both take the
state that ``prepare`` builds.  ``exact`` restates the operators in 64 bits.

Operators (rows are voxels in z-order or Hilbert order, ragged samples one after another; sums in at least 32 bits):

window_attention  row i of a sample sits at place t = i + (keys - rows) of the sample's keys and attends the keys j with
                  j <= t + right and (j >= t - left or j < sinks) whose mask is set: out = softmax(scale q k^T) v, query
                  heads sharing key heads; a row with no key gives zeros and lse = -inf.  left, right: -1 for no bound.
gated_scan        h_t = a_t h_{t-1} + (1 - a_t) x_t ("mix") or a_t h_{t-1} + x_t ("sum"), a = sigmoid(gate), per channel
                  along a sample's rows (from the last row where reversed) from its initial state; the rows' h and the
                  samples' final states.
layer_norm        y = (s - mean s) / sqrt(var s + eps) w + b over a row's channels, with s = x, or s = residual +
                  dropout(x), which is an output as well.
dropout           y = x * keep * 65536 / (65536 - t), plus a residual where given: element e of the flattened tensor is
                  kept where its 16 random bits are at least t = round(65536 p).  The bits are half-word e mod 8 (low half
                  of a word first) of Philox-4x32 with ten rounds of counter (e div 8, layer, step low, step high) and
                  key (seed low, seed high); seed and step are inputs.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5
LAYER = 3  # which of a network's dropout layers the cases stand for


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------

def _text(lens):
    return ",".join(map(str, lens))


def _ints(text):
    return [int(v) for v in text.split(",")]


def _window(q_lens, kv_lens, heads_q, heads_kv, dim, dtype, left, right, sinks, mask="none", packed=False, train=False):
    return {"op": "window_attention", "q_lens": _text(q_lens), "kv_lens": _text(kv_lens), "heads_q": heads_q, "heads_kv": heads_kv,
            "dim": dim, "dtype": dtype, "left": left, "right": right, "sinks": sinks, "mask": mask, "packed": packed, "train": train}


def _scan(lens, channels, dtype, form="mix", reverse=False, state=False, packed=False, train=False):
    return {"op": "gated_scan", "lens": _text(lens), "channels": channels, "dtype": dtype, "form": form, "reverse": reverse,
            "state": state, "packed": packed, "train": train}


def _norm(n, channels, dtype, residual=False, p=0.0, affine=True, train=False):
    return {"op": "layer_norm", "n": n, "channels": channels, "dtype": dtype, "residual": residual, "p": p, "affine": affine,
            "train": train}


def _dropout(n, channels, dtype, p, residual=False, train=False):
    return {"op": "dropout", "n": n, "channels": channels, "dtype": dtype, "p": p, "residual": residual, "train": train}


def listed():
    return [
        # the next row of one sample while serving, over a cache of the largest 256^3 shell's rows: the call's latency
        dict(_window([1], [211026], 4, 4, 64, "bf16", 1023, 0, 4), name="window one row"),
        # the 2 x 64^3 shells workload's rows, windows of 257 and four register rows, from a packed projection, inference
        dict(_window([11302, 11115], [11302, 11115], 4, 4, 64, "f16", 128, 128, 4, packed=True), name="window 64^3"),
        # training at the 4 x 256^3 shells' 0.8M rows and 256 channels, windows of 1,025: the longest sequences
        dict(_window([199911, 203045, 185530, 211026], [199911, 203045, 185530, 211026], 4, 4, 64, "bf16", 512, 512, 4, train=True),
             name="window 256^3 train"),
        # ragged fp32 batch, causal, an empty sample, grouped heads of an odd size, masked rows, training
        dict(_window([700, 0, 333, 1, 838], [700, 129, 333, 77, 838], 6, 2, 40, "f32", 100, 0, 1, mask="random", train=True),
             name="window ragged train f32"),
        # one more row of each of 32 sequences while serving at 1,024 channels, from their states
        dict(_scan([1] * 32, 1024, "bf16", state=True), name="scan one row"),
        # the 2 x 64^3 shells at 64 channels, from the last row, x and gate of a packed projection, training
        dict(_scan([11302, 11115], 64, "f16", reverse=True, packed=True, train=True), name="scan 64^3 train"),
        # ragged fp32 batch with empty samples and initial states, 40 channels, training
        dict(_scan([700, 0, 333, 1, 838], 40, "f32", form="sum", state=True, train=True), name="scan ragged train f32"),
        # the 128^3 random-occupancy workload's rows at its 1,024 channels, training: the largest streaming case
        dict(_scan([629000], 1024, "bf16", train=True), name="scan 128^3 train"),
        # one pooled token while serving
        dict(_norm(1, 256, "bf16"), name="norm one row"),
        # the 128^3 workload's rows at its 1,024 channels: dropout, residual and norm of a training step
        dict(_norm(629000, 1024, "bf16", residual=True, p=0.1, train=True), name="norm 128^3 train"),
        # the 32^3 shell's rows, fp32, an odd width
        dict(_dropout(1872, 40, "f32", 0.1), name="dropout 32^3 f32"),
        # the 4 x 256^3 shells at 256 channels, with the residual, training
        dict(_dropout(799512, 256, "bf16", 0.1, residual=True, train=True), name="dropout 256^3 train"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def _size(dtype):
    return 4 if dtype == "f32" else 2


def _channels(rng, dtype, lo, hi):
    step = 4 if dtype == "f32" else 8  # rows are whole 16-byte vectors
    return max(step, _log(rng, lo, hi) // step * step) if rng.random() < 0.5 else rng.choice([32, 64, 128, 256, 512, 1024])


def _draw_window(rng):
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    dim = rng.choice([32, 40, 48, 64, 64, 72, 80, 96, 128])
    heads_kv = rng.choice([1, 2, 4, 8])
    heads_q = heads_kv * rng.choice([1, 1, 2, 4])
    samples = rng.choice([1, 2, 3, 4, 7])
    form = rng.choice(["self", "self", "causal", "next"])
    left, sinks = rng.choice([0, _log(rng, 1, 4096), _log(rng, 16, 1024)]), rng.choice([0, 0, 1, 4, 17, 64])
    right = 0 if form != "self" else rng.choice([left, left, _log(rng, 1, 1024)])
    train = form != "next" and rng.random() < 0.6
    hi = _log(rng, 2, 200000)
    # no more than a third of the largest listed case's products, and for fp32 a fifth of that
    most = 7e10 / (heads_q * dim) * (0.2 if dtype == "f32" else 1.0) * (1.0 if train else 3.0)
    seen = left + right + 1 + sinks
    while form != "next" and samples * hi * min(hi, seen) > most:
        hi = max(2, int(hi * 0.8))
    kv_lens = [max(1, int(hi * rng.uniform(0.6, 1.0))) for _ in range(samples)]
    q_lens = [min(rng.choice([1, 1, 1, 5]), m) for m in kv_lens] if form == "next" else list(kv_lens)
    if samples > 2 and rng.random() < 0.4:
        q_lens[1] = 0
    if form == "self" and rng.random() < 0.1:
        left = -1 if samples * hi * hi < most else left
    return _window(q_lens, kv_lens, heads_q, heads_kv, dim, dtype, left, right, sinks, rng.choice(["none", "none", "tail", "random"]),
                   rng.random() < 0.4, train)


def _draw_scan(rng):
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    channels = _channels(rng, dtype, 8, 1024)
    train = rng.random() < 0.6
    rows = _log(rng, 1, min(800000, 0.9 * 629000 * 1024 * 2 / (channels * _size(dtype))))
    samples = min(rows, rng.choice([1, 1, 2, 4, 32, 300]))
    cuts = sorted(rng.randint(0, rows) for _ in range(samples - 1))  # an empty sample now and then
    lens = [b - a for a, b in zip([0] + cuts, cuts + [rows])]
    return _scan(lens, channels, dtype, rng.choice(["mix", "mix", "sum"]), rng.random() < 0.4, rng.random() < 0.5, rng.random() < 0.4, train)


def _draw_norm(rng):
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    channels = _channels(rng, dtype, 8, 4096)
    rows = _log(rng, 1, min(800000, 0.9 * 629000 * 1024 * 2 / (channels * _size(dtype))))
    residual = rng.random() < 0.6
    return _norm(rows, channels, dtype, residual, rng.choice([0.0, 0.1, 0.37]) if residual else 0.0, rng.random() < 0.8, rng.random() < 0.6)


def _draw_dropout(rng):
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    channels = _log(rng, 1, 2048)
    rows = _log(rng, 1, min(800000, 0.9 * 799512 * 256 * 2 / (channels * _size(dtype))))
    return _dropout(rows, channels, dtype, rng.choice([0.0, 0.05, 0.1, 0.5, 0.93]), rng.random() < 0.5, rng.random() < 0.5)


def draw(rng):
    return rng.choice([_draw_window, _draw_window, _draw_scan, _draw_scan, _draw_norm, _draw_dropout])(rng)


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------

def _rows(n, *shape, gen, dev, dtype, centres=None):
    """Rows of standard normal values, scattered around a few directions where given, as a trained projection's are."""
    x = torch.empty(n, *shape, device=dev, dtype=dtype)
    for lo in range(0, n, 1 << 17):
        hi = min(n, lo + (1 << 17))
        y = torch.randn(hi - lo, *shape, generator=gen, device=dev)
        if centres is not None:
            y += centres[torch.randint(0, centres.shape[0], (hi - lo,), generator=gen, device=dev)]
        x[lo:hi] = y.to(dtype)
    return x


def _pack(parts):
    """The same values as views of one packed projection."""
    whole = torch.cat(parts, dim=1)
    at, views = 0, []
    for p in parts:
        views.append(whole[:, at:at + p.shape[1]])
        at += p.shape[1]
    return views


def _offsets(lens, dev):
    return torch.tensor([sum(lens[:b]) for b in range(len(lens) + 1)], dtype=torch.int32, device=dev)


def _prepare_window(case, st, make, gen, dev):
    hq, hk, dim = case["heads_q"], case["heads_kv"], case["dim"]
    q_lens, kv_lens = _ints(case["q_lens"]), _ints(case["kv_lens"])
    nq, nk = sum(q_lens), sum(kv_lens)
    centres = 0.8 * torch.randn(24, 1, dim, generator=gen, device=dev)
    q, k = make(nq, hq, dim, centres=centres), make(nk, hk, dim, centres=centres)
    v = make(nk, hk, dim)
    st["kv_mask"] = None
    if case["mask"] != "none":
        keep = torch.ones(nk, dtype=torch.bool, device=dev)
        at = 0
        for m in kv_lens:
            if case["mask"] == "tail":
                keep[at:at + m] = torch.arange(m, device=dev) < torch.randint(m // 2, m + 1, (1,), generator=gen, device=dev)
            else:
                keep[at:at + m] = torch.rand(m, generator=gen, device=dev) < 0.8
            at += m
        st["kv_mask"] = keep
        k[~keep] = float("nan")  # padding rows hold whatever was in memory
        v[~keep] = float("inf")
    if case["packed"]:
        k, v = _pack([k, v])
    st.update(q=q, k=k, v=v, q_offsets=_offsets(q_lens, dev), kv_offsets=_offsets(kv_lens, dev), q_lens=q_lens, kv_lens=kv_lens)
    st["scale"] = 1.0 / math.sqrt(dim)
    if case["train"]:
        st["dout"] = 0.1 * make(nq, hq, dim)


def _prepare_scan(case, st, make, gen, dev):
    lens, c = _ints(case["lens"]), case["channels"]
    n = sum(lens)
    x = make(n, c)
    # channels remember from two to a few hundred rows
    gate = (make(n, c).float() + torch.linspace(0.0, 6.0, c, device=dev)).to(st["dtype"])
    if case["packed"]:
        x, gate = _pack([x, gate])
    st.update(x=x, gate=gate, lens=lens, offsets=_offsets(lens, dev))
    st["h0"] = torch.randn(len(lens), c, generator=gen, device=dev) if case["state"] else None
    if case["train"]:
        st["dy"] = make(n, c)
        st["dlast"] = torch.randn(len(lens), c, generator=gen, device=dev) if case["state"] else None


def prepare(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    st = {"case": case, "op": case["op"], "train": case["train"], "dtype": dtype}

    def make(*shape, centres=None):
        return _rows(*shape, gen=gen, dev=dev, dtype=dtype, centres=centres)

    if case["op"] == "window_attention":
        _prepare_window(case, st, make, gen, dev)
    elif case["op"] == "gated_scan":
        _prepare_scan(case, st, make, gen, dev)
    else:
        n, c = case["n"], case["channels"]
        st["x"] = make(n, c)
        st["residual"] = make(n, c) if case["residual"] else None
        st["rng"] = torch.randint(0, 1 << 62, (2,), generator=gen, device=dev)  # a program's seed and step
        if case["op"] == "layer_norm":
            st["weight"] = (1 + 0.2 * torch.randn(c, generator=gen, device=dev)).to(dtype) if case["affine"] else None
            st["bias"] = (0.2 * torch.randn(c, generator=gen, device=dev)).to(dtype) if case["affine"] else None
        if case["train"]:
            st["dy"] = make(n, c)
            if case["op"] == "layer_norm" and case["residual"]:
                st["ds"] = make(n, c)
    return st


# ---------------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------------

def _bits(rng, blocks):
    """[blocks, 8] the 16-bit halves of Philox-4x32-10's four words for counters (block, LAYER, step)."""
    low = 0xFFFFFFFF
    c0 = torch.arange(blocks, dtype=torch.int64, device=rng.device)
    c1, c2, c3 = torch.full_like(c0, LAYER), (rng[1] & low).expand(blocks), (rng[1] >> 32 & low).expand(blocks)
    k0, k1 = rng[0] & low, rng[0] >> 32 & low
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # 64-bit products: their bits wrap as unsigned ones' do
        c0, c1, c2, c3 = (p1 >> 32 & low) ^ c1 ^ k0, p1 & low, (p0 >> 32 & low) ^ c3 ^ k1, p0 & low
        k0, k1 = k0 + 0x9E3779B9 & low, k1 + 0xBB67AE85 & low
    return torch.stack([w >> s & 0xFFFF for w in (c0, c1, c2, c3) for s in (0, 16)], dim=1).to(torch.int32)


def _kept(st, shape):
    """(truth of the kept elements, factor), or None for no dropout."""
    t = int(math.floor(st["case"]["p"] * 65536 + 0.5))
    if t == 0:
        return None
    count = math.prod(shape)
    keep = _bits(st["rng"], (count + 7) // 8).view(-1)[:count].view(shape) >= t
    return keep, 65536.0 / (65536 - t)


def _drop(x, kept):
    return x if kept is None else torch.where(kept[0], x * kept[1], 0.0)


def _plain_dropout(st):
    kept = _kept(st, st["x"].shape)
    y = _drop(st["x"].float(), kept)
    if st["residual"] is not None:
        y = y + st["residual"].float()
    outs = {"y": y.to(st["dtype"])}
    if st["train"]:
        outs["dx"] = _drop(st["dy"].float(), kept).to(st["dtype"])
    return outs


def _plain_norm(st):
    kept = _kept(st, st["x"].shape)
    s = _drop(st["x"].float(), kept)
    outs = {}
    if st["residual"] is not None:
        s = s + st["residual"].float()
        outs["s"] = s.to(st["dtype"])
    mean = s.mean(-1, keepdim=True)
    d = s - mean
    r = torch.rsqrt((d * d).mean(-1, keepdim=True) + EPS)
    xn = d * r
    wf = 1.0 if st["weight"] is None else st["weight"].float()
    outs["y"] = (xn * wf if st["bias"] is None else xn * wf + st["bias"].float()).to(st["dtype"])
    if st["train"]:
        dy = st["dy"].float()
        g = dy * wf
        ds = (g - g.mean(-1, keepdim=True) - xn * (g * xn).mean(-1, keepdim=True)) * r
        if st["residual"] is not None:
            ds = ds + st["ds"].float()
            outs["dresidual"] = ds.to(st["dtype"])
        outs["dx"] = _drop(ds, kept).to(st["dtype"])
        if st["weight"] is not None:
            outs["dweight"] = (dy * xn).sum(0).to(st["dtype"])
            outs["dbias"] = dy.sum(0).to(st["dtype"])
    return outs


def _recur(a, b, piece=64):
    """h_t = a_t h_{t-1} + b_t along the rows from zero: rows in pieces, walked side by side, then the pieces' ends."""
    n, c = a.shape
    pad = -n % piece
    if pad:
        a, b = (torch.cat([t, t.new_zeros(pad, c)]) for t in (a, b))
    a, b = a.view(-1, piece, c), b.view(-1, piece, c)
    h, prod = b.clone(), a.clone()
    for t in range(1, piece):
        h[:, t].addcmul_(a[:, t], h[:, t - 1])
        prod[:, t].mul_(prod[:, t - 1])
    if len(a) > 1:
        ends = h[:, -1] if len(a) < piece else None
        if ends is None:
            ends = _recur(prod[:, -1].contiguous(), h[:, -1].contiguous(), piece)
        else:
            ends = ends.clone()
            for i in range(1, len(a)):
                ends[i].addcmul_(prod[i, -1], ends[i - 1])
        h[1:].addcmul_(prod[1:], ends[:-1, None])
    return h.view(-1, c)[:n]


def _plain_scan(st):
    lens, form = st["lens"], st["case"]["form"]
    x, gate = st["x"].float(), st["gate"].float()
    n, c = x.shape
    off = st["offsets"].long()
    some = off[1:] > off[:-1]
    first, last = off[:-1][some], off[1:][some] - 1
    if st["case"]["reverse"]:  # mirrored rows run forward
        x, gate = x.flip(0), gate.flip(0)
        first, last = n - 1 - last, n - 1 - first
    a, keep = torch.sigmoid(gate), torch.sigmoid(-gate)
    b = keep * x if form == "mix" else x.clone()
    h0 = x.new_zeros(len(lens), c) if st["h0"] is None else st["h0"]
    b[first] += a[first] * h0[some]
    inside = a.clone()
    inside[first] = 0.0
    h = _recur(inside, b)
    end = h0.clone()
    end[some] = h[last]
    flip = (lambda t: t.flip(0)) if st["case"]["reverse"] else (lambda t: t)
    outs = {"y": flip(h).to(st["dtype"]), "last": end}
    if not st["train"]:
        return outs
    g = flip(st["dy"].float())
    g = g.clone()
    if st["dlast"] is not None:
        g[last] += st["dlast"][some]
    after = torch.cat([inside[1:], inside.new_zeros(1, c)])  # the row behind takes a_{t+1} of this one, not over an end
    d = _recur(after.flip(0), g.flip(0)).flip(0)
    before = torch.cat([h.new_zeros(1, c), h[:-1]])
    before[first] = h0[some]
    outs["dx"] = flip(keep * d if form == "mix" else d).to(st["dtype"])
    outs["dgate"] = flip(a * keep * d * (before - x if form == "mix" else before)).to(st["dtype"])
    if st["h0"] is not None:
        dh0 = torch.zeros_like(h0) if st["dlast"] is None else st["dlast"].clone()
        dh0[some] = (a * d)[first]
        outs["dh0"] = dh0
    return outs


def _bounds(case):
    far = 1 << 30
    return (far if case["left"] < 0 else case["left"]), (far if case["right"] < 0 else case["right"]), case["sinks"]


def _plain_window(st, block=1024):
    q, k, v, dev = st["q"], st["k"], st["v"], st["q"].device
    (nq, hq, dim), (nk, hk) = q.shape, k.shape[:2]
    g, scale = hq // hk, st["scale"]
    left, right, sinks = _bounds(st["case"])
    out, lse = torch.zeros(nq, hq, dim, device=dev), torch.full((nq, hq), float("-inf"), device=dev)
    if st["train"]:
        dq, dk, dv = torch.zeros(nq, hq, dim, device=dev), torch.zeros(nk, hk, dim, device=dev), torch.zeros(nk, hk, dim, device=dev)
    q_at = kv_at = 0
    for lq, lk in zip(st["q_lens"], st["kv_lens"]):
        shift = lk - lq
        for lo in range(0, lq, block):
            hi = min(lo + block, lq)
            m = hi - lo
            j1 = min(lk, hi + shift + right)
            j0 = min(max(0, lo + shift - left), max(j1, 0))
            top = min(sinks, j0)
            if j1 - j0 + top <= 0:
                continue
            keys = torch.cat([torch.arange(top, device=dev), torch.arange(j0, j1, device=dev)])
            place = torch.arange(lo, hi, device=dev)[:, None] + shift
            seen = (keys <= place + right) & ((keys >= place - left) | (keys < sinks))
            parts = [slice(kv_at, kv_at + top), slice(kv_at + j0, kv_at + j1)]
            kf, vf = (torch.cat([t[p] for p in parts]).float() for t in (k, v))
            if st["kv_mask"] is not None:
                on = st["kv_mask"][keys + kv_at]
                seen = seen & on
                kf, vf = (torch.where(on[:, None, None], t, 0.0) for t in (kf, vf))
            kf, vf = kf.transpose(0, 1).contiguous(), vf.transpose(0, 1).contiguous()

            def by_head(x):  # [m, Hq, D] -> [Hk, G m, D]
                return x.float().view(m, hk, g, dim).permute(1, 2, 0, 3).reshape(hk, g * m, dim)

            def by_row(x):
                return x.view(hk, g, m, -1).permute(2, 0, 1, 3).reshape(m, hq, -1)

            rows = slice(q_at + lo, q_at + hi)
            qf = by_head(q[rows])
            s = torch.matmul(qf, kf.transpose(1, 2)).mul_(scale)
            s.masked_fill_(~seen.repeat(g, 1), float("-inf"))
            top_s = s.amax(-1, keepdim=True)
            top_s = torch.where(top_s == float("-inf"), 0.0, top_s)
            p = s.sub_(top_s).exp_()
            total = p.sum(-1, keepdim=True)
            p.mul_(torch.where(total > 0, 1.0 / total, 0.0))
            o = torch.matmul(p, vf)
            out[rows] = by_row(o)
            lse[rows] = by_row(torch.where(total > 0, top_s + total.log(), float("-inf")))[..., 0]
            if st["train"]:
                do = by_head(st["dout"][rows])
                pv = torch.matmul(p.transpose(1, 2), do).transpose(0, 1)
                ds = torch.matmul(do, vf.transpose(1, 2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
                dq[rows] = by_row(torch.matmul(ds, kf))
                pk = torch.matmul(ds.transpose(1, 2), qf).transpose(0, 1)
                for total_of, part in ((dk, pk), (dv, pv)):
                    total_of[parts[0]] += part[:top]
                    total_of[parts[1]] += part[top:]
        q_at, kv_at = q_at + lq, kv_at + lk
    outs = {"out": out.to(st["dtype"]), "lse": lse.t().contiguous()}
    if st["train"]:
        if st["kv_mask"] is not None:
            dk[~st["kv_mask"]] = 0.0
            dv[~st["kv_mask"]] = 0.0
        outs.update(dq=dq.to(st["dtype"]), dk=dk.to(st["dtype"]), dv=dv.to(st["dtype"]))
    return outs


# ---------------------------------------------------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------------------------------------------------

def _own_window(st):
    import sparse_submanifold_convolution_amd as ssc
    case = st["case"]
    where = (st["q_offsets"], st["kv_offsets"])
    kw = {"left": None if case["left"] < 0 else case["left"], "right": None if case["right"] < 0 else case["right"],
          "sinks": case["sinks"], "kv_mask": st["kv_mask"], "scale": st["scale"]}
    out, lse = ssc.window_attention_fwd(st["q"], st["k"], st["v"], *where, **kw)
    outs = {"out": out, "lse": lse}
    if st["train"]:
        dq, dk, dv = ssc.window_attention_bwd(st["q"], st["k"], st["v"], out, lse, st["dout"], *where, **kw)
        outs.update(dq=dq, dk=dk, dv=dv)
    return outs


def _own_scan(st):
    import sparse_submanifold_convolution_amd as ssc
    kw = {"h0": st["h0"], "reverse": st["case"]["reverse"], "form": st["case"]["form"]}
    y, last, carries = ssc.gated_scan_fwd(st["x"], st["gate"], st["offsets"], need_carries=st["train"], **kw)
    outs = {"y": y, "last": last}
    if st["train"]:
        dx, dgate, dh0 = ssc.gated_scan_bwd(st["x"], st["gate"], carries, st["dy"], st["offsets"], dlast=st["dlast"], **kw)
        outs.update(dx=dx, dgate=dgate)
        if st["h0"] is not None:
            outs["dh0"] = dh0
    return outs


def _own_norm(st):
    import sparse_submanifold_convolution_amd as ssc
    w, b = st["weight"], st["bias"]
    if st["residual"] is None:
        outs = {"y": ssc.layer_norm_fwd(st["x"], w, b, EPS)}
        if st["train"]:
            outs["dx"], dw, db = ssc.layer_norm_bwd(st["x"], st["dy"], w, b, EPS)
    else:
        drop = {"p": st["case"]["p"], "rng": st["rng"], "layer": LAYER}
        y, s = ssc.add_layer_norm_fwd(st["x"], st["residual"], w, b, EPS, **drop)
        outs = {"s": s, "y": y}
        if st["train"]:
            outs["dx"], dr, dw, db = ssc.add_layer_norm_bwd(s, st["dy"], st["ds"], w, b, EPS, **drop)
            outs["dresidual"] = dr
    if st["train"] and w is not None:
        outs.update(dweight=dw, dbias=db)
    return outs


def _own_dropout(st):
    import sparse_submanifold_convolution_amd as ssc
    kw = {"p": st["case"]["p"], "rng": st["rng"], "layer": LAYER}
    outs = {"y": ssc.dropout_fwd(st["x"], residual=st["residual"], **kw)}
    if st["train"]:
        outs["dx"] = ssc.dropout_bwd(st["dy"], **kw)
    return outs


_NAMES = ("out", "lse", "dq", "dk", "dv", "s", "y", "last", "dx", "dresidual", "dgate", "dh0", "dweight", "dbias")


def run(state):
    op = state["op"]
    if own:
        outs = {"window_attention": _own_window, "gated_scan": _own_scan, "layer_norm": _own_norm, "dropout": _own_dropout}[op](state)
    else:
        outs = {"window_attention": _plain_window, "gated_scan": _plain_scan, "layer_norm": _plain_norm, "dropout": _plain_dropout}[op](state)
    return {name: outs[name] for name in _NAMES if name in outs}


# ---------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------------

def _pairs(case):
    """(pairs of rows and keys they see, keys any row sees) of a window case, masks aside."""
    left, right, sinks = _bounds(case)
    pairs = keys = 0
    for lq, lk in zip(_ints(case["q_lens"]), _ints(case["kv_lens"])):
        t = torch.arange(lq, dtype=torch.int64) + (lk - lq)
        hi = (t + right + 1).clamp(0, lk)
        lo = torch.minimum((t - left).clamp(0, lk), hi)
        pairs += int((hi - lo + torch.minimum(lo, torch.tensor(sinks))).sum())
        if lq:
            keys += int(hi[-1] - lo[0] + min(int(lo[0]), sinks))
    return pairs, keys


def work(case):
    size = _size(case["dtype"])
    if case["op"] == "window_attention":
        hq, hk, dim = case["heads_q"], case["heads_kv"], case["dim"]
        nq = sum(_ints(case["q_lens"]))
        pairs, keys = _pairs(case)
        # forward: q, k, v in, out and lse out; training: dout in and dq, dk, dv out as well
        moved = (2 * nq * hq + 2 * keys * hk) * dim * size * (2 if case["train"] else 1)
        moved += nq * hq * 4 + (keys if case["mask"] != "none" else 0)
        return {"bytes": moved, "flops": pairs * hq * dim * 2 * (7 if case["train"] else 2)}
    if case["op"] == "gated_scan":
        lens, c = _ints(case["lens"]), case["channels"]
        state = len(lens) * c * 4
        elements = sum(lens) * c
        # x, gate in, h out; training: dy in, dx and dgate out as well
        moved = elements * size * (6 if case["train"] else 3) + state * (1 + case["state"]) * (2 if case["train"] else 1)
        return {"bytes": moved, "flops": elements * (30 if case["train"] else 12)}
    elements = case["n"] * case["channels"]
    if case["op"] == "dropout":
        streams = 2 + case["residual"] + (2 if case["train"] else 0)
        return {"bytes": elements * size * streams, "flops": elements * (16 if case["train"] else 8)}
    streams = 4 if case["residual"] else 2  # x (and residual) in, y (and s) out
    if case["train"]:
        streams += 2 if not case["residual"] else 3 + (case["p"] > 0)  # dy (and ds) in, dx (and the residual's, where they differ) out
    weights = 2 * case["channels"] * size * (2 if case["train"] else 1) if case["affine"] else 0
    return {"bytes": elements * size * streams + weights, "flops": elements * (30 if case["train"] else 10)}


# ---------------------------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------------------------------

def _exact_keep(st, lo, hi):
    """Factors 0 or 65536 / (65536 - t) of elements lo .. hi - 1, lo a multiple of 8: each product's halves from 16-bit limbs."""
    t = int(math.floor(st["case"]["p"] * 65536 + 0.5))
    dev = st["rng"].device
    if t == 0:
        return torch.ones(hi - lo, dtype=torch.float64, device=dev)
    seed, step = (int(v) for v in st["rng"].tolist())
    word = [torch.arange(lo // 8, (hi + 7) // 8, dtype=torch.int64, device=dev)] + [LAYER, step % (1 << 32), step >> 32]
    word = [word[0]] + [torch.full_like(word[0], v) for v in word[1:]]
    key = [seed % (1 << 32), seed >> 32]

    def halves(x, m):
        x0, x1, m0, m1 = x % 65536, x // 65536, m % 65536, m // 65536
        low = x0 * m0
        mid = x1 * m0 + low // 65536
        mid2 = x0 * m1 + mid % 65536
        return x1 * m1 + mid // 65536 + mid2 // 65536, mid2 % 65536 * 65536 + low % 65536

    for r in range(10):
        h0, l0 = halves(word[0], 0xD2511F53)
        h1, l1 = halves(word[2], 0xCD9E8D57)
        ka, kb = (key[0] + r * 0x9E3779B9) % (1 << 32), (key[1] + r * 0xBB67AE85) % (1 << 32)
        word = [h1 ^ word[1] ^ ka, l1, h0 ^ word[3] ^ kb, l0]
    out = torch.empty(len(word[0]), 8, dtype=torch.float64, device=dev)
    for i in range(8):
        w = word[i // 2]
        out[:, i] = ((w // 65536 if i % 2 else w % 65536) >= t).double() * (65536.0 / (65536 - t))
    return out.view(-1)[:hi - lo]


def _exact_dropout(st):
    x = st["x"]
    n, c = x.shape
    names = ["y"] + (["dx"] if st["train"] else [])
    outs = {name: torch.empty(n * c, dtype=torch.float64, device=x.device) for name in names}
    for lo in range(0, n * c, 1 << 27):
        hi = min(n * c, lo + (1 << 27))
        f = _exact_keep(st, lo, hi)
        outs["y"][lo:hi] = f * x.reshape(-1)[lo:hi].double()
        if st["residual"] is not None:
            outs["y"][lo:hi] += st["residual"].reshape(-1)[lo:hi].double()
        if st["train"]:
            outs["dx"][lo:hi] = f * st["dy"].reshape(-1)[lo:hi].double()
    return {name: t.view(n, c) for name, t in outs.items()}


def _exact_norm(st):
    x, res, train = st["x"], st["residual"], st["train"]
    n, c = x.shape
    dev = x.device
    names = (["s"] if res is not None else []) + ["y"] + (["dx"] if train else []) + (["dresidual"] if train and res is not None else [])
    outs = {name: torch.empty(n, c, dtype=torch.float64, device=dev) for name in names}
    w = torch.ones(c, dtype=torch.float64, device=dev) if st["weight"] is None else st["weight"].double()
    b = torch.zeros(c, dtype=torch.float64, device=dev) if st["bias"] is None else st["bias"].double()
    dw, db = torch.zeros_like(w), torch.zeros_like(b)
    step = max(8, (1 << 27) // c // 8 * 8)
    for lo in range(0, n, step):
        hi = min(n, lo + step)
        f = _exact_keep(st, lo * c, hi * c).view(hi - lo, c)
        s = f * x[lo:hi].double()
        if res is not None:
            s += res[lo:hi].double()
            outs["s"][lo:hi] = s
        var, mean = torch.var_mean(s, 1, correction=0, keepdim=True)
        sigma = (var + EPS).sqrt()
        z = (s - mean) / sigma
        outs["y"][lo:hi] = z * w + b
        if train:
            up = st["dy"][lo:hi].double()
            dw += (up * z).sum(0)
            db += up.sum(0)
            t = up * w
            # the part of t that moves neither the row's mean nor its size
            d = (t - t.sum(1, keepdim=True) / c - z * ((t * z).sum(1, keepdim=True) / c)) / sigma
            if res is not None:
                d += st["ds"][lo:hi].double()
                outs["dresidual"][lo:hi] = d
            outs["dx"][lo:hi] = f * d
    if train and st["weight"] is not None:
        outs.update(dweight=dw, dbias=db)
    return outs


def _doubling(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 0 from zero, each round reaching twice as far back."""
    a, b, reach = a.clone(), b.clone(), 1
    while reach < len(a):
        b[reach:] = b[reach:] + a[reach:] * b[:-reach]
        a[reach:] = a[reach:] * a[:-reach]
        reach *= 2
    return b


def _exact_scan(st):
    case, lens = st["case"], st["lens"]
    n, c = st["x"].shape
    dev, train, mix = st["x"].device, st["train"], case["form"] == "mix"
    names = ["y"] + (["dx", "dgate"] if train else [])
    outs = {name: torch.zeros(n, c, dtype=torch.float64, device=dev) for name in names}
    h0 = torch.zeros(len(lens), c, dtype=torch.float64, device=dev) if st["h0"] is None else st["h0"].double()
    outs["last"] = h0.clone()
    dh0 = torch.zeros_like(h0) if not train or st["dlast"] is None else st["dlast"].double()
    wide = max(1, (1 << 27) // max(max(lens), 1))
    at = 0
    for s, m in enumerate(lens):
        for c0 in range(0, c if m else 0, wide):
            cols = slice(c0, min(c, c0 + wide))
            order = torch.arange(at, at + m, device=dev)
            if case["reverse"]:
                order = order.flip(0)
            x, a = st["x"][order, cols].double(), 1.0 / (1.0 + torch.exp(-st["gate"][order, cols].double()))
            b = (1.0 - a) * x if mix else x.clone()
            b[0] += a[0] * h0[s, cols]
            h = _doubling(a, b)
            outs["y"][order, cols] = h
            outs["last"][s, cols] = h[-1]
            if train:
                up = st["dy"][order, cols].double()
                if st["dlast"] is not None:
                    up[-1] += st["dlast"][s, cols].double()
                d = _doubling(torch.cat([a[1:], a[:1]]).flip(0), up.flip(0)).flip(0)
                prev = torch.cat([h0[s, cols][None], h[:-1]])
                outs["dx"][order, cols] = d * (1.0 - a) if mix else d
                outs["dgate"][order, cols] = d * (prev - x if mix else prev) * a * (1.0 - a)
                dh0[s, cols] = a[0] * d[0]
        at += m
    if train and st["h0"] is not None:
        outs["dh0"] = dh0
    return outs


def _exact_window(st):
    q, k, v = st["q"], st["k"], st["v"]
    (nq, hq, dim), (nk, hk) = q.shape, k.shape[:2]
    dev, g, scale = q.device, hq // hk, st["scale"]
    left, right, sinks = _bounds(st["case"])
    out, dq = (torch.zeros(nq, hq, dim, dtype=torch.float64, device=dev) for _ in range(2))
    dk, dv = (torch.zeros(nk, hk, dim, dtype=torch.float64, device=dev) for _ in range(2))
    lse = torch.full((hq, nq), float("-inf"), dtype=torch.float64, device=dev)
    q_at = kv_at = 0
    for lq, lk in zip(st["q_lens"], st["kv_lens"]):
        every = torch.arange(lk, device=dev)
        if st["kv_mask"] is not None:
            every = every[st["kv_mask"][kv_at:kv_at + lk]]
        places = every.tolist() if lk < 4096 else None
        at = 0
        while at < lq:
            end = min(lq, at + 2048)
            t = torch.arange(at, end, device=dev) + (lk - lq)
            t0, t1 = at + lk - lq, end - 1 + lk - lq
            if places is None:
                some = every[((every >= t0 - left) | (every < sinks)) & (every <= t1 + right)]
            else:
                some = torch.tensor([j for j in places if (j >= t0 - left or j < sinks) and j <= t1 + right], dtype=torch.int64, device=dev)
            apart = some[None, :] - t[:, None]
            hidden = (apart > right) | ((apart < -left) & (some >= sinks)[None, :])
            rows = slice(q_at + at, q_at + end)
            for h in range(hq if len(some) else 0):
                kh, vh, qh = k[kv_at + some, h // g].double(), v[kv_at + some, h // g].double(), q[rows, h].double()
                s = (qh @ kh.t().contiguous() * scale).masked_fill_(hidden, float("-inf"))
                z = torch.logsumexp(s, 1)
                lse[h, rows] = z
                p = torch.nan_to_num((s - z[:, None]).exp(), nan=0.0)  # a row that sees no key: -inf - -inf
                out[rows, h] = p @ vh
                if st["train"]:
                    up = st["dout"][rows, h].double()
                    dv[kv_at + some, h // g] += p.t() @ up
                    d = p * (up @ vh.t().contiguous() - (up * out[rows, h]).sum(1, keepdim=True)) * scale
                    dq[rows, h] = d @ kh
                    dk[kv_at + some, h // g] += d.t() @ qh
            at = end
        q_at, kv_at = q_at + lq, kv_at + lk
    outs = {"out": out, "lse": lse}
    if st["train"]:
        outs.update(dq=dq, dk=dk, dv=dv)
    return outs


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    outs = {"window_attention": _exact_window, "gated_scan": _exact_scan, "layer_norm": _exact_norm, "dropout": _exact_dropout}[op](st)
    return {name: outs[name] for name in _NAMES if name in outs}
