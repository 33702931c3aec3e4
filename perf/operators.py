"""Measured cases of the voxel-attention operators: the queries' and keys' norm with position rotation, and cross attention.

``own`` is False: ``run`` computes an operator from elementary torch operations in 32 bits, rounded once at the end.
``own`` is True: ``run`` makes the calls of ``sparse_submanifold_convolution_amd`` that a program makes.  Both take the
state that ``prepare`` builds.  ``exact`` restates the operators in 64 bits, sample by sample and head by head.

Operators (formulas; D = head dimension, all sums in at least 32 bits):

qk_norm_rope   y = R(pos) (x * rsqrt(mean(x^2) + eps) * w) for every head of the queries and of the keys, where R turns
               pair j of the head by 2 pi * turns[j] * pos[axis[j]]; its backward gives dx and dw.
cross_attention  rows of sample b attend that sample's encoder rows: out = softmax(scale q k^T) v over the keys whose mask
               is set, with query heads sharing key heads in groups; a row with no key gives zeros and lse = -inf.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6
THETA = 10000.0


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------

def _rope(n, heads_q, heads_kv, dim, dtype, pairs, layout="interleaved", weight="shared", packed=False, train=False, side=64):
    return {"op": "qk_norm_rope", "n": n, "heads_q": heads_q, "heads_kv": heads_kv, "dim": dim, "dtype": dtype, "axis_pairs": pairs,
            "layout": layout, "weight": weight, "packed": packed, "train": train, "side": side}


def _attn(q_lens, kv_lens, heads_q, heads_kv, dim, dtype, mask="none", packed=False, train=False):
    return {"op": "cross_attention", "q_lens": ",".join(map(str, q_lens)), "kv_lens": ",".join(map(str, kv_lens)), "heads_q": heads_q,
            "heads_kv": heads_kv, "dim": dim, "dtype": dtype, "mask": mask, "packed": packed, "train": train}


def listed():
    return [
        # the pooled query token of one object while serving: a single row, where the call's latency is all there is
        dict(_rope(1, 4, 4, 64, "bf16", "10,10,10"), name="rope one row"),
        # the 32^3 shell workload's 1,872 rows in fp32, odd head size, grouped keys, halves layout, training
        dict(_rope(1872, 6, 2, 40, "f32", "6,7,7", layout="halves", weight="head", train=True, side=32), name="rope 32^3 train f32"),
        # the 2 x 64^3 shells workload's rows, read from a packed query/key/value projection of 256 channels
        dict(_rope(22417, 4, 4, 64, "f16", "10,11,11", weight="head", packed=True), name="rope 64^3 packed"),
        # the 128^3 random-occupancy workload's rows at its 1,024 channels, training: the largest streaming case
        dict(_rope(629000, 16, 16, 64, "bf16", "10,10,10", weight="head", train=True, side=128), name="rope 128^3 train"),
        # one query row over a short encoder sequence (16 x 16 patches and a class token): serving latency
        dict(_attn([1], [257], 8, 2, 64, "f16"), name="attn one query"),
        # attention pooling while serving: one query token per sample over all voxels of the 4 x 256^3 shells
        dict(_attn([1, 1, 1, 1], [199911, 203045, 185530, 211026], 4, 4, 64, "bf16"), name="attn pool 256^3"),
        # voxels of the 2 x 64^3 shells reading padded encoder states (masked tail), inference
        dict(_attn([11302, 11115], [257, 257], 4, 4, 64, "f16", mask="tail"), name="attn cross 64^3"),
        # training: voxels of the 4 x 256^3 shells at their 256 channels reading 32 x 32 patches and a class token
        dict(_attn([199911, 203045, 185530, 211026], [1025, 1025, 1025, 1025], 4, 4, 64, "bf16", train=True), name="attn cross 256^3 train"),
        # training: self attention among the voxels of each 64^3 sample at 1,024 channels
        dict(_attn([11302, 11115], [11302, 11115], 16, 16, 64, "bf16", train=True), name="attn self 64^3 train"),
        # ragged batch in fp32 with empty samples, an all-masked one, grouped heads and an odd head size, training
        dict(_attn([700, 0, 333, 1, 838], [77, 129, 0, 513, 1], 6, 2, 40, "f32", mask="random", train=True), name="attn ragged train f32"),
        # inference with wide heads over a long encoder sequence (several views)
        dict(_attn([22417], [4099], 8, 8, 128, "f16"), name="attn wide heads"),
        # latent queries pooling the voxels of each 64^3 sample, training: few rows, long key axis
        dict(_attn([16, 16, 15], [11302, 11115, 9001], 8, 4, 96, "bf16", mask="tail", packed=True, train=True), name="attn latents train"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_rope(rng):
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    dim = rng.choice([32, 40, 48, 64, 64, 72, 80, 96, 128])
    heads_kv = rng.choice([1, 2, 3, 4, 8, 16])
    heads_q = heads_kv * rng.choice([1, 1, 2, 3])
    layout = rng.choice(["interleaved", "interleaved", "halves"])
    axes = rng.choice([1, 2, 3, 3, 3])
    step = 1 if layout == "interleaved" else (4 if dtype == "f32" else 8)  # halves: whole 16-byte vectors
    total = dim // 2 // step * step
    if layout == "interleaved" and rng.random() < 0.5:
        total = dim // 2 // axes * axes
    pairs = [total // axes] * axes
    pairs[-1] += total - sum(pairs)
    most = max(1, int(629000 * 2 * 16 * 64 * 2 / ((heads_q + heads_kv) * dim * (4 if dtype == "f32" else 2))))
    return _rope(_log(rng, 1, min(629000, most)), heads_q, heads_kv, dim, dtype, ",".join(map(str, pairs)), layout,
                 rng.choice(["none", "shared", "head", "head"]), rng.random() < 0.4, rng.random() < 0.5,
                 rng.choice([32, 64, 128, 256, 1024, 1 << 20]))


def _draw_attn(rng):
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    dim = rng.choice([32, 40, 48, 64, 64, 72, 80, 96, 128])
    heads_kv = rng.choice([1, 2, 4, 8])
    heads_q = heads_kv * rng.choice([1, 1, 2, 4])
    samples = rng.choice([1, 2, 3, 4, 7])
    form = rng.choice(["few", "cross", "cross", "self"])
    mask = rng.choice(["none", "none", "tail", "random"])
    train = rng.random() < 0.5
    q_max, kv_max = {"few": (16, 200000), "cross": (200000, 1025), "self": (11000, 11000)}[form]
    q_hi, kv_hi = _log(rng, 1, q_max), _log(rng, 16, kv_max)
    if form == "self":
        q_hi = kv_hi
    # no more than half of the largest listed case's products, and for fp32 a quarter of that
    most = 2.0e11 / (heads_q * dim) * (0.25 if dtype == "f32" else 1.0)
    while samples * q_hi * kv_hi > most:
        q_hi, kv_hi = max(1, int(q_hi * 0.8)), max(16, int(kv_hi * (0.8 if form == "self" else 0.9)))
    kv_lens = [max(1, int(kv_hi * rng.uniform(0.6, 1.0))) for _ in range(samples)]
    q_lens = kv_lens if form == "self" else [max(1, int(q_hi * rng.uniform(0.7, 1.0))) for _ in range(samples)]
    if samples > 2 and rng.random() < 0.4:
        kv_lens = [0] + kv_lens[1:]
    if samples > 2 and rng.random() < 0.4:
        q_lens = q_lens[:-1] + [0]
    return _attn(q_lens, kv_lens, heads_q, heads_kv, dim, dtype, mask, rng.random() < 0.4, train)


def _sizes(case):
    yield from (case["heads_q"] * case["dim"], case["heads_kv"] * case["dim"], (case["heads_q"] + 2 * case["heads_kv"]) * case["dim"])
    yield from ([case["n"]] if "n" in case else _ints(case["q_lens"]) + _ints(case["kv_lens"]))


def draw(rng):
    while True:
        case = _draw_rope(rng) if rng.random() < 0.4 else _draw_attn(rng)
        if 3072 not in _sizes(case):
            return case


def _ints(text):
    return [int(v) for v in text.split(",")]


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------

def _shell_positions(n, side, gen, dev):
    """Voxel coordinates (b, x, y, z) near the surface of an ellipsoid in a side^3 grid: the rows a sparse network holds."""
    d = torch.randn(n, 3, generator=gen, device=dev, dtype=torch.float32)
    d = d / d.norm(dim=1, keepdim=True).clamp_min(1e-6)
    axes = torch.tensor([0.45, 0.38, 0.30], device=dev)
    xyz = ((0.5 + d * axes) * (side - 1)).round().to(torch.int32).clamp_(0, side - 1)
    return torch.cat([torch.zeros(n, 1, dtype=torch.int32, device=dev), xyz], dim=1).contiguous()


def _heads(n, heads, dim, gen, dev, dtype, centres=None):
    """Rows of `heads` vectors, scattered around a few directions as a trained projection's are."""
    x = torch.empty(n, heads, dim, device=dev, dtype=dtype)
    for lo in range(0, n, 1 << 17):
        hi = min(n, lo + (1 << 17))
        y = torch.randn(hi - lo, heads, dim, generator=gen, device=dev)
        if centres is not None:
            y += centres[torch.randint(0, centres.shape[0], (hi - lo,), generator=gen, device=dev)]
        x[lo:hi] = y.to(dtype)
    return x


def _pack(parts):
    """The same values as views of one packed projection [n, heads of all parts, dim]."""
    whole = torch.cat(parts, dim=1)
    at, views = 0, []
    for p in parts:
        views.append(whole[:, at:at + p.shape[1]])
        at += p.shape[1]
    return views


def prepare(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    hq, hk, dim = case["heads_q"], case["heads_kv"], case["dim"]
    st = {"case": case, "op": case["op"], "train": case["train"], "dtype": dtype}
    if case["op"] == "qk_norm_rope":
        n = case["n"]
        st["positions"] = _shell_positions(n, case["side"], gen, dev)[:, 1:1 + len(_ints(case["axis_pairs"]))]
        q, k = (_heads(n, h, dim, gen, dev, dtype) for h in (hq, hk))
        if case["packed"]:
            q, k, _ = _pack([q, k, _heads(n, hk, dim, gen, dev, dtype)])
        st["q"], st["k"] = q, k
        pairs = _ints(case["axis_pairs"])
        st["turns"] = torch.tensor([THETA ** (-j / m) / (2 * math.pi) for m in pairs for j in range(m)], dtype=torch.float64, device=dev)
        st["axis"] = torch.tensor([a for a, m in enumerate(pairs) for _ in range(m)], dtype=torch.int32, device=dev)
        st["layout"] = case["layout"]
        for name, h in (("q_weight", hq), ("k_weight", hk)):
            shape = {"none": None, "shared": (dim,), "head": (h, dim)}[case["weight"]]
            st[name] = None if shape is None else (1 + 0.2 * torch.randn(shape, generator=gen, device=dev)).to(dtype)
        if case["train"]:
            st["dq"], st["dk"] = (_heads(n, h, dim, gen, dev, dtype) for h in (hq, hk))
        return st
    q_lens, kv_lens = _ints(case["q_lens"]), _ints(case["kv_lens"])
    nq, nk = sum(q_lens), sum(kv_lens)
    # keys and queries share a few directions: some scores stand out, as after training
    centres = 0.8 * torch.randn(24, 1, dim, generator=gen, device=dev)
    q, k = (_heads(n, h, dim, gen, dev, dtype, centres) for n, h in ((nq, hq), (nk, hk)))
    v = _heads(nk, hk, dim, gen, dev, dtype)
    st["kv_mask"] = None
    if case["mask"] != "none":
        keep = torch.ones(nk, dtype=torch.bool, device=dev)
        at = 0
        for b, m in enumerate(kv_lens):
            if case["mask"] == "tail":
                part = torch.arange(m, device=dev) < torch.randint(m // 2, m + 1, (1,), generator=gen, device=dev)
            else:
                part = torch.rand(m, generator=gen, device=dev) < 0.8
            keep[at:at + m] = part
            if b == 1 and len(kv_lens) > 2:
                keep[at:at + m] = False  # a sample whose keys are all masked
            at += m
        st["kv_mask"] = keep
        # padding rows hold whatever was in memory
        k[~keep] = float("nan")
        v[~keep] = float("inf")
    if case["packed"]:
        k, v = _pack([k, v])
    st["q"], st["k"], st["v"] = q, k, v
    for name, lens in (("q_offsets", q_lens), ("kv_offsets", kv_lens)):
        st[name] = torch.tensor([sum(lens[:b]) for b in range(len(lens) + 1)], dtype=torch.int32, device=dev)
    st["q_lens"], st["kv_lens"] = q_lens, kv_lens
    st["scale"] = 1.0 / math.sqrt(dim)
    if case["train"]:
        st["dout"] = 0.1 * _heads(nq, hq, dim, gen, dev, dtype)
    return st


# ---------------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------------

def _cos_sin(st):
    """[n, 1, P] cosine and sine of every pair's angle: the turns are reduced in 64 bits, where far positions keep their phase."""
    t = st["positions"].to(torch.float64)[:, st["axis"].long()] * st["turns"]
    t = ((t - t.round()) * (2 * math.pi)).to(torch.float32)
    return t.cos()[:, None], t.sin()[:, None]


def _rotate(x, cos, sin, layout):
    """Pairs are (2j, 2j + 1) of a head (interleaved) or (j, j + P) (halves); dimensions past the pairs stay."""
    p = cos.shape[-1]
    if layout == "interleaved":
        a, b = x[..., 0:2 * p:2], x[..., 1:2 * p:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    else:
        a, b = x[..., :p], x[..., p:2 * p]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    return torch.cat([turned, x[..., 2 * p:]], dim=-1)


def _in_order(outs):
    return {name: outs[name] for name in ("q", "k", "dq", "dk", "q_weight_grad", "k_weight_grad") if name in outs}


def _plain_rope(st):
    cos, sin = _cos_sin(st)
    outs = {}
    for name in ("q", "k"):
        x = st[name].float()
        w = st[name + "_weight"]
        wf = 1.0 if w is None else w.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        outs[name] = _rotate(x * r * wf, cos, sin, st["layout"]).to(st["dtype"])
        if st["train"]:
            g = _rotate(st["d" + name].float(), cos, -sin, st["layout"])
            xn = x * r
            if w is not None:
                dw = (g * xn).sum(dim=(0, 1) if w.dim() == 1 else 0)
                outs[name + "_weight_grad"] = dw.to(st["dtype"])
            gw = g * wf
            outs["d" + name] = ((gw - xn * (gw * xn).mean(-1, keepdim=True)) * r).to(st["dtype"])
    return _in_order(outs)


def _sample_rows(offsets, lens, n, dev):
    """Row numbers [B, longest] (clamped), their truth [B, longest], and each row's sample and place."""
    longest = max(max(lens), 1)
    place = torch.arange(longest, device=dev)
    start, end = offsets[:-1, None].long(), offsets[1:, None].long()
    rows = start + place
    row = torch.arange(n, device=dev)
    sample = torch.bucketize(row, offsets[1:].long(), right=True)
    return rows.clamp(max=max(n - 1, 0)), rows < end, sample, row - offsets[:-1].long()[sample]


def _plain_attention(st):
    q, k, v, dev = st["q"], st["k"], st["v"], st["q"].device
    (nq, hq, dim), (nk, hk) = q.shape, k.shape[:2]
    g = hq // hk
    batch = len(st["q_lens"])
    qr, _, q_sample, q_place = _sample_rows(st["q_offsets"], st["q_lens"], nq, dev)
    kr, k_ok, k_sample, k_place = _sample_rows(st["kv_offsets"], st["kv_lens"], nk, dev)
    if st["kv_mask"] is not None:
        k_ok = k_ok & st["kv_mask"][kr]
    lq, lk = qr.shape[1], kr.shape[1]

    def by_query(x):  # [n, Hq, D] -> [B, Hk, G * Lq, D]
        return x[qr].float().view(batch, lq, hk, g, dim).permute(0, 2, 3, 1, 4).reshape(batch, hk, g * lq, dim)

    def from_query(x):  # back to rows
        return x.view(batch, hk, g, lq, -1)[q_sample, :, :, q_place].reshape(nq, hq, -1)

    def by_key(x):  # masked rows are left out whatever they hold
        return torch.where(k_ok[:, :, None, None], x[kr].float(), 0.0).permute(0, 2, 1, 3).contiguous()

    qf, kf, vf = by_query(q), by_key(k), by_key(v)
    s = torch.matmul(qf, kf.transpose(2, 3)).mul_(st["scale"])
    s.masked_fill_(~k_ok[:, None, None, :], float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    some = total > 0
    p.mul_(torch.where(some, 1.0 / total, 0.0))
    o = torch.matmul(p, vf)
    lse = torch.where(some, m + total.log(), float("-inf"))
    outs = {"out": from_query(o).to(st["dtype"]), "lse": from_query(lse)[..., 0].t().contiguous()}
    if not st["train"]:
        return outs
    do = by_query(st["dout"])
    # rows past a sample's end stand for no query: they add nothing to the keys' gradients
    do = do * (torch.arange(lq, device=dev) < (st["q_offsets"][1:, None] - st["q_offsets"][:-1, None])).repeat(1, g)[:, None, :, None]
    dv = torch.matmul(p.transpose(2, 3), do)
    ds = torch.matmul(do, vf.transpose(2, 3)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(st["scale"])
    outs["dq"] = from_query(torch.matmul(ds, kf)).to(st["dtype"])
    dk = torch.matmul(ds.transpose(2, 3), qf)
    for name, x in (("dk", dk), ("dv", dv)):
        outs[name] = torch.where(k_ok[:, None, :, None], x, 0.0)[k_sample, :, k_place].to(st["dtype"])
    return outs


# ---------------------------------------------------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------------------------------------------------

def _own_rope(st):
    import sparse_submanifold_convolution_amd as ssc
    table = ssc.RopeTable(st["turns"], st["axis"])
    w = {"q_weight": st["q_weight"], "k_weight": st["k_weight"], "eps": EPS, "layout": st["layout"]}
    q, k = ssc.qk_norm_rope_fwd(st["q"], st["k"], st["positions"], table, **w)
    outs = {"q": q, "k": k}
    if st["train"]:
        dq, dk, dqw, dkw = ssc.qk_norm_rope_bwd(st["q"], st["k"], st["positions"], table, st["dq"], st["dk"], **w)
        outs.update(dq=dq, dk=dk)
        if dqw is not None:
            outs.update(q_weight_grad=dqw, k_weight_grad=dkw)
    return outs


def _own_attention(st):
    import sparse_submanifold_convolution_amd as ssc
    where = (st["q_offsets"], st["kv_offsets"])
    kw = {"kv_mask": st["kv_mask"], "scale": st["scale"]}
    out, lse = ssc.cross_attention_fwd(st["q"], st["k"], st["v"], *where, **kw)
    outs = {"out": out, "lse": lse}
    if st["train"]:
        dq, dk, dv = ssc.cross_attention_bwd(st["q"], st["k"], st["v"], out, lse, st["dout"], *where, **kw)
        outs.update(dq=dq, dk=dk, dv=dv)
    return outs


def run(state):
    if state["op"] == "qk_norm_rope":
        return _own_rope(state) if own else _plain_rope(state)
    return _own_attention(state) if own else _plain_attention(state)


# ---------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------------

def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    hq, hk, dim = case["heads_q"], case["heads_kv"], case["dim"]
    if case["op"] == "qk_norm_rope":
        n, axes = case["n"], len(_ints(case["axis_pairs"]))
        rows = n * (hq + hk) * dim
        weights = {"none": 0, "shared": 2 * dim, "head": (hq + hk) * dim}[case["weight"]] * size
        # forward: read and write the rows; backward: also the output gradients in and the input gradients out
        streams = 4 if case["train"] else 2
        return {"bytes": streams * rows * size + n * axes * 4 + weights * (2 if case["train"] else 1),
                "flops": rows * (18 if case["train"] else 7)}
    q_lens, kv_lens = _ints(case["q_lens"]), _ints(case["kv_lens"])
    nq, nk = sum(q_lens), sum(kv_lens)
    products = sum(a * b for a, b in zip(q_lens, kv_lens)) * hq * dim * 2
    # forward: q, k, v in, out and lse out; training: dout in and dq, dk, dv out as well
    moved = (2 * nq * hq + 2 * nk * hk) * dim * size + nq * hq * 4 + (nk if case["mask"] != "none" else 0)
    if case["train"]:
        moved += (2 * nq * hq + 2 * nk * hk) * dim * size
    return {"bytes": moved, "flops": products * (7 if case["train"] else 2)}


# ---------------------------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------------------------------

def _exact_rope(st):
    case = st["case"]
    pairs = _ints(case["axis_pairs"])
    total, dim = sum(pairs), case["dim"]
    pos = st["positions"].double()
    angles = torch.cat([pos[:, a:a + 1] * (THETA ** (-torch.arange(m, dtype=torch.float64, device=pos.device) / m))
                        for a, m in enumerate(pairs) if m], dim=1)
    turn = torch.polar(torch.ones_like(angles), angles)[:, None]  # [n, 1, P] complex
    first = torch.arange(total, device=pos.device) * (2 if case["layout"] == "interleaved" else 1)
    second = first + (1 if case["layout"] == "interleaved" else total)

    def rotated(x, by):
        z = torch.complex(x[..., first], x[..., second]) * by
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    outs = {}
    for name, heads in (("q", case["heads_q"]), ("k", case["heads_kv"])):
        x = st[name].double()
        w = st[name + "_weight"]
        weight = torch.ones(heads, dim, dtype=torch.float64, device=x.device) if w is None else w.double().expand(heads, dim)
        rms = ((x ** 2).sum(-1, keepdim=True) / dim + EPS).sqrt()
        outs[name] = rotated(x / rms * weight, turn)
        if st["train"]:
            up = rotated(st["d" + name].double(), turn.conj())
            if w is not None:
                dw = torch.einsum("nhd,nhd->hd", up, x / rms)
                outs[name + "_weight_grad"] = dw if w.dim() == 2 else dw.sum(0)
            inner = (up * weight * x).sum(-1, keepdim=True)
            outs["d" + name] = up * weight / rms - x * inner / (dim * rms ** 3)
    return _in_order(outs)


def _exact_attention(st):
    q, k, v = st["q"], st["k"], st["v"]
    (nq, hq, dim), (nk, hk) = q.shape, k.shape[:2]
    dev, g, scale = q.device, hq // hk, st["scale"]
    out, dq = (torch.zeros(nq, hq, dim, dtype=torch.float64, device=dev) for _ in range(2))
    dk, dv = (torch.zeros(nk, hk, dim, dtype=torch.float64, device=dev) for _ in range(2))
    lse = torch.full((hq, nq), float("-inf"), dtype=torch.float64, device=dev)
    q_at = kv_at = 0
    for lq, lk in zip(st["q_lens"], st["kv_lens"]):
        keys = torch.arange(kv_at, kv_at + lk, device=dev)
        if st["kv_mask"] is not None:
            keys = keys[st["kv_mask"][keys]]
        step = max(1, (1 << 28) // max(1, len(keys)))
        for h in range(hq if len(keys) else 0):
            kh, vh = k[keys, h // g].double(), v[keys, h // g].double()
            for lo in range(q_at, q_at + lq, step):
                hi = min(lo + step, q_at + lq)
                qh = q[lo:hi, h].double()
                s = qh @ kh.t().contiguous() * scale
                z = torch.logsumexp(s, 1)
                lse[h, lo:hi] = z
                p = (s - z[:, None]).exp()
                del s
                out[lo:hi, h] = p @ vh
                if st["train"]:
                    up = st["dout"][lo:hi, h].double()
                    dv[keys, h // g] += p.t() @ up
                    d = p * (up @ vh.t().contiguous() - (up * out[lo:hi, h]).sum(1, keepdim=True)) * scale
                    dq[lo:hi, h] = d @ kh
                    dk[keys, h // g] += d.t() @ qh
        q_at, kv_at = q_at + lq, kv_at + lk
    outs = {"out": out, "lse": lse}
    if st["train"]:
        outs.update(dq=dq, dk=dk, dv=dv)
    return outs


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_rope(st) if case["op"] == "qk_norm_rope" else _exact_attention(st)
