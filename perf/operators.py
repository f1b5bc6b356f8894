"""Cases of the training-block operators over voxel features: layer norm, 8-bit activation checkpoints and
cross attention to an encoder's states. Row counts are those of this package's workloads (a 7,130-voxel
shell, a LiDAR frame of about 43 thousand voxels, bands and boxes of millions), channels those of its
layers (8 to 256)."""
import math

import torch

own = False

GROUP = 64  # channels that share a checkpoint scale
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # The smallest call: the norm after the first fp32 8 -> 8 layer on the shell scene (launch latency).
        {"name": "norm-f32-shell", "op": "norm", "dtype": "f32", "rows": 7130, "channels": 8},
        # A norm between two 64-channel layers of a narrow band, an odd number of rows.
        {"name": "norm-bf16-band", "op": "norm", "dtype": "bf16", "rows": 2000003, "channels": 64},
        # Its gradient in the widest layer of a large scene (the most bytes of all cases).
        {"name": "norm-grad-bf16-large", "op": "norm_grad", "dtype": "bf16", "rows": 4000037, "channels": 256},
        # fp32 features of the dense boxes packed after the forward pass and restored in the backward pass.
        {"name": "pack-f32-boxes", "op": "pack", "dtype": "f32", "rows": 4100003, "channels": 16},
        # A block's norm that keeps its normalised input in 8 bits ...
        {"name": "norm8-bf16-band", "op": "norm8", "dtype": "bf16", "rows": 2000003, "channels": 128},
        # ... and that norm's backward pass.
        {"name": "norm8-grad-bf16-band", "op": "norm8_grad", "dtype": "bf16", "rows": 2000003, "channels": 128},
        # Weight gradient of a 128 -> 128 convolution over a LiDAR-sized scene from the 8-bit input.
        {"name": "conv8-wgrad-lidar", "op": "conv8", "dtype": "bf16", "side": 208, "cin": 128, "cout": 128},
        # One query token for each of 64 sequences over ragged states (serving: reads the states once).
        {"name": "attn-bf16-token", "op": "attn", "dtype": "bf16", "batch": 64, "queries": 64, "keys": 262147,
         "skew": 1.5, "heads": 8, "kv_heads": 8, "dim": 64, "masked": 0.0},
        # Object queries over one frame's voxels in fp32: few rows, a long axis.
        {"name": "attn-f32-objects", "op": "attn", "dtype": "f32", "batch": 1, "queries": 300, "keys": 43217,
         "skew": 0.0, "heads": 8, "kv_heads": 8, "dim": 32, "masked": 0.0},
        # The voxels of five frames attending to five sets of image states of differing lengths.
        {"name": "attn-bf16-frames", "op": "attn", "dtype": "bf16", "batch": 5, "queries": 215003, "keys": 5120,
         "skew": 0.4, "heads": 4, "kv_heads": 4, "dim": 64, "masked": 0.0},
        # Training on three scenes, padded states masked out, pairs of query heads on one key head.
        {"name": "attn-grad-bf16-scenes", "op": "attn_grad", "dtype": "bf16", "batch": 3, "queries": 100003, "keys": 2400,
         "skew": 0.5, "heads": 4, "kv_heads": 2, "dim": 64, "masked": 0.1},
        # A small fp32 scene against a short text, sizes that fill no tile.
        {"name": "attn-grad-f32-short", "op": "attn_grad", "dtype": "f32", "batch": 2, "queries": 7130, "keys": 141,
         "skew": 0.3, "heads": 2, "kv_heads": 2, "dim": 40, "masked": 0.0},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "norm_grad", "pack", "norm8", "norm8_grad", "conv8", "token", "attn", "attn_grad"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("norm", "norm_grad", "pack", "norm8", "norm8_grad"):
        channels = rng.choice([log(3, 1024), 8 * log(1, 64), rng.choice([8, 16, 32, 64, 128, 256])])
        rows = log(50, min(3000000, 400000000 // channels))
        # The checkpoint of a normalised row is a computed value rounded to 8 bits: in bf16, where one step
        # of a code weighs as little as the output's own rounding.
        return {"op": op, "dtype": "bf16" if op == "norm8" else dtype, "rows": rows, "channels": channels}
    if op == "conv8":
        return {"op": op, "dtype": "bf16", "side": rng.randint(24, 208), "cin": rng.choice([32, 64, 128]),
                "cout": rng.choice([64, 128])}
    kv_heads = rng.choice([1, 2, 4])
    case = {"op": "attn_grad" if op == "attn_grad" else "attn", "dtype": dtype, "batch": rng.randint(1, 6), "skew": rng.uniform(0, 0.8),
            "heads": kv_heads * rng.choice([1, 1, 2]), "kv_heads": kv_heads, "dim": rng.choice([16, 32, 40, 64, 96, 128]),
            "masked": rng.choice([0.0, 0.0, 0.2])}
    if op == "token":
        case["batch"] = case["queries"] = rng.randint(1, 64)
        case["keys"] = case["batch"] * log(16, 4096)
    else:
        case["queries"] = case["batch"] * log(20, 20000)
        case["keys"] = case["batch"] * log(10, 1500)
    return case


def lengths(total, parts, skew):
    """`parts` lengths of the sum `total`, the longest up to 1 + skew times the mean or so."""
    w = [1.0 + skew * (((7 * i + 3) % parts) / max(1, parts - 1) - 0.5) for i in range(parts)]
    got = [int(total * x / sum(w)) for x in w]
    got[-1] += total - sum(got)
    return got


def pairs(case):
    """Query-key pairs of all sequences, masked keys left out."""
    lq, lk = lengths(case["queries"], case["batch"], case["skew"]), lengths(case["keys"], case["batch"], -case["skew"])
    return (1.0 - case["masked"]) * sum(a * b for a, b in zip(lq, lk))


def work(case):
    op, es = case["op"], 4 if case["dtype"] == "f32" else 2
    if op.startswith("attn"):
        nq, nk = case["queries"] * case["heads"] * case["dim"], case["keys"] * case["kv_heads"] * case["dim"]
        flops = pairs(case) * case["heads"] * case["dim"] * (4 if op == "attn" else 10)
        moved = (2 * nq + 2 * nk) * es if op == "attn" else (4 * nq + 4 * nk) * es
        return {"bytes": moved + 4 * case["queries"] * case["heads"], "flops": flops}
    if op == "conv8":
        n, cin, cout = case["side"] ** 2, case["cin"], case["cout"]
        # About 8.6 of the 27 offsets of a sheet's voxel lead to a voxel.
        return {"bytes": n * (cin + 4 * -(-cin // GROUP) + 2 * cout + 27 * 4) + 27 * cin * cout * 4, "flops": 2 * 8.6 * n * cin * cout}
    n, c = case["rows"], case["channels"]
    scales = 4 * n * -(-c // GROUP)
    moved = {"norm": 2 * n * c * es + 8 * n, "norm_grad": 3 * n * c * es + 8 * n, "pack": 2 * (n * c * (es + 1) + scales),
             "norm8": n * c * (2 * es + 1) + scales + 4 * n + n * c * es + n * c + scales,
             "norm8_grad": n * c * (2 * es + 1) + scales + 4 * n}[op]
    return {"bytes": moved + 2 * c * es, "flops": n * c * {"norm": 8, "norm_grad": 14, "pack": 6, "norm8": 13, "norm8_grad": 14}[op]}


# ----------------------------------------------------------------------------------------- inputs

def sheet(side, gen):
    """Voxels of a rough height field over side x side columns, in the grid's row order, and the
    27-offset neighbour map over them (-1: no voxel there)."""
    u = torch.arange(side, device="cuda")
    ph = torch.rand(4, generator=gen, device="cuda") * 6.28
    i, j = [t.reshape(-1) for t in torch.meshgrid(u, u, indexing="ij")]
    z = 40 + 12 * torch.sin(i * 0.05 + ph[0]) + 12 * torch.cos(j * 0.07 + ph[1]) + 3 * torch.sin((i + j) * 0.11 + ph[2])
    k = z.round().long()
    up = ((i >> 7) << 10) | ((j >> 7) << 5) | (k >> 7)
    low = ((i >> 3 & 15) << 8) | ((j >> 3 & 15) << 4) | (k >> 3 & 15)
    order = ((up << 21) | (low << 9) | ((i & 7) << 6) | ((j & 7) << 3) | (k & 7)).argsort()
    ijk = torch.stack([i, j, k], 1)[order]
    code = ((ijk[:, 0] + 1) * 1024 + ijk[:, 1] + 1) * 1024 + ijk[:, 2] + 1
    by_code, row = code.sort()
    d = torch.tensor([-1, 0, 1], device="cuda")
    off = torch.stack(torch.meshgrid(d, d, d, indexing="ij"), -1).reshape(27, 3)
    want = code + (off[:, 0:1] * 1024 + off[:, 1:2]) * 1024 + off[:, 2:3]
    at = torch.searchsorted(by_code, want).clamp(max=code.numel() - 1)
    return ijk.int().contiguous(), torch.where(by_code[at] == want, row[at], -1).int().contiguous()


def packed(x):
    """8-bit codes and scales of float32 rows."""
    n, c = x.shape
    g = -(-c // GROUP)
    x = torch.nn.functional.pad(x, (0, g * GROUP - c)).view(n, g, GROUP)
    a = x.abs().amax(2, keepdim=True)
    small = a < 2.0 ** -100
    inv = torch.where(small, 0.0, 127.0 / a)
    codes = torch.round(x * inv).to(torch.int8).view(n, g * GROUP)[:, :c].contiguous()
    return codes, torch.where(small, 0.0, a / 127.0).view(n, g)


def restored(codes, scales):
    return codes.float() * scales.repeat_interleave(GROUP, 1)[:, :codes.shape[1]]


def inputs(case, seed):
    """The tensors a case works on, all on the GPU."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std)

    if op.startswith("attn"):
        lq, lk = lengths(case["queries"], case["batch"], case["skew"]), lengths(case["keys"], case["batch"], -case["skew"])
        s = {"lq": max(lq), "lk": max(lk), "scale": case["dim"] ** -0.5,
             "q_offsets": torch.tensor([0] + lq, device="cuda").cumsum(0).int(), "kv_offsets": torch.tensor([0] + lk, device="cuda").cumsum(0).int()}
        s["q"] = normal(case["queries"], case["heads"], case["dim"], std=1.5).to(dt)
        # Keys and values as one projection of the states gives them: two slices of one tensor.
        kv = normal(case["keys"], 2, case["kv_heads"], case["dim"]).to(dt)
        s["k"], s["v"] = kv[:, 0], kv[:, 1]
        s["key_mask"] = torch.rand(case["keys"], generator=gen, device="cuda") >= case["masked"] if case["masked"] else None
        if op == "attn_grad":
            s["dout"] = normal(case["queries"], case["heads"], case["dim"], std=0.1).to(dt)
        return s
    if op == "conv8":
        ijk, kmap = sheet(case["side"], gen)
        codes, scales = packed(torch.relu(normal(ijk.shape[0], case["cin"])).to(dt).float())
        return {"ijk": ijk, "kmap": kmap, "codes": codes, "scales": scales, "dout": normal(ijk.shape[0], case["cout"], std=0.1).to(dt),
                "weights": normal(27, case["cin"], case["cout"], std=0.02).to(dt)}
    n, c = case["rows"], case["channels"]
    x = (normal(n, c) * (0.5 + torch.rand(c, generator=gen, device="cuda")) + normal(c, std=0.3)).to(dt)
    s = {"x": x, "weight": (1 + normal(c, std=0.1)).to(dt), "bias": normal(c, std=0.1).to(dt)}
    if op.endswith("_grad"):
        s["dy"] = normal(n, c, std=0.1).to(dt)
        s["mean"], s["rstd"] = statistics(x.float())
        if op == "norm8_grad":
            s["codes"], s["scales"] = packed((x.float() - s["mean"][:, None]) * s["rstd"][:, None])
            del s["x"], s["mean"]
    return s


def prepare(case, seed):
    s = inputs(case, seed)
    s["op"] = case["op"]
    if case["op"] == "attn_grad":  # what the forward pass left
        s["out"], s["lse"] = attend(s)
    if own:
        import sparse_convolution_amd as igc
        s["igc"] = igc
        if "codes" in s:
            s["ckpt"] = igc.Checkpoint8(s["codes"], s["scales"], DTYPES[case["dtype"]])
        if case["op"] == "conv8":
            s["grid"] = igc.grid_build(s["ijk"])
    return s


# ------------------------------------------------------------------------------------ plain forms

EPS = 1e-5


def statistics(x):
    mean = x.mean(1)
    return mean, 1.0 / torch.sqrt((x - mean[:, None]).square().mean(1) + EPS)


def norm_gradients(dy, xhat, rstd, weight, dt):
    dy = dy.float()
    g = dy * weight.float()
    dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    return dx.to(dt), (dy * xhat).sum(0), dy.sum(0)


def padded(offsets, most, total):
    """Rows [batch, most] of each sequence, and which of them exist."""
    at = offsets[:-1, None].long() + torch.arange(most, device=offsets.device)
    return at.clamp(max=total - 1), at < offsets[1:, None]


def places(offsets, total):
    """(sequence, position) of each packed row."""
    r = torch.arange(total, device=offsets.device)
    b = torch.searchsorted(offsets[1:].long().contiguous(), r, right=True)
    return b, r - offsets[b].long()


def scores(s):
    """Scaled scores [B, Hkv, G * Lq, Lk] with -inf where there is no key, and q, k, v padded alike."""
    q, k, v = s["q"], s["k"], s["v"]
    (nq, h, d), (nk, hk, _) = q.shape, k.shape
    qi, qok = padded(s["q_offsets"], s["lq"], nq)
    ki, kok = padded(s["kv_offsets"], s["lk"], nk)
    if s["key_mask"] is not None:
        kok = kok & s["key_mask"][ki]
    b, lq = qi.shape

    def rows(x):  # [nq, h, d] -> [b, hk, g * lq, d]
        return (x.float()[qi] * qok[:, :, None, None]).view(b, lq, hk, h // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, (h // hk) * lq, d)

    kp, vp = [(x.float()[ki] * kok[:, :, None, None]).permute(0, 2, 1, 3).contiguous() for x in (k, v)]
    qp = rows(q) * s["scale"]
    sc = torch.matmul(qp, kp.transpose(2, 3).contiguous())
    return sc.masked_fill_(~kok[:, None, None, :], -math.inf), qp, kp, vp, rows


def probabilities(sc):
    top = sc.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(sc - top)
    total = p.sum(3, keepdim=True)
    return p / torch.where(total == 0, 1.0, total), (top + torch.log(total)).squeeze(3)


def attend(s):
    (nq, h, d), hk = s["q"].shape, s["k"].shape[1]
    sc, _, _, vp, _ = scores(s)
    p, lse = probabilities(sc)
    b, at = places(s["q_offsets"], nq)
    out = torch.matmul(p, vp).view(-1, h, s["lq"], d)[b, :, at]
    return out.to(s["q"].dtype), lse.view(-1, h, s["lq"])[b, :, at]


def attend_gradients(s):
    (nq, h, d), (nk, hk, _) = s["q"].shape, s["k"].shape
    sc, qp, kp, vp, rows = scores(s)
    p, _ = probabilities(sc)
    do = rows(s["dout"])
    dv = torch.matmul(p.transpose(2, 3).contiguous(), do)
    dp = torch.matmul(do, vp.transpose(2, 3).contiguous())
    ds = p * (dp - (p * dp).sum(3, keepdim=True))
    dq = torch.matmul(ds, kp) * s["scale"]
    dk = torch.matmul(ds.transpose(2, 3).contiguous(), qp)
    qb, qat = places(s["q_offsets"], nq)
    kb, kat = places(s["kv_offsets"], nk)
    dt = s["q"].dtype
    return dq.view(-1, h, s["lq"], d)[qb, :, qat].to(dt), dk[kb, :, kat].to(dt), dv[kb, :, kat].to(dt)


def plain(s):
    op = s["op"]
    if op == "attn":
        return attend(s)
    if op == "attn_grad":
        return attend_gradients(s)
    if op == "conv8":
        n, cin = s["codes"].shape
        # The checkpoint stands for values of the activation's type.
        x = restored(s["codes"], s["scales"]).to(s["dout"].dtype).float()
        near = x[s["kmap"].clamp(min=0).long().t()] * (s["kmap"].t() >= 0)[:, :, None]
        return torch.matmul(near.reshape(n, 27 * cin).t(), s["dout"].float()).view(27, cin, -1)
    if op == "norm8_grad":
        return norm_gradients(s["dy"], restored(s["codes"], s["scales"]), s["rstd"], s["weight"], s["dy"].dtype)
    x, dt = s["x"].float(), s["x"].dtype
    if op == "pack":
        return restored(*packed(x)).to(dt)
    if op == "norm_grad":
        return norm_gradients(s["dy"], (x - s["mean"][:, None]) * s["rstd"][:, None], s["rstd"], s["weight"], dt)
    mean, rstd = statistics(x)
    xhat = (x - mean[:, None]) * rstd[:, None]
    y = (xhat * s["weight"].float() + s["bias"].float()).to(dt)
    return (y, mean, rstd) if op == "norm" else (y, restored(*packed(xhat)).to(dt), rstd)


# ------------------------------------------------------------------------------------------- runs

def run(state):
    if not own:
        return plain(state)
    s, igc, op = state, state["igc"], state["op"]
    if op == "norm":
        return igc.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)
    if op == "norm_grad":
        return igc.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"])
    if op == "pack":
        return igc.checkpoint_unpack(igc.checkpoint_pack(s["x"]))
    if op == "norm8":
        y, ckpt, rstd = igc.layer_norm_checkpoint(s["x"], s["weight"], s["bias"], eps=EPS)
        return y, igc.checkpoint_unpack(ckpt), rstd
    if op == "norm8_grad":
        return igc.layer_norm_checkpoint_backward(s["dy"], s["ckpt"], s["rstd"], s["weight"])
    if op == "conv8":
        return igc.sparse_conv_backward(s["grid"], s["ckpt"], s["weights"], s["dout"], s["kmap"], need_dfeats=False)[1]
    where = {"q_offsets": s["q_offsets"], "kv_offsets": s["kv_offsets"], "key_mask": s["key_mask"], "scale": s["scale"]}
    if op == "attn":
        return igc.cross_attention(s["q"], s["k"], s["v"], **where)
    return igc.cross_attention_backward(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], **where)


# ------------------------------------------------------------------------------ in 64 bits, apart

def codes64(x):
    """Values of the 8-bit checkpoint of float64 rows, group by group."""
    out = torch.empty_like(x)
    for c in range(0, x.shape[1], GROUP):
        part = x[:, c:c + GROUP]
        a = part.abs().max(1).values.unsqueeze(1)
        out[:, c:c + GROUP] = torch.where(a < 2.0 ** -100, 0.0, torch.round(part / a * 127) * a / 127)
    return out


def exact(case, seed):
    op, s = case["op"], inputs(case, seed)
    if op.startswith("attn"):
        return attend64(case, s)
    if op == "conv8":
        n = s["codes"].shape[0]
        scales = torch.stack([s["scales"][:, c // GROUP] for c in range(case["cin"])], 1)
        x = (s["codes"] * scales).bfloat16().double()
        dw = torch.zeros(27, case["cin"], case["cout"], dtype=torch.float64, device="cuda")
        for o in range(27):
            r = torch.nonzero(s["kmap"][o] >= 0).flatten()
            dw[o] = x[s["kmap"][o][r].long()].t().contiguous() @ s["dout"][r].double()
        return dw
    if op == "pack":
        return codes64(s["x"].double())
    w, b = s["weight"].double(), s["bias"].double()
    if op.endswith("_grad"):
        if op == "norm8_grad":
            xhat = s["codes"].double() * torch.stack([s["scales"][:, c // GROUP] for c in range(case["channels"])], 1)
        else:
            xhat = s["x"].double().sub_(s["mean"].double().unsqueeze(1)).mul_(s["rstd"].double().unsqueeze(1))
        dy, c = s["dy"].double(), case["channels"]
        dw, db = torch.einsum("nc,nc->c", dy, xhat), torch.einsum("nc->c", dy)
        dy.mul_(w)
        m1, m2 = torch.einsum("nc->n", dy) / c, torch.einsum("nc,nc->n", dy, xhat) / c
        dy.sub_(m1.unsqueeze(1)).sub_(xhat.mul_(m2.unsqueeze(1))).mul_(s["rstd"].double().unsqueeze(1))
        return dy, dw, db
    x = s["x"].double()
    var, mean = torch.var_mean(x, 1, correction=0)
    xhat = (x - mean.unsqueeze(1)) * torch.rsqrt(var + EPS).unsqueeze(1)
    y = torch.addcmul(b, xhat, w)
    return (y, mean, torch.rsqrt(var + EPS)) if op == "norm" else (y, codes64(xhat), torch.rsqrt(var + EPS))


def attend64(case, s):
    """One sequence and one head at a time, straight from the formulas."""
    h, hk = case["heads"], case["kv_heads"]
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    grads = case["op"] == "attn_grad"
    do = s["dout"].double() if grads else None
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    qo, ko = s["q_offsets"].tolist(), s["kv_offsets"].tolist()
    for b in range(case["batch"]):
        rows = slice(qo[b], qo[b + 1])
        keys = torch.arange(ko[b], ko[b + 1], device="cuda")
        if s["key_mask"] is not None:
            keys = keys[s["key_mask"][keys]]
        if not keys.numel():
            continue
        for i in range(h):
            j = i * hk // h
            kk, vv, qq = k[keys, j], v[keys, j], q[rows, i]
            sc = qq @ kk.t().contiguous() * s["scale"]
            lse[rows, i] = torch.logsumexp(sc, 1)
            p = torch.softmax(sc, 1)
            out[rows, i] = p @ vv
            if grads:
                g = do[rows, i]
                ds = p * (g @ vv.t().contiguous() - (g * out[rows, i]).sum(1, keepdim=True))
                dq[rows, i] = ds @ kk * s["scale"]
                dk[keys, j] += ds.t().contiguous() @ qq * s["scale"]
                dv[keys, j] += p.t().contiguous() @ g
    return (dq, dk, dv) if grads else (out, lse)
