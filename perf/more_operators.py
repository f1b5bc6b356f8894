"""Cases of the self-attention operators over voxels in grid order: attention in a sliding window with first tokens
that stay visible, the norm of queries and keys with the rotation by their positions, and dropout from a counter-based
generator. Row counts are those of this package's workloads (a 7,130-voxel shell, a LiDAR frame of about 43 thousand
voxels, bands of millions), heads and channels those of its layers and of its cross attention."""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


# ------------------------------------------------------------------------------------------ cases
# left, right: keys that stay visible before and after a query's own position (-1: all of them).

def listed():
    return [
        # One new token for each of 64 sequences over caches of about 4,096 (serving: latency, few keys of a long cache).
        {"name": "window-bf16-token", "op": "window", "dtype": "bf16", "batch": 64, "queries": 64, "keys": 262147, "skew": 0.8,
         "left": 1023, "right": 0, "sinks": 4, "heads": 8, "kv_heads": 4, "dim": 64, "masked": 0.0},
        # The shell scene in fp32 with a scene token in front, narrow windows to both sides.
        {"name": "window-f32-shell", "op": "window", "dtype": "f32", "batch": 1, "queries": 7131, "keys": 7131, "skew": 0.0,
         "left": 64, "right": 64, "sinks": 1, "heads": 2, "kv_heads": 2, "dim": 32, "masked": 0.0},
        # A narrow band's voxels in grid order, eight scene tokens.
        {"name": "window-bf16-band", "op": "window", "dtype": "bf16", "batch": 1, "queries": 200003, "keys": 200003, "skew": 0.0,
         "left": 256, "right": 256, "sinks": 8, "heads": 4, "kv_heads": 4, "dim": 64, "masked": 0.0},
        # Training on three padded scenes, pairs of query heads on one key head.
        {"name": "window-grad-bf16-scenes", "op": "window_grad", "dtype": "bf16", "batch": 3, "queries": 100003, "keys": 100003, "skew": 0.5,
         "left": 512, "right": 512, "sinks": 16, "heads": 4, "kv_heads": 2, "dim": 64, "masked": 0.1},
        # Training on short fp32 sequences generated token by token, sizes that fill no tile.
        {"name": "window-grad-f32-causal", "op": "window_grad", "dtype": "f32", "batch": 2, "queries": 9001, "keys": 9001, "skew": 0.3,
         "left": 255, "right": 0, "sinks": 4, "heads": 2, "kv_heads": 2, "dim": 40, "masked": 0.0},
        # The new tokens' queries and keys before they meet the caches: far positions, half of each head turned (the smallest call).
        {"name": "qk-bf16-token", "op": "qk", "dtype": "bf16", "rows": 64, "heads": 8, "kv_heads": 4, "dim": 64, "axes": 1, "pairs": 16,
         "layout": "interleaved", "amplitude": 1.2, "reach": 1000000, "stretch": 8.0},
        # Queries and keys of one LiDAR frame by voxel coordinates in fp32.
        {"name": "qk-f32-lidar", "op": "qk", "dtype": "f32", "rows": 43217, "heads": 8, "kv_heads": 8, "dim": 32, "axes": 3, "pairs": 5,
         "layout": "half", "amplitude": 1.0, "reach": 2048, "stretch": 1.0},
        # A band of a million voxels by their coordinates ...
        {"name": "qk-bf16-band", "op": "qk", "dtype": "bf16", "rows": 1000003, "heads": 4, "kv_heads": 4, "dim": 64, "axes": 3, "pairs": 10,
         "layout": "half", "amplitude": 1.0, "reach": 2048, "stretch": 1.0},
        # ... and its gradients.
        {"name": "qk-grad-bf16-band", "op": "qk_grad", "dtype": "bf16", "rows": 1000003, "heads": 4, "kv_heads": 4, "dim": 64, "axes": 3,
         "pairs": 10, "layout": "half", "amplitude": 1.0, "reach": 2048, "stretch": 1.0},
        # The rotation alone over dense boxes' voxels in fp32.
        {"name": "rotary-f32-boxes", "op": "rotary", "dtype": "f32", "rows": 500003, "heads": 4, "kv_heads": 0, "dim": 48, "axes": 3,
         "pairs": 8, "layout": "half", "amplitude": 1.0, "reach": 2048, "stretch": 1.0},
        # Dropout in the backward pass of a small fp32 block.
        {"name": "dropout-grad-f32-shell", "op": "dropout_grad", "dtype": "f32", "rows": 7131, "channels": 64, "p": 0.1},
        # A block's output dropped and added to its input over a band (the most bytes of all cases).
        {"name": "dropout-bf16-band", "op": "dropout", "dtype": "bf16", "rows": 2000003, "channels": 128, "p": 0.1},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["window", "window_grad", "token", "chunk", "qk", "qk_grad", "rotary", "dropout", "dropout_grad"])
    dtype = rng.choice(["f32", "bf16"])
    if op.startswith("dropout"):
        channels = rng.choice([log(3, 1024), 8 * log(1, 64), rng.choice([8, 16, 32, 64, 128, 256])])
        return {"op": op, "dtype": dtype, "rows": log(50, min(2000000, 120000000 // channels)), "channels": channels,
                "p": rng.choice([0.05, 0.1, 0.3, rng.uniform(0.0, 0.9)])}
    kv_heads = rng.choice([1, 2, 4])
    case = {"op": op, "dtype": dtype, "heads": kv_heads * rng.choice([1, 1, 2]), "kv_heads": kv_heads,
            "dim": rng.choice([16, 32, 40, 64, 96, 128])}
    if op in ("qk", "qk_grad", "rotary"):
        if op == "rotary":
            case["kv_heads"] = 0
        axes = rng.choice([1, 3])
        most = case["dim"] // 2 // axes
        case.update(axes=axes, pairs=rng.choice([most, rng.randint(1, most)]), layout=rng.choice(["half", "interleaved"]),
                    amplitude=rng.choice([1.0, 1.3]), reach=rng.choice([2048, 1000000]), stretch=rng.choice([1.0, 4.0]),
                    rows=log(20, 60000000 // (case["dim"] * (case["heads"] + case["kv_heads"]))))
        return case
    case.update(batch=rng.randint(1, 6), skew=rng.uniform(0, 0.8), masked=rng.choice([0.0, 0.0, 0.2]), sinks=rng.choice([0, 0, 1, 4, 70]),
                left=log(1, 500), right=rng.choice([0, log(1, 500)]))
    if op == "token":
        case.update(op="window", batch=rng.randint(1, 64), left=log(16, 4000), right=0)
        case["queries"], case["keys"] = case["batch"], case["batch"] * log(16, 6000)
        return case
    if op == "chunk":  # some new tokens behind a cache
        case.update(op="window", right=0)
        case["queries"], case["keys"] = case["batch"] * rng.randint(2, 300), case["batch"] * log(400, 6000)
        return case
    # At most the work of the largest listed case; fp32 takes several times as long.
    most = 25600000 // (case["batch"] * case["heads"] * case["dim"] * (4 if dtype == "f32" else 1))
    if rng.random() < 0.15:  # no limit to one side
        case["left"] = -1
        most = min(most, 1500)
    case["queries"] = case["batch"] * log(20, min(12000, most))
    case["keys"] = case["queries"]
    return case


def lengths(total, parts, skew):
    """`parts` lengths of the sum `total`, the longest up to 1 + skew times the mean or so."""
    w = [1.0 + skew * (((7 * i + 3) % parts) / max(1, parts - 1) - 0.5) for i in range(parts)]
    got = [int(total * x / sum(w)) for x in w]
    got[-1] += total - sum(got)
    return got


def sequences(case):
    """Queries and keys of each sequence."""
    lk = lengths(case["keys"], case["batch"], case["skew"])
    return (lk if case["queries"] == case["keys"] else lengths(case["queries"], case["batch"], 0.0)), lk


def pairs(case):
    """Visible query-key pairs of all sequences, masked keys left out."""
    total = 0
    for lq, lk in zip(*sequences(case)):
        p = torch.arange(lk - lq, lk)
        hi = torch.full_like(p, lk) if case["right"] < 0 else (p + case["right"] + 1).clamp(0, lk)
        lo = torch.zeros_like(p) if case["left"] < 0 else (p - case["left"]).clamp(0, lk)
        total += int(((hi - lo).clamp(min=0) + torch.minimum(hi, lo).clamp(max=case["sinks"])).sum())
    return (1.0 - case["masked"]) * total


def seen(case):
    """Keys that some query sees."""
    total = 0
    for lq, lk in zip(*sequences(case)):
        first = 0 if case["left"] < 0 else max(0, lk - lq - case["left"])
        total += lk - first + min(first, case["sinks"])
    return total


def work(case):
    op, es = case["op"], 4 if case["dtype"] == "f32" else 2
    if op.startswith("window"):
        nq, nk = case["queries"] * case["heads"] * case["dim"], seen(case) * case["kv_heads"] * case["dim"]
        flops = pairs(case) * case["heads"] * case["dim"] * (4 if op == "window" else 10)
        return {"bytes": (2 * nq + 2 * nk if op == "window" else 4 * nq + 4 * nk) * es + 4 * case["queries"] * case["heads"], "flops": flops}
    if op.startswith("dropout"):
        n = case["rows"] * case["channels"]
        return {"bytes": n * es * (3 if op == "dropout" else 2), "flops": 2 * n}
    n = case["rows"] * (case["heads"] + case["kv_heads"]) * case["dim"]
    return {"bytes": n * es * (3 if op == "qk_grad" else 2) + 4 * case["rows"] * case["axes"],
            "flops": n * {"qk": 7, "qk_grad": 14, "rotary": 3}[op]}


# ----------------------------------------------------------------------------------------- inputs

def inputs(case, seed):
    """The tensors a case works on, all on the GPU."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * std

    if op.startswith("window"):
        lq, lk = sequences(case)
        s = {"scale": case["dim"] ** -0.5, "left": case["left"], "right": case["right"], "sinks": case["sinks"],
             "q_offsets": torch.tensor([0] + lq, device="cuda").cumsum(0).int(), "kv_offsets": torch.tensor([0] + lk, device="cuda").cumsum(0).int()}
        # Queries, keys and values as projections give them; keys and values are slices of one tensor.
        s["q"] = normal(case["queries"], case["heads"], case["dim"], std=1.5).to(dt)
        kv = normal(case["keys"], 2, case["kv_heads"], case["dim"]).to(dt)
        s["k"], s["v"] = kv[:, 0], kv[:, 1]
        s["key_mask"] = torch.rand(case["keys"], generator=gen, device="cuda") >= case["masked"] if case["masked"] else None
        if op == "window_grad":
            s["dout"] = normal(case["queries"], case["heads"], case["dim"], std=0.1).to(dt)
        return s
    if op.startswith("dropout"):
        s = {"p": case["p"], "seed": 1234567890123 + 7919 * seed, "offset": 3 + seed,
             "x": normal(case["rows"], case["channels"]).to(dt), "residual": None}
        if op == "dropout":
            s["residual"] = normal(case["rows"], case["channels"]).to(dt)
        return s
    n, h, hk, d = case["rows"], case["heads"], case["kv_heads"], case["dim"]
    s = {"layout": case["layout"], "amplitude": case["amplitude"]}
    # Voxel coordinates around the origin, or positions along a sequence.
    low, high = (-case["reach"], case["reach"]) if case["axes"] > 1 else (0, case["reach"])
    s["positions"] = torch.randint(low, high, (n, case["axes"]), generator=gen, device="cuda", dtype=torch.int32)
    i = torch.arange(case["pairs"], dtype=torch.float64)
    s["frequencies"] = (10000.0 ** (-i / case["pairs"]) / case["stretch"]).float().expand(case["axes"], -1).contiguous().cuda()
    # Slices of the one projection that gives queries, keys and values (the values stay where they are).
    packed = (normal(n, h + 2 * hk, d) * (0.5 + torch.rand(d, generator=gen, device="cuda"))).to(dt)
    s["q"], s["k"] = packed[:, :h], packed[:, h:h + hk] if hk else None
    if op != "rotary":
        s["q_weight"], s["k_weight"] = 1 + normal(d, std=0.1), 1 + normal(d, std=0.1)
    if op == "qk_grad":
        s["dq"], s["dk"] = normal(n, h, d, std=0.1).to(dt), normal(n, hk, d, std=0.1).to(dt)
    return s


def prepare(case, seed):
    s = inputs(case, seed)
    s["op"] = case["op"]
    if case["op"].startswith("window"):
        s["plan"] = blocks(case)
    if case["op"] == "window_grad":  # what the forward pass left
        s["out"], s["lse"] = attend(s)
    if own:
        import sparse_convolution_amd as igc
        s["igc"] = igc
    return s


# ------------------------------------------------------------------------------------ plain forms

def blocks(case):
    """Blocks of up to 512 queries of one sequence, and the keys that they may see: rows [blocks, width] of queries and of
    keys, which of them exist, and their positions in the sequence."""
    lq, lk = sequences(case)
    width = min(512, max(lq))
    limited = case["left"] >= 0 and case["right"] >= 0
    span = min(max(lk), width + case["left"] + case["right"]) if limited else max(lk)
    table, q0, k0 = [], 0, 0
    for a, b in zip(lq, lk):
        for i in range(0, a, width):
            p = i + b - a
            start = max(0, min(p - case["left"], b - span)) if limited else 0
            table.append((q0, i, a, k0, b, start))
        q0, k0 = q0 + a, k0 + b
    q0, i, a, k0, b, start = torch.tensor(table, device="cuda").t()[:, :, None]
    qp = i + torch.arange(width, device="cuda")
    first = torch.arange(case["sinks"], device="cuda").expand(len(table), -1)
    kp = torch.cat([torch.where(first < start, first, b), start + torch.arange(span, device="cuda")], 1)
    qok, kok = qp < a, kp < b
    return {"q_rows": torch.where(qok, q0 + qp, 0), "k_rows": torch.where(kok, k0 + kp, 0), "q_ok": qok, "k_ok": kok,
            "q_at": qp + b - a, "k_at": kp}


def scores(s):
    """Scaled scores [blocks, kv_heads, group * queries, keys] with -inf where a key is out of sight; q, k, v alike."""
    t, (nq, h, d), hk = s["plan"], s["q"].shape, s["k"].shape[1]
    kok = t["k_ok"] if s["key_mask"] is None else t["k_ok"] & s["key_mask"][t["k_rows"]]
    p, j = t["q_at"][:, :, None], t["k_at"][:, None, :]
    near = kok[:, None, :].expand(-1, p.shape[1], -1)
    if s["right"] >= 0:
        near = near & (j <= p + s["right"])
    if s["left"] >= 0:
        near = near & ((j >= p - s["left"]) | (j < s["sinks"]))
    n, width = t["q_rows"].shape
    g = h // hk

    def rows(x):
        return (x.float()[t["q_rows"]] * t["q_ok"][:, :, None, None]).view(n, width, hk, g, d).permute(0, 2, 3, 1, 4).reshape(n, hk, g * width, d)

    kp, vp = [(x.float()[t["k_rows"]] * kok[:, :, None, None]).permute(0, 2, 1, 3).contiguous() for x in (s["k"], s["v"])]
    qp = rows(s["q"]) * s["scale"]
    sc = torch.matmul(qp, kp.transpose(2, 3).contiguous()).view(n, hk, g, width, -1).masked_fill_(~near[:, None, None], -math.inf)
    return sc.view(n, hk, g * width, -1), qp, kp, vp, rows


def probabilities(sc):
    top = sc.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(sc - top)
    total = p.sum(3, keepdim=True)
    return p / torch.where(total == 0, 1.0, total), (top + torch.log(total)).squeeze(3)


def unblocked(s, x):
    """[blocks, heads, queries, ...] back to rows."""
    t = s["plan"]
    out = torch.empty((s["q"].shape[0], x.shape[1]) + x.shape[3:], device=x.device)
    out[t["q_rows"][t["q_ok"]]] = x.transpose(1, 2)[t["q_ok"]]
    return out


def attend(s):
    h, width = s["q"].shape[1], s["plan"]["q_rows"].shape[1]
    sc, _, _, vp, _ = scores(s)
    p, lse = probabilities(sc)
    n, d = sc.shape[0], vp.shape[3]
    return unblocked(s, torch.matmul(p, vp).view(n, h, width, d)).to(s["q"].dtype), unblocked(s, lse.view(n, h, width))


def attend_gradients(s):
    (nq, h, d), (nk, hk, _), t, dt = s["q"].shape, s["k"].shape, s["plan"], s["q"].dtype
    sc, qp, kp, vp, rows = scores(s)
    p, _ = probabilities(sc)
    do = rows(s["dout"])
    dv = torch.matmul(p.transpose(2, 3).contiguous(), do)
    dp = torch.matmul(do, vp.transpose(2, 3).contiguous())
    ds = p * (dp - (p * dp).sum(3, keepdim=True))
    dq = torch.matmul(ds, kp) * s["scale"]
    dk = torch.matmul(ds.transpose(2, 3).contiguous(), qp)
    to = t["k_rows"].reshape(-1)
    dk, dv = [torch.zeros(nk, hk, d, device=x.device).index_add_(0, to, x.transpose(1, 2).reshape(-1, hk, d)) for x in (dk, dv)]
    return unblocked(s, dq.view(sc.shape[0], h, -1, d)).to(dt), dk.to(dt), dv.to(dt)


def turns(s):
    """Cosines and sines [rows, 1, axes * pairs] of the angles (in 64 bits: far positions), times the amplitude."""
    angle = (s["positions"].double()[:, :, None] * s["frequencies"].double()).flatten(1)[:, None]
    return (torch.cos(angle) * s["amplitude"]).float(), (torch.sin(angle) * s["amplitude"]).float()


def turned(x, cos, sin, layout):
    n = cos.shape[2]
    if layout == "half":
        a, b = x[..., :n], x[..., n:2 * n]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], 2)
    else:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], 3).flatten(2)
    return torch.cat([y, x[..., 2 * n:]], 2)


def norm_gradients(dy, x, weight, cos, sin, layout):
    g = turned(dy.float(), cos, -sin, layout)
    xf = x.float()
    rstd = 1.0 / torch.sqrt(xf.square().mean(2, keepdim=True) + EPS)
    xhat = xf * rstd
    gw = g * weight
    return (rstd * (gw - xhat * (gw * xhat).mean(2, keepdim=True))).to(x.dtype), (g * xhat).sum((0, 1))


def kept(shape, p, seed, offset):
    """Which elements stay: 16 bits of each against p, eight elements a counter of Philox 4x32 with ten rounds."""
    n = shape[0] * shape[1]
    low = (1 << 32) - 1
    at = torch.arange((n + 7) // 8, device="cuda")
    c = [at & low, at >> 32, torch.full_like(at, offset & low), torch.full_like(at, offset >> 32)]
    k0, k1 = seed & low, seed >> 32 & low
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57  # the low 64 bits, whatever their sign
        c = [(b >> 32 & low) ^ c[1] ^ k0, b & low, (a >> 32 & low) ^ c[3] ^ k1, a & low]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    bits = torch.stack([w >> shift & 0xFFFF for w in c for shift in (0, 16)], 1)
    return (bits >= round(65536 * p)).view(-1)[:n].view(shape)


def plain(s):
    op = s["op"]
    if op == "window":
        return attend(s)
    if op == "window_grad":
        return attend_gradients(s)
    if op.startswith("dropout"):
        drop = round(65536 * s["p"])
        y = torch.where(kept(s["x"].shape, s["p"], s["seed"], s["offset"]), s["x"].float() * (65536 / (65536 - drop)), 0.0)
        return (y if s["residual"] is None else y + s["residual"].float()).to(s["x"].dtype)
    cos, sin = turns(s)
    if op == "rotary":
        return turned(s["q"].float(), cos, sin, s["layout"]).to(s["q"].dtype)
    if op == "qk_grad":
        dq, dqw = norm_gradients(s["dq"], s["q"], s["q_weight"], cos, sin, s["layout"])
        dk, dkw = norm_gradients(s["dk"], s["k"], s["k_weight"], cos, sin, s["layout"])
        return dq, dk, dqw, dkw
    got = []
    for x, weight in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        xf = x.float()
        got.append(turned(xf / torch.sqrt(xf.square().mean(2, keepdim=True) + EPS) * weight, cos, sin, s["layout"]).to(x.dtype))
    return tuple(got)


# ------------------------------------------------------------------------------------------- runs

def run(state):
    if not own:
        return plain(state)
    s, igc, op = state, state["igc"], state["op"]
    if op.startswith("window"):
        where = {"left": None if s["left"] < 0 else s["left"], "right": None if s["right"] < 0 else s["right"], "sinks": s["sinks"],
                 "q_offsets": s["q_offsets"], "kv_offsets": s["kv_offsets"], "key_mask": s["key_mask"], "scale": s["scale"]}
        if op == "window":
            return igc.window_attention(s["q"], s["k"], s["v"], **where)
        return igc.window_attention_backward(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], **where)
    if op == "dropout":
        return igc.dropout(s["x"], s["p"], s["seed"], s["offset"], residual=s["residual"])
    if op == "dropout_grad":
        return igc.dropout_backward(s["x"], s["p"], s["seed"], s["offset"])
    how = {"layout": s["layout"], "amplitude": s["amplitude"]}
    if op == "rotary":
        return igc.rotary(s["q"], s["positions"], s["frequencies"], **how)
    if op == "qk":
        return igc.qk_norm_rotary(s["q"], s["k"], s["positions"], s["frequencies"], s["q_weight"], s["k_weight"], eps=EPS, **how)
    return igc.qk_norm_rotary_backward(s["dq"], s["dk"], s["q"], s["k"], s["positions"], s["frequencies"], s["q_weight"], s["k_weight"],
                                       eps=EPS, **how)


# ------------------------------------------------------------------------------ in 64 bits, apart

def exact(case, seed):
    op, s = case["op"], inputs(case, seed)
    if op.startswith("window"):
        return window64(case, s)
    if op.startswith("dropout"):
        y = s["x"].double().flatten()
        drop = round(65536 * s["p"])
        for at in range(0, y.numel(), 1 << 26):  # a piece at a time
            part = y[at:at + (1 << 26)]
            stay = bits64(at, part.numel(), s["seed"], s["offset"]) >= drop
            part.mul_(65536 / (65536 - drop)).masked_fill_(~stay, 0.0)
        y = y.view(s["x"].shape)
        return y if s["residual"] is None else y + s["residual"].double()
    z = torch.polar(torch.full((), s["amplitude"], dtype=torch.float64, device="cuda"),
                    torch.cat([s["positions"][:, a:a + 1].double() * s["frequencies"][a].double() for a in range(case["axes"])], 1))[:, None]
    if op == "rotary":
        return turn64(s["q"].double(), z, s["layout"])
    if op == "qk":
        return tuple(turn64(x.double() * (x.double().pow(2).sum(2, keepdim=True) / case["dim"] + EPS).rsqrt() * w.double(), z, s["layout"])
                     for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])))
    dxs, dws = [], []
    for dy, x, w in ((s["dq"], s["q"], s["q_weight"]), (s["dk"], s["k"], s["k_weight"])):
        g, x = turn64(dy.double(), z.conj(), s["layout"]), x.double()
        r = (x.pow(2).sum(2, keepdim=True) / case["dim"] + EPS).rsqrt()
        dws.append(torch.einsum("nhd,nhd->d", g, x * r))
        g = g * w.double()
        dxs.append(r * g - x * (r.pow(3) * (g * x).sum(2, keepdim=True) / case["dim"]))
    return (*dxs, *dws)


def turn64(x, z, layout):
    n = z.shape[2]
    first, second = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    w = torch.complex(x[..., first], x[..., second]) * z
    y = x.clone()
    y[..., first], y[..., second] = w.real, w.imag
    return y


def bits64(first, count, seed, offset):
    """The 16 bits of `count` elements from `first` (a multiple of 8) on; products in two halves, within 63 bits."""
    def product(x, m):
        p, r = x * (m & 0xFFFF), x * (m >> 16)  # x m = p + 2^16 r
        t = (p >> 16) + r
        return t >> 16, (t & 0xFFFF) << 16 | p & 0xFFFF

    block = torch.arange(first // 8, (first + count + 7) // 8, device="cuda")
    x0, x1 = block % (1 << 32), block // (1 << 32)
    x2, x3 = torch.full_like(block, offset % (1 << 32)), torch.full_like(block, offset // (1 << 32))
    for i in range(10):
        hi0, lo0 = product(x0, 0xD2511F53)
        hi1, lo1 = product(x2, 0xCD9E8D57)
        x0, x1 = hi1 ^ x1 ^ (seed + i * 0x9E3779B9) % (1 << 32), lo1
        x2, x3 = hi0 ^ x3 ^ (seed // (1 << 32) + i * 0xBB67AE85) % (1 << 32), lo0
    words = torch.stack([x0, x1, x2, x3], 1)
    return torch.stack([words % 65536, words // 65536], 2).flatten()[:count]


def window64(case, s):
    """One sequence, one head and some queries at a time, straight from the formulas."""
    h, hk, grads = case["heads"], case["kv_heads"], case["op"] == "window_grad"
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    do = s["dout"].double() if grads else None
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    qo, ko = s["q_offsets"].tolist(), s["kv_offsets"].tolist()
    for b in range(case["batch"]):
        lq, lk = qo[b + 1] - qo[b], ko[b + 1] - ko[b]
        for first in range(0, lq, 2000):
            last = min(lq, first + 2000)
            rows = slice(qo[b] + first, qo[b] + last)
            place = torch.arange(first, last, device="cuda").unsqueeze(1) + (lk - lq)
            key = torch.arange(lk, device="cuda")
            some = torch.ones_like(key, dtype=torch.bool)
            if case["right"] >= 0:
                some &= key <= last - 1 + lk - lq + case["right"]
            if case["left"] >= 0:
                some &= (key >= first + lk - lq - case["left"]) | (key < case["sinks"])
            if s["key_mask"] is not None:
                some &= s["key_mask"][ko[b]:ko[b + 1]]
            key = key[some]
            if not key.numel():
                continue
            gap = key - place
            hidden = torch.zeros_like(gap, dtype=torch.bool)
            if case["right"] >= 0:
                hidden |= gap > case["right"]
            if case["left"] >= 0:
                hidden |= (-gap > case["left"]) & (key >= case["sinks"])
            blind = hidden.all(1, keepdim=True)
            key = key + ko[b]
            for i in range(h):
                j = i * hk // h
                kk, vv, qq = k[key, j], v[key, j], q[rows, i]
                sc = (qq @ kk.t().contiguous() * s["scale"]).masked_fill_(hidden, -math.inf)
                lse[rows, i] = torch.logsumexp(sc, 1)
                p = torch.softmax(sc, 1).masked_fill_(blind, 0.0)
                out[rows, i] = p @ vv
                if grads:
                    g = do[rows, i]
                    ds = p * (g @ vv.t().contiguous() - (g * out[rows, i]).sum(1, keepdim=True))
                    dq[rows, i] = ds @ kk * s["scale"]
                    dk[key, j] += ds.t().contiguous() @ qq * s["scale"]
                    dv[key, j] += p.t().contiguous() @ g
    return (dq, dk, dv) if grads else (out, lse)
