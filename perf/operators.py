"""What is measured of the operators around the block-sparse attention in a video transformer layer.

Two operators, each with its backward pass:

  rope   the per-head RMS norm of queries and keys with the position rotation, which also moves
         q, k and v from the projection's token order [B, S, H, D] into the attention's
         [B, H, rows, D], cube by cube for video (`rope_fwd`, `rope_bwd`);
  cross  attention of the video tokens (or of single tokens) to an encoder's states of another
         length, with shared key heads and a length for each batch entry (`cross_fwd`,
         `cross_bwd`).

With `own` false, run() computes them in plain torch operations in 32 bits, rounded once at the
end; with `own` true it calls block_sparse_video_tok_gb300.layer.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CUBE = 4
EPS = 1e-6
LOG2E = 1.4426950408889634
THETA = 10000.0


# ------------------------------------------------------------------------------------- cases

def _rope(name, op, B, S, grid, H, Hk, D, dtype, wdtype, rot, halves):
    return {"name": name, "op": op, "B": B, "S": S, "grid": grid, "H": H, "Hk": Hk, "D": D,
            "dtype": dtype, "wdtype": wdtype, "rot": rot, "halves": halves}


def _cross(name, op, B, Sq, Sk, H, Hk, lens):
    return {"name": name, "op": op, "B": B, "Sq": Sq, "Sk": Sk, "H": H, "Hk": Hk, "lens": lens}


def listed():
    return [
        # One layer of the 480P workload (12 heads, a 21 x 60 x 104 latent in 4x4x4 cubes): the
        # largest forward, bound by HBM.
        _rope("rope_fwd_video", "rope_fwd", 1, 131040, "21x60x104", 12, 12, 128, "bf16", "bf16", 128,
              False),
        # Training on the 21 x 30 x 52 workload with batch 2 and fp32 norm weights.
        _rope("rope_bwd_video", "rope_bwd", 2, 32760, "21x30x52", 12, 12, 128, "bf16", "fp32", 128,
              False),
        # Serving: one token for each of eight sequences at far positions of their own, key heads
        # shared by four.
        _rope("rope_fwd_token", "rope_fwd", 8, 1, "", 8, 2, 128, "bf16", "bf16", 128, True),
        # A text-side layer in fp16: odd length, a head size that is no power of two, a part of
        # each head rotated, no video order.
        _rope("rope_bwd_odd", "rope_bwd", 2, 1021, "", 10, 5, 96, "fp16", "fp16", 64, True),
        # A small model in fp32.
        _rope("rope_fwd_fp32", "rope_fwd", 1, 777, "", 8, 8, 64, "fp32", "fp32", 64, False),
        # 480P video tokens attending to 512 text states: the largest forward.
        _cross("cross_fwd_video_text", "cross_fwd", 1, 131040, 512, 12, 12, ""),
        # Training of one such layer at 21 x 30 x 52.
        _cross("cross_bwd_video_text", "cross_bwd", 1, 32760, 512, 12, 12, ""),
        # A ragged batch with shared key heads; one entry has no state at all.
        _cross("cross_fwd_ragged", "cross_fwd", 3, 4095, 257, 12, 4, "257,0,100"),
        # Single tokens of eight sequences on text of their own lengths.
        _cross("cross_fwd_token", "cross_fwd", 8, 1, 512, 12, 12, "512,77,301,1,480,256,33,129"),
        # A single token on a long encoder output.
        _cross("cross_fwd_token_long", "cross_fwd", 1, 1, 32768, 8, 2, ""),
        # A few learned queries reading a long sequence (a resampler), in training.
        _cross("cross_bwd_few_queries", "cross_bwd", 2, 64, 8191, 8, 8, ""),
        # A short ragged training batch with shared key heads.
        _cross("cross_bwd_ragged", "cross_bwd", 2, 1111, 77, 8, 2, "77,31"),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _dearest():
    works = [work(c) for c in listed()]
    return max(w["bytes"] for w in works), max(w["flops"] for w in works)


def draw(rng):
    most_bytes, most_flops = _dearest()
    while True:
        op = rng.choice(["rope_fwd", "rope_bwd", "cross_fwd", "cross_bwd"])
        B = rng.choice([1, 1, 2, 3, 8])
        Hk = rng.choice([1, 2, 4, 5, 8, 12])
        H = Hk * rng.choice([1, 1, 2, 4])
        if op.startswith("rope"):
            D = rng.choice([64, 80, 96, 128, 128, 128, 256])
            rot = rng.choice([D, D, D // 2 if D % 32 == 0 else D])
            halves = rng.random() < 0.5
            dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
            wdtype = rng.choice([dtype, "fp32"])
            if rng.random() < 0.5:
                g = [_between(rng, 1, 24), _between(rng, 3, 60), _between(rng, 3, 104)]
                case = _rope("", op, B, g[0] * g[1] * g[2], "%dx%dx%d" % tuple(g), H, Hk, D, dtype,
                             wdtype, rot, halves)
            else:
                S = 1 if rng.random() < 0.2 else _between(rng, 2, 70000)
                case = _rope("", op, B, S, "", H, Hk, D, dtype, wdtype, rot, halves)
        else:
            short, long = _between(rng, 1, 1500), _between(rng, 64, 70000)
            Sq, Sk = (long, short) if rng.random() < 0.5 else (short, long)
            if op == "cross_fwd" and rng.random() < 0.3:
                Sq = 1
            lens = ""
            if rng.random() < 0.5:
                lens = ",".join(str(rng.choice([0, 1, Sk, rng.randint(0, Sk), rng.randint(0, Sk)]))
                                for _ in range(B))
            case = _cross("", op, B, Sq, Sk, H, Hk, lens)
        w = work(case)
        if w["bytes"] <= most_bytes and w["flops"] <= most_flops:
            del case["name"]
            return case


# ------------------------------------------------------------------------------------- inputs

def _video_order(grid):
    """Token order of a (T, H, W) grid cut into 4x4x4 cubes (t-major): src[row] is the raster token
    of each attention row, the tokens of a clipped cube first and -1 on the rest of its 64 rows;
    dst[token] is the token's row."""
    g = np.array([int(x) for x in grid.split("x")])
    n = -(-g // CUBE)
    t, h, w = np.meshgrid(*[np.arange(x) for x in g], indexing="ij")
    cube = ((t // CUBE * n[1] + h // CUBE) * n[2] + w // CUBE).reshape(-1)
    tokens = np.argsort(cube, kind="stable")          # raster order within a cube
    first = np.searchsorted(cube[tokens], np.arange(n.prod()))
    rows = cube[tokens] * CUBE ** 3 + np.arange(cube.size) - first[cube[tokens]]
    src = np.full(n.prod() * CUBE ** 3, -1, np.int32)
    src[rows] = tokens
    dst = np.empty(cube.size, np.int32)
    dst[tokens] = rows
    return src, dst


def _table(case, gen):
    """cos and sin of the rotation angles, fp32 from angles in 64 bits: three axes share the pairs
    of a video head; other inputs have one axis, and far positions of their own for each sequence
    where they are single tokens."""
    half = case["rot"] // 2
    if case["grid"]:
        g = [int(x) for x in case["grid"].split("x")]
        pos = torch.cartesian_prod(*[torch.arange(x, dtype=torch.float64) for x in g]).reshape(-1, 3)
        share = [half - 2 * (half // 3), half // 3, half // 3]
    else:
        if case["S"] == 1:
            pos = torch.randint(0, 1 << 20, (case["B"], 1, 1), generator=gen).double()
        else:
            pos = torch.arange(case["S"], dtype=torch.float64)[:, None]
        share = [half]
    angle = torch.cat([pos[..., a:a + 1] * THETA ** -(torch.arange(s, dtype=torch.float64) / max(s, 1))
                       for a, s in enumerate(share)], -1)
    return torch.cos(angle).float().cuda(), torch.sin(angle).float().cuda()


def prepare(case, seed):
    gen = torch.Generator().manual_seed(int(seed) + 1)
    dev = torch.Generator("cuda").manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=dev, device="cuda").to(dtype)

    B, H, Hk = case["B"], case["H"], case["Hk"]
    s = {"op": case["op"], "H": H, "Hk": Hk}
    if case["op"].startswith("rope"):
        S, D, dtype = case["S"], case["D"], DTYPES[case["dtype"]]
        s["D"], s["halves"] = D, case["halves"]
        # One projection's output: the heads of q, then of k, then of v, with a scale of its own
        # for each token.
        scale = torch.exp(0.5 * normal(B, S, 1))
        s["qkv"] = (normal(B, S, (H + 2 * Hk) * D) * scale).to(dtype)
        s["wq"], s["wk"] = ((1 + 0.1 * normal(D)).to(DTYPES[case["wdtype"]]) for _ in range(2))
        s["cos"], s["sin"] = _table(case, gen)
        s["src"] = s["dst"] = None
        rows = S
        if case["grid"]:
            src, dst = _video_order(case["grid"])
            s["src"], s["dst"] = torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda()
            rows = src.size
        if case["op"] == "rope_bwd":
            s["dq"] = normal(B, H, rows, D, dtype=dtype)
            s["dk"], s["dv"] = (normal(B, Hk, rows, D, dtype=dtype) for _ in range(2))
        return s
    Sq, Sk, D, dtype = case["Sq"], case["Sk"], 128, torch.bfloat16
    s["scale"] = D ** -0.5
    s["q"] = normal(B, Sq, H, D, dtype=dtype)                     # a projection's output each
    s["kv"] = normal(B, Sk, 2, Hk, D, dtype=dtype)
    s["lens"] = None
    if case["lens"]:
        s["lens"] = torch.tensor([int(x) for x in case["lens"].split(",")], dtype=torch.int32,
                                 device="cuda")
    if case["op"] == "cross_bwd":
        s["do"] = normal(B, Sq, H, D, dtype=dtype)
        o, s["lse"] = _cross_fwd_plain(*_cross_views(s), s["lens"], s["scale"])
        s["o"] = o.transpose(1, 2).contiguous()
        del o
    return s


def _rope_views(s):
    B, S, _ = s["qkv"].shape
    x = s["qkv"].view(B, S, s["H"] + 2 * s["Hk"], s["D"])
    return x[:, :, :s["H"]], x[:, :, s["H"]:s["H"] + s["Hk"]], x[:, :, s["H"] + s["Hk"]:]


def _cross_views(s):
    """q, k, v as [B, heads, tokens, 128] views of the projections' outputs."""
    return s["q"].transpose(1, 2), s["kv"][:, :, 0].transpose(1, 2), s["kv"][:, :, 1].transpose(1, 2)


# ------------------------------------------------------------------------------- plain forms

def _turn(x, cos, sin, halves):
    """The leading 2 * cos.shape[-1] values of each head of x [B, S, H, D] turned by the table."""
    n = cos.shape[-1]
    c, s = cos.unsqueeze(-2), sin.unsqueeze(-2)
    if halves:
        a, b = x[..., :n], x[..., n:2 * n]
        return torch.cat([a * c - b * s, b * c + a * s, x[..., 2 * n:]], -1)
    a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
    y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([y, x[..., 2 * n:]], -1)


def _to_rows(x, src, dtype):
    """[B, S, H, D] in token order -> [B, H, rows, D] in attention order, zeros where src is -1."""
    x = x.transpose(1, 2)
    if src is not None:
        x = x[:, :, src.clamp(min=0).long()] * (src >= 0)[:, None]
    return x.to(dtype).contiguous()


def _to_tokens(y, dst):
    """The reverse, in 32 bits: [B, H, rows, D] -> [B, S, H, D]."""
    y = y.float().transpose(1, 2)
    return y if dst is None else y[:, dst.long()]


def _rope_one(x, w, s):
    x32 = x.float()
    y = x32 * torch.rsqrt(x32.square().mean(-1, keepdim=True) + EPS) * w.float()
    return _to_rows(_turn(y, s["cos"], s["sin"], s["halves"]), s["src"], x.dtype)


def _rope_one_bwd(dy, x, w, s):
    x32 = x.float()
    r = torch.rsqrt(x32.square().mean(-1, keepdim=True) + EPS)
    g = _turn(_to_tokens(dy, s["dst"]), s["cos"], -s["sin"], s["halves"])
    n = x32 * r
    gw = g * w.float()
    dx = r * (gw - n * (gw * n).mean(-1, keepdim=True))
    dw = (g * n).sum((0, 1, 2), dtype=torch.float64)
    return dx.to(x.dtype), dw.to(w.dtype)


def _scores(q, k, lens, scale):
    """Scores in log2 units [B, Hk, G, Sq, Sk] in 32 bits, -inf past each length."""
    B, H, Sq, D = q.shape
    Hk, Sk = k.shape[1], k.shape[2]
    s = q.float().reshape(B, Hk, -1, D) @ k.float().transpose(-1, -2)
    s = s.view(B, Hk, H // Hk, Sq, Sk) * (scale * LOG2E)
    if lens is not None:
        hidden = torch.arange(Sk, device=q.device) >= lens[:, None]
        s = s.masked_fill(hidden[:, None, None, None], -math.inf)
    return s


def _values(v, lens):
    """v in 32 bits with the rows past each length zeroed."""
    v = v.float()
    if lens is None:
        return v
    hidden = torch.arange(v.shape[2], device=v.device) >= lens[:, None]
    return v.masked_fill(hidden[:, None, :, None], 0.0)


def _cross_fwd_plain(q, k, v, lens, scale):
    B, H, Sq, D = q.shape
    s = _scores(q, k, lens, scale)
    m = s.amax(-1, keepdim=True)
    p = torch.exp2(s - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    o = p.flatten(2, 3) @ _values(v, lens)
    o = o.view(B, H, Sq, D) / torch.where(l == 0, 1.0, l).view(B, H, Sq, 1)
    return o.to(q.dtype), (m + torch.log2(l)).view(B, H, Sq)


def _cross_bwd_plain(do, q, k, v, o, lse, lens, scale):
    B, H, Sq, D = q.shape
    Hk, Sk = k.shape[1], k.shape[2]
    grouped = (B, Hk, H // Hk, Sq, 1)
    lse = lse.view(grouped)
    p = torch.exp2(_scores(q, k, lens, scale) - torch.where(lse == -math.inf, 0.0, lse)).flatten(2, 3)
    do32 = do.float().reshape(B, Hk, -1, D)
    delta = (o.float() * do.float()).sum(-1).view(B, Hk, -1, 1)
    ds = p * (do32 @ _values(v, lens).transpose(-1, -2) - delta)
    dq = (ds @ _values(k, lens)).view(B, H, Sq, D) * scale
    dk = ds.transpose(-1, -2) @ q.float().reshape(B, Hk, -1, D) * scale
    dv = p.transpose(-1, -2) @ do32
    return dq.to(q.dtype), dk.to(k.dtype), dv.to(v.dtype)


# ------------------------------------------------------------------------------------- passes

def run(s):
    if s["op"] == "rope_fwd":
        q, k, v = _rope_views(s)
        if own:
            from block_sparse_video_tok_gb300 import layer
            return layer.vsa_norm_rope(q, k, v, s["wq"], s["wk"], s["cos"], s["sin"], src=s["src"],
                                       halves=s["halves"], eps=EPS)
        return _rope_one(q, s["wq"], s), _rope_one(k, s["wk"], s), _to_rows(v, s["src"], v.dtype)
    if s["op"] == "rope_bwd":
        q, k, v = _rope_views(s)
        if own:
            from block_sparse_video_tok_gb300 import layer
            return layer.vsa_norm_rope_bwd(s["dq"], s["dk"], s["dv"], q, k, s["wq"], s["wk"],
                                           s["cos"], s["sin"], dst=s["dst"], halves=s["halves"],
                                           eps=EPS)
        dq, dwq = _rope_one_bwd(s["dq"], q, s["wq"], s)
        dk, dwk = _rope_one_bwd(s["dk"], k, s["wk"], s)
        return dq, dk, _to_tokens(s["dv"], s["dst"]).to(v.dtype), dwq, dwk
    q, k, v = _cross_views(s)
    if s["op"] == "cross_fwd":
        if own:
            from block_sparse_video_tok_gb300 import layer
            return layer.vsa_cross_fwd(q, k, v, s["lens"], s["scale"])
        return _cross_fwd_plain(q, k, v, s["lens"], s["scale"])
    do, o = s["do"].transpose(1, 2), s["o"].transpose(1, 2)
    if own:
        from block_sparse_video_tok_gb300 import layer
        return layer.vsa_cross_bwd(do, q, k, v, o, s["lse"], s["lens"], s["scale"])
    return _cross_bwd_plain(do, q, k, v, o, s["lse"], s["lens"], s["scale"])


def work(case):
    B, H, Hk = case["B"], case["H"], case["Hk"]
    if case["op"].startswith("rope"):
        S, D, e = case["S"], case["D"], DTYPES[case["dtype"]].itemsize
        tokens, rows = B * S, S
        table = (B if S == 1 and not case["grid"] else 1) * S * case["rot"] * 4
        weights = 2 * D * DTYPES[case["wdtype"]].itemsize
        index = 0
        if case["grid"]:
            rows = CUBE ** 3 * math.prod(-(-int(x) // CUBE) for x in case["grid"].split("x"))
            index = 4 * (rows if case["op"] == "rope_fwd" else S)
        if case["op"] == "rope_fwd":
            return {"bytes": (tokens + B * rows) * (H + 2 * Hk) * D * e + table + weights + index,
                    "flops": tokens * (H + Hk) * D * 8}
        # Reads q, k and the rows' gradients that a token has; writes dq, dk, dv.
        return {"bytes": tokens * (3 * H + 5 * Hk) * D * e + table + 2 * weights + index,
                "flops": tokens * (H + Hk) * D * 16}
    Sq, Sk, D = case["Sq"], case["Sk"], 128
    keys = sum(int(x) for x in case["lens"].split(",")) if case["lens"] else B * Sk
    rows = B * H * Sq
    pairs = H * Sq * keys
    lens = 4 * B if case["lens"] else 0
    if case["op"] == "cross_fwd":
        return {"bytes": rows * (4 * D + 4) + keys * Hk * 4 * D + lens, "flops": 4 * D * pairs}
    return {"bytes": rows * (8 * D + 4) + keys * Hk * 4 * D + B * Sk * Hk * 4 * D + lens,
            "flops": 10 * D * pairs}


# ------------------------------------------------------------------------- values in 64 bits

def _exact_rotation(cos, sin, D, halves):
    """The rotation of each token as a matrix [..., S, D, D]."""
    n = cos.shape[-1]
    i = torch.arange(n, device=cos.device)
    a, b = (i, i + n) if halves else (2 * i, 2 * i + 1)
    r = torch.eye(D, dtype=torch.float64, device=cos.device).repeat(*cos.shape[:-1], 1, 1)
    r[..., a, a] = cos.double()
    r[..., b, b] = cos.double()
    r[..., a, b] = -sin.double()
    r[..., b, a] = sin.double()
    return r


def _exact_rope(case, s):
    """Token by token in chunks: y = R (x / sqrt(mean x^2 + eps) * w) and its vector-Jacobian."""
    B, S, H, Hk, D = case["B"], case["S"], case["H"], case["Hk"], case["D"]
    forward = case["op"] == "rope_fwd"
    x = s["qkv"].reshape(B, S, H + 2 * Hk, D)
    w = torch.cat([s["wq"].double().expand(H, D), s["wk"].double().expand(Hk, D)])
    rows = S if s["src"] is None else s["src"].numel()
    row = torch.arange(S, device="cuda") if s["dst"] is None else s["dst"].long()
    if forward:
        out = torch.zeros(B, H + 2 * Hk, rows, D, dtype=torch.float64, device="cuda")
    else:
        out = torch.empty(B, S, H + 2 * Hk, D, dtype=torch.float64, device="cuda")
        dw = torch.zeros(H + Hk, D, dtype=torch.float64, device="cuda")
        dy = torch.cat([s["dq"], s["dk"], s["dv"]], 1)
    step = 2048
    for t0 in range(0, S, step):
        t = slice(t0, min(S, t0 + step))
        rot = _exact_rotation(s["cos"][..., t, :], s["sin"][..., t, :], D, case["halves"])
        xt = x[:, t, :H + Hk].double()
        inv = 1.0 / torch.sqrt((xt * xt).sum(-1, keepdim=True) / D + EPS)
        n = xt * inv
        if forward:
            y = (rot @ (n * w).transpose(-1, -2)).transpose(-1, -2)
            out[:, :, row[t]] = torch.cat([y, x[:, t, H + Hk:].double()], 2).transpose(1, 2)
        else:
            g = dy[:, :, row[t]].transpose(1, 2).double()
            u = g[:, :, :H + Hk] @ rot                       # R^T g, as rows
            dw += (u * n).sum((0, 1))
            uw = u * w
            out[:, t, :H + Hk] = inv * (uw - n * (uw * n).sum(-1, keepdim=True) / D)
            out[:, t, H + Hk:] = g[:, :, H + Hk:]
    if forward:
        return out[:, :H], out[:, H:H + Hk], out[:, H + Hk:]
    return out[:, :, :H], out[:, :, H:H + Hk], out[:, :, H + Hk:], dw[:H].sum(0), dw[H:].sum(0)


def _exact_cross(case, s):
    """Head by head, on the keys that each entry has, query rows in chunks."""
    B, H, Hk, Sq, Sk, D = case["B"], case["H"], case["Hk"], case["Sq"], case["Sk"], 128
    f64 = dict(dtype=torch.float64, device="cuda")
    forward = case["op"] == "cross_fwd"
    lens = [int(x) for x in case["lens"].split(",")] if case["lens"] else [Sk] * B
    o, lse = torch.zeros(B, H, Sq, D, **f64), torch.full((B, H, Sq), -math.inf, **f64)
    dq = torch.zeros(B, H, Sq, D, **f64)
    dk, dv = torch.zeros(B, Hk, Sk, D, **f64), torch.zeros(B, Hk, Sk, D, **f64)
    step = max(1, (1 << 27) // Sk)
    for b in range(B):
        n = lens[b]
        for h in range(H if n else 0):
            kh, vh = (s["kv"][b, :n, i, h // (H // Hk)].double() for i in range(2))
            for r0 in range(0, Sq, step):
                r = slice(r0, min(Sq, r0 + step))
                z = s["q"][b, r, h].double() @ kh.T * s["scale"]          # natural units
                if forward:
                    log = torch.logsumexp(z, -1)
                    o[b, h, r] = torch.exp(z - log[:, None]) @ vh
                    lse[b, h, r] = log / math.log(2.0)
                    continue
                p = torch.exp(z - s["lse"][b, h, r].double()[:, None] * math.log(2.0))
                g = s["do"][b, r, h].double()
                ds = p * (g @ vh.T - (g * s["o"][b, r, h].double()).sum(-1, keepdim=True))
                dq[b, h, r] = ds @ kh * s["scale"]
                dk[b, h // (H // Hk), :n] += ds.T @ s["q"][b, r, h].double() * s["scale"]
                dv[b, h // (H // Hk), :n] += p.T @ g
    return (o, lse) if forward else (dq, dk, dv)


def exact(case, seed):
    if work(case)["flops"] > 4e12:                   # over about 20 seconds in 64 bits
        return None
    s = prepare(case, seed)
    return _exact_rope(case, s) if case["op"].startswith("rope") else _exact_cross(case, s)
