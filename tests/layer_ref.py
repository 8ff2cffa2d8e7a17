"""Plain 64-bit forms of the layer operators and how far a kernel may be from them.

Each function returns (value, bound) pairs in float64.  A bound adds up, element by element:
  - half a step of the output's type, `half_step(dtype)` times the value;
  - for cross attention, half a bf16 step of every P or dS that a 16-bit tensor-core operand holds
    (2^-8 relative each, at worst all with one sign);
  - the rounding of the fp32 arithmetic.  A sum of n products in fp32 is off by at most about
    n 2^-24 of the sum of its terms' magnitudes; sums here have at most 256 terms in a row
    (2^-16) before they are joined, and the exponentials and reciprocal square roots of the
    device are good to 2^-21.  F32 = 2^-15 of the magnitudes covers a chain of two such steps.
"""
import math

import torch

F32 = 2.0 ** -15
LOG2E = 1.4426950408889634


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Where relative rounding ends: half the smallest subnormal."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def check(name, got, ref, bound):
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    got = got.double()
    same = (got == ref) | (got.isnan() & ref.isnan())
    off = torch.where(same, 0.0, (got - ref).abs())
    bad = ~(off <= bound)
    assert not bad.any(), "%s: %d of %d outside, worst %.3g of its bound" % (
        name, int(bad.sum()), bad.numel(), float((off / bound)[bad].max()))


# ------------------------------------------------------------------------------- norm_rope

def _pairs(D, n, halves, device):
    i = torch.arange(n, device=device)
    return (i, i + n) if halves else (2 * i, 2 * i + 1)


def _turn(x, cos, sin, halves, inverse=False, magnitude=False):
    """R x (or R^T x) of x [B, S, H, D]; with magnitude, the sums of the terms' magnitudes."""
    if cos is None:
        return x.clone()
    a, b = _pairs(x.shape[-1], cos.shape[-1], halves, x.device)
    c, s = cos.double().unsqueeze(-2), sin.double().unsqueeze(-2)
    if inverse:
        s = -s
    y = x.clone()
    if magnitude:
        c, s = c.abs(), s.abs()
        y[..., a] = x[..., a] * c + x[..., b] * s
    else:
        y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def _gather(x, order):
    """x [B, n, H, D] taken at order (zeros at entries outside [0, n))."""
    if order is None:
        return x
    ok = (order >= 0) & (order < x.shape[1])
    return x[:, torch.where(ok, order, 0).long()] * ok[:, None, None]


def _norm(x, w, eps):
    x = x.double()
    r = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    w = torch.ones(x.shape[-1], dtype=torch.float64, device=x.device) if w is None else w.double()
    return x * r, r, w


def norm_rope_one(x, w, cos, sin, src, halves, eps, dtype):
    n, _, w = _norm(x, w, eps)
    y = _gather(_turn(n * w, cos, sin, halves), src).transpose(1, 2)
    mag = _gather(_turn((n * w).abs(), cos, sin, halves, magnitude=True), src).transpose(1, 2)
    return y, half_step(dtype) * y.abs() + F32 * mag + tiny(dtype)


def move(x, src):
    return _gather(x, src).transpose(1, 2).double()


def norm_rope_one_bwd(dy, x, w, cos, sin, dst, halves, eps, dtype, wdtype):
    """((dx, bound), (dw, bound))."""
    n, r, w = _norm(x, w, eps)
    g = _gather(dy.transpose(1, 2), dst).double()
    u = _turn(g, cos, sin, halves, inverse=True)
    um = _turn(g.abs(), cos, sin, halves, magnitude=True)
    dx = r * (u * w - n * (u * w * n).mean(-1, keepdim=True))
    dxm = r * (um * w.abs() + n.abs() * (um * w.abs() * n.abs()).mean(-1, keepdim=True))
    dw, dwm = (u * n).sum((0, 1, 2)), (um * n.abs()).sum((0, 1, 2))
    return ((dx, half_step(dtype) * dx.abs() + F32 * dxm + tiny(dtype)),
            (dw, half_step(wdtype) * dw.abs() + F32 * dwm + tiny(wdtype)))


# ------------------------------------------------------------------------- cross attention

def _masked(q, k, v, kv_len, scale):
    """Scores in log2 units and the magnitudes of their sums [B, H, Sq, Sk], -inf where hidden,
    and k, v expanded to the query heads with hidden rows zeroed."""
    B, H, Sq, D = q.shape
    Sk, share = k.shape[2], H // k.shape[1]
    n = torch.full((B,), Sk, device=q.device) if kv_len is None else kv_len.clamp(0, Sk)
    hidden = (torch.arange(Sk, device=q.device) >= n[:, None])[:, None]
    k, v = (x.double().masked_fill(hidden[..., None], 0.0).repeat_interleave(share, 1)
            for x in (k, v))
    q = q.double()
    s = (q @ k.transpose(-1, -2) * (scale * LOG2E)).masked_fill(hidden[:, :, None], -math.inf)
    mag = q.abs() @ k.abs().transpose(-1, -2) * abs(scale * LOG2E)
    return s, mag, k, v


def cross_fwd(q, k, v, kv_len, scale):
    """((o, bound), (lse, bound))."""
    s, mag, _, v = _masked(q, k, v, kv_len, scale)
    m = s.amax(-1, keepdim=True)
    p = torch.exp2(s - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    p = p / torch.where(l == 0, 1.0, l)
    o = p @ v
    lse = (m + torch.log2(l)).squeeze(-1)
    # P is off by 2^-8 as an operand, and by the fp32 rounding of its exponent (in log2 units).
    rel = 2.0 ** -8 + F32 + math.log(2.0) * 2 * F32 * mag.amax(-1, keepdim=True)
    bound = 2.0 ** -8 * o.abs() + rel * (p @ v.abs()) + 1e-30
    return (o, bound), (lse, F32 * (1 + mag.amax(-1)) + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0))


def cross_bwd(do, q, k, v, o, lse, kv_len, scale):
    """((dq, bound), (dk, bound), (dv, bound))."""
    B, H, Sq, D = q.shape
    Hk = k.shape[1]
    s, mag, k, v = _masked(q, k, v, kv_len, scale)
    lse = lse.double()[..., None]
    p = torch.exp2(s - torch.where(lse == -math.inf, 0.0, lse))
    do, q = do.double(), q.double()
    delta = (o.double() * do).sum(-1, keepdim=True)
    dmag = (o.double() * do).abs().sum(-1, keepdim=True)
    ds = p * (do @ v.transpose(-1, -2) - delta)
    # fp32: dP and Delta of their magnitudes, P of its exponent's; operand: 2^-8 of dS.
    prel = F32 + math.log(2.0) * 2 * F32 * (mag + lse.abs().nan_to_num(posinf=0))
    dsb = (2.0 ** -8 + prel) * ds.abs() + F32 * p * (do.abs() @ v.abs().transpose(-1, -2) + dmag)
    pb = p * (2.0 ** -8 + prel)

    def shared(x):
        return x.view(B, Hk, H // Hk, *x.shape[2:]).sum(2)

    c = abs(scale)
    dq, dqb = ds @ k * scale, dsb @ k.abs() * c + F32 * (ds.abs() @ k.abs()) * c
    dk = shared(ds.transpose(-1, -2) @ q) * scale
    dkb = shared((dsb + F32 * ds.abs()).transpose(-1, -2) @ q.abs()) * c
    dv, dvb = shared(p.transpose(-1, -2) @ do), shared((pb + F32 * p).transpose(-1, -2) @ do.abs())
    return tuple((x, b + 2.0 ** -8 * x.abs() + 1e-30) for x, b in ((dq, dqb), (dk, dkb), (dv, dvb)))
