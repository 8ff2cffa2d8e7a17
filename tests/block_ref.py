"""Plain 64-bit forms of the block operators and how far a kernel may be from them.

Each function returns (value, bound) pairs in float64, the bounds built as in layer_ref: half a step
of the output's type times the value; half a step for what is rounded as a 16-bit operand of a product
(dz); and F32 = 2^-15 of the magnitudes that an fp32 computation adds up, which covers sums of up to
512 terms in a row at 2^-24 each and the device's exponentials, roots and quotients (2^-20).  An error
d of an intermediate value goes on as |slope| d; the activations' slopes are at most 1.13 in magnitude.
"""
import math

import torch

from tests.layer_ref import F32, check, half_step, tiny  # noqa: F401

SLOPE = 1.13


# ------------------------------------------------------------------------------- gate_norm

def _of_token(m, S):
    if m is None:
        return None
    m = m.double()
    m = m[:, None] if m.dim() == 2 else m
    return m.repeat_interleave(S // m.shape[1], 1)


def _wide(t):
    return None if t is None else t.double()


def _branch(y, gate, post_weight, post_eps, S):
    """gate u, its fp32 error, n_y, 1 / root of y."""
    y = y.double()
    ny, ry = y, torch.ones_like(y[..., :1])
    u = y
    if post_weight is not None:
        ry = 1 / torch.sqrt(y.square().mean(-1, keepdim=True) + post_eps)
        ny = y * ry
        u = ny * post_weight.double()
    g = _of_token(gate, S)
    return (u if g is None else u * g), ny, ry


def _norm(x, mag, kind, eps):
    """(n, 1 / deviation, error of n) of x, whose own fp32 error is F32 mag."""
    c = x - x.mean(-1, keepdim=True) if kind == "layer" else x
    r = 1 / torch.sqrt(c.square().mean(-1, keepdim=True) + eps)
    n = c * r
    return n, r, F32 * (r * (mag + mag.mean(-1, keepdim=True)) + n.abs() * (1 + r * mag.mean(-1, keepdim=True)))


def gate_norm(x, y, gate, post_weight, weight, bias, scale, shift, kind, eps, post_eps, hdtype):
    """((x', bound), (h, bound))."""
    S = x.shape[1]
    xd = x.double()
    mag = xd.abs()
    if y is not None:
        u, _, _ = _branch(y, gate, post_weight, post_eps, S)
        xd, mag = xd + u, mag + u.abs()
    n, _, dn = _norm(xd, mag, kind, eps)
    one = torch.ones_like(n) if scale is None else 1 + _of_token(scale, S)
    a = one if weight is None else one * weight.double()
    c = torch.zeros_like(n) if bias is None else one * bias.double()
    cm = c.abs()
    if shift is not None:
        c, cm = c + _of_token(shift, S), cm + _of_token(shift, S).abs()
    h = n * a + c
    hb = half_step(hdtype) * h.abs() + a.abs() * dn + F32 * ((n * a).abs() + cm) + tiny(hdtype)
    return (xd, half_step(x.dtype) * xd.abs() + F32 * mag + tiny(x.dtype)), (h, hb)


def gate_norm_bwd(dh, dx_out, x, y, gate, post_weight, weight, bias, scale, shift, kind, eps, post_eps):
    """(dx, dy, dgate, dpost_weight, dweight, dbias, dscale, dshift), (value, bound) or None each."""
    B, S, C = x.shape
    xd, g = x.double(), dh.double()
    n, r, dn = _norm(xd, xd.abs(), kind, eps)
    one = torch.ones_like(n) if scale is None else 1 + _of_token(scale, S)
    w = torch.ones(C, dtype=torch.float64, device=x.device) if weight is None else weight.double()
    ga = g * one * w
    gm = ga.abs()

    def mean(t):
        return t.mean(-1, keepdim=True)

    o = 0 if dx_out is None else dx_out.double()
    dx = o + r * (ga - (mean(ga) if kind == "layer" else 0) - n * mean(ga * n))
    dxb = F32 * (abs(o) + r * (gm + mean(gm) + n.abs() * mean(gm * n.abs()))) + \
        r * (dn * mean(gm * n.abs()) + n.abs() * mean(gm * dn))
    out = dict.fromkeys(("dx", "dy", "dgate", "dpost_weight", "dweight", "dbias", "dscale", "dshift"))
    out["dx"] = dx, dxb + half_step(x.dtype) * dx.abs() + tiny(x.dtype)

    def sums(value, bound, like):
        """Over the tokens of a modulation row (or all), rounded to like's type."""
        if like.dim() == 1:
            v, b = value.sum((0, 1)), bound.sum((0, 1))
        else:
            G = 1 if like.dim() == 2 else like.shape[1]
            v, b = (t.view(B, G, S // G, C).sum(2).view(like.shape) for t in (value, bound))
        return v, b + half_step(like.dtype) * v.abs() + tiny(like.dtype)

    if shift is not None:
        out["dshift"] = sums(g, F32 * g.abs(), shift)
    b0 = 0 if bias is None else bias.double()
    if scale is not None:
        out["dscale"] = sums(g * (n * w + b0), g.abs() * (w.abs() * dn + F32 * ((n * w).abs() + abs(b0))), scale)
    if bias is not None:
        out["dbias"] = sums(g * one, F32 * (g * one).abs(), bias)
    if weight is not None:
        out["dweight"] = sums(g * one * n, (g * one).abs() * (dn + F32 * n.abs()), weight)
    if y is not None:
        _, ny, ry = _branch(y, gate, post_weight, post_eps, S)
        p = 1 if post_weight is None else post_weight.double()
        gt = 1 if gate is None else _of_token(gate, S)
        ub = dxb * ny.abs() + F32 * (dx * ny).abs()
        if gate is not None:
            out["dgate"] = sums(dx * ny * p, ub * abs(p) if post_weight is not None else ub, gate)
        du, dub = dx * gt, (dxb + F32 * dx.abs()) * abs(gt)
        if post_weight is not None:
            out["dpost_weight"] = sums(du * ny, dub * ny.abs() + F32 * (du * ny).abs(), post_weight)
            q, qb = du * p, dub * abs(p)
            du = ry * (q - ny * mean(q * ny))
            dub = ry * (qb + ny.abs() * mean(qb * ny.abs()) + F32 * (q.abs() + 2 * ny.abs() * mean((q * ny).abs())))
        out["dy"] = du, dub + half_step(y.dtype) * du.abs() + tiny(y.dtype)
    return tuple(out.values())


# ------------------------------------------------------------------------------- linear

def act(z, name):
    """In forms that keep their precision where the result is small: Phi(z) = erfc(-z / sqrt 2) / 2,
    (1 + tanh u) / 2 = sigmoid(2 u)."""
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z / 2 ** 0.5)
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z) if name == "silu" else z


def slope(z, name):
    if name is None:
        return torch.ones_like(z)
    z = z.detach().requires_grad_(True)
    with torch.enable_grad():
        return torch.autograd.grad(act(z, name).sum(), z)[0]


def linear(x, weight, bias, name, residual):
    """((out, bound), (pre, bound)) of x [M, K]."""
    x, w, dtype = x.double(), weight.double(), x.dtype
    z, mag = x @ w.T, x.abs() @ w.abs().T
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    zb = F32 * mag
    out = act(z, name)
    bound = SLOPE * zb + F32 * out.abs()
    if residual is not None:
        out = out + residual.double()
        bound = bound + F32 * residual.double().abs()
    return ((out, bound + half_step(dtype) * out.abs() + tiny(dtype)),
            (z, zb + half_step(dtype) * z.abs() + tiny(dtype)))


def linear_bwd(dout, x, weight, bias, name, pre, x_name, x_pre):
    """((dx, bound), (dweight, bound), (dbias, bound) or None)."""
    dtype = x.dtype
    x, w, dz = x.double(), weight.double(), dout.double()
    dzb = torch.zeros_like(dz)
    if name is not None:
        dzb = F32 * SLOPE * dz.abs()
        dz = dz * slope(pre.double(), name)
        dzb = dzb + half_step(dtype) * dz.abs() + tiny(dtype)
    dzb = dzb + F32 * dz.abs()
    dx, dxb = dz @ w, dzb @ w.abs()
    if x_name is not None:
        s = slope(x_pre.double(), x_name)
        dx, dxb = dx * s, SLOPE * (dxb + F32 * dx.abs())
    dw, dwb = dz.T @ x, dzb.T @ x.abs()
    res = [(dx, dxb + half_step(dtype) * dx.abs() + tiny(dtype)),
           (dw, dwb + half_step(dtype) * dw.abs() + tiny(dtype)), None]
    if bias is not None:
        db = dz.sum(0)
        res[2] = db, dzb.sum(0) + half_step(bias.dtype) * db.abs() + tiny(bias.dtype)
    return tuple(res)
