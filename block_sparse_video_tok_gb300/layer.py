"""The operators around the block-sparse attention in a video transformer layer: thin binding of
include/vsa_layer.h, with the C entry points' names.

    q, k, v = layer.vsa_norm_rope(q, k, v, q_weight, k_weight, cos, sin, src=src)
    o, lse = layer.vsa_cross_fwd(q, k, v, kv_len, sm_scale)

Tensors of heads are [B, H, S, D] views (norm_rope takes [B, S, H, D] token order in, and gives
[B, H, rows, D]) of any strides whose last dimension is contiguous and whose other strides are
multiples of 16 bytes.  Argument marshalling only, as in `vsa`: every step runs in libvsa.so's
kernels on the caller's stream, and outputs and workspaces that are not passed are allocated here
with torch (on that stream).  `autograd.norm_rope` and `autograd.cross_attention` are the
differentiable forms.
"""
import contextlib
import ctypes
import math

import numpy as np
import torch

from . import vsa
from .workloads import VIDEO_CUBE

DEVERR_ORDER = 0x40
DEVERR_KV_LEN = 0x80

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


class VsaHeads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("heads", ctypes.c_int32)]


class VsaNormRope(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("tokens", ctypes.c_int32), ("rows", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("weight_dtype", ctypes.c_int32), ("rot", ctypes.c_int32),
                ("halves", ctypes.c_int32), ("eps", ctypes.c_float),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("cosines", ctypes.c_void_p), ("sines", ctypes.c_void_p),
                ("table_batch_stride", ctypes.c_int64), ("order", ctypes.c_void_p)]


class VsaCross(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("q_tokens", ctypes.c_int32), ("kv_tokens", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("sm_scale", ctypes.c_float),
                ("kv_len", ctypes.c_void_p)]


_H = ctypes.POINTER(VsaHeads)
_N = ctypes.POINTER(VsaNormRope)
_C = ctypes.POINTER(VsaCross)
_P = ctypes.c_void_p
_SZ = ctypes.c_size_t

# Every symbol include/vsa_layer.h declares, with its (restype, argtypes).
SIGNATURES = {
    "vsa_norm_rope_fwd": (ctypes.c_int, [_N] + [_H] * 6 + [_P]),
    "vsa_norm_rope_bwd_workspace_bytes": (_SZ, [_N]),
    "vsa_norm_rope_bwd": (ctypes.c_int, [_N] + [_H] * 8 + [_P, _P, _P, _SZ, _P]),
    "vsa_cross_fwd_workspace_bytes": (_SZ, [_C]),
    "vsa_cross_bwd_workspace_bytes": (_SZ, [_C]),
    "vsa_cross_fwd": (ctypes.c_int, [_C] + [_H] * 4 + [_P, _P, _SZ, _P]),
    "vsa_cross_bwd": (ctypes.c_int, [_C] + [_H] * 5 + [_P] + [_H] * 3 + [_P, _SZ, _P]),
    "vsa_layer_device_error": (ctypes.c_int, [ctypes.POINTER(ctypes.c_uint32), _P]),
}

_fns = None


def _lib():
    """The library's functions of this header (raises if libvsa.so has not been built)."""
    global _fns
    if _fns is None:
        handle = vsa.lib()
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _fns = handle
    return _fns


# ------------------------------------------------------------------------------- arguments

def _heads(t, name, shape, dtype, device):
    """The [B, H, S, D] view t as a VsaHeads, after checking it."""
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise TypeError("%s must be a tensor on %s" % (name, device))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    sb, sh, ss, sd = t.stride()
    unit = 16 // t.element_size()
    B, H, S, D = shape
    if sd != 1 or t.data_ptr() % 16 or (B > 1 and sb % unit) or (H > 1 and sh % unit) or \
            (S > 1 and ss % unit):
        raise ValueError("%s: the last dimension must be contiguous, and the data and the other "
                         "strides multiples of 16 bytes (strides %s)" % (name, t.stride()))
    return VsaHeads(t.data_ptr(), sb, sh, ss, H)


def _cuda(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dim() != 4:
        raise ValueError("%s must be 4-D, got %s" % (name, tuple(t.shape)))
    if t.numel() == 0:
        raise ValueError("%s is empty: %s" % (name, tuple(t.shape)))
    if t.device.index != torch.cuda.current_device():
        raise ValueError("%s is on %s, which is not the current device" % (name, t.device))


def _vector(t, name, dtype, n, device):
    """The address of a contiguous 1-D tensor, or None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype != dtype:
        raise TypeError("%s must be a %s tensor on %s" % (name, dtype, device))
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError("%s must be contiguous with shape (%d,), got %s" % (name, n, tuple(t.shape)))
    return t.data_ptr()


def _on(stream):
    """Context for allocations that are used on `stream` (None: the current one)."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _handle(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _check(status, what):
    if status != 0:
        vsa._check(status, what)


def _workspace(given, need, device, stream):
    """(workspace tensor, address, bytes); allocated if not given."""
    if need == 0:
        return None, None, 0
    if given is None:
        with _on(stream):
            given = torch.empty(need, dtype=torch.uint8, device=device)
        return given, given.data_ptr(), need
    if not isinstance(given, torch.Tensor) or given.device != device or not given.is_contiguous():
        raise TypeError("workspace must be a contiguous tensor on %s" % device)
    return given, given.data_ptr(), given.numel() * given.element_size()


# ------------------------------------------------------------------------------- norm_rope

def _norm_rope_op(x, rows, weights, cos, sin, order, order_len, halves, eps):
    """(VsaNormRope, kept tensors) for activations shaped and typed like x [B, S, H, D]."""
    B, S, _, D = x.shape
    dtype, device = x.dtype, x.device
    if dtype not in _DTYPES:
        raise TypeError("activations must be bf16, fp16 or fp32, got %s" % dtype)
    if D % 8 or not 8 <= D <= 256:
        raise ValueError("head_dim must be a multiple of 8 up to 256, got %d" % D)
    wdtype = next((w.dtype for w in weights if isinstance(w, torch.Tensor)), dtype)
    if wdtype not in (dtype, torch.float32):
        raise TypeError("weights must be fp32 or %s, got %s" % (dtype, wdtype))
    wp = [_vector(w, n, wdtype, D, device) for w, n in zip(weights, ("q_weight", "k_weight"))]
    rot, stride, cp, sp = 0, 0, None, None
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    if cos is not None:
        for t, n in ((cos, "cos"), (sin, "sin")):
            if not isinstance(t, torch.Tensor) or t.device != device or t.dtype != torch.float32:
                raise TypeError("%s must be an fp32 tensor on %s" % (n, device))
            if t.dim() not in (2, 3) or t.shape != cos.shape or t.shape[-2] != S or \
                    (t.dim() == 3 and t.shape[0] != B):
                raise ValueError("%s must be [%d, rot / 2] or [%d, %d, rot / 2], got %s" %
                                 (n, S, B, S, tuple(t.shape)))
            if not t.is_contiguous() or t.data_ptr() % 16:
                raise ValueError("%s must be contiguous and 16-byte aligned" % n)
        rot = 2 * cos.shape[-1]
        stride = S * cos.shape[-1] if cos.dim() == 3 else 0
        cp, sp = cos.data_ptr(), sin.data_ptr()
        if rot > D or rot % (16 if halves else 8):
            raise ValueError("cos and sin turn %d of %d elements of a head: at most all, in "
                             "multiples of %d" % (rot, D, 16 if halves else 8))
    op = _vector(order, "the order", torch.int32, order_len, device)
    return VsaNormRope(B, S, rows, D, _DTYPES[dtype], _DTYPES[wdtype], rot, 1 if halves else 0,
                       eps, wp[0], wp[1], cp, sp, stride, op)


def _tokens_view(t):
    """[B, S, H, D] as [B, H, S, D]."""
    return t.transpose(1, 2)


def vsa_norm_rope(q, k=None, v=None, q_weight=None, k_weight=None, cos=None, sin=None, src=None,
                  halves=False, eps=1e-6, q_out=None, k_out=None, v_out=None, stream=None):
    """RMS norm of each head of q and k, rotation by the table, and the move from token order to
    attention rows; v is only moved.

    q, k, v: [B, S, H, D] (bf16, fp16 or fp32; D a multiple of 8 up to 256; k and v may be None or
    have other head counts).  q_weight, k_weight: [D], fp32 or the activations' type (None: ones).
    cos, sin: fp32 [S, rot / 2] or [B, S, rot / 2] of each token's angles (None: no rotation); the
    first rot elements of a head are turned, in pairs (2i, 2i + 1) or, with halves, (i, i + rot/2).
    src: int32 [rows], the token of each output row, -1 for a row of zeros (None: row t is token
    t).  Returns (q_out, k_out, v_out), [B, H, rows, D]; None where the input is None."""
    _cuda(q, "q")
    B, S, _, D = q.shape
    rows = S if src is None else src.numel()
    op = _norm_rope_op(q, rows, (q_weight, k_weight), cos, sin, src, rows, halves, eps)
    ins, outs = [], []
    res = []
    for x, y, name in ((q, q_out, "q"), (k, k_out, "k"), (v, v_out, "v")):
        if x is None:
            if y is not None:
                raise ValueError("%s_out is given without %s" % (name, name))
            ins.append(None)
            outs.append(None)
            res.append(None)
            continue
        if not isinstance(x, torch.Tensor) or x.dim() != 4 or x.shape[2] == 0:
            raise ValueError("%s must be [B, S, H, D]" % name)
        H = x.shape[2]
        ins.append(_heads(_tokens_view(x), name, (B, H, S, D), q.dtype, q.device))
        if y is None:
            with _on(stream):
                y = torch.empty((B, H, rows, D), dtype=q.dtype, device=q.device)
        outs.append(_heads(y, name + "_out", (B, H, rows, D), q.dtype, q.device))
        res.append(y)
    _check(_lib().vsa_norm_rope_fwd(op, *ins, *outs, _handle(stream)), "vsa_norm_rope_fwd")
    return tuple(res)


def vsa_norm_rope_bwd(dq_out, dk_out, dv_out, q, k=None, q_weight=None, k_weight=None, cos=None,
                      sin=None, dst=None, halves=False, eps=1e-6, dq=None, dk=None, dv=None,
                      need_dweight=True, workspace=None, stream=None):
    """Gradients of vsa_norm_rope: dq_out, dk_out, dv_out [B, H, rows, D] are the gradients of its
    outputs (dk_out with k, dv_out may be None), q and k its inputs.  dst: int32 [S], the row of
    each token, -1 for a token that no row takes (None: row t).  Returns (dq, dk, dv, dq_weight,
    dk_weight): dq, dk, dv in token order [B, S, H, D]; weight gradients in the weights' type, None
    for a weight that is None (or with need_dweight false)."""
    _cuda(q, "q")
    _cuda(dq_out, "dq_out")
    if (k is None) != (dk_out is None):
        raise ValueError("k and dk_out come together")
    B, S, _, D = q.shape
    rows = dq_out.shape[2]
    if dst is None and rows != S:
        raise ValueError("dq_out has %d rows for %d tokens, without dst" % (rows, S))
    op = _norm_rope_op(q, rows, (q_weight, k_weight), cos, sin, dst, S, halves, eps)
    dys, xs, dxs, res, dws = [], [], [], [], []
    for dy, x, dx, w, name in ((dq_out, q, dq, q_weight, "q"), (dk_out, k, dk, k_weight, "k"),
                               (dv_out, None, dv, None, "v")):
        if dy is None:
            if dx is not None:
                raise ValueError("d%s is given without d%s_out" % (name, name))
            dys.append(None)
            dxs.append(None)
            if name != "v":
                xs.append(None)
                dws.append(None)
            res.append(None)
            continue
        if not isinstance(dy, torch.Tensor) or dy.dim() != 4 or dy.shape[1] == 0:
            raise ValueError("d%s_out must be [B, H, rows, D]" % name)
        H = dy.shape[1]
        dys.append(_heads(dy, "d%s_out" % name, (B, H, rows, D), q.dtype, q.device))
        if x is not None:
            if x.dim() != 4:
                raise ValueError("%s must be [B, S, H, D]" % name)
            xs.append(_heads(_tokens_view(x), name, (B, H, S, D), q.dtype, q.device))
        with _on(stream):
            if dx is None:
                dx = torch.empty((B, S, H, D), dtype=q.dtype, device=q.device)
            if name != "v":
                dws.append(torch.empty_like(w) if w is not None and need_dweight else None)
        dxs.append(_heads(_tokens_view(dx), "d" + name, (B, H, S, D), q.dtype, q.device))
        res.append(dx)
    need = 0
    if any(w is not None for w in dws):
        need = _lib().vsa_norm_rope_bwd_workspace_bytes(op)
    keep, wp, wn = _workspace(workspace, need, q.device, stream)
    _check(_lib().vsa_norm_rope_bwd(op, *dys, *xs, *dxs, *(None if w is None else w.data_ptr()
                                                           for w in dws), wp, wn,
                                    _handle(stream)), "vsa_norm_rope_bwd")
    return (*res, *dws)


def video_token_order(grid, cube=VIDEO_CUBE, device="cuda"):
    """Token order of a (T, H, W) latent grid cut into cubes (t-major), as the block-sparse
    attention takes it: (src, dst, vbs), int32.  src [rows]: the raster token of each row, a
    cube's tokens first in raster order and -1 on the rest of its rows; dst [T * H * W]: the row
    of each token; vbs: valid tokens of each cube."""
    g, c = np.asarray(grid, np.int64), np.asarray(cube, np.int64)
    if g.shape != (3,) or c.shape != (3,) or (g < 1).any() or (c < 1).any():
        raise ValueError("grid and cube must be three sizes of at least 1")
    n = -(-g // c)
    t, h, w = np.indices(g).reshape(3, -1)
    block = ((t // c[0]) * n[1] + h // c[1]) * n[2] + w // c[2]
    per, nb = int(c.prod()), int(n.prod())
    if nb * per > 0x7FFFFFFF:
        raise ValueError("the grid has too many tokens for int32 rows")
    vbs = np.bincount(block, minlength=nb).astype(np.int32)
    tokens = np.argsort(block, kind="stable")
    start = np.cumsum(vbs) - vbs
    ranked = block[tokens]
    rows = ranked * per + np.arange(block.size) - start[ranked]
    src = np.full(nb * per, -1, np.int32)
    src[rows] = tokens
    dst = np.empty(block.size, np.int32)
    dst[tokens] = rows
    return tuple(torch.from_numpy(x).to(device) for x in (src, dst, vbs))


def rotation_table(positions, rot, theta=10000.0, device="cuda"):
    """cos and sin [..., rot / 2] (fp32) of the rotation angles of `positions` [..., axes]: the
    pairs are shared out over the axes (the first axis takes what is left over), and pair i of the
    n of an axis turns by position * theta^(-i / n).  Angles are taken in 64 bits, so that far
    positions keep their phase."""
    pos = torch.as_tensor(positions).to(torch.float64)
    half, axes = rot // 2, pos.shape[-1]
    if rot % 2 or half < axes:
        raise ValueError("rot = %d is not a number of pairs for %d axes" % (rot, axes))
    share = [half - (axes - 1) * (half // axes)] + [half // axes] * (axes - 1)
    angle = torch.cat([pos[..., a:a + 1] *
                       theta ** -(torch.arange(s, dtype=torch.float64, device=pos.device) / s)
                       for a, s in enumerate(share)], -1)
    return angle.cos().float().to(device), angle.sin().float().to(device)


# ------------------------------------------------------------------------- cross attention

def _cross_op(q, k, kv_len, sm_scale):
    _cuda(q, "q")
    _cuda(k, "k")
    B, H, Sq, D = q.shape
    Hk, Sk = k.shape[1], k.shape[2]
    if D != vsa.HEAD_DIM:
        raise ValueError("head_dim must be %d, got %d" % (vsa.HEAD_DIM, D))
    if H % Hk:
        raise ValueError("%d query heads do not share %d key heads evenly" % (H, Hk))
    if sm_scale is None:
        sm_scale = D ** -0.5
    if not math.isfinite(sm_scale):
        raise ValueError("sm_scale must be finite")
    n = _vector(kv_len, "kv_len", torch.int32, B, q.device)
    return VsaCross(B, H, Hk, Sq, Sk, D, sm_scale, n), (B, H, Sq, D), (B, Hk, Sk, D)


def _bf16(t, name, shape, device):
    h = _heads(t, name, shape, torch.bfloat16, device)
    if (shape[1] > 1 and h.head_stride == 0) or (shape[2] > 1 and h.token_stride == 0):
        raise ValueError("%s must not be broadcast over its heads or tokens" % name)
    return h


def _lse(lse, B, H, Sq, device):
    if not isinstance(lse, torch.Tensor) or lse.device != device or lse.dtype != torch.float32:
        raise TypeError("lse must be an fp32 tensor on %s" % device)
    if lse.shape != (B, H, Sq) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous [%d, %d, %d], got %s" % (B, H, Sq, tuple(lse.shape)))
    return lse.data_ptr()


def vsa_cross_fwd(q, k, v, kv_len=None, sm_scale=None, o=None, lse=None, workspace=None,
                  stream=None):
    """Attention of q [B, H, Sq, 128] to k, v [B, Hk, Sk, 128] (bf16; H a multiple of Hk), over the
    first kv_len[b] keys (int32 [B]; None: all).  sm_scale defaults to 1/sqrt(128).  Returns (o in
    q's memory order, lse fp32 [B, H, Sq], base 2); without a visible key o = 0 and lse = -inf."""
    op, qs, ks = _cross_op(q, k, kv_len, sm_scale)
    dev = q.device
    with _on(stream):
        if o is None:
            o = torch.empty_like(q)
        if lse is None:
            lse = torch.empty(qs[:3], dtype=torch.float32, device=dev)
    args = (_bf16(q, "q", qs, dev), _bf16(k, "k", ks, dev), _bf16(v, "v", ks, dev),
            _bf16(o, "o", qs, dev), _lse(lse, *qs[:3], dev))
    lib = _lib()
    keep, wp, wn = _workspace(workspace, lib.vsa_cross_fwd_workspace_bytes(op), dev, stream)
    _check(lib.vsa_cross_fwd(op, *args, wp, wn, _handle(stream)), "vsa_cross_fwd")
    return o, lse


def vsa_cross_bwd(dout, q, k, v, o, lse, kv_len=None, sm_scale=None, dq=None, dk=None, dv=None,
                  workspace=None, stream=None):
    """Gradients of vsa_cross_fwd from dout, its inputs, and the o and lse that it returned.
    Returns (dq, dk, dv), each in its input's memory order; rows of dk and dv at or past
    kv_len[b] are exact zeros."""
    op, qs, ks = _cross_op(q, k, kv_len, sm_scale)
    dev = q.device
    with _on(stream):
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        dv = torch.empty_like(v) if dv is None else dv
    args = (_bf16(dout, "dout", qs, dev), _bf16(q, "q", qs, dev), _bf16(k, "k", ks, dev),
            _bf16(v, "v", ks, dev), _bf16(o, "o", qs, dev), _lse(lse, *qs[:3], dev),
            _bf16(dq, "dq", qs, dev), _bf16(dk, "dk", ks, dev), _bf16(dv, "dv", ks, dev))
    lib = _lib()
    keep, wp, wn = _workspace(workspace, lib.vsa_cross_bwd_workspace_bytes(op), dev, stream)
    _check(lib.vsa_cross_bwd(op, *args, wp, wn, _handle(stream)), "vsa_cross_bwd")
    return dq, dk, dv


def vsa_layer_device_error(stream=None):
    """Synchronise the stream; return and clear the device error bits that these operators have
    raised on the current device since the last call."""
    bits = ctypes.c_uint32(0)
    _check(_lib().vsa_layer_device_error(ctypes.byref(bits), _handle(stream)),
           "vsa_layer_device_error")
    return int(bits.value)
