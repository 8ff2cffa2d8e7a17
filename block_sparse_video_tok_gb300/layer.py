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
import ctypes
import functools
import math
import struct

import numpy as np
import torch

from . import vsa
from .workloads import VIDEO_CUBE

DEVERR_ORDER = 0x40
DEVERR_KV_LEN = 0x80

_current = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # device index -> stream handle

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
                ("table_batch_stride", ctypes.c_int64), ("order", ctypes.c_void_p),
                ("inverse", ctypes.c_void_p)]


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

# The wrappers below hand structures over as packed bytes: a single call into C builds one, where
# a ctypes.Structure converts field by field, which would cost more than a small kernel.
_pack_heads = struct.Struct("@4Pi4x").pack
_pack_norm = struct.Struct("@8if4PqPP").pack
_pack_cross = struct.Struct("@6ifP").pack

_fns = None
_calls = None


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


def _call(name, *args):
    """The named function on packed structures."""
    global _calls
    if _calls is None:
        lib, calls = _lib(), {}
        for n, (res, types) in SIGNATURES.items():
            fn = calls[n] = lib[n]              # a function object of its own
            fn.restype = res
            fn.argtypes = [ctypes.c_char_p if t in (_H, _N, _C) else t for t in types]
        _calls = calls
    status = _calls[name](*args)
    if status != 0:
        vsa._check(status, name)


# ------------------------------------------------------------------------------- arguments

def _heads(t, name, shape, dtype, device, transposed=False, whole=False):
    """The [B, H, S, D] tensor t (transposed: [B, S, H, D]) as a packed vsa_heads, after checking it
    against `shape` (as t has it), its type and its device's index.  whole: its heads and tokens
    must not be broadcast."""
    if not isinstance(t, torch.Tensor) or t.get_device() != device:
        raise TypeError("%s must be a tensor on cuda:%d" % (name, device))
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    ptr = t.data_ptr()
    if transposed:
        B, S, H, _ = shape
        sb, ss, sh, sd = t.stride()
    else:
        B, H, S, _ = shape
        sb, sh, ss, sd = t.stride()
    # A dimension of length 1 may have any stride.  (16 bytes: 4 fp32 or 8 16-bit elements.)
    used = (sb if B > 1 else 0) | (sh if H > 1 else 0) | (ss if S > 1 else 0)
    if sd != 1 or ptr & 15 or used & (3 if dtype is torch.float32 else 7):
        raise ValueError("%s: the last dimension must be contiguous, and the data and the other "
                         "strides multiples of 16 bytes (strides %s)" % (name, t.stride()))
    if whole and ((sh == 0 and H > 1) or (ss == 0 and S > 1)):
        raise ValueError("%s must not be broadcast over its heads or tokens" % name)
    return _pack_heads(ptr, sb, sh, ss, H)


def _cuda(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dim() != 4:
        raise ValueError("%s must be 4-D, got %s" % (name, tuple(t.shape)))
    if t.numel() == 0:
        raise ValueError("%s is empty: %s" % (name, tuple(t.shape)))
    if t.get_device() != torch._C._cuda_getDevice():
        raise ValueError("%s is on %s, which is not the current device" % (name, t.device))


def _vector(t, name, dtype, n, like):
    """The address of a contiguous 1-D tensor, or None."""
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor) or t.get_device() != like.get_device() or t.dtype is not dtype:
        raise TypeError("%s must be a %s tensor on %s" % (name, dtype, like.device))
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError("%s must be contiguous with shape (%d,), got %s" % (name, n, tuple(t.shape)))
    return t.data_ptr()


def _on(stream, f, *args, **kwargs):
    """f with `stream` as the current one, so that what it allocates belongs to it."""
    with torch.cuda.stream(stream):
        return f(*args, **kwargs)


def _workspace(given, need, like):
    """(workspace tensor, address, bytes); allocated if not given."""
    if need == 0:
        return None, None, 0
    if given is None:
        given = torch.empty(need, dtype=torch.uint8, device=like.device)
        return given, given.data_ptr(), need
    if not isinstance(given, torch.Tensor) or given.get_device() != like.get_device() or \
            not given.is_contiguous():
        raise TypeError("workspace must be a contiguous tensor on %s" % like.device)
    return given, given.data_ptr(), given.numel() * given.element_size()


@functools.lru_cache(maxsize=256)
def _cross_workspace(name, device, *sizes):
    """Workspace bytes of a cross attention of these sizes (a pure function of them)."""
    return getattr(_lib(), name)(VsaCross(*sizes, 1.0, None))


@functools.lru_cache(maxsize=64)
def _norm_workspace(device, head_dim):
    return _lib().vsa_norm_rope_bwd_workspace_bytes(
        VsaNormRope(1, 1, 1, head_dim, 0, 0, 0, 0, 0.0, None, None, None, None, 0, None, None))


# ------------------------------------------------------------------------------- norm_rope

def _norm_rope_op(x, rows, q_weight, k_weight, cos, sin, order, order_len, inverse, inverse_len, halves, eps):
    """The packed vsa_norm_rope for activations shaped and typed like x [B, S, H, D]."""
    B, S, _, D = x.shape
    dtype = x.dtype
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError("activations must be bf16, fp16 or fp32, got %s" % dtype)
    if D % 8 or not 8 <= D <= 256:
        raise ValueError("head_dim must be a multiple of 8 up to 256, got %d" % D)
    w = k_weight if q_weight is None else q_weight
    wdtype = dtype if w is None else getattr(w, "dtype", None)
    if wdtype is not dtype and wdtype is not torch.float32:
        raise TypeError("weights must be fp32 or %s, got %s" % (dtype, wdtype))
    wq = _vector(q_weight, "q_weight", wdtype, D, x)
    wk = _vector(k_weight, "k_weight", wdtype, D, x)
    rot = stride = cp = sp = 0
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    if cos is not None:
        for t, n in ((cos, "cos"), (sin, "sin")):
            if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32 or \
                    t.get_device() != x.get_device():
                raise TypeError("%s must be an fp32 tensor on %s" % (n, x.device))
        shape = cos.shape
        if len(shape) not in (2, 3) or sin.shape != shape or shape[-2] != S or \
                (len(shape) == 3 and shape[0] != B):
            raise ValueError("cos and sin must be [%d, rot / 2] or [%d, %d, rot / 2], got %s and %s" %
                             (S, B, S, tuple(shape), tuple(sin.shape)))
        cp, sp = cos.data_ptr(), sin.data_ptr()
        if not cos.is_contiguous() or not sin.is_contiguous() or (cp | sp) & 15:
            raise ValueError("cos and sin must be contiguous and 16-byte aligned")
        rot = 2 * shape[-1]
        stride = S * shape[-1] if len(shape) == 3 else 0
        if rot > D or rot % (16 if halves else 8):
            raise ValueError("cos and sin turn %d of %d elements of a head: at most all, in "
                             "multiples of %d" % (rot, D, 16 if halves else 8))
    if inverse is not None and order is None:
        raise ValueError("src and dst come together")
    return _pack_norm(B, S, rows, D, code, _DTYPES[wdtype], rot, 1 if halves else 0, eps, wq, wk, cp,
                      sp, stride, _vector(order, "the order", torch.int32, order_len, x),
                      _vector(inverse, "the other order", torch.int32, inverse_len, x))


def vsa_norm_rope(q, k=None, v=None, q_weight=None, k_weight=None, cos=None, sin=None, src=None,
                  halves=False, eps=1e-6, q_out=None, k_out=None, v_out=None, stream=None, dst=None):
    """RMS norm of each head of q and k by itself (not over all heads together), rotation by the
    table, and the move from token order to attention rows; v is only moved.

    q, k, v: [B, S, H, D] (bf16, fp16 or fp32; D a multiple of 8 up to 256; k and v may be None or
    have other head counts).  q_weight, k_weight: [D], fp32 or the activations' type (None: ones).
    cos, sin: fp32 [S, rot / 2] or [B, S, rot / 2] of each token's angles (None: no rotation); the
    first rot elements of a head are turned, in pairs (2i, 2i + 1) or, with halves, (i, i + rot/2).
    src: int32 [rows], the token of each output row, -1 for a row of zeros (None: row t is token
    t).  dst: the order that the backward will be given, if src is to be checked against it: a row
    whose token it does not send back raises DEVERR_ORDER (a token may go to several rows, but its
    gradients come from one).  Returns (q_out, k_out, v_out), [B, H, rows, D]; None where the input
    is None."""
    if stream is not None:
        return _on(stream, vsa_norm_rope, q, k, v, q_weight, k_weight, cos, sin, src, halves, eps,
                   q_out, k_out, v_out, dst=dst)
    _cuda(q, "q")
    B, S, _, D = q.shape
    rows = S if src is None else src.numel()
    op = _norm_rope_op(q, rows, q_weight, k_weight, cos, sin, src, rows, dst, S, halves, eps)
    dtype, where, device = q.dtype, q.device, q.get_device()
    ins, outs, res = [], [], []
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
        ins.append(_heads(x, name, (B, S, H, D), dtype, device, True))
        if y is None:
            y = torch.empty((B, H, rows, D), dtype=dtype, device=where)
            outs.append(_pack_heads(y.data_ptr(), H * rows * D, rows * D, D, H))
        else:
            outs.append(_heads(y, name + "_out", (B, H, rows, D), dtype, device))
        res.append(y)
    _call("vsa_norm_rope_fwd", op, *ins, *outs, _current(device))
    return tuple(res)


def vsa_norm_rope_bwd(dq_out, dk_out, dv_out, q, k=None, q_weight=None, k_weight=None, cos=None,
                      sin=None, dst=None, halves=False, eps=1e-6, dq=None, dk=None, dv=None,
                      need_dweight=True, workspace=None, stream=None, src=None):
    """Gradients of vsa_norm_rope: dq_out, dk_out, dv_out [B, H, rows, D] are the gradients of its
    outputs (dk_out with k, dv_out may be None), q and k its inputs.  dst: int32 [S], the row of
    each token, -1 for a token that no row takes (None: row t).  src: the order that the forward was
    given, if dst is to be checked against it: a token whose row it does not fill from the token
    raises DEVERR_ORDER.  Returns (dq, dk, dv, dq_weight, dk_weight): dq, dk, dv in token order
    [B, S, H, D]; weight gradients in the weights' type, None for a weight that is None (or with
    need_dweight false)."""
    if stream is not None:
        return _on(stream, vsa_norm_rope_bwd, dq_out, dk_out, dv_out, q, k, q_weight, k_weight, cos,
                   sin, dst, halves, eps, dq, dk, dv, need_dweight, workspace, src=src)
    _cuda(q, "q")
    _cuda(dq_out, "dq_out")
    if (k is None) != (dk_out is None):
        raise ValueError("k and dk_out come together")
    B, S, _, D = q.shape
    rows = dq_out.shape[2]
    if dst is None and rows != S:
        raise ValueError("dq_out has %d rows for %d tokens, without dst" % (rows, S))
    op = _norm_rope_op(q, rows, q_weight, k_weight, cos, sin, dst, S, src, rows, halves, eps)
    dtype, where, device = q.dtype, q.device, q.get_device()
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
        dys.append(_heads(dy, "d%s_out" % name, (B, H, rows, D), dtype, device))
        shape = (B, S, H, D)
        if name != "v":
            xs.append(_heads(x, name, shape, dtype, device, True))
            dws.append(torch.empty_like(w) if w is not None and need_dweight else None)
        if dx is None:
            dx = torch.empty(shape, dtype=dtype, device=where)
            dxs.append(_pack_heads(dx.data_ptr(), S * H * D, D, H * D, H))
        else:
            dxs.append(_heads(dx, "d" + name, shape, dtype, device, True))
        res.append(dx)
    dwq, dwk = dws
    need = 0 if dwq is None and dwk is None else _norm_workspace(device, D)
    keep, wp, wn = _workspace(workspace, need, q)
    _call("vsa_norm_rope_bwd", op, *dys, *xs, *dxs, None if dwq is None else dwq.data_ptr(),
          None if dwk is None else dwk.data_ptr(), wp, wn, _current(device))
    return (*res, dwq, dwk)


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
    """(packed vsa_cross, its sizes)."""
    _cuda(q, "q")
    if not isinstance(k, torch.Tensor) or k.dim() != 4 or k.numel() == 0:
        raise ValueError("k must be a 4-D tensor with elements")
    B, H, Sq, D = q.shape
    _, Hk, Sk, _ = k.shape
    if D != vsa.HEAD_DIM:
        raise ValueError("head_dim must be %d, got %d" % (vsa.HEAD_DIM, D))
    if H % Hk:
        raise ValueError("%d query heads do not share %d key heads evenly" % (H, Hk))
    if sm_scale is None:
        sm_scale = D ** -0.5
    if not math.isfinite(sm_scale):
        raise ValueError("sm_scale must be finite")
    sizes = (B, H, Hk, Sq, Sk, D)
    return _pack_cross(*sizes, sm_scale, _vector(kv_len, "kv_len", torch.int32, B, q)), sizes


def _operand(t, name, shape, device):
    return _heads(t, name, shape, torch.bfloat16, device, False, True)


def _lse(lse, shape, like):
    if not isinstance(lse, torch.Tensor) or lse.get_device() != like.get_device() or \
            lse.dtype is not torch.float32:
        raise TypeError("lse must be an fp32 tensor on %s" % like.device)
    if lse.shape != shape or not lse.is_contiguous():
        raise ValueError("lse must be contiguous %s, got %s" % (tuple(shape), tuple(lse.shape)))
    return lse.data_ptr()


def vsa_cross_fwd(q, k, v, kv_len=None, sm_scale=None, o=None, lse=None, workspace=None,
                  stream=None):
    """Attention of q [B, H, Sq, 128] to k, v [B, Hk, Sk, 128] (bf16; H a multiple of Hk), over the
    first kv_len[b] keys (int32 [B]; None: all).  sm_scale defaults to 1/sqrt(128).  Returns (o in
    q's memory order, lse fp32 [B, H, Sq], base 2); without a visible key o = 0 and lse = -inf."""
    if stream is not None:
        return _on(stream, vsa_cross_fwd, q, k, v, kv_len, sm_scale, o, lse, workspace)
    op, sizes = _cross_op(q, k, kv_len, sm_scale)
    B, H, Hk, Sq, Sk, D = sizes
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, Sq), dtype=torch.float32, device=q.device)
    qs, ks, device = (B, H, Sq, D), (B, Hk, Sk, D), q.get_device()
    args = (_operand(q, "q", qs, device), _operand(k, "k", ks, device), _operand(v, "v", ks, device),
            _operand(o, "o", qs, device), _lse(lse, qs[:3], q))
    keep, wp, wn = _workspace(workspace, _cross_workspace("vsa_cross_fwd_workspace_bytes", device,
                                                          *sizes), q)
    _call("vsa_cross_fwd", op, *args, wp, wn, _current(device))
    return o, lse


def vsa_cross_bwd(dout, q, k, v, o, lse, kv_len=None, sm_scale=None, dq=None, dk=None, dv=None,
                  workspace=None, stream=None):
    """Gradients of vsa_cross_fwd from dout, its inputs, and the o and lse that it returned.
    Returns (dq, dk, dv), each in its input's memory order; rows of dk and dv at or past
    kv_len[b] are exact zeros."""
    if stream is not None:
        return _on(stream, vsa_cross_bwd, dout, q, k, v, o, lse, kv_len, sm_scale, dq, dk, dv,
                   workspace)
    op, sizes = _cross_op(q, k, kv_len, sm_scale)
    B, H, Hk, Sq, Sk, D = sizes
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    qs, ks, device = (B, H, Sq, D), (B, Hk, Sk, D), q.get_device()
    args = (_operand(dout, "dout", qs, device), _operand(q, "q", qs, device),
            _operand(k, "k", ks, device), _operand(v, "v", ks, device),
            _operand(o, "o", qs, device), _lse(lse, qs[:3], q), _operand(dq, "dq", qs, device),
            _operand(dk, "dk", ks, device), _operand(dv, "dv", ks, device))
    keep, wp, wn = _workspace(workspace, _cross_workspace("vsa_cross_bwd_workspace_bytes", device,
                                                          *sizes), q)
    _call("vsa_cross_bwd", op, *args, wp, wn, _current(device))
    return dq, dk, dv


def vsa_layer_device_error(stream=None):
    """Synchronise the stream; return and clear the device error bits that these operators have
    raised on the current device since the last call."""
    bits = ctypes.c_uint32(0)
    handle = (torch.cuda.current_stream() if stream is None else stream).cuda_stream
    vsa._check(_lib().vsa_layer_device_error(ctypes.byref(bits), handle), "vsa_layer_device_error")
    return int(bits.value)
