"""The operators that make a whole transformer block of the attention layer: thin binding of
include/vsa_block.h, with the C entry points' names.

    x, h = block.vsa_gate_norm(x, y, gate, scale=scale, shift=shift)   # x + gate y, norm, modulation
    out, _ = block.vsa_linear(h, weight, bias, act="gelu_tanh")

Argument marshalling only, as in `layer`: every step runs in libvsa.so's kernels on the caller's
stream, and outputs and workspaces that are not passed are allocated here with torch (on that
stream).  Device error bits are those of `layer.vsa_layer_device_error`.  `autograd.gate_norm`,
`autograd.linear` and `autograd.mlp` are the differentiable forms.
"""
import ctypes
import functools
import struct

import torch

from . import vsa
from .layer import _DTYPES, _current, _on, _workspace

KINDS = {"layer": 0, "rms": 1}
MAX_TOKENS = 1 << 30      # and rows
ACTS = {None: 0, "gelu": 1, "gelu_tanh": 2, "silu": 3}


class VsaTokens(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64)]


class VsaModulation(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64),
                ("group_stride", ctypes.c_int64)]


class VsaGateNorm(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("tokens", ctypes.c_int32), ("channels", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("kind", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("branch_dtype", ctypes.c_int32), ("mod_dtype", ctypes.c_int32),
                ("weight_dtype", ctypes.c_int32), ("eps", ctypes.c_float), ("post_eps", ctypes.c_float),
                ("gate", VsaModulation), ("scale", VsaModulation), ("shift", VsaModulation),
                ("post_weight", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p)]


class VsaGateNormGrads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("gate", "scale", "shift", "post_weight", "weight", "bias")]


class VsaMatrix(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64)]


class VsaLinear(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("bias_dtype", ctypes.c_int32), ("act", ctypes.c_int32),
                ("weight", VsaMatrix), ("bias", ctypes.c_void_p)]


_G = ctypes.POINTER(VsaGateNorm)
_T = ctypes.POINTER(VsaTokens)
_GG = ctypes.POINTER(VsaGateNormGrads)
_L = ctypes.POINTER(VsaLinear)
_M = ctypes.POINTER(VsaMatrix)
_P = ctypes.c_void_p
_SZ = ctypes.c_size_t

# Every symbol include/vsa_block.h declares, with its (restype, argtypes).
SIGNATURES = {
    "vsa_gate_norm_fwd": (ctypes.c_int, [_G] + [_T] * 4 + [_P]),
    "vsa_gate_norm_bwd_workspace_bytes": (_SZ, [_G]),
    "vsa_gate_norm_bwd": (ctypes.c_int, [_G] + [_T] * 6 + [_GG, _P, _SZ, _P]),
    "vsa_linear_fwd_workspace_bytes": (_SZ, [_L]),
    "vsa_linear_bwd_workspace_bytes": (_SZ, [_L]),
    "vsa_linear_fwd": (ctypes.c_int, [_L] + [_M] * 4 + [_P, _SZ, _P]),
    "vsa_linear_bwd": (ctypes.c_int, [_L, ctypes.c_int32] + [_M] * 6 + [_P, _P, _SZ, _P]),
}

# Structures go over as packed bytes, one call into C each (see layer.py).
_pack_tokens = struct.Struct("@P2q").pack
_pack_norm = struct.Struct("@9i2fPqqPqqPqq3P").pack
_pack_grads = struct.Struct("@6P").pack
_pack_matrix = struct.Struct("@Pq").pack
_pack_linear = struct.Struct("@6iPqP").pack

_Tensor, _empty, _empty_like = torch.Tensor, torch.empty, torch.empty_like


def _current_device():
    return torch._C._cuda_getDevice()


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
            fn.argtypes = [ctypes.c_char_p if t in (_G, _T, _GG, _L, _M) else t for t in types]
        _calls = calls
    status = _calls[name](*args)
    if status != 0:
        vsa._check(status, name)


# ------------------------------------------------------------------------------- arguments

def _first(t, name, dims):
    """The index of the current device, after checking that the tensor is on it."""
    if isinstance(t, _Tensor):
        device = t.get_device()
        if device >= 0 and device == _current_device() and dims[0] <= t.dim() <= dims[1] and t.numel():
            return device
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dim() < dims[0] or t.dim() > dims[1]:
        raise ValueError("%s has %d dimensions" % (name, t.dim()))
    if t.numel() == 0:
        raise ValueError("%s is empty: %s" % (name, tuple(t.shape)))
    raise ValueError("%s is on %s, which is not the current device" % (name, t.device))


def _like(t, name, shape, dtype, device):
    if not isinstance(t, torch.Tensor) or t.get_device() != device:
        raise TypeError("%s must be a tensor on cuda:%d" % (name, device))
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _misaligned(name, t):
    return ValueError("%s: the last dimension must be contiguous, and the data and the other strides "
                      "multiples of 16 bytes (strides %s)" % (name, t.stride()))


def _strides3(t, name):
    """(address, stride of dimension 0, of dimension 1) of a 3-D tensor."""
    s0, s1, s2 = t.stride()
    n0, n1, n2 = t.shape
    ptr = t.data_ptr()
    used = (s0 if n0 > 1 else 0) | (s1 if n1 > 1 else 0)
    if (s2 != 1 and n2 > 1) or ptr & 15 or used & (3 if t.dtype is torch.float32 else 7):
        raise _misaligned(name, t)
    return ptr, s0, s1


def _tokens(t, name, shape, dtype, device):
    """The [B, S, C] tensor t as a packed vsa_tokens, after checking it."""
    if not isinstance(t, _Tensor) or t.get_device() != device or t.dtype is not dtype or t.shape != shape:
        _like(t, name, shape, dtype, device)
    s0, s1, s2 = t.stride()
    ptr = t.data_ptr()
    if s1 != shape[2] or s0 != shape[1] * s1 or s2 != 1 or ptr & 15:      # not the usual case
        return _pack_tokens(*_strides3(t, name))
    return _pack_tokens(ptr, s0, s1)


def _new_tokens(like, shape, dtype):
    """A tensor for an output shaped like `like`, contiguous, and its packed vsa_tokens."""
    # (empty_like takes three quarters of empty's time.)
    if like.dtype is dtype and like.is_contiguous():
        t = _empty_like(like)
    else:
        t = _empty(shape, dtype=dtype, device=like.device)
    return t, _pack_tokens(t.data_ptr(), shape[1] * shape[2], shape[2])


def _vector(t, name, dtype, n, device):
    """The address of a contiguous 1-D tensor, or 0 for None."""
    if t is None:
        return 0
    if not isinstance(t, _Tensor) or t.get_device() != device or t.dtype is not dtype or t.shape != (n,):
        _like(t, name, (n,), dtype, device)
    ptr = t.data_ptr()
    if ptr & 15 or not t.is_contiguous():
        raise ValueError("%s must be contiguous and 16-byte aligned" % name)
    return ptr


def _param_dtype(tensors, branch, what):
    """The one type of the parameters that are given: fp32 or the branch's."""
    dtype = None
    for t in tensors:
        if t is not None:
            d = getattr(t, "dtype", None)
            if d is not dtype:
                if dtype is not None or (d is not branch and d is not torch.float32):
                    raise TypeError("%s must all be fp32 or all %s" % (what, branch))
                dtype = d
    return branch if dtype is None else dtype


# ------------------------------------------------------------------------------- gate_norm

_NO_MODULATION = (0, 0, 0, None)


def _modulation(m, name, B, S, C, dtype, device):
    """(address, batch stride, group stride, groups) of a [B, C] or [B, G, C] modulation."""
    if m is None:
        return _NO_MODULATION
    if not isinstance(m, _Tensor) or m.dim() not in (2, 3):
        raise TypeError("%s must be a [B, C] or [B, groups, C] tensor" % name)
    if m.dim() == 2:
        m = m.unsqueeze(1)
    n0, G, n2 = m.shape
    if m.get_device() != device or m.dtype is not dtype or n0 != B or n2 != C:
        _like(m, name, (B, G, C), dtype, device)
    if G < 1 or S % G:
        raise ValueError("%s: %d tokens do not share %d groups evenly" % (name, S, G))
    s0, s1, s2 = m.stride()
    ptr = m.data_ptr()
    if s2 != 1 or ptr & 15 or (s0 | s1) & 7:                                # not the usual case
        ptr, s0, s1 = _strides3(m, name)
    return ptr, s0, s1, G


def _gate_norm_op(x, branch, y, gate, post_weight, weight, bias, scale, shift, kind, eps, post_eps):
    """(packed vsa_gate_norm, its batch, tokens, channels, groups)."""
    B, S, C = x.shape
    dtype, device = x.dtype, x.get_device()
    if dtype not in _DTYPES:
        raise TypeError("the stream must be bf16, fp16 or fp32, got %s" % dtype)
    if branch is not dtype and (dtype is not torch.float32 or branch not in _DTYPES):
        raise TypeError("the branch must be %s%s, got %s" %
                        (dtype, " or 16-bit" if dtype is torch.float32 else "", branch))
    if C % 8 or not 8 <= C <= 8192:
        raise ValueError("channels must be a multiple of 8 up to 8192, got %d" % C)
    if B * S > MAX_TOKENS:
        raise ValueError("there may be up to 2^30 tokens, got %d" % (B * S))
    if kind not in KINDS:
        raise ValueError("kind must be one of %s, got %r" % (sorted(KINDS), kind))
    if y is None and (gate is not None or post_weight is not None):
        raise ValueError("gate and post_weight need y")
    mdtype = _param_dtype((gate, scale, shift), branch, "gate, scale and shift")
    wdtype = _param_dtype((post_weight, weight, bias), branch, "the weights and the bias")
    gp, gs0, gs1, G = _modulation(gate, "gate", B, S, C, mdtype, device)
    cp, cs0, cs1, G1 = _modulation(scale, "scale", B, S, C, mdtype, device)
    tp, ts0, ts1, G2 = _modulation(shift, "shift", B, S, C, mdtype, device)
    G = G or G1 or G2 or 1
    if (G1 or G) != G or (G2 or G) != G:
        raise ValueError("gate, scale and shift must have the same groups, got %s" %
                         sorted({n for n in (G, G1, G2) if n}))
    op = _pack_norm(B, S, C, G, KINDS[kind], _DTYPES[dtype], _DTYPES[branch], _DTYPES[mdtype],
                    _DTYPES[wdtype], eps, post_eps, gp, gs0, gs1, cp, cs0, cs1, tp, ts0, ts1,
                    _vector(post_weight, "post_weight", wdtype, C, device),
                    _vector(weight, "weight", wdtype, C, device), _vector(bias, "bias", wdtype, C, device))
    return op, (B, S, C, G)


@functools.lru_cache(maxsize=256)
def _norm_workspace(device, B, S, C, G, dtype, branch, weights):
    """Workspace bytes of a backward of these sizes and types (a pure function of them), with the gradients of
    weights or without."""
    some, dtype, branch = VsaModulation(16, 0, 0), _DTYPES[dtype], _DTYPES[branch]
    return _lib().vsa_gate_norm_bwd_workspace_bytes(
        VsaGateNorm(B, S, C, G, 0, dtype, branch, branch, branch, 0.0, 0.0, some, some, some, 16 if weights else None,
                    None, None))


def vsa_gate_norm(x, y=None, gate=None, post_weight=None, weight=None, bias=None, scale=None,
                  shift=None, kind="layer", eps=1e-6, post_eps=1e-6, h_dtype=None, x_out=None, h=None,
                  stream=None):
    """The end of one branch and the start of the next: x' = x + gate * u with u = y, or the RMS norm
    of y times post_weight; h = (norm(x') * weight + bias) * (1 + scale) + shift.  What is None drops
    out; without y, x' is x.

    x: [B, S, C] (bf16, fp16 or fp32; C a multiple of 8 up to 8192).  y: [B, S, C] of x's type, or
    16-bit with an fp32 x.  gate, scale, shift: [B, C], or [B, G, C] with a row for every S / G
    tokens; post_weight, weight, bias: [C]; each of the two sets in fp32 or all of y's type.  kind:
    "layer" or "rms".  h_dtype: without y, the type of h (x's, or 16-bit with an fp32 x).  x_out may
    be x, for a stream that is updated in place.  Returns (x', h)."""
    if stream is not None:
        return _on(stream, vsa_gate_norm, x, y, gate, post_weight, weight, bias, scale, shift, kind, eps,
                   post_eps, h_dtype, x_out, h)
    device = _first(x, "x", (3, 3))
    branch = getattr(y, "dtype", None) if y is not None else x.dtype if h_dtype is None else h_dtype
    if h_dtype is not None and h_dtype is not branch:
        raise TypeError("h has y's type, %s" % branch)
    op, (B, S, C, _) = _gate_norm_op(x, branch, y, gate, post_weight, weight, bias, scale, shift, kind,
                                     eps, post_eps)
    shape, dtype = x.shape, x.dtype
    xs = _tokens(x, "x", shape, dtype, device)
    if h is None:
        h, hs = _new_tokens(x if y is None else y, shape, branch)
    else:
        hs = _tokens(h, "h", shape, branch, device)
    if y is None:
        if x_out is not None:
            raise ValueError("x_out is given without y")
        _call("vsa_gate_norm_fwd", op, xs, None, None, hs, _current(device))
        return x, h
    ys = _tokens(y, "y", shape, branch, device)
    if x_out is None:
        x_out, os = _new_tokens(x, shape, dtype)
    else:
        os = _tokens(x_out, "x_out", shape, dtype, device)
    _call("vsa_gate_norm_fwd", op, xs, ys, os, hs, _current(device))
    return x_out, h


def vsa_gate_norm_bwd(dh, dx_out, x_out, y=None, gate=None, post_weight=None, weight=None, bias=None,
                      scale=None, shift=None, kind="layer", eps=1e-6, post_eps=1e-6, need_dparams=True,
                      dx=None, dy=None, workspace=None, stream=None):
    """Gradients of vsa_gate_norm from those of its outputs (dx_out None: zero), the x' that it
    returned and its other inputs.  Returns (dx, dy, dgate, dpost_weight, dweight, dbias, dscale,
    dshift), None for what is None; the parameters' gradients have their types.  need_dparams: whether
    those are wanted, or six of it, for gate, post_weight, weight, bias, scale and shift.  dx may be
    dx_out."""
    if stream is not None:
        return _on(stream, vsa_gate_norm_bwd, dh, dx_out, x_out, y, gate, post_weight, weight, bias, scale,
                   shift, kind, eps, post_eps, need_dparams, dx, dy, workspace)
    device = _first(x_out, "x_out", (3, 3))
    branch = getattr(dh if y is None else y, "dtype", None)
    op, sizes = _gate_norm_op(x_out, branch, y, gate, post_weight, weight, bias, scale, shift, kind, eps,
                              post_eps)
    B, S, C, _ = sizes
    shape, dtype, where = x_out.shape, x_out.dtype, x_out.device
    ins = [_tokens(dh, "dh", shape, branch, device),
           None if dx_out is None else _tokens(dx_out, "dx_out", shape, dtype, device),
           _tokens(x_out, "x_out", shape, dtype, device),
           None if y is None else _tokens(y, "y", shape, branch, device)]
    if dx is None:
        dx, packed = _new_tokens(x_out, shape, dtype)
        ins.append(packed)
    else:
        ins.append(_tokens(dx, "dx", shape, dtype, device))
    if y is None:
        if dy is not None:
            raise ValueError("dy is given without y")
        ins.append(None)
    elif dy is None:
        dy, packed = _new_tokens(y, shape, branch)
        ins.append(packed)
    else:
        ins.append(_tokens(dy, "dy", shape, branch, device))
    wanted = need_dparams if isinstance(need_dparams, (tuple, list)) else (need_dparams,) * 6
    if len(wanted) != 6:
        raise ValueError("need_dparams must be one or six truth values, got %d" % len(wanted))
    grads = [None if p is None or not n else _empty_like(p) if p.is_contiguous() else
             _empty(p.shape, dtype=p.dtype, device=where)
             for p, n in zip((gate, post_weight, weight, bias, scale, shift), wanted)]
    dgate, dpost, dweight, dbias, dscale, dshift = grads
    weights = dpost is not None or dweight is not None or dbias is not None
    need = 0
    if weights or dgate is not None or dscale is not None or dshift is not None:
        need = _norm_workspace(device, *sizes, dtype, branch, weights)
    keep, wp, wn = _workspace(workspace, need, x_out)
    places = _pack_grads(*(0 if g is None else g.data_ptr()
                           for g in (dgate, dscale, dshift, dpost, dweight, dbias)))
    _call("vsa_gate_norm_bwd", op, *ins, places, wp, wn, _current(device))
    return dx, dy, dgate, dpost, dweight, dbias, dscale, dshift


# ------------------------------------------------------------------------------- linear

def _matrix(t, name, rows, columns, dtype, device):
    """A tensor [..., columns] of `rows` rows at one stride, as a packed vsa_matrix."""
    if not isinstance(t, _Tensor) or t.get_device() != device:
        raise TypeError("%s must be a tensor on cuda:%d" % (name, device))
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    shape = t.shape
    if len(shape) < 1 or shape[-1] != columns or t.numel() != rows * columns:
        raise ValueError("%s must have %d rows of %d, got %s" % (name, rows, columns, tuple(shape)))
    ptr = t.data_ptr()
    if t.is_contiguous():
        if ptr & 15:
            raise _misaligned(name, t)
        return _pack_matrix(ptr, columns)
    strides = t.stride()
    step = count = None
    for n, s in zip(reversed(shape[:-1]), reversed(strides[:-1])):
        if n == 1:
            continue
        if step is None:
            step, count = s, n
        elif s != step * count:
            raise ValueError("%s: the rows must lie at one stride (shape %s, strides %s)" %
                             (name, tuple(shape), strides))
        else:
            count *= n
    if step is None:
        step = columns
    if strides[-1] != 1 or ptr & 15 or step & 7:
        raise _misaligned(name, t)
    if step < columns:
        raise ValueError("%s: the rows must not overlap (strides %s)" % (name, strides))
    return _pack_matrix(ptr, step)


def _linear_op(x, weight, bias, act):
    """(packed vsa_linear, rows, in_features, out_features)."""
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2 or weight.numel() == 0:
        raise ValueError("weight must be [out_features, in_features]")
    N, K = weight.shape
    dtype, device = x.dtype, x.get_device()
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise TypeError("matrices must be bf16 or fp16, got %s" % dtype)
    if K % 8 or N % 8:
        raise ValueError("in_features and out_features must be multiples of 8, got %d and %d" % (K, N))
    if act not in ACTS:
        raise ValueError("act must be None, 'gelu', 'gelu_tanh' or 'silu', got %r" % (act,))
    bdtype = dtype if bias is None else getattr(bias, "dtype", None)
    if bdtype is not dtype and bdtype is not torch.float32:
        raise TypeError("bias must be fp32 or %s, got %s" % (dtype, bdtype))
    ptr = _vector(bias, "bias", bdtype, N, device)
    _like(weight, "weight", (N, K), dtype, device)
    at, step = weight.data_ptr(), weight.stride(0) if N > 1 else K
    if (weight.stride(1) != 1 and K > 1) or at & 15 or step & 7:
        raise _misaligned("weight", weight)
    if step < K:
        raise ValueError("weight: the rows must not overlap (strides %s)" % (weight.stride(),))

    def make(rows):
        if rows > MAX_TOKENS:
            raise ValueError("there may be up to 2^30 rows, got %d" % rows)
        return _pack_linear(rows, K, N, _DTYPES[dtype], _DTYPES[bdtype], ACTS[act], at, step, ptr)
    return make, N, K


@functools.lru_cache(maxsize=256)
def _linear_workspace(name, device, rows, K, N, act):
    """Workspace bytes of a call of these sizes (a pure function of them)."""
    return getattr(_lib(), name)(VsaLinear(rows, K, N, 0, 0, act, VsaMatrix(16, K), None))


def vsa_linear(x, weight, bias=None, act=None, residual=None, need_pre=False, out=None, pre=None,
               workspace=None, stream=None):
    """out = act(x weight^T + bias) + residual.

    x: [..., K] (bf16 or fp16), its rows at one stride; weight: [N, K] of x's type; bias: [N], fp32 or
    x's type; K and N multiples of 8.  act: None, "gelu", "gelu_tanh" or "silu".  residual: [..., N].
    Returns (out [..., N], pre), pre being x weight^T + bias rounded to x's type, which the backward of
    an activation takes (None unless need_pre or a place for it is given)."""
    if stream is not None:
        return _on(stream, vsa_linear, x, weight, bias, act, residual, need_pre, out, pre, workspace)
    device = _first(x, "x", (1, 64))
    make, N, K = _linear_op(x, weight, bias, act)
    dtype = x.dtype
    rows = x.numel() // x.shape[-1]
    op = make(rows)
    xs = _matrix(x, "x", rows, K, dtype, device)
    rs = None if residual is None else _matrix(residual, "residual", rows, N, dtype, device)
    shape = (*x.shape[:-1], N)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=x.device)
    if pre is None and need_pre:
        pre = _empty_like(out) if out.is_contiguous() else _empty(shape, dtype=dtype, device=x.device)
    keep, wp, wn = _workspace(workspace, _linear_workspace("vsa_linear_fwd_workspace_bytes", device, rows, K, N,
                                                           ACTS[act]), x)
    _call("vsa_linear_fwd", op, xs, rs, _matrix(out, "out", rows, N, dtype, device),
          None if pre is None else _matrix(pre, "pre", rows, N, dtype, device), wp, wn, _current(device))
    return out, pre


def vsa_linear_bwd(dout, x, weight, bias=None, act=None, pre=None, x_act=None, x_pre=None, need_dx=True,
                   need_dweight=True, dx=None, dweight=None, dbias=None, workspace=None, stream=None):
    """Gradients of vsa_linear from dout (which is also the residual's), its inputs and, with an
    activation, the pre that it returned.  With x_act, x is x_act(x_pre) and dx is taken on through it:
    the gradient of x_pre.  bias is taken for its type alone.  Returns (dx [..., K], dweight [N, K],
    dbias [N]), None for what is not wanted (dbias: without a bias)."""
    if stream is not None:
        return _on(stream, vsa_linear_bwd, dout, x, weight, bias, act, pre, x_act, x_pre, need_dx,
                   need_dweight, dx, dweight, dbias, workspace)
    device = _first(x, "x", (1, 64))
    make, N, K = _linear_op(x, weight, bias, act)
    if x_act not in ACTS:
        raise ValueError("x_act must be None, 'gelu', 'gelu_tanh' or 'silu', got %r" % (x_act,))
    if (act is None) != (pre is None) or (x_act is None) != (x_pre is None):
        raise ValueError("an activation and what went into it come together")
    dtype, where = x.dtype, x.device
    rows = x.numel() // x.shape[-1]
    op = make(rows)
    if dx is None and need_dx:
        dx = _empty_like(x) if x.is_contiguous() else _empty(x.shape, dtype=dtype, device=where)
    if dweight is None and need_dweight:
        dweight = _empty_like(weight) if weight.is_contiguous() else _empty((N, K), dtype=dtype, device=where)
    if bias is None:
        if dbias is not None:
            raise ValueError("dbias is given without bias")
    elif dbias is None:
        dbias = _empty_like(bias)
    if dx is None and dweight is None and dbias is None:
        return None, None, None

    def matrix(t, name, n):
        return None if t is None else _matrix(t, name, rows, n, dtype, device)

    if dweight is not None and dweight.shape != (N, K):
        raise ValueError("dweight must be %s, got %s" % ((N, K), tuple(dweight.shape)))
    keep, wp, wn = _workspace(workspace, _linear_workspace("vsa_linear_bwd_workspace_bytes", device, rows, K, N,
                                                           ACTS[act]), x)
    _call("vsa_linear_bwd", op, ACTS[x_act], matrix(dout, "dout", N), matrix(x, "x", K), matrix(pre, "pre", N),
          matrix(x_pre, "x_pre", K), matrix(dx, "dx", K),
          None if dweight is None else _matrix(dweight, "dweight", N, K, dtype, device),
          _vector(dbias, "dbias", None if bias is None else bias.dtype, N, device), wp, wn, _current(device))
    return dx, dweight, dbias
