"""torch.autograd binding of the block-sparse attention path.

`block_sparse_attention(q, k, v, q2k_idx, q2k_num, vbs, sm_scale)` returns O and records, for
the backward, what the backward kernels consume: Q, K, V, O, the base-2 lse (M form) of the
forward, and the inverted selection k2q.  The FastVideo autograd path inverts the selection
(q2k -> k2q) right before its sm_100a backward (block_sparse_attn_bwd_sm100a.py,
block_sparse_attn_backward_sm100a; the custom op's backward in the compare page
main...vsa_bwd_fix, _backward_sm100a); here the forward does it once and saves the result, so
the backward starts on its preprocess at once, and a caller whose layers share one selection can
invert it once for all of them (`k2q=` below).

Argument marshalling only: every step runs in libvsa.so's kernels through `vsa`.  Nothing here can be
differentiated twice: doing so raises.

A backward is captured into a CUDA graph together with its forward, after warm-up on a side stream, and
while no autograd graph of the same leaves that was made outside the capture is alive: torch accumulates a
leaf's gradient on the stream its graph was made on, which a capture cannot join.
"""
import functools

import torch

from . import block, layer, vsa


class _FirstDerivative(torch.autograd.Function):
    """compute(), as a function of the tensors it depends on that has no derivative."""

    @staticmethod
    def forward(ctx, compute, *tensors):
        return compute()

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("the gradients of these operators can be taken once only: their backward "
                           "kernels have no derivative")


def _once(backward):
    """A backward whose results refuse to be differentiated.  The kernels record nothing, so with
    create_graph the results would pass for constants.  (torch's once_differentiable refuses only
    where the incoming gradients require one; the results depend on the saved tensors too, and on
    them alone where the loss is a sum.)"""
    @functools.wraps(backward)
    def wrapper(ctx, *grads):
        if not torch.is_grad_enabled():              # no create_graph
            return backward(ctx, *grads)
        return _FirstDerivative.apply(lambda: backward(ctx, *grads), *grads, *ctx.saved_tensors)
    return wrapper


class BlockSparseAttention(torch.autograd.Function):
    """O = block-sparse softmax(Q K^T * sm_scale) V over 64- or 128-token blocks.

    Inputs: bf16 [B, H, S, 128] q, k, v (S = block * nb); int32 q2k_idx [B, H, nb, topk] and
    q2k_num [B, H, nb] (the kv blocks each q block attends to, a set: duplicates count once);
    int32 vbs [nb] (valid tokens of each kv block); sm_scale; k2q_idx / k2q_num: the inverted
    selection (vsa_invert_indices of q2k), or None to invert it here.  Outputs O (bf16, same
    shape as q) and lse (fp32 [B, H, S], not differentiable).  Gradients flow to q, k and v; dq
    and dk carry sm_scale, dv does not.
    """

    @staticmethod
    def forward(ctx, q, k, v, q2k_idx, q2k_num, vbs, sm_scale, k2q_idx=None, k2q_num=None):
        o, lse = vsa.vsa_fwd(q, k, v, q2k_idx, q2k_num, vbs, sm_scale)
        if k2q_idx is None or k2q_num is None:
            k2q_idx, k2q_num = vsa.vsa_invert_indices(q2k_idx, q2k_num, vbs.numel())
        ctx.save_for_backward(q, k, v, o, lse, k2q_idx, k2q_num, vbs)
        ctx.sm_scale = sm_scale
        ctx.mark_non_differentiable(lse)
        return o, lse

    @staticmethod
    @_once
    def backward(ctx, do, _dlse):
        q, k, v, o, lse, k2q_idx, k2q_num, vbs = ctx.saved_tensors
        dq, dk, dv = vsa.vsa_bwd(_aligned(do.contiguous()), q, k, v, o, lse, k2q_idx, k2q_num, vbs,
                                 ctx.sm_scale)
        return dq, dk, dv, None, None, None, None, None, None


def block_sparse_attention(q, k, v, q2k_idx, q2k_num, vbs, sm_scale=None, k2q=None):
    """O of block-sparse attention, differentiable in q, k and v (see BlockSparseAttention).
    sm_scale defaults to 1/sqrt(head_dim).  k2q: optional (k2q_idx, k2q_num) of this selection,
    from vsa.vsa_invert_indices, for callers that reuse one selection in several calls; without
    it the forward inverts the selection once and saves it for the backward."""
    if sm_scale is None:
        sm_scale = q.shape[-1] ** -0.5
    k2q_idx, k2q_num = k2q if k2q is not None else (None, None)
    o, _ = BlockSparseAttention.apply(q, k, v, q2k_idx, q2k_num, vbs, float(sm_scale), k2q_idx,
                                      k2q_num)
    return o


class NormRope(torch.autograd.Function):
    """vsa_norm_rope of layer.py; gradients flow to q, k, v and the weights."""

    @staticmethod
    def forward(ctx, q, k, v, q_weight, k_weight, cos, sin, src, dst, halves, eps,
                recorded=True):
        recorded = recorded and any(ctx.needs_input_grad)
        if recorded and (src is None) != (dst is None):
            raise ValueError("a gradient needs both of the order's (src, dst)")
        out = layer.vsa_norm_rope(q, k, v, q_weight, k_weight, cos, sin, src, halves, eps,
                                  dst=dst if recorded else None)
        ctx.save_for_backward(q, k, q_weight, k_weight, cos, sin, src, dst)
        ctx.halves, ctx.eps, ctx.rows = halves, eps, out[0].shape[2]
        ctx.v_heads = None if v is None else v.shape[2]
        return out

    @staticmethod
    @_once
    def backward(ctx, dq_out, dk_out, dv_out):
        q, k, q_weight, k_weight, cos, sin, src, dst = ctx.saved_tensors
        grads = []
        for g, heads in ((dq_out, q.shape[2]), (dk_out, None if k is None else k.shape[2]),
                         (dv_out, ctx.v_heads)):
            if g is None and heads is not None:      # an output that the loss does not reach
                g = q.new_zeros((q.shape[0], heads, ctx.rows, q.shape[3]))
            grads.append(g if g is None else _aligned(g))
        need = ctx.needs_input_grad[3] or ctx.needs_input_grad[4]
        return layer.vsa_norm_rope_bwd(*grads, q, k, q_weight, k_weight, cos, sin, dst, ctx.halves,
                                       ctx.eps, need_dweight=need, src=src) + (None,) * 7


class CrossAttention(torch.autograd.Function):
    """vsa_cross of layer.py: (o, lse); gradients flow to q, k and v (lse is not differentiable)."""

    @staticmethod
    def forward(ctx, q, k, v, kv_len, sm_scale):
        o, lse = layer.vsa_cross_fwd(q, k, v, kv_len, sm_scale)
        ctx.save_for_backward(q, k, v, o, lse, kv_len)
        ctx.sm_scale = sm_scale
        ctx.mark_non_differentiable(lse)
        return o, lse

    @staticmethod
    @_once
    def backward(ctx, do, _dlse):
        q, k, v, o, lse, kv_len = ctx.saved_tensors
        return layer.vsa_cross_bwd(_aligned(do), q, k, v, o, lse, kv_len, ctx.sm_scale) + (None,) * 2


class GateNorm(torch.autograd.Function):
    """vsa_gate_norm of block.py: (x', h), or h alone without y; gradients flow to x, y and every
    parameter."""

    @staticmethod
    def forward(ctx, x, y, gate, post_weight, weight, bias, scale, shift, kind, eps, post_eps, h_dtype):
        ctx.set_materialize_grads(False)
        x_out, h = block.vsa_gate_norm(x, y, gate, post_weight, weight, bias, scale, shift, kind, eps,
                                       post_eps, h_dtype)
        ctx.save_for_backward(x_out, y, gate, post_weight, weight, bias, scale, shift)
        ctx.settings, ctx.h_dtype = (kind, eps, post_eps), h.dtype
        return h if y is None else (x_out, h)

    @staticmethod
    @_once
    def backward(ctx, *grads):
        dx_out, dh = grads if len(grads) == 2 else (None, grads[0])
        if dx_out is None and dh is None:
            return (None,) * 12
        x_out, y, *params = ctx.saved_tensors
        dh = torch.zeros(x_out.shape, dtype=ctx.h_dtype, device=x_out.device) if dh is None else _aligned(dh)
        return block.vsa_gate_norm_bwd(dh, None if dx_out is None else _aligned(dx_out), x_out, y, *params,
                                       *ctx.settings, need_dparams=ctx.needs_input_grad[2:8]) + (None,) * 4


class Linear(torch.autograd.Function):
    """vsa_linear of block.py; gradients flow to x, the weight, the bias and the residual."""

    @staticmethod
    def forward(ctx, x, weight, bias, residual, act, recorded=True):
        recorded = recorded and any(ctx.needs_input_grad)
        out, pre = block.vsa_linear(x, weight, bias, act, residual, need_pre=recorded and act is not None)
        ctx.save_for_backward(x, weight, bias, pre)
        ctx.act, ctx.residual = act, _shape(residual)
        return out

    @staticmethod
    @_once
    def backward(ctx, dout):
        x, weight, bias, pre = ctx.saved_tensors
        need = ctx.needs_input_grad
        g = _flat(dout)
        dx, dw, db = block.vsa_linear_bwd(g, x, weight, bias if need[2] else None, ctx.act, pre,
                                          need_dx=need[0], need_dweight=need[1])
        return dx, dw, db, dout.reshape(ctx.residual) if need[3] else None, None, None


class Mlp(torch.autograd.Function):
    """Two products with an activation between them; the backward of the second goes through the
    activation in the epilogue of its product."""

    @staticmethod
    def forward(ctx, x, w1, b1, w2, b2, residual, act, recorded=True):
        recorded = recorded and any(ctx.needs_input_grad)
        mid, pre = block.vsa_linear(x, w1, b1, act, need_pre=recorded)
        out, _ = block.vsa_linear(mid, w2, b2, residual=residual)
        ctx.save_for_backward(x, w1, b1, w2, b2, mid, pre)
        ctx.act, ctx.residual = act, _shape(residual)
        return out

    @staticmethod
    @_once
    def backward(ctx, dout):
        x, w1, b1, w2, b2, mid, pre = ctx.saved_tensors
        need = ctx.needs_input_grad
        first = need[0] or need[1] or need[2]
        dz, dw2, db2 = block.vsa_linear_bwd(_flat(dout), mid, w2, b2 if need[4] else None, x_act=ctx.act,
                                            x_pre=pre, need_dx=first, need_dweight=need[3])
        dx = dw1 = db1 = None
        if first:
            dx, dw1, db1 = block.vsa_linear_bwd(dz, x, w1, b1 if need[2] else None, need_dx=need[0],
                                                need_dweight=need[1])
        return dx, dw1, db1, dw2, db2, dout.reshape(ctx.residual) if need[5] else None, None, None


def _shape(t):
    return None if t is None else t.shape


def _aligned(g):
    """g, copied where its address or strides are not the kernels' (a slice that starts off 16 bytes, an
    expanded or a transposed gradient)."""
    unit = 16 // g.element_size()
    if g.data_ptr() % 16:
        return g.clone(memory_format=torch.contiguous_format)
    if g.stride(-1) == 1 and all(s and s % unit == 0 for s in g.stride()[:-1]):
        return g
    return g.contiguous()


def _flat(g):
    """_aligned, and copied where its rows do not lie at one stride (a gradient with its leading dimensions
    permuted)."""
    g = _aligned(g)
    if not g.is_contiguous():
        try:
            g.view(-1, g.shape[-1])
        except RuntimeError:
            return g.contiguous()
    return g


def norm_rope(q, k=None, v=None, q_weight=None, k_weight=None, cos=None, sin=None, order=None,
              halves=False, eps=1e-6):
    """Differentiable layer.vsa_norm_rope: the per-head norm and rotation of q and k in the pass
    that moves q, k and v [B, S, H, D] to [B, H, rows, D].  order: (src, dst) as from
    layer.video_token_order, or None.  The two must name each other, dst[src[r]] == r wherever
    src[r] >= 0 and src[dst[t]] == t wherever dst[t] >= 0, so that no token goes to two rows: the
    gradients follow dst alone, and where that does not hold, forward and backward raise
    layer.DEVERR_ORDER in the device's error word.  Returns (q, k, v) for block_sparse_attention."""
    src, dst = order if order is not None else (None, None)
    return NormRope.apply(q, k, v, q_weight, k_weight, cos, sin, src, dst, bool(halves), float(eps),
                          torch.is_grad_enabled())


def cross_attention(q, k, v, kv_len=None, sm_scale=None):
    """O of the attention of q [B, H, Sq, 128] to the first kv_len[b] of the keys and values
    [B, Hk, Sk, 128], differentiable in q, k and v (see layer.vsa_cross_fwd)."""
    if sm_scale is None:
        sm_scale = q.shape[-1] ** -0.5
    return CrossAttention.apply(q, k, v, kv_len, float(sm_scale))[0]


def gate_norm(x, y=None, gate=None, post_weight=None, weight=None, bias=None, scale=None, shift=None,
              kind="layer", eps=1e-6, post_eps=1e-6, h_dtype=None):
    """Differentiable block.vsa_gate_norm: (x', h) with x' = x + gate * y (y normalised first with a
    post_weight) and h = (norm(x') * weight + bias) * (1 + scale) + shift.  Without y, x' is x."""
    out = GateNorm.apply(x, y, gate, post_weight, weight, bias, scale, shift, kind, float(eps),
                         float(post_eps), h_dtype)
    return (x, out) if y is None else out


def linear(x, weight, bias=None, act=None, residual=None):
    """Differentiable block.vsa_linear: act(x weight^T + bias) + residual.  The residual has the output's rows,
    in any leading dimensions, and so has its gradient."""
    return Linear.apply(x, weight, bias, residual, act, torch.is_grad_enabled())


def mlp(x, w1, b1, w2, b2, act="gelu_tanh", residual=None):
    """act(x w1^T + b1) w2^T + b2 + residual, differentiable in all of them.  The backward keeps both
    sides of the activation, [..., w1's rows] each; the gradient between them is rounded to x's type once,
    and b1's sums it up so."""
    if act is None:
        raise ValueError("mlp needs an activation")
    return Mlp.apply(x, w1, b1, w2, b2, residual, act, torch.is_grad_enabled())
