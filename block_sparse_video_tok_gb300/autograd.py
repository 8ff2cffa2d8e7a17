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
"""
import functools

import torch

from . import layer, vsa


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


def _aligned(g):
    """g, copied where its address or strides are not the kernels' (a slice that starts off 16 bytes, an
    expanded or a transposed gradient)."""
    unit = 16 // g.element_size()
    if g.data_ptr() % 16:
        return g.clone(memory_format=torch.contiguous_format)
    if g.stride(-1) == 1 and all(s and s % unit == 0 for s in g.stride()[:-1]):
        return g
    return g.contiguous()


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
