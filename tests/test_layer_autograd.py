"""The torch bindings of autograd.py without a GPU: the kernels are replaced by plain torch forms that,
like them, record nothing, so what is tested is what the bindings do with gradients."""
import pytest
import torch

from block_sparse_video_tok_gb300 import autograd, layer, vsa
from tests import layer_ref as ref

F64 = torch.float64


@pytest.fixture
def plain(monkeypatch):
    """The kernels' entry points as torch forms in 64 bits, without a graph."""

    def norm_rope(q, k, v, q_weight, k_weight, cos, sin, src, halves, eps, *more, **names):
        def one(x, w):
            return None if x is None else ref.norm_rope_one(x, w, cos, sin, src, halves, eps, F64)[0].contiguous()
        return one(q, q_weight), one(k, k_weight), None if v is None else ref.move(v, src).contiguous()

    def norm_rope_bwd(dq, dk, dv, q, k, q_weight, k_weight, cos, sin, dst, halves, eps, need_dweight=True, **names):
        def one(dy, x, w):
            if x is None:
                return None, None
            (dx, _), (dw, _) = ref.norm_rope_one_bwd(dy, x, w, cos, sin, dst, halves, eps, F64, F64)
            return dx, dw if w is not None and need_dweight else None
        (dxq, dwq), (dxk, dwk) = one(dq, q, q_weight), one(dk, k, k_weight)
        return dxq, dxk, None if dv is None else ref.move(dv.transpose(1, 2), dst).transpose(1, 2), dwq, dwk

    def cross_fwd(q, k, v, kv_len, sm_scale):
        (o, _), (lse, _) = ref.cross_fwd(q, k, v, kv_len, sm_scale)
        return o, lse

    def cross_bwd(do, q, k, v, o, lse, kv_len, sm_scale):
        return tuple(x for x, _ in ref.cross_bwd(do, q, k, v, o, lse, kv_len, sm_scale))

    def sparse_fwd(q, k, v, idx, num, vbs, sm_scale):
        return cross_fwd(q, k, v, None, sm_scale)

    def sparse_bwd(do, q, k, v, o, lse, idx, num, vbs, sm_scale):
        return cross_bwd(do, q, k, v, o, lse, None, sm_scale)

    for module, name, f in ((layer, "vsa_norm_rope", norm_rope), (layer, "vsa_norm_rope_bwd", norm_rope_bwd),
                            (layer, "vsa_cross_fwd", cross_fwd), (layer, "vsa_cross_bwd", cross_bwd),
                            (vsa, "vsa_fwd", sparse_fwd), (vsa, "vsa_bwd", sparse_bwd),
                            (vsa, "vsa_invert_indices", lambda idx, num, nb: (idx, num))):
        monkeypatch.setattr(module, name, torch.no_grad()(f))


def randn(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed + sum(shape)), dtype=F64)


def operators():
    """name: (function of the leaves, leaves)."""
    cos, sin = layer.rotation_table(torch.arange(6)[:, None], 8, device="cpu")
    one = torch.zeros(1, dtype=torch.int32)
    heads = [randn(1, 2, 5, 128, seed=i) for i in range(3)]
    return {
        "norm_rope": (lambda q, k, v, wq, wk: autograd.norm_rope(q, k, v, wq, wk, cos, sin),
                      [randn(1, 6, h, 8, seed=h) for h in (2, 1, 1)] + [1 + randn(8, seed=i) / 4 for i in (4, 5)]),
        "norm_rope_alone": (lambda q: autograd.norm_rope(q)[:1], [randn(1, 6, 2, 8)]),
        "cross_attention": (lambda q, k, v: (autograd.cross_attention(q, k, v),), heads),
        "block_sparse_attention": (lambda q, k, v: (autograd.block_sparse_attention(q, k, v, one, one, one),), heads),
    }


@pytest.mark.parametrize("name", list(operators()))
def test_a_second_derivative_is_refused(plain, name):
    """Gradients taken with create_graph have the values of those taken without, and differentiating
    them raises: they would count as constants, and a loss of them and of other terms would lose their
    part.  (x^2 and x^3 as in a gradient penalty next to another term.)"""
    f, leaves = operators()[name]
    leaves = [x.requires_grad_(True) for x in leaves]
    want = torch.autograd.grad(sum((y * y).sum() for y in f(*leaves)), leaves)
    assert not any(g.requires_grad for g in want)
    got = torch.autograd.grad(sum((y * y).sum() for y in f(*leaves)), leaves, create_graph=True)
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    for total in (lambda y: (y * y).sum(), lambda y: y.sum()):    # the latter's own gradient needs none
        got = torch.autograd.grad(sum(total(y) for y in f(*leaves)), leaves, create_graph=True)
        with pytest.raises(RuntimeError, match="once"):
            (sum((g * g).sum() for g in got) + sum((x ** 3).sum() for x in leaves)).backward()
