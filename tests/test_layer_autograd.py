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


def sixteen_byte_view(t):
    return t.stride(-1) == 1 and t.data_ptr() % 16 == 0 and \
        all(n == 1 or (s and s * t.element_size() % 16 == 0) for n, s in zip(t.shape[:-1], t.stride()))


def test_gradients_reach_the_kernels_aligned():
    """Whatever the memory of an incoming gradient (a slice that starts off 16 bytes, as behind a
    torch.cat of flattened tensors; broadcast; transposed; odd strides), the kernels get its values with
    16-byte aligned data and strides; one that has them already is not copied."""
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.randn(2, 3, 4, 128).to(dtype)
        flat = torch.zeros(x.numel() + 9, dtype=dtype)
        for offset in (1, 3, 8, 9):
            flat[offset:offset + x.numel()] = x.flatten()
            g = flat[offset:offset + x.numel()].view(x.shape)
            a = autograd._aligned(g)
            assert sixteen_byte_view(a) and torch.equal(a, x)
            assert (a.data_ptr() == g.data_ptr()) == (g.data_ptr() % 16 == 0)
            one = autograd._aligned(g[:1, :1, :1])               # strides of single entries do not count
            assert sixteen_byte_view(one) and torch.equal(one, x[:1, :1, :1])
        for g in (x[:, :1].expand(-1, 3, -1, -1), x.mT.contiguous().mT, torch.cat([x, x[..., :1]], -1)[..., :128],
                  x[:1, :1, :1, :1].expand(2, 3, 4, 128)):
            a = autograd._aligned(g)
            assert sixteen_byte_view(a) and torch.equal(a, g)
        assert autograd._aligned(x.transpose(1, 2)).data_ptr() == x.data_ptr()


def test_block_sparse_gradient_that_starts_anywhere(plain, monkeypatch):
    """block_sparse_attention's backward takes a contiguous gradient at a 16-byte address, wherever and
    however the incoming one lies."""
    seen, bwd = [], vsa.vsa_bwd
    monkeypatch.setattr(vsa, "vsa_bwd", lambda do, *args: seen.append(do) or bwd(do, *args))
    one = torch.zeros(1, dtype=torch.int32)
    leaves = [randn(1, 2, 5, 128, seed=i).requires_grad_(True) for i in range(3)]
    g = randn(1, 2, 5, 128, seed=7)
    want = None
    for before in (2, 1):
        y = autograd.block_sparse_attention(*leaves, one, one, one)
        got = torch.autograd.grad(torch.cat([torch.zeros(before, dtype=F64), y.flatten()]), leaves,
                                  torch.cat([torch.zeros(before, dtype=F64), g.flatten()]))
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    y = autograd.block_sparse_attention(*leaves, one, one, one)
    got = torch.autograd.grad(y.transpose(2, 3), leaves, g.transpose(2, 3).contiguous())
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for do in seen:
        assert do.is_contiguous() and do.data_ptr() % 16 == 0 and torch.equal(do, g)


def test_half_an_order_gives_no_gradient(plain):
    """norm_rope's backward cannot do without the order of the other direction."""
    x, one = randn(1, 4, 2, 8).requires_grad_(True), torch.arange(4, dtype=torch.int32)
    for order in ((one, None), (None, one)):
        with pytest.raises(ValueError, match="order"):
            autograd.norm_rope(x, order=order)
    with torch.no_grad():
        assert autograd.norm_rope(x, order=(one, None))[0].shape == (1, 2, 4, 8)
    assert autograd.norm_rope(x, order=(one, one))[0].requires_grad


def test_an_order_to_check_against_is_refused():
    from block_sparse_video_tok_gb300 import build
    build.build()
    at = 0x100000
    h = layer.VsaHeads(at, 4 * 10 * 128, 10 * 128, 128, 4)
    for order, inverse in ((None, at), (at, at + 2)):               # none to check; misaligned
        op = layer.VsaNormRope(batch=1, tokens=10, rows=10, head_dim=128, eps=1e-6, order=order, inverse=inverse)
        assert layer._lib().vsa_norm_rope_fwd(op, h, None, None, h, None, None, None) == 1
        assert layer._lib().vsa_norm_rope_bwd(op, h, None, None, h, None, h, *[None] * 5, 0, None) == 1
