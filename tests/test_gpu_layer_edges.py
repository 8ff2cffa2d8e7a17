"""GPU: the layer operators on values that are not finite, forward and backward, with layer_ref's bounds."""
import math

import pytest
import torch

from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
SCALE = 128 ** -0.5


@pytest.fixture(scope="module")
def layer():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    from block_sparse_video_tok_gb300 import build
    build.build()
    from block_sparse_video_tok_gb300 import layer as binding
    return binding


@pytest.fixture(autouse=True)
def no_device_error(layer):
    layer.vsa_layer_device_error()
    yield
    assert layer.vsa_layer_device_error() == 0


def randn(*shape, seed=0):
    g = torch.Generator("cuda").manual_seed(seed + 17 * len(shape) + sum(shape))
    return torch.randn(shape, generator=g, device="cuda").to(BF16)


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ---------------------------------------------------------------------- values that are not finite

SHAPES = {
    # B, Sq, Sk, H, Hk
    "token": (2, 1, 300, 4, 4),
    "token_parts": (1, 1, 5000, 2, 2),
    "token_two_rows": (2, 1, 300, 4, 2),
    "token_two_rows_parts": (1, 1, 5000, 4, 2),
    "few": (2, 5, 300, 4, 4),
    "few_parts": (1, 5, 3000, 2, 2),
    "few_shared": (2, 3, 300, 8, 2),
    "half_tile": (1, 64, 300, 2, 2),
    "tile": (1, 128, 256, 4, 2),
    "tile_and_a_row": (2, 129, 300, 2, 2),
    "long": (1, 2500, 300, 4, 2),
}


def inputs(name):
    B, Sq, Sk, H, Hk = SHAPES[name]
    q, do = (randn(B, Sq, H, 128, seed=i).transpose(1, 2) for i in (1, 2))
    k, v = (randn(B, Sk, Hk, 128, seed=i).transpose(1, 2) for i in (3, 4))
    return do, q, k, v, H // Hk


def with_value(x, at, value):
    y = x.clone()
    y[at] = value
    return y


@pytest.mark.parametrize("name", list(SHAPES))
def test_forward_keeps_what_is_not_finite_apart(layer, name):
    """A NaN or an infinity in a query row makes that row NaN, one in a key the rows that read its key head,
    one in a value their column; nothing else changes by a bit."""
    _, q, k, v, share = inputs(name)
    o, lse = layer.vsa_cross_fwd(q, k, v)
    h = q.shape[1] - 1
    kh = h // share
    heads = slice(kh * share, (kh + 1) * share)
    for value in (math.nan, math.inf):
        for x, at in ((q, (0, h, -1)), (k, (0, kh, 5))):
            args = [with_value(y, at, value) if y is x else y for y in (q, k, v)]
            o2, lse2 = layer.vsa_cross_fwd(*args)
            hit = torch.zeros_like(lse, dtype=torch.bool)
            hit[(0, h, -1) if x is q else (0, heads)] = True
            assert o2[hit].isnan().all() and lse2[hit].isnan().all()
            assert same(o2[~hit], o[~hit]) and same(lse2[~hit], lse[~hit])
        o2, lse2 = layer.vsa_cross_fwd(q, k, with_value(v, (0, kh, 5, 9), value))
        hit = torch.zeros_like(o, dtype=torch.bool)
        hit[0, heads, :, 9] = True
        assert not o2[hit].isfinite().any()
        assert same(o2[~hit], o[~hit]) and same(lse2, lse)


@pytest.mark.parametrize("name", list(SHAPES))
def test_backward_keeps_what_is_not_finite_apart(layer, name):
    """A NaN in a row of q, dout or o reaches that row of dQ and, over the rows' sums, the keys' gradients
    of its key head as the formulas have it; nothing else changes by a bit."""
    do, q, k, v, share = inputs(name)
    o, lse = layer.vsa_cross_fwd(q, k, v)
    dq, dk, dv = layer.vsa_cross_bwd(do, q, k, v, o, lse)
    h = q.shape[1] - 1
    kh = h // share
    for i, x in enumerate((do, q, o)):
        do2, q2, o2 = (with_value(y, (0, h, -1), math.nan) if y is x else y for y in (do, q, o))
        dq2, dk2, dv2 = layer.vsa_cross_bwd(do2, q2, k, v, o2, lse)
        hit = torch.zeros_like(lse, dtype=torch.bool)
        hit[0, h, -1] = True
        assert dq2[hit].isnan().all() and same(dq2[~hit], dq[~hit])
        hit = torch.zeros(dk.shape[:3], dtype=torch.bool, device="cuda")
        hit[0, kh] = True
        assert dk2[hit].isnan().all() and same(dk2[~hit], dk[~hit])
        if x is o:                                                   # dV = P^T dO has no O
            assert same(dv2, dv)
        else:
            assert dv2[hit].isnan().all() and same(dv2[~hit], dv[~hit])


@pytest.mark.parametrize("name", list(SHAPES))
def test_a_key_that_every_score_hides(layer, name):
    """A key whose scores are all -inf takes no part: O, lse and the other keys' gradients are those
    without it, its own gradients are zeros, whatever the number of query rows beside a full tile.  (dQ
    has 0 x inf in the column where the key is infinite.)"""
    do, q, k, v, _ = inputs(name)
    q, k = q.clone(), k.clone()
    q[..., 0] = q[..., 0].abs() + 0.5
    k[:, :, 5] = 0
    k[:, :, 5, 0] = -math.inf
    o, lse = layer.vsa_cross_fwd(q, k, v)
    rest = torch.arange(k.shape[2], device="cuda") != 5
    less = k[:, :, rest], v[:, :, rest]
    (wo, bo), (wl, bl) = ref.cross_fwd(q, *less, None, SCALE)
    ref.check("o", o, wo, bo)
    ref.check("lse", lse, wl, bl)
    dq, dk, dv = layer.vsa_cross_bwd(do, q, k, v, o, lse)
    (wq, bq), (wk, bk), (wv, bv) = ref.cross_bwd(do, q, *less, o, lse, None, SCALE)
    ref.check("dk", dk[:, :, rest], wk, bk)
    ref.check("dv", dv[:, :, rest], wv, bv)
    ref.check("dq", dq[..., 1:], wq[..., 1:], bq[..., 1:])
    assert not dv[:, :, 5].any() and not dk[:, :, 5].any()
