"""GPU: the layer operators on values that are not finite, on sums of tens of thousands of terms and at
offsets past 2^31 elements, forward and backward.

The bounds are layer_ref's with F32, the rounding of the fp32 sums, set for the sums at hand: a sum of n
terms that are added one after another in fp32 is off by at most n 2^-24 of the sum of its terms'
magnitudes.  (One accumulator in tensor memory takes all keys of a part, for dQ and O, or all query rows of
all heads that share a key head, for dK and dV, so n is their number.)"""
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


@pytest.mark.parametrize("name", ["token", "few_parts", "half_tile", "long"])
def test_scale_zero_on_large_scores(layer, name):
    """With scale 0 every visible key has the same weight, however large the finite scores are."""
    do, q, k, v, _ = inputs(name)
    q = (q.float() * 1e34).to(BF16)
    lens = torch.full((q.shape[0],), k.shape[2] - 7, dtype=torch.int32, device="cuda")
    o, lse = layer.vsa_cross_fwd(q, k, v, lens, 0.0)
    (wo, bo), (wl, bl) = ref.cross_fwd(q, k, v, lens, 0.0)
    ref.check("o", o, wo, bo)
    ref.check("lse", lse, wl, bl)
    got = layer.vsa_cross_bwd(do, q, k, v, o, lse, lens, 0.0)
    for n, g, (w, b) in zip(("dq", "dk", "dv"), got, ref.cross_bwd(do, q, k, v, o, lse, lens, 0.0)):
        ref.check(n, g, w, b)


# ---------------------------------------------------------------------- long sums

@pytest.mark.parametrize("Sq, Sk, H, Hk", [(40000, 130, 2, 2), (11000, 130, 4, 1), (130, 40000, 2, 1), (3, 60000, 1, 1)])
def test_long_sums(layer, monkeypatch, Sq, Sk, H, Hk):
    """Tens of thousands of query rows to a key tile, or keys to a query tile, against 64 bits."""
    do, q = (randn(1, H, Sq, 128, seed=i) for i in (11, 12))
    k, v = (randn(1, Hk, Sk, 128, seed=i) for i in (13, 14))
    o, lse = layer.vsa_cross_fwd(q, k, v)
    got = layer.vsa_cross_bwd(do, q, k, v, o, lse)

    def bounds(terms):
        monkeypatch.setattr(ref, "F32", max(2.0 ** -15, terms * 2.0 ** -24))

    bounds(Sk)
    (wo, bo), (wl, bl) = ref.cross_fwd(q, k, v, None, SCALE)
    ref.check("o", o, wo, bo)
    ref.check("lse", lse, wl, bl)
    ref.check("dq", got[0], *ref.cross_bwd(do, q, k, v, o, lse, None, SCALE)[0])
    bounds(Sq * H // Hk)
    _, dk, dv = ref.cross_bwd(do, q, k, v, o, lse, None, SCALE)
    ref.check("dk", got[1], *dk)
    ref.check("dv", got[2], *dv)


@pytest.mark.parametrize("Sq, H, Hk", [(50000, 1, 1), (12500, 4, 1)])
def test_long_sum_of_equal_weights(layer, Sq, H, Hk):
    """q = 0 and 2^n keys: every P is exactly 2^-n, and dV is the sum of dO's rows, head after head, times
    it.  An addition in fp32 is off by at most 2^-24 of what the sum has reached, so all of them by n 2^-24
    of the largest it reaches (the order of the rows within a tile does not matter for a bound that takes
    the largest over every tile's start and adds the tile's magnitudes); dQ and dK are zeros but for
    what is left of dP - Delta, which is taken away here by equal values."""
    Sk = 128
    do = randn(1, H, Sq, 128, seed=21)
    k, v = randn(1, Hk, Sk, 128, seed=22), randn(1, Hk, 1, 128, seed=23).expand(-1, -1, Sk, -1).contiguous()
    q = torch.zeros_like(do)
    o, lse = layer.vsa_cross_fwd(q, k, v)
    assert same(o, v[:, :, :1].repeat_interleave(H // Hk, 1).expand_as(o)) and (lse == 7).all()
    dv = layer.vsa_cross_bwd(do, q, k, v, o, lse)[2]
    rows = do.double().flatten(1, 2) / Sk                            # [1, H Sq, 128]
    want = rows.sum(1)[:, None, None]
    tiles = torch.nn.functional.pad(rows, (0, 0, 0, -rows.shape[1] % 128)).unflatten(1, (-1, 128))
    # (Heads of a number of rows that is no multiple of 128 end within these tiles: one more tile's
    # magnitudes cover that.)
    reached = tiles.sum(2).cumsum(1).abs().amax(1) + 2 * tiles.abs().sum(2).amax(1)
    bound = 2.0 ** -8 * want.abs() + rows.shape[1] * 2.0 ** -24 * reached[:, None, None]
    assert bool(((dv.double() - want).abs() <= bound).all())


# ---------------------------------------------------------------------- offsets past 2^31 elements

def fused(n, heads, seed):
    """Two [1, heads, n, 128] views of one [1, n, 2, heads, 128] buffer of more than 2^31 elements."""
    x = torch.empty((1, n, 2, heads, 128), dtype=BF16, device="cuda")
    assert x.numel() > 1 << 31
    for i in range(0, n, n // 10):
        if seed is None:
            x[:, i:i + n // 10] = math.nan
        else:
            x[:, i:i + n // 10] = randn(1, min(n // 10, n - i), 2, heads, 128, seed=seed + i)
    return x[:, :, 0].transpose(1, 2), x[:, :, 1].transpose(1, 2)


@pytest.mark.parametrize("Sq, Sk", [(3, 66000), (66000, 90)])
def test_cross_backward_past_32_bits(layer, monkeypatch, Sq, Sk):
    """Keys and values, then queries and their gradients, in and out, whose last heads and rows lie past
    2^31 elements and 2^32 bytes."""
    monkeypatch.setattr(ref, "F32", max(Sq, Sk) * 2.0 ** -24)
    H = 130
    if Sq < Sk:
        (k, v), (dk, dv) = fused(Sk, H, 31), fused(Sk, H, None)
        q, do = randn(1, H, Sq, 128, seed=32), randn(1, H, Sq, 128, seed=33)
        o, lse = layer.vsa_cross_fwd(q, k, v)
        dq, _, _ = layer.vsa_cross_bwd(do, q, k, v, o, lse, dk=dk, dv=dv)
    else:
        (q, do), (dq, o) = fused(Sq, H, 31), fused(Sq, H, None)
        k, v = randn(1, H, Sk, 128, seed=32), randn(1, H, Sk, 128, seed=33)
        _, lse = layer.vsa_cross_fwd(q, k, v, o=o)
        _, dk, dv = layer.vsa_cross_bwd(do, q, k, v, o, lse, dq=dq)
    for h in (0, H - 1):
        part = [x[:, h:h + 1] for x in (do, q, k, v, o, lse)]
        whole = [x[:, h:h + 1] for x in (dq, dk, dv)]
        alone = layer.vsa_cross_bwd(*part)
        (wo, bo), _ = ref.cross_fwd(*part[1:4], None, SCALE)
        ref.check("o", part[4], wo, bo)
        for n, g, a, (w, b) in zip(("dq", "dk", "dv"), whole, alone, ref.cross_bwd(*part, None, SCALE)):
            ref.check(n, g, w, b)
            ref.check(n, a, w, b)                   # (other parts than in the whole, so other bits)


def test_norm_rope_past_32_bits(layer):
    """Rows in reverse order in buffers of more than 2^31 elements: the first and last tokens, forward and
    backward, have the bits of a short call on them."""
    S, H, D = 470000, 36, 128
    x = torch.empty((1, S, H, D), dtype=BF16, device="cuda")
    assert x.numel() > 1 << 31
    for i in range(0, S, 47000):
        x[:, i:i + 47000] = randn(1, 47000, H, D, seed=i)
    w = 1 + randn(D) / 4
    cos, sin = layer.rotation_table(torch.arange(S)[:, None], D)
    back = torch.arange(S - 1, -1, -1, dtype=torch.int32, device="cuda")
    y = torch.full((1, S, H, D), math.nan, dtype=BF16, device="cuda").transpose(1, 2)     # rows in token order
    layer.vsa_norm_rope(x[:, :, :20], x[:, :, 20:], None, w, w, cos, sin, src=back, q_out=y[:, :20], k_out=y[:, 20:],
                        dst=back)
    n = 300
    near = torch.arange(n - 1, -1, -1, dtype=torch.int32, device="cuda")
    ends = [(slice(0, n), slice(S - n, S)), (slice(S - n, S), slice(0, n))]               # tokens, rows
    for t, r in ends:
        short = layer.vsa_norm_rope(x[:, t], None, None, w, None, cos[t], sin[t], src=near)[0]
        assert same(y[:, :, r], short)
    del short
    dx = torch.full((1, S, H, D), math.nan, dtype=BF16, device="cuda")
    layer.vsa_norm_rope_bwd(y[:, :20], y[:, 20:], None, x[:, :, :20], x[:, :, 20:], w, w, cos, sin, dst=back,
                            dq=dx[:, :, :20], dk=dx[:, :, 20:], src=back)
    for t, r in ends:
        short = layer.vsa_norm_rope_bwd(y[:, :, r], None, None, x[:, t], None, w, None, cos[t], sin[t], dst=near)[0]
        assert same(dx[:, t], short)
