"""GPU: the operators around the block-sparse attention (layer.py) against plain 64-bit forms.

The bounds are layer_ref's, derived there from the rounding of the outputs, of the 16-bit operands
and of fp32 sums."""
import math

import pytest
import torch

from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


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


def randn(*shape, dtype=BF16, seed=0, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed + 17 * len(shape) + sum(shape))
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


# ------------------------------------------------------------------------------- norm_rope

def norm_case(layer, B, S, H, Hk, D, rot, halves, dtype, wdtype, order=None, per_batch=False,
              weights=True, seed=0):
    qkv = randn(B, S, (H + 2 * Hk) * D, dtype=dtype, seed=seed) * 2
    x = qkv.view(B, S, H + 2 * Hk, D)
    c = dict(q=x[:, :, :H], k=x[:, :, H:H + Hk], v=x[:, :, H + Hk:], halves=halves, src=None,
             dst=None, cos=None, sin=None, wq=None, wk=None, rows=S)
    if weights:
        c["wq"], c["wk"] = (1 + randn(D, dtype=wdtype, seed=seed + i, scale=0.2) for i in (1, 2))
    if rot:
        pos = torch.arange(B * S).reshape(B, S, 1) * 37 if per_batch else torch.arange(S)[:, None]
        c["cos"], c["sin"] = layer.rotation_table(pos, rot)
    if order is not None:
        c["src"], c["dst"], vbs = layer.video_token_order(order)
        assert c["dst"].numel() == S
        c["rows"] = c["src"].numel()
    return c


NORM_CASES = {
    # B, S, H, Hk, D, rot, halves, dtype, weight dtype
    "video": dict(B=2, S=5 * 6 * 7, H=3, Hk=3, D=128, rot=128, halves=False, dtype=BF16, wdtype=BF16, order=(5, 6, 7)),
    "video_fp32_weights": dict(B=1, S=9 * 4 * 13, H=4, Hk=2, D=128, rot=128, halves=True, dtype=BF16, wdtype=FP32, order=(9, 4, 13)),
    "one_token": dict(B=1, S=1, H=12, Hk=12, D=128, rot=128, halves=False, dtype=BF16, wdtype=BF16),
    "token_per_batch": dict(B=8, S=1, H=8, Hk=2, D=128, rot=128, halves=True, dtype=BF16, wdtype=BF16, per_batch=True),
    "table_per_batch": dict(B=3, S=33, H=2, Hk=1, D=64, rot=32, halves=False, dtype=FP16, wdtype=FP16, per_batch=True),
    "d8": dict(B=2, S=19, H=5, Hk=1, D=8, rot=8, halves=False, dtype=BF16, wdtype=BF16),
    "d16_halves": dict(B=1, S=50, H=3, Hk=3, D=16, rot=16, halves=True, dtype=FP32, wdtype=FP32),
    "d72_part": dict(B=1, S=77, H=7, Hk=7, D=72, rot=48, halves=True, dtype=FP16, wdtype=FP32),
    "d80": dict(B=2, S=31, H=6, Hk=3, D=80, rot=80, halves=True, dtype=BF16, wdtype=BF16),
    "d96_part": dict(B=1, S=1021, H=10, Hk=5, D=96, rot=64, halves=True, dtype=FP16, wdtype=FP16),
    "d256": dict(B=1, S=65, H=4, Hk=1, D=256, rot=256, halves=True, dtype=BF16, wdtype=FP32),
    "d200_fp32": dict(B=1, S=40, H=3, Hk=2, D=200, rot=104, halves=False, dtype=FP32, wdtype=FP32),
    "no_rotation": dict(B=1, S=17, H=2, Hk=2, D=128, rot=0, halves=False, dtype=BF16, wdtype=BF16),
    "no_weights": dict(B=1, S=17, H=9, Hk=2, D=128, rot=128, halves=False, dtype=BF16, wdtype=BF16, weights=False),
    "long_sum": dict(B=1, S=20000, H=6, Hk=6, D=64, rot=64, halves=False, dtype=FP32, wdtype=FP32),
}


@pytest.mark.parametrize("name", list(NORM_CASES))
def test_norm_rope(layer, name):
    spec = NORM_CASES[name]
    c = norm_case(layer, **spec)
    got = layer.vsa_norm_rope(c["q"], c["k"], c["v"], c["wq"], c["wk"], c["cos"], c["sin"], src=c["src"],
                              halves=c["halves"])
    for n, g, x, w in (("q", got[0], c["q"], c["wq"]), ("k", got[1], c["k"], c["wk"])):
        ref.check(n, g, *ref.norm_rope_one(x, w, c["cos"], c["sin"], c["src"], c["halves"], 1e-6, spec["dtype"]))
    assert torch.equal(got[2].double(), ref.move(c["v"], c["src"]))
    again = layer.vsa_norm_rope(c["q"], c["k"], c["v"], c["wq"], c["wk"], c["cos"], c["sin"], src=c["src"],
                                halves=c["halves"])
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("name", list(NORM_CASES))
def test_norm_rope_bwd(layer, name):
    spec = NORM_CASES[name]
    c = norm_case(layer, **spec, seed=5)
    B, D, dt = spec["B"], spec["D"], spec["dtype"]
    dq, dk, dv = (randn(B, h, c["rows"], D, dtype=dt, seed=9 + i)
                  for i, h in enumerate((spec["H"], spec["Hk"], spec["Hk"])))
    args = (dq, dk, dv, c["q"], c["k"], c["wq"], c["wk"], c["cos"], c["sin"])
    got = layer.vsa_norm_rope_bwd(*args, dst=c["dst"], halves=c["halves"])
    for n, g, gw, dy, x, w in (("q", got[0], got[3], dq, c["q"], c["wq"]), ("k", got[1], got[4], dk, c["k"], c["wk"])):
        dx, dw = ref.norm_rope_one_bwd(dy, x, w, c["cos"], c["sin"], c["dst"], c["halves"], 1e-6, dt, spec["wdtype"])
        ref.check("d" + n, g, *dx)
        if w is None:
            assert gw is None
        else:
            assert gw.dtype == spec["wdtype"]
            ref.check("dw" + n, gw, *dw)
    assert torch.equal(got[2].transpose(1, 2).double(), ref.move(dv.transpose(1, 2), c["dst"]))
    again = layer.vsa_norm_rope_bwd(*args, dst=c["dst"], halves=c["halves"])
    assert all(torch.equal(a, b) for a, b in zip(got, again) if a is not None)


def test_norm_rope_gradient_against_differences(layer):
    """The fp32 gradients against central differences of the 64-bit forward along random
    directions: with step h the difference is off by O(h^2) ~ 1e-8 of the third derivative."""
    c = norm_case(layer, 1, 2 * 3 * 5, 2, 1, 64, 48, True, FP32, FP32, order=(2, 3, 5), seed=3)
    dq = randn(1, 2, c["rows"], 64, dtype=FP32, seed=4)
    dk = randn(1, 1, c["rows"], 64, dtype=FP32, seed=5)
    gq, gk, _, gwq, gwk = layer.vsa_norm_rope_bwd(dq, dk, None, c["q"], c["k"], c["wq"], c["wk"], c["cos"], c["sin"],
                                                  dst=c["dst"], halves=True)
    for dy, x, w, gx, gw in ((dq, c["q"], c["wq"], gq, gwq), (dk, c["k"], c["wk"], gk, gwk)):
        f = lambda x, w: (ref.norm_rope_one(x, w, c["cos"], c["sin"], c["src"], True, 1e-6, FP32)[0]  # noqa: E731
                          * dy.double()).sum()
        ex, ew = randn(*x.shape, dtype=torch.float64, seed=6), randn(*w.shape, dtype=torch.float64, seed=7)
        h = 1e-4
        want = (f(x.double() + h * ex, w.double() + h * ew) - f(x.double() - h * ex, w.double() - h * ew)) / (2 * h)
        have = (gx.double() * ex).sum() + (gw.double() * ew).sum()
        size = (gx.double() * ex).abs().sum() + (gw.double() * ew).abs().sum()
        assert abs(float(want - have)) <= 1e-5 * float(size)


def test_norm_rope_parts_and_strides(layer):
    """q alone, q and k alone, q and v alone; outputs in token order; a broadcast batch."""
    c = norm_case(layer, 2, 30, 4, 2, 128, 128, False, BF16, BF16, seed=11)
    args = (c["wq"], c["wk"], c["cos"], c["sin"])
    full = layer.vsa_norm_rope(c["q"], c["k"], c["v"], *args)
    q, k, v = layer.vsa_norm_rope(c["q"], None, None, *args)
    assert k is None and v is None and torch.equal(q, full[0])
    q, k, v = layer.vsa_norm_rope(c["q"], c["k"], None, *args)
    assert v is None and torch.equal(k, full[1])
    out = torch.full((2, 30, 4, 128), math.nan, dtype=BF16, device="cuda").transpose(1, 2)
    q, k, v = layer.vsa_norm_rope(c["q"], None, c["v"], *args, q_out=out)
    assert k is None and torch.equal(out, full[0]) and torch.equal(v, full[2])
    wide = c["q"][:1].expand(2, -1, -1, -1)
    q, _, _ = layer.vsa_norm_rope(wide, None, None, *args)
    assert torch.equal(q[0], full[0][0]) and torch.equal(q[1], full[0][0])
    # Gradients of q alone, without the weights', from a strided gradient.
    dy = randn(2, 30, 4, 128, seed=12).transpose(1, 2)
    one = layer.vsa_norm_rope_bwd(dy, None, None, c["q"], None, *args, need_dweight=False)
    assert one[1:] == (None,) * 4
    both = layer.vsa_norm_rope_bwd(dy.contiguous(), randn(2, 2, 30, 128), None, c["q"], c["k"], *args)
    assert torch.equal(one[0], both[0])


def test_norm_rope_orders(layer):
    """Tokens that no row takes, rows without a token, a token taken twice, entries out of range."""
    c = norm_case(layer, 1, 8, 2, 1, 128, 128, True, BF16, BF16, seed=13)
    src = torch.tensor([3, -1, 0, 3, 7, -1], dtype=torch.int32, device="cuda")
    q, k, v = layer.vsa_norm_rope(c["q"], c["k"], c["v"], c["wq"], c["wk"], c["cos"], c["sin"], src=src, halves=True)
    ref.check("q", q, *ref.norm_rope_one(c["q"], c["wq"], c["cos"], c["sin"], src, True, 1e-6, BF16))
    assert torch.equal(v.double(), ref.move(c["v"], src))
    assert torch.equal(q[:, :, 0], q[:, :, 3]) and not q[:, :, 1].any()
    dst = torch.tensor([2, -1, -1, 0, -1, -1, -1, 4], dtype=torch.int32, device="cuda")
    dy = randn(1, 2, 6, 128, seed=14)
    dq, _, _, dw, _ = layer.vsa_norm_rope_bwd(dy, None, None, c["q"], None, c["wq"], None, c["cos"], c["sin"],
                                              dst=dst, halves=True)
    want, wantw = ref.norm_rope_one_bwd(dy, c["q"], c["wq"], c["cos"], c["sin"], dst, True, 1e-6, BF16, BF16)
    ref.check("dq", dq, *want)
    ref.check("dw", dw, *wantw)
    assert not dq[:, 1].any()
    assert layer.vsa_layer_device_error() == 0
    bad = torch.tensor([3, -2, 8, 1 << 30, -(1 << 31), 7], dtype=torch.int32, device="cuda")
    q, _, _ = layer.vsa_norm_rope(c["q"], None, None, c["wq"], None, c["cos"], c["sin"], src=bad, halves=True)
    assert layer.vsa_layer_device_error() == layer.DEVERR_ORDER
    assert not q[:, :, 1:5].any() and q[:, :, 0].any() and q[:, :, 5].any()


def test_norm_rope_special_values(layer):
    """A row of zeros stays zero (eps > 0), one NaN stays in its head, tiny and huge rows."""
    q = randn(1, 6, 2, 128, dtype=FP32, seed=15)
    q[0, 0] = 0
    q[0, 1, 0, 5] = math.nan
    q[0, 2] *= 1e-15
    q[0, 3] *= 1e15
    y, _, _ = layer.vsa_norm_rope(q)
    want, bound = ref.norm_rope_one(q, None, None, None, None, False, 1e-6, FP32)
    keep = torch.ones_like(want, dtype=torch.bool)
    keep[0, 0, 1] = False
    ref.check("y", y[keep], want[keep], bound[keep])
    assert y[0, 0, 1].isnan().all() and not y[0, :, 0].any()


# ------------------------------------------------------------------------- cross attention

def cross_case(B, Sq, Sk, H, Hk, lens=None, seed=0, scale=128 ** -0.5, qscale=1.0):
    c = dict(q=randn(B, Sq, H, 128, seed=seed, scale=qscale).transpose(1, 2), scale=scale, lens=None)
    kv = randn(B, Sk, 2, Hk, 128, seed=seed + 1)
    c["k"], c["v"] = kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
    c["do"] = randn(B, Sq, H, 128, seed=seed + 2).transpose(1, 2)
    if lens is not None:
        c["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for b, n in enumerate(lens):                      # what is past the length must not matter
            c["k"][b, :, n:] = math.nan
            c["v"][b, :, n:] = -math.inf if b % 2 else math.nan
    return c


CROSS_CASES = {
    # B, Sq, Sk, H, Hk, lens
    "one_one": dict(B=1, Sq=1, Sk=1, H=1, Hk=1),
    "token": dict(B=8, Sq=1, Sk=512, H=12, Hk=12, lens=[512, 77, 301, 1, 0, 256, 33, 129]),
    "token_shared": dict(B=3, Sq=1, Sk=300, H=8, Hk=2, lens=[300, 0, 7]),
    "token_shared_16": dict(B=1, Sq=1, Sk=1000, H=16, Hk=1),
    "two_tokens_shared": dict(B=2, Sq=2, Sk=131, H=6, Hk=2),
    "token_long": dict(B=1, Sq=1, Sk=20011, H=8, Hk=2),
    "few_long": dict(B=1, Sq=5, Sk=9000, H=4, Hk=4, lens=[8191]),
    "two_rows": dict(B=3, Sq=2, Sk=700, H=2, Hk=2, lens=[700, 0, 9]),
    "two_rows_long": dict(B=1, Sq=1, Sk=5000, H=4, Hk=2),
    "many_parts_64": dict(B=1, Sq=64, Sk=7000, H=2, Hk=2, lens=[6500]),
    "many_parts_100": dict(B=1, Sq=100, Sk=7000, H=1, Hk=1),
    "few_64": dict(B=2, Sq=64, Sk=1500, H=3, Hk=3, lens=[1500, 1409]),
    "tile": dict(B=1, Sq=128, Sk=128, H=2, Hk=2),
    "tile_plus": dict(B=1, Sq=129, Sk=129, H=2, Hk=2),
    "two_tiles": dict(B=1, Sq=256, Sk=256, H=2, Hk=1),
    "tiles_minus": dict(B=2, Sq=255, Sk=383, H=2, Hk=2, lens=[127, 382]),
    "lens": dict(B=6, Sq=200, Sk=257, H=2, Hk=2, lens=[0, 1, 64, 128, 129, 257]),
    "empty": dict(B=2, Sq=70, Sk=40, H=2, Hk=1, lens=[0, 0]),
    "long_queries": dict(B=1, Sq=5000, Sk=77, H=4, Hk=2, lens=[70]),
    "text": dict(B=2, Sq=2100, Sk=512, H=3, Hk=3, lens=[512, 333]),
    "square": dict(B=1, Sq=1300, Sk=1300, H=4, Hk=4),
    "one_key": dict(B=2, Sq=300, Sk=1, H=3, Hk=1),
    "shared_4": dict(B=2, Sq=333, Sk=200, H=8, Hk=2, lens=[200, 150]),
    "many_heads": dict(B=5, Sq=3, Sk=20, H=40, Hk=20),
    "steep": dict(B=1, Sq=300, Sk=700, H=2, Hk=2, qscale=30.0),
    "negative_scale": dict(B=1, Sq=140, Sk=300, H=2, Hk=2, scale=-0.3, lens=[290]),
    "zero_scale": dict(B=1, Sq=140, Sk=300, H=2, Hk=2, scale=0.0, lens=[290]),
    "token_steep": dict(B=2, Sq=1, Sk=700, H=4, Hk=2, qscale=30.0, lens=[700, 650]),
    "token_zero_scale": dict(B=1, Sq=1, Sk=300, H=2, Hk=2, scale=0.0, lens=[290]),
}


def both(f):
    """f() twice: the outputs, which have to be the same bits."""
    a, b = f(), f()
    assert all(torch.equal(x.view(torch.int16 if x.element_size() == 2 else torch.int32),
                           y.view(torch.int16 if y.element_size() == 2 else torch.int32)) for x, y in zip(a, b))
    return a


@pytest.mark.parametrize("name", list(CROSS_CASES))
def test_cross_fwd(layer, name):
    c = cross_case(**CROSS_CASES[name])
    o, lse = both(lambda: layer.vsa_cross_fwd(c["q"], c["k"], c["v"], c["lens"], c["scale"]))
    (wo, bo), (wl, bl) = ref.cross_fwd(c["q"], c["k"], c["v"], c["lens"], c["scale"])
    assert o.stride() == c["q"].stride() or 1 in o.shape
    ref.check("lse", lse, wl, bl)
    ref.check("o", o, wo, bo)
    if c["lens"] is not None:
        for b in torch.nonzero(c["lens"] == 0).flatten().tolist():
            assert not o[b].any() and (lse[b] == -math.inf).all()


@pytest.mark.parametrize("name", list(CROSS_CASES))
def test_cross_bwd(layer, name):
    c = cross_case(**CROSS_CASES[name], seed=3)
    o, lse = layer.vsa_cross_fwd(c["q"], c["k"], c["v"], c["lens"], c["scale"])
    args = (c["do"], c["q"], c["k"], c["v"], o, lse, c["lens"], c["scale"])
    got = both(lambda: layer.vsa_cross_bwd(*args))
    for n, g, (w, b) in zip(("dq", "dk", "dv"), got, ref.cross_bwd(*args)):
        ref.check(n, g, w, b)
    if c["lens"] is not None:
        for b, n in enumerate(c["lens"].tolist()):
            for g in got[1:]:
                assert not g[b, :, n:].contiguous().view(torch.int16).any()


def test_cross_gradient_against_differences(layer):
    """Directional derivatives of the 64-bit forward by central differences (h = 1e-4, so off by
    about 1e-8 of the third derivative) against the bf16 gradients, within their bounds."""
    c = cross_case(1, 40, 90, 4, 2, lens=[85], seed=21)
    for x in (c["k"], c["v"]):
        x[:, :, 85:] = 0
    o, lse = layer.vsa_cross_fwd(c["q"], c["k"], c["v"], c["lens"], c["scale"])
    args = (c["do"], c["q"], c["k"], c["v"], o, lse, c["lens"], c["scale"])
    got, want = layer.vsa_cross_bwd(*args), ref.cross_bwd(*args)
    h = 1e-4
    for i, n in enumerate("qkv"):
        e = randn(*c[n].shape, dtype=torch.float64, seed=22 + i)
        f = lambda s: (ref.cross_fwd(*[c[m].double() + s * e if m == n else c[m] for m in "qkv"],  # noqa: E731
                                     c["lens"], c["scale"])[0][0] * c["do"].double()).sum()
        d = float((f(h) - f(-h)) / (2 * h))
        # Delta is taken from the rounded O: it moves dS by up to 2^-8 P |dO| |O|, within the
        # bound's 2^-8 |dS| and half-step terms summed in magnitude, doubled here for it.
        assert abs(float((got[i].double() * e).sum()) - d) <= 2 * float((want[i][1] * e.abs()).sum())


def test_cross_strides(layer):
    """Contiguous heads, a slice of a fused projection, a batch of shared states (stride 0), given
    outputs in another memory order."""
    c = cross_case(2, 150, 140, 4, 2, seed=31)
    base = layer.vsa_cross_fwd(c["q"], c["k"], c["v"], None, c["scale"])
    flat = layer.vsa_cross_fwd(*(c[n].contiguous() for n in "qkv"), None, c["scale"])
    assert torch.equal(base[0], flat[0]) and torch.equal(base[1], flat[1])
    out = torch.full((150, 2, 4, 136), math.nan, dtype=BF16, device="cuda")[..., :128].permute(1, 2, 0, 3)
    layer.vsa_cross_fwd(c["q"], c["k"], c["v"], None, c["scale"], o=out)
    assert torch.equal(out, base[0])
    k, v = (c[n][:1].expand(2, -1, -1, -1) for n in "kv")
    shared = layer.vsa_cross_fwd(c["q"], k, v, None, c["scale"])
    copied = layer.vsa_cross_fwd(c["q"], k.contiguous(), v.contiguous(), None, c["scale"])
    assert torch.equal(shared[0], copied[0])
    do, o, lse = c["do"], *shared
    g = layer.vsa_cross_bwd(do, c["q"], k, v, o, lse, None, c["scale"])
    w = layer.vsa_cross_bwd(do.contiguous(), c["q"].contiguous(), k.contiguous(), v.contiguous(), o.contiguous(), lse,
                            None, c["scale"])
    assert all(torch.equal(a, b) for a, b in zip(g, w))
    dk = torch.full((2, 140, 2, 2, 128), math.nan, dtype=BF16, device="cuda")
    layer.vsa_cross_bwd(do, c["q"], k, v, o, lse, None, c["scale"], dk=dk[:, :, 0].transpose(1, 2),
                        dv=dk[:, :, 1].transpose(1, 2))
    assert torch.equal(dk[:, :, 0].transpose(1, 2), g[1]) and torch.equal(dk[:, :, 1].transpose(1, 2), g[2])
    one = layer.vsa_cross_fwd(c["q"][:, :, :1], k, v, None, c["scale"])     # single tokens, shared states
    ref.check("token", one[0], *ref.cross_fwd(c["q"][:, :, :1], k, v, None, c["scale"])[0])


def test_cross_lengths_out_of_range(layer):
    c = cross_case(3, 20, 50, 2, 2, seed=41)
    bad = torch.tensor([-1, 51, 1 << 30], dtype=torch.int32, device="cuda")
    o, lse = layer.vsa_cross_fwd(c["q"], c["k"], c["v"], bad, c["scale"])
    assert layer.vsa_layer_device_error() == layer.DEVERR_KV_LEN
    want = layer.vsa_cross_fwd(c["q"], c["k"], c["v"], bad.clamp(0, 50), c["scale"])
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    g = layer.vsa_cross_bwd(c["do"], c["q"], c["k"], c["v"], o, lse, bad, c["scale"])
    assert layer.vsa_layer_device_error() == layer.DEVERR_KV_LEN
    w = layer.vsa_cross_bwd(c["do"], c["q"], c["k"], c["v"], o, lse, bad.clamp(0, 50), c["scale"])
    assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_cross_non_finite_inputs(layer):
    """A NaN in one query row stays in that row's O; an infinite visible score gives NaN there as
    the formula does, and nowhere else."""
    c = cross_case(1, 140, 150, 2, 1, seed=43)
    clean = layer.vsa_cross_fwd(c["q"], c["k"], c["v"], None, c["scale"])[0]
    c["q"][0, 0, 3, 7] = math.nan
    c["q"][0, 1, 130] = math.inf
    o, lse = layer.vsa_cross_fwd(c["q"], c["k"], c["v"], None, c["scale"])
    hit = torch.zeros(2, 140, dtype=torch.bool, device="cuda")
    hit[0, 3] = hit[1, 130] = True
    assert torch.equal(o[0][~hit], clean[0][~hit])
    assert o[0][hit].isnan().all()


def test_cross_offsets_past_32_bits(layer):
    """Keys and values of more than 2^32 bytes and 2^31 elements: the last heads and keys."""
    Sk, Hk = 66000, 130
    kv = torch.empty((1, Sk, 2, Hk, 128), dtype=BF16, device="cuda")
    assert kv.numel() > 1 << 31
    for i in range(0, Sk, 6600):
        kv[:, i:i + 6600] = randn(1, 6600, 2, Hk, 128, seed=i)
    k, v = kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
    for Sq in (1, 3):
        q = randn(1, Sq, Hk, 128, seed=51).transpose(1, 2)
        o, lse = layer.vsa_cross_fwd(q, k, v)
        for h in (0, 1, Hk - 1):
            part = [x[:, h:h + 1] for x in (q, k, v)]
            (wo, bo), (wl, bl) = ref.cross_fwd(*part, None, 128 ** -0.5)
            ref.check("o", o[:, h:h + 1], wo, bo)
            ref.check("lse", lse[:, h:h + 1], wl, bl)


# ------------------------------------------------------------------------------- using them

def test_other_stream(layer):
    c = cross_case(1, 300, 200, 2, 2, seed=61)
    n = norm_case(layer, 1, 300, 2, 2, 128, 128, False, BF16, BF16, seed=62)
    want = layer.vsa_cross_fwd(c["q"], c["k"], c["v"])
    wn = layer.vsa_norm_rope(n["q"], n["k"], n["v"], n["wq"], n["wk"], n["cos"], n["sin"])
    wg = layer.vsa_cross_bwd(c["do"], c["q"], c["k"], c["v"], *want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = layer.vsa_cross_fwd(c["q"], c["k"], c["v"], stream=side)
    gg = layer.vsa_cross_bwd(c["do"], c["q"], c["k"], c["v"], *got, stream=side)
    gn = layer.vsa_norm_rope(n["q"], n["k"], n["v"], n["wq"], n["wk"], n["cos"], n["sin"], stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*want, *wn, *wg), (*got, *gn, *gg)))


def test_graph_capture(layer):
    """Forward and backward of both operators in one graph, replayed on new inputs."""
    cs = [cross_case(2, 260, 300, 4, 2, lens=lens, seed=71) for lens in ([300, 0], [17, 299])]
    for c in cs:
        for x in (c["k"], c["v"]):
            x.nan_to_num_(0, 0, 0)
    ns = [norm_case(layer, 1, 60, 3, 3, 128, 128, False, BF16, BF16, order=(3, 4, 5), seed=s) for s in (72, 73)]

    def step(c, n):
        y = layer.vsa_norm_rope(n["q"], n["k"], n["v"], n["wq"], n["wk"], n["cos"], n["sin"], src=n["src"])
        dx = layer.vsa_norm_rope_bwd(*y, n["q"], n["k"], n["wq"], n["wk"], n["cos"], n["sin"], dst=n["dst"])
        o, lse = layer.vsa_cross_fwd(c["q"], c["k"], c["v"], c["lens"], c["scale"])
        return (*y, *dx, o, lse, *layer.vsa_cross_bwd(c["do"], c["q"], c["k"], c["v"], o, lse, c["lens"], c["scale"]))

    want = [[t.clone() for t in step(c, n)] for c, n in zip(cs, ns)]
    c = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in cs[0].items()}
    n = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in ns[0].items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(c, n)
    for i in (0, 1, 0):
        for k, v in c.items():
            if isinstance(v, torch.Tensor):
                v.copy_(cs[i][k])
        for k, v in n.items():
            if isinstance(v, torch.Tensor):
                v.copy_(ns[i][k])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i])), i


def test_autograd(layer):
    """norm_rope into cross_attention: gradients equal the binding's, through an expanded gradient
    of the output and with an output that the loss does not reach."""
    from block_sparse_video_tok_gb300.autograd import cross_attention, norm_rope
    n = norm_case(layer, 2, 60, 4, 2, 128, 128, False, BF16, FP32, order=(3, 4, 5), seed=81)
    kv = cross_case(2, 1, 90, 4, 2, lens=[90, 31], seed=82)
    for x in (kv["k"], kv["v"]):
        x.nan_to_num_(0, 0, 0)
    leaves = [n["q"].contiguous(), n["k"].contiguous(), n["v"].contiguous(), n["wq"].clone(), n["wk"].clone(),
              kv["k"].clone(), kv["v"].clone()]
    for t in leaves:
        t.requires_grad_(True)
    q, k, v, wq, wk, ek, ev = leaves
    y, yk, yv = norm_rope(q, k, v, wq, wk, n["cos"], n["sin"], (n["src"], n["dst"]))
    o = cross_attention(y, ek, ev, kv["lens"])
    (o.sum() + yk.float().square().sum()).backward()                # yv is not reached
    with torch.no_grad():
        y2, yk2, _ = layer.vsa_norm_rope(q, k, v, wq, wk, n["cos"], n["sin"], src=n["src"])
        o2, lse = layer.vsa_cross_fwd(y2, ek, ev, kv["lens"])
        dy, dek, dev = layer.vsa_cross_bwd(torch.ones_like(o2), y2, ek, ev, o2, lse, kv["lens"])
        dx = layer.vsa_norm_rope_bwd(dy, (2 * yk2.float()).to(BF16), torch.zeros_like(yk2), q, k, wq, wk, n["cos"],
                                     n["sin"], dst=n["dst"])
    assert torch.equal(o, o2)
    for g, w in zip((q.grad, k.grad, v.grad, wq.grad, wk.grad, ek.grad, ev.grad), (*dx, dek, dev)):
        assert torch.equal(g, w)
    assert not v.grad.any()


def test_binding_refusals(layer):
    x = randn(1, 20, 4, 128)
    q, k = x.transpose(1, 2), randn(1, 30, 2, 128).transpose(1, 2)
    cos = torch.ones(20, 64, device="cuda")
    with pytest.raises(TypeError):
        layer.vsa_cross_fwd(q.float(), k, k)
    with pytest.raises(TypeError):
        layer.vsa_cross_fwd(q, k, k, kv_len=torch.ones(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        layer.vsa_cross_fwd(q, k, k, kv_len=torch.ones(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        layer.vsa_cross_fwd(q[..., :64], k[..., :64], k[..., :64])
    with pytest.raises(ValueError):
        layer.vsa_cross_fwd(q[:, :3], k, k)
    with pytest.raises(ValueError):
        layer.vsa_cross_fwd(q, k, k[:, :, :29])
    with pytest.raises(ValueError):
        layer.vsa_cross_fwd(q, k, k, sm_scale=math.nan)
    with pytest.raises(ValueError):
        layer.vsa_cross_fwd(q, k[:, :, :0], k[:, :, :0])
    with pytest.raises(ValueError):
        layer.vsa_cross_fwd(randn(1, 4, 20, 129)[..., 1:], k, k)
    with pytest.raises(TypeError):
        layer.vsa_norm_rope(x.double())
    with pytest.raises(TypeError):
        layer.vsa_norm_rope(x, q_weight=torch.ones(128, device="cuda", dtype=FP16))
    with pytest.raises(ValueError):
        layer.vsa_norm_rope(x, q_weight=torch.ones(64, device="cuda"))
    with pytest.raises(ValueError):
        layer.vsa_norm_rope(x, cos=cos)
    with pytest.raises(ValueError):
        layer.vsa_norm_rope(x, cos=cos[:10], sin=cos[:10])
    with pytest.raises(ValueError):
        layer.vsa_norm_rope(x, cos=cos[:, :4].contiguous(), sin=cos[:, :4].contiguous(), halves=True)
    with pytest.raises(TypeError):
        layer.vsa_norm_rope(x, src=torch.zeros(20, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        layer.vsa_norm_rope(x[:, :, :, :100].contiguous())
    with pytest.raises(ValueError):
        layer.vsa_norm_rope_bwd(randn(1, 4, 19, 128), None, None, x)
    with pytest.raises(ValueError):
        layer.vsa_norm_rope_bwd(q, None, None, x, k=x)
