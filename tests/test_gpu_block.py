"""GPU: the operators that make a whole block (block.py) against plain 64-bit forms, with the bounds
that block_ref derives."""
import pytest
import torch

from tests import block_ref as ref

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def block():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    from block_sparse_video_tok_gb300 import build
    build.build()
    from block_sparse_video_tok_gb300 import block as binding
    return binding


@pytest.fixture(autouse=True)
def no_device_error(block):
    from block_sparse_video_tok_gb300 import layer
    layer.vsa_layer_device_error()
    yield
    assert layer.vsa_layer_device_error() == 0


def randn(*shape, dtype=BF16, seed=0, scale=1.0, offset=0.0):
    g = torch.Generator("cuda").manual_seed(seed + 17 * len(shape) + sum(shape))
    return (torch.randn(shape, generator=g, device="cuda") * scale + offset).to(dtype)


def same_bits(a, b):
    return all(x is y is None or torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
               for x, y in zip(a, b))


# ------------------------------------------------------------------------------- gate_norm

PARAMS = ("y", "gate", "post_weight", "weight", "bias", "scale", "shift")


def norm_case(B, S, C, kind="layer", have="y gate scale shift", G=None, dtype=BF16, branch=None, mod=None,
              wdtype=None, seed=0):
    """Inputs; G None: modulations [B, C], chunks of one [B, 6, C] projection; else [B, G, C]."""
    branch = branch or dtype
    mod, wdtype, have = mod or branch, wdtype or branch, have.split()
    c = dict.fromkeys(PARAMS)
    c["x"] = (randn(B, S, C, seed=seed, dtype=FP32) * torch.exp(randn(B, S, 1, seed=seed + 1, dtype=FP32)) +
              randn(B, S, 1, seed=seed + 2, dtype=FP32)).to(dtype)
    six = randn(*((B, 6, C) if G is None else (B, G, 6, C)), dtype=mod, seed=seed + 3, scale=0.4)
    for i, n in enumerate(("gate", "scale", "shift")):
        if n in have:
            c[n] = six[..., i + 1, :]
    if "y" in have:
        c["y"] = randn(B, S, C, dtype=branch, seed=seed + 4)
    for i, n in enumerate(("post_weight", "weight", "bias")):
        if n in have:
            c[n] = randn(C, dtype=wdtype, seed=seed + 5 + i, scale=0.2, offset=float(n != "bias"))
    return c, kind


NORM_CASES = {
    "block": dict(B=2, S=130, C=1536),
    "one_token": dict(B=1, S=1, C=1536),
    "tokens": dict(B=8, S=1, C=1536, G=1, mod=FP32),
    "plain": dict(B=1, S=77, C=1024, have=""),
    "affine": dict(B=3, S=33, C=264, have="weight bias", wdtype=FP32),
    "rms": dict(B=2, S=65, C=1000, kind="rms", have="y weight", dtype=FP16),
    "add": dict(B=1, S=200, C=512, have="y weight bias", dtype=FP32),
    "fp32_stream": dict(B=2, S=50, C=1024, have="y gate weight bias scale shift", dtype=FP32, branch=BF16, wdtype=FP32),
    "fp32_stream_fp16": dict(B=2, S=21, C=72, have="y gate post_weight scale", dtype=FP32, branch=FP16, mod=FP32),
    "post": dict(B=2, S=90, C=768, kind="rms", have="y gate post_weight weight scale shift", wdtype=FP32, mod=FP32),
    "post_layer": dict(B=1, S=41, C=2048, have="y post_weight weight bias", dtype=FP16),
    "post_add": dict(B=1, S=64, C=1536, kind="rms", have="y post_weight"),
    "frames": dict(B=2, S=7 * 13, C=640, G=13),
    "frames_all": dict(B=3, S=5 * 6, C=320, G=5, have="y gate post_weight weight bias scale shift", mod=FP32, wdtype=FP32),
    "per_token": dict(B=2, S=19, C=264, G=19, kind="rms", have="y gate weight scale shift"),
    "gate_alone": dict(B=2, S=37, C=128, have="y gate"),
    "scale_alone": dict(B=2, S=37, C=128, have="scale bias"),
    "shift_alone": dict(B=2, S=37, C=128, have="shift weight", dtype=FP16, mod=FP32),
    "c8": dict(B=3, S=50, C=8, have="y gate weight bias scale shift"),
    "c64": dict(B=1, S=1021, C=64),
    "c2056": dict(B=1, S=17, C=2056, have="y gate weight bias scale shift"),
    "c4096": dict(B=1, S=40, C=4096, mod=FP32),
    "c4104": dict(B=1, S=9, C=4104, have="y gate post_weight weight bias scale shift", dtype=FP16),
    "c8192": dict(B=2, S=5, C=8192, dtype=FP32, have="y gate post_weight weight bias scale shift"),
    "many_tokens": dict(B=1, S=20011, C=256, have="y gate weight bias scale shift", mod=FP32, wdtype=FP32),
    "many_groups": dict(B=2, S=3000, C=64, G=1500, have="y gate weight scale shift", wdtype=FP32),
}


def forward(block, c, kind, **kw):
    return block.vsa_gate_norm(c["x"], *(c[n] for n in PARAMS), kind=kind, **kw)


@pytest.mark.parametrize("name", list(NORM_CASES))
def test_gate_norm(block, name):
    c, kind = norm_case(**NORM_CASES[name])
    x, h = forward(block, c, kind)
    hdtype = c["x"].dtype if c["y"] is None else c["y"].dtype
    want_x, want_h = ref.gate_norm(c["x"], *(c[n] for n in PARAMS), kind, 1e-6, 1e-6, hdtype)
    if c["y"] is None:
        assert x is c["x"]
    else:
        assert x.dtype == c["x"].dtype
        ref.check("x", x, *want_x)
    assert h.dtype == hdtype
    ref.check("h", h, *want_h)
    assert same_bits(forward(block, c, kind), (x, h))


GRADS = ("dx", "dy", "dgate", "dpost_weight", "dweight", "dbias", "dscale", "dshift")


@pytest.mark.parametrize("name", list(NORM_CASES))
def test_gate_norm_bwd(block, name):
    c, kind = norm_case(**NORM_CASES[name], seed=11)
    hdtype = c["x"].dtype if c["y"] is None else c["y"].dtype
    dh, dx_out = randn(*c["x"].shape, dtype=hdtype, seed=21), randn(*c["x"].shape, dtype=c["x"].dtype, seed=22)
    for o in (dx_out, None):
        got = block.vsa_gate_norm_bwd(dh, o, c["x"], *(c[n] for n in PARAMS), kind=kind)
        want = ref.gate_norm_bwd(dh, o, c["x"], *(c[n] for n in PARAMS), kind, 1e-6, 1e-6)
        for n, g, w in zip(GRADS, got, want):
            assert (g is None) == (w is None), n
            if g is not None:
                assert n in ("dx", "dy") or g.dtype == c[n[1:]].dtype
                ref.check(n, g, *w)
        assert same_bits(block.vsa_gate_norm_bwd(dh, o, c["x"], *(c[n] for n in PARAMS), kind=kind), got)
    alone = block.vsa_gate_norm_bwd(dh, None, c["x"], *(c[n] for n in PARAMS), kind=kind, need_dparams=False)
    assert same_bits(alone[:2], got[:2]) and alone[2:] == (None,) * 6


def test_gate_norm_h_dtype(block):
    x = randn(2, 9, 264, dtype=FP32)
    for t in (BF16, FP16):
        _, h = block.vsa_gate_norm(x, h_dtype=t)
        ref.check("h", h, *ref.gate_norm(x, *[None] * 7, "layer", 1e-6, 1e-6, t)[1])


def test_gate_norm_in_place(block):
    c, kind = norm_case(2, 301, 1536)
    want = forward(block, c, kind)
    x = c["x"].clone()
    got = block.vsa_gate_norm(x, *(c[n] for n in PARAMS), kind=kind, x_out=x)
    assert got[0] is x and same_bits(got, want)
    dh, g = randn(2, 301, 1536, seed=1), randn(2, 301, 1536, seed=2)
    want = block.vsa_gate_norm_bwd(dh, g, x, *(c[n] for n in PARAMS))
    got = block.vsa_gate_norm_bwd(dh, g, x, *(c[n] for n in PARAMS), dx=g)
    assert got[0] is g and same_bits(got, want)


def test_gate_norm_strides(block):
    """Slices of wider tensors, tokens before batch, modulations that all entries share; what lies
    between the outputs' rows stays as it was."""
    B, S, C = 3, 37, 264
    wide = randn(S, B, 2 * C + 8, seed=1)
    x, y = wide[:, :, :C].transpose(0, 1), wide[:, :, C + 8:].transpose(0, 1)
    gate = randn(1, C, seed=2).expand(B, C)
    scale, shift = randn(B, C, seed=3), randn(1, 1, C, seed=4).expand(B, 1, C)
    want = block.vsa_gate_norm(x.contiguous(), y.contiguous(), gate.contiguous(), scale=scale, shift=shift.contiguous())
    room = torch.full((S, B, 2 * C + 16), 7.0, dtype=BF16, device="cuda")
    got = block.vsa_gate_norm(x, y, gate, scale=scale, shift=shift, x_out=room[:, :, :C].transpose(0, 1),
                              h=room[:, :, C + 8:2 * C + 8].transpose(0, 1))
    assert same_bits(got, want)
    assert bool((room[:, :, C:C + 8] == 7).all()) and bool((room[:, :, 2 * C + 8:] == 7).all())


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_gate_norm_far_from_zero(block, kind):
    """Tokens a thousand deviations from zero, in fp32: the variance is taken around the mean."""
    x = randn(1, 50, 1536, dtype=FP32) + 1000 * randn(1, 50, 1, dtype=FP32, seed=1)
    _, h = block.vsa_gate_norm(x, kind=kind)
    ref.check("h", h, *ref.gate_norm(x, *[None] * 7, kind, 1e-6, 1e-6, FP32)[1])


def test_gate_norm_gradient_against_differences(block):
    """fp32 gradients against central differences of the 64-bit forward along random directions:
    with step h the difference is off by O(h^2) ~ 1e-8 of the third derivative."""
    c, kind = norm_case(2, 12, 64, have="y gate post_weight weight bias scale shift", G=3, dtype=FP32)
    dh, dxo = randn(2, 12, 64, dtype=FP32, seed=31), randn(2, 12, 64, dtype=FP32, seed=32)

    def value(inputs):
        (x, _), (h, _) = ref.gate_norm(inputs["x"], *(inputs[n] for n in PARAMS), kind, 1e-6, 1e-6, FP32)
        return float((x * dxo.double()).sum() + (h * dh.double()).sum())

    x_out, _ = forward(block, c, kind)
    grads = dict(zip(GRADS, block.vsa_gate_norm_bwd(dh, dxo, x_out, *(c[n] for n in PARAMS))))
    for i, n in enumerate(("x", *PARAMS)):
        d = randn(*c[n].shape, dtype=torch.float64, seed=40 + i)
        step = 1e-4
        wide = {k: v.double() for k, v in c.items()}
        up, down = value({**wide, n: wide[n] + step * d}), value({**wide, n: wide[n] - step * d})
        got, want = float((grads["d" + n].double() * d).sum()), (up - down) / (2 * step)
        scale = float((grads["d" + n].double() * d).abs().sum())
        assert abs(got - want) <= 2e-5 * scale, (n, got, want, scale)


# ------------------------------------------------------------------------------- linear

LINEAR_SIZES = [
    # rows, in, out
    (1, 8, 8), (1, 1536, 264), (2, 64, 64), (3, 4096, 1000), (5, 24, 136), (8, 1536, 2048), (9, 520, 72), (16, 256, 256),
    (17, 72, 8), (33, 1000, 40), (64, 128, 512), (127, 64, 264), (128, 64, 256), (129, 136, 128), (255, 320, 256),
    (256, 256, 256), (257, 264, 520), (500, 8, 1000), (1021, 1000, 264), (2048, 512, 8), (3000, 2048, 1536),
]


def linear_case(M, K, N, dtype=BF16, bdtype=None, bias=True, residual=False, seed=0):
    return dict(x=randn(M, K, dtype=dtype, seed=seed), weight=randn(N, K, dtype=dtype, seed=seed + 1, scale=K ** -0.5),
                bias=randn(N, dtype=bdtype or dtype, seed=seed + 2) if bias else None,
                residual=randn(M, N, dtype=dtype, seed=seed + 3) if residual else None)


@pytest.mark.parametrize("size", LINEAR_SIZES, ids=str)
def test_linear(block, size):
    for i, (act, dtype, bdtype, bias, residual) in enumerate((
            (None, BF16, None, False, False), ("gelu_tanh", BF16, FP32, True, True), ("gelu", FP16, None, True, False),
            ("silu", FP16, FP32, True, True))):
        c = linear_case(*size, dtype, bdtype, bias, residual, seed=i)
        args = (c["x"], c["weight"], c["bias"], act, c["residual"])
        out, pre = block.vsa_linear(*args, need_pre=True)
        want, want_pre = ref.linear(c["x"], c["weight"], c["bias"], act, c["residual"])
        ref.check("out", out, *want)
        ref.check("pre", pre, *want_pre)
        again, none = block.vsa_linear(*args)
        assert none is None and same_bits((again,), (out,))


@pytest.mark.parametrize("size", LINEAR_SIZES, ids=str)
def test_linear_bwd(block, size):
    M, K, N = size
    for i, (act, x_act, dtype, bdtype, bias) in enumerate((
            (None, None, BF16, None, False), ("gelu_tanh", "silu", BF16, FP32, True), ("gelu", None, FP16, None, True),
            ("silu", "gelu", FP16, FP32, True), (None, "gelu_tanh", BF16, None, True))):
        c = linear_case(*size, dtype, bdtype, bias, seed=i)
        dout = randn(M, N, dtype=dtype, seed=50 + i)
        x_pre = c["x"] if x_act else None
        x = ref.act(c["x"].double(), x_act).to(dtype)
        pre = ref.linear(x, c["weight"], c["bias"], None, None)[0][0].to(dtype) if act else None
        args = (dout, x, c["weight"], c["bias"], act, pre, x_act, x_pre)
        got = block.vsa_linear_bwd(*args)
        want = ref.linear_bwd(*args)
        for n, g, w in zip(("dx", "dweight", "dbias"), got, want):
            assert (g is None) == (w is None), n
            if g is not None:
                ref.check(n, g, *w)
        assert same_bits(block.vsa_linear_bwd(*args), got)
        # Each gradient by itself is the same.
        one = block.vsa_linear_bwd(*args, need_dweight=False)
        assert one[1] is None and same_bits((one[0], one[2]), (got[0], got[2]))
        one = block.vsa_linear_bwd(*args, need_dx=False)
        assert one[0] is None and same_bits(one[1:], got[1:])


def test_linear_strides(block):
    """Rows of wider tensors, a weight that is a slice, leading dimensions; what lies between the
    outputs' rows stays as it was."""
    B, S, K, N = 2, 75, 136, 264
    wide = randn(B, S, K + 24, seed=1)
    x = wide[..., 16:16 + K]
    w = randn(N + 8, K + 8, seed=2)[8:, 8:]
    r = randn(B, S, 2 * N, seed=3)[..., N:]
    want = block.vsa_linear(x.contiguous(), w.contiguous(), None, "silu", r.contiguous(), need_pre=True)
    room = torch.full((2, B, S, N + 16), 7.0, dtype=BF16, device="cuda")
    got = block.vsa_linear(x, w, None, "silu", r, out=room[0, ..., 8:8 + N], pre=room[1, ..., 8:8 + N])
    assert got[0].shape == (B, S, N) and same_bits(got, want)
    assert bool((room[..., :8] == 7).all()) and bool((room[..., 8 + N:] == 7).all())
    dout = randn(B, S, 2 * N, seed=4)[..., N:]
    want = block.vsa_linear_bwd(dout.contiguous(), x.contiguous(), w.contiguous(), None, "silu", want[1])
    room_x = torch.full((B, S, K + 16), 7.0, dtype=BF16, device="cuda")
    room_w = torch.full((N, K + 8), 7.0, dtype=BF16, device="cuda")
    got = block.vsa_linear_bwd(dout, x, w, None, "silu", got[1], dx=room_x[..., 8:8 + K], dweight=room_w[:, :K])
    assert same_bits(got, want)
    assert bool((room_x[..., :8] == 7).all()) and bool((room_x[..., 8 + K:] == 7).all()) and bool((room_w[:, K:] == 7).all())


def test_linear_values_that_are_not_finite(block):
    """An infinite or undefined element reaches its row (or column) alone, also where a tile's rows,
    columns or sum end inside it."""
    M, K, N = 130, 72, 136
    c = linear_case(M, K, N, bias=False)
    base, _ = block.vsa_linear(c["x"], c["weight"])
    x = c["x"].clone()
    x[3, 5], x[129, 71] = float("inf"), float("nan")
    out, _ = block.vsa_linear(x, c["weight"])
    rows = torch.ones(M, dtype=torch.bool, device="cuda")
    rows[[3, 129]] = False
    assert not torch.isfinite(out[~rows].float()).any() and same_bits((out[rows],), (base[rows],))
    dout = randn(M, N, seed=9)
    dx, dw, _ = block.vsa_linear_bwd(dout, c["x"], c["weight"])
    d2 = dout.clone()
    d2[129, 135] = float("nan")
    dx2, dw2, _ = block.vsa_linear_bwd(d2, c["x"], c["weight"])
    assert torch.isnan(dx2[129].float()).all() and same_bits((dx2[:129],), (dx[:129],))
    assert torch.isnan(dw2[135].float()).all() and same_bits((dw2[:135],), (dw[:135],))


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_linear_activations_over_their_range(block, act, dtype):
    """Every size of z, through a weight of ones on the diagonal: the tails keep the result's
    precision."""
    z = torch.cat([torch.linspace(-12, 12, 4001), torch.logspace(-6, 4, 500), -torch.logspace(-6, 4, 500)])
    z = torch.cat([z, z.new_zeros(-z.numel() % 8)]).view(-1, 8).to("cuda", dtype)
    eye = torch.eye(8, device="cuda", dtype=dtype)
    out, pre = block.vsa_linear(z, eye, None, act, need_pre=True)
    assert torch.equal(pre, z)
    want = ref.act(z.double(), act)
    # The quotient and exponential are relative; the exponent itself is off by 2^-22 of its size, up to 60
    # before the result is below fp16's and 88 before it is below bf16's smallest value.
    bound = (ref.half_step(dtype) + 2.0 ** -14) * want.abs() + ref.tiny(dtype) + 1e-37
    ref.check(act, out, want, bound)
    dout = torch.ones_like(z)
    dz, _, _ = block.vsa_linear_bwd(dout, dout, eye, None, None, None, act, z, need_dweight=False)
    want = ref.slope(z.double(), act)
    ref.check(act + "'", dz, want, ref.half_step(dtype) * want.abs() + 2.0 ** -14 * (want.abs() + 2.0 ** -6) + ref.tiny(dtype))


def test_graph_replays(block):
    """Both operators, forward and backward, captured in one graph and replayed on other inputs."""
    c, kind = norm_case(2, 130, 512)
    w = randn(1024, 512, seed=5, scale=512 ** -0.5)
    b = randn(1024, seed=6)
    dh, dxo = randn(2, 130, 512, seed=7), randn(2, 130, 512, seed=8)
    dout = randn(2, 130, 1024, seed=9)

    def step():
        x, h = forward(block, c, kind)
        out, pre = block.vsa_linear(h, w, b, "gelu_tanh", need_pre=True)
        dx, dw, db = block.vsa_linear_bwd(dout, h, w, b, "gelu_tanh", pre)
        return [x, h, out, pre, dx, dw, db, *block.vsa_gate_norm_bwd(dx, dxo, x, *(c[n] for n in PARAMS))[:3]]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (60, 61):
        for t in (c["x"], c["y"], dout):
            t.copy_(randn(*t.shape, seed=seed))
        graph.replay()
        torch.cuda.synchronize()
        assert same_bits(outs, step())


def test_other_stream(block):
    """A call on a stream of its own sees what that stream did before it."""
    c = linear_case(300, 512, 264)
    want = block.vsa_linear(c["x"], c["weight"], c["bias"], "silu", need_pre=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    x = torch.zeros_like(c["x"])
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(2000000)
        x.copy_(c["x"])
    got = block.vsa_linear(x, c["weight"], c["bias"], "silu", need_pre=True, stream=s)
    s.synchronize()
    assert same_bits(got, want)


def every_value(dtype):
    """All values of a 16-bit type but NaNs, [.., 8]."""
    z = torch.arange(1 << 16, device="cuda").to(torch.int16).view(dtype)
    z = z[~z.isnan()]
    return torch.cat([z, z.new_zeros(-z.numel() % 8)]).view(-1, 8)


def wanted_slope(z, act):
    """The slope in 64 bits, its limits at the infinities, and its bound: as a sum of terms of its own size
    and of 2^-6, each good to 2^-14."""
    want = torch.where(z.isinf(), (z > 0).double(), ref.slope(z.double().nan_to_num(0.0, 0.0, 0.0), act))
    return want, ref.half_step(z.dtype) * want.abs() + 2.0 ** -14 * (want.abs() + 2.0 ** -6) + ref.tiny(z.dtype)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_linear_slopes_of_every_value(block, act, dtype):
    """Also where z^2 leaves the range of fp32, and at the infinities that a pre rounded to 16 bits may be."""
    z = every_value(dtype)
    eye = torch.eye(8, device="cuda", dtype=dtype)
    one = torch.ones_like(z)
    want = wanted_slope(z, act)
    # The slopes' own pass, then those of the products' epilogues: small tiles, and pairs of CTAs.
    dz, _, db = block.vsa_linear_bwd(one, one, eye, torch.zeros(8, device="cuda"), act, z, need_dweight=False)
    ref.check(act + "' before the products", dz, *want)
    assert torch.isfinite(db).all()
    few = z[-2000:]
    dz = block.vsa_linear_bwd(one[:2000], one[:2000], eye, None, None, None, act, few, need_dweight=False)[0]
    ref.check(act + "' in small tiles", dz, *(t[-2000:] for t in want))
    wide = torch.zeros(8 * z.shape[0], 64, device="cuda", dtype=dtype)
    for i in range(8):
        wide.view(8, -1, 64)[i, :, 8 * i:8 * i + 8] = z
    one = torch.ones_like(wide)
    dz = block.vsa_linear_bwd(one, one, torch.eye(64, device="cuda", dtype=dtype), None, None, None, act, wide,
                              need_dweight=False)[0]
    ref.check(act + "' in pairs", dz, *wanted_slope(wide, act))
    # An undefined value stays undefined, in its element.
    few = few.clone()
    few[3, 5] = float("nan")
    got = block.vsa_linear_bwd(one[:2000, :8].contiguous(), few, eye, None, None, None, act, few, need_dweight=False)[0]
    assert got[3, 5].isnan() and int(got.isnan().sum()) == 1


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_linear_activations_of_every_finite_value(block, act, dtype):
    z = every_value(dtype)
    z = torch.where(z.isinf(), 0, z)
    out, pre = block.vsa_linear(z, torch.eye(8, device="cuda", dtype=dtype), None, act, need_pre=True)
    assert torch.equal(pre, z)
    want = ref.act(z.double(), act)
    # Relative as in the test of their range; a logistic function below 2^-126, of a z up to 104, is zero.
    ref.check(act, out, want, (ref.half_step(dtype) + 2.0 ** -14) * want.abs() + ref.tiny(dtype) + 104 * 2.0 ** -126)


def off(got, want):
    """Norm of the difference over the norm."""
    return ((got.double() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("size", [s for s in LINEAR_SIZES if s[0] > 1] + [(9000, 256, 520)], ids=str)
@pytest.mark.parametrize("act,x_act,dtype", [("gelu_tanh", None, BF16), ("silu", "gelu", FP16), (None, "silu", BF16)], ids=str)
def test_linear_in_the_norm(block, size, act, x_act, dtype):
    """Where single elements may be off by all roundings at once, whole results may not: each rounding is off by at
    most half a step relative to its value, so results are by half a step of their norm, and dz's roundings, which
    have no sign of their own, come out of the products as large beside dx and dweight as they were beside dz.
    2^-10 of the norm more covers fp32 sums (2^-15 of magnitudes up to 2^5 times the result's)."""
    M, K, N = size
    step = ref.half_step(dtype)
    c = linear_case(M, K, N, dtype, residual=True, seed=3)
    x = ref.act(c["x"].double(), x_act).to(dtype)
    out, pre = block.vsa_linear(x, c["weight"], c["bias"], act, c["residual"], need_pre=True)
    (want, _), (want_pre, _) = ref.linear(x, c["weight"], c["bias"], act, c["residual"])
    assert off(out, want) <= step + 2.0 ** -10 and off(pre, want_pre) <= step + 2.0 ** -10
    dout = randn(M, N, dtype=dtype, seed=70)
    args = (dout, x, c["weight"], c["bias"], act, pre if act else None, x_act, c["x"] if x_act else None)
    for n, got, (value, _) in zip(("dx", "dweight", "dbias"), block.vsa_linear_bwd(*args), ref.linear_bwd(*args)):
        # (A rounding of dz is at most half a step of its value, 0.6 of one in the root of the mean square; with few
        # terms the sums of signed errors may stand out, twice that covers them.)
        bound = step + (2 * step if act and n != "dbias" else 0.0) + 2.0 ** -10
        assert off(got, value) <= bound, (n, off(got, value), bound)


@pytest.mark.parametrize("dtype,branch", [(FP32, BF16), (BF16, BF16)], ids=str)
def test_gate_norm_long_video_in_the_norm(block, dtype, branch):
    """A stream of thousands of tokens of a whole block's width, fp32 or bf16, forward and backward: each result is
    off by half a step of its type in the norm, 2^-12 more for fp32."""
    c, kind = norm_case(2, 8190, 1536, have="y gate weight bias scale shift", dtype=dtype, branch=branch, mod=FP32, wdtype=FP32)
    x, h = forward(block, c, kind)
    (want_x, _), (want_h, _) = ref.gate_norm(c["x"], *(c[n] for n in PARAMS), kind, 1e-6, 1e-6, branch)
    assert off(x, want_x) <= ref.half_step(dtype) + 2.0 ** -12 and off(h, want_h) <= ref.half_step(branch) + 2.0 ** -12
    dh, dx_out = randn(2, 8190, 1536, dtype=branch, seed=21), randn(2, 8190, 1536, dtype=dtype, seed=22)
    args = (dh, dx_out, x, *(c[n] for n in PARAMS))
    for n, got, want in zip(GRADS, block.vsa_gate_norm_bwd(*args), ref.gate_norm_bwd(*args, kind, 1e-6, 1e-6)):
        if got is not None:
            assert off(got, want[0]) <= ref.half_step(got.dtype) + 2.0 ** -12, n


def test_gate_norm_inputs_that_are_broadcast(block):
    """Tokens, entries and gradients of stride 0, and one tensor in several places."""
    B, S, C = 3, 41, 264
    one, row = randn(1, S, C, seed=1), randn(1, 1, C, seed=2)
    gate, scale = randn(B, C, seed=3), randn(1, C, seed=4).expand(B, C)
    w = randn(C, seed=5)
    for x, y in ((one.expand(B, S, C), row.expand(B, S, C)), (row.expand(B, S, C), one.expand(B, S, C))):
        args = (y, gate, None, w, w, scale, scale)
        got = block.vsa_gate_norm(x, *args)
        assert same_bits(got, block.vsa_gate_norm(x.contiguous(), y.contiguous(), *args[1:]))
        bwd = block.vsa_gate_norm_bwd(y, x, x, *args)
        assert same_bits(bwd, block.vsa_gate_norm_bwd(*(t.contiguous() for t in (y, x, x, y)), *args[1:]))
    x = one.expand(B, S, C).contiguous()
    assert same_bits(block.vsa_gate_norm(x, x, gate, scale=gate, shift=gate),
                     block.vsa_gate_norm(x, x.clone(), gate, scale=gate.clone(), shift=gate.clone()))
