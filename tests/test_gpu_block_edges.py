"""GPU: the block operators where sizes, values and surroundings are unusual: sums of tens of thousands
of terms, offsets past 2^31 elements, norms of nothing but zeros, values that are not finite, two
streams at once."""
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
    torch.cuda.empty_cache()


def randn(*shape, dtype=BF16, seed=0, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed + sum(shape))
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def same_bits(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))


def test_long_sums_of_parameters(block):
    """A token gradient of one sign, 70000 tokens: the sums keep fp32's precision.  A unit adds at most 512
    terms in a row (2^-15 of their magnitudes), the parts as many again."""
    B, S, C = 2, 35000, 64
    x, y = randn(B, S, C), randn(B, S, C, seed=1)
    dh = randn(B, S, C, seed=2).abs() + 1
    mods = [randn(B, C, dtype=FP32, seed=3 + i) for i in range(3)]
    w, b = randn(C, dtype=FP32, seed=6), randn(C, dtype=FP32, seed=7)
    args = (dh, None, x, y, mods[0], None, w, b, mods[1], mods[2])
    for g, r in zip(block.vsa_gate_norm_bwd(*args), ref.gate_norm_bwd(*args, "layer", 1e-6, 1e-6)):
        if g is not None:
            ref.check("grad", g, r[0], 2 * r[1])


def test_long_sums_of_products(block):
    """Products of one sign over 70000 rows (dweight, dbias) and over 65536 features (out): all operands 1,
    so that every partial sum is whole and results are exact up to their rounding."""
    M, K, N = 70000, 64, 72
    x, w = torch.ones(M, K, dtype=BF16, device="cuda"), torch.ones(N, K, dtype=BF16, device="cuda")
    dout = torch.ones(M, N, dtype=BF16, device="cuda")
    _, dw, db = block.vsa_linear_bwd(dout, x, w, torch.zeros(N, device="cuda"), need_dx=False)
    assert bool((db == 70000).all()) and bool((dw == torch.tensor(70000.0).to(BF16)).all())
    for M in (1, 16, 100, 300):
        x, w = (torch.ones(n, 1 << 16, dtype=FP16, device="cuda") * 0.5 for n in (M, 264))
        out, _ = block.vsa_linear(x, w)
        assert bool((out == 16384).all()), M


def test_gate_norm_past_2_31_elements(block):
    """The last tokens of tensors of more than 2^31 elements are those of the same tokens by themselves."""
    S, C = (1 << 31) // 2048 + 40, 2048
    x = torch.zeros(1, S, C, dtype=BF16, device="cuda")
    y = torch.zeros(1, S, C, dtype=BF16, device="cuda")
    tail = slice(S - 64, S)
    x[:, tail], y[:, tail] = randn(1, 64, C), randn(1, 64, C, seed=1)
    gate, scale, shift = (randn(1, C, seed=2 + i) for i in range(3))
    xo, h = block.vsa_gate_norm(x, y, gate, scale=scale, shift=shift, x_out=x)
    got = xo[:, tail].clone(), h[:, tail].clone()
    torch.cuda.synchronize()
    small = [randn(1, 64, C), randn(1, 64, C, seed=1)]
    assert same_bits(block.vsa_gate_norm(*small, gate, scale=scale, shift=shift), got)
    h.zero_()
    h[:, tail] = randn(1, 64, C, seed=7)
    out = block.vsa_gate_norm_bwd(h, None, xo, y, gate, scale=scale, shift=shift, need_dparams=False, dx=xo)
    want = block.vsa_gate_norm_bwd(randn(1, 64, C, seed=7), None, got[0], small[1], gate, scale=scale, shift=shift,
                                   need_dparams=False)
    assert same_bits((out[0][:, tail], out[1][:, tail]), want[:2])


def test_linear_past_2_31_elements(block):
    M, K, N = (1 << 31) // 512 + 300, 64, 512
    x = torch.zeros(M, K, dtype=BF16, device="cuda")
    x[-600:] = randn(600, K)
    w, b = randn(N, K, seed=1), randn(N, seed=2)
    out, _ = block.vsa_linear(x, w, b, "silu")
    want, _ = block.vsa_linear(x[-600:], w, b, "silu")
    bound = ref.linear(x[-600:], w, b, "silu", None)[0]
    ref.check("out", out[-600:], *bound)
    ref.check("want", want, *bound)
    assert bool((out[:8] == block.vsa_linear(x[:8], w, b, "silu")[0]).all())
    out.zero_()
    out[-600:] = randn(600, N, seed=3)
    dx, dw, db = block.vsa_linear_bwd(out, x, w, b)
    (rx, bx), (rw, bw), (rb, bb) = ref.linear_bwd(out[-600:], x[-600:], w, b, None, None, None, None)
    ref.check("dx", dx[-600:], rx, bx)
    ref.check("dw", dw, rw, bw)
    ref.check("db", db, rb, bb)
    assert not dx[:-600].any()


def test_tokens_of_zeros(block):
    """Zeros with an eps are zeros, without one undefined in their token alone; a constant token is a zero
    of the layer norm."""
    x, dh = randn(1, 6, 264), randn(1, 6, 264, seed=1)
    x[0, 2] = 0
    for kind in ("layer", "rms"):
        _, h = block.vsa_gate_norm(x, kind=kind)
        assert not h[0, 2].any() and torch.isfinite(h.float()).all()
        dx = block.vsa_gate_norm_bwd(dh, None, x, kind=kind)[0]
        assert torch.isfinite(dx.float()).all()
        _, h0 = block.vsa_gate_norm(x, kind=kind, eps=0.0)
        rest = [0, 1, 3, 4, 5]
        assert torch.isfinite(h0[0, rest].float()).all()
    x[0, 3] = 5
    assert not block.vsa_gate_norm(x)[1][0, 3].any()


def test_values_that_are_not_finite_stay_in_their_token(block):
    B, S, C = 2, 40, 520
    x, y, dh, g = (randn(B, S, C, seed=i) for i in range(4))
    gate = randn(B, C, seed=5)
    base = block.vsa_gate_norm(x, y, gate)
    base_b = block.vsa_gate_norm_bwd(dh, g, x, y, gate, need_dparams=False)
    bad = x.clone()
    bad[0, 7, 3], bad[1, 39, 519], bad[1, 0, 0] = float("inf"), float("nan"), -float("inf")
    keep = torch.ones(B, S, dtype=torch.bool, device="cuda")
    keep[0, 7] = keep[1, 39] = keep[1, 0] = False
    for got, want in ((block.vsa_gate_norm(bad, y, gate), base),
                      (block.vsa_gate_norm_bwd(dh, g, bad, y, gate, need_dparams=False)[:2], base_b[:2])):
        assert same_bits([t[keep] for t in got], [t[keep] for t in want])
        assert torch.isnan(got[1][~keep].float()).any(-1).all()


def test_two_streams_at_once(block):
    """Calls on two streams, each with its own workspaces, do not meet."""
    cases = []
    for i in range(2):
        x, w = randn(300, 4096, seed=i), randn(1536, 4096, seed=2 + i, scale=1 / 64)
        cases.append((x, w, randn(300, 1536, seed=4 + i), randn(1, 300, 1536, seed=6 + i)))

    def all_of(x, w, dout, t):
        out, _ = block.vsa_linear(x, w)
        return [out, *block.vsa_linear_bwd(dout, x, w)[:2], *block.vsa_gate_norm_bwd(t, None, t, weight=t[0, 0])[::4]]

    want = [all_of(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = all_of(*cases[i])
        torch.cuda.synchronize()
        assert all(same_bits(g, w) for g, w in zip(got, want))


def test_the_current_device_is_the_tensors(block):
    """A tensor of a device that is not the current one is refused (with one GPU: nothing to refuse)."""
    if torch.cuda.device_count() < 2:
        pytest.skip("one GPU")
    x = torch.zeros(1, 4, 64, dtype=BF16, device="cuda:1")
    with pytest.raises(ValueError):
        block.vsa_gate_norm(x)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("size", [(1, 8, 8), (64, 64, 64), (40, 256, 256), (17, 1000, 264), (300, 1000, 264),
                                  (1021, 1000, 264), (2000, 64, 136), (20, 64, 2048), (20, 2048, 64), (512, 1024, 512),
                                  (4096, 64, 64), (256, 1536, 1536)], ids=str)
def test_linear_bwd_alone_and_together(block, size, dtype):
    # Both gradients may come from one launch whose tiles are shared by different numbers of CTAs: the bits
    # are those of each gradient asked for alone.
    M, K, N = size
    dout, x, w = randn(M, N, dtype=dtype, seed=1), randn(M, K, dtype=dtype, seed=2), randn(N, K, dtype=dtype, seed=3, scale=K ** -0.5)
    x_pre = randn(M, K, dtype=dtype, seed=4)
    for more in ({}, {"x_act": "silu", "x_pre": x_pre}):
        dx, dw, _ = block.vsa_linear_bwd(dout, x, w, **more)
        alone_x = block.vsa_linear_bwd(dout, x, w, need_dweight=False, **more)[0]
        alone_w = block.vsa_linear_bwd(dout, x, w, need_dx=False)[1]
        assert same_bits((dx, dw), (alone_x, alone_w))
        want = dout.double().t() @ x.double()
        err = (dw.double() - want).abs().max() / want.abs().max().clamp(min=1e-6)
        # One rounding, and M sums in fp32 of products that are exact there, relative to the largest of them all.
        big = (dout.double().abs().t() @ x.double().abs()).max() / want.abs().max().clamp(min=1e-6)
        assert err <= torch.finfo(dtype).eps / 2 + big * M * 2.0 ** -24


@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("case", [(2, 1, 1000, 400), (1, 2, 8, 64), (32, 1, 4104, 9), (33, 1, 4104, 9), (8, 8, 2056, 32),
                                  (65, 1, 2056, 5), (64, 2, 264, 34), (3, 43, 264, 86), (43, 1, 64, 3000), (7, 23, 1536, 69),
                                  (300, 1, 1536, 20), (1100, 1, 128, 3), (129, 1, 256, 130)], ids=str)
def test_gate_norm_bwd_rows(block, case, weights):
    # The joins of the units' sums are chosen by the number of modulation rows, of channels and of units.
    B, G, C, S = case
    x, y, dh = (randn(B, S, C, seed=i) for i in range(3))
    mods = [randn(*((B, C) if G == 1 else (B, G, C)), seed=10 + i, scale=0.4) for i in range(3)]
    w, b = (randn(C, dtype=FP32, seed=20), randn(C, dtype=FP32, seed=21)) if weights else (None, None)
    args = (y, mods[0], None, w, b, mods[1], mods[2])
    got = block.vsa_gate_norm_bwd(dh, None, x, *args)
    want = ref.gate_norm_bwd(dh, None, x, *args, "layer", 1e-6, 1e-6)
    for n, g, v in zip(("dx", "dy", "dgate", "dpost_weight", "dweight", "dbias", "dscale", "dshift"), got, want):
        assert (g is None) == (v is None), n
        if g is not None:
            ref.check(n, g, *v)
    again = block.vsa_gate_norm_bwd(dh, None, x, *args)
    assert same_bits([g for g in got if g is not None], [g for g in again if g is not None])


@pytest.mark.parametrize("mod", [BF16, FP32])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("case", [(1, 500, 1536, 500), (2, 700, 4104, 700), (1, 1300, 1024, 2600), (1, 3000, 64, 3000),
                                  (2, 900, 128, 6300), (1, 600, 128, 4800), (3, 1, 8, 1), (1, 1001, 6152, 1001),
                                  (1, 400, 2056, 800)], ids=str)
def test_gate_norm_modulations_of_few_tokens(block, case, kind, mod):
    # A modulation row that one unit covers: its sums become its gradients without the workspace.
    B, G, C, S = case
    x, y, dh = (randn(B, S, C, seed=i) for i in range(3))
    mods = [randn(B, G, C, dtype=mod, seed=10 + i, scale=0.4) for i in range(3)]
    args = (y, mods[0], None, None, None, mods[1], mods[2])
    x2, h = block.vsa_gate_norm(x, *args, kind=kind)
    want_x, want_h = ref.gate_norm(x, *args, kind, 1e-6, 1e-6, BF16)
    ref.check("x", x2, *want_x)
    ref.check("h", h, *want_h)
    got = block.vsa_gate_norm_bwd(dh, None, x, *args, kind=kind)
    want = ref.gate_norm_bwd(dh, None, x, *args, kind, 1e-6, 1e-6)
    for n, g, v in zip(("dx", "dy", "dgate", "dpost_weight", "dweight", "dbias", "dscale", "dshift"), got, want):
        assert (g is None) == (v is None), n
        if g is not None:
            ref.check(n, g, *v)
    again = block.vsa_gate_norm_bwd(dh, None, x, *args, kind=kind)
    assert same_bits([g for g in got if g is not None], [g for g in again if g is not None])


@pytest.mark.parametrize("size", [(20000, 8, 264), (9001, 64, 1528), (5003, 520, 2056), (6000, 768, 1536), (6000, 776, 1032),
                                  (5000, 1024, 2000), (5000, 1032, 2000), (40000, 64, 40), (30000, 40, 72)], ids=str)
def test_linear_epilogues(block, size):
    # Many rows of few features: the epilogue's warps and what it leaves out are chosen by the features.
    M, K, N = size
    x, w, r = randn(M, K, seed=1), randn(N, K, seed=2, scale=K ** -0.5), randn(M, N, seed=3)
    b = randn(N, dtype=FP32, seed=4)
    for act, residual, bias in ((None, None, None), (None, None, b), (None, r, b), ("gelu_tanh", None, b), ("silu", r, None),
                                ("gelu", None, None)):
        out, pre = block.vsa_linear(x, w, bias, act, residual, need_pre=True)
        want, want_pre = ref.linear(x, w, bias, act, residual)
        ref.check("out", out, *want)
        ref.check("pre", pre, *want_pre)
        assert same_bits((block.vsa_linear(x, w, bias, act, residual)[0],), (out,))
    # dx of K features from N, with and without a slope; dweight over the many rows.
    dout, x_pre = randn(M, K, seed=5), r
    for act in (None, "gelu_tanh"):
        args = (dout, r if act is None else ref.act(r.double(), act).to(BF16), randn(K, N, seed=6, scale=K ** -0.5), None,
                None, None, act, None if act is None else x_pre)
        got, want = block.vsa_linear_bwd(*args), ref.linear_bwd(*args)
        ref.check("dx", got[0], *want[0])
        ref.check("dweight", got[1], *want[1])
        assert same_bits(block.vsa_linear_bwd(*args)[:2], got[:2])


@pytest.mark.parametrize("size", [(8, 8192, 5000), (9, 8192, 3040), (16, 8192, 3048), (16, 8192, 3056), (17, 1000, 1000), (17, 8192, 1224),
                                  (23, 5000, 2000), (24, 24, 16), (24, 5000, 2008), (25, 1536, 1536)], ids=str)
def test_linear_few_rows(block, size):
    # On both sides of where a few rows stop having a kernel of their own.
    M, K, N = size
    x, w, r = randn(M, K, seed=1), randn(N, K, seed=2, scale=K ** -0.5), randn(M, N, seed=3)
    b = randn(N, dtype=FP32, seed=4)
    for act, residual, bias in ((None, None, None), ("gelu_tanh", r, b), ("silu", None, b)):
        out, pre = block.vsa_linear(x, w, bias, act, residual, need_pre=True)
        want, want_pre = ref.linear(x, w, bias, act, residual)
        ref.check("out", out, *want)
        ref.check("pre", pre, *want_pre)
        assert same_bits((block.vsa_linear(x, w, bias, act, residual)[0],), (out,))


@pytest.mark.parametrize("C", [8, 56, 120, 224, 488, 656, 1000, 1272, 1536, 2024, 4080, 6080, 8160])
@pytest.mark.parametrize("dtype,branch", [(FP32, FP32), (FP32, BF16), (FP16, FP16), (BF16, BF16)], ids=str)
def test_constant_tokens_are_zeros_of_the_layer_norm(block, C, dtype, branch):
    """Tokens of one whole number, whose sums are exact in fp32: n is zero in the backward as it is in the
    forward, so nothing of it reaches dscale or dweight, and dx = (g - mean(g)) / sqrt(eps)."""
    top = (1 << 24) // C
    values = [v for v in (5, 120, 1000, 15000, 12345, top) if v <= top and (dtype == FP32 or v <= 60000)]
    x = torch.tensor(values, device="cuda", dtype=torch.float64)
    x = x[x.to(dtype).double() == x]
    S = x.numel()
    x = x.to(dtype).view(1, S, 1).expand(1, S, C).contiguous()
    dh = randn(1, S, C, dtype=branch, seed=1, scale=0.25)
    scale, w = randn(1, S, C, dtype=FP32, seed=2, scale=0.4), randn(C, dtype=FP32, seed=3)
    _, h = block.vsa_gate_norm(x, scale=scale, h_dtype=branch)
    assert not h.any()
    one, g1 = 1 + scale.double(), dh.double()
    for weight in (None, w):
        dx, _, _, _, dweight, _, dscale, _ = block.vsa_gate_norm_bwd(dh, None, x, weight=weight, scale=scale)
        assert not dscale.any() and (dweight is None or not dweight.any())
        g = g1 * one * (1 if weight is None else weight.double())
        want = 1000 * (g - g.mean(-1, keepdim=True))
        bound = 1000 * ref.F32 * (g.abs() + g.abs().mean(-1, keepdim=True)) + ref.half_step(dtype) * want.abs()
        ref.check("dx", dx, want, bound)
    # The sums of many tokens' units likewise.
    x = x[:, -1:].expand(1, 700, C).contiguous()
    _, _, _, _, dweight, _, _, _ = block.vsa_gate_norm_bwd(randn(1, 700, C, dtype=branch, seed=4), None, x, weight=w)
    assert not dweight.any()


def test_gate_norm_bwd_without_a_workspace(block):
    """Modulations of single tokens: their gradients come with a null workspace, with weights whose own are not
    wanted too, and are those of all gradients asked for together."""
    import ctypes
    B, S, C = 2, 3000, 1536
    x, y, dh = (randn(B, S, C, seed=i) for i in range(3))
    mods = [randn(B, S, C, seed=10 + i, scale=0.4) for i in range(3)]
    w, b = randn(C, seed=20), randn(C, seed=21)
    want = block.vsa_gate_norm_bwd(dh, None, x, y, mods[0], None, w, b, *mods[1:])
    outs = [torch.empty_like(x) for _ in range(5)]
    op = block.VsaGateNorm(B, S, C, S, 0, 0, 0, 0, 0, 1e-6, 1e-6, *(block.VsaModulation(m.data_ptr(), S * C, C) for m in mods),
                           None, w.data_ptr(), b.data_ptr())
    view = [block.VsaTokens(t.data_ptr(), S * C, C) for t in (dh, x, y, *outs[:2])]
    grads = block.VsaGateNormGrads(*(t.data_ptr() for t in outs[2:]))
    status = block._lib().vsa_gate_norm_bwd(op, view[0], None, *view[1:], grads, None, 0,
                                            ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert status == 0
    for got, ref_ in zip(outs, (want[0], want[1], want[2], want[6], want[7])):
        ref.check("alone", got, ref_.double(), 2 * ref.half_step(BF16) * ref_.double().abs() + 2.0 ** -20)
    one = block.vsa_gate_norm_bwd(dh, None, x, y, mods[0], None, w, b, *mods[1:],
                                  need_dparams=(True, False, False, False, True, True))
    assert one[3] is one[4] is one[5] is None and same_bits((one[0], one[1], one[2], one[6], one[7]), outs)
    with pytest.raises(ValueError):
        block.vsa_gate_norm_bwd(dh, None, x, y, need_dparams=(True, False))


def test_gate_norm_bwd_memory_of_frozen_weights(block):
    """Through autograd: a modulation that is trained beside weights that are not takes no workspace."""
    from block_sparse_video_tok_gb300 import autograd
    B, S, C = 1, 8192, 1536
    x, dh, w, shift = randn(B, S, C), randn(B, S, C, seed=1), randn(C, seed=2), randn(B, S, C, seed=4)
    scale = randn(B, S, C, seed=3, scale=0.4).requires_grad_(True)
    _, h = autograd.gate_norm(x, weight=w, scale=scale, shift=shift)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    (got,) = torch.autograd.grad(h, scale, dh)
    assert torch.cuda.max_memory_allocated() - before <= 2 * got.numel() * got.element_size() + (1 << 20)
    want = ref.gate_norm_bwd(dh, None, x, None, None, None, w, None, scale.detach(), shift, "layer", 1e-6, 1e-6)[6]
    ref.check("dscale", got, *want)


@pytest.mark.parametrize("case", [(2, 1, 1000, 400), (1, 7, 64, 700), (3, 43, 264, 86), (300, 1, 1536, 20), (1, 900, 1536, 900),
                                  (1, 900, 128, 1800), (1, 300, 6152, 300)], ids=str)
def test_gate_norm_bwd_of_some_parameters(block, case):
    """Each parameter's gradient asked for alone, in pairs, and all but it, is what it is among all of them, but for
    the order of fp32 sums (2^-15 of magnitudes that are at most some dozens of times the sums)."""
    B, G, C, S = case
    x, y, dh = (randn(B, S, C, seed=i) for i in range(3))
    gate, scale, shift = (randn(*((B, C) if G == 1 else (B, G, C)), dtype=FP32, seed=10 + i, scale=0.4) for i in range(3))
    post, w, b = (randn(C, dtype=FP32, seed=20 + i) for i in range(3))
    args = (dh, None, x, y, gate, post, w, b, scale, shift)
    every = block.vsa_gate_norm_bwd(*args)
    some = [[i == j for j in range(6)] for i in range(6)] + [[i != j for j in range(6)] for i in range(6)]
    some += [[j in (i, (i + 1) % 6) for j in range(6)] for i in range(6)] + [[True, False, False, False, True, True]]
    for wanted in some:
        got = block.vsa_gate_norm_bwd(*args, need_dparams=wanted)
        assert same_bits(got[:2], every[:2])
        for n, g, r in zip(wanted, got[2:], every[2:]):
            assert (g is not None) == n
            if n:
                assert ((g.double() - r.double()).norm() / r.double().norm()).item() <= 2.0 ** -14


def test_more_tokens_than_there_may_be(block):
    """Sizes past 2^30 and past 2^31 are refused by name, before anything is allocated for them."""
    for n in ((1 << 30) + 8, (1 << 31) + 8):
        x = torch.zeros(1, 1, 8, dtype=BF16, device="cuda").expand(1, n, 8)
        before = torch.cuda.max_memory_allocated()
        with pytest.raises(ValueError):
            block.vsa_gate_norm(x)
        with pytest.raises(ValueError):
            block.vsa_gate_norm_bwd(x, None, x)
        assert torch.cuda.max_memory_allocated() == before
        rows = torch.empty(n, 8, dtype=BF16, device="cuda")
        w = torch.zeros(8, 8, dtype=BF16, device="cuda")
        with pytest.raises(ValueError):
            block.vsa_linear(rows, w)
        with pytest.raises(ValueError):
            block.vsa_linear_bwd(rows, rows, w)
        del rows
        torch.cuda.empty_cache()
