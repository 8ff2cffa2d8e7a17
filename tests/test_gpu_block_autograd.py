"""GPU: the block operators through autograd, in the surroundings of a user's program, and a whole block
of them with the attention operators against plain operations in 64 bits."""
import pytest
import torch

from tests import block_ref as ref

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def autograd():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    from block_sparse_video_tok_gb300 import build
    build.build()
    from block_sparse_video_tok_gb300 import autograd as binding
    return binding


@pytest.fixture(autouse=True)
def no_device_error(autograd):
    from block_sparse_video_tok_gb300 import layer
    layer.vsa_layer_device_error()
    yield
    assert layer.vsa_layer_device_error() == 0


def randn(*shape, dtype=BF16, seed=0, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed + sum(shape))
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def leaves(*tensors):
    return [t.requires_grad_(True) for t in tensors]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_gate_norm_gives_the_binding_s_gradients(autograd):
    from block_sparse_video_tok_gb300 import block
    B, S, C = 2, 30, 264
    ts = leaves(randn(B, S, C), randn(B, S, C, seed=1), randn(B, 3, C, seed=2), randn(C, seed=3), randn(C, seed=4),
                randn(C, seed=5), randn(B, 3, C, seed=6), randn(B, 3, C, seed=7))
    x, h = autograd.gate_norm(*ts, kind="rms")
    dx, dh = randn(B, S, C, seed=8), randn(B, S, C, seed=9)
    got = torch.autograd.grad([x, h], ts, [dx, dh])
    assert same(got, block.vsa_gate_norm_bwd(dh, dx, x.detach(), *(t.detach() for t in ts[1:]), kind="rms"))
    # One output alone: the other's gradient is zero.
    x, h = autograd.gate_norm(*ts, kind="rms")
    got = torch.autograd.grad(h, ts, dh, retain_graph=True)
    assert same(got, block.vsa_gate_norm_bwd(dh, None, x.detach(), *(t.detach() for t in ts[1:]), kind="rms"))
    got = torch.autograd.grad(x, ts[:3], dx, allow_unused=True)
    want = block.vsa_gate_norm_bwd(torch.zeros_like(dh), dx, x.detach(), *(t.detach() for t in ts[1:]), kind="rms")
    assert same(got, want)


def test_gate_norm_without_a_branch(autograd):
    from block_sparse_video_tok_gb300 import block
    x, w = leaves(randn(2, 9, 64, dtype=FP32), randn(64, dtype=FP32, seed=1))
    same_x, h = autograd.gate_norm(x, weight=w, h_dtype=BF16)
    assert same_x is x and h.dtype is BF16
    dh = randn(2, 9, 64, seed=2)
    got = torch.autograd.grad(h, (x, w), dh)
    want = block.vsa_gate_norm_bwd(dh, None, x.detach(), weight=w.detach())
    assert same(got, (want[0], want[4]))


def test_modulations_that_are_broadcast(autograd):
    """One modulation for all entries: its gradient is the sum of the entries'."""
    B, S, C = 3, 17, 64
    x, y = randn(B, S, C, dtype=FP32), randn(B, S, C, dtype=FP32, seed=1)
    one = leaves(*(randn(1, C, dtype=FP32, seed=2 + i) for i in range(3)))
    each = leaves(*(t.detach().repeat(B, 1) for t in one))
    grads = []
    for ts in (one, each):
        gate, scale, shift = (t.expand(B, C) for t in ts)
        a, h = autograd.gate_norm(x, y, gate, scale=scale, shift=shift)
        grads.append(torch.autograd.grad((a * h).sum(), ts))
    for a, b in zip(*grads):
        assert torch.allclose(a, b.sum(0, keepdim=True), rtol=1e-5, atol=1e-5)


def test_linear_gives_the_binding_s_gradients(autograd):
    from block_sparse_video_tok_gb300 import block
    x, w, b, r = leaves(randn(3, 50, 136), randn(264, 136, seed=1, scale=0.1), randn(264, dtype=FP32, seed=2),
                        randn(3, 50, 264, seed=3))
    out = autograd.linear(x, w, b, "gelu", r)
    dout = randn(3, 50, 264, seed=4)
    got = torch.autograd.grad(out, (x, w, b, r), dout)
    d = [t.detach() for t in (x, w, b, r)]
    want, pre = block.vsa_linear(*d[:3], "gelu", d[3], need_pre=True)
    assert torch.equal(out, want) and torch.equal(got[3], dout)
    assert same(got, block.vsa_linear_bwd(dout, *d[:3], "gelu", pre))
    # What is not asked for is not computed.
    out = autograd.linear(x, w.detach(), None, "gelu", r.detach())
    assert torch.autograd.grad(out, x, dout)[0].shape == x.shape
    with torch.no_grad():
        assert autograd.linear(x, w, b, "gelu", r).grad_fn is None


def test_mlp_is_the_two_products(autograd):
    ts = leaves(randn(2, 40, 64), randn(256, 64, seed=1, scale=0.1), randn(256, seed=2),
                randn(64, 256, seed=3, scale=0.1), randn(64, seed=4), randn(2, 40, 64, seed=5))
    dout = randn(2, 40, 64, seed=6)
    x, w1, b1, w2, b2, r = ts
    out = autograd.mlp(x, w1, b1, w2, b2, "silu", r)
    got = torch.autograd.grad(out, ts, dout)
    two = autograd.linear(autograd.linear(x, w1, b1, "silu"), w2, b2, None, r)
    assert torch.equal(out, two)
    want = torch.autograd.grad(two, ts, dout)
    # Through the middle, dz is rounded once here and twice there (the gradient of the middle, then dz):
    # half a bf16 step of difference in each of its elements, 2^-8 of the magnitudes that follow.
    wide = [t.detach().double() for t in ts]
    pre = wide[0].flatten(0, 1) @ wide[1].T + wide[2]
    dmid = (dout.double().flatten(0, 1) @ wide[3]).abs() * ref.slope(pre, "silu").abs()
    bound = {0: (dmid @ wide[1].abs()).view_as(x), 1: dmid.T @ wide[0].flatten(0, 1).abs(), 2: dmid.sum(0)}
    for i, (a, b) in enumerate(zip(got, want)):
        if i in bound:
            assert bool(((a.double() - b.double()).abs() <= 2.0 ** -6 * bound[i]).all()), i
        else:
            assert torch.equal(a, b), i


@pytest.mark.parametrize("name", ["gate_norm", "linear", "mlp"])
def test_gradient_that_starts_anywhere(autograd, name):
    """An odd number of elements before an output moves its gradient off 16 bytes, and an expanded or
    transposed one has other strides; no bit of what comes back changes."""
    if name == "gate_norm":
        f, ts = lambda x, y: autograd.gate_norm(x, y)[1], leaves(randn(2, 30, 64), randn(2, 30, 64, seed=1))
    elif name == "linear":
        f, ts = lambda x, w: autograd.linear(x, w, None, "silu"), leaves(randn(2, 30, 64), randn(64, 64, seed=1))
    else:
        f = lambda x, w, v: autograd.mlp(x, w, None, v, None)  # noqa: E731
        ts = leaves(randn(2, 30, 64), randn(128, 64, seed=1), randn(64, 128, seed=2))
    g = randn(2, 30, 64, seed=3)
    want = torch.autograd.grad(f(*ts), ts, g)
    for before in (1, 7, 8):
        room = torch.zeros(before + g.numel(), dtype=BF16, device="cuda")
        room[before:] = g.flatten()
        assert same(torch.autograd.grad(f(*ts), ts, room[before:].view(2, 30, 64)), want), before
    for a, b in ((1, 2), (0, 1)):
        assert same(torch.autograd.grad(f(*ts), ts, g.transpose(a, b).contiguous().transpose(a, b)), want), (a, b)
    wide = torch.zeros(2, 30, 72, dtype=BF16, device="cuda")
    wide[..., 8:] = g
    assert same(torch.autograd.grad(f(*ts), ts, wide[..., 8:]), want)
    row = randn(64, seed=4)
    assert same(torch.autograd.grad(f(*ts), ts, row.expand(2, 30, 64)),
                torch.autograd.grad(f(*ts), ts, row.expand(2, 30, 64).contiguous()))


def test_second_derivatives_raise(autograd):
    x, w = leaves(randn(4, 64), randn(64, 64, seed=1))
    (g,) = torch.autograd.grad(autograd.linear(x, w).float().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.float().sum().backward()
    x = randn(1, 4, 64).requires_grad_(True)
    (g,) = torch.autograd.grad(autograd.gate_norm(x)[1].float().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.float().sum().backward()


def test_refusals(autograd):
    """Arguments that the kernels do not take raise in the binding, by name."""
    from block_sparse_video_tok_gb300 import block
    x, m = randn(2, 12, 64), randn(2, 64, seed=1)
    for bad in (dict(gate=m), dict(scale=randn(2, 5, 64)), dict(scale=m, shift=randn(2, 3, 64)), dict(kind="batch"),
                dict(weight=randn(72)), dict(scale=randn(3, 64)), dict(x_out=x)):
        with pytest.raises((ValueError, TypeError)):
            block.vsa_gate_norm(x, **bad)
    with pytest.raises(TypeError):
        block.vsa_gate_norm(x, scale=m, shift=m.float())
    with pytest.raises(TypeError):
        block.vsa_gate_norm(x, h_dtype=FP16)
    for t in (x[:, :, ::2], x[:, :, 4:], x.flatten()[1:1 + 2 * 11 * 64].view(2, 11, 64), x[:, :0], x[:, :, :60].contiguous()):
        with pytest.raises(ValueError):
            block.vsa_gate_norm(t)
    w = randn(64, 64, seed=2)
    for args in ((x, w[:60]), (x, w[:, :56]), (x[..., :60].contiguous(), w[:, :60].contiguous()), (x, w, randn(56)),
                 (x, w, None, "relu"), (x, w, None, None, x[:1]), (x[:, ::2].transpose(0, 1), w), (x[:, :1].expand(2, 12, 64), w),
                 (x[:, :0], w)):
        with pytest.raises(ValueError):
            block.vsa_linear(*args)
    for args in ((x.float(), w), (x, w.half()), (x, w, randn(64, dtype=FP16))):
        with pytest.raises(TypeError):
            block.vsa_linear(*args)
    with pytest.raises(ValueError):
        block.vsa_linear_bwd(x, x, w, act="gelu")
    with pytest.raises(ValueError):
        block.vsa_linear_bwd(x, x, w, x_act="gelu")


def test_backward_in_a_graph(autograd):
    """A whole training step of the operators, captured and replayed on other inputs."""
    ts = leaves(randn(2, 40, 64), randn(2, 40, 64, seed=1), randn(2, 64, seed=2), randn(2, 64, seed=3),
                randn(2, 64, seed=4), randn(256, 64, seed=5, scale=0.1), randn(256, seed=6),
                randn(64, 256, seed=7, scale=0.1), randn(64, seed=8))

    def step():
        x, y, gate, scale, shift, w1, b1, w2, b2 = ts
        x, h = autograd.gate_norm(x, y, gate, scale=scale, shift=shift)
        return torch.autograd.grad(autograd.mlp(h, w1, b1, w2, b2, residual=x).float().square().sum(), ts)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = step()
    for seed in (70, 71):
        with torch.no_grad():
            ts[0].copy_(randn(2, 40, 64, seed=seed))
            ts[5].copy_(randn(256, 64, seed=seed, scale=0.1))
        graph.replay()
        torch.cuda.synchronize()
        assert same(grads, step())


def test_residual_of_other_leading_dimensions(autograd):
    """A residual of as many rows as the output: its gradient has its own shape."""
    ts = leaves(randn(2, 30, 64), randn(64, 64, seed=1, scale=0.1), randn(64, 64, seed=2, scale=0.1))
    x, w1, w2 = ts
    dout = randn(2, 30, 64, seed=3)
    wide = torch.zeros(2, 30, 72, dtype=BF16, device="cuda")
    wide[..., 8:] = dout
    for f in (lambda r: autograd.linear(x, w1, None, None, r), lambda r: autograd.linear(x, w1, None, "silu", r),
              lambda r: autograd.mlp(x, w1, None, w2, None, "silu", r)):
        for shape in ((60, 64), (1, 60, 64), (6, 10, 64), (2, 30, 1, 64)):
            (r,) = leaves(randn(60, 64, seed=4).view(shape))
            (same_r,) = leaves(r.detach().view(2, 30, 64))
            want = torch.autograd.grad(f(same_r), (x, w1, same_r), dout)
            for g in (dout, wide[..., 8:]):
                got = torch.autograd.grad(f(r), (x, w1, r), g)
                assert got[2].shape == shape and same(got[:2], want[:2]) and torch.equal(got[2].view_as(dout), want[2])


def test_a_chain_of_the_operators_in_the_norm(autograd):
    """Norm, two products and the gated sum with the next norm, against plain operations in 64 bits.  Some ten
    bf16 results forward and as many back, half a step each, independent of one another: in the root of the sum of
    squares sqrt(20) 2^-8, taken twice for the slopes, gates and 1 / deviations they pass through."""
    B, S, C, W = 2, 150, 264, 1032
    x, y = randn(B, S, C, dtype=FP32), randn(B, S, C, seed=1)
    mods = [randn(B, C, seed=2 + i, scale=0.4) for i in range(6)]
    w1, b1, w2, b2 = randn(W, C, seed=8, scale=C ** -0.5), randn(W, seed=9), randn(C, W, seed=10, scale=W ** -0.5), randn(C, seed=11)
    nw, nb = randn(C, seed=12, scale=0.1) + 1, randn(C, seed=13, scale=0.1)
    ts = leaves(x, y, *mods, w1, b1, w2, b2, nw, nb)
    dx, dh = randn(B, S, C, dtype=FP32, seed=14), randn(B, S, C, seed=15)

    def own(x, y, g1, s1, t1, g2, s2, t2, w1, b1, w2, b2, nw, nb):
        x, h = autograd.gate_norm(x, y, g1, scale=s1, shift=t1)
        return autograd.gate_norm(x, autograd.mlp(h, w1, b1, w2, b2, "gelu_tanh"), g2, weight=nw, bias=nb, scale=s2, shift=t2)

    def plain(x, y, g1, s1, t1, g2, s2, t2, w1, b1, w2, b2, nw, nb):
        def norm(x):
            c = x - x.mean(-1, keepdim=True)
            return c / torch.sqrt(c.square().mean(-1, keepdim=True) + 1e-6)
        x = x + g1[:, None] * y
        h = norm(x) * (1 + s1[:, None]) + t1[:, None]
        x = x + g2[:, None] * (ref.act(h @ w1.T + b1, "gelu_tanh") @ w2.T + b2)
        return x, (norm(x) * nw + nb) * (1 + s2[:, None]) + t2[:, None]

    got = own(*ts)
    wide = leaves(*(t.detach().double() for t in ts))
    want = plain(*wide)
    bound = 2 * 20 ** 0.5 * 2.0 ** -8
    pairs = list(zip(got, want)) + list(zip(torch.autograd.grad(got, ts, [dx, dh]),
                                            torch.autograd.grad(want, wide, [dx.double(), dh.double()])))
    for i, (a, b) in enumerate(pairs):
        error = ((a.detach().double() - b.detach()).norm() / b.detach().norm()).item()
        assert error <= bound, (i, error, bound)
