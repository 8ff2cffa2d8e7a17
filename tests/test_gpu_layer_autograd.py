"""GPU: the layer operators through autograd, in the surroundings of a user's program."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


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
    g = torch.Generator("cuda").manual_seed(seed + sum(shape))
    return torch.randn(shape, generator=g, device="cuda").to(BF16)


def behind_a_cat(f, leaves, before):
    """Gradients of the leaves through torch.cat([.., f(leaves) flattened]), which gives f's outputs
    gradients that start `before` elements into a buffer."""
    y = f(*leaves).flatten()
    head = randn(before).requires_grad_(True)
    g = torch.cat([randn(before, seed=1), torch.linspace(-1, 1, y.numel(), device="cuda").to(BF16)])
    return torch.autograd.grad(torch.cat([head, y]), leaves, g)


@pytest.mark.parametrize("name", ["norm_rope", "cross_attention"])
def test_gradient_that_starts_anywhere(layer, name):
    """An odd number of elements before an output moves its gradient off 16 bytes and changes no bit of
    what comes back."""
    from block_sparse_video_tok_gb300 import autograd
    if name == "norm_rope":
        f, leaves = lambda x, w: autograd.norm_rope(x, q_weight=w)[0], [randn(2, 37, 4, 128), randn(128)]
    else:
        f = autograd.cross_attention
        leaves = [randn(2, 4, 70, 128), randn(2, 2, 50, 128, seed=1), randn(2, 2, 50, 128, seed=2)]
    leaves = [x.requires_grad_(True) for x in leaves]
    want = behind_a_cat(f, leaves, 8)
    for before in (1, 7, 12):
        got = behind_a_cat(f, leaves, before)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), before


def test_error_bits_of_another_stream_are_not_lost(layer):
    """A bit that a call on another stream raises while the word is read and cleared is in that read or in
    the next.  The call starts after a wait of 0 to 200000 cycles, so that some fall on the read."""
    q = randn(1, 1, 1, 128)
    bad = torch.tensor([9], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    lost = 0
    for i in range(6000):
        with torch.cuda.stream(side):
            torch.cuda._sleep(1000 * (i % 200))
        layer.vsa_cross_fwd(q, q, q, bad, stream=side)
        first = layer.vsa_layer_device_error()
        side.synchronize()
        lost += (first | layer.vsa_layer_device_error()) != layer.DEVERR_KV_LEN
    assert lost == 0


def test_orders_that_do_not_fit(layer):
    """norm_rope's gradients follow dst alone: a token that goes to two rows, one that no row takes although
    dst says so and one whose row dst leaves out raise DEVERR_ORDER, in the forward or the backward that
    meets it.  Orders that fit raise nothing, and a forward without gradients may repeat tokens."""
    from block_sparse_video_tok_gb300.autograd import norm_rope
    q = randn(2, 4, 3, 128).requires_grad_(True)

    def bits(src, dst, grad=True):
        src, dst = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (src, dst))
        with torch.set_grad_enabled(grad):
            y = norm_rope(q, order=(src, dst))[0]
        forward = layer.vsa_layer_device_error()
        if grad:
            y.float().sum().backward()
        return forward, layer.vsa_layer_device_error()

    fits = [([0, 1, 2, 3], [0, 1, 2, 3]), ([3, -1, 0, 2, 1], [2, 4, 3, 0]), ([2, -1, -1], [-1, -1, 0, -1])]
    for src, dst in fits:
        assert bits(src, dst) == (0, 0), (src, dst)
    bad = layer.DEVERR_ORDER
    assert bits([3, -1, 0, 3, 1], [2, 4, -1, 0]) == (bad, 0)        # token 3 in rows 0 and 3
    assert bits([3, -1, 0, 2, 1], [2, 4, -1, 0]) == (bad, 0)        # token 2 left out
    assert bits([3, -1, 0, -1, 1], [2, 4, 3, 0]) == (0, bad)        # row 3 is empty
    assert bits([1, 0, 2, 3], [0, 1, 2, 3]) == (bad, bad)           # two rows exchanged
    assert bits([3, -1, 0, 3, 1], [2, 4, -1, 0], grad=False) == (0, 0)
    for src, dst in ((None, torch.arange(4, dtype=torch.int32, device="cuda")),
                     (torch.arange(4, dtype=torch.int32, device="cuda"), None)):
        with pytest.raises(ValueError):
            norm_rope(q, order=(src, dst))
