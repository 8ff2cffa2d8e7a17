"""GPU: the waits inside the product kernels of vsa_linear -- many tiles handed from warp to warp without
a mistake, and time limits that fire without planting a defect (a limit far below the time that a
normal wait takes)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

SHORT_NS = 200
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def block():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    from block_sparse_video_tok_gb300 import build
    build.build()
    from block_sparse_video_tok_gb300 import block as binding
    return binding


def randn(*shape, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(BF16)


def case(M, K, N, seed):
    return dict(x=randn(M, K, seed=seed), w=randn(N, K, seed=seed + 1), b=randn(N, seed=seed + 2),
                r=randn(M, N, seed=seed + 3), dout=randn(M, N, seed=seed + 4))


def every(block, c):
    """Each of the products, with and without what their epilogues load."""
    out, pre = block.vsa_linear(c["x"], c["w"], c["b"], "silu", need_pre=True)
    both, _ = block.vsa_linear(c["x"], c["w"], c["b"], "silu", c["r"])
    return [out, pre, both, *block.vsa_linear_bwd(c["dout"], c["x"], c["w"], c["b"], "silu", pre),
            *block.vsa_linear_bwd(c["dout"], c["x"], c["w"], None, None, None, "silu", c["x"])[:2]]


def same_bits(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("size", [
    (40000, 64, 512),      # several tiles to a pair of CTAs, a single step of k each
    (5000, 712, 5000),     # whole tiles and tiles in parts
    (300, 4000, 520),      # tiles in parts alone
    (100, 2000, 136),      # clusters
], ids=str)
def test_many_tiles(block, size):
    """Calls that follow one another without a wait give the same bits every time, and no wait runs out."""
    from block_sparse_video_tok_gb300 import layer
    layer.vsa_layer_device_error()
    cases = [case(*size, seed) for seed in (1, 11)]
    want = [every(block, c) for c in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [every(block, c) for c in cases * 2]
        torch.cuda.synchronize()
        for i, x in enumerate(got):
            assert same_bits(x, want[i % 2])
    assert layer.vsa_layer_device_error() == 0


@pytest.mark.parametrize("size, long", [((9000, 2048, 4096), True), ((300, 2048, 512), False), ((1024, 1280, 1536), False)],
                         ids=["pairs", "clusters", "many_steps"])
def test_short_wait_limit_reports_timeout_then_recovers(block, size, long):
    """long: waits of tens of microseconds among them.  A probe of a barrier is suspended by the hardware for
    some microseconds before it fails and the limit is looked at, which is longer than the whole of a
    small product: there the limit may fire or not, and either way the next calls are right."""
    from block_sparse_video_tok_gb300 import layer, vsa
    layer.vsa_layer_device_error()
    c = case(*size, seed=5)
    want = every(block, c)
    torch.cuda.synchronize()
    assert layer.vsa_layer_device_error() == 0
    calls = [lambda: block.vsa_linear(c["x"], c["w"], c["b"], "silu"),
             lambda: block.vsa_linear(c["x"], c["w"], c["b"], None, c["r"]),
             lambda: block.vsa_linear_bwd(c["dout"], c["x"], c["w"], need_dweight=False),
             lambda: block.vsa_linear_bwd(c["dout"], c["x"], c["w"], need_dx=False)]
    prev = vsa.vsa_set_wait_limit_ns(SHORT_NS)
    bits = []
    try:
        for call in calls:
            call()
            bits.append(layer.vsa_layer_device_error())
    finally:
        vsa.vsa_set_wait_limit_ns(prev)
    assert all(b == vsa.DEVERR_TIMEOUT or (b == 0 and not long) for b in bits), bits
    # The context is intact: the same calls with the normal limit give the same bits.
    got = every(block, c)
    torch.cuda.synchronize()
    assert layer.vsa_layer_device_error() == 0
    assert same_bits(got, want)


@pytest.mark.parametrize("size", [(64, 256, 256), (128, 1000, 264), (512, 512, 512), (300, 4096, 64), (1021, 1000, 264)], ids=str)
def test_short_wait_limit_stops_small_products(block, size):
    """Products in small tiles, alone, in clusters and two to a launch: a limit below the time of one copy runs out
    in each, is reported, and the calls after it are right."""
    from block_sparse_video_tok_gb300 import layer, vsa
    layer.vsa_layer_device_error()
    c = case(*size, seed=7)
    want = every(block, c)
    torch.cuda.synchronize()
    assert layer.vsa_layer_device_error() == 0
    calls = [lambda: block.vsa_linear(c["x"], c["w"], c["b"], "silu", need_pre=True),
             lambda: block.vsa_linear(c["x"], c["w"], c["b"], None, c["r"]),
             lambda: block.vsa_linear_bwd(c["dout"], c["x"], c["w"], need_dweight=False),
             lambda: block.vsa_linear_bwd(c["dout"], c["x"], c["w"], need_dx=False),
             lambda: block.vsa_linear_bwd(c["dout"], c["x"], c["w"])]
    for _ in range(3):
        prev = vsa.vsa_set_wait_limit_ns(SHORT_NS)
        bits = []
        try:
            for call in calls:
                call()
                bits.append(layer.vsa_layer_device_error())
        finally:
            vsa.vsa_set_wait_limit_ns(prev)
        assert bits == [vsa.DEVERR_TIMEOUT] * len(calls)
        got = every(block, c)
        torch.cuda.synchronize()
        assert layer.vsa_layer_device_error() == 0
        assert same_bits(got, want)


@pytest.mark.parametrize("size, own", [
    ((8, 4096, 8192), True), ((8, 8192, 8192), False), ((1, 8192, 8192), False), ((8, 1536, 32768), True), ((8, 16384, 6144), False),
    ((16, 1536, 9216), True), ((16, 4096, 5120), False), ((24, 2048, 4096), True), ((17, 1536, 7168), True), ((24, 1024, 8192), False),
    ((24, 4096, 4096), False), ((25, 256, 256), False)], ids=str)
def test_which_few_rows_have_a_kernel_of_their_own(block, size, own):
    """That kernel waits for nothing, the tiles' kernels do: a limit that no wait keeps tells which of them ran."""
    from block_sparse_video_tok_gb300 import layer, vsa
    layer.vsa_layer_device_error()
    M, K, N = size
    x, w = randn(M, K, seed=1), randn(N, K, seed=2)
    prev = vsa.vsa_set_wait_limit_ns(SHORT_NS)
    try:
        block.vsa_linear(x, w)
        bits = layer.vsa_layer_device_error()
    finally:
        vsa.vsa_set_wait_limit_ns(prev)
    assert bits == (0 if own else vsa.DEVERR_TIMEOUT)
    out, want = block.vsa_linear(x, w)[0].double(), x.double() @ w.double().T
    mag = x.double().abs() @ w.double().abs().T
    # One rounding, and sums of K terms in fp32.
    assert bool(((out - want).abs() <= 2.0 ** -8 * want.abs() + K * 2.0 ** -24 * mag).all())
    assert layer.vsa_layer_device_error() == 0
