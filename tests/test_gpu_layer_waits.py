"""GPU: the waits inside the cross-attention kernels -- many short units handed from warp to warp
without a mistake, and time limits that fire without planting a defect (a limit far below the time
that a normal wait takes)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

SHORT_NS = 200
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def layer():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    from block_sparse_video_tok_gb300 import build
    build.build()
    from block_sparse_video_tok_gb300 import layer as binding
    return binding


def cross_inputs(B, Sq, Sk, H, Hk, seed):
    g = torch.Generator("cuda").manual_seed(seed)

    def heads(S, n):
        return torch.randn((B, S, n, 128), generator=g, device="cuda").to(BF16).transpose(1, 2)
    return heads(Sq, H), heads(Sq, H), heads(Sk, Hk), heads(Sk, Hk)  # do, q, k, v


def both(layer, do, q, k, v):
    o, lse = layer.vsa_cross_fwd(q, k, v)
    return (o, lse, *layer.vsa_cross_bwd(do, q, k, v, o, lse))


def same_bits(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("Sq, Sk, H, Hk", [
    (14207, 1, 20, 5),      # query tiles of a single short step: what a unit needs is prepared ahead
    (15701, 141, 12, 12),   # two steps
    (100, 15000, 8, 4),     # key tiles of a single query tile
], ids=["one_key", "two_key_tiles", "one_query_tile"])
def test_many_short_units(layer, Sq, Sk, H, Hk):
    """Calls that follow one another without a wait give the same bits every time, and no wait
    runs out."""
    layer.vsa_layer_device_error()
    cases = [cross_inputs(1, Sq, Sk, H, Hk, seed) for seed in (1, 2)]
    want = [both(layer, *c) for c in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [both(layer, *c) for c in cases * 2]
        torch.cuda.synchronize()
        for i, x in enumerate(got):
            assert same_bits(x, want[i % 2])
    assert layer.vsa_layer_device_error() == 0
    # One key: P is 1, o is v, and dv is the sum of do over the rows of the heads that share it.
    if Sk == 1:
        do, q, k, v = cases[0]
        assert torch.equal(want[0][0], v.repeat_interleave(H // Hk, 1).expand_as(q))
        dv = do.double().sum(2).view(1, Hk, H // Hk, 128).sum(2)
        terms = do.double().abs().sum(2).view(1, Hk, H // Hk, 128).sum(2)
        # fp32 sums of n terms, at most n steps of 2^-24 each of the terms' magnitudes (and P = 2^x
        # with an x off 0 by the rounding of a score, far below bf16's 2^-8 of the result).
        bound = dv.abs() * 2.0 ** -8 + terms * (Sq * H // Hk * 2.0 ** -24 + 2.0 ** -18)
        assert bool(((want[0][4][:, :, 0].double() - dv).abs() <= bound).all())


def test_short_wait_limit_reports_timeout_then_recovers(layer):
    from block_sparse_video_tok_gb300 import vsa
    layer.vsa_layer_device_error()
    args = cross_inputs(2, 4096, 4096, 4, 2, 5)
    want = both(layer, *args)
    torch.cuda.synchronize()
    assert layer.vsa_layer_device_error() == 0
    do, q, k, v = args
    prev = vsa.vsa_set_wait_limit_ns(SHORT_NS)
    try:
        layer.vsa_cross_fwd(q, k, v)
        fwd_bits = layer.vsa_layer_device_error()
        layer.vsa_cross_bwd(do, q, k, v, want[0], want[1])
        bwd_bits = layer.vsa_layer_device_error()
    finally:
        vsa.vsa_set_wait_limit_ns(prev)
    assert fwd_bits & vsa.DEVERR_TIMEOUT, hex(fwd_bits)
    assert bwd_bits & vsa.DEVERR_TIMEOUT, hex(bwd_bits)
    # The context is intact: the same calls with the normal limit give the same bits.
    got = both(layer, *args)
    torch.cuda.synchronize()
    assert layer.vsa_layer_device_error() == 0
    assert same_bits(got, want)
