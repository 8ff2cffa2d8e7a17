"""GPU: the example layer (norm and rotation, block-sparse attention, cross attention together)
against the same layer of plain PyTorch operations in 64 bits, and its training steps."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

GRID = (5, 6, 7)


@pytest.fixture(scope="module")
def example():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    from block_sparse_video_tok_gb300 import build
    build.build()
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "video_layer.py")
    spec = importlib.util.spec_from_file_location("video_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def rms(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w


def turn(x, cos, sin):
    a, b = x[..., 0::2], x[..., 1::2]
    c, s = cos[:, None], sin[:, None]
    return torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)


def attend(q, k, v, seen):
    s = (q @ k.transpose(-1, -2) * q.shape[-1] ** -0.5).masked_fill(~seen, -torch.inf)
    return s.softmax(-1) @ v


def plain(net, p, x, text, lens, idx):
    """net's forward in raster order with the parameters p, the selection given."""
    heads = net.heads
    q, k, v = (x @ p["qkv.weight"].T).unflatten(-1, (3, heads, 128)).unbind(2)
    cos, sin = net.cos.double(), net.sin.double()
    q, k = (turn(rms(y, p[w]), cos, sin) for y, w in ((q, "q_norm"), (k, "k_norm")))
    cube = net.order[1].long() // 64                             # of each token
    n = net.vbs.numel()
    picked = torch.zeros(*idx.shape[:3], n, dtype=torch.bool, device=x.device).scatter_(3, idx.long(), True)
    seen = picked[:, :, cube][..., cube]                         # [B, H, token, token]
    q, k, v = (y.transpose(1, 2) for y in (q, k, v))
    x = x + attend(q, k, v, seen).transpose(1, 2).flatten(2) @ p["out.weight"].T
    q = rms((x @ p["text_q.weight"].T).unflatten(-1, (heads, 128)), p["text_q_norm"])
    k, v = (text @ p["text_kv.weight"].T).unflatten(-1, (2, net.text_heads, 128)).unbind(2)
    k = rms(k, p["text_k_norm"])
    q, k, v = (y.transpose(1, 2) for y in (q, k, v))
    k, v = (y.repeat_interleave(heads // net.text_heads, 1) for y in (k, v))
    seen = torch.arange(text.shape[1], device=x.device) < lens[:, None, None, None]
    o = attend(q, k, v, seen)
    return x + o.transpose(1, 2).flatten(2) @ p["text_out.weight"].T


def test_layer_against_plain(example):
    torch.manual_seed(3)
    net = example.VideoAttention(GRID, heads=4, text_heads=2, density=0.5)
    x = torch.randn(2, GRID[0] * GRID[1] * GRID[2], 512, device="cuda", dtype=torch.bfloat16)
    text = torch.randn(2, 70, 512, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    lens = torch.tensor([70, 13], dtype=torch.int32, device="cuda")
    chosen = []
    select = net.select

    def record(q, k):
        chosen.append(select(q, k))
        return chosen[0]

    net.select = record
    g = torch.randn_like(x)
    got = net(x, text, lens)
    got.backward(g)
    p = {n: w.detach().double().requires_grad_(True) for n, w in net.named_parameters()}
    t64 = text.detach().double().requires_grad_(True)
    want = plain(net, p, x.double(), t64, lens, chosen[0][0])
    want.backward(g.double())

    # Each of the layer's bf16 results on the way is off by at most 2^-8 of a value (2^-9 rms); a
    # dozen of them in a row, taken as adding up in full, stay below 12 * 2^-8 of the result's norm.
    # A gradient passes them twice, forward and back.
    def near(a, b, bound, name):
        off = ((a.double() - b).norm() / b.norm()).item()
        assert off <= bound, "%s: %.3g > %.3g" % (name, off, bound)

    near(got.detach(), want.detach(), 12 * 2.0 ** -8, "output")
    near(text.grad, t64.grad, 24 * 2.0 ** -8, "text")
    for name, w in net.named_parameters():
        near(w.grad, p[name].grad, 24 * 2.0 ** -8, name)


def test_training_steps(example):
    losses = example.train(GRID, heads=2, text=40, batch=2, steps=4)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
