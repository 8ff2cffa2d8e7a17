"""GPU: the example block (every operator of the package together) against the same block of plain PyTorch
operations in 64 bits, and its training steps."""
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
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "video_block.py")
    spec = importlib.util.spec_from_file_location("video_block", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def rms(x, w):
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w


def layer_norm(x):
    c = x - x.mean(-1, keepdim=True)
    return c / torch.sqrt(c.square().mean(-1, keepdim=True) + 1e-6)


def turn(x, cos, sin):
    a, b = x[..., 0::2], x[..., 1::2]
    c, s = cos[:, None], sin[:, None]
    return torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)


def attend(q, k, v, seen):
    s = (q @ k.transpose(-1, -2) * q.shape[-1] ** -0.5).masked_fill(~seen, -torch.inf)
    return s.softmax(-1) @ v


def plain(net, p, x, step, text, lens, idx):
    """net's forward in raster order with the parameters p, the selection given."""
    def product(name, t):
        return t @ p[name + "_w"].T + p[name + "_b"]

    heads = net.heads
    e = product("embed", step)
    shift1, scale1, gate1, shift2, scale2, gate2 = (
        t[:, None] for t in product("modulation", e * torch.sigmoid(e)).unflatten(-1, (6, net.dim)).unbind(1))
    q, k, v = product("qkv", layer_norm(x) * (1 + scale1) + shift1).unflatten(-1, (3, heads, 128)).unbind(2)
    cos, sin = net.cos.double(), net.sin.double()
    q, k = (turn(rms(y, p[w]), cos, sin) for y, w in ((q, "q_norm"), (k, "k_norm")))
    cube = net.order[1].long() // 64                             # of each token
    picked = torch.zeros(*idx.shape[:3], net.vbs.numel(), dtype=torch.bool, device=x.device).scatter_(3, idx.long(), True)
    seen = picked[:, :, cube][..., cube]                         # [B, H, token, token]
    o = attend(*(y.transpose(1, 2) for y in (q, k, v)), seen)
    x = x + gate1 * product("out", o.transpose(1, 2).flatten(2))
    h = layer_norm(x) * p["cross_weight"] + p["cross_bias"]
    q, k, v = (product(n, t).unflatten(-1, (heads, 128)) for n, t in (("text_q", h), ("text_k", text), ("text_v", text)))
    q, k = rms(q, p["text_q_norm"]), rms(k, p["text_k_norm"])
    seen = torch.arange(text.shape[1], device=x.device) < lens[:, None, None, None]
    o = attend(*(y.transpose(1, 2) for y in (q, k, v)), seen)
    x = x + product("text_out", o.transpose(1, 2).flatten(2))
    z = product("up", layer_norm(x) * (1 + scale2) + shift2)
    z = z * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3))
    return x + gate2 * product("down", z)


def test_block_against_plain(example):
    torch.manual_seed(3)
    net = example.VideoBlock(GRID, heads=4, density=0.5)
    x = torch.randn(2, GRID[0] * GRID[1] * GRID[2], 512, device="cuda", requires_grad=True)
    step = torch.randn(2, 256, device="cuda", dtype=torch.bfloat16)
    text = torch.randn(2, 70, 512, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    lens = torch.tensor([70, 13], dtype=torch.int32, device="cuda")
    chosen = []
    select = net.select

    def record(q, k):
        chosen.append(select(q, k))
        return chosen[0]

    net.select = record
    g = torch.randn_like(x)
    got = net(x, step, text, lens)
    assert got.dtype is torch.float32
    got.backward(g)
    p = {n: w.detach().double().requires_grad_(True) for n, w in net.named_parameters()}
    x64, t64 = (t.detach().double().requires_grad_(True) for t in (x, text))
    want = plain(net, p, x64, step.double(), t64, lens, chosen[0][0])
    want.backward(g.double())

    # Each of the block's bf16 results on the way is off by at most 2^-8 of a value (2^-9 rms); two
    # dozen of them in a row, taken as adding up in full, stay below 24 * 2^-8 of the result's norm.  A
    # gradient passes them twice, forward and back.
    def near(a, b, bound, name):
        off = ((a.double() - b).norm() / b.norm()).item()
        assert off <= bound, "%s: %.3g > %.3g" % (name, off, bound)

    near(got.detach(), want.detach(), 24 * 2.0 ** -8, "output")
    near(x.grad, x64.grad, 48 * 2.0 ** -8, "x")
    near(text.grad, t64.grad, 48 * 2.0 ** -8, "text")
    for name, w in net.named_parameters():
        near(w.grad, p[name].grad, 48 * 2.0 ** -8, name)


def test_training_steps_run(example):
    losses = example.train(GRID, heads=2, text=40, batch=2, steps=3)
    assert len(losses) == 3 and all(x == x and x < float("inf") for x in losses)
