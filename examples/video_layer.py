"""The attention part of a video transformer layer on the package's operators, trained for a few
steps on synthetic data:

    projections -> norm_rope (norm, rotation, raster order -> 4x4x4 cubes)
                -> block_sparse_attention -> back to raster order, output projection
    query projection -> norm_rope (norm alone) -> cross_attention to text states -> projection

    python examples/video_layer.py [--grid 21x30x52] [--text 512] [--steps 5]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

from block_sparse_video_tok_gb300 import layer  # noqa: E402
from block_sparse_video_tok_gb300.autograd import (  # noqa: E402
    block_sparse_attention, cross_attention, norm_rope)

HEAD_DIM = 128


class VideoAttention(torch.nn.Module):
    """Self attention over the cubes that each cube scores highest (by its mean query and the
    others' mean keys), then attention to text states of each batch entry's own length."""

    def __init__(self, grid, heads=12, text_heads=None, density=0.125, device="cuda"):
        super().__init__()
        self.heads, self.text_heads = heads, text_heads or heads
        dim = heads * HEAD_DIM

        def linear(n_in, n_out):
            return torch.nn.Linear(n_in, n_out, bias=False, device=device, dtype=torch.bfloat16)

        def weight():
            return torch.nn.Parameter(torch.ones(HEAD_DIM, device=device))

        self.qkv, self.out = linear(dim, 3 * dim), linear(dim, dim)
        self.text_q, self.text_out = linear(dim, dim), linear(dim, dim)
        self.text_kv = linear(dim, 2 * self.text_heads * HEAD_DIM)
        self.q_norm, self.k_norm, self.text_q_norm, self.text_k_norm = (weight() for _ in range(4))
        src, dst, self.vbs = layer.video_token_order(grid, device=device)
        self.order = src, dst
        t, h, w = (torch.arange(n) for n in grid)
        positions = torch.cartesian_prod(t, h, w)
        self.cos, self.sin = layer.rotation_table(positions, HEAD_DIM, device=device)
        self.topk = max(1, round(density * self.vbs.numel()))

    def select(self, q, k):
        """The top cubes of each cube, ascending: q2k_idx [B, H, cubes, topk], q2k_num."""
        with torch.no_grad():
            n = self.vbs.numel()
            mean_q, mean_k = (x.unflatten(2, (n, -1)).float().sum(3) / self.vbs[:, None] for x in (q, k))
            idx = (mean_q @ mean_k.transpose(-1, -2)).topk(self.topk).indices.sort().values.int()
            return idx, torch.full(idx.shape[:3], self.topk, dtype=torch.int32, device=idx.device)

    def forward(self, x, text, text_len=None):
        """x [B, T * H * W, dim] in raster order, text [B, n, dim], its lengths int32 [B] or None."""
        q, k, v = self.qkv(x).unflatten(-1, (3, self.heads, HEAD_DIM)).unbind(2)
        q, k, v = norm_rope(q, k, v, self.q_norm, self.k_norm, self.cos, self.sin, self.order)
        o = block_sparse_attention(q, k, v, *self.select(q, k), self.vbs)
        o = o.index_select(2, self.order[1]).transpose(1, 2).flatten(2)
        x = x + self.out(o)

        q = self.text_q(x).unflatten(-1, (self.heads, HEAD_DIM))
        k, v = self.text_kv(text).unflatten(-1, (2, self.text_heads, HEAD_DIM)).unbind(2)
        q, _, _ = norm_rope(q, q_weight=self.text_q_norm)
        k, _, v = norm_rope(k, v=v, q_weight=self.text_k_norm)
        o = cross_attention(q, k, v, text_len)
        return x + self.text_out(o.transpose(1, 2).flatten(2))


def train(grid=(21, 30, 52), heads=12, text=512, batch=1, steps=5, seed=0, lr=1e-3):
    """Fits the layer to a fixed random target; the losses of the steps."""
    torch.manual_seed(seed)
    net = VideoAttention(grid, heads)
    tokens, dim = grid[0] * grid[1] * grid[2], heads * HEAD_DIM
    x, target = (torch.randn(batch, tokens, dim, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    states = torch.randn(batch, text, dim, device="cuda", dtype=torch.bfloat16)
    lens = torch.randint(1, text + 1, (batch,), device="cuda", dtype=torch.int32)
    opt = torch.optim.Adam(net.parameters(), lr=lr)
    losses = []
    for _ in range(steps):
        opt.zero_grad()
        loss = (net(x, states, lens).float() - target.float()).square().mean()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    bits = layer.vsa_layer_device_error()
    if bits:
        raise RuntimeError("device error bits %#x" % bits)
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--grid", default="21x30x52")
    ap.add_argument("--heads", type=int, default=12)
    ap.add_argument("--text", type=int, default=512)
    ap.add_argument("--batch", type=int, default=1)
    ap.add_argument("--steps", type=int, default=5)
    a = ap.parse_args()
    shape = tuple(int(n) for n in a.grid.split("x"))
    for i, loss in enumerate(train(shape, a.heads, a.text, a.batch, a.steps)):
        print("step %d  loss %.6f" % (i, loss))
