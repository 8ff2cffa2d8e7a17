"""A whole video transformer block on the package's operators, trained for a few steps on synthetic data.
The stream is fp32, the branches bf16; the step's embedding modulates the norms and gates the branches:

    embedding -> linear (silu) -> linear: six modulations
    gate_norm -> qkv product -> norm_rope -> block_sparse_attention -> output product
    gate_norm (gated sum, norm) -> query product -> norm_rope -> cross_attention -> output product
    gate_norm (sum, norm, modulation) -> mlp -> gated sum

    python examples/video_block.py [--grid 21x30x52] [--text 512] [--steps 5]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

from block_sparse_video_tok_gb300 import layer  # noqa: E402
from block_sparse_video_tok_gb300.autograd import (  # noqa: E402
    block_sparse_attention, cross_attention, gate_norm, linear, mlp, norm_rope)

HEAD_DIM = 128


class VideoBlock(torch.nn.Module):
    """Self attention over the cubes that each cube scores highest, attention to text states, and two
    products with a gelu between them; each branch normalised before and gated after."""

    def __init__(self, grid, heads=12, density=0.125, widen=4, embed=256, device="cuda"):
        super().__init__()
        self.heads, self.dim = heads, heads * HEAD_DIM
        dim = self.dim

        def parameter(*shape, scale=0.0, offset=0.0, dtype=torch.bfloat16):
            return torch.nn.Parameter((torch.randn(shape, device=device) * scale + offset).to(dtype))

        def product(name, n_in, n_out):
            setattr(self, name + "_w", parameter(n_out, n_in, scale=n_in ** -0.5))
            setattr(self, name + "_b", parameter(n_out))

        for name, n_in, n_out in (("embed", embed, dim), ("modulation", dim, 6 * dim), ("qkv", dim, 3 * dim),
                                  ("out", dim, dim), ("text_q", dim, dim), ("text_k", dim, dim), ("text_v", dim, dim),
                                  ("text_out", dim, dim), ("up", dim, widen * dim), ("down", widen * dim, dim)):
            product(name, n_in, n_out)
        self.cross_weight, self.cross_bias = parameter(dim, offset=1.0), parameter(dim)
        for name in ("q_norm", "k_norm", "text_q_norm", "text_k_norm"):
            setattr(self, name, parameter(HEAD_DIM, offset=1.0, dtype=torch.float32))
        src, dst, self.vbs = layer.video_token_order(grid, device=device)
        self.order = src, dst
        positions = torch.cartesian_prod(*(torch.arange(n) for n in grid))
        self.cos, self.sin = layer.rotation_table(positions, HEAD_DIM, device=device)
        self.topk = max(1, round(density * self.vbs.numel()))

    def product(self, name, x, act=None):
        return linear(x, getattr(self, name + "_w"), getattr(self, name + "_b"), act)

    def select(self, q, k):
        """The top cubes of each cube, ascending: q2k_idx [B, H, cubes, topk], q2k_num."""
        with torch.no_grad():
            n = self.vbs.numel()
            mean_q, mean_k = (x.unflatten(2, (n, -1)).float().sum(3) / self.vbs[:, None] for x in (q, k))
            idx = (mean_q @ mean_k.transpose(-1, -2)).topk(self.topk).indices.sort().values.int()
            return idx, torch.full(idx.shape[:3], self.topk, dtype=torch.int32, device=idx.device)

    def heads_of(self, x):
        return x.unflatten(-1, (-1, HEAD_DIM))

    def forward(self, x, step, text, text_len=None):
        """x fp32 [B, T * H * W, dim] in raster order, step [B, embed] of the diffusion step, text
        [B, n, dim] bf16, its lengths int32 [B] or None."""
        six = self.product("modulation", self.product("embed", step, "silu")).unflatten(-1, (6, self.dim))
        shift1, scale1, gate1, shift2, scale2, gate2 = six.unbind(1)

        _, h = gate_norm(x, scale=scale1, shift=shift1, h_dtype=torch.bfloat16)
        q, k, v = self.heads_of(self.product("qkv", h)).unflatten(2, (3, self.heads)).unbind(2)
        q, k, v = norm_rope(q, k, v, self.q_norm, self.k_norm, self.cos, self.sin, self.order)
        o = block_sparse_attention(q, k, v, *self.select(q, k), self.vbs)
        y = self.product("out", o.index_select(2, self.order[1]).transpose(1, 2).flatten(2))

        x, h = gate_norm(x, y, gate1, weight=self.cross_weight, bias=self.cross_bias)
        q, _, _ = norm_rope(self.heads_of(self.product("text_q", h)), q_weight=self.text_q_norm)
        k, _, v = norm_rope(self.heads_of(self.product("text_k", text)), v=self.heads_of(self.product("text_v", text)),
                            q_weight=self.text_k_norm)
        o = cross_attention(q, k, v, text_len)
        y = self.product("text_out", o.transpose(1, 2).flatten(2))

        x, h = gate_norm(x, y, scale=scale2, shift=shift2)
        y = mlp(h, self.up_w, self.up_b, self.down_w, self.down_b, "gelu_tanh")
        return gate_norm(x, y, gate2)[0]            # (in a stack, with the next block's first norm)


def train(grid=(21, 30, 52), heads=12, text=512, batch=1, steps=5, seed=0, lr=1e-3):
    """Fits the block to a fixed random target; the losses of the steps."""
    torch.manual_seed(seed)
    net = VideoBlock(grid, heads)
    tokens = grid[0] * grid[1] * grid[2]
    x, target = (torch.randn(batch, tokens, net.dim, device="cuda") for _ in range(2))
    step = torch.randn(batch, 256, device="cuda", dtype=torch.bfloat16)
    states = torch.randn(batch, text, net.dim, device="cuda", dtype=torch.bfloat16)
    lens = torch.randint(1, text + 1, (batch,), device="cuda", dtype=torch.int32)
    opt = torch.optim.Adam(net.parameters(), lr=lr)
    losses = []
    for _ in range(steps):
        opt.zero_grad()
        loss = (net(x, step, states, lens) - target).square().mean()
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
