"""The layer operators without a GPU: include/vsa_layer.h's symbols, its refusals (made on the host
before anything touches the device), the binding's refusals, and the token order and angle
helpers."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

from block_sparse_video_tok_gb300 import build as vsa_build
from block_sparse_video_tok_gb300 import workloads

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PTR = 0x100000


@pytest.fixture(scope="module")
def layer():
    vsa_build.build()
    from block_sparse_video_tok_gb300 import layer as binding
    return binding


def test_every_declared_symbol_is_exported(layer):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "vsa_layer.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(vsa_[a-z_]+)\s*\(", text)))
    assert len(names) == 8 and sorted(layer.SIGNATURES) == names
    for name in names:
        assert hasattr(layer._lib(), name), name


def norm_op(layer, **changes):
    f = dict(batch=2, tokens=10, rows=10, head_dim=128, dtype=0, weight_dtype=0, rot=64, halves=0,
             eps=1e-6, q_weight=PTR, k_weight=PTR, cosines=PTR, sines=PTR, table_batch_stride=0,
             order=None)
    f.update(changes)
    return layer.VsaNormRope(**f)


def heads(layer, H=4, S=10, D=128, ptr=PTR, **changes):
    f = dict(data=ptr, batch_stride=H * S * D, head_stride=S * D, token_stride=D, heads=H)
    f.update(changes)
    return layer.VsaHeads(**f)


def norm_fwd(layer, op, x=None, y=None):
    x, y = x or heads(layer), y or heads(layer)
    return layer._lib().vsa_norm_rope_fwd(op, x, None, None, y, None, None, None)


@pytest.mark.parametrize("status,changes", [
    (1, dict(batch=0)), (1, dict(tokens=0)), (1, dict(rows=0)), (1, dict(rows=11)),
    (2, dict(head_dim=0)), (2, dict(head_dim=100)), (2, dict(head_dim=264)), (2, dict(dtype=3)),
    (2, dict(weight_dtype=1)), (1, dict(rot=-8)), (1, dict(rot=136)), (2, dict(rot=60)),
    (2, dict(rot=40, halves=1)), (1, dict(eps=math.nan)), (1, dict(eps=-1.0)),
    (1, dict(cosines=None)), (1, dict(sines=PTR + 4)), (1, dict(table_batch_stride=-4)),
    (1, dict(table_batch_stride=2)), (1, dict(q_weight=PTR + 2)), (1, dict(order=PTR + 1)),
    (2, dict(tokens=1 << 30, rows=1 << 30, batch=4)),
])
def test_norm_rope_refuses_bad_operators(layer, status, changes):
    assert norm_fwd(layer, norm_op(layer, **changes)) == status
    assert layer._lib().vsa_norm_rope_bwd_workspace_bytes(norm_op(layer, **changes)) == 0


@pytest.mark.parametrize("changes", [
    dict(ptr=PTR + 8), dict(heads=0), dict(token_stride=132), dict(head_stride=4),
    dict(batch_stride=-128),
])
def test_norm_rope_refuses_bad_tensors(layer, changes):
    assert norm_fwd(layer, norm_op(layer), x=heads(layer, **changes)) == 1


@pytest.mark.parametrize("changes", [
    dict(heads=5), dict(token_stride=0), dict(token_stride=64), dict(head_stride=128),
    dict(batch_stride=128), dict(data=None),
])
def test_norm_rope_refuses_overlapping_or_unfit_outputs(layer, changes):
    assert norm_fwd(layer, norm_op(layer), y=heads(layer, **changes)) == 1


def test_norm_rope_bwd_refuses(layer):
    lib, op, h = layer._lib(), norm_op(layer), heads(layer)
    p = ctypes.c_void_p(PTR)
    need = lib.vsa_norm_rope_bwd_workspace_bytes(op)
    assert need > 0
    assert lib.vsa_norm_rope_bwd(op, *[None] * 8, None, None, None, 0, None) == 1      # nothing
    full = [h, None, None, h, None, h, None, None]
    assert lib.vsa_norm_rope_bwd(op, *full, p, None, None, 0, None) == 3               # workspace
    assert lib.vsa_norm_rope_bwd(op, *full, p, None, p, need - 1, None) == 3
    assert lib.vsa_norm_rope_bwd(op, *full, p, None, ctypes.c_void_p(PTR + 16), need, None) == 3
    for missing in (0, 3, 5):                                                          # dy, x, dx
        args = list(full)
        args[missing] = None
        assert lib.vsa_norm_rope_bwd(op, *args, None, None, None, 0, None) == 1
    # A weight gradient without its tensor.
    assert lib.vsa_norm_rope_bwd(op, *full, None, p, p, need, None) == 1


def cross_op(layer, **changes):
    f = dict(batch=2, heads=4, kv_heads=2, q_tokens=10, kv_tokens=20, head_dim=128, sm_scale=0.1,
             kv_len=None)
    f.update(changes)
    return layer.VsaCross(**f)


def cross_tensors(layer):
    return heads(layer), heads(layer, 2, 20), heads(layer, 2, 20), heads(layer)


@pytest.mark.parametrize("status,changes", [
    (1, dict(batch=0)), (1, dict(heads=0)), (1, dict(kv_heads=0)), (1, dict(kv_heads=3)),
    (1, dict(q_tokens=0)), (1, dict(kv_tokens=0)), (2, dict(head_dim=64)),
    (1, dict(sm_scale=math.inf)), (1, dict(sm_scale=math.nan)), (2, dict(batch=65535)),
    (2, dict(q_tokens=1 << 30)), (2, dict(kv_tokens=1 << 30)), (1, dict(kv_len=PTR + 2)),
])
def test_cross_refuses_bad_operators(layer, status, changes):
    lib, op, p = layer._lib(), cross_op(layer, **changes), ctypes.c_void_p(PTR)
    q, k, v, o = cross_tensors(layer)
    assert lib.vsa_cross_fwd(op, q, k, v, o, p, p, 1 << 40, None) == status
    assert lib.vsa_cross_bwd(op, q, q, k, v, q, p, o, k, v, p, 1 << 40, None) == status
    assert lib.vsa_cross_fwd_workspace_bytes(op) == 0
    assert lib.vsa_cross_bwd_workspace_bytes(op) == 0


def test_cross_refuses_bad_tensors(layer):
    lib, op, p = layer._lib(), cross_op(layer), ctypes.c_void_p(PTR)
    good = cross_tensors(layer)
    for i in range(4):
        for bad in (None, heads(layer, 3, 20), heads(layer, ptr=PTR + 2), heads(layer, token_stride=130)):
            args = list(good)
            args[i] = bad
            assert lib.vsa_cross_fwd(op, *args, p, p, 1 << 40, None) == 1
    assert lib.vsa_cross_fwd(op, *good, None, p, 1 << 40, None) == 1                    # lse
    for dim in ("head_stride", "token_stride"):                                          # broadcast
        assert lib.vsa_cross_fwd(op, heads(layer, **{dim: 0}), *good[1:], p, p, 1 << 40, None) == 1
    assert lib.vsa_cross_fwd(op, *good[:3], heads(layer, token_stride=0), p, p, 1 << 40, None) == 1
    q, k, v, o = good
    need = lib.vsa_cross_bwd_workspace_bytes(op)
    assert need > 0
    assert lib.vsa_cross_bwd(op, q, q, k, v, q, p, o, k, v, None, 0, None) == 3
    assert lib.vsa_cross_bwd(op, q, q, k, v, q, p, o, k, v, p, need - 1, None) == 3
    assert lib.vsa_cross_bwd(op, q, q, k, v, q, None, o, k, v, p, need, None) == 1
    assert lib.vsa_cross_bwd(op, q, q, k, v, q, p, o, None, v, p, need, None) == 1


def test_device_error_needs_a_place(layer):
    assert layer._lib().vsa_layer_device_error(None, None) == 1


def test_binding_refuses_cpu_tensors(layer):
    x = torch.zeros(1, 4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        layer.vsa_norm_rope(x)
    with pytest.raises(TypeError):
        layer.vsa_cross_fwd(x, x, x)


@pytest.mark.parametrize("grid,cube", [((21, 30, 52), (4, 4, 4)), ((1, 1, 1), (4, 4, 4)),
                                       ((5, 3, 9), (4, 4, 4)), ((6, 8, 10), (4, 4, 8)),
                                       ((2, 3, 4), (1, 1, 1))])
def test_video_token_order(layer, grid, cube):
    src, dst, vbs = (t.numpy() for t in layer.video_token_order(grid, cube, device="cpu"))
    per = int(np.prod(cube))
    assert np.array_equal(vbs, workloads.video_cube_sizes(grid, cube))
    assert dst.size == np.prod(grid) and src.size == vbs.size * per
    assert np.array_equal(src[dst], np.arange(dst.size))
    valid = np.arange(per)[None, :] < vbs[:, None]           # a cube's tokens come first
    assert np.array_equal(src.reshape(-1, per) >= 0, valid)
    pos = np.stack(np.unravel_index(np.arange(dst.size), grid), -1) // np.array(cube)
    n = -(-np.array(grid) // np.array(cube))
    assert np.array_equal(dst // per, (pos[:, 0] * n[1] + pos[:, 1]) * n[2] + pos[:, 2])


def test_video_token_order_refuses(layer):
    for grid, cube in (((4, 4), (4, 4, 4)), ((0, 4, 4), (4, 4, 4)), ((4, 4, 4), (4, 0, 4))):
        with pytest.raises(ValueError):
            layer.video_token_order(grid, cube, device="cpu")


def test_rotation_table(layer):
    pos = torch.tensor([[0, 0, 0], [1, 2, 3], [1 << 24, 1, 0]])
    cos, sin = layer.rotation_table(pos, 128, device="cpu")
    assert cos.shape == (3, 64) and cos.dtype == torch.float32
    assert torch.equal(cos[0], torch.ones(64)) and torch.equal(sin[0], torch.zeros(64))
    # 64 pairs over three axes: 22, 21, 21; pair i of n turns by position * theta^(-i / n).
    angle = [p * 10000.0 ** -(i / n) for p, n in ((1, 22), (2, 21), (3, 21)) for i in range(n)]
    assert np.abs(cos[1].numpy() - np.cos(angle)).max() <= 2.0 ** -24
    far = float(1 << 24) * 10000.0 ** -(np.arange(22) / 22)
    assert np.abs(sin[2, :22].numpy() - np.sin(far)).max() <= 2.0 ** -24 + 1e-8
    with pytest.raises(ValueError):
        layer.rotation_table(pos, 4, device="cpu")
