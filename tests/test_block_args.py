"""The block operators without a GPU: include/vsa_block.h's symbols, its refusals (made on the host
before anything touches the device) and the binding's refusals."""
import ctypes
import math
import os
import re

import pytest
import torch

from block_sparse_video_tok_gb300 import build as vsa_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PTR = 0x100000
C = 64


@pytest.fixture(scope="module")
def block():
    vsa_build.build()
    from block_sparse_video_tok_gb300 import block as binding
    return binding


def test_every_declared_symbol_is_exported(block):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "vsa_block.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(vsa_[a-z_]+)\s*\(", text)))
    assert len(names) == 7 and sorted(block.SIGNATURES) == names
    for name in names:
        assert hasattr(block._lib(), name), name


def test_packed_structures_have_the_header_s_layout(block):
    for pack, type_, values in (
            (block._pack_tokens, block.VsaTokens, 3), (block._pack_norm, block.VsaGateNorm, 23),
            (block._pack_grads, block.VsaGateNormGrads, 6), (block._pack_matrix, block.VsaMatrix, 2),
            (block._pack_linear, block.VsaLinear, 9)):
        assert len(pack(*range(values))) == ctypes.sizeof(type_)
    op = block.VsaGateNorm.from_buffer_copy(block._pack_norm(*range(23)))
    assert (op.batch, op.weight_dtype, op.post_eps, op.gate.data, op.shift.group_stride, op.bias) == (0, 8, 10.0, 11, 19, 22)
    op = block.VsaLinear.from_buffer_copy(block._pack_linear(*range(9)))
    assert (op.rows, op.act, op.weight.data, op.weight.row_stride, op.bias) == (0, 5, 6, 7, 8)


# ------------------------------------------------------------------------------- gate_norm

def norm_op(block, **changes):
    mod = block.VsaModulation(PTR, 6 * C, 6 * C)
    f = dict(batch=2, tokens=12, channels=C, groups=1, kind=0, dtype=0, branch_dtype=0, mod_dtype=0,
             weight_dtype=0, eps=1e-6, post_eps=1e-6, gate=mod, scale=mod, shift=mod, post_weight=PTR,
             weight=PTR, bias=PTR)
    f.update(changes)
    return block.VsaGateNorm(**f)


def tokens(block, **changes):
    f = dict(data=PTR, batch_stride=12 * C, token_stride=C)
    f.update(changes)
    return block.VsaTokens(**f)


BAD_NORM = [
    (1, dict(batch=0)), (1, dict(tokens=0)), (1, dict(groups=0)), (1, dict(groups=5)),
    (2, dict(channels=0)), (2, dict(channels=60)), (2, dict(channels=8200)), (2, dict(kind=2)),
    (2, dict(dtype=3)), (2, dict(branch_dtype=1)), (2, dict(branch_dtype=2)), (2, dict(mod_dtype=1)),
    (2, dict(weight_dtype=1)), (2, dict(dtype=2, branch_dtype=0, mod_dtype=1)),
    (1, dict(eps=math.nan)), (1, dict(eps=-1.0)), (1, dict(post_eps=math.inf)),
    (1, dict(post_weight=PTR + 8)), (1, dict(weight=PTR + 4)), (1, dict(bias=PTR + 2)),
    (2, dict(tokens=1 << 30)),
]


@pytest.mark.parametrize("status,changes", BAD_NORM)
def test_gate_norm_refuses_bad_operators(block, status, changes):
    lib, op, t = block._lib(), norm_op(block, **changes), tokens(block)
    assert lib.vsa_gate_norm_fwd(op, t, t, t, t, None) == status
    assert lib.vsa_gate_norm_bwd(op, t, t, t, t, t, t, None, None, 0, None) == status
    assert lib.vsa_gate_norm_bwd_workspace_bytes(op) == 0


@pytest.mark.parametrize("name", ["gate", "scale", "shift"])
def test_gate_norm_refuses_bad_modulations(block, name):
    lib, t = block._lib(), tokens(block)
    for changes in (dict(data=PTR + 2), dict(batch_stride=-C), dict(batch_stride=C + 4), dict(group_stride=C + 1)):
        mod = block.VsaModulation(**{**dict(data=PTR, batch_stride=C, group_stride=C), **changes})
        assert lib.vsa_gate_norm_fwd(norm_op(block, groups=2, **{name: mod}), t, t, t, t, None) == 1
    none = block.VsaModulation(None, 0, 0)
    bare = norm_op(block, groups=2, gate=none, scale=none, shift=none)
    assert lib.vsa_gate_norm_fwd(bare, t, t, t, t, None) == 1                 # groups of nothing


def test_gate_norm_refuses_bad_tensors(block):
    lib, op, t = block._lib(), norm_op(block), tokens(block)
    bad = [None, tokens(block, data=None), tokens(block, data=PTR + 8), tokens(block, batch_stride=-C),
           tokens(block, token_stride=C + 4)]
    overlapping = [tokens(block, token_stride=0), tokens(block, token_stride=C // 2), tokens(block, batch_stride=C),
                   tokens(block, batch_stride=0), tokens(block, batch_stride=C, token_stride=C)]
    for i in range(4):                                                        # x, y, x_out, h
        for x in bad + (overlapping if i >= 2 else []):
            args = [t] * 4
            args[i] = x
            assert lib.vsa_gate_norm_fwd(op, *args, None) == 1, i
    for i in (0, 2, 3, 4, 5):                                                 # dh, x_out, y, dx, dy
        for x in bad + (overlapping if i >= 4 else []):
            args = [t] * 6
            args[i] = x
            assert lib.vsa_gate_norm_bwd(op, *args, None, None, 0, None) == 1, i
    for x in bad[2:]:                                                         # dx_out may be absent
        assert lib.vsa_gate_norm_bwd(op, t, x, t, t, t, t, None, None, 0, None) == 1
    # A gate or a post norm without y.
    none = block.VsaModulation(None, 0, 0)
    for o in (norm_op(block, post_weight=None), norm_op(block, gate=none)):
        assert lib.vsa_gate_norm_fwd(o, t, None, None, t, None) == 1
        assert lib.vsa_gate_norm_bwd(o, t, t, t, None, t, None, None, None, 0, None) == 1


def test_gate_norm_bwd_refuses_bad_places(block):
    lib, t = block._lib(), tokens(block)
    p = ctypes.c_void_p(PTR)
    op = norm_op(block)
    need = lib.vsa_gate_norm_bwd_workspace_bytes(op)
    assert need > 0
    fields = ("gate", "scale", "shift", "post_weight", "weight", "bias")
    for name in fields:
        grads = block.VsaGateNormGrads(**{name: PTR})
        for ws, n in ((None, 0), (p, need - 1), (ctypes.c_void_p(PTR + 16), need)):
            assert lib.vsa_gate_norm_bwd(op, t, t, t, t, t, t, grads, ws, n, None) == 3
        grads = block.VsaGateNormGrads(**{name: PTR + 4})
        assert lib.vsa_gate_norm_bwd(op, t, t, t, t, t, t, grads, p, need, None) == 1
        # The gradient of a parameter that is absent.
        none = block.VsaModulation(None, 0, 0) if name in fields[:3] else None
        grads = block.VsaGateNormGrads(**{name: PTR})
        assert lib.vsa_gate_norm_bwd(norm_op(block, **{name: none}), t, t, t, t, t, t, grads, p, need, None) == 1


# ------------------------------------------------------------------------------- linear

def linear_op(block, **changes):
    f = dict(rows=40, in_features=64, out_features=48, dtype=0, bias_dtype=0, act=0,
             weight=block.VsaMatrix(PTR, 64), bias=PTR)
    f.update(changes)
    return block.VsaLinear(**f)


def matrices(block):
    return block.VsaMatrix(PTR, 64), block.VsaMatrix(PTR, 48)


@pytest.mark.parametrize("status,changes", [
    (1, dict(rows=0)), (2, dict(rows=(1 << 30) + 1)), (2, dict(rows=1 << 30, out_features=1 << 20)),
    (2, dict(in_features=1 << 23, out_features=1 << 23)), (2, dict(in_features=0)), (2, dict(in_features=60)),
    (2, dict(out_features=4)), (2, dict(out_features=1 << 25)), (2, dict(dtype=2)), (2, dict(bias_dtype=1)),
    (2, dict(act=4)), (2, dict(act=-1)), (1, dict(bias=PTR + 4)), (1, dict(weight=(None, 64))),
    (1, dict(weight=(PTR + 2, 64))), (1, dict(weight=(PTR, 56))), (1, dict(weight=(PTR, 68))), (1, dict(weight=(PTR, -64))),
])
def test_linear_refuses_bad_operators(block, status, changes):
    if "weight" in changes:
        changes = dict(weight=block.VsaMatrix(*changes["weight"]))
    lib, op, p = block._lib(), linear_op(block, **changes), ctypes.c_void_p(PTR)
    x, o = matrices(block)
    assert lib.vsa_linear_fwd(op, x, None, o, None, p, 1 << 40, None) == status
    assert lib.vsa_linear_bwd(op, 0, o, x, None, None, x, None, None, p, 1 << 40, None) == status
    assert lib.vsa_linear_fwd_workspace_bytes(op) == 0 and lib.vsa_linear_bwd_workspace_bytes(op) == 0


def test_linear_refuses_bad_matrices(block):
    lib, p = block._lib(), ctypes.c_void_p(PTR)
    x, o = matrices(block)

    def bad(columns):
        return [block.VsaMatrix(*a) for a in ((PTR + 8, columns), (PTR, columns - 8), (PTR, columns + 4), (PTR, 0))]

    op = linear_op(block)
    for i, columns in ((0, 64), (1, 48), (2, 48), (3, 48)):                   # x, residual, out, pre
        for m in bad(columns) + ([None] if i in (0, 2) else []):
            args = [x, o, o, o]
            args[i] = m
            assert lib.vsa_linear_fwd(op, *args, p, 1 << 40, None) == 1, i
    op = linear_op(block, act=2)
    good = [o, x, o, x, x, block.VsaMatrix(PTR, 64)]                          # dout, x, pre, x_pre, dx, dweight
    for i, columns in enumerate((48, 64, 48, 64, 64, 64)):
        for m in bad(columns) + ([None] if i < 4 else []):
            args = list(good)
            args[i] = m
            assert lib.vsa_linear_bwd(op, 3, *args, p, p, 1 << 40, None) == 1, i
    assert lib.vsa_linear_bwd(op, 4, *good, p, p, 1 << 40, None) == 2
    assert lib.vsa_linear_bwd(op, 3, *good, ctypes.c_void_p(PTR + 4), p, 1 << 40, None) == 1
    assert lib.vsa_linear_bwd(op, 0, *good, p, p, 1 << 40, None) == 1         # x_pre without x_act
    assert lib.vsa_linear_bwd(linear_op(block), 3, *good, p, p, 1 << 40, None) == 1   # pre without act
    assert lib.vsa_linear_bwd(op, 3, *good[:4], None, None, None, p, 1 << 40, None) == 1  # nothing wanted


def test_linear_refuses_a_workspace_that_is_too_small(block):
    lib, p = block._lib(), ctypes.c_void_p(PTR)
    op = linear_op(block, rows=512, in_features=8192, out_features=1536, act=1, weight=block.VsaMatrix(PTR, 8192))
    x, o = block.VsaMatrix(PTR, 8192), block.VsaMatrix(PTR, 1536)
    need = lib.vsa_linear_fwd_workspace_bytes(op)                             # (0 without a GPU to plan for)
    for ws, n in () if need == 0 else ((None, 0), (p, need - 1), (ctypes.c_void_p(PTR + 16), need)):
        assert lib.vsa_linear_fwd(op, x, None, o, None, ws, n, None) == 3
    need = lib.vsa_linear_bwd_workspace_bytes(op)
    assert need >= 512 * 1536 * 2                                             # dz
    for ws, n in ((None, 0), (p, need - 1), (ctypes.c_void_p(PTR + 16), need)):
        assert lib.vsa_linear_bwd(op, 0, o, x, o, None, x, None, None, ws, n, None) == 3


# ------------------------------------------------------------------------------- binding

def test_binding_refuses_cpu_tensors(block):
    x = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, 64, dtype=torch.bfloat16)
    for call in (lambda: block.vsa_gate_norm(x), lambda: block.vsa_gate_norm_bwd(x, None, x),
                 lambda: block.vsa_linear(x, w), lambda: block.vsa_linear_bwd(x, x, w)):
        with pytest.raises(TypeError):
            call()


def test_mlp_needs_an_activation(block):
    from block_sparse_video_tok_gb300.autograd import mlp
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mlp(x, x, None, x, None, act=None)


def test_gate_norm_bwd_workspace_is_what_is_used(block):
    """A modulation for every token: its gradients need none, the weights' do; a long row's need some either way."""
    lib = block._lib()
    none = dict(post_weight=None, weight=None, bias=None)
    for dtype, branch in ((0, 0), (1, 1), (2, 0), (2, 2)):
        f = dict(dtype=dtype, branch_dtype=branch, mod_dtype=branch, weight_dtype=branch, batch=1, tokens=131040,
                 channels=1536)
        token, row = norm_op(block, groups=131040, **f, **none), norm_op(block, groups=1, **f, **none)
        assert lib.vsa_gate_norm_bwd_workspace_bytes(token) == 0
        assert lib.vsa_gate_norm_bwd_workspace_bytes(row) > 0
        for name in none:
            need = lib.vsa_gate_norm_bwd_workspace_bytes(norm_op(block, groups=131040, **f, **{**none, name: PTR}))
            assert 131040 * 1536 * 12 < need <= 131040 * 1536 * 12 * 17 // 16 + 1536 * 12 * 1024
    bare = block.VsaModulation(None, 0, 0)
    assert lib.vsa_gate_norm_bwd_workspace_bytes(norm_op(block, gate=bare, scale=bare, shift=bare, **none)) == 0
    # The weights are there but only a modulation's gradient is wanted: the size says so without them, and the
    # call asks for it where it is not zero.
    t = tokens(block, token_stride=1536, batch_stride=0)
    op = norm_op(block, batch=1, tokens=5000, channels=1536, groups=1)
    need = lib.vsa_gate_norm_bwd_workspace_bytes(op)
    grads = block.VsaGateNormGrads(gate=PTR)
    assert need > 0 and lib.vsa_gate_norm_bwd(op, t, t, t, t, t, t, grads, ctypes.c_void_p(PTR), need - 1, None) == 3
