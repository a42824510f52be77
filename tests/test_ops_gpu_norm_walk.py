"""Norm + rotation and its gradient where a warp walks through many tokens: rows requested ahead across tokens and
batches, several rounds of blocks, sums of dw over tokens.

Tolerances as in test_ops_gpu_norm_rope.py; before fp64 takes over, a chain of dw here has at most 81 tokens (with
weights per head; the others are shorter), two levels of lane groups and eight warps, and each term ten roundings:
101 * 2^-24 of the sum of |terms|.
"""
import numpy as np
import pytest

import oracle.block_oracle as BO
from gpu_util import bf16_to_f64
from test_ops_gpu_norm_rope import EPS, Case
from vsa_synth import LayerConfig

pytestmark = pytest.mark.gpu


def config(batch, heads, d, grid, segments=(77,)):
    T, H, W = grid
    shapes = ((4, 4, 4), (2, 4, 8), (1, 8, 8), (16, 2, 2), (4, 4, 4))
    return LayerConfig(name="walk", batch=batch, heads=heads, head_dim=d, T=T, H=H, W=W, segments=segments,
                       tile_shapes=tuple(shapes[i % 5] for i in range(heads)), score_mode="meanpool_gate", proj_dim=d,
                       sparsity=(0.5,), seed=5)


CONFIGS = {"three batches, d 64": lambda: config(3, 3, 64, (11, 19, 29)),     # 6,138 tokens each: eight to a warp
           "three batches, d 128": lambda: config(3, 5, 128, (11, 19, 29)),
           "one batch": lambda: config(1, 2, 128, (9, 31, 33), ()),           # 9,207 tokens
           "short batches": lambda: config(3001, 1, 64, (3, 3, 3), ()),       # a step passes over hundreds of batches
           "rounds": lambda: config(3, 5, 64, (31, 40, 41))}                  # packed: two rounds of blocks


def check_backward(c, i, dy, dx, dw):
    d = c.shape[3]
    x = bf16_to_f64((c.q, c.k)[i])
    want, dw_want, dw_abs = BO.norm_rope_grad(dy, x, c.w[i], c.cos, c.sin, c.layout, EPS, c.per_head)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
    gmax = (np.abs(dy) * np.abs(c.w[i]).max()).max(-1, keepdims=True) * np.sqrt(2)
    slack = (d + 16) * 2.0 ** -24 * r * gmax * (1 + np.abs(x * r))
    assert np.all(np.abs(bf16_to_f64(dx) - want) <= 2.0 ** -8 * np.abs(want) + slack)
    assert np.all(np.abs(dw.double().cpu().numpy() - dw_want) <= 101 * 2.0 ** -24 * dw_abs + 2.0 ** -24 * np.abs(dw_want))


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("name", sorted(CONFIGS))
def test_backward(name, packed, per_head):
    import torch
    c = Case(CONFIGS[name](), "halves" if packed else "interleaved", per_head)
    p, bf = c.plan, torch.bfloat16
    dy = [torch.randn(*c.shape, generator=c.gen).to(bf).cuda() for _ in range(3 if packed else 2)]
    dw = [torch.full_like(c.norm.w_q, 9.0) for _ in range(2)]
    ws = torch.empty(p.norm_bwd_workspace_bytes(), dtype=torch.uint8, device="cuda")
    if name == "rounds":     # the partial sums of two rounds of two blocks per SM
        assert ws.numel() == 4 * torch.cuda.get_device_properties(0).multi_processor_count * 2 * 64 * 4
    dqkv = torch.full((c.shape[0], c.shape[1], 3, *c.shape[2:]), 7.0, dtype=bf, device="cuda")
    pk = [torch.empty(p.info.packed_elems, dtype=bf, device="cuda") for _ in range(3)]

    def run(out_dw):
        if packed:
            p.tile_norm_rope_bwd(*pk, c.q, c.k, c.norm, dqkv[:, :, 0], dqkv[:, :, 1], dqkv[:, :, 2], *out_dw, ws)
        else:
            p.qk_norm_rope_bwd(dy[0], dy[1], c.q, c.k, c.norm, dqkv[:, :, 0], dqkv[:, :, 1], *out_dw, ws)
        p.check()

    if packed:
        p.tile_pack(*dy, *pk)
    run(dw)
    for i in range(2):
        check_backward(c, i, bf16_to_f64(dy[i]), dqkv[:, :, i], dw[i])
    assert torch.equal(dqkv[:, :, 2], dy[2]) if packed else torch.all(dqkv[:, :, 2] == 7)
    again = [torch.empty_like(t) for t in dw]
    first = dqkv.clone()
    run(again)
    assert torch.equal(again[0], dw[0]) and torch.equal(again[1], dw[1]) and torch.equal(first, dqkv)


@pytest.mark.parametrize("layout", ["interleaved", "halves"])
@pytest.mark.parametrize("name", ["rounds", "short batches"])
def test_forward(name, layout):
    """More tokens over the batch than warps in all rounds (16 x 3 x 8 to an SM)."""
    import torch
    c = Case(CONFIGS[name](), layout, True)
    assert c.shape[0] * c.shape[1] > torch.cuda.get_device_properties(0).multi_processor_count * 16 * 3 * 8
    qo, ko = (torch.full(c.shape, 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c.plan.qk_norm_rope(c.q, c.k, c.norm, qo, ko)
    c.plan.check()
    for i, got in enumerate((qo, ko)):
        c.check_forward(got, c.oracle(i))
    c.plan.qk_norm_rope(c.q, c.k, c.norm, c.q, c.k)       # in place
    c.plan.check()
    assert torch.equal(c.q, qo) and torch.equal(c.k, ko)
