"""Norm + rotation and its gradient against the fp64 oracle.

Tolerances: one bf16 rounding of the result (half a step, 2^-8 relative) plus the fp32 arithmetic before it.
Forward: the mean's rsqrt (2 units of 2^-24) and at most ten roundings of products of |n| <= the row's
largest, so 16 * 2^-24 of (|a| + |b|) <= 2^-19 of the row's largest |n| is above it. Backward: dx is a
difference of r g and r xr mean(g xr), |xr| <= sqrt(d); its terms are at most r (|g| + |xr| max|g| sqrt(d)),
and a row sum of d products adds d roundings: (d + 16) 2^-24 of that. dw is a sum whose chains are joined in
fp64; each chain is at most 64 terms long at these sizes and each term has ten roundings: 80 * 2^-24 of the
sum of |terms|.
"""
import numpy as np
import pytest

import oracle.block_oracle as BO
import oracle.vsa_oracle as O
from gpu_util import bf16_to_f64, no_prefix_config, ragged_gpu_config, to_device
from vsa_synth import LayerConfig, get_config

pytestmark = pytest.mark.gpu

EPS = 1e-6


def one_token_config():
    return LayerConfig(name="one", batch=1, heads=1, head_dim=128, T=1, H=1, W=1, segments=(),
                       tile_shapes=((4, 4, 4),), score_mode="meanpool_gate", proj_dim=128, sparsity=(0.0,), seed=9)


def three_heads_config():
    """No multiple of the four rows of 64 channels that a warp takes, 105 tokens."""
    return LayerConfig(name="three", batch=1, heads=3, head_dim=64, T=3, H=5, W=7, segments=(),
                       tile_shapes=((4, 4, 4),) * 3, score_mode="meanpool_gate", proj_dim=64, sparsity=(0.0,), seed=9)


CONFIGS = {"ragged128": lambda: ragged_gpu_config(128, batch=2), "ragged64_trip": lambda: ragged_gpu_config(64, "tripool"),
           "noprefix": no_prefix_config, "tiny": lambda: get_config("tiny"), "one": one_token_config}


class Case:
    def __init__(self, cfg, layout, per_head, weights=True, table=True, strided=True, seed=0):
        import torch
        import tile_sparse_video_pack_b200 as T
        self.cfg, self.layout, self.per_head = cfg, layout, per_head
        g = torch.Generator().manual_seed(seed)
        B, N, Hh, d = self.shape = (cfg.batch, cfg.n_tokens, cfg.heads, cfg.head_dim)
        bf = lambda *s: (torch.randn(*s, generator=g) * 1.5).to(torch.bfloat16)
        if strided:                     # q, k, v: slices of one projection's output
            self.qkv = bf(B, N, 3, Hh, d).cuda()
            self.q, self.k, self.v = (self.qkv[:, :, i] for i in range(3))
        else:
            self.q, self.k, self.v = (bf(B, N, Hh, d).cuda() for _ in range(3))
        ws = (Hh, d) if per_head else (d,)
        w = [(1 + 0.3 * torch.randn(*ws, generator=g)).float() if weights else None for _ in range(2)]
        ang = BO.rope_angles(cfg.T, cfg.H, cfg.W, cfg.n_prefix_tokens, d // 2) + 0.25
        tab = [f(ang).astype(np.float32) if table else None for f in (np.cos, np.sin)]
        dev = lambda t: None if t is None else torch.as_tensor(t).cuda()
        self.norm = T.NormRope(dev(w[0]), dev(w[1]), dev(tab[0]), dev(tab[1]), layout=layout, eps=EPS)
        self.w = [np.ones(d) if t is None else t.double().numpy() for t in w]
        self.cos, self.sin = (None if t is None else t.astype(np.float64) for t in tab)
        k = [1] * Hh
        self.plan = T.Plan.from_config(cfg, 0.5, k_per_head=k)
        self.gen = g

    def oracle(self, i):
        x = bf16_to_f64((self.q, self.k)[i])
        return BO.norm_rope(x, self.w[i], self.cos, self.sin, self.layout, EPS)

    def check_forward(self, got, want):
        got = bf16_to_f64(got)
        slack = 2.0 ** -19 * np.abs(want).max(-1, keepdims=True) * np.sqrt(2)   # a rotated pair's |a| + |b|
        assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + slack)


@pytest.mark.parametrize("layout", ["interleaved", "halves"])
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("name", sorted(CONFIGS))
def test_forward(name, layout, per_head):
    import torch
    c = Case(CONFIGS[name](), layout, per_head)
    qo, ko = torch.empty(c.shape, dtype=torch.bfloat16, device="cuda"), torch.empty(c.shape, dtype=torch.bfloat16, device="cuda")
    c.plan.qk_norm_rope(c.q, c.k, c.norm, qo, ko)
    c.plan.check()
    c.check_forward(qo, c.oracle(0))
    c.check_forward(ko, c.oracle(1))
    # in place, into the projection's own buffer: the same bits, and v untouched
    v = c.v.clone()
    c.plan.qk_norm_rope(c.q, c.k, c.norm, c.q, c.k)
    c.plan.check()
    assert torch.equal(c.q, qo) and torch.equal(c.k, ko) and torch.equal(c.v, v)


@pytest.mark.parametrize("weights,table", [(False, True), (True, False), (False, False)])
def test_without_weights_or_table(weights, table):
    import torch
    c = Case(ragged_gpu_config(128), "halves", False, weights, table, strided=False)
    qo, ko = torch.empty_like(c.q), torch.empty_like(c.k)
    c.plan.qk_norm_rope(c.q, c.k, c.norm, qo, ko)
    c.plan.check()
    c.check_forward(qo, c.oracle(0))
    c.check_forward(ko, c.oracle(1))


def test_zero_and_special_rows():
    """A row of zeros stays zero; one with an infinity or a NaN is the formula's, and no other row changes."""
    import torch
    c = Case(ragged_gpu_config(64), "interleaved", False, strided=False)
    qo, ko = torch.empty_like(c.q), torch.empty_like(c.k)
    c.plan.qk_norm_rope(c.q, c.k, c.norm, qo, ko)
    base = qo.clone()
    c.q[0, 3, 1] = 0
    c.q[0, 5, 2, 7] = float("inf")
    c.q[0, 6, 0, 0] = float("nan")
    c.plan.qk_norm_rope(c.q, c.k, c.norm, qo, ko)
    c.plan.check()
    assert torch.all(qo[0, 3, 1] == 0)
    assert torch.isnan(qo[0, 6, 0]).all()
    assert torch.isnan(qo[0, 5, 2, 6:8]).any() and torch.all(qo[0, 5, 2, :6] == 0)   # x / inf = 0, inf / inf = NaN
    same = torch.ones(c.shape[:3], dtype=torch.bool, device="cuda")
    same[0, 3, 1] = same[0, 5, 2] = same[0, 6, 0] = False
    assert torch.equal(qo[same], base[same])


@pytest.mark.parametrize("layout", ["interleaved", "halves"])
@pytest.mark.parametrize("name", sorted(CONFIGS))
def test_pack_equals_forward_then_pack(name, layout):
    """The fused pass: packed tiles and descriptors bit for bit those of the two calls."""
    import torch
    c = Case(CONFIGS[name](), layout, name == "ragged128")
    p, bf = c.plan, torch.bfloat16
    qo, ko = (torch.empty(c.shape, dtype=bf, device="cuda") for _ in range(2))
    p.qk_norm_rope(c.q, c.k, c.norm, qo, ko)
    two, one = p.allocate(), p.allocate()
    for b in (two, one):
        for x in ("qp", "kp", "vp"):
            b[x].fill_(7)
        b["workspace"].zero_()
    p.tile_pack_pool(qo, ko, c.v.contiguous(), two["qp"], two["kp"], two["vp"], two["workspace"])
    p.tile_norm_rope_pack_pool(c.q, c.k, c.v, c.norm, one["qp"], one["kp"], one["vp"], one["workspace"])
    p.check()
    for x in ("qp", "kp", "vp"):
        assert torch.equal(two[x].view(torch.int16), one[x].view(torch.int16)), x
    for a, b in zip(p.pooled(two["workspace"]), p.pooled(one["workspace"])):
        assert torch.equal(a, b)
    want, n = O.pack(bf16_to_f64(qo), c.cfg)
    assert np.array_equal(bf16_to_f64(one["qp"]), want)


def test_pack_of_many_heads_per_block():
    """Enough tiles that a block works through several heads, equal and different shapes in turn."""
    import torch
    shapes = ((4, 4, 4), (4, 4, 4), (1, 8, 8), (1, 8, 8), (1, 8, 8), (16, 2, 2), (2, 4, 8), (4, 4, 4), (2, 4, 8),
              (2, 4, 8), (16, 2, 2), (4, 4, 4), (8, 4, 2))
    cfg = LayerConfig(name="many", batch=1, heads=13, head_dim=64, T=18, H=46, W=78, segments=(77, 512),
                      tile_shapes=shapes, score_mode="tripool", proj_dim=64, sparsity=(0.5,), seed=6)
    c = Case(cfg, "interleaved", True)
    p = c.plan
    qo, ko = (torch.empty(c.shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    p.qk_norm_rope(c.q, c.k, c.norm, qo, ko)
    two, one = p.allocate(), p.allocate()
    two["workspace"].zero_()
    one["workspace"].fill_(1)
    p.tile_pack_pool(qo, ko, c.v.contiguous(), two["qp"], two["kp"], two["vp"], two["workspace"])
    p.tile_norm_rope_pack_pool(c.q, c.k, c.v, c.norm, one["qp"], one["kp"], one["vp"], one["workspace"])
    p.check()
    for x in ("qp", "kp", "vp"):
        assert torch.equal(two[x].view(torch.int16), one[x].view(torch.int16)), x
    for a, b in zip(p.pooled(two["workspace"]), p.pooled(one["workspace"])):
        assert torch.equal(a, b)


def check_backward(c, i, dy, dx, dw):
    x, d = bf16_to_f64((c.q, c.k)[i]), c.shape[3]
    want, dw_want, dw_abs = BO.norm_rope_grad(dy, x, c.w[i], c.cos, c.sin, c.layout, EPS, c.per_head)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
    gmax = (np.abs(dy) * np.abs(c.w[i]).max()).max(-1, keepdims=True) * np.sqrt(2)
    slack = (d + 16) * 2.0 ** -24 * r * gmax * (1 + np.abs(x * r))
    assert np.all(np.abs(bf16_to_f64(dx) - want) <= 2.0 ** -8 * np.abs(want) + slack)
    assert np.all(np.abs(dw.double().cpu().numpy() - dw_want) <= 80 * 2.0 ** -24 * dw_abs + 2.0 ** -24 * np.abs(dw_want))


@pytest.mark.parametrize("layout", ["interleaved", "halves"])
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("name", sorted(CONFIGS))
def test_backward(name, packed, per_head, layout):
    import torch
    c = Case(CONFIGS[name](), layout, per_head)
    p, bf = c.plan, torch.bfloat16
    dy = [torch.randn(*c.shape, generator=c.gen).to(bf).cuda() for _ in range(3)]
    dw = [torch.full_like(c.norm.w_q, 9.0) for _ in range(2)]
    ws = torch.empty(p.norm_bwd_workspace_bytes(), dtype=torch.uint8, device="cuda")
    dqkv = torch.empty(c.shape[0], c.shape[1], 3, *c.shape[2:], dtype=bf, device="cuda")

    def run(out_dw):
        if packed:
            pk = [torch.empty(p.info.packed_elems, dtype=bf, device="cuda") for _ in range(3)]
            p.tile_pack(*dy, *pk)
            p.tile_norm_rope_bwd(*pk, c.q, c.k, c.norm, dqkv[:, :, 0], dqkv[:, :, 1], dqkv[:, :, 2], *out_dw, ws)
            assert torch.equal(dqkv[:, :, 2], dy[2])
        else:
            p.qk_norm_rope_bwd(dy[0], dy[1], c.q, c.k, c.norm, dqkv[:, :, 0], dqkv[:, :, 1], *out_dw, ws)
        p.check()

    run(dw)
    for i in range(2):
        check_backward(c, i, bf16_to_f64(dy[i]), dqkv[:, :, i], dw[i])
    again = [torch.empty_like(t) for t in dw]
    run(again)
    assert torch.equal(again[0], dw[0]) and torch.equal(again[1], dw[1])   # the same on every call
    run((None, None))                                                      # without the weights' gradient


def test_backward_in_place():
    import torch
    c = Case(ragged_gpu_config(128), "halves", False, strided=False)
    dy = [torch.randn(*c.shape, generator=c.gen).to(torch.bfloat16).cuda() for _ in range(2)]
    ws = torch.empty(c.plan.norm_bwd_workspace_bytes(), dtype=torch.uint8, device="cuda")
    out = [torch.empty_like(t) for t in dy]
    c.plan.qk_norm_rope_bwd(*dy, c.q, c.k, c.norm, *out, None, None, ws)
    c.plan.qk_norm_rope_bwd(*dy, c.q, c.k, c.norm, *dy, None, None, ws)
    c.plan.check()
    assert torch.equal(out[0], dy[0]) and torch.equal(out[1], dy[1])


def test_refusals():
    import torch
    import tile_sparse_video_pack_b200 as T
    c = Case(ragged_gpu_config(128), "halves", False, strided=False)
    p, n = c.plan, c.norm
    qo, ko = torch.empty_like(c.q), torch.empty_like(c.k)
    with pytest.raises(TypeError):
        p.qk_norm_rope(c.q.float(), c.k, n, qo, ko)
    with pytest.raises(TypeError):
        p.qk_norm_rope(c.q.cpu(), c.k, n, qo, ko)
    with pytest.raises(ValueError):
        p.qk_norm_rope(c.q[:, :-1], c.k, n, qo, ko)
    with pytest.raises(ValueError):
        p.qk_norm_rope(c.q.transpose(2, 3), c.k, n, qo, ko)
    with pytest.raises(ValueError):
        p.qk_norm_rope(c.q, c.k, T.NormRope(n.w_q[:64], n.w_k[:64]), qo, ko)
    with pytest.raises(ValueError):
        p.qk_norm_rope(c.q, c.k, T.NormRope(cos=n.cos[:-1], sin=n.sin[:-1]), qo, ko)
    with pytest.raises(ValueError):
        p.tile_norm_rope_pack_pool(c.q, c.k, c.v, n, qo, ko, qo, torch.empty(16, dtype=torch.uint8, device="cuda"))
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(T.VsaError):
            p.qk_norm_rope(c.q, c.k, T.NormRope(eps=eps), qo, ko)
    # a base address off by one element
    flat = torch.empty(c.q.numel() + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(T.VsaError):
        p.qk_norm_rope(flat[1:1 + c.q.numel()].view(c.shape), c.k, n, qo, ko)
    # a token stride that is no multiple of eight
    wide = torch.empty(c.shape[0], c.shape[1], c.shape[2] * c.shape[3] + 4, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(T.VsaError):
        p.qk_norm_rope(wide[..., :-4].unflatten(2, c.shape[2:]), c.k, n, qo, ko)
    p.check()


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_backward_without_epsilon(packed, per_head, monkeypatch):
    """Lanes without a row (an odd head count, the last tokens) hold zeros, whose norm has no value with eps 0: they
    add nothing to dw."""
    import sys
    import torch
    monkeypatch.setattr(sys.modules[__name__], "EPS", 0.0)
    c = Case(three_heads_config(), "halves", per_head)
    p, bf = c.plan, torch.bfloat16
    dy = [torch.randn(*c.shape, generator=c.gen).to(bf).cuda() for _ in range(3)]
    dw = [torch.empty_like(c.norm.w_q) for _ in range(2)]
    ws = torch.empty(p.norm_bwd_workspace_bytes(), dtype=torch.uint8, device="cuda")
    dq, dk, dv = (torch.empty(c.shape, dtype=bf, device="cuda") for _ in range(3))
    if packed:
        pk = [torch.empty(p.info.packed_elems, dtype=bf, device="cuda") for _ in range(3)]
        p.tile_pack(*dy, *pk)
        p.tile_norm_rope_bwd(*pk, c.q, c.k, c.norm, dq, dk, dv, *dw, ws)
    else:
        p.qk_norm_rope_bwd(dy[0], dy[1], c.q, c.k, c.norm, dq, dk, *dw, ws)
    p.check()
    for i, dx in enumerate((dq, dk)):
        check_backward(c, i, bf16_to_f64(dy[i]), dx, dw[i])


def test_packed_backward_in_place():
    import torch
    c = Case(ragged_gpu_config(128, batch=2), "interleaved", False, strided=False)
    p, bf = c.plan, torch.bfloat16
    pk = [torch.empty(p.info.packed_elems, dtype=bf, device="cuda") for _ in range(3)]
    p.tile_pack(*(torch.randn(*c.shape, generator=c.gen).to(bf).cuda() for _ in range(3)), *pk)
    ws = torch.empty(p.norm_bwd_workspace_bytes(), dtype=torch.uint8, device="cuda")
    out = [torch.empty(c.shape, dtype=bf, device="cuda") for _ in range(3)]
    p.tile_norm_rope_bwd(*pk, c.q, c.k, c.norm, *out, None, None, ws)
    p.tile_norm_rope_bwd(*pk, c.q, c.k, c.norm, c.q, c.k, c.v, None, None, ws)
    p.check()
    assert all(torch.equal(a, b) for a, b in zip(out, (c.q, c.k, c.v)))


def test_batches_inside_tokens_and_shared_inputs():
    """[N, B, heads, d] outputs are taken, inputs may be one batch for all, outputs that overlap are refused."""
    import torch
    import tile_sparse_video_pack_b200 as T
    c = Case(ragged_gpu_config(128, batch=2), "halves", False, strided=False)
    p, (B, N, Hh, d) = c.plan, c.shape
    new = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
    qo, ko = new(*c.shape), new(*c.shape)
    p.qk_norm_rope(c.q, c.k, c.norm, qo, ko)
    qt, kt = (new(N, B, Hh, d).transpose(0, 1) for _ in range(2))
    p.qk_norm_rope(c.q, c.k, c.norm, qt, kt)
    assert torch.equal(qt, qo) and torch.equal(kt, ko)
    one = c.q[:1].expand(B, N, Hh, d)
    p.qk_norm_rope(one, one, c.norm, qt, kt)
    assert torch.equal(qt[0], qo[0]) and torch.equal(qt[1], qo[0])
    ws = torch.empty(p.norm_bwd_workspace_bytes(), dtype=torch.uint8, device="cuda")
    shared = new(1, N, Hh, d).expand(B, N, Hh, d)
    with pytest.raises(T.VsaError):
        p.qk_norm_rope(c.q, c.k, c.norm, shared, ko)
    with pytest.raises(T.VsaError):
        p.qk_norm_rope(c.q, c.k, c.norm, qo, new(N * B + 1, Hh, d)[:N + 1].as_strided(c.shape, (Hh * d, Hh * d, d, 1)))
    with pytest.raises(T.VsaError):
        p.qk_norm_rope_bwd(qo, ko, c.q, c.k, c.norm, qt, shared, None, None, ws)
    pk = [torch.empty(p.info.packed_elems, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    with pytest.raises(T.VsaError):
        p.tile_norm_rope_bwd(*pk, c.q, c.k, c.norm, qt, kt, shared, None, None, ws)
    p.check()
