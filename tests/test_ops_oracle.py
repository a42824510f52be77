"""Pins of oracle/block_oracle.py (CPU): every gradient against central differences of its forward, the
forwards against torch in fp64, and planted mistakes that the pins catch."""
import numpy as np
import pytest
import torch

import oracle.block_oracle as BO
import oracle.vsa_oracle as O
from vsa_synth import LayerConfig

RNG = np.random.default_rng


def numeric_grad(f, x, dy, n=12, eps=1e-5, seed=0):
    """Central differences of <f(x), dy> at n random entries of x: (index, value) pairs."""
    rng = RNG(seed)
    out = []
    for flat in rng.choice(x.size, size=min(n, x.size), replace=False):
        at = np.unravel_index(flat, x.shape)
        a, b = x.copy(), x.copy()
        a[at] += eps
        b[at] -= eps
        out.append((at, float(((f(a) - f(b)) * dy).sum() / (2 * eps))))
    return out


def assert_grad(grad, pairs, tol=1e-6):
    scale = np.abs(grad).max()
    for at, want in pairs:
        assert abs(grad[at] - want) <= tol * max(scale, 1.0), (at, grad[at], want)


@pytest.mark.parametrize("layout", ["interleaved", "halves"])
@pytest.mark.parametrize("per_head", [False, True])
def test_norm_rope_and_gradient(layout, per_head):
    rng = RNG(1)
    B, N, Hh, d = 2, 5, 3, 64
    x, dy = rng.normal(size=(B, N, Hh, d)), rng.normal(size=(B, N, Hh, d))
    w = 1 + 0.3 * rng.normal(size=(Hh, d) if per_head else d)
    ang = rng.uniform(-3, 3, size=(N, d // 2))
    cos, sin = np.cos(ang), np.sin(ang)
    y = BO.norm_rope(x, w, cos, sin, layout, 1e-6)
    # the same through complex numbers
    n = torch.tensor(x) * torch.rsqrt(torch.tensor(x).square().mean(-1, keepdim=True) + 1e-6) * torch.tensor(w)
    a, b = (n[..., :d // 2], n[..., d // 2:]) if layout == "halves" else (n[..., 0::2], n[..., 1::2])
    z = torch.complex(a, b) * torch.polar(torch.ones(N, d // 2, dtype=torch.float64), torch.tensor(ang))[None, :, None]
    want = torch.cat([z.real, z.imag], -1) if layout == "halves" else torch.stack([z.real, z.imag], -1).flatten(-2)
    assert np.abs(y - want.numpy()).max() < 1e-12
    dx, dw, _ = BO.norm_rope_grad(dy, x, w, cos, sin, layout, 1e-6, per_head)
    f = lambda t: BO.norm_rope(t, w, cos, sin, layout, 1e-6)
    assert_grad(dx, numeric_grad(f, x, dy))
    assert_grad(dw, numeric_grad(lambda t: BO.norm_rope(x, t, cos, sin, layout, 1e-6), w, dy))
    # planted: rotating the gradient forward instead of back is caught by the differences
    wrong = BO.norm_rope_grad(BO.rotate(BO.rotate(dy, cos, sin, layout), cos, sin, layout), x, w, cos, sin, layout,
                              1e-6, per_head)[0]
    with pytest.raises(AssertionError):
        assert_grad(wrong, numeric_grad(f, x, dy))


@pytest.mark.parametrize("act", ["none", "gelu_tanh", "silu"])
def test_linear_and_gradient(act):
    rng = RNG(2)
    x, w, bias = rng.normal(size=(6, 8)), rng.normal(size=(16, 8)), rng.normal(size=16)
    gate, res, dy = rng.normal(size=(2, 16)), rng.normal(size=(6, 16)), rng.normal(size=(6, 16))
    y, z = BO.linear(x, w, bias, act, gate, res)
    tz = torch.tensor(x) @ torch.tensor(w).T + torch.tensor(bias)
    ta = {"none": lambda t: t, "silu": torch.nn.functional.silu,
          "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[act](tz)
    want = torch.tensor(res) + ta * torch.tensor(gate).repeat_interleave(3, 0)
    assert np.abs(y - want.numpy()).max() < 1e-12
    g = BO.linear_grad(dy, x, w, act, z, gate)
    assert_grad(g["dx"], numeric_grad(lambda t: BO.linear(t, w, bias, act, gate, res)[0], x, dy))
    assert_grad(g["dw"], numeric_grad(lambda t: BO.linear(x, t, bias, act, gate, res)[0], w, dy))
    assert_grad(g["dbias"], numeric_grad(lambda t: BO.linear(x, w, t, act, gate, res)[0], bias, dy))
    assert_grad(g["dgate"], numeric_grad(lambda t: BO.linear(x, w, bias, act, t, res)[0], gate, dy))


def tiny_cfg(**kw):
    base = dict(name="t", batch=1, heads=2, head_dim=64, T=2, H=5, W=9, segments=(70,), seed=1,
                tile_shapes=((4, 4, 4), (1, 8, 8)), score_mode="meanpool_gate", proj_dim=64, sparsity=(0.5,))
    return LayerConfig(**{**base, **kw})


def test_attention_gradient_by_differences_and_autograd():
    cfg = tiny_cfg()
    rng = RNG(3)
    shape = (1, cfg.n_tokens, 2, 64)
    q, k, v, do = (rng.normal(size=shape) for _ in range(4))
    kept = [[[sorted(rng.choice(len(O.head_tiling(cfg, h).video), size=2, replace=False))
              for _ in O.head_tiling(cfg, h).video] for h in range(2)]]
    dq, dk, dv, lse, o, bq, bk, bv = BO.attention_grad(cfg, q, k, v, do, kept, bound=True)[:8]
    for h in range(2):                       # autograd of a masked softmax, fp64
        til = O.head_tiling(cfg, h)
        allowed = np.zeros((cfg.n_tokens, cfg.n_tokens), dtype=bool)
        for n, rows in enumerate(til.all):
            i = n - til.n_prefix
            allowed[np.ix_(rows, O.query_key_tokens(til, n, [] if i < 0 else kept[0][h][i]))] = True
        t = [torch.tensor(a[0, :, h], requires_grad=True) for a in (q, k, v)]
        s = (t[0] @ t[1].T / 8).masked_fill(~torch.tensor(allowed), -torch.inf)
        out = torch.softmax(s, 1) @ t[2]
        out.backward(torch.tensor(do[0, :, h]))
        assert np.abs(out.detach().numpy() - o[0, :, h]).max() < 1e-12
        assert np.abs(torch.logsumexp(s, 1).detach().numpy() - lse[0, :, h]).max() < 1e-12
        for got, x in zip((dq, dk, dv), t):
            assert np.abs(got[0, :, h] - x.grad.numpy()).max() < 1e-12
    f = lambda a, b, c: BO.attention_grad(cfg, a, b, c, do, kept)[4]
    assert_grad(dq, numeric_grad(lambda t: f(t, k, v), q, do, n=3), 1e-5)
    assert_grad(dk, numeric_grad(lambda t: f(q, t, v), k, do, n=3), 1e-5)
    assert_grad(dv, numeric_grad(lambda t: f(q, k, t), v, do, n=3), 1e-5)
    for g, b in ((dq, bq), (dk, bk), (dv, bv)):
        assert np.all(np.abs(g) <= b * (1 + 1e-9))
    # planted: a query tile's list moved by one tile changes dk
    shifted = [[[[(j + 1) % len(O.head_tiling(cfg, h).video) for j in row] for row in kept[0][h]] for h in range(2)]]
    assert np.abs(BO.attention_grad(cfg, q, k, v, do, shifted)[1] - dk).max() > 1e-3


def test_rope_angles_axes():
    a = BO.rope_angles(2, 3, 4, 5, 32)
    assert a.shape == (5 + 24, 32) and np.all(a[:5] == 0)
    last = a[5 + (1 * 3 + 2) * 4 + 3]
    assert last[0] == 1 and last[12] == 2 and last[22] == 3      # split 12, 10, 10: pair 0 of an axis turns by its position
    assert np.isclose(last[13], 2 * 10000.0 ** (-1 / 10))
