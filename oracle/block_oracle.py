"""The operators around the attention layer and their gradients, in plain fp64 numpy.

Slow and direct: each function follows its formula with loops over heads and tiles where that is the
plainest form, and shares no code with the CUDA path. Next to a gradient, ``bound=True`` returns the same
sum over absolute values, which is what a rounding of each term can move the result by at most.
"""
from __future__ import annotations

import numpy as np

from .vsa_oracle import head_tiling, query_key_tokens


def rope_angles(T, H, W, n_prefix, half, theta=10000.0, split=None):
    """Angle of every token (prefix first, unrotated) and channel pair: the pairs are divided among t, h
    and w, and pair j of an axis with n pairs turns by position * theta^(-j/n)."""
    split = split or (half - 2 * (half // 3), half // 3, half // 3)
    out = np.zeros((n_prefix + T * H * W, half))
    i = n_prefix
    for t in range(T):
        for h in range(H):
            for w in range(W):
                out[i] = np.concatenate([p * theta ** (-np.arange(n) / n) for p, n in zip((t, h, w), split) if n])
                i += 1
    return out


def _pairs(d, layout):
    """Channels (first, second) of every rotation pair."""
    i = np.arange(d // 2)
    return (i, i + d // 2) if layout == "halves" else (2 * i, 2 * i + 1)


def rotate(x, cos, sin, layout, back=False):
    """x [B, N, heads, d], tables [N, d / 2]: every channel pair turned by the token's angle (back: by minus it)."""
    a, b = _pairs(x.shape[-1], layout)
    c, s = cos[None, :, None], (-sin if back else sin)[None, :, None]
    out = np.empty_like(x)
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., a] * s + x[..., b] * c
    return out


def norm_rope(x, w, cos, sin, layout, eps):
    x = np.asarray(x, dtype=np.float64)
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return n if cos is None else rotate(n, cos, sin, layout)


def norm_rope_grad(dy, x, w, cos, sin, layout, eps, per_head):
    """(dx, dw, sum of |terms| of dw)."""
    x, dy = np.asarray(x, dtype=np.float64), np.asarray(dy, dtype=np.float64)
    dn = dy if cos is None else rotate(dy, cos, sin, layout, back=True)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    axes = (0, 1) if per_head else (0, 1, 2)
    dw = (dn * x * r).sum(axes)
    g = dn * w
    dx = r * g - x * r ** 3 * (g * x).mean(-1, keepdims=True)
    return dx, dw, np.abs(dn * x * r).sum(axes)


def act(z, name):
    if name == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z / (1 + np.exp(-z))
    return z


def act_grad(z, name):
    if name == "gelu_tanh":
        t = np.tanh(np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * np.sqrt(2 / np.pi) * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = 1 / (1 + np.exp(-z))
        return s + z * s * (1 - s)
    return np.ones_like(z)


def linear(x, w, bias=None, act_name="none", gate=None, residual=None):
    """(y, z): y = residual + gate[sample] * act(z), z = x w^T + bias."""
    z = x @ w.T + (0 if bias is None else bias)
    y = act(z, act_name)
    if gate is not None:
        y = y * np.repeat(gate, len(x) // len(gate), axis=0)
    return (y if residual is None else y + residual), z


def linear_grad(dy, x, w, act_name="none", z=None, gate=None):
    """{"dz", "dx", "dw", "dbias", "dgate"}; z: the pre-activation the derivative is taken at."""
    out = {}
    per = len(dy) // len(gate) if gate is not None else 0
    if gate is not None:
        out["dgate"] = (dy * act(z, act_name)).reshape(len(gate), per, -1).sum(1) if z is not None else None
        dy = dy * np.repeat(gate, per, axis=0)
    dz = dy * act_grad(z, act_name) if act_name != "none" else dy
    return {**out, "dz": dz, "dx": dz @ w, "dw": dz.T @ x, "dbias": dz.sum(0)}


def attention_grad(cfg, q, k, v, do, kept, kept_ref=None, lse=None, o=None, bound=False):
    """Gradient of the tile-sparse attention for token-major [B, N, heads, d] inputs.

    kept[b][h]: kept video key tiles per video query tile. lse [B, N, heads] and o: the forward's outputs
    to take P and delta from (None: the exact ones). Returns (dq, dk, dv, lse, o) and with bound=True also
    (bq, bk, bv): for each gradient the sum of |terms| of its last product, and (fq, fk, fv): what the fp32
    accumulation of dP and delta (head_dim additions, 2^-23 of the sum of |terms| each) moves it by at most."""
    q, k, v, do = (np.asarray(a, dtype=np.float64) for a in (q, k, v, do))
    scale = 1.0 / np.sqrt(cfg.head_dim)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(q), np.zeros_like(q)
    bq, bk, bv, fq, fk = (np.zeros_like(q) for _ in range(5))
    lse_out, o_out = np.zeros(q.shape[:3]), np.zeros_like(q)
    from .vsa_oracle import ref_tiles
    for b in range(q.shape[0]):
        for h in range(cfg.heads):
            til = head_tiling(cfg, h)
            for n, rows in enumerate(til.all):
                i = n - til.n_prefix
                sel = [] if i < 0 else kept[b][h][i]
                if kept_ref is not None:
                    keys = query_key_tokens(til, n, sel, ref_tiles(cfg), [] if i < 0 else kept_ref[b][h][i])
                else:
                    keys = query_key_tokens(til, n, sel)
                kk, vv, qq, dd = k[b, keys, h], v[b, keys, h], q[b, rows, h], do[b, rows, h]
                s = scale * qq @ kk.T
                m = s.max(1, keepdims=True)
                exact = (m + np.log(np.exp(s - m).sum(1, keepdims=True)))[:, 0]
                l = exact if lse is None else lse[b, rows, h]
                p = np.exp(s - l[:, None])
                oo = np.exp(s - exact[:, None]) @ vv
                lse_out[b, rows, h], o_out[b, rows, h] = exact, oo
                if o is not None:
                    oo = o[b, rows, h]
                dp = dd @ vv.T
                ds = p * (dp - (dd * oo).sum(1, keepdims=True))
                dq[b, rows, h] = scale * ds @ kk
                np.add.at(dk[b, :, h], keys, scale * ds.T @ qq)
                np.add.at(dv[b, :, h], keys, p.T @ dd)
                if bound:
                    fp32 = p * (np.abs(dd) @ np.abs(vv).T + (np.abs(dd) * np.abs(oo)).sum(1, keepdims=True))
                    fp32 *= cfg.head_dim * 2.0 ** -23
                    bq[b, rows, h] = scale * np.abs(ds) @ np.abs(kk)
                    fq[b, rows, h] = scale * fp32 @ np.abs(kk)
                    np.add.at(bk[b, :, h], keys, scale * np.abs(ds).T @ np.abs(qq))
                    np.add.at(fk[b, :, h], keys, scale * fp32.T @ np.abs(qq))
                    np.add.at(bv[b, :, h], keys, p.T @ np.abs(dd))
    return (dq, dk, dv, lse_out, o_out) + ((bq, bk, bv, fq, fk, np.zeros_like(q)) if bound else ())
