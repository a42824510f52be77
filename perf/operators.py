"""The operators around the tile-sparse attention layer that are measured, case by case.

Three families, each reached through a method of ``Plan``:

* norm + rotation -- RMS norm of every head's query and key row and the rotary position embedding in one
  pass: token-major (``qk_norm_rope``), fused with the tile pack and the score stage's pooling
  (``tile_norm_rope_pack_pool``), and its gradient from token-major or packed gradients
  (``qk_norm_rope_bwd``, ``tile_norm_rope_bwd``);
* linear -- y = residual + gate * act(x W^T + bias) in one product with its epilogue (``linear``) and the
  gradients of x, W, bias and gate (``linear_bwd``);
* the gradient of the tile-sparse attention over each query tile's kept key tiles (``sparse_attn_bwd``).

``run`` computes a case in plain torch operations in fp32 (``own = False``) or through the framework
(``own = True``); ``exact`` computes it in fp64, written apart from both.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
TILE = 64
CYCLE = ((4, 4, 4), (1, 8, 8), (16, 2, 2), (2, 4, 8))     # the head-aware tile shapes


# ------------------------------------------------------------------- cases ----

def listed():
    """Twelve cases: every operator from its smallest call to its largest."""
    clip = {"T": 28, "H": 48, "W": 80, "segments": "512,3840,640"}        # 107,520 video + 4,992 prefix tokens
    return [
        # the smallest layer: two heads of 64, 384 tokens; launch latency counts
        dict(name="norm rope small", op="norm", batch=1, heads=2, d=64, T=4, H=8, W=8, segments="64,64", shapes="444",
             k=2, layout="halves", per_head=False),
        # a 5 s clip of 1344x768: q, k, v straight from a fused projection into packed tiles and descriptors
        dict(name="norm rope pack clip", op="norm_pack", batch=1, heads=24, d=128, **clip, shapes="444", k=420,
             layout="interleaved", per_head=False, score="meanpool_gate"),
        # its gradient on the same clip: packed gradients back to the fused projection's layout
        dict(name="norm rope pack clip bwd", op="norm_pack_bwd", batch=1, heads=24, d=128, **clip, shapes="444", k=420,
             layout="interleaved", per_head=False),
        # two ragged samples with a weight per head: token-major gradient, odd grid, odd prefix
        dict(name="norm rope ragged bwd", op="norm_bwd", batch=2, heads=5, d=128, T=7, H=18, W=26, segments="77,130",
             shapes="cycle", k=3, layout="halves", per_head=True),
        # the conditioning of one denoising step: two timestep embeddings to six modulation vectors
        dict(name="linear modulation", op="linear", rows=2, n_in=2048, n_out=12288, act="none", bias=True, gate=False,
             residual=False, pre=False, samples=1),
        # a short prompt's projection, 77 tokens
        dict(name="linear prompt", op="linear", rows=77, n_in=1480, n_out=2056, act="gelu_tanh", bias=True, gate=False,
             residual=False, pre=False, samples=1),
        # the output projection of two short clips of 9,280 tokens: a gate per sample, added to the residual stream
        dict(name="linear output", op="linear", rows=18560, n_in=2048, n_out=2048, act="none", bias=True, gate=True,
             residual=True, pre=False, samples=2),
        # the feed-forward's first product over the whole clip, pre-activation kept for training
        dict(name="linear feed-forward", op="linear", rows=112512, n_in=2048, n_out=8192, act="gelu_tanh", bias=True,
             gate=False, residual=False, pre=True, samples=1),
        # its gradient over a short clip of 9,280 tokens
        dict(name="linear feed-forward bwd", op="linear_bwd", rows=9280, n_in=2048, n_out=8192, act="gelu_tanh",
             bias=True, gate=False, samples=1),
        # a small conditioning network's gradient: odd rows, three samples with a gate each
        dict(name="linear ragged bwd", op="linear_bwd", rows=1005, n_in=200, n_out=328, act="silu", bias=True, gate=True,
             samples=3),
        # attention gradient with partial tiles, head-aware shapes, head_dim 64, two samples
        dict(name="attention ragged bwd", op="attn_bwd", batch=2, heads=4, d=64, T=6, H=10, W=14, segments="100,30",
             shapes="cycle", k=4),
        # one rank's three heads (24 split over 8) of the clip at 75 % sparsity
        dict(name="attention clip bwd", op="attn_bwd", batch=1, heads=3, d=128, **clip, shapes="444", k=420),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_pack", "norm_pack_bwd", "norm_bwd", "linear", "linear", "linear_bwd", "attn_bwd",
                     "attn_bwd"])
    if op in ("linear", "linear_bwd"):
        while True:
            c = dict(op=op, rows=_log(rng, 1, 112512), n_in=8 * _log(rng, 4, 1024), n_out=8 * _log(rng, 4, 1536),
                     act=rng.choice(["none", "gelu_tanh", "silu"]), bias=rng.random() < 0.7, gate=rng.random() < 0.4,
                     samples=rng.choice([1, 1, 2, 3]))
            c["rows"] = max(1, c["rows"] // c["samples"]) * c["samples"]
            if op == "linear":
                c.update(residual=rng.random() < 0.4, pre=rng.random() < 0.3)
            if c["rows"] * c["n_in"] * c["n_out"] <= (1.8e12 if op == "linear" else 1.5e11):
                return c
    while True:
        d = rng.choice([64, 128, 128])
        c = dict(op=op, batch=rng.choice([1, 1, 2]), heads=_log(rng, 1, 24), d=d, T=_log(rng, 1, 28), H=_log(rng, 2, 48),
                 W=_log(rng, 2, 80), segments=rng.choice(["", "64", "512", "%d,%d" % (_log(rng, 1, 600), _log(rng, 1, 4000))]),
                 shapes=rng.choice(["444", "444", "cycle"]))
        n = _tokens(c)
        if c["batch"] * c["heads"] * n * d > 24 * 112512 * 128:
            continue
        low = min(_video_tiles(c, h) for h in range(c["heads"]))
        c["k"] = rng.choice([1, low, max(1, low // 2), max(1, low // 4), max(1, low // 10)])
        if op == "attn_bwd":
            if _pairs(c) * d > 1.2e12 or c["batch"] * c["heads"] * n * n * d > 4e12:
                continue
        else:
            c.update(layout=rng.choice(["interleaved", "halves"]), per_head=rng.random() < 0.3)
            if op == "norm_pack":
                c["score"] = rng.choice(["meanpool_gate", "tripool"])
        return c


# ---------------------------------------------------------------- geometry ----

def _segments(c):
    return [int(s) for s in c["segments"].split(",") if s]


def _shape(c, h):
    return (4, 4, 4) if c["shapes"] == "444" else CYCLE[h % len(CYCLE)]


def _tokens(c):
    return sum(_segments(c)) + c["T"] * c["H"] * c["W"]


def _video_tiles(c, h):
    pt, ph, pw = _shape(c, h)
    return -(-c["T"] // pt) * -(-c["H"] // ph) * -(-c["W"] // pw)


def _prefix_tiles(c):
    return sum(-(-s // TILE) for s in _segments(c))


def _nt_max(c):
    return _prefix_tiles(c) + max(_video_tiles(c, h) for h in range(c["heads"]))


def _rows_of(c, h, device="cpu"):
    """The packed row (tile * 64 + slot) of every token of one head, in token order."""
    out, tile = [], 0
    for s in _segments(c):
        j = torch.arange(s, device=device)
        out.append((tile + j // TILE) * TILE + j % TILE)
        tile += -(-s // TILE)
    pt, ph, pw = _shape(c, h)
    T, H, W = c["T"], c["H"], c["W"]
    t = torch.arange(T, device=device).view(T, 1, 1)
    y = torch.arange(H, device=device).view(1, H, 1)
    x = torch.arange(W, device=device).view(1, 1, W)
    eh = torch.clamp(H - (y // ph) * ph, max=ph)
    ew = torch.clamp(W - (x // pw) * pw, max=pw)
    n = ((t // pt) * -(-H // ph) + y // ph) * -(-W // pw) + x // pw
    slot = ((t % pt) * eh + y % ph) * ew + x % pw
    out.append(((tile + n) * TILE + slot).expand(T, H, W).reshape(-1))
    return torch.cat(out)


def _counts(c, h, device="cpu"):
    """Valid tokens of every packed tile of one head, [nt_max]."""
    return torch.bincount(_rows_of(c, h, device) // TILE, minlength=_nt_max(c))


def _pairs(c):
    """(query row, key row) pairs the attention computes, at most: whole tiles for the kept ones."""
    pre, n = sum(_segments(c)), _tokens(c)
    return c["batch"] * c["heads"] * (pre * n + (n - pre) * (pre + min(c["k"] * TILE, n - pre)))


# ------------------------------------------------------------------ inputs ----

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=BF16, scale=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=F32).mul_(scale).to(dtype)


def _table(c):
    """cos, sin [tokens, d / 2] of a rotation along t, h and w; prefix tokens stay unrotated."""
    half = c["d"] // 2
    split = (half - 2 * (half // 3), half // 3, half // 3)
    T, H, W = c["T"], c["H"], c["W"]
    grid = torch.stack(torch.meshgrid(torch.arange(T), torch.arange(H), torch.arange(W), indexing="ij"), -1)
    pos = grid.reshape(-1, 3).to(F64).cuda()
    ang = [pos[:, a:a + 1] * (10000.0 ** (-torch.arange(n, dtype=F64, device="cuda") / n)) for a, n in enumerate(split)]
    ang = torch.cat(ang, 1)
    ang = torch.cat([torch.zeros(sum(_segments(c)), half, dtype=F64, device="cuda"), ang])
    return ang.cos().to(F32), ang.sin().to(F32)


def _plan(c):
    import tile_sparse_video_pack_b200 as T
    trip = c.get("score") == "tripool"
    heads = c["heads"]
    return T.Plan(T.make_desc(c["batch"], heads, c["d"], c["T"], c["H"], c["W"], _segments(c),
                              [_shape(c, h) for h in range(heads)], [c["k"]] * heads,
                              "tripool" if trip else "meanpool_gate", 64 if trip else c["d"]))


def _kept(c, g):
    """Kept key tiles of every video query tile, ascending: a noisy score that favours near tiles."""
    B, Hh, k = c["batch"], c["heads"], c["k"]
    ntv_max = max(_video_tiles(c, h) for h in range(Hh))
    idx = torch.zeros(B, Hh, ntv_max, k, dtype=torch.int32, device="cuda")
    for h in range(Hh):
        pt, ph, pw = _shape(c, h)
        nT, nY, nX = -(-c["T"] // pt), -(-c["H"] // ph), -(-c["W"] // pw)
        n = nT * nY * nX
        at = torch.arange(n, device="cuda")
        xyz = torch.stack([at // (nY * nX), at // nX % nY, at % nX], 1).to(F32)
        near = torch.exp(-0.1 * (xyz[:, None] - xyz[None]).pow(2).sum(-1)).mul_(2.0)
        for b in range(B):
            s = near + torch.randn(n, n, generator=g, device="cuda")
            idx[b, h, :n] = s.topk(k, dim=1).indices.sort(dim=1).values.to(torch.int32)
    return idx


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = {"case": c}
    if c["op"] in ("linear", "linear_bwd"):
        M, K, N, S = c["rows"], c["n_in"], c["n_out"], c["samples"]
        st["x"] = _randn(g, M, K)
        st["w"] = _randn(g, N, K, scale=K ** -0.5)
        st["bias"] = _randn(g, N, dtype=F32, scale=0.1) if c["bias"] else None
        st["gate"] = _randn(g, S, N, dtype=F32, scale=0.5) if c["gate"] else None
        if c["op"] == "linear":
            st["residual"] = _randn(g, M, N) if c["residual"] else None
        else:
            st["dy"] = _randn(g, M, N)
            st["pre"] = _randn(g, M, N) if c["act"] != "none" or c["gate"] else None
        if own:
            import tile_sparse_video_pack_b200 as T
            st["plan"] = p = T.Plan(T.make_desc(1, 1, 64, 1, 8, 8, [], [(4, 4, 4)], [1]))
            new = lambda *s, t=BF16: torch.empty(*s, dtype=t, device="cuda")
            if c["op"] == "linear_bwd":
                st["ws"] = new(p.linear_bwd_workspace_bytes(M, K, N, samples=S if c["gate"] else 0), t=torch.uint8)
                st.update(dx=new(M, K), dw=new(N, K), dbias=new(N, t=F32) if c["bias"] else None,
                          dgate=new(S, N, t=F32) if c["gate"] else None)
            else:
                st.update(y=new(M, N), z=new(M, N) if c["pre"] else None)
        return st

    B, Hh, d, n = c["batch"], c["heads"], c["d"], _tokens(c)
    packed = (B, Hh, _nt_max(c), TILE, d)

    def pack(t):                                # [B, n, heads, d] -> packed tiles, zero in unused slots
        out = torch.zeros(B, Hh, packed[2] * TILE, d, dtype=t.dtype, device="cuda")
        for h in range(Hh):
            out[:, h, _rows_of(c, h, "cuda")] = t[:, :, h]
        return out.view(packed)

    if own:
        st["plan"] = _plan(c)
    if c["op"] == "attn_bwd":
        q, k, v, do = (pack(_randn(g, B, n, Hh, d)) for _ in range(4))
        st.update(q=q, k=k, v=v, do=do, idx=_kept(c, g))
        o, lse = torch.zeros_like(q), torch.zeros(packed[:4], dtype=F32, device="cuda")
        _attend(c, st, o, lse)
        st.update(o=o, lse=lse)
        if own:
            p = st["plan"]
            st.update(dq=torch.empty_like(q), dk=torch.empty_like(q), dv=torch.empty_like(q),
                      ws=torch.empty(p.attn_bwd_workspace_bytes(), dtype=torch.uint8, device="cuda"))
        return st

    wshape = (Hh, d) if c["per_head"] else (d,)
    st["w_q"], st["w_k"] = (1.0 + _randn(g, *wshape, dtype=F32, scale=0.2) for _ in range(2))
    st["cos"], st["sin"] = _table(c)
    # q, k, v as one projection's output: strided views, as a layer has them
    qkv = _randn(g, B, n, 3, Hh, d, scale=1.5)
    st["q"], st["k"], st["v"] = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
    if c["op"] == "norm_bwd":
        st["dqo"], st["dko"] = _randn(g, B, n, Hh, d), _randn(g, B, n, Hh, d)
    if c["op"] == "norm_pack_bwd":
        st["dqp"], st["dkp"], st["dvp"] = (pack(_randn(g, B, n, Hh, d)) for _ in range(3))
    if own:
        import tile_sparse_video_pack_b200 as T
        p = st["plan"]
        st["norm"] = T.NormRope(st["w_q"], st["w_k"], st["cos"], st["sin"], layout=c["layout"], eps=1e-6)
        new = lambda *s, t=BF16: torch.empty(*s, dtype=t, device="cuda")
        if c["op"] == "norm":
            st.update(qo=new(B, n, Hh, d), ko=new(B, n, Hh, d))
        elif c["op"] == "norm_pack":
            st.update({x: new(*packed) for x in ("qp", "kp", "vp")})
            st["ws"] = new(p.info.workspace_bytes, t=torch.uint8)
        else:
            dqkv = new(B, n, 3, Hh, d)
            st.update(dq=dqkv[:, :, 0], dk=dqkv[:, :, 1], dv=dqkv[:, :, 2], dw_q=new(*wshape, t=F32),
                      dw_k=new(*wshape, t=F32), ws=new(p.norm_bwd_workspace_bytes(), t=torch.uint8))
    return st


# --------------------------------------------------------------- plain forms ----

def _act(z, act):
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "gelu_tanh":
        a = math.sqrt(2.0 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3 * 0.044715 * z * z)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return torch.ones_like(z)


def _rotate(x, cos, sin, layout, sign=1.0):
    """Rotates the channel pairs of x [B, n, heads, d] by the table's angles (sign -1: back)."""
    cos, sin = cos[None, :, None], sign * sin[None, :, None]
    if layout == "halves":
        a, b = x.chunk(2, dim=-1)
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)


def _norm_rope(st, x, w):
    x = x.to(F32)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    return _rotate(x * r * w, st["cos"], st["sin"], st["case"]["layout"])


def _norm_rope_grad(st, dy, x, w):
    x = x.to(F32)
    dn = _rotate(dy.to(F32), st["cos"], st["sin"], st["case"]["layout"], -1.0)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    xr = x * r
    dw = (dn * xr).sum((0, 1) if st["case"]["per_head"] else (0, 1, 2))
    g = dn * w
    return (r * (g - xr * (g * xr).mean(-1, keepdim=True))).to(BF16), dw


def _pack_index(c):
    """For every packed row of every head the token it holds, or the number of tokens where it holds none."""
    n, rows = _tokens(c), _nt_max(c) * TILE
    out = torch.full((c["heads"], rows), n, dtype=torch.int64, device="cuda")
    for h in range(c["heads"]):
        out[h, _rows_of(c, h, "cuda")] = torch.arange(n, device="cuda")
    return out


def _pack_plain(c, x):
    """[B, n, heads, d] -> packed tiles by a gather, a row of zeros standing for unused slots."""
    B, n, Hh, d = x.shape
    x = torch.cat([x, torch.zeros_like(x[:, :1])], 1)
    at = _pack_index(c)
    return torch.stack([x[:, at[h], h] for h in range(Hh)], 1).view(B, Hh, -1, TILE, d)


def _unpack_plain(c, x):
    B, Hh, _, _, d = x.shape
    flat = x.reshape(B, Hh, -1, d)
    return torch.stack([flat[:, h, _rows_of(c, h, "cuda")] for h in range(Hh)], 2)


def _pool_plain(c, xp):
    """Descriptors of every video tile of packed xp: mean over its tokens, for TripPool maximum and minimum too."""
    pre, ntv_max = _prefix_tiles(c), max(_video_tiles(c, h) for h in range(c["heads"]))
    out = []
    for h in range(c["heads"]):
        n = _counts(c, h, "cuda")[pre:]
        x = xp[:, h, pre:].to(F32)
        has = (torch.arange(TILE, device="cuda") < n[:, None])[None, :, :, None]
        real = (n > 0)[None, :, None]
        parts = [x.sum(2) / n.clamp(min=1)[None, :, None]]
        if c["score"] == "tripool":
            parts += [torch.where(has, x, -math.inf).amax(2), torch.where(has, x, math.inf).amin(2)]
        out.append(torch.where(real, torch.cat(parts, -1), 0.0))
    return torch.stack(out, 1)


def _chunks(c, h, idx_bh):
    """Query tiles of one head in blocks that share a shape: (query tile ids, their key tile ids)."""
    pre, ntv = _prefix_tiles(c), _video_tiles(c, h)
    every = torch.arange(pre + ntv, device="cuda")
    step = max(1, 3000 // (pre + ntv))
    for a in range(0, pre, step):
        q = torch.arange(a, min(pre, a + step), device="cuda")
        yield q, every[None].expand(len(q), -1)
    keys = torch.cat([torch.arange(pre, device="cuda")[None].expand(ntv, -1), pre + idx_bh[:ntv].long()], 1)
    step = max(1, 20000 // keys.shape[1])
    for a in range(0, ntv, step):
        yield torch.arange(pre + a, pre + min(ntv, a + step), device="cuda"), keys[a:a + step]


def _masks(counts, qt, kt):
    slot = torch.arange(TILE, device="cuda")
    rows = (slot < counts[qt][:, None])[:, :, None]
    cols = (slot < counts[kt][..., None]).flatten(1)[:, None]
    return rows, cols


def _attend(c, st, o, lse):
    """Forward: the output and row log-sum-exp that a training step holds when its gradient is asked for."""
    scale = c["d"] ** -0.5
    for b in range(c["batch"]):
        for h in range(c["heads"]):
            n = _counts(c, h, "cuda")
            for qt, kt in _chunks(c, h, st["idx"][b, h]):
                rows, cols = _masks(n, qt, kt)
                s = st["q"][b, h, qt].to(F32) @ st["k"][b, h, kt].flatten(1, 2).to(F32).mT
                s = torch.where(cols, s.mul_(scale), -math.inf)
                m = s.amax(-1, keepdim=True)
                p = torch.exp(s - m)
                l = p.sum(-1, keepdim=True)
                o[b, h, qt] = torch.where(rows, (p @ st["v"][b, h, kt].flatten(1, 2).to(F32)) / l, 0.0).to(BF16)
                lse[b, h, qt] = torch.where(rows, m + torch.log(l), 0.0)[..., 0]


def _attend_grad(c, st):
    scale, d = c["d"] ** -0.5, c["d"]
    out = []
    dq, dk, dv = (torch.zeros(st["q"].shape, dtype=F32, device="cuda") for _ in range(3))
    delta = (st["do"].to(F32) * st["o"].to(F32)).sum(-1, keepdim=True)
    for b in range(c["batch"]):
        for h in range(c["heads"]):
            n = _counts(c, h, "cuda")
            dkh, dvh = dk[b, h].view(-1, TILE * d), dv[b, h].view(-1, TILE * d)
            for qt, kt in _chunks(c, h, st["idx"][b, h]):
                rows, cols = _masks(n, qt, kt)
                q, do = st["q"][b, h, qt].to(F32), st["do"][b, h, qt].to(F32)
                kk, vv = (st[x][b, h, kt].flatten(1, 2).to(F32) for x in ("k", "v"))
                p = torch.exp((q @ kk.mT).mul_(scale).sub_(st["lse"][b, h, qt][..., None]))
                p = torch.where(rows & cols, p, 0.0)
                ds = (do @ vv.mT).sub_(delta[b, h, qt]).mul_(p).mul_(scale)
                dq[b, h, qt] = ds @ kk
                dkh.index_add_(0, kt.reshape(-1), (ds.mT @ q).reshape(-1, TILE * d))
                dvh.index_add_(0, kt.reshape(-1), (p.mT @ do).reshape(-1, TILE * d))
    out = [x.to(BF16) for x in (dq, dk, dv)]
    return {"dq": out[0], "dk": out[1], "dv": out[2]}


def run(state):
    st, c = state, state["case"]
    op = c["op"]
    if own:
        return _run_own(st, c, op)
    if op == "linear":
        z = st["x"].to(F32) @ st["w"].to(F32).T
        if st["bias"] is not None:
            z += st["bias"]
        y = _act(z, c["act"])
        if st["gate"] is not None:
            y = y * st["gate"].repeat_interleave(c["rows"] // c["samples"], 0)
        if st["residual"] is not None:
            y = y + st["residual"].to(F32)
        out = {"y": y.to(BF16)}
        if c["pre"]:
            out["pre"] = z.to(BF16)
        return out
    if op == "linear_bwd":
        per = c["rows"] // c["samples"]
        dy, out = st["dy"].to(F32), {}
        z = st["pre"].to(F32) if st["pre"] is not None else None
        if st["gate"] is not None:
            out["dgate"] = (dy * _act(z, c["act"])).view(c["samples"], per, -1).sum(1)
            dy = dy * st["gate"].repeat_interleave(per, 0)
        dz = dy * _act_grad(z, c["act"]) if c["act"] != "none" else dy
        if c["bias"]:
            out["dbias"] = dz.sum(0)
        out["dx"] = (dz @ st["w"].to(F32)).to(BF16)
        out["dw"] = (dz.T @ st["x"].to(F32)).to(BF16)
        return out
    if op == "attn_bwd":
        return _attend_grad(c, st)
    if op == "norm":
        return {x: _norm_rope(st, st[x], st["w_" + x]).to(BF16) for x in ("q", "k")}
    if op == "norm_pack":
        qp, kp = (_pack_plain(c, _norm_rope(st, st[x], st["w_" + x]).to(BF16)) for x in ("q", "k"))
        return {"qp": qp, "kp": kp, "vp": _pack_plain(c, st["v"]), "pool_q": _pool_plain(c, qp),
                "pool_k": _pool_plain(c, kp)}
    packed = op == "norm_pack_bwd"
    dqo = _unpack_plain(c, st["dqp"]) if packed else st["dqo"]
    dko = _unpack_plain(c, st["dkp"]) if packed else st["dko"]
    dq, dw_q = _norm_rope_grad(st, dqo, st["q"], st["w_q"])
    dk, dw_k = _norm_rope_grad(st, dko, st["k"], st["w_k"])
    out = {"dq": dq, "dk": dk, "dw_q": dw_q, "dw_k": dw_k}
    if packed:
        out["dv"] = _unpack_plain(c, st["dvp"])
    return out


def _run_own(st, c, op):
    p = st["plan"]
    if op == "linear":
        p.linear(st["x"], st["w"], st["y"], bias=st["bias"], act=c["act"], gate=st["gate"], residual=st["residual"],
                 pre=st["z"])
        return {"y": st["y"], "pre": st["z"]} if c["pre"] else {"y": st["y"]}
    if op == "linear_bwd":
        p.linear_bwd(st["dy"], st["x"], st["w"], st["dx"], st["dw"], act=c["act"], pre=st["pre"], gate=st["gate"],
                     dbias=st["dbias"], dgate=st["dgate"], workspace=st["ws"])
        out = {"dgate": st["dgate"]} if c["gate"] else {}
        if c["bias"]:
            out["dbias"] = st["dbias"]
        return {**out, "dx": st["dx"], "dw": st["dw"]}
    if op == "attn_bwd":
        p.sparse_attn_bwd(st["q"], st["k"], st["v"], st["o"], st["lse"], st["do"], st["idx"], st["dq"], st["dk"],
                          st["dv"], st["ws"])
        return {"dq": st["dq"], "dk": st["dk"], "dv": st["dv"]}
    if op == "norm":
        p.qk_norm_rope(st["q"], st["k"], st["norm"], st["qo"], st["ko"])
        return {"q": st["qo"], "k": st["ko"]}
    if op == "norm_pack":
        p.tile_norm_rope_pack_pool(st["q"], st["k"], st["v"], st["norm"], st["qp"], st["kp"], st["vp"], st["ws"])
        pool_q, pool_k = p.pooled(st["ws"])
        return {"qp": st["qp"], "kp": st["kp"], "vp": st["vp"], "pool_q": pool_q, "pool_k": pool_k}
    if op == "norm_bwd":
        p.qk_norm_rope_bwd(st["dqo"], st["dko"], st["q"], st["k"], st["norm"], st["dq"], st["dk"], st["dw_q"],
                           st["dw_k"], st["ws"])
    else:
        p.tile_norm_rope_bwd(st["dqp"], st["dkp"], st["dvp"], st["q"], st["k"], st["norm"], st["dq"], st["dk"],
                             st["dv"], st["dw_q"], st["dw_k"], st["ws"])
    out = {"dq": st["dq"], "dk": st["dk"], "dw_q": st["dw_q"], "dw_k": st["dw_k"]}
    if op == "norm_pack_bwd":
        out["dv"] = st["dv"]
    return out


# --------------------------------------------------------------------- work ----

def work(case):
    c = case
    if c["op"] in ("linear", "linear_bwd"):
        M, K, N, S = c["rows"], c["n_in"], c["n_out"], c["samples"]
        vec = 4 * N * (c["bias"] + S * c["gate"])
        if c["op"] == "linear":
            return {"bytes": 2 * (M * K + N * K + M * N * (1 + c["residual"] + c["pre"])) + vec, "flops": 2 * M * N * K}
        pre = c["act"] != "none" or c["gate"]
        return {"bytes": 2 * (2 * M * K + 2 * N * K + M * N * (1 + pre)) + vec + 4 * N * S * c["gate"],
                "flops": 4 * M * N * K}
    B, Hh, d, n = c["batch"], c["heads"], c["d"], _tokens(c)
    row, prow = B * Hh * n * d, B * Hh * _nt_max(c) * TILE * d
    if c["op"] == "attn_bwd":
        ntv = sum(_video_tiles(c, h) for h in range(Hh))
        return {"bytes": 2 * 5 * row + 2 * 3 * prow + 4 * B * (Hh * n + ntv * c["k"]), "flops": 10 * d * _pairs(c)}
    w = 4 * 2 * d * (Hh if c["per_head"] else 1)
    table = 4 * n * d
    if c["op"] == "norm":
        return {"bytes": 2 * 4 * row + table + w, "flops": 20 * row}
    if c["op"] == "norm_pack":
        nv = sum(_video_tiles(c, h) for h in range(Hh))
        pool = 4 * 2 * B * nv * d * (3 if c["score"] == "tripool" else 1)
        return {"bytes": 2 * 3 * (row + prow) + table + w + pool, "flops": 22 * row}
    return {"bytes": 2 * (6 + 2 * (c["op"] == "norm_pack_bwd")) * row + table + 2 * w, "flops": 40 * row}


# -------------------------------------------------------------------- exact ----

def _turn(x, cos, sin, layout, back=False):
    """The rotation as a product of complex numbers, fp64."""
    turn = torch.complex(cos, -sin if back else sin)[None, :, None]
    half = x.shape[-1] // 2
    if layout == "halves":
        z = torch.complex(x[..., :half], x[..., half:]) * turn
        return torch.cat([z.real, z.imag], -1)
    return torch.view_as_real(torch.view_as_complex(x.reshape(*x.shape[:-1], half, 2)) * turn).flatten(-2)


def _scatter(c, x):
    B, n, Hh, d = x.shape
    out = torch.zeros(B, Hh, _nt_max(c) * TILE, d, dtype=x.dtype, device=x.device)
    for h in range(Hh):
        out[:, h].index_copy_(1, _rows_of(c, h, "cuda"), x[:, :, h])
    return out.view(B, Hh, -1, TILE, d)


def _exact_linear(c, st):
    per = c["rows"] // c["samples"]
    parts = {"y": [], "pre": []}
    w = st["w"].to(F64)
    step = max(1, (1 << 28) // c["n_out"])                 # rows at a time
    for a in range(0, c["rows"], step):
        z = torch.mm(st["x"][a:a + step].to(F64), w.t())
        if c["bias"]:
            z += st["bias"].to(F64)
        y = z
        if c["act"] == "gelu_tanh":
            u = z * (1 + 0.044715 * z * z) * math.sqrt(8 / math.pi)
            y = z * torch.sigmoid(u)                       # (1 + tanh(u / 2)) / 2 = sigmoid(u)
        elif c["act"] == "silu":
            y = z * torch.sigmoid(z)
        if c["gate"]:
            at = torch.arange(a, a + len(z), device="cuda") // per
            y = y * st["gate"].to(F64)[at]
        if c["residual"]:
            y = y + st["residual"][a:a + step].to(F64)
        parts["y"].append(y)
        if c["pre"]:
            parts["pre"].append(z)
    return {k: torch.cat(v) for k, v in parts.items() if v}


def _exact_linear_bwd(c, st):
    M, S = c["rows"], c["samples"]
    dy, out = st["dy"].to(F64), {}
    f, slope = torch.ones_like(dy), torch.ones_like(dy)
    if st["pre"] is not None:
        z = st["pre"].to(F64)
        f = z
        if c["act"] != "none":
            if c["act"] == "gelu_tanh":
                b = math.sqrt(8 / math.pi)
                g, du = torch.sigmoid(b * (z + 0.044715 * z ** 3)), b * (1 + 3 * 0.044715 * z * z)
            else:
                g, du = torch.sigmoid(z), 1.0
            f, slope = z * g, g + z * g * (1 - g) * du
    at = torch.arange(M, device="cuda") // (M // S)
    if c["gate"]:
        out["dgate"] = torch.zeros(S, c["n_out"], dtype=F64, device="cuda").index_add_(0, at, dy * f)
        dy = dy * st["gate"].to(F64)[at]
    dz = dy * slope
    if c["bias"]:
        out["dbias"] = torch.mv(dz.t(), torch.ones(M, dtype=F64, device="cuda"))
    out["dx"] = torch.mm(dz, st["w"].to(F64))
    out["dw"] = torch.mm(dz.t(), st["x"].to(F64))
    return out


def _exact_attention(c, st):
    """Every query row against every key of its head, kept or not, under a boolean mask."""
    scale, pre = c["d"] ** -0.5, _prefix_tiles(c)
    grads = [torch.zeros(st["q"].shape, dtype=F64, device="cuda") for _ in range(3)]
    for b in range(c["batch"]):
        for h in range(c["heads"]):
            rows = _rows_of(c, h, "cuda")
            tile = rows // TILE
            q, k, v, do, o = (st[x][b, h].reshape(-1, c["d"])[rows].to(F64) for x in ("q", "k", "v", "do", "o"))
            lse = st["lse"][b, h].reshape(-1)[rows].to(F64)
            allowed = torch.ones(_nt_max(c), _nt_max(c), dtype=torch.bool, device="cuda")
            allowed[pre:, pre:] = False
            ntv = _video_tiles(c, h)
            allowed[pre:pre + ntv].scatter_(1, pre + st["idx"][b, h, :ntv].long(), True)
            dk, dv = torch.zeros_like(k), torch.zeros_like(v)
            dq = torch.empty_like(q)
            step = max(TILE, (1 << 28) // len(rows))
            for a in range(0, len(rows), step):
                s = slice(a, a + step)
                w = torch.where(allowed[tile[s]][:, tile], torch.exp(q[s] @ k.t() * scale - lse[s, None]), 0.0)
                dv += w.t() @ do[s]
                w *= do[s] @ v.t() - (do[s] * o[s]).sum(1, keepdim=True)
                dq[s] = w @ k * scale
                dk += w.t() @ q[s] * scale
            for g, x in zip(grads, (dq, dk, dv)):
                g[b, h].view(-1, c["d"])[rows] = x
    return {"dq": grads[0], "dk": grads[1], "dv": grads[2]}


def exact(case, seed):
    c = case
    st = _inputs_only(case, seed)
    if c["op"] == "linear":
        return _exact_linear(c, st)
    if c["op"] == "linear_bwd":
        return _exact_linear_bwd(c, st)
    if c["op"] == "attn_bwd":
        return _exact_attention(c, st)
    cos, sin = st["cos"].to(F64), st["sin"].to(F64)

    def forward(x, w):
        x = x.to(F64)
        return _turn(x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.to(F64), cos, sin, c["layout"])

    if c["op"] == "norm":
        return {x: forward(st[x], st["w_" + x]) for x in ("q", "k")}
    if c["op"] == "norm_pack":
        qp, kp = (_scatter(c, forward(st[x], st["w_" + x])) for x in ("q", "k"))
        # the descriptors are pooled from the tiles as they are stored, so they have no value apart from that rounding
        return {"qp": qp, "kp": kp, "vp": _scatter(c, st["v"].to(F64)), "pool_q": None, "pool_k": None}
    packed = c["op"] == "norm_pack_bwd"
    back = {}
    for x in ("q", "k"):
        dy = torch.empty(c["batch"], _tokens(c), c["heads"], c["d"], dtype=F64, device="cuda")
        for h in range(c["heads"]):
            src = st["d%sp" % x][:, h].reshape(c["batch"], -1, c["d"]) if packed else None
            dy[:, :, h] = src[:, _rows_of(c, h, "cuda")] if packed else st["d%so" % x][:, :, h]
        dn = _turn(dy, cos, sin, c["layout"], back=True)
        del dy
        v, w = st[x].to(F64), st["w_" + x].to(F64)
        inv = 1 / torch.sqrt(v.square().mean(-1, keepdim=True) + 1e-6)
        unit = v * inv
        gw = torch.einsum("bnhd,bnhd->hd", dn, unit)
        back["dw_" + x] = gw if c["per_head"] else gw.sum(0)
        dn *= w
        back["d" + x] = inv * (dn - unit * (dn * unit).mean(-1, keepdim=True))
    out = {"dq": back["dq"], "dk": back["dk"], "dw_q": back["dw_q"], "dw_k": back["dw_k"]}
    if packed:
        flat = st["dvp"].reshape(c["batch"], c["heads"], -1, c["d"]).to(F64)
        out["dv"] = torch.stack([flat[:, h, _rows_of(c, h, "cuda")] for h in range(c["heads"])], 2)
    return out


def _inputs_only(case, seed):
    """prepare's inputs without the framework's plan and buffers."""
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was
