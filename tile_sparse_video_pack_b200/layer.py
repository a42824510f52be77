"""One tile-sparse attention layer -- a plan, its device buffers and its score weights -- and the parts of a
transformer block around it: projections, norm and rotation, feed-forward, and their gradients."""
from __future__ import annotations

from .vsa import NormRope, Plan, make_desc, k_from_sparsity


class TileSparseAttention:
    """Runs pack -> score -> select -> sparse attention -> unpack on token-major bf16 Q, K, V.

    ``proj_q`` / ``proj_k``: fp32 CUDA tensors -- the gate G ([d, d], the same
    tensor for both) for mean-pool scoring, or per-head TripPool projections
    ([heads, 3d, p]). ``direct=True`` (plans with ``info.direct_attn``) runs
    pool -> score -> select -> sparse attention straight on the token-major
    tensors and allocates no packed copies: less memory, about three times the
    attention time (see vsa_sparse_attn_direct).
    """

    def __init__(self, plan: Plan, proj_q, proj_k, with_lse: bool = False, device=None, direct: bool = False):
        self.plan = plan
        self.proj_q = proj_q
        self.proj_k = proj_k
        if direct and not plan.info.direct_attn:
            raise ValueError("this plan's tiles are not boxes of the token-major tensors (info.direct_attn == 0)")
        self.direct = direct
        self.runs = 0        # forwards so far: whose tiles the buffers hold
        self.bufs = plan.allocate(device, with_lse=with_lse, packed=not direct)

    @classmethod
    def from_config(cls, cfg, sparsity, proj_q, proj_k, k_per_head=None, **kw):
        return cls(Plan.from_config(cfg, sparsity, k_per_head=k_per_head), proj_q, proj_k, **kw)

    def forward(self, q, k, v, out=None, stream=None):
        """Token-major ``[B, N, heads, d]`` bf16 CUDA tensors -> output of the same shape."""
        import torch
        if out is None:
            out = torch.empty_like(q)
        if self.plan.info.n_ref_tiles or self.direct:
            return self.stages(q, k, v, out, stream)   # R2VA budgets, or tiles straight from q, k, v
        self.runs += 1
        self.plan.layer_forward(q, k, v, self.proj_q, self.proj_k, self.bufs, out, stream=stream)
        return out

    __call__ = forward

    def stages(self, q, k, v, out, stream=None):
        """The calls one by one (same result as :meth:`forward`); with reference segments,
        the reference tiles are scored and selected and the attention uses that selection."""
        b, p = self.bufs, self.plan
        if self.direct:
            self.runs += 1
            p.tile_pool(q, k, b["workspace"], stream)
            p.tile_score_pooled(self.proj_q, self.proj_k, b["scores"], b["workspace"], stream)
            p.topk_select(b["scores"], b["idx"], stream)
            p.sparse_attn_direct(q, k, v, b["idx"], out, b["lse"], stream)
            return out
        p.tile_pack_pool(q, k, v, b["qp"], b["kp"], b["vp"], b["workspace"], stream)
        return self.attend(out, stream)

    def attend(self, out, stream=None):
        """The stages after packing, from the packed tiles and descriptors in the layer's buffers."""
        self.runs += 1
        b, p = self.bufs, self.plan
        p.tile_score_pooled(self.proj_q, self.proj_k, b["scores"], b["workspace"], stream)
        p.topk_select(b["scores"], b["idx"], stream)
        if p.info.n_ref_tiles:
            p.ref_score(b["kp"], self.proj_k, b["scores_ref"], b["workspace"], stream)
            p.topk_select_ref(b["scores_ref"], b["idx_ref"], stream)
            p.sparse_attn_ref(b["qp"], b["kp"], b["vp"], b["idx"], b["idx_ref"], b["op"], b["lse"], stream)
        else:
            p.sparse_attn(b["qp"], b["kp"], b["vp"], b["idx"], b["op"], b["lse"], stream)
        p.tile_unpack(b["op"], out, stream)
        return out


def axial_rope_table(plan, theta: float = 10000.0, split=None, device=None):
    """cos, sin (fp32 [n_tokens, head_dim / 2], for :class:`NormRope`) of a rotation along t, h and w: the channel
    pairs are divided among the three axes (``split``; by default h and w a third each, t the rest) and pair j
    of an axis with n pairs turns by position * theta^(-j / n). Prefix tokens are not rotated. Angles in fp64."""
    import torch
    d = plan.desc
    half = d.head_dim // 2
    split = (half - 2 * (half // 3), half // 3, half // 3) if split is None else tuple(split)
    if len(split) != 3 or sum(split) != half or min(split) < 0:
        raise ValueError(f"split must be three counts with sum {half}, got {split}")
    dev = torch.device("cuda") if device is None else torch.device(device)
    f64 = dict(dtype=torch.float64, device=dev)
    n_pre = sum(d.seg_len[i] for i in range(d.n_segments))
    angles = []
    for axis, (size, n) in enumerate(zip((d.T, d.H, d.W), split)):
        if n == 0:
            continue
        a = torch.arange(size, **f64)[:, None] * theta ** (-torch.arange(n, **f64) / n)
        shape = [1, 1, 1, n]
        shape[axis] = size
        angles.append(a.view(shape).expand(d.T, d.H, d.W, n).reshape(-1, n))
    video = torch.cat(angles, 1)
    table = torch.cat([torch.zeros(n_pre, half, **f64), video])
    return table.cos().float().contiguous(), table.sin().float().contiguous()


def _new(like, *shape, dtype=None):
    import torch
    return torch.empty(*shape, dtype=dtype or torch.bfloat16, device=like.device)


def _workspace(like, n):
    import torch
    return torch.empty(n, dtype=torch.uint8, device=like.device)


def _check_bias(name, b, n):
    if b is not None and tuple(b.shape) != (n,):
        raise ValueError(f"{name} must be [{n}], got {tuple(b.shape)}")


def _row_bytes(t):
    """Bytes from row to row of a [..., cols] view whose leading dimensions form one row axis, else None."""
    try:
        m = t.view(-1, t.shape[-1])
    except RuntimeError:
        return None
    return m.stride(0) * t.element_size() if m.stride(1) == 1 else None


def _keeps(x, out, save):
    """Refuses an output over the input that backward needs."""
    if not save or out is None or x.numel() == 0 or out.numel() == 0:
        return
    lo = [t.data_ptr() for t in (x, out)]
    hi = [a + (1 + sum((n - 1) * st for n, st in zip(t.shape, t.stride()))) * t.element_size() for a, t in zip(lo, (x, out))]
    if lo[0] < hi[1] and lo[1] < hi[0]:
        row = _row_bytes(x)
        if row and row == _row_bytes(out):     # column slices of one buffer may lie side by side
            at = (lo[1] - lo[0]) % row
            if x.shape[-1] * x.element_size() <= at and at + out.shape[-1] * out.element_size() <= row:
                return
        raise ValueError("out overlaps x, which backward needs: save=True takes another output")


def _saved_tensors(saved):
    """What a forward kept, ready for backward on the current stream: another stream than the forward's, whose pool
    the tensors go back to with the next forward, must have been waited for before they are used again."""
    import torch
    stream = torch.cuda.current_stream()
    made_on, tensors = saved
    if stream != made_on:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
    return tensors


class TileSparseBlock:
    """The attention half of a transformer block: y = residual + gate * (attention(norm, rotation(x w_qkv^T + b_qkv))
    w_out^T + b_out), with its gradient.

    ``layer``: a :class:`TileSparseAttention`. ``w_qkv`` [3 heads head_dim, channels] and ``w_out`` [channels,
    heads head_dim] bf16, biases fp32 or None, ``norm`` a :class:`NormRope`. q, k and v are written by one
    product and read in place by the norm-and-pack pass; with ``layer.direct`` each has its own product and the
    norm runs token-major. ``forward(..., save=True)`` keeps what :meth:`backward` needs (the gradient follows
    the selected tiles as given; not with ``layer.direct``). The packed tiles stay in the layer's buffers, which
    its next forward overwrites: backward refuses then, so blocks that are trained need a layer each. (A replayed
    graph's forward is not noticed: capture a forward and its backward together.) With ``stream`` the whole call, its
    allocations too, is that stream's; a backward on another stream than its forward's waits for that one first, and
    the next forward, which fills the layer's buffers anew, for the backward's (``wait_stream``).
    """

    def __init__(self, layer: TileSparseAttention, w_qkv, w_out, norm: NormRope, b_qkv=None, b_out=None):
        p = layer.plan
        d = p.desc
        width = d.heads * d.head_dim
        if w_qkv.dim() != 2 or w_qkv.shape[0] != 3 * width:
            raise ValueError(f"w_qkv must be [{3 * width}, channels], got {tuple(w_qkv.shape)}")
        if w_out.dim() != 2 or w_out.shape[1] != width:
            raise ValueError(f"w_out must be [channels, {width}], got {tuple(w_out.shape)}")
        _check_bias("b_qkv", b_qkv, 3 * width)
        _check_bias("b_out", b_out, w_out.shape[0])
        self.layer, self.norm = layer, norm
        self.w_qkv, self.b_qkv, self.w_out, self.b_out = w_qkv, b_qkv, w_out, b_out
        self._saved = None

    def forward(self, x, residual=None, gate=None, out=None, save=False, stream=None):
        """x [B, N, channels] bf16, residual [B, N, out channels], gate [B, out channels] fp32 -> y."""
        import torch
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.forward(x, residual, gate, out, save)
        L, b = self.layer, self.layer.bufs
        p = L.plan
        B, N, heads, d = p.shapes()["tokens"]
        if tuple(x.shape) != (B, N, self.w_qkv.shape[1]):
            raise ValueError(f"x must be {(B, N, self.w_qkv.shape[1])}, got {tuple(x.shape)}")
        _keeps(x, out, save)
        if save and L.direct:
            raise ValueError("the direct path keeps no packed tiles: its gradient is not available")
        width = heads * d
        o = _new(x, B, N, heads, d)
        if L.direct:
            q, k, v = (_new(x, B, N, heads, d) for _ in range(3))
            for i, t in enumerate((q, k, v)):
                bias = None if self.b_qkv is None else self.b_qkv[i * width:(i + 1) * width]
                p.linear(x, self.w_qkv[i * width:(i + 1) * width], t.view(B, N, width), bias=bias)
            p.qk_norm_rope(q, k, self.norm, q, k)
            L.stages(q, k, v, o)
            qkv = None
        else:
            qkv = _new(x, B, N, 3, heads, d)
            p.linear(x, self.w_qkv, qkv.view(B, N, 3 * width), bias=self.b_qkv)
            p.tile_norm_rope_pack_pool(qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2], self.norm, b["qp"], b["kp"], b["vp"],
                                       b["workspace"])
            if save and b["lse"] is None:
                b["lse"] = torch.empty(p.shapes()["lse"], dtype=torch.float32, device=x.device)
            L.attend(o)
        y = _new(x, B, N, self.w_out.shape[0]) if out is None else out
        pre = _new(x, B, N, self.w_out.shape[0]) if save and gate is not None else None
        p.linear(o.view(B, N, width), self.w_out, y, bias=self.b_out, gate=gate, residual=residual, pre=pre)
        self._saved = (torch.cuda.current_stream(), (x, qkv, o, gate, pre)) if save else None
        self._run = L.runs
        return y

    __call__ = forward

    def backward(self, dy, stream=None):
        """Gradients of the last ``forward(..., save=True)`` from dy: a dict with "x", "w_qkv", "b_qkv", "w_out",
        "b_out", "gate", "w_q", "w_k" (None where the forward had none); the residual's is dy itself."""
        import torch
        if self._saved is None:
            raise ValueError("backward follows a forward with save=True")
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.backward(dy)
        L, b = self.layer, self.layer.bufs
        if L.runs != self._run:
            raise ValueError("the layer has run again since this block's forward: its tiles are another's")
        x, qkv, o, gate, pre = _saved_tensors(self._saved)
        p = L.plan
        B, N, heads, d = p.shapes()["tokens"]
        width, f32 = heads * d, torch.float32
        samples = gate.shape[0] if gate is not None else 0
        g = {"x": torch.empty_like(x), "w_qkv": torch.empty_like(self.w_qkv), "w_out": torch.empty_like(self.w_out),
             "b_qkv": None if self.b_qkv is None else torch.empty_like(self.b_qkv),
             "b_out": None if self.b_out is None else torch.empty_like(self.b_out),
             "gate": None if gate is None else torch.empty_like(gate),
             "w_q": None if self.norm.w_q is None else torch.empty_like(self.norm.w_q),
             "w_k": None if self.norm.w_k is None else torch.empty_like(self.norm.w_k)}
        rows = B * N
        ws = _workspace(x, max(p.linear_bwd_workspace_bytes(rows, width, self.w_out.shape[0], samples),
                               p.linear_bwd_workspace_bytes(rows, x.shape[2], 3 * width),
                               p.attn_bwd_workspace_bytes(), p.norm_bwd_workspace_bytes()))
        do = torch.empty_like(o)
        p.linear_bwd(dy, o.view(B, N, width), self.w_out, dx=do.view(B, N, width), dw=g["w_out"], pre=pre, gate=gate,
                     dbias=g["b_out"], dgate=g["gate"], workspace=ws)
        packed = p.shapes()["packed"]
        dop, dqp, dkp, dvp = (_new(x, *packed) for _ in range(4))
        p.tile_pack(do, None, None, dop, None, None)
        args = (b["qp"], b["kp"], b["vp"], b["op"], b["lse"], dop, b["idx"])
        if p.info.n_ref_tiles:
            p.sparse_attn_ref_bwd(*args, b["idx_ref"], dqp, dkp, dvp, ws)
        else:
            p.sparse_attn_bwd(*args, dqp, dkp, dvp, ws)
        dqkv = torch.empty_like(qkv)
        p.tile_norm_rope_bwd(dqp, dkp, dvp, qkv[:, :, 0], qkv[:, :, 1], self.norm, dqkv[:, :, 0], dqkv[:, :, 1],
                             dqkv[:, :, 2], g["w_q"], g["w_k"], ws)
        p.linear_bwd(dqkv.view(B, N, 3 * width), x, self.w_qkv, dx=g["x"], dw=g["w_qkv"], dbias=g["b_qkv"],
                     workspace=ws)
        return g


class FeedForward:
    """The other half of the block: y = residual + gate * (act(x w_up^T + b_up) w_down^T + b_down), with its gradient.
    ``plan`` names the device; weights bf16, biases and gate [samples, channels] fp32 (or None). A backward on another
    stream than its forward's waits for that one first (``wait_stream``); the next forward need not wait for it."""

    def __init__(self, plan: Plan, w_up, w_down, b_up=None, b_down=None, act="gelu_tanh"):
        if w_up.dim() != 2 or w_down.dim() != 2 or w_up.shape[0] != w_down.shape[1]:
            raise ValueError(f"w_up {tuple(w_up.shape)} and w_down {tuple(w_down.shape)} do not follow each other")
        _check_bias("b_up", b_up, w_up.shape[0])
        _check_bias("b_down", b_down, w_down.shape[0])
        self.plan, self.act = plan, act
        self.w_up, self.b_up, self.w_down, self.b_down = w_up, b_up, w_down, b_down
        self._saved = None

    def forward(self, x, residual=None, gate=None, out=None, save=False, stream=None):
        import torch
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.forward(x, residual, gate, out, save)
        _keeps(x, out, save)
        p, lead = self.plan, x.shape[:-1]
        h = _new(x, *lead, self.w_up.shape[0])
        hidden = _new(x, *lead, self.w_up.shape[0]) if save else None
        p.linear(x, self.w_up, h, bias=self.b_up, act=self.act, pre=hidden)
        y = _new(x, *lead, self.w_down.shape[0]) if out is None else out
        pre = _new(x, *lead, self.w_down.shape[0]) if save and gate is not None else None
        p.linear(h, self.w_down, y, bias=self.b_down, gate=gate, residual=residual, pre=pre)
        self._saved = (torch.cuda.current_stream(), (x, hidden, h, gate, pre)) if save else None
        return y

    __call__ = forward

    def backward(self, dy, stream=None):
        """Gradients of the last ``forward(..., save=True)``: "x", "w_up", "b_up", "w_down", "b_down", "gate"."""
        import torch
        if self._saved is None:
            raise ValueError("backward follows a forward with save=True")
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.backward(dy)
        x, hidden, h, gate, pre = _saved_tensors(self._saved)
        p = self.plan
        like = lambda t: None if t is None else torch.empty_like(t)
        g = {"x": torch.empty_like(x), "w_up": torch.empty_like(self.w_up), "w_down": torch.empty_like(self.w_down),
             "b_up": like(self.b_up), "b_down": like(self.b_down), "gate": like(gate)}
        rows, n_mid, n_out = x.numel() // x.shape[-1], self.w_up.shape[0], self.w_down.shape[0]
        ws = _workspace(x, max(p.linear_bwd_workspace_bytes(rows, n_mid, n_out, gate.shape[0] if gate is not None else 0),
                               p.linear_bwd_workspace_bytes(rows, x.shape[-1], n_mid)))
        dh = torch.empty_like(h)
        p.linear_bwd(dy, h, self.w_down, dx=dh, dw=g["w_down"], pre=pre, gate=gate, dbias=g["b_down"], dgate=g["gate"],
                     workspace=ws)
        p.linear_bwd(dh, x, self.w_up, dx=g["x"], dw=g["w_up"], act=self.act, pre=hidden, dbias=g["b_up"], workspace=ws)
        return g


__all__ = ["TileSparseAttention", "TileSparseBlock", "FeedForward", "axial_rope_table", "NormRope", "Plan", "make_desc",
           "k_from_sparsity"]
