"""The operators together, as a transformer block runs them: projection, norm + rotation + pack, score, select,
attention, unpack, output projection with gate and residual -- and back -- against fp64.

The kept tiles are the GPU's own. Tolerance: the chain rounds qkv, the normed q and k, P, o and y (backward: do,
P, dS, the packed gradients, dqkv and the results) to bf16, each by at most 2^-8 / sqrt(3) rms of its value.
A rounding before the softmax moves a logit |s| < 8 by at most 8 * 2 * 2^-8 / sqrt(3) = 0.036, and with it a
weight P by that share in the worst row; ten independent contributions of up to 0.036 / sqrt(10) rms of the
result each stay below 2^-4 / 2 of its norm: 2^-5.
"""
import numpy as np
import pytest

import oracle.vsa_oracle as O
from gpu_util import bf16_to_f64, n_video_tiles, r2va_gpu_config, ragged_gpu_config
from vsa_synth import get_config

pytestmark = pytest.mark.gpu

REL = 2.0 ** -5


def f64(t):
    import torch
    return None if t is None else t.detach().double().cpu()


class Block:
    def __init__(self, cfg, channels=192, gate=True, layout="interleaved", direct=False, seed=0):
        import torch
        import tile_sparse_video_pack_b200 as T
        self.cfg = cfg
        g = torch.Generator().manual_seed(seed)
        bf = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(torch.bfloat16).cuda()
        f32 = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).cuda()
        d, W = cfg.head_dim, cfg.heads * cfg.head_dim
        self.x = bf(cfg.batch, cfg.n_tokens, channels)
        self.residual, self.dy = bf(*self.x.shape), bf(*self.x.shape)
        self.gate = f32(cfg.batch, channels) if gate else None
        if cfg.score_mode == "tripool":
            proj = [f32(cfg.heads, 3 * d, cfg.proj_dim, scale=(3 * d) ** -0.5) for _ in range(2)]
        else:
            proj = [f32(d, d, scale=d ** -0.5)] * 2
        self.layer = T.TileSparseAttention.from_config(cfg, 0.5, *proj, direct=direct)
        cos, sin = T.axial_rope_table(self.layer.plan)
        norm = T.NormRope(1 + f32(d, scale=0.2), 1 + f32(d, scale=0.2), cos, sin, layout=layout)
        self.block = T.TileSparseBlock(self.layer, bf(3 * W, channels, scale=channels ** -0.5),
                                       bf(channels, W, scale=W ** -0.5), norm, f32(3 * W, scale=0.1),
                                       f32(channels, scale=0.1))
        if self.layer.bufs["op"] is not None:
            self.layer.bufs["op"].zero_()

    def run(self, save=False, **kw):
        y = self.block(self.x, residual=self.residual, gate=self.gate, save=save, **kw)
        self.layer.plan.check()
        return y

    def reference(self):
        """fp64 autograd of the same block with the GPU's kept tiles: (y, leaves)."""
        import torch
        cfg, blk = self.cfg, self.block
        leaves = {k: f64(v).requires_grad_() for k, v in
                  dict(x=self.x, w_qkv=blk.w_qkv, b_qkv=blk.b_qkv, w_out=blk.w_out, b_out=blk.b_out, w_q=blk.norm.w_q,
                       w_k=blk.norm.w_k).items()}
        if self.gate is not None:
            leaves["gate"] = f64(self.gate).requires_grad_()
        B, N, Hh, d = cfg.batch, cfg.n_tokens, cfg.heads, cfg.head_dim
        qkv = (leaves["x"] @ leaves["w_qkv"].T + leaves["b_qkv"]).view(B, N, 3, Hh, d)
        turn = torch.complex(f64(blk.norm.cos), f64(blk.norm.sin))[None, :, None]

        def normed(t, w):
            n = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + blk.norm.eps) * w
            if blk.norm.layout == "halves":
                z = torch.complex(n[..., :d // 2], n[..., d // 2:]) * turn
                return torch.cat([z.real, z.imag], -1)
            z = torch.complex(n[..., 0::2], n[..., 1::2]) * turn
            return torch.stack([z.real, z.imag], -1).flatten(-2)

        q, k, v = normed(qkv[:, :, 0], leaves["w_q"]), normed(qkv[:, :, 1], leaves["w_k"]), qkv[:, :, 2]
        ref = O.ref_tiles(cfg) if any(cfg.seg_ref) else None
        heads = []
        for h in range(Hh):
            til = O.head_tiling(cfg, h)
            per_b = []
            for b in range(B):
                allowed = torch.zeros(N, N, dtype=torch.bool)
                for n, rows in enumerate(til.all):
                    i = n - til.n_prefix
                    kh = self.layer.plan.k_per_head[h]
                    kept = [] if i < 0 else self.layer.bufs["idx"][b, h, i, :kh].cpu().numpy()
                    kr = None if ref is None or i < 0 else self.layer.bufs["idx_ref"][b, h, i, :cfg.k_ref].cpu().numpy()
                    keys = O.query_key_tokens(til, n, kept) if ref is None else \
                        O.query_key_tokens(til, n, kept, ref, [] if kr is None else kr)
                    allowed[np.ix_(rows, keys)] = True
                s = (q[b, :, h] @ k[b, :, h].T / d ** 0.5).masked_fill(~allowed, -torch.inf)
                per_b.append(torch.softmax(s, -1) @ v[b, :, h])
            heads.append(torch.stack(per_b))
        o = torch.stack(heads, 2).reshape(B, N, Hh * d)
        y = o @ leaves["w_out"].T + leaves["b_out"]
        if self.gate is not None:
            y = y * leaves["gate"][:, None]
        return y + f64(self.residual), leaves


def near(got, want, what):
    err = float((f64(got) - want).norm() / want.norm())
    assert err <= REL, (what, err)


CONFIGS = {"ragged128": lambda: ragged_gpu_config(128, batch=2), "ragged64_trip": lambda: ragged_gpu_config(64, "tripool"),
           "r2va": lambda: r2va_gpu_config(128), "tiny": lambda: get_config("tiny")}


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("layout", ["interleaved", "halves"])
@pytest.mark.parametrize("name", sorted(CONFIGS))
def test_block_forward_and_backward(name, layout, gate):
    c = Block(CONFIGS[name](), gate=gate, layout=layout)
    y = c.run(save=True)
    want, leaves = c.reference()
    near(y, want.detach(), "y")
    want.backward(f64(c.dy))
    g = c.block.backward(c.dy)
    c.layer.plan.check()
    for k, t in leaves.items():
        near(g[k], t.grad, k)
    assert gate or g["gate"] is None


@pytest.mark.parametrize("d", [64, 128])
def test_direct_block_equals_packed_block(d):
    """The direct path (own products, token-major norm) gives the packed path's bits."""
    import torch
    a, b = Block(ragged_gpu_config(d)), Block(ragged_gpu_config(d), direct=True)
    assert torch.equal(a.run(), b.run())
    with pytest.raises(ValueError):
        b.run(save=True)
    with pytest.raises(ValueError):
        a.block.backward(a.dy)               # the last forward saved nothing


def test_feed_forward():
    import torch
    import tile_sparse_video_pack_b200 as T
    plan = T.Plan(T.make_desc(1, 1, 64, 1, 8, 8, [], [(4, 4, 4)], [1]))
    g = torch.Generator().manual_seed(5)
    bf = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(torch.bfloat16).cuda()
    f32 = lambda *s: (torch.randn(*s, generator=g) * 0.3).cuda()
    x, res, dy = bf(2, 77, 192), bf(2, 77, 192), bf(2, 77, 192)
    gate, bu, bd = f32(2, 192), f32(520), f32(192)
    wu, wd = bf(520, 192, scale=192 ** -0.5), bf(192, 520, scale=520 ** -0.5)
    ff = T.FeedForward(plan, wu, wd, bu, bd)
    y = ff(x, residual=res, gate=gate, save=True)
    grads = ff.backward(dy)
    plan.check()
    leaves = {k: f64(v).requires_grad_() for k, v in dict(x=x, w_up=wu, b_up=bu, w_down=wd, b_down=bd, gate=gate).items()}
    h = torch.nn.functional.gelu(leaves["x"] @ leaves["w_up"].T + leaves["b_up"], approximate="tanh")
    want = f64(res) + leaves["gate"][:, None] * (h @ leaves["w_down"].T + leaves["b_down"])
    near(y, want.detach(), "y")
    want.backward(f64(dy))
    for k, t in leaves.items():
        near(grads[k], t.grad, k)


def test_block_on_a_stream_and_in_a_graph():
    """Forward and backward on a side stream, then captured and replayed: the same bits, and new inputs in the
    same buffers are followed."""
    import torch
    c = Block(ragged_gpu_config(128))
    y0 = c.run(save=True)
    g0 = c.block.backward(c.dy)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y1 = c.block(c.x, residual=c.residual, gate=c.gate, save=True)
        g1 = c.block.backward(c.dy)
        graph = torch.cuda.CUDAGraph()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            y2 = c.block(c.x, residual=c.residual, gate=c.gate, save=True)
            g2 = c.block.backward(c.dy)
    torch.cuda.synchronize()
    for _ in range(3):
        graph.replay()
    c.layer.plan.check()
    assert torch.equal(y0, y1) and torch.equal(y0, y2)
    for k, t in g0.items():
        assert torch.equal(t, g1[k]) and torch.equal(t, g2[k]), k
    c.x.copy_(c.x.flip(1))
    c.dy.mul_(2)
    graph.replay()
    c.layer.plan.check()
    y3 = c.run(save=True)
    g3 = c.block.backward(c.dy)
    c.layer.plan.check()
    assert torch.equal(y2, y3)
    for k, t in g3.items():
        assert torch.equal(t, g2[k]), k


def test_stream_argument_and_shared_layer():
    """stream=: the call's own allocations are that stream's; a layer that has run again refuses the older backward."""
    import torch
    c = Block(ragged_gpu_config(128))
    want = c.run(save=True)
    g0 = c.block.backward(c.dy)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        y = c.block(c.x, residual=c.residual, gate=c.gate, save=True, stream=s)
        g1 = c.block.backward(c.dy, stream=s)
        torch.empty(1 << 20, device="cuda").fill_(7)      # the current stream's allocations meanwhile
    c.layer.plan.check()
    assert torch.equal(want, y) and all(torch.equal(t, g1[k]) for k, t in g0.items())
    q = torch.randn(*c.layer.plan.shapes()["tokens"], device="cuda").to(torch.bfloat16)
    c.layer(q, q, q)
    with pytest.raises(ValueError, match="run again"):
        c.block.backward(c.dy)
    c.layer.plan.check()


def test_two_plans_on_two_streams():
    """Blocks with a plan each, at once on two streams: each gives what it gives alone."""
    import torch
    blocks = [Block(ragged_gpu_config(128), seed=i) for i in range(2)]
    alone = []
    for c in blocks:
        y = c.run(save=True)
        alone.append((y, c.block.backward(c.dy)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    both = [None, None]
    for _ in range(5):
        for i, (c, s) in enumerate(zip(blocks, streams)):
            with torch.cuda.stream(s):
                both[i] = (c.block(c.x, residual=c.residual, gate=c.gate, save=True), c.block.backward(c.dy))
    torch.cuda.synchronize()
    for c, (y, g), (y1, g1) in zip(blocks, alone, both):
        c.layer.plan.check()
        assert torch.equal(y, y1)
        for k, t in g.items():
            assert torch.equal(t, g1[k]), k


def test_rope_table():
    import torch
    import oracle.block_oracle as BO
    import tile_sparse_video_pack_b200 as T
    cfg = ragged_gpu_config(128)
    plan = T.Plan.from_config(cfg, 0.5)
    for split in (None, (20, 22, 22), (64, 0, 0)):
        cos, sin = T.axial_rope_table(plan, split=split)
        a = BO.rope_angles(cfg.T, cfg.H, cfg.W, cfg.n_prefix_tokens, 64, split=split)
        assert np.abs(cos.double().cpu().numpy() - np.cos(a)).max() <= 2.0 ** -24
        assert np.abs(sin.double().cpu().numpy() - np.sin(a)).max() <= 2.0 ** -24
    with pytest.raises(ValueError):
        T.axial_rope_table(plan, split=(1, 2, 3))


def test_block_refusals():
    import torch
    import tile_sparse_video_pack_b200 as T
    c = Block(get_config("tiny"))
    with pytest.raises(ValueError):
        c.block(c.x[:, :-1])
    with pytest.raises(ValueError):
        T.TileSparseBlock(c.layer, c.block.w_qkv[:-1], c.block.w_out, c.block.norm)
    with pytest.raises(ValueError):
        T.TileSparseBlock(c.layer, c.block.w_qkv, c.block.w_out[:, :-8], c.block.norm)
    with pytest.raises(ValueError):
        T.FeedForward(c.layer.plan, c.block.w_out, c.block.w_out)


def test_output_over_the_input():
    """Without save the residual's x may be written over; backward's x may not."""
    import torch
    import tile_sparse_video_pack_b200 as T
    c = Block(get_config("tiny"))
    x, channels = c.x, c.x.shape[2]
    g = torch.Generator().manual_seed(6)
    w_out = (torch.randn(channels, c.block.w_out.shape[1], generator=g) * 0.05).to(torch.bfloat16).cuda()
    w_up = (torch.randn(264, channels, generator=g) * 0.05).to(torch.bfloat16).cuda()
    block = T.TileSparseBlock(c.layer, c.block.w_qkv, w_out, c.block.norm)
    for part in (block, T.FeedForward(c.layer.plan, w_up, w_up.t().contiguous())):
        with pytest.raises(ValueError):
            part(x, residual=x, out=x, save=True)
        want = part(x, residual=x)
        over = x.clone()
        assert part(over, residual=over, out=over) is over
        c.layer.plan.check()
        assert torch.equal(over, want)
        both = torch.empty(2, *x.shape, dtype=torch.bfloat16, device="cuda")   # neighbours in one buffer are taken
        both[0].copy_(x)
        assert torch.equal(part(both[0], residual=both[0], out=both[1], save=True), want)
