"""The gradient of the tile-sparse attention against the fp64 oracle.

Both sides take P from the same lse (fp32) and delta from the same o (bf16). Per element: P and dS are
rounded to bf16 for their products, half a step each, so 2^-8 of the sum of |terms| (the oracle's bound) and
the fp32 accumulation of dP and delta (the oracle's second bound, which is all there is where a row's only
key makes dS zero: dP and delta are then the same sum in two orders); the exponent is an fp32 product of |s log2 e| < 64
with its own rounding, so 2^-16 of the same sum covers it and the accumulation; the result's rounding is
2^-8 of the value. The roundings are independent, so the norms are held to 2^-7 and the second bound's.
"""
import numpy as np
import pytest

import oracle.block_oracle as BO
import oracle.vsa_oracle as O
from gpu_util import bf16_to_f64, n_video_tiles, no_prefix_config, r2va_gpu_config, ragged_gpu_config
from vsa_synth import LayerConfig, get_config

pytestmark = pytest.mark.gpu


def long_rows_config(d=128):
    """Odd grid, many tiles: lists of several words, odd list lengths, three query tiles past a multiple of 32."""
    return LayerConfig(name="words", batch=1, heads=2, head_dim=d, T=9, H=18, W=23, segments=(65, 1),
                       tile_shapes=((4, 4, 4), (1, 8, 8)), score_mode="meanpool_gate", proj_dim=d, sparsity=(0.5,),
                       seed=4)


CONFIGS = {"ragged128": lambda: ragged_gpu_config(128, batch=2), "ragged64": lambda: ragged_gpu_config(64),
           "noprefix": no_prefix_config, "tiny": lambda: get_config("tiny"), "words128": lambda: long_rows_config(128),
           "words64": lambda: long_rows_config(64),
           "one": lambda: LayerConfig(name="one", batch=1, heads=1, head_dim=128, T=1, H=1, W=1, segments=(),
                                      tile_shapes=((4, 4, 4),), score_mode="meanpool_gate", proj_dim=128,
                                      sparsity=(0.0,), seed=9)}


class Case:
    def __init__(self, cfg, k_per_head, seed=0, with_ref=False, spread=1.0):
        import torch
        import tile_sparse_video_pack_b200 as T
        self.cfg, self.k = cfg, k_per_head
        rng = np.random.default_rng(seed)
        self.plan = p = T.Plan.from_config(cfg, 0.5, k_per_head=k_per_head)
        shape = (cfg.batch, cfg.n_tokens, cfg.heads, cfg.head_dim)
        tok = [torch.tensor(rng.normal(size=shape) * (spread if i < 2 else 1)).to(torch.bfloat16).cuda() for i in range(4)]
        self.f = [bf16_to_f64(t) for t in tok]
        self.kept = [[[np.sort(rng.choice(n_video_tiles(cfg, h), size=k_per_head[h], replace=False))
                       for _ in range(n_video_tiles(cfg, h))] for h in range(cfg.heads)] for _ in range(cfg.batch)]
        idx = np.zeros(p.shapes()["idx"], dtype=np.int32)
        for b in range(cfg.batch):
            for h in range(cfg.heads):
                idx[b, h, :n_video_tiles(cfg, h), :k_per_head[h]] = np.stack(self.kept[b][h])
        self.idx = torch.tensor(idx).cuda()
        self.kept_ref = self.idx_ref = None
        if with_ref:
            n_ref = p.info.n_ref_tiles
            self.kept_ref = [[[np.sort(rng.choice(n_ref, size=cfg.k_ref, replace=False))
                               for _ in range(n_video_tiles(cfg, h))] for h in range(cfg.heads)] for _ in range(cfg.batch)]
            ir = np.zeros(p.shapes()["idx_ref"], dtype=np.int32)
            for b in range(cfg.batch):
                for h in range(cfg.heads):
                    ir[b, h, :n_video_tiles(cfg, h), :cfg.k_ref] = np.stack(self.kept_ref[b][h])
            self.idx_ref = torch.tensor(ir).cuda()
        new = lambda: torch.empty(p.shapes()["packed"], dtype=torch.bfloat16, device="cuda")
        self.pk = [new() for _ in range(4)]                       # q, k, v, do
        p.tile_pack(*tok[:3], *self.pk[:3])
        p.tile_pack(tok[3], None, None, self.pk[3], None, None)
        # the forward's outputs: by the framework's own forward
        self.op = torch.zeros_like(self.pk[0])
        self.lse = torch.zeros(p.shapes()["lse"], dtype=torch.float32, device="cuda")
        if with_ref:
            p.sparse_attn_ref(*self.pk[:3], self.idx, self.idx_ref, self.op, self.lse)
        else:
            p.sparse_attn(*self.pk[:3], self.idx, self.op, self.lse)
        self.grads = [torch.full_like(self.pk[0], 7) for _ in range(3)]
        self.ws = torch.empty(p.attn_bwd_workspace_bytes(), dtype=torch.uint8, device="cuda")
        p.check()

    def run(self, k_per_head=None):
        if self.idx_ref is not None:
            self.plan.sparse_attn_ref_bwd(*self.pk[:3], self.op, self.lse, self.pk[3], self.idx, self.idx_ref, *self.grads,
                                          self.ws, k_per_head=k_per_head)
        else:
            self.plan.sparse_attn_bwd(*self.pk[:3], self.op, self.lse, self.pk[3], self.idx, *self.grads, self.ws,
                                      k_per_head=k_per_head)

    def check(self):
        cfg = self.cfg
        lse_p = self.lse.double().cpu().numpy()
        lse = O.unpack(lse_p[..., None], cfg)[..., 0]
        o = O.unpack(bf16_to_f64(self.op), cfg)
        out = BO.attention_grad(cfg, *self.f, self.kept, self.kept_ref, lse=lse, o=o, bound=True)
        for name, got, want, bound, fp32 in zip(("dq", "dk", "dv"), self.grads, out[:3], out[5:8], out[8:]):
            g = bf16_to_f64(got)
            wp, counts = O.pack(want, cfg)
            bp, fp = O.pack(bound, cfg)[0], O.pack(fp32, cfg)[0]
            err = np.abs(g - wp)
            tol = (2.0 ** -8 + 2.0 ** -16) * bp + fp + 2.0 ** -8 * np.abs(wp)     # 0 in unused slots and tiles
            assert np.all(err <= tol), (name, np.max(err / np.maximum(tol, 1e-30)))
            assert np.linalg.norm(err) <= 2.0 ** -7 * np.linalg.norm(wp) + np.linalg.norm(fp), name


@pytest.mark.parametrize("share", ["one", "half", "all"])
@pytest.mark.parametrize("name", sorted(CONFIGS))
def test_gradient(name, share):
    import torch
    cfg = CONFIGS[name]()
    n = [n_video_tiles(cfg, h) for h in range(cfg.heads)]
    c = Case(cfg, {"one": [1] * cfg.heads, "half": [max(1, x // 2) for x in n], "all": n}[share])
    c.run()
    c.plan.check()
    c.check()
    first = [g.clone() for g in c.grads]
    c.ws.fill_(255)                          # nothing is kept in the workspace between calls
    c.run()
    c.plan.check()
    assert all(torch.equal(a, b) for a, b in zip(first, c.grads))


@pytest.mark.parametrize("d", [64, 128])
def test_reference_budgets(d):
    cfg = r2va_gpu_config(d)
    c = Case(cfg, [max(1, n_video_tiles(cfg, h) // 2) for h in range(cfg.heads)], with_ref=True)
    c.run()
    c.plan.check()
    c.check()


def test_sharp_softmax():
    """Logits of tens: rows with one dominant key and many that underflow."""
    cfg = ragged_gpu_config(128)
    c = Case(cfg, [2] * cfg.heads, spread=3.0)
    c.run()
    c.plan.check()
    c.check()


def test_smaller_k_than_the_plan():
    cfg = ragged_gpu_config(128)
    c = Case(cfg, [4, 2, 4, 4])
    k = [2, 1, 3, 4]
    c.plan.sparse_attn(*c.pk[:3], c.idx, c.op, c.lse, k_per_head=k)
    c.kept = [[[row[:k[h]] for row in c.kept[b][h]] for h in range(cfg.heads)] for b in range(cfg.batch)]
    c.run(k_per_head=k)
    c.plan.check()
    c.check()


def test_bad_list_is_reported_and_left_out():
    """A list that is not ascending or out of range latches the error; its query tile has no gradient and takes
    no part in the others', which stay right."""
    import torch
    import tile_sparse_video_pack_b200 as T
    cfg = get_config("tiny")
    c = Case(cfg, [2, 2])
    for bad in ([3, 1], [1, 1], [2, 4], [-1, 2]):
        keep = c.idx[0, 1, 2].clone()
        c.idx[0, 1, 2] = torch.tensor(bad, dtype=torch.int32)
        c.run()
        with pytest.raises(T.VsaError, match="BAD_INDEX"):
            c.plan.check()
        c.idx[0, 1, 2] = keep
        dq = c.grads[0]
        assert torch.all(dq[0, 1, 2 + 2] == 0) and torch.all(torch.isfinite(torch.stack(c.grads).float()))
        assert torch.any(dq[0, 0, 4] != 0)
    c.run()
    c.plan.check()
    c.check()


def test_medium_layer_sampled_rows():
    """The medium clip, two heads: the whole gradient."""
    cfg = get_config("medium").with_(heads=2, tile_shapes=((4, 4, 4), (2, 4, 8)))
    c = Case(cfg, [30, 30])
    c.run()
    c.plan.check()
    c.check()


def test_timeout_is_reported():
    """A wait limit of a microsecond runs out: the call returns, check reports it, and the next call is right."""
    import tile_sparse_video_pack_b200 as T
    cfg = ragged_gpu_config(128)
    c = Case(cfg, [2] * cfg.heads)
    c.plan.set_wait_limit(1000)
    c.run()
    try:
        c.plan.check()
    except T.VsaError as e:
        assert "TIMEOUT" in str(e)
    c.plan.set_wait_limit(0)
    c.run()
    c.plan.check()
    c.check()


def test_refusals():
    import torch
    import tile_sparse_video_pack_b200 as T
    cfg = ragged_gpu_config(128)
    c = Case(cfg, [2] * cfg.heads)
    p = c.plan
    good = [*c.pk[:3], c.op, c.lse, c.pk[3], c.idx, *c.grads, c.ws]
    for i, wrong in ((0, c.pk[0].float()), (4, c.lse.double()), (6, c.idx.long())):
        with pytest.raises(TypeError):
            p.sparse_attn_bwd(*good[:i], wrong, *good[i + 1:])
    for i in (0, 4, 6, 8, 10):
        with pytest.raises(ValueError):
            p.sparse_attn_bwd(*good[:i], good[i].view(-1)[:-1], *good[i + 1:])
    with pytest.raises(T.VsaError):
        p.sparse_attn_bwd(*good, k_per_head=[3] * cfg.heads)
    with pytest.raises(T.VsaError):
        p.sparse_attn_bwd(*good, k_per_head=[0] * cfg.heads)
    big = torch.empty(c.ws.numel() + 256, dtype=torch.uint8, device="cuda")
    with pytest.raises(T.VsaError):
        p.sparse_attn_bwd(*good[:-1], big[16:16 + c.ws.numel()])
    with pytest.raises(T.VsaError):          # no reference segments in this plan
        p.sparse_attn_ref_bwd(*good[:7], torch.zeros(0, dtype=torch.int32, device="cuda"), *good[7:])
    p.check()
