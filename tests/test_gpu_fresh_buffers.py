"""A layer's buffers do not depend on what the memory held before: entries past a head's own tiles, which the calls
leave unwritten, are zero."""
import pytest

from gpu_util import LayerRun, n_video_tiles, r2va_gpu_config, ragged_gpu_config

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ref", [False, True])
def test_entries_past_a_heads_own_tiles_are_zero(ref):
    import torch
    cfg = r2va_gpu_config() if ref else ragged_gpu_config()
    names = ["scores", "idx", "op", "lse"] + (["scores_ref", "idx_ref"] if ref else [])
    sizes = [b.numel() * b.element_size() for b in LayerRun(cfg, 0.5).bufs.values() if b is not None]
    torch.cuda.synchronize()
    used = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    torch.cuda.synchronize()
    del used                             # the allocator hands these out next, as they are
    r = LayerRun(cfg, 0.5)
    if not ref:
        r.bufs = r.plan.allocate(with_lse=True)
    r.run(fused=True)
    n_pre = r.plan.info.n_prefix_tiles
    n = [n_video_tiles(cfg, h) for h in range(cfg.heads)]
    assert min(n) < max(n)
    for name in names:
        for h in range(cfg.heads):
            past = r.bufs[name][:, h, (n_pre if name in ("op", "lse") else 0) + n[h]:]
            assert not past.any(), (name, h)
            if name == "scores":
                assert not r.bufs[name][:, h, :, n[h]:].any(), h
