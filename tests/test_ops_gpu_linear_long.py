"""A weight gradient over so many rows that one CTA's sum takes longer than the wait limit: the limit bounds a wait for the
next 64 rows, not the length of the sum.

Entries are -1, 0 and 1, so that every partial sum is a whole number below 2^24 and exact in fp32: the result is the
exact sum, rounded once.
"""
import pytest

import tile_sparse_video_pack_b200 as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,with_dx", [((1 << 22) + 40, True), ((1 << 23) - 8, False)])
def test_a_long_sum_outlasts_the_limit(rows, with_dx):
    import torch
    plan = T.Plan(T.make_desc(1, 1, 64, 1, 8, 8, [], [(4, 4, 4)], [1]))
    g = torch.Generator(device="cuda").manual_seed(3)
    new = lambda: torch.randint(-1, 2, (rows, 8), generator=g, device="cuda").to(torch.bfloat16)
    dy, x = new(), new()
    w = torch.randint(-1, 2, (8, 8), generator=g, device="cuda").to(torch.bfloat16)
    dw = torch.full((8, 8), 7.0, dtype=torch.bfloat16, device="cuda")
    dx = torch.full_like(x, 7.0) if with_dx else None
    ws = torch.empty(plan.linear_bwd_workspace_bytes(rows, 8, 8), dtype=torch.uint8, device="cuda")
    plan.linear_bwd(dy, x, w, dx=dx, dw=dw, workspace=ws)       # warm
    plan.check()
    t0, t1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    plan.set_wait_limit(500_000)
    t0.record()
    plan.linear_bwd(dy, x, w, dx=dx, dw=dw, workspace=ws)
    t1.record()
    plan.check()
    assert t0.elapsed_time(t1) > 1.0                            # ms: more than the limit, so the case tests something
    assert torch.equal(dw, (dy.double().T @ x.double()).to(torch.bfloat16))
    if with_dx:
        assert torch.equal(dx, (dy.float() @ w.float()).to(torch.bfloat16))
