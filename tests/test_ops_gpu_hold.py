"""The wait limit of the products and of the attention's gradient, run out on purpose and without a fault: with the plan's
test hold, warps wait on a barrier nothing arrives on. The call must end near the limit, the status must reach the
host, and the next call on the same plan, hold off, must be right.
"""
import pytest

import tile_sparse_video_pack_b200 as T
from gpu_util import ragged_gpu_config
from test_ops_gpu_attn_bwd import Case, long_rows_config
from test_ops_gpu_linear import check_backward, check_forward, tensors, workspace

pytestmark = pytest.mark.gpu
LIMIT = 20_000_000
NONE = dict(bias=False, gate=False, residual=False)


def runs_out(plan, call):
    import torch
    t0, t1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    plan.set_wait_limit(LIMIT)
    plan.set_test_hold(True)
    t0.record()
    call()
    t1.record()
    with pytest.raises(T.VsaError) as e:
        plan.check()
    assert e.value.status == 4                        # VSA_ERR_DEVICE_TIMEOUT
    assert t0.elapsed_time(t1) < 1000.0               # near the short limit, not the default
    plan.set_test_hold(False)
    plan.set_wait_limit(0)
    call()
    plan.check()


def tiling(plan, M, N):
    """Which kernel a product of this size takes on this device (linear.cu's use_pairs and run_products)."""
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    up = lambda a, b: -(-a // b)
    units = lambda n: up(M, 128) * up(N, n)
    if 11 * up(up(M, 256) * up(N, 256), sms // 2) < 10 * up(units(128), sms):
        return "pairs"
    return "128x128" if units(64) > sms else "clusters" if units(64) * 2 <= sms * 9 // 10 else "128x64"


@pytest.mark.parametrize("M,K,N,kind", [(64, 2048, 128, "clusters"), (1000, 256, 1024, "128x64"),
                                        (1000, 64, 2048, "128x128"), (1000, 1024, 2048, "128x128"),
                                        (3000, 1024, 1304, "pairs"), (7000, 64, 1304, "pairs")])
def test_linear(M, K, N, kind):
    """K of 64: one k block to a tile, so that the producer has left long before the limit."""
    import torch
    plan = T.Plan(T.make_desc(1, 1, 64, 1, 8, 8, [], [(4, 4, 4)], [1]))
    assert tiling(plan, M, N) == kind
    t = tensors(M, K, N, 1)
    y = torch.zeros_like(t["residual"])
    runs_out(plan, lambda: plan.linear(t["x"], t["w"], y))
    check_forward(t, y, None, "none", NONE)


def test_linear_gradient():
    import torch
    plan = T.Plan(T.make_desc(1, 1, 64, 1, 8, 8, [], [(4, 4, 4)], [1]))
    M, K, N = 1000, 264, 1024
    t = tensors(M, K, N, 1, seed=1)
    pre = tensors(M, K, N, 1, seed=2)["residual"]
    out = dict(dx=torch.zeros_like(t["x"]), dw=torch.zeros_like(t["w"]), dbias=torch.zeros_like(t["bias"]))
    ws = workspace(plan, M, K, N)
    runs_out(plan, lambda: plan.linear_bwd(t["dy"], t["x"], t["w"], act="silu", pre=pre, workspace=ws, **out))
    check_backward(t, out, "silu", pre, False)


@pytest.mark.parametrize("name", ["ragged64", "ragged128", "words128"])
def test_attention_gradient(name):
    cfg = {"ragged64": lambda: ragged_gpu_config(64), "ragged128": lambda: ragged_gpu_config(128, batch=2),
           "words128": lambda: long_rows_config(128)}[name]()
    c = Case(cfg, [2] * cfg.heads)
    runs_out(c.plan, c.run)
    c.check()


def test_linear_of_few_rows_has_no_waits():
    import torch
    plan = T.Plan(T.make_desc(1, 1, 64, 1, 8, 8, [], [(4, 4, 4)], [1]))
    t = tensors(16, 64, 128, 1)
    y = torch.zeros_like(t["residual"])
    plan.set_test_hold(True)
    plan.linear(t["x"], t["w"], y)
    plan.check()
    check_forward(t, y, None, "none", NONE)
