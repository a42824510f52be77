"""The linear layer's activations far out: pre-activations whose square is infinite in fp32, infinities and NaN.

Expected from the definitions: z or 0 (exact: z is a bf16 value times 1, its sigmoid 1 or 0), a derivative of 1 or 0.
At -infinity the products z * 0 of both definitions are NaN, as PyTorch's are. Ordinary pre-activations among
them keep the tolerances of test_ops_gpu_linear.py.
"""
import numpy as np
import pytest

import oracle.block_oracle as BO
from gpu_util import bf16_to_f64
from test_ops_gpu_linear import check_backward, f64, plan, tensors, workspace  # noqa: F401

pytestmark = pytest.mark.gpu
FAR = [1e20, -1e20, 2e19, -2e19, 3e38, -3e38, float("inf"), -float("inf"), float("nan"), 1e4, -1e4, 0.0]


# up to 8 and 16 rows, clusters that share K, 128 x 64, 128 x 128 and pairs of CTAs on 256 x 256 tiles
SIZES = [(1, 64, 64), (13, 72, 264), (60, 512, 136), (515, 64, 1000), (1300, 72, 1544), (1200, 64, 2304)]


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_forward(plan, M, K, N, act):  # noqa: F811
    import torch
    z = torch.linspace(-6, 6, N)
    z[1::3] = torch.tensor(FAR).repeat(N)[:len(z[1::3])]
    w = torch.zeros(N, K)
    w[:, 5] = z
    x = torch.zeros(M, K)
    x[:, 5] = 1.0
    w, x = w.to(torch.bfloat16).cuda(), x.to(torch.bfloat16).cuda()
    y, pre = (torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    plan.linear(x, w, y, act=act, pre=pre)
    plan.check()
    zz = bf16_to_f64(w[:, 5].contiguous())
    with np.errstate(all="ignore"):
        want = BO.act(zz, act)
    got = bf16_to_f64(y)
    assert np.array_equal(bf16_to_f64(pre), np.broadcast_to(zz, (M, N)), equal_nan=True)
    far = ~(np.abs(zz) < 1e4)
    assert np.array_equal(got[:, far], np.broadcast_to(want[far], (M, far.sum())), equal_nan=True)
    near = ~far
    assert np.all(np.abs(got[:, near] - want[near]) <= 2.0 ** -17 * (np.abs(zz[near]) + 1e-3) + 2.0 ** -8 * np.abs(want[near]))


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,K,N", [(6, 64, 72), (515, 64, 1000), (1200, 64, 2304)])
def test_backward(plan, M, K, N, gated, act):  # noqa: F811
    """Finite pre-activations (with a gate up to 1e30: dgate adds up to the rows' dy act(z) in fp32)."""
    import torch
    t = tensors(M, K, N, 1, seed=1)
    pre = tensors(M, K, N, 1, seed=2)["residual"]
    far = [1e20, -1e20, 2e19, -2e19, 1e30, -1e30] if gated else [v for v in FAR if np.isfinite(v)]
    flat = pre.view(-1)
    flat[1::5] = torch.tensor(far, dtype=torch.bfloat16, device="cuda").repeat(len(flat))[:len(flat[1::5])]
    out = dict(dx=torch.full_like(t["x"], 7), dw=torch.full_like(t["w"], 7), dbias=torch.full_like(t["bias"], 7),
               dgate=torch.full_like(t["gate"], 7) if gated else None)
    ws = workspace(plan, M, K, N, samples=1 if gated else 0)
    plan.linear_bwd(t["dy"], t["x"], t["w"], act=act, pre=pre, gate=t["gate"] if gated else None, workspace=ws, **out)
    plan.check()
    check_backward(t, out, act, pre, gated)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_backward_at_infinity(plan, act):  # noqa: F811
    """The derivative is 1 and 0 there; a NaN spoils its row of dx, its row of dw and its dbias, nothing else."""
    import torch
    M, K, N = 40, 64, 72
    t = tensors(M, K, N, 1, seed=1)
    pre = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    pre[:, 0], pre[:, 1], pre[7, 2] = float("inf"), -float("inf"), float("nan")
    dbias = torch.full_like(t["bias"], 7)
    dx, dw = torch.full_like(t["x"], 7), torch.full_like(t["w"], 7)
    ws = workspace(plan, M, K, N)
    plan.linear_bwd(t["dy"], t["x"], t["w"], act=act, pre=pre, dbias=dbias, dx=dx, dw=dw, workspace=ws)
    plan.check()
    dy = f64(t["dy"])
    assert abs(float(dbias[0]) - dy[:, 0].sum()) <= 2.0 ** -17 * np.abs(dy[:, 0]).sum() and float(dbias[1]) == 0.0
    assert torch.isnan(dbias[2]) and int(torch.isnan(dbias).sum()) == 1
    assert torch.isnan(dw[2]).all() and int(torch.isnan(dw).sum()) == K and torch.all(dw[1] == 0)
    assert torch.isnan(dx[7]).all() and int(torch.isnan(dx).sum()) == K
