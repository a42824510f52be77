"""Calls that the documentation allows, in the ways a program makes them: a sum into the residual by every kind of tile, two
calls at once on one plan, graphs replayed with other data, the same buffers back to back."""
import pytest

import tile_sparse_video_pack_b200 as T
from gpu_util import ragged_gpu_config
from test_ops_gpu_attn_bwd import Case as AttnCase, long_rows_config
from test_ops_gpu_hold import tiling
from test_ops_gpu_linear import check_backward, check_forward, plan, tensors, workspace  # noqa: F401
from test_ops_gpu_norm_rope import Case as NormCase

pytestmark = pytest.mark.gpu
ALL = dict(bias=True, gate=True, residual=True)


@pytest.mark.parametrize("M,K,N,kind", [(3, 520, 72, "few"), (15, 1032, 264, "few"), (63, 2048, 136, "clusters"),
                                        (999, 256, 1024, "128x64"), (999, 200, 2048, "128x128"), (3000, 136, 1304, "pairs")])
def test_a_sum_into_the_residual(plan, M, K, N, kind):  # noqa: F811
    import torch
    assert kind == "few" or tiling(plan, M, N) == kind
    t = tensors(M, K, N, 3)
    y = torch.empty_like(t["residual"])
    plan.linear(t["x"], t["w"], y, bias=t["bias"], act="silu", gate=t["gate"], residual=t["residual"])
    inplace = t["residual"].clone()
    plan.linear(t["x"], t["w"], inplace, bias=t["bias"], act="silu", gate=t["gate"], residual=inplace)
    plan.check()
    check_forward(t, y, None, "silu", ALL)
    assert torch.equal(y, inplace)


def test_a_chain_of_calls_without_a_wait(plan):  # noqa: F811
    """Each call reads what the one before wrote, and writes what an earlier one read (dependent launches)."""
    import torch
    M, C = 300, 256
    t = tensors(M, C, C, 3)
    a, b = t["x"].clone(), torch.empty_like(t["x"])
    steps = []
    for i in range(40):                       # buffers swap roles every step; sizes that take three kernels
        rows = (300, 12, 300, 140)[i % 4]
        plan.linear(a[:rows], t["w"], b[:rows], bias=t["bias"], act=("gelu_tanh", "silu")[i % 2], residual=a[:rows])
        steps.append(b[:rows].clone())
        a, b = b, a
        b[rows:].copy_(a[rows:])
        a[rows:].copy_(b[rows:])
    plan.check()
    a, b = t["x"].clone(), torch.empty_like(t["x"])
    for i in range(40):
        rows = (300, 12, 300, 140)[i % 4]
        torch.cuda.synchronize()
        plan.linear(a[:rows], t["w"], b[:rows], bias=t["bias"], act=("gelu_tanh", "silu")[i % 2], residual=a[:rows])
        torch.cuda.synchronize()
        assert torch.equal(steps[i], b[:rows]), i
        a, b = b, a
        b[rows:].copy_(a[rows:])
        a[rows:].copy_(b[rows:])


@pytest.mark.parametrize("d", [64, 128])
def test_two_attention_gradients_at_once_on_one_plan(d):
    import torch
    cfg = long_rows_config(d)
    n = [4, 6]
    cases = [AttnCase(cfg, n, seed=i) for i in range(2)]
    p = cases[0].plan
    for c in cases:
        c.plan = p
        c.run()
    p.check()
    for c in cases:
        c.check()
    want = [[g.clone() for g in c.grads] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        for c in cases:
            for g in c.grads:
                g.fill_(7)
        torch.cuda.synchronize()
        for c, s in zip(cases, streams):
            p.sparse_attn_bwd(*c.pk[:3], c.op, c.lse, c.pk[3], c.idx, *c.grads, c.ws, stream=s)
        p.check()
        for c, w in zip(cases, want):
            assert all(torch.equal(a, b) for a, b in zip(c.grads, w))


def test_a_captured_attention_gradient_follows_its_inputs():
    """Other lists, tiles and incoming gradients in the captured buffers: the replay gives theirs."""
    import torch
    cfg = ragged_gpu_config(128, batch=2)
    k = [2] * cfg.heads
    a, b = AttnCase(cfg, k, seed=1), AttnCase(cfg, k, seed=2)
    a.run()
    a.plan.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run()
    b.run()
    b.plan.check()
    for mine, other in zip([*a.pk, a.op, a.lse, a.idx], [*b.pk, b.op, b.lse, b.idx]):
        mine.copy_(other)
    for _ in range(2):
        for g in a.grads:
            g.fill_(7)
        graph.replay()
    a.plan.check()
    assert all(torch.equal(x, y) for x, y in zip(a.grads, b.grads))
    a.kept, a.f = b.kept, b.f
    a.check()


def test_norms_at_once_on_one_plan():
    import torch
    c = NormCase(ragged_gpu_config(128, batch=2), "halves", True, strided=False)
    p, new = c.plan, lambda: torch.empty(c.shape, dtype=torch.bfloat16, device="cuda")
    dy = [torch.randn(*c.shape, generator=c.gen).to(torch.bfloat16).cuda() for _ in range(2)]

    def run(out, stream=None):
        p.qk_norm_rope(c.q, c.k, c.norm, out[0], out[1], stream=stream)
        p.qk_norm_rope_bwd(*dy, c.q, c.k, c.norm, out[2], out[3], out[4], out[5], out[6], stream=stream)

    outs = [[new() for _ in range(4)] + [torch.empty_like(c.norm.w_q) for _ in range(2)] +
            [torch.empty(p.norm_bwd_workspace_bytes(), dtype=torch.uint8, device="cuda")] for _ in range(3)]
    run(outs[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for o, s in zip(outs[1:], streams):
            run(o, s)
    p.check()
    for o in outs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(outs[0][:6], o[:6]))


def test_a_captured_linear_gradient_follows_its_inputs(plan):  # noqa: F811
    import torch
    M, K, N = 515, 328, 1000
    t, u = tensors(M, K, N, 1, seed=1), tensors(M, K, N, 1, seed=5)
    pre = [tensors(M, K, N, 1, seed=s)["residual"] for s in (2, 6)]
    out = dict(dx=torch.empty_like(t["x"]), dw=torch.empty_like(t["w"]), dbias=torch.empty_like(t["bias"]),
               dgate=torch.empty_like(t["gate"]))
    ws = workspace(plan, M, K, N, samples=1)
    call = lambda: plan.linear_bwd(t["dy"], t["x"], t["w"], act="silu", pre=pre[0], gate=t["gate"], workspace=ws, **out)
    call()
    plan.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in t:
        t[k].copy_(u[k])
    pre[0].copy_(pre[1])
    ws.fill_(255)
    for _ in range(2):
        graph.replay()
    plan.check()
    check_backward(u, out, "silu", pre[1], True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("slow", ["q", "do", "k", "v"])
def test_attention_gradient_with_one_tensor_out_of_cache(d, slow):
    """Copies of one tensor arrive late, those of the others at once: the same bits as with all of them in cache."""
    import torch
    cfg = long_rows_config(d)
    c = AttnCase(cfg, [4, 6])
    c.run()
    c.plan.check()
    c.check()
    want = [g.clone() for g in c.grads]
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    hot = [t for t, name in zip(c.pk, ("q", "k", "v", "do")) if name != slow]
    for _ in range(20):
        flush.fill_(1)
        for t in hot:
            t.sum()
        for g in c.grads:
            g.fill_(7)
        c.run()
        c.plan.check()
        assert all(torch.equal(a, b) for a, b in zip(c.grads, want))
