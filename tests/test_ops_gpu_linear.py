"""The linear layer with its epilogue and its gradient against the fp64 oracle.

Tolerances, per element. Products: K fp32 additions of exact bf16 products, at most 2^-23 of the sum of
|terms| each (the tensor cores may truncate where they align): K 2^-23 sum|x||w|. The epilogue's few fp32
roundings and its exponential (2 + |u| units of 2^-24, |u| < 32 where it matters): 2^-17 of |z| + |act|.
Output rounding: half a bf16 step, 2^-8 of the value. In the gradient dz is rounded to bf16 first: 2^-8 of
the sum of |terms| of its two products. Those roundings are independent, each at most 2^-8 and 2^-8/sqrt(3)
rms of its term, so the error of an output has an rms of at most 2^-8/sqrt(3) times the root of the sum of
its squared terms and its own square; over an output tensor the norm of the error stays below 2^-8 of that
root. (The terms, not the result, set the scale: eight terms of one row can cancel, as 1.7e-3 against a result
of 0.14 showed for one row of eight, where the terms' root is 0.5.) Column sums: fp32 chains of at most
64 terms, each term off by 2^-17: (64 2^-24 + 2^-17) of the sum of |terms|.
"""
import numpy as np
import pytest

import oracle.block_oracle as BO
from gpu_util import bf16_to_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def plan():
    import tile_sparse_video_pack_b200 as T
    return T.Plan(T.make_desc(1, 1, 64, 1, 8, 8, [], [(4, 4, 4)], [1]))


def tensors(M, K, N, samples, seed=0):
    import torch
    g = torch.Generator().manual_seed(seed)
    bf = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(torch.bfloat16).cuda()
    f32 = lambda *s: torch.randn(*s, generator=g).cuda()
    return dict(x=bf(M, K), w=bf(N, K, scale=K ** -0.5), bias=f32(N), gate=f32(samples, N), residual=bf(M, N),
                dy=bf(M, N))


def f64(t):
    import torch
    if t is None:
        return None
    return bf16_to_f64(t) if t.dtype == torch.bfloat16 else t.double().cpu().numpy()


def workspace(plan, *a, **kw):
    import torch
    return torch.empty(plan.linear_bwd_workspace_bytes(*a, **kw), dtype=torch.uint8, device="cuda")


def check_forward(t, got, pre, act, use):
    x, w = f64(t["x"]), f64(t["w"])
    arg = {k: f64(t[k]) if use[k] else None for k in ("bias", "gate", "residual")}
    y, z = BO.linear(x, w, arg["bias"], act, arg["gate"], arg["residual"])
    acc = x.shape[1] * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T) + 2.0 ** -17 * (np.abs(z) + 1e-3)
    gate = np.repeat(np.abs(arg["gate"]), len(x) // len(arg["gate"]), 0) if use["gate"] else 1.0
    tol = 1.2 * acc * gate + 2.0 ** -23 * np.abs(y) + 2.0 ** -8 * np.abs(y)     # |act'| < 1.13
    assert np.all(np.abs(f64(got) - y) <= tol), np.max(np.abs(f64(got) - y) / tol)
    if pre is not None:
        assert np.all(np.abs(f64(pre) - z) <= acc + 2.0 ** -8 * np.abs(z))


SIZES = [(1, 8, 8), (1, 2048, 328), (2, 136, 1040), (3, 1480, 64), (8, 256, 2056), (9, 520, 200), (16, 64, 128),
         (17, 72, 264), (64, 128, 256), (77, 1480, 520), (127, 64, 136), (128, 128, 128), (129, 200, 72),
         (200, 2048, 96), (257, 512, 512), (515, 328, 1000), (1200, 192, 2304), (2500, 64, 640),
         (3000, 136, 1304), (1100, 2600, 2904), (7201, 520, 520), (2, 72, 9480), (7, 1032, 9480), (4, 520, 1024),
         (16, 2048, 9480), (13, 136, 40), (12, 1096, 1544), (5, 1560, 72), (1, 8, 16), (77, 2048, 1024)]


@pytest.mark.parametrize("act", ["none", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_forward(plan, M, K, N, act):
    import torch
    t = tensors(M, K, N, M if M < 4 else 1)
    y, pre = torch.full_like(t["residual"], 7), torch.full_like(t["residual"], 7)
    for use in (dict(bias=False, gate=False, residual=False), dict(bias=True, gate=True, residual=True)):
        plan.linear(t["x"], t["w"], y, act=act, pre=pre if use["bias"] else None,
                    **{k: t[k] if v else None for k, v in use.items()})
        plan.check()
        check_forward(t, y, pre if use["bias"] else None, act, use)


def test_gate_per_sample_and_views(plan):
    """Three samples of 43 rows; x, y and the residual are column slices of wider buffers; y in place of the
    residual; columns outside the slices keep their values."""
    import torch
    M, K, N = 129, 136, 264
    t = tensors(M, K, N, 3)
    wide = {k: torch.full((M, v.shape[1] + 24), 5.0, dtype=v.dtype, device="cuda") for k, v in t.items()
            if k in ("x", "residual")}
    for k, v in wide.items():
        v[:, 8:-16] = t[k]
    x, r = wide["x"][:, 8:-16], wide["residual"][:, 8:-16]
    use = dict(bias=True, gate=True, residual=True)
    plan.linear(x, t["w"], r, bias=t["bias"], act="silu", gate=t["gate"], residual=r)
    plan.check()
    check_forward(t, r, None, "silu", use)
    assert torch.all(wide["residual"][:, :8] == 5) and torch.all(wide["residual"][:, -16:] == 5)
    y3 = torch.empty(3, 43, N, dtype=torch.bfloat16, device="cuda")      # three-dimensional x and y
    plan.linear(t["x"].view(3, 43, K), t["w"], y3, bias=t["bias"], act="silu", gate=t["gate"],
                residual=t["residual"].view(3, 43, N))
    plan.check()
    assert torch.equal(y3.view(M, N), r)


def check_backward(t, out, act, pre, use_gate):
    x, w, dy = f64(t["x"]), f64(t["w"]), f64(t["dy"])
    z, gate = f64(pre), f64(t["gate"]) if use_gate else None
    g = BO.linear_grad(dy, x, w, act, z, gate)
    rounded = act != "none" or use_gate
    adz = np.abs(g["dz"])
    for name, K, terms, squares in (("dx", w.shape[0], adz @ np.abs(w), adz ** 2 @ w ** 2),
                                    ("dw", len(x), adz.T @ np.abs(x), (adz ** 2).T @ x ** 2)):
        got, want = f64(out[name]), g[name]
        tol = (K * 2.0 ** -23 + 2.0 ** -17 + (2.0 ** -8 if rounded else 0)) * terms + 2.0 ** -8 * np.abs(want)
        err = np.abs(got - want)
        assert np.all(err <= tol), (name, np.max(err / tol))
        assert np.linalg.norm(err) <= 2.0 ** -8 * np.sqrt(squares.sum() + (want ** 2).sum()), name
    col = (64 * 2.0 ** -24 + 2.0 ** -17)
    assert np.all(np.abs(f64(out["dbias"]) - g["dbias"]) <= col * adz.sum(0) + 1e-30)
    if use_gate and out.get("dgate") is not None:
        S = len(gate)
        terms = np.abs(dy * BO.act(z, act)).reshape(S, len(dy) // S, -1).sum(1)
        assert np.all(np.abs(f64(out["dgate"]) - g["dgate"]) <= col * terms + 1e-30)


@pytest.mark.parametrize("act", ["none", "gelu_tanh", "silu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_backward(plan, M, K, N, gated, act):
    import torch
    S = M if M < 4 else (3 if M % 3 == 0 else 1)
    t = tensors(M, K, N, S, seed=1)
    pre = tensors(M, K, N, S, seed=2)["residual"]
    out = dict(dx=torch.full_like(t["x"], 7), dw=torch.full_like(t["w"], 7), dbias=torch.full_like(t["bias"], 7),
               dgate=torch.full_like(t["gate"], 7) if gated else None)
    ws = workspace(plan, M, K, N, samples=S if gated else 0)
    plan.linear_bwd(t["dy"], t["x"], t["w"], act=act, pre=pre, gate=t["gate"] if gated else None, workspace=ws, **out)
    plan.check()
    check_backward(t, out, act, pre, gated)
    again = {k: None if v is None else torch.empty_like(v) for k, v in out.items()}
    plan.linear_bwd(t["dy"], t["x"], t["w"], act=act, pre=pre, gate=t["gate"] if gated else None, workspace=ws, **again)
    plan.check()
    for k, v in out.items():
        assert v is None or torch.equal(v, again[k]), k       # the same on every call
    # each output alone (K may be split otherwise, so to the same tolerances and not to the bit)
    for k in ("dx", "dw", "dbias"):
        one = torch.empty_like(out[k])
        plan.linear_bwd(t["dy"], t["x"], t["w"], act=act, pre=pre, gate=t["gate"] if gated else None, workspace=ws,
                        **{k: one})
        plan.check()
        check_backward(t, {**out, k: one}, act, pre, gated)


def test_no_rows(plan):
    import torch
    t = tensors(1, 64, 128, 1)
    e = lambda n: torch.empty(0, n, dtype=torch.bfloat16, device="cuda")
    assert plan.linear_bwd_workspace_bytes(0, 64, 128) == 0
    plan.linear(e(64), t["w"], e(128), bias=t["bias"], act="silu")
    dw, db = torch.full_like(t["w"], 7), torch.full_like(t["bias"], 7)
    plan.linear_bwd(e(128), e(64), t["w"], dx=e(64), dw=dw, dbias=db)
    plan.check()
    assert torch.all(dw == 0) and torch.all(db == 0)


def test_special_values_stay_in_their_rows(plan):
    """A row with an infinity or a NaN spoils its own output row only; large |z| saturates the activation."""
    import torch
    t = tensors(130, 128, 256, 1)
    y = torch.empty_like(t["residual"])
    plan.linear(t["x"], t["w"], y, act="gelu_tanh")
    base = y.clone()
    t["x"][5, 3] = float("nan")
    t["x"][129, 0] = float("inf")
    plan.linear(t["x"], t["w"], y, act="gelu_tanh")
    plan.check()
    rows = [i for i in range(130) if i not in (5, 129)]
    assert torch.equal(y[rows], base[rows]) and torch.isnan(y[5]).all()
    t = tensors(4, 128, 256, 1)
    t["x"] *= 200
    for act in ("silu", "gelu_tanh"):
        plan.linear(t["x"], t["w"], y[:4], act=act)
        plan.check()
        check_forward(t, y[:4], None, act, dict(bias=False, gate=False, residual=False))


@pytest.mark.parametrize("M,K,N", [(64, 2048, 128), (1200, 192, 2304), (3000, 1024, 1304)])
def test_timeout_is_reported(M, K, N):
    """A wait limit of a microsecond runs out (clusters that share K, single CTAs, CTA pairs): the call returns,
    check reports it, and the next call is right."""
    import torch
    import tile_sparse_video_pack_b200 as T
    plan = T.Plan(T.make_desc(1, 1, 64, 1, 8, 8, [], [(4, 4, 4)], [1]))
    t = tensors(M, K, N, 1)
    y = torch.empty_like(t["residual"])
    plan.set_wait_limit(1000)
    plan.linear(t["x"], t["w"], y)
    try:
        plan.check()
    except T.VsaError as e:
        assert "TIMEOUT" in str(e)
    plan.set_wait_limit(0)
    plan.linear(t["x"], t["w"], y)
    plan.check()
    check_forward(t, y, None, "none", dict(bias=False, gate=False, residual=False))


def test_two_streams_share_a_plan(plan):
    """Calls on one plan keep nothing in it: two streams at once give what one gives."""
    import torch
    cases = [tensors(300, 512, 1024, 1, seed=i) for i in range(2)]
    want = []
    for t in cases:
        want.append(torch.empty_like(t["residual"]))
        plan.linear(t["x"], t["w"], want[-1], bias=t["bias"], act="silu")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[torch.empty_like(w) for _ in range(8)] for w in want]
    for i in range(8):
        for t, s, g in zip(cases, streams, got):
            plan.linear(t["x"], t["w"], g[i], bias=t["bias"], act="silu", stream=s)
    plan.check()
    for w, g in zip(want, got):
        assert all(torch.equal(w, x) for x in g)


def test_refusals(plan):
    import torch
    import tile_sparse_video_pack_b200 as T
    t = tensors(6, 64, 128, 2)
    y = torch.empty_like(t["residual"])
    with pytest.raises(TypeError):
        plan.linear(t["x"].half(), t["w"], y)
    with pytest.raises(TypeError):
        plan.linear(t["x"], t["w"], y, bias=t["bias"].to(torch.bfloat16))
    with pytest.raises(ValueError):
        plan.linear(t["x"][:, :32], t["w"], y)
    with pytest.raises(ValueError):
        plan.linear(t["x"], t["w"], y[:4])
    with pytest.raises(ValueError):
        plan.linear(t["x"], t["w"], y, act="relu")
    with pytest.raises(ValueError):
        plan.linear(t["x"], t["w"], y, gate=torch.ones(4, 128, device="cuda"))     # 4 does not divide 6 rows
    with pytest.raises(ValueError):
        plan.linear(t["x"].t().contiguous().t(), t["w"], y)                        # columns not contiguous
    with pytest.raises(ValueError):
        plan.linear(t["x"], t["w"].t().contiguous().t(), y)
    with pytest.raises(T.VsaError):
        plan.linear(t["x"][:, :60].contiguous(), t["w"][:, :60].contiguous(), y)   # n_in not a multiple of 8
    with pytest.raises(T.VsaError):
        plan.linear_bwd_workspace_bytes(-1, 64, 64)
    with pytest.raises(ValueError):
        plan.linear_bwd(t["dy"], t["x"], t["w"], dx=torch.empty_like(t["x"]), act="silu")   # no pre
    with pytest.raises(ValueError):
        plan.linear_bwd(t["dy"], t["x"], t["w"], dgate=t["gate"])
    with pytest.raises(ValueError):
        plan.linear_bwd(t["dy"], None, t["w"], dw=torch.empty_like(t["w"]))
    with pytest.raises(ValueError):                                                # a workspace that is too small
        plan.linear_bwd(t["dy"], t["x"], t["w"], dbias=t["bias"], workspace=torch.empty(1, dtype=torch.uint8, device="cuda"))
    plan.check()


def test_widths_have_a_limit(plan):
    import tile_sparse_video_pack_b200 as T
    assert plan.linear_bwd_workspace_bytes(8, 64, 1 << 20) > 0
    for n_in, n_out in ((64, (1 << 20) + 8), ((1 << 20) + 8, 64)):
        with pytest.raises(T.VsaError):
            plan.linear_bwd_workspace_bytes(8, n_in, n_out)


def test_widest(plan):
    """2^20 columns out with one row, and 2^20 in: offsets of the weights past 32 bits."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    K, N = 2056, 1 << 20                         # 2.16e9 weights
    w = torch.randn(N, K, generator=g, device="cuda", dtype=torch.bfloat16)
    for rows in (3, 20):                         # both kernels that read W by rows and by tiles
        x = torch.randn(rows, K, generator=g, device="cuda").bfloat16()
        y = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
        plan.linear(x, w, y)
        plan.check()
        for at in (0, N // 2 - 8, N - 16):
            want = x.double() @ w[at:at + 16].double().T
            terms = x.double().abs() @ w[at:at + 16].double().abs().T
            assert bool(((y[:, at:at + 16].double() - want).abs() <= K * 2.0 ** -23 * terms + 2.0 ** -8 * want.abs()).all())


def test_no_rows_with_a_gate(plan):
    import torch
    bf, K, N = torch.bfloat16, 64, 136
    new = lambda *s, dtype=bf: torch.full(s, 7.0, dtype=dtype, device="cuda")
    x, dx, y = new(2, 0, K), new(2, 0, K), new(2, 0, N)
    w, dw, gate, dgate = new(N, K), new(N, K), new(2, N, dtype=torch.float32), new(2, N, dtype=torch.float32)
    dbias = new(N, dtype=torch.float32)
    plan.linear(x, w, y, gate=gate, residual=y)
    for stream in (None, torch.cuda.Stream()):
        for t in (dw, dbias, dgate):
            t.fill_(7.0)
        torch.cuda.synchronize()
        plan.linear_bwd(y, x, w, dx=dx, dw=dw, pre=y, gate=gate, dbias=dbias, dgate=dgate, stream=stream)
        plan.check()
        assert not dw.any() and not dbias.any() and not dgate.any()
