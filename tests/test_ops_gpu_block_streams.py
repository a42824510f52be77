"""A block's backward on another stream than its forward's."""
import pytest

import tile_sparse_video_pack_b200 as T

pytestmark = pytest.mark.gpu


def test_feed_forward_keeps_its_tensors_until_backward_has_read_them():
    """The next forward, on the first stream, drops what the last one kept while backward is still to run on the other:
    the first stream's new tensors must not take its memory."""
    import torch
    plan = T.Plan(T.make_desc(1, 1, 64, 1, 8, 8, [], [(4, 4, 4)], [1]))
    g = torch.Generator(device="cuda").manual_seed(3)
    bf = lambda *s, scale=1.0: (torch.randn(*s, generator=g, device="cuda") * scale).to(torch.bfloat16)
    rows, n, m = 2048, 256, 1024
    ff = T.FeedForward(plan, bf(m, n, scale=n ** -0.5), bf(n, m, scale=m ** -0.5))
    data = bf(rows, n)
    dy = bf(rows, n)
    gate = torch.randn(4, n, generator=g, device="cuda")
    ff.forward(data, gate=gate, save=True)
    want = ff.backward(dy)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for _ in range(3):
        ff.forward(data.clone(), gate=gate.clone(), save=True)        # backward's only reference to x and gate
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(other):
            torch.cuda._sleep(100_000_000)                             # some 50 ms
        got = ff.backward(dy, stream=other)
        ff.forward(data, save=True)
        spoil = [torch.full((rows, w), 3.0, dtype=torch.bfloat16, device="cuda") for w in (n, m) for _ in range(6)]
        spoil += [torch.full((4, n), 3.0, device="cuda") for _ in range(6)]
        torch.cuda.synchronize()
        plan.check()
        for k, v in want.items():
            assert v is None or torch.equal(v, got[k]), k
        del spoil
