"""The norm and the router's training side where offsets pass 32 bits, on
several streams at once, and as masks of either type: every row's result is
that of the same rows alone."""

import numpy as np
import pytest
import torch

from helpers import say
from oracle import balance as ob

pytestmark = pytest.mark.gpu


def test_norm_past_four_gib():
    import mixture_experts_layer_04_amd as moe
    T, H = 320000, 7168  # x, h and y of 4.6 GB each
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    x.normal_()
    w = torch.rand(H, device="cuda") + 0.5
    say("norm", T, H)
    y, h, q, s = moe.rms_norm(x, w, x, 1e-6, "fp8")
    rows = torch.cat([torch.arange(5), torch.arange(T // 2, T // 2 + 5), torch.arange(T - 5, T)]).cuda()
    few = x[rows]
    y1, h1, q1, s1 = moe.rms_norm(few, w, few, 1e-6, "fp8")
    torch.cuda.synchronize()
    for a, b in ((y, y1), (h, h1), (q, q1), (s, s1)):
        assert torch.equal(a[rows], b)
    del q, s
    dx, _ = moe.rms_norm_grad(y, h, w, 1e-6, dh=x, dx=x, with_weight=False)
    want, _ = moe.rms_norm_grad(y[rows], h[rows], w, 1e-6, dh=few, with_weight=False)
    torch.cuda.synchronize()
    assert torch.equal(dx[rows], want)


def test_norm_of_more_rows_than_one_grid_holds():
    import mixture_experts_layer_04_amd as moe
    T, H = (1 << 22) + 3, 8192  # 1024 threads a row; x of 69 GB
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 1, (1 << 21) - 1, 1 << 21, (1 << 21) + 1, (1 << 22) - 1, 1 << 22, T - 1], device="cuda")
    few = torch.randn(len(rows), H, device="cuda").bfloat16()
    x[rows] = few
    w = torch.rand(H, device="cuda") + 0.5
    say("norm", T, H)
    y, _ = moe.rms_norm(x, w, y=x)
    want, _ = moe.rms_norm(few, w)
    torch.cuda.synchronize()
    assert torch.equal(y[rows], want)
    del x, y
    torch.cuda.empty_cache()


def test_gate_grad_past_four_gib():
    import mixture_experts_layer_04_amd as moe
    T, H, E = 320000, 7168, 24
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    x.normal_()
    gate = torch.randn(E, H, device="cuda")
    d = torch.randn(T, E, device="cuda")
    say("gate_grad", T, H, E)
    dx, dg = moe.gate_grad(x, gate, d, x)
    rows = torch.cat([torch.arange(5), torch.arange(T // 2, T // 2 + 5), torch.arange(T - 5, T)]).cuda()
    one, _ = moe.gate_grad(x[rows], gate, d[rows], x[rows], with_gate=False)
    torch.cuda.synchronize()
    assert torch.equal(dx[rows], one)
    del dx
    want = torch.zeros(E, H, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(want)
    for t in range(0, T, 20000):
        a, b = d[t:t + 20000].double().t().contiguous(), x[t:t + 20000].double()
        want += a @ b
        mag += a.abs() @ b.abs()
    # exact products, 3 per 32-token step, each addition within 4 u of its sum
    bound = mag * 4 * (3 * (T // 32) + 64) * 2.0 ** -24
    assert torch.all((dg.double() - want).abs() <= bound)
    # and on the whole far closer: the errors of sums in any order average out
    assert float((dg.double() - want).norm() / want.norm()) < 1e-4


def test_router_past_four_gib():
    import mixture_experts_layer_04_amd as moe
    T, E, k = 4000000, 288, 2  # logits of 4.6 GB
    lg = torch.empty(T, E, device="cuda")
    lg.normal_()
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda")
    off = torch.tensor([0, T - 40, T], dtype=torch.int32, device="cuda")
    say("router", T, E)
    losses, counts, probs, tokens = moe.balance_loss(lg, ids, "sigmoid", off)
    dw = torch.randn(T, k, device="cuda")
    d = moe.route_grad(lg, ids, "sigmoid", True, 1.0, dw)
    tail = slice(T - 40, T)
    c1 = moe.balance_loss(lg[tail].clone(), ids[tail].clone(), "sigmoid")
    d1 = moe.route_grad(lg[tail].clone(), ids[tail].clone(), "sigmoid", True, 1.0, dw[tail].clone())
    torch.cuda.synchronize()
    assert tokens.tolist() == [T - 40, 40, T, 2]
    assert torch.equal(counts[1], c1[1][0]) and int(counts.sum()) == T * k
    assert torch.allclose(probs[1], c1[2][0], rtol=2.0 ** -16) and abs(float(probs[0].sum()) - 1) < 2.0 ** -16
    assert torch.equal(d[tail], d1)


def test_streams_at_once():
    import mixture_experts_layer_04_amd as moe
    T, H, E, k = 700, 1024, 128, 4
    sets = []
    for i in range(3):
        g = torch.Generator().manual_seed(i)
        lg = torch.randn(T, E, generator=g).cuda()
        sets.append((lg, lg.topk(k, 1).indices.int(), torch.randn(T, H, generator=g).to(torch.bfloat16).cuda(),
                     torch.randn(E, H, generator=g).cuda()))
    off = torch.tensor([0, 300, 700], dtype=torch.int32, device="cuda")
    dl = torch.ones(2, device="cuda")

    def chain(lg, ids, x, gate):
        r = moe.balance_loss(lg, ids, "softmax", off)
        d = moe.route_grad(lg, ids, "softmax", d_losses=dl, counts=r[1], tokens=r[3], seq_offsets=off)
        return (*r, d, *moe.gate_grad(x, gate, d))

    want = [chain(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(4):
        got = []
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(chain(*s))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_two_graphs_at_once():
    """Two captured chains, replayed together on two streams: their scratch
    memory is their own."""
    import mixture_experts_layer_04_amd as moe
    T, H, E = 600, 512, 288
    runs = []
    for i in range(2):
        g = torch.Generator().manual_seed(i)
        lg = torch.randn(T, E, generator=g).cuda()
        ids = lg.topk(4, 1).indices.int()
        x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
        gate = torch.randn(E, H, generator=g).cuda()
        w = torch.rand(H, generator=g).cuda()
        dl = torch.ones(2, device="cuda")

        def chain(lg=lg, ids=ids, x=x, gate=gate, w=w, dl=dl):
            r = moe.balance_loss(lg, ids, "sigmoid")
            d = moe.route_grad(lg, ids, "sigmoid", d_losses=dl, counts=r[1], tokens=r[3])
            dx, dg = moe.gate_grad(x, gate, d)
            return (*r, d, dg, *moe.rms_norm_grad(dx, x, w))

        want = chain()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = chain()
        runs.append((graph, out, want, torch.cuda.Stream(), chain))  # the chain holds the inputs
    for _ in range(4):
        for _, out, _, _, _ in runs:
            for t in out:
                t.zero_()
        torch.cuda.synchronize()
        for graph, _, _, st, _ in runs:
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for _, out, want, _, _ in runs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_bool_mask():
    import mixture_experts_layer_04_amd as moe
    lg = torch.randn(300, 64, device="cuda")
    ids = lg.topk(4, 1).indices.int()
    mask = torch.rand(300, device="cuda") < 0.6
    a = moe.balance_loss(lg, ids, token_mask=mask)
    b = moe.balance_loss(lg, ids, token_mask=mask.to(torch.uint8) * 255)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    ref = ob.balance_loss(lg.double().cpu().numpy(), ids.cpu().numpy(), "softmax", None, mask.cpu().numpy())
    assert np.array_equal(a[1].cpu().numpy(), ref["counts"]) and int(a[3][0]) == int(mask.sum())
