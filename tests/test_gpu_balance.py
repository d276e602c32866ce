"""moe_balance_loss, moe_route_grad and moe_gate_grad on the GPU against the
float64 oracle, alone and as the router's backward pass uses them together.

Error bounds (u = 2^-24): a probability is exp(l - m) over a sum of at most
1024 of them; l - m is rounded (|l - m| u, with |l - m| <= 60 for every value
that matters below) and the functions are within a few u, the sums within
(E / 16 + 6) u: 2^-17 in all.  Means and losses add positive terms to that,
at most 2^11 of them one after another: 2^-12 u, so 2^-16 covers them.  The z
loss's lse is within 2^-18 of 1 + |max| + |lse|.  The gradients add terms
with those errors: 2^-15 of the sum of their magnitudes.
"""

import numpy as np
import pytest
import torch

from helpers import say
from oracle import balance as ob

pytestmark = pytest.mark.gpu

SCORINGS = ["softmax", "sigmoid", "sqrtsoftplus"]


def f64(t):
    return None if t is None else t.detach().to(torch.float64).cpu().numpy()


def make(T, E, k, seed=0, n_shared=0, std=2.0):
    g = torch.Generator().manual_seed(seed * 7919 + T * 31 + E)
    lg = torch.randn(T, E, generator=g) * std + torch.randn(E, generator=g)
    ids = lg.topk(k, dim=1).indices
    if n_shared:
        ids = torch.cat([ids, torch.full((T, 1), E)], dim=1)
    return lg.cuda(), ids.to(torch.int32).cuda()


def ranges(T, kind, seed=0):
    """Sequence offsets (on the CPU, a list) of a batch of T rows."""
    rng = np.random.default_rng(seed)
    if kind == "one":
        return None
    if kind == "single":
        return [0, T]
    if kind == "inner":  # rows before the first and behind the last
        a, b = T // 5, T - T // 7
        return [a, (a + b) // 2, b]
    if kind == "empty":
        return [0, 0, 0, T // 2, T // 2, T, T]
    if kind == "none":
        return [T // 2, T // 2]
    return [0] + sorted(rng.integers(0, T + 1, size=40).tolist()) + [T]


def check_loss(got, ref, lg, seq):
    losses, counts, probs, tokens = (t.cpu() for t in got)
    assert np.array_equal(counts.numpy(), ref["counts"])
    assert np.array_equal(tokens.numpy(), ref["tokens"])
    assert np.all(np.abs(f64(probs) - ref["probs"]) <= ref["probs"] * 2.0 ** -16 + 1e-30)
    assert abs(float(losses[0]) - ref["losses"][0]) <= 2.0 ** -16 * ref["losses"][0]
    live = seq >= 0
    size = np.abs(f64(lg)).max(axis=1, initial=0.0) + 8.0  # lse <= max + ln 1024
    bound = 2.0 ** -16 * np.mean(size[live] ** 2) if live.any() else 0.0
    assert abs(float(losses[1]) - ref["losses"][1]) <= bound


def to_dev(off, mask):
    return (None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda"),
            None if mask is None else torch.tensor(mask, dtype=torch.uint8, device="cuda"))


CASES = [(1, 1, 1), (1, 8, 2), (5, 7, 3), (17, 60, 6), (64, 128, 8), (300, 100, 1), (129, 256, 8), (512, 288, 8),
         (1000, 320, 4), (77, 384, 8), (40, 500, 8), (33, 513, 8), (50, 700, 16), (90, 1024, 8), (20000, 64, 6),
         (40000, 16, 2)]


@pytest.mark.parametrize("T,E,k", CASES)
@pytest.mark.parametrize("scoring", SCORINGS)
def test_balance_and_gradient(T, E, k, scoring):
    """Every kind of sequence cut and mask at every shape."""
    import mixture_experts_layer_04_amd as moe
    lg, ids = make(T, E, k)
    big = T * E > 600000
    for n, kind in enumerate(["ragged"] if big else ["one", "single", "inner", "empty", "none", "ragged"]):
        off = ranges(T, kind, T + n)
        mask = None if n % 2 == 0 else (np.random.default_rng(n).random(T) < 0.7).astype(np.uint8)
        offd, maskd = to_dev(off, mask)
        got = moe.balance_loss(lg, ids, scoring, offd, maskd)
        torch.cuda.synchronize()
        ref = ob.balance_loss(f64(lg), ids.cpu().numpy(), scoring, off, mask)
        seq, _ = ob.members(T, off, mask)
        check_loss(got, ref, lg, seq)
        g = torch.Generator().manual_seed(n)
        dw = torch.randn(T, k, generator=g).cuda()
        dl = torch.tensor([0.3 * T, 0.02 * T], device="cuda")
        for use_w, use_l in ((True, True), (False, True), (True, False)):
            renorm = (n + use_w) % 2 == 0
            d = moe.route_grad(lg, ids, scoring, renorm, 2.5, dw if use_w else None, dl if use_l else None,
                               got[1] if use_l else None, got[3] if use_l else None, offd, maskd)
            torch.cuda.synchronize()
            want, mag = ob.route_grad(f64(lg), ids.cpu().numpy(), scoring, renorm, 2.5, f64(dw) if use_w else None,
                                      f64(dl) if use_l else None, ref["counts"], off, mask)
            err = np.abs(f64(d) - want)
            assert np.all(err <= mag * 2.0 ** -15 + 1e-35), f"{kind}: {np.max(err / (mag + 1e-30))}"
            if not use_w:
                assert np.all(f64(d)[seq < 0] == 0)


@pytest.mark.parametrize("E", [321, 400, 449, 577, 640, 641, 768, 897, 1023])
@pytest.mark.parametrize("scoring", SCORINGS)
def test_many_experts(E, scoring):
    """Above 320 experts a token's logits lie in 32 or 64 lanes: all 16 slots,
    ids that repeat in the first and the last of them, foreign ones, and
    rows of a wave that take no part beside ones that do."""
    import mixture_experts_layer_04_amd as moe
    T, k = 77, 16
    lg, ids = make(T, E, k)
    ids[0, :] = E - 1
    ids[1, 15] = ids[1, 0]
    ids[2, ::2] = 0
    ids[3, 7] = E
    ids[4, :] = -1
    mask = (np.arange(T) % 3 != 1).astype(np.uint8)
    off = [2, 40, 40, T - 3]
    offd, maskd = to_dev(off, mask)
    got = moe.balance_loss(lg, ids, scoring, offd, maskd)
    ref = ob.balance_loss(f64(lg), ids.cpu().numpy(), scoring, off, mask)
    seq, _ = ob.members(T, off, mask)
    check_loss(got, ref, lg, seq)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(E)).cuda()
    dw[::5] = 0
    dl = torch.tensor([20.0, 3.0], device="cuda")
    for renorm in (True, False):
        d = moe.route_grad(lg, ids, scoring, renorm, 2.5, dw, dl, got[1], got[3], offd, maskd)
        torch.cuda.synchronize()
        want, mag = ob.route_grad(f64(lg), ids.cpu().numpy(), scoring, renorm, 2.5, f64(dw), f64(dl), ref["counts"],
                                  off, mask)
        assert np.all(np.abs(f64(d) - want) <= mag * 2.0 ** -15 + 1e-35)


def test_shared_slot_foreign_and_repeated_ids():
    import mixture_experts_layer_04_amd as moe
    T, E, k = 90, 64, 4
    lg, ids = make(T, E, k, n_shared=1)
    ids[3, 1] = -1
    ids[4, :4] = -1
    ids[5, 2] = E + 7
    ids[6, :4] = 9           # the same expert in every slot
    ids[7, 3] = ids[7, 0]
    dw = torch.randn(T, k + 1, device="cuda")
    for scoring in SCORINGS:
        for renorm in (True, False):
            got = moe.balance_loss(lg, ids, scoring, n_shared=1)
            d = moe.route_grad(lg, ids, scoring, renorm, 1.5, dw, torch.ones(2, device="cuda"), got[1], got[3],
                               n_shared=1)
            torch.cuda.synchronize()
            routed = ids.cpu().numpy()[:, :k]
            ref = ob.balance_loss(f64(lg), routed, scoring)
            check_loss(got, ref, lg, np.zeros(T, dtype=int))
            want, mag = ob.route_grad(f64(lg), routed, scoring, renorm, 1.5, f64(dw)[:, :k], np.ones(2),
                                      ref["counts"])
            assert np.all(np.abs(f64(d) - want) <= mag * 2.0 ** -15 + 1e-35)


@pytest.mark.parametrize("scoring", SCORINGS)
def test_extreme_logits(scoring):
    """-inf experts, rows of -inf, the type's lowest value, and rows with NaN
    that the mask leaves out."""
    import mixture_experts_layer_04_amd as moe
    T, E, k = 70, 96, 4
    lg, ids = make(T, E, k)
    lg[1, 5:40] = float("-inf")
    lg[2, :] = float("-inf")
    lg[3, :50] = torch.finfo(torch.float32).min
    lg[4, :] = 80.0
    lg[5, 7] = 200.0
    lg[6, :] = -95.0
    lg[7, 3] = float("nan")
    lg[8, :] = float("nan")
    lg[9, 0] = float("inf")
    mask = np.ones(T, dtype=np.uint8)
    mask[7:10] = 0
    _, maskd = to_dev(None, mask)
    got = moe.balance_loss(lg, ids, scoring, None, maskd)
    dl = torch.tensor([3.0, 0.1], device="cuda")
    d = moe.route_grad(lg, ids, scoring, True, 1.0, None, dl, got[1], got[3], None, maskd)
    torch.cuda.synchronize()
    clean = lg.clone()
    clean[7:10] = 0.0
    ref = ob.balance_loss(f64(clean), ids.cpu().numpy(), scoring, None, mask)
    losses, counts, probs, tokens = (t.cpu() for t in got)
    assert np.array_equal(counts.numpy(), ref["counts"]) and np.array_equal(tokens.numpy(), ref["tokens"])
    assert np.all(np.abs(f64(probs) - ref["probs"]) <= ref["probs"] * 2.0 ** -16 + 1e-30)
    assert abs(float(losses[0]) - ref["losses"][0]) <= 2.0 ** -16 * ref["losses"][0]
    assert abs(float(losses[1]) - ref["losses"][1]) <= 2.0 ** -15 * ref["losses"][1]
    want, mag = ob.route_grad(f64(clean), ids.cpu().numpy(), scoring, True, 1.0, None, f64(dl), ref["counts"], None,
                              mask)
    # exp flushes what lies below 2^-126 to zero
    assert np.all(np.abs(f64(d) - want) <= mag * 2.0 ** -15 + 1e-35)
    assert torch.all(d[7:10] == 0)
    # a NaN in a row that takes part reaches the losses
    bad = moe.balance_loss(lg, ids, scoring)[0]
    torch.cuda.synchronize()
    assert torch.all(torch.isnan(bad))


def test_a_row_without_gradients_is_zero():
    import mixture_experts_layer_04_amd as moe
    lg, ids = make(40, 64, 4)
    lg[3] = float("nan")
    dw = torch.randn(40, 4, device="cuda")
    dw[3] = 0.0
    ids[5] = -1
    d = moe.route_grad(lg, ids, "sigmoid", d_weights=dw)
    torch.cuda.synchronize()
    assert torch.all(d[3] == 0) and torch.all(d[5] == 0) and torch.all(torch.isfinite(d))


def test_offsets_out_of_order_stay_inside():
    """Undefined numbers, but every access is clamped: the call ends and the
    words around its outputs are as they were."""
    import mixture_experts_layer_04_amd as moe
    T, E, k = 500, 64, 4
    lg, ids = make(T, E, k)
    for off in ([0, 400, 100, T], [-50, 20, 10 ** 9, T], [T, 0], [2 ** 31 - 1, -2 ** 31, 5, 4]):
        offd, _ = to_dev(off, None)
        got = moe.balance_loss(lg, ids, "softmax", offd)
        d = moe.route_grad(lg, ids, "softmax", d_losses=torch.ones(2, device="cuda"), counts=got[1], tokens=got[3],
                           seq_offsets=offd)
        torch.cuda.synchronize()
        assert got[1].shape == (len(off) - 1, E) and d.shape == (T, E)
    got = moe.balance_loss(lg, ids, "softmax")
    torch.cuda.synchronize()
    assert np.array_equal(got[1].cpu().numpy(), ob.balance_loss(f64(lg), ids.cpu().numpy(), "softmax")["counts"])


def test_empty_batch():
    import mixture_experts_layer_04_amd as moe
    lg = torch.empty(0, 8, device="cuda")
    ids = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    losses, counts, probs, tokens = moe.balance_loss(lg, ids)
    d = moe.route_grad(lg, ids, d_losses=torch.ones(2, device="cuda"), counts=counts, tokens=tokens)
    torch.cuda.synchronize()
    assert not losses.any() and not counts.any() and not probs.any() and not tokens.any() and d.shape == (0, 8)


def test_the_same_every_time_and_in_a_graph():
    import mixture_experts_layer_04_amd as moe
    T, E, k = 3000, 256, 8
    lg, ids = make(T, E, k)
    off, mask = to_dev(ranges(T, "ragged"), (np.random.default_rng(0).random(T) < 0.8).astype(np.uint8))
    dl = torch.tensor([1.0, 0.1], device="cuda")
    dw = torch.randn(T, k, device="cuda")

    def both():
        r = moe.balance_loss(lg, ids, "sigmoid", off, mask)
        return (*r, moe.route_grad(lg, ids, "sigmoid", True, 2.5, dw, dl, r[1], r[3], off, mask))

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for i in range(4):
        lg.copy_(make(T, E, k, seed=i + 1)[0])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, both()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


GATE = [(1, 128, 1), (3, 256, 8), (33, 128, 60), (128, 384, 64), (130, 1024, 100), (300, 2048, 128), (512, 4096, 288),
        (257, 512, 320), (1000, 256, 513), (40, 640, 1024), (4099, 1024, 256), (8192, 128, 16)]


@pytest.mark.parametrize("T,H,E", GATE)
@pytest.mark.parametrize("gt", [torch.float32, torch.bfloat16])
def test_gate_grad(T, H, E, gt):
    """dx: an operand's hi plane is within 2^-8 of it (a half step of bf16), hi
    and mid within 2^-16, so the parts left out (mid mid and the two lo parts)
    are below 3 2^-16 < 2^-14 of each product; the sum's own error is below (E
    / 32 + 4) 3 u 2, then comes one bf16 rounding of 2^-8; d_gate:
    exact products, 3 per 32-token step and operand, added with a relative
    error of at most 4 u each."""
    import mixture_experts_layer_04_amd as moe
    g = torch.Generator().manual_seed(T + H + E)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    gate = (torch.randn(E, H, generator=g) * 0.02).to(gt).cuda()
    d = torch.randn(T, E, generator=g).cuda() * torch.exp(torch.randn(T, 1, generator=g).cuda() * 3)
    dx_in = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    u = 2.0 ** -24
    for add in (dx_in, None):
        dx, dg = moe.gate_grad(x, gate, d, add)
        torch.cuda.synchronize()
        ref = ob.gate_grad(f64(x), f64(gate), f64(d), f64(add))
        assert np.all(np.abs(f64(dx) - ref["dx"]) <=
                      np.abs(ref["dx"]) * 2.0 ** -8 + ref["dx_mag"] * (2.0 ** -14 + (E / 32 + 4) * 6 * u) * 1.01)
        assert np.all(np.abs(f64(dg) - ref["d_gate"]) <= ref["d_gate_mag"] * 4 * (3 * (-(-T // 32)) + 8) * u)
    only_dx, none = moe.gate_grad(x, gate, d, with_gate=False)
    none2, only_dg = moe.gate_grad(x, gate, d, with_dx=False)
    again, _ = moe.gate_grad(x, gate, d, dx_in, dx=dx_in)
    torch.cuda.synchronize()
    assert none is None and none2 is None and torch.equal(only_dx, dx) and torch.equal(only_dg, dg)
    assert again is dx_in


def test_gate_grad_in_place_graph_and_rows_behind():
    import mixture_experts_layer_04_amd as moe
    T, H, E = 200, 512, 96
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    gate = torch.randn(E, H, device="cuda")
    d = torch.randn(T, E, device="cuda")
    buf = torch.full((T + 9, H), 3.0, dtype=torch.bfloat16, device="cuda")
    want, _ = moe.gate_grad(x, gate, d, buf[:T].clone())
    moe.gate_grad(x, gate, d, buf[:T], dx=buf[:T])
    torch.cuda.synchronize()
    assert torch.equal(buf[:T], want) and torch.all(buf[T:] == 3.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx, dg = moe.gate_grad(x, gate, d)
    for i in range(3):
        d.copy_(torch.randn(T, E, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        a, b = moe.gate_grad(x, gate, d)
        torch.cuda.synchronize()
        assert torch.equal(dx, a) and torch.equal(dg, b)


def test_gate_grad_not_finite_and_empty():
    import mixture_experts_layer_04_amd as moe
    T, H, E = 70, 256, 40
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    gate = torch.randn(E, H, device="cuda")
    d = torch.randn(T, E, device="cuda")
    clean, cleang = moe.gate_grad(x, gate, d)
    d[5, 3] = float("nan")
    d[6, 4] = float("inf")
    dx, dg = moe.gate_grad(x, gate, d)
    torch.cuda.synchronize()
    keep = [t for t in range(T) if t not in (5, 6)]
    assert torch.equal(dx[keep], clean[keep]) and not torch.any(torch.isfinite(dx[[5, 6]]))
    rows = [e for e in range(E) if e not in (3, 4)]
    assert torch.equal(dg[rows], cleang[rows]) and not torch.any(torch.isfinite(dg[[3, 4]]))
    dx, dg = moe.gate_grad(x[:0], gate, d[:0])
    torch.cuda.synchronize()
    assert dx.shape == (0, H) and torch.all(dg == 0)


def test_router_backward_as_a_whole():
    """A scalar of the routing weights and both losses, as a function of the
    hidden states and the gate: the calls in a row give the gradient that
    central differences of the float64 forward give."""
    import mixture_experts_layer_04_amd as moe
    from oracle import router as orouter
    T, H, E, k = 24, 128, 16, 3
    g = torch.Generator().manual_seed(11)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    gate = torch.randn(E, H, generator=g) * 0.1
    dw = torch.randn(T, k, generator=g)
    dl = torch.tensor([0.8, 0.05])
    off = [0, 10, 24]
    offd, _ = to_dev(off, None)
    for scoring in SCORINGS:
        ids, w, lg = moe.route(x.cuda(), gate.cuda(), None, k, scoring, return_logits=True, routed_scale=1.7)
        losses, counts, probs, tokens = moe.balance_loss(lg, ids, scoring, offd)
        d = moe.route_grad(lg, ids, scoring, True, 1.7, dw.cuda(), dl.cuda(), counts, tokens, offd)
        dx, dg = moe.gate_grad(x.cuda(), gate.cuda(), d)
        torch.cuda.synchronize()
        idn = ids.cpu().numpy()

        def f(x, gate):
            l = x @ gate.T
            r = ob.balance_loss(l, idn, scoring, off)
            return np.dot(f64(dl), r["losses"]) + np.sum(f64(dw) * ob.weights(l, idn, scoring, True, 1.7))

        assert np.allclose(f64(w), ob.weights(f64(lg), idn, scoring, True, 1.7), rtol=1e-5, atol=1e-6)
        assert orouter.SCORINGS and abs(np.dot(f64(dl), f64(losses)) + np.sum(f64(dw) * f64(w)) -
                                        f(f64(x), f64(gate))) < 1e-3
        rng = np.random.default_rng(0)
        vx, vg = rng.normal(size=x.shape), rng.normal(size=gate.shape)
        step = 1e-5
        px = (f(f64(x) + step * vx, f64(gate)) - f(f64(x) - step * vx, f64(gate))) / (2 * step)
        pg = (f(f64(x), f64(gate) + step * vg) - f(f64(x), f64(gate) - step * vg)) / (2 * step)
        # dx is bf16 (2^-8 of each element); d_gate and the logits' gradient
        # are fp32, on fp32 logits (2^-15 of their size in every derivative)
        assert abs(np.sum(f64(dx) * vx) - px) <= np.sum(np.abs(f64(dx) * vx)) * 2.0 ** -7 + 1e-6
        assert abs(np.sum(f64(dg) * vg) - pg) <= np.sum(np.abs(f64(dg) * vg)) * 2.0 ** -10 + 1e-6
    say("router backward follows the differences")


def test_refusals():
    import mixture_experts_layer_04_amd as moe
    lg, ids = make(16, 32, 4)
    one = torch.ones(2, device="cuda")
    off = torch.tensor([0, 16], dtype=torch.int32, device="cuda")
    losses, counts, probs, tokens = moe.balance_loss(lg, ids)
    x = torch.zeros(16, 128, dtype=torch.bfloat16, device="cuda")
    gate = torch.zeros(32, 128, device="cuda")
    bad = [lambda: moe.balance_loss(lg.double(), ids), lambda: moe.balance_loss(lg, ids.long()),
           lambda: moe.balance_loss(lg, ids[:8]), lambda: moe.balance_loss(lg, ids, seq_offsets=off.long()),
           lambda: moe.balance_loss(lg, ids, seq_offsets=off[:1]), lambda: moe.balance_loss(lg[:, ::2], ids),
           lambda: moe.balance_loss(lg, ids, token_mask=torch.ones(15, device="cuda", dtype=torch.uint8)),
           lambda: moe.balance_loss(lg.cpu(), ids), lambda: moe.route_grad(lg, ids),
           lambda: moe.route_grad(lg, ids, d_losses=one), lambda: moe.route_grad(lg, ids, d_weights=one),
           lambda: moe.route_grad(lg, ids, d_losses=one, counts=counts[:, :8], tokens=tokens),
           lambda: moe.gate_grad(x, gate, lg[:8]), lambda: moe.gate_grad(x, gate.half(), lg),
           lambda: moe.gate_grad(x, gate, lg, dx_in=x, with_dx=False)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    errors = [lambda: moe.balance_loss(lg, ids, n_shared=2), lambda: moe.balance_loss(lg, ids[:, :0].contiguous()),
              lambda: moe.gate_grad(x, gate, lg, with_dx=False, with_gate=False),
              lambda: moe.gate_grad(x[:, :64].contiguous(), gate[:, :64].contiguous(), lg)]
    for f in errors:
        with pytest.raises(moe.MoeError):
            f()


def test_many_sequences():
    """More sequences than one launch totals by its last workgroup, most of
    them one or two tokens long or empty."""
    import mixture_experts_layer_04_amd as moe
    T, E, k = 700, 40, 4
    lg, ids = make(T, E, k)
    rng = np.random.default_rng(3)
    off = np.sort(rng.integers(0, T + 1, size=1500)).tolist()
    offd, _ = to_dev(off, None)
    got = moe.balance_loss(lg, ids, "sigmoid", offd)
    d = moe.route_grad(lg, ids, "sigmoid", d_losses=torch.tensor([900.0, 30.0], device="cuda"), counts=got[1],
                       tokens=got[3], seq_offsets=offd)
    torch.cuda.synchronize()
    ref = ob.balance_loss(f64(lg), ids.cpu().numpy(), "sigmoid", off)
    check_loss(got, ref, lg, ob.members(T, off)[0])
    want, mag = ob.route_grad(f64(lg), ids.cpu().numpy(), "sigmoid", True, 1.0, None, np.array([900.0, 30.0]),
                              ref["counts"], off)
    assert np.all(np.abs(f64(d) - want) <= mag * 2.0 ** -15 + 1e-35)
