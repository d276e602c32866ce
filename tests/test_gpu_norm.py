"""moe_rms_norm, its gradient and moe_norm_layer on the GPU against the
float64 oracle.

Error bounds (u = 2^-24, the half step of fp32): a row's sum of squares adds
at most 32 values per thread, 7 lane steps and 16 waves, each with a relative
error of u, so r = rsqrt(...) is within 2^-18 (half of the sum's 55 u, the
division's and the hardware root's 3 u); y adds 2 u and one bf16 rounding of
2^-8.  The gradient's second sum has the same depth: within 2^-17 of the sum
of the magnitudes with the three factors r; with the row's other factors
2^-16 covers it.  The weight's gradient adds at most T / groups + 81 terms
of relative error u and r's 2^-18: 2^-16 of the magnitudes for T <= 16384.
"""

import numpy as np
import pytest
import torch

from helpers import check_output, oracle_layer, oracle_route, routing_for_layer, say
from oracle import norm as onorm
from synth import get_config, make_weights

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
HALF_BF16 = torch.finfo(BF16).eps / 2


def f64(t):
    return None if t is None else t.detach().to(torch.float64).cpu().numpy()


def make(T, H, res, w, seed=0, big=True):
    g = torch.Generator().manual_seed(1000 * T + H + seed)
    x = torch.randn(T, H, generator=g)
    if big and H > 3:
        x[:, 3] *= 50.0
    r = None if res is None else torch.randn(T, H, generator=g).mul(3.0).to(res).cuda()
    return x.to(BF16).cuda(), r, torch.randn(H, generator=g).mul(0.3).add(1.0).to(w).cuda()


def check_norm(x, r, w, y, h, eps=1e-6):
    rh, ry = onorm.rms_norm(f64(x), f64(w), eps, f64(r))
    assert np.all(np.abs(f64(y) - ry) <= np.abs(ry) * (HALF_BF16 + 2.0 ** -17))
    if r is None:
        assert h is None
    else:
        half = torch.finfo(r.dtype).eps / 2
        assert h.dtype == r.dtype
        assert np.all(np.abs(f64(h) - rh) <= np.abs(rh) * (half + 2.0 ** -24) * (1 + 2.0 ** -20))
    return rh, ry


SHAPES = [(1, 1), (1, 7), (3, 8), (1, 64), (5, 100), (2, 512), (3, 513), (7, 777), (4, 1001), (300, 1024), (2, 2050),
          (1, 4095), (64, 4096), (3, 5120), (1, 7168), (300, 7168), (2, 8200), (3, 16384), (2, 32768)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("res,w", [(None, BF16), (BF16, BF16), (BF16, FP32), (FP32, FP32)])
def test_norm(T, H, res, w):
    import mixture_experts_layer_04_amd as moe
    x, r, wt = make(T, H, res, w)
    y, h = moe.rms_norm(x, wt, r, 1e-6)
    torch.cuda.synchronize()
    check_norm(x, r, wt, y, h)


def e4m3(q):
    return q.view(torch.float8_e4m3fn).to(torch.float64).cpu().numpy()


def check_quant(quant, q, s, ry):
    """Codes and scales against the float64 values they stand for."""
    T, H = ry.shape
    width = 128 if quant == "fp8" else 32
    grp = ry.reshape(T, H // width, width)
    amax = np.abs(grp).max(axis=2)
    if quant == "fp8":
        sc = f64(s)
        assert np.all(np.abs(sc - amax / 448)[amax > 0] <= (amax / 448 * 2.0 ** -16)[amax > 0])
        assert np.all(sc[amax == 0] == 1.0)
    else:
        sc = np.exp2(s.cpu().numpy().astype(np.float64) - 127)
        some = amax > 0
        assert np.all(sc[some] >= amax[some] / 448 * (1 - 2.0 ** -16))
        assert np.all(sc[some] / 2 < amax[some] / 448 * (1 + 2.0 ** -16))
        assert np.all(sc[~some] == 1.0)
    got = e4m3(q).reshape(grp.shape)
    want = grp / sc[:, :, None]
    # half an e4m3 step: 2^-4 of the value, 2^-10 among the subnormals
    bound = np.maximum(np.abs(want) * 2.0 ** -4, 2.0 ** -10) * (1 + 2.0 ** -12) + np.abs(want) * 2.0 ** -16
    assert np.all(np.abs(got - want) <= bound)
    # and all but the values next to a rounding border are the nearest code
    near = torch.from_numpy(want).clamp(-448, 448).to(FP32).to(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.mean(got != near) <= 1e-3


@pytest.mark.parametrize("quant", ["fp8", "mxfp4"])
@pytest.mark.parametrize("T,H", [(1, 128), (3, 256), (17, 1024), (1, 7168), (300, 7168), (5, 4096), (2, 1152),
                                 (2, 32768)])
@pytest.mark.parametrize("res", [None, BF16, FP32])
def test_norm_quantised(quant, T, H, res):
    import mixture_experts_layer_04_amd as moe
    x, r, wt = make(T, H, res, FP32)
    wt[: min(H, 128)] *= 0.0 if T == 3 else 1.0  # a group of zeros
    x[-1, 128:] *= 2.0 ** -20  # groups of very different sizes in one row
    y, h, q, s = moe.rms_norm(x, wt, r, 1e-6, quant)
    torch.cuda.synchronize()
    _, ry = check_norm(x, r, wt, y, h)
    check_quant(quant, q, s, ry)
    y2, h2, q2, s2 = moe.rms_norm(x, wt, r, 1e-6, quant, with_y=False)
    assert y2 is None and torch.equal(q2, q) and torch.equal(s2, s)


def test_mx_widths_of_one_group():
    import mixture_experts_layer_04_amd as moe
    for H in (32, 96, 544):
        x, r, wt = make(4, H, BF16, BF16)
        y, h, q, s = moe.rms_norm(x, wt, r, 1e-6, "mxfp4")
        torch.cuda.synchronize()
        _, ry = check_norm(x, r, wt, y, h)
        check_quant("mxfp4", q, s, ry)


def test_norm_rows_do_not_mix():
    """A row's result is the same alone and in a batch, and a row of NaN,
    infinities or zeros leaves the others alone."""
    import mixture_experts_layer_04_amd as moe
    for T, H in ((9, 1024), (300, 7168), (5, 200)):
        x, r, wt = make(T, H, FP32, BF16)
        y, h = moe.rms_norm(x, wt, r)
        x2 = x.clone()
        x2[1] = 0
        r[1] = 0
        x2[2, 5] = float("nan")
        x2[4, 7] = float("inf")
        y2, _ = moe.rms_norm(x2, wt, r)
        torch.cuda.synchronize()
        keep = [i for i in range(T) if i not in (1, 2, 4)]
        assert torch.equal(y2[keep], y[keep])
        assert torch.all(y2[1] == 0) and torch.all(torch.isnan(y2[2]))
        assert torch.isnan(y2[4, 7]) and torch.all(y2[4, :7] == 0)
    x, r, wt = make(3, 256, None, BF16)
    x[1, 9] = float("nan")
    for quant in ("fp8", "mxfp4"):
        y, _, q, s = moe.rms_norm(x, wt, None, 1e-6, quant)
        torch.cuda.synchronize()
        assert torch.all((q[1] & 0x7F) == 0x7F) and not torch.any((q[[0, 2]] & 0x7F) == 0x7F)
        assert torch.all(s[1] == (1.0 if quant == "fp8" else 127))


def test_norm_in_place():
    import mixture_experts_layer_04_amd as moe
    for T, H in ((1, 7168), (300, 4096), (7, 777)):
        x, r, wt = make(T, H, BF16, BF16)
        y, h = moe.rms_norm(x, wt, r)
        moe.rms_norm(x, wt, r, y=x, h=r)
        torch.cuda.synchronize()
        assert torch.equal(x, y) and torch.equal(r, h)
        x2, _, _ = make(T, H, BF16, BF16)
        r2, _, _ = make(T, H, BF16, BF16, seed=1)
        y, h = moe.rms_norm(x2, wt, r2)
        moe.rms_norm(x2, wt, r2, h=x2)
        torch.cuda.synchronize()
        assert torch.equal(x2, h)


def test_norm_leaves_the_rows_behind_alone():
    import mixture_experts_layer_04_amd as moe
    T, H = 5, 1001
    x, r, wt = make(T, H, FP32, BF16)
    y = torch.full((T + 3, H), 7.0, dtype=BF16, device="cuda")
    h = torch.full((T + 3, H), 7.0, device="cuda")
    moe.rms_norm(x, wt, r, y=y[:T], h=h[:T])
    torch.cuda.synchronize()
    assert torch.all(y[T:] == 7) and torch.all(h[T:] == 7)


def test_norm_of_an_offset_view():
    """Rows that start at any element: nothing needs a wider alignment."""
    import mixture_experts_layer_04_amd as moe
    for H in (64, 1001, 4096):
        base = torch.randn(3 * H + 8, device="cuda").to(BF16)
        x = base[1:1 + 3 * H].view(3, H)
        _, _, wt = make(3, H, None, BF16)
        y, _ = moe.rms_norm(x, wt)
        want, _ = moe.rms_norm(x.clone(), wt)
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_norm_empty():
    import mixture_experts_layer_04_amd as moe
    x = torch.empty(0, 256, dtype=BF16, device="cuda")
    w = torch.ones(256, device="cuda")
    y, h = moe.rms_norm(x, w, torch.empty(0, 256, device="cuda"))
    assert y.shape == (0, 256) and h.shape == (0, 256)
    dx, dw = moe.rms_norm_grad(x, x, w)
    torch.cuda.synchronize()
    assert dx.shape == (0, 256) and torch.all(dw == 0)


GRAD_SHAPES = [(1, 1), (2, 9), (1, 64), (5, 100), (3, 513), (70, 777), (33, 1001), (64, 2048), (1500, 1024),
               (1, 7168), (1100, 7168), (5000, 256), (3, 8200), (2, 32768)]


@pytest.mark.parametrize("T,H", GRAD_SHAPES)
@pytest.mark.parametrize("ht,w,with_dh", [(BF16, BF16, True), (FP32, FP32, True), (BF16, FP32, False)])
def test_norm_grad(T, H, ht, w, with_dh):
    import mixture_experts_layer_04_amd as moe
    x, h, wt = make(T, H, ht, w)
    dy = make(T, H, None, w, seed=5, big=False)[0]
    dh = make(T, H, ht, w, seed=6)[1] if with_dh else None
    dx, dw = moe.rms_norm_grad(dy, h, wt, 1e-6, dh)
    torch.cuda.synchronize()
    ref = onorm.rms_norm_grad(f64(dy), f64(h), f64(wt), 1e-6, f64(dh))
    half = torch.finfo(ht).eps / 2
    assert dx.dtype == ht and dw.dtype == FP32
    assert np.all(np.abs(f64(dx) - ref["dx"]) <= np.abs(ref["dx"]) * half + ref["dx_mag"] * 2.0 ** -16)
    assert np.all(np.abs(f64(dw) - ref["dw"]) <= ref["dw_mag"] * 2.0 ** -16)
    dx2, none = moe.rms_norm_grad(dy, h, wt, 1e-6, dh, with_weight=False)
    assert none is None and torch.equal(dx2, dx)
    dx3, dw3 = moe.rms_norm_grad(dy, h, wt, 1e-6, dh, dx=h if dh is None else dh)
    torch.cuda.synchronize()
    assert torch.equal(dx3, dx) and torch.equal(dw3, dw)  # in place, and the same sums every time


NARROW = [(1, 3), (77, 5), (1003, 7), (64, 8), (513, 9), (300, 31), (5, 40), (1001, 63), (4097, 64), (33, 65),
          (515, 127), (9000, 128), (1030, 129), (70, 200), (2, 255), (2053, 256), (129, 257)]


@pytest.mark.parametrize("T,H", NARROW)
@pytest.mark.parametrize("res,w", [(None, FP32), (BF16, BF16), (FP32, BF16)])
def test_narrow_rows(T, H, res, w):
    """Rows of up to 256 values share a wave (8, 4 or 2 of them): the norm, in
    place too, and its gradient, with rows in the last wave that do not
    exist."""
    test_norm(T, H, res, w)
    test_norm_grad(T, H, BF16 if res is None else res, w, res is not None)
    import mixture_experts_layer_04_amd as moe
    x, r, wt = make(T, H, res, w)
    y, h = moe.rms_norm(x, wt, r)
    y1, h1 = moe.rms_norm(x, wt, r, y=x, h=r)
    torch.cuda.synchronize()
    assert torch.equal(y1, y) and (h is None or torch.equal(h1, h))


@pytest.mark.parametrize("quant", ["fp8", "mxfp4"])
@pytest.mark.parametrize("T,H", [(1001, 32), (1001, 64), (259, 96), (1001, 128), (67, 160), (515, 256)])
def test_narrow_rows_quantised(quant, T, H):
    import mixture_experts_layer_04_amd as moe
    if quant == "fp8" and H % 128:
        with pytest.raises(ValueError):
            moe.rms_norm(*make(T, H, None, FP32)[::2], quant=quant)
        return
    x, r, wt = make(T, H, BF16, FP32)
    x[T // 2], r[T // 2] = 0, 0
    y, h, q, s = moe.rms_norm(x, wt, r, 1e-6, quant)
    torch.cuda.synchronize()
    _, ry = check_norm(x, r, wt, y, h)
    check_quant(quant, q, s, ry)


@pytest.mark.parametrize("T,H", [(700, 20001), (300, 16385), (3, 32767), (260, 24576)])
@pytest.mark.parametrize("ht", [BF16, FP32])
def test_wide_rows(T, H, ht):
    """Above 16384 values the weight gradient's sums lie in LDS, over several
    rows of a workgroup; odd widths in place."""
    test_norm_grad(T, H, ht, FP32 if ht == BF16 else BF16, True)


def test_norm_grad_follows_differences_of_the_forward():
    """The step of y along a direction, taken in the fp32 forward, is the
    gradient's inner product with it."""
    T, H, eps = 4, 96, 1e-6
    import mixture_experts_layer_04_amd as moe
    g = torch.Generator().manual_seed(1)
    h = torch.randn(T, H, generator=g)
    wt = torch.randn(H, generator=g)
    dy = torch.randn(T, H, generator=g).to(BF16)
    step = torch.randn(T, H, generator=g)
    dx, _ = moe.rms_norm_grad(dy.cuda(), h.cuda(), wt.cuda(), eps)
    f = lambda v: np.sum(f64(dy) * onorm.rms_norm(f64(v.double()), f64(wt), eps)[1])  # noqa: E731
    d = (f(h.double() + 1e-5 * step) - f(h.double() - 1e-5 * step)) / 2e-5
    got = float((dx.cpu().double() * step.double()).sum())
    # the differences' own error is O(1e-10); dx is within 2^-16 of its terms
    mag = onorm.rms_norm_grad(f64(dy), f64(h), f64(wt), eps)["dx_mag"]
    assert abs(got - d) <= 2.0 ** -15 * np.sum(mag * np.abs(f64(step))) + 1e-6


LAYERS = [("qwen3", dict(E=16, F=256), 1, None), ("qwen3", dict(E=16, F=256), 70, FP32),
          ("dsv3", dict(E=32, F=512, H=1024), 3, BF16), ("dsv3", dict(E=32, F=512, H=1024), 200, FP32),
          ("dsv4", dict(E=16, F=512, H=1024), 2, BF16), ("dsv4", dict(E=16, F=512, H=1024), 300, None)]


@pytest.mark.parametrize("name,over,T,res", LAYERS)
def test_norm_layer(name, over, T, res):
    """The layer on the norm of x + residual, against the oracle's layer on
    the oracle's norm; the steps called one by one give the same routing,
    and for bf16 experts the same bits."""
    import mixture_experts_layer_04_amd as moe
    cfg = get_config(name, **over)
    wts = make_weights(cfg, "cuda")
    x, r, nw = make(T, cfg.H, res, BF16, big=False)
    kw = dict(scoring=cfg.scoring, n_group=cfg.n_group, topk_group=cfg.topk_group, renormalize=cfg.renormalize,
              routed_scale=cfg.routed_scale, wformat=cfg.wformat, w13_scale=wts["w13_scale"],
              w2_scale=wts["w2_scale"], return_routing=True)
    y, h, ids, w = moe.norm_layer(x, nw, wts["gate"], wts["bias"], wts["w13"], wts["w2"], cfg.k, residual=r, **kw)
    yn, hn = moe.rms_norm(x, nw, r)
    y1, ids1, w1 = moe.layer(yn, wts["gate"], wts["bias"], wts["w13"], wts["w2"], cfg.k, **kw)
    torch.cuda.synchronize()
    check_norm(x, r, nw, yn, hn)
    assert torch.equal(ids, ids1) and torch.equal(w, w1)
    assert (h is None) == (r is None) and (r is None or torch.equal(h, hn))
    if cfg.wformat == "bf16":
        assert torch.equal(y, y1)
    ro = oracle_route(cfg, yn, wts["gate"], wts["bias"])
    routing = routing_for_layer(cfg, ro, ids.cpu().numpy())
    ref = oracle_layer(cfg, yn, routing, wts)
    check_output(f64(y), ref, {"bf16": 2e-2, "fp8": 5e-2, "mxfp4": 5e-2}[cfg.wformat])


def test_norm_and_gradient_in_a_graph():
    import mixture_experts_layer_04_amd as moe
    T, H = 130, 1024
    x, r, wt = make(T, H, BF16, BF16)
    dy = make(T, H, None, BF16, seed=2)[0]
    y, h = torch.empty_like(x), torch.empty_like(r)
    moe.rms_norm(x, wt, r, y=y, h=h)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.rms_norm(x, wt, r, y=y, h=h)
        dx, dw = moe.rms_norm_grad(dy, h, wt)
    for i in range(4):
        x.copy_(make(T, H, None, BF16, seed=10 + i)[0])
        graph.replay()
        torch.cuda.synchronize()
        y1, h1 = moe.rms_norm(x, wt, r)
        dx1, dw1 = moe.rms_norm_grad(dy, h1, wt)
        torch.cuda.synchronize()
        assert torch.equal(y, y1) and torch.equal(h, h1) and torch.equal(dx, dx1) and torch.equal(dw, dw1)


def test_two_streams_at_once():
    import mixture_experts_layer_04_amd as moe
    sets = [make(700, 2048, FP32, BF16, seed=i) for i in range(2)]
    dys = [make(700, 2048, None, BF16, seed=20 + i)[0] for i in range(2)]
    want = [moe.rms_norm_grad(dy, s[1], s[2]) for dy, s in zip(dys, sets)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = moe.rms_norm_grad(dys[i], sets[i][1], sets[i][2])
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_norm_refusals():
    import mixture_experts_layer_04_amd as moe
    x, r, wt = make(4, 256, BF16, BF16)
    bad = [lambda: moe.rms_norm(x.float(), wt), lambda: moe.rms_norm(x[0], wt), lambda: moe.rms_norm(x, wt[:128]),
           lambda: moe.rms_norm(x, wt.half()), lambda: moe.rms_norm(x, wt, r[:2]),
           lambda: moe.rms_norm(x.t(), wt), lambda: moe.rms_norm(x, wt, r.cpu()), lambda: moe.rms_norm(x, wt, h=r),
           lambda: moe.rms_norm(x, wt, r, h=r.float()), lambda: moe.rms_norm(x, wt, quant="int8"),
           lambda: moe.rms_norm(x, wt, q=torch.empty(4, 256, dtype=torch.uint8, device="cuda")),
           lambda: moe.rms_norm(x[:, :200].contiguous(), wt[:200], quant="fp8"),
           lambda: moe.rms_norm(x[:, :48].contiguous(), wt[:48], quant="mxfp4"),
           lambda: moe.rms_norm_grad(x, r.float(), wt, dh=r), lambda: moe.rms_norm_grad(x, r, wt, dx=r.float()),
           lambda: moe.rms_norm_grad(x, r[:, :128], wt)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(moe.MoeError):
            moe.rms_norm(x, wt, eps=eps)
    wide = torch.zeros(1, 32776, dtype=BF16, device="cuda")
    with pytest.raises(moe.MoeError):
        moe.rms_norm(wide, torch.ones(32776, device="cuda"))
    say("refusals raised")
