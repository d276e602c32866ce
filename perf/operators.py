"""The operators around the MoE layer as measured cases: the norm in front of
it and the router's training side, each in a plain form (elementary torch
operations in 32 bits) and as the calls a user makes of the package.

Operators ("op" of a case):

* ``norm``       h = x + residual, y = h rsqrt(mean h^2 + eps) w, with y in
                 bf16 and, with "quant", also in e4m3 with one fp32 scale per
                 128 values ("fp8") or one power-of-two scale per 32 ("mxfp4")
* ``norm_grad``  its gradient: dx (the incoming gradient of h added) and dw
* ``balance``    the load-balance loss over ragged sequences, the z loss and
                 the per-expert counts, from the router's logits and choices
* ``route_grad`` the gradient of both losses and of the routing weights with
                 respect to the logits
* ``gate_grad``  from there to the gate and the hidden states
"""

import math

import torch

own = False

EPS = 1e-6

# Widths of the five layer shapes, and generic ones: norms also run over
# widths that are no multiple of a vector (a shard's or a head's).
_WIDTHS = (256, 1024, 2048, 4096, 5120, 7168)
_ODD_WIDTHS = (100, 777, 1001, 2050, 4095)
_EXPERTS = (8, 60, 64, 100, 128, 160, 256, 288)


def listed():
    return [
        # one decoded token in front of an fp8 layer (H 7168): latency
        dict(name="norm_decode_fp8", op="norm", T=1, H=7168, res="bf16", w="bf16", quant="fp8"),
        # a decode batch with an fp32 residual stream and an fp32 weight
        dict(name="norm_batch_fp32", op="norm", T=64, H=2048, res="fp32", w="fp32", quant="none"),
        # a width that no vector load divides, no residual (a first norm)
        dict(name="norm_odd", op="norm", T=3001, H=1001, res="none", w="bf16", quant="none"),
        # prefill in front of an MXFP4 layer (8192 tokens, H 4096)
        dict(name="norm_prefill_mx", op="norm", T=8192, H=4096, res="bf16", w="bf16", quant="mxfp4"),
        # a small micro-batch's backward
        dict(name="norm_grad_small", op="norm_grad", T=64, H=2048, res="bf16", w="bf16", dh=True),
        # a large micro-batch's backward with an fp32 residual stream
        dict(name="norm_grad_large", op="norm_grad", T=8192, H=7168, res="fp32", w="fp32", dh=True),
        # the losses of a small batch, softmax over 128 experts, one sequence
        dict(name="balance_small", op="balance", T=64, E=128, k=8, seqs=0, mask=False, scoring="softmax"),
        # a packed training batch: ragged sequences, sigmoid over 256 experts, padded tokens masked
        dict(name="balance_packed", op="balance", T=131072, E=256, k=8, seqs=37, mask=True, scoring="sigmoid"),
        # the router's gradient at an ordinary micro-batch, 288 experts
        dict(name="route_grad_512", op="route_grad", T=512, E=288, k=8, seqs=0, mask=False, scoring="sigmoid",
             renorm=True),
        # the same for a packed batch of softmax routing over 128 experts
        dict(name="route_grad_packed", op="route_grad", T=65536, E=128, k=8, seqs=16, mask=True, scoring="softmax",
             renorm=True),
        # gate and hidden-state gradients at a small micro-batch, bf16 gate
        dict(name="gate_grad_512", op="gate_grad", T=512, H=4096, E=288, gate="bf16", dx_in=True),
        # and at a large one (H 7168, 256 experts), fp32 gate
        dict(name="gate_grad_8192", op="gate_grad", T=8192, H=7168, E=256, gate="fp32", dx_in=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "balance", "route_grad", "gate_grad"])
    if op == "norm":
        quant = rng.choice(["none", "fp8", "mxfp4"])
        H = rng.choice(_WIDTHS + (_ODD_WIDTHS if quant == "none" else ()))
        return dict(op=op, T=_log_int(rng, 1, 8192), H=H, res=rng.choice(["none", "bf16", "fp32"]),
                    w=rng.choice(["bf16", "fp32"]), quant=quant)
    if op == "norm_grad":
        return dict(op=op, T=_log_int(rng, 1, 8192), H=rng.choice(_WIDTHS + _ODD_WIDTHS),
                    res=rng.choice(["bf16", "fp32"]), w=rng.choice(["bf16", "fp32"]), dh=rng.random() < 0.7)
    if op in ("balance", "route_grad"):
        E = rng.choice(_EXPERTS)
        T = _log_int(rng, 1, 131072 * 256 // max(E, 128))
        c = dict(op=op, T=T, E=E, k=min(E, rng.choice([1, 2, 6, 8])), seqs=rng.choice([0, 1, 5, 60]),
                 mask=rng.random() < 0.5, scoring=rng.choice(["softmax", "sigmoid", "sqrtsoftplus"]))
        if op == "route_grad":
            c["renorm"] = rng.random() < 0.7
        return c
    return dict(op=op, T=_log_int(rng, 1, 8192), H=rng.choice(_WIDTHS), E=rng.choice(_EXPERTS),
                gate=rng.choice(["bf16", "fp32"]), dx_in=rng.random() < 0.7)


# ---------------------------------------------------------------------------
# inputs

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32, std=1.0, mean=0.0):
    t = torch.randn(*shape, generator=g, device="cuda")
    return (t * std + mean).to(dtype)


def _hidden(g, T, H, dtype):
    """Hidden states: N(0, 1) with a few channels of much larger spread."""
    t = torch.randn(T, H, generator=g, device="cuda")
    t[:, ::97] *= 12.0
    return t.to(dtype)


def _router_state(c, g):
    """Logits of a gate with uneven experts, the choice of the k best scores,
    and the ragged sequences with their padded tokens."""
    T, E, k, S = c["T"], c["E"], c["k"], c["seqs"]
    s = {"logits": _randn(g, T, E, std=1.3) + _randn(g, E, std=0.5)}
    s["ids"] = s["logits"].topk(k, dim=1).indices.to(torch.int32)
    s["offsets"] = s["mask"] = None
    if S:
        # cut points anywhere in the batch (so some sequences may be empty)
        # and rows behind the last sequence
        end = T - T // 50
        cuts = (torch.rand(S - 1, generator=g, device="cuda") * (end + 1)).long().clamp(max=end).sort().values
        s["offsets"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), end)]).to(torch.int32)
    if c["mask"]:
        s["mask"] = (torch.rand(T, generator=g, device="cuda") < 0.9).to(torch.uint8)
    return s


def prepare(case, seed):
    c, g = case, _gen(seed)
    op = c["op"]
    s = {"case": c}
    if op == "norm":
        T, H = c["T"], c["H"]
        s["x"] = _hidden(g, T, H, torch.bfloat16)
        s["residual"] = None if c["res"] == "none" else _hidden(g, T, H, _TYPES[c["res"]])
        s["weight"] = _randn(g, H, std=0.2, mean=1.0, dtype=_TYPES[c["w"]])
        # the buffers that a serving program keeps between its layers
        s["y"] = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        s["h"] = None if s["residual"] is None else torch.empty_like(s["residual"])
        s["q"] = s["s"] = s["q_values"] = s["s_values"] = None
        if c["quant"] != "none":
            s["q"] = torch.empty(T, H, dtype=torch.uint8, device="cuda")
            s["q_values"] = s["q"].view(torch.float8_e4m3fn)
            if c["quant"] == "fp8":
                s["s"] = s["s_values"] = torch.empty(T, H // 128, device="cuda")
            else:
                s["s"] = torch.empty(T, H // 32, dtype=torch.uint8, device="cuda")
                s["s_values"] = s["s"].view(torch.float8_e8m0fnu)
    elif op == "norm_grad":
        T, H = c["T"], c["H"]
        s["h"] = _hidden(g, T, H, _TYPES[c["res"]])
        s["weight"] = _randn(g, H, std=0.2, mean=1.0, dtype=_TYPES[c["w"]])
        s["dy"] = _randn(g, T, H, std=1e-2, dtype=torch.bfloat16)
        s["dh"] = _randn(g, T, H, std=1e-2, dtype=_TYPES[c["res"]]) if c["dh"] else None
    elif op == "balance":
        s.update(_router_state(c, g))
    elif op == "route_grad":
        s.update(_router_state(c, g))
        T, E, k = c["T"], c["E"], c["k"]
        s["d_weights"] = _randn(g, T, k, std=1e-2)
        s["d_losses"] = torch.tensor([1e-2, 1e-3], device="cuda") * (1.0 + torch.rand(2, generator=g, device="cuda"))
        # what the forward call left: counts and token numbers
        seg, n = _segments(s, T)
        s["counts"] = _counts(s["ids"], seg, n, E)
        tokens = (seg[:, None] == torch.arange(n, device="cuda")).sum(0)
        s["tokens"] = torch.cat([tokens, tokens.sum()[None], (tokens > 0).sum()[None]]).to(torch.int32)
    elif op == "gate_grad":
        T, H, E = c["T"], c["H"], c["E"]
        s["x"] = _hidden(g, T, H, torch.bfloat16)
        s["gate"] = _randn(g, E, H, std=0.02, dtype=_TYPES[c["gate"]])
        # small gradients of the losses everywhere, larger ones at the chosen experts
        d = _randn(g, T, E, std=1e-5)
        k = min(E, 8)
        at = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices
        s["d_logits"] = d.scatter_add_(1, at, _randn(g, T, k, std=1e-3))
        s["dx_in"] = _randn(g, T, H, std=1e-3, dtype=torch.bfloat16) if c["dx_in"] else None
    return s


# ---------------------------------------------------------------------------
# the plain forms

def _segments(s, T):
    """The sequence of every token (-1: in none, or masked) and how many."""
    rows = torch.arange(T, device="cuda")
    n = 1
    seg = torch.zeros_like(rows)
    if s["offsets"] is not None:
        off = s["offsets"].long()
        n = off.numel() - 1
        seg = (rows[:, None] >= off[1:][None, :]).sum(1)
        seg = torch.where((rows >= off[0]) & (rows < off[-1]), seg, -1)
    if s["mask"] is not None:
        seg = torch.where(s["mask"] != 0, seg, -1)
    return seg, n


def _counts(ids, seg, n, E):
    """Assignments per (sequence, expert), int32 [n, E]."""
    cell = torch.where(seg[:, None] >= 0, seg[:, None] * E + ids.long(), n * E)
    out = torch.zeros(n * E + 1, dtype=torch.int32, device="cuda")
    out.scatter_add_(0, cell.reshape(-1), torch.ones(cell.numel(), dtype=torch.int32, device="cuda"))
    return out[: n * E].reshape(n, E)


def _scores(l, scoring):
    if scoring == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
        return e / e.sum(1, keepdim=True)
    if scoring == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    return torch.sqrt(l.clamp(min=0) + torch.log1p(torch.exp(-l.abs())))


def _plain_norm(s):
    c = s["case"]
    h = s["x"].float()
    h_out = None
    if s["residual"] is not None:
        h = h + s["residual"].float()
        h_out = h.to(s["residual"].dtype)
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"].float()
    out = {"y": y.to(torch.bfloat16), "h": h_out}
    if c["quant"] != "none":
        T, H = y.shape
        width = 128 if c["quant"] == "fp8" else 32
        grp = y.reshape(T, H // width, width)
        amax = grp.abs().amax(2)
        if c["quant"] == "fp8":
            scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
            out["s"] = scale
        else:
            scale = torch.where(amax > 0, torch.exp2(torch.ceil(torch.log2(amax.double() / 448.0))).float(),
                                torch.ones_like(amax))
            out["s"] = scale.to(torch.float8_e8m0fnu)
        q = (grp / scale[:, :, None]).clamp(-448.0, 448.0)
        out["q"] = q.reshape(T, H).to(torch.float8_e4m3fn)
    return out


def _plain_norm_grad(s):
    h, w, dy = s["h"].float(), s["weight"].float(), s["dy"].float()
    r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    g = dy * w
    dx = r * g - h * (r * r * r * (g * h).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    dw = (dy * h * r).sum(0, dtype=torch.float64).float()
    return {"dx": dx.to(s["h"].dtype), "dw": dw}


def _plain_balance(s):
    c = s["case"]
    l, E, k = s["logits"], c["E"], c["k"]
    seg, n = _segments(s, c["T"])
    live = seg >= 0
    p = _scores(l, c["scoring"])
    if c["scoring"] != "softmax":
        p = p / (p.sum(1, keepdim=True) + 1e-20)
    m = l.amax(1)
    lse = m + torch.log(torch.exp(l - m[:, None]).sum(1))
    counts = _counts(s["ids"], seg, n, E)
    tokens = (seg[:, None] == torch.arange(n, device="cuda")).sum(0)
    total, full = tokens.sum(), (tokens > 0).sum()
    # sums over up to every token of the batch: in 64 bits
    member = (seg[None, :] == torch.arange(n, device="cuda")[:, None]).double()
    sums = torch.matmul(member, p.double())
    probs = sums / tokens.clamp(min=1)[:, None]
    f = counts.double() * E / (k * tokens.clamp(min=1)[:, None])
    loss = (f * probs).sum() / full.clamp(min=1)
    z = torch.where(live, lse, torch.zeros_like(lse)).double().square().sum() / total.clamp(min=1)
    return {"losses": torch.stack([loss, z]).float(), "counts": counts, "probs": probs.float(),
            "tokens": torch.cat([tokens, total[None], full[None]]).to(torch.int32)}


def _plain_route_grad(s):
    c = s["case"]
    l, E, k = s["logits"], c["E"], c["k"]
    seg, n = _segments(s, c["T"])
    live = (seg >= 0)[:, None]
    at = seg.clamp(min=0)
    tokens = s["tokens"][:n].float().clamp(min=1)
    total, full = s["tokens"][n].float().clamp(min=1), s["tokens"][n + 1].float().clamp(min=1)
    gb = s["d_losses"][0] * E / k * s["counts"].float() / (tokens[:, None] * tokens[:, None] * full)
    gb = torch.where(live, gb[at], torch.zeros((), device="cuda"))
    sc = _scores(l, c["scoring"])
    ids = s["ids"].long()
    sel = sc.gather(1, ids)
    dw = s["d_weights"] * SCALE
    if c["renorm"]:
        den = sel.sum(1, keepdim=True) + 1e-20
        dsel = (dw - (dw * sel).sum(1, keepdim=True) / den) / den
    else:
        dsel = dw
    gw = torch.zeros_like(l).scatter_add_(1, ids, dsel)
    m = l.amax(1, keepdim=True)
    e = torch.exp(l - m)
    es = e.sum(1, keepdim=True)
    soft, lse = e / es, m + torch.log(es)
    if c["scoring"] == "softmax":
        g = gb + gw
        d = sc * (g - (sc * g).sum(1, keepdim=True))
    else:
        tot = sc.sum(1, keepdim=True) + 1e-20
        ds = (gb - (sc * gb).sum(1, keepdim=True) / tot) / tot + gw
        sig = 1.0 / (1.0 + torch.exp(-l))
        d = ds * (sig * (1.0 - sig) if c["scoring"] == "sigmoid" else sig / (2.0 * sc))
    return d + torch.where(live, s["d_losses"][1] * 2.0 / total * lse * soft, torch.zeros((), device="cuda"))


def _plain_gate_grad(s):
    d = s["d_logits"]
    dx = torch.matmul(d, s["gate"].float())
    if s["dx_in"] is not None:
        dx = dx + s["dx_in"].float()
    return {"dx": dx.to(torch.bfloat16), "d_gate": torch.matmul(d.t(), s["x"].float())}


SCALE = 2.5  # the routed scale of the weights whose gradient route_grad takes

_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "balance": _plain_balance,
          "route_grad": _plain_route_grad, "gate_grad": _plain_gate_grad}


# ---------------------------------------------------------------------------
# the package's calls

def _own(s):
    import mixture_experts_layer_04_amd as moe
    c = s["case"]
    op = c["op"]
    if op == "norm":
        quant = None if c["quant"] == "none" else c["quant"]
        moe.rms_norm(s["x"], s["weight"], s["residual"], EPS, quant, y=s["y"], h=s["h"], q=s["q"], s=s["s"])
        out = {"y": s["y"], "h": s["h"]}
        if quant is not None:
            out["q"], out["s"] = s["q_values"], s["s_values"]
        return out
    if op == "norm_grad":
        dx, dw = moe.rms_norm_grad(s["dy"], s["h"], s["weight"], EPS, dh=s["dh"])
        return {"dx": dx, "dw": dw}
    if op == "balance":
        losses, counts, probs, tokens = moe.balance_loss(s["logits"], s["ids"], c["scoring"], s["offsets"], s["mask"])
        return {"losses": losses, "counts": counts, "probs": probs, "tokens": tokens}
    if op == "route_grad":
        return moe.route_grad(s["logits"], s["ids"], c["scoring"], c["renorm"], SCALE, d_weights=s["d_weights"],
                              d_losses=s["d_losses"], counts=s["counts"], tokens=s["tokens"],
                              seq_offsets=s["offsets"], token_mask=s["mask"])
    dx, d_gate = moe.gate_grad(s["x"], s["gate"], s["d_logits"], dx_in=s["dx_in"])
    return {"dx": dx, "d_gate": d_gate}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


def work(case):
    c = case
    op, T = c["op"], c["T"]
    size = {"bf16": 2, "fp32": 4, "none": 0}
    if op == "norm":
        H, r = c["H"], size[c["res"]]
        b = T * H * (2 + 2 * r + 2) + H * size[c["w"]]
        if c["quant"] != "none":
            b += T * H + (T * H // 128 * 4 if c["quant"] == "fp8" else T * H // 32)
        return {"bytes": b, "flops": 6 * T * H}
    if op == "norm_grad":
        H, r = c["H"], size[c["res"]]
        return {"bytes": T * H * (2 + 2 * r + (r if c["dh"] else 0)) + H * (size[c["w"]] + 4), "flops": 12 * T * H}
    if op in ("balance", "route_grad"):
        E, k, n = c["E"], c["k"], max(1, c["seqs"])
        b = 4 * T * E + 4 * T * k + (T if c["mask"] else 0) + 4 * n * E
        if op == "balance":
            return {"bytes": b + 4 * n * E, "flops": 8 * T * E}
        return {"bytes": b + 4 * T * k + 4 * T * E, "flops": 16 * T * E}
    H, E = c["H"], c["E"]
    b = T * H * (2 + 2 + (2 if c["dx_in"] else 0)) + 4 * T * E + E * H * (size[c["gate"]] + 4)
    return {"bytes": b, "flops": 4 * T * E * H}


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_rows(s, T):
    """Indicator [n, T] of the tokens of each sequence, in 64 bits."""
    off = [0, T] if s["offsets"] is None else s["offsets"].tolist()
    ind = torch.zeros(len(off) - 1, T, dtype=torch.float64, device="cuda")
    for i in range(len(off) - 1):
        ind[i, off[i]:off[i + 1]] = 1.0
    if s["mask"] is not None:
        ind *= s["mask"].double()
    return ind


def _exact_chosen(ids, E):
    """Times each token chose each expert, [T, E]."""
    out = torch.zeros(ids.shape[0], E, dtype=torch.float64, device="cuda")
    for j in range(ids.shape[1]):
        out[torch.arange(ids.shape[0], device="cuda"), ids[:, j].long()] += 1.0
    return out


def _exact_score(l, scoring):
    """(score, its derivative by the expert's own logit for the scores taken
    expert by expert, None for softmax)."""
    if scoring == "softmax":
        return torch.exp(l - torch.logsumexp(l, 1, keepdim=True)), None
    sig = torch.sigmoid(l)
    if scoring == "sigmoid":
        return sig, sig * torch.sigmoid(-l)
    sc = torch.logaddexp(l, torch.zeros_like(l)).sqrt()
    return sc, sig / (2 * sc)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    op = c["op"]
    if op == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h += s["residual"].double()
        y = s["weight"].double() * h / (torch.linalg.vector_norm(h, dim=1, keepdim=True).square() / c["H"] + EPS).sqrt()
        out = {"y": y, "h": None if s["residual"] is None else h}
        if c["quant"] != "none":
            width = 128 if c["quant"] == "fp8" else 32
            parts = y.unflatten(1, (-1, width))
            top = parts.abs().amax(-1, keepdim=True) / 448
            if c["quant"] == "mxfp4":
                frac, exponent = torch.frexp(top)
                top = torch.ldexp(torch.ones_like(frac), exponent - (frac == 0.5).to(exponent.dtype))
            out["s"] = top[..., 0]
            out["q"] = (parts / top).float().to(torch.float8_e4m3fn).double().flatten(1)
        return out
    if op == "norm_grad":
        h, w, dy = s["h"].double(), s["weight"].double(), s["dy"].double()
        size = (h.square().sum(1, keepdim=True) / c["H"] + EPS).sqrt()
        unit = h / size
        g = dy * w
        dx = (g - unit * (g * unit).sum(1, keepdim=True) / c["H"]) / size
        if s["dh"] is not None:
            dx += s["dh"].double()
        return {"dx": dx, "dw": (dy * unit).sum(0)}
    if op in ("balance", "route_grad"):
        l, E, k, T = s["logits"].double(), c["E"], c["k"], c["T"]
        ind = _exact_rows(s, T)
        tokens = ind.sum(1)
        full = max(1.0, float((tokens > 0).sum()))
        total = max(1.0, float(tokens.sum()))
        some = tokens.clamp(min=1)[:, None]
        sc, ds_dl = _exact_score(l, c["scoring"])
        if op == "balance":
            p = (sc / sc.sum(1, keepdim=True)) * ind.sum(0)[:, None]
            upto = torch.cat([p.new_zeros(1, E), p.cumsum(0)])
            off = torch.tensor([0, T]) if s["offsets"] is None else s["offsets"].long().cpu()
            probs = (upto[off[1:].cuda()] - upto[off[:-1].cuda()]) / some
            share = E / k * (ind @ _exact_chosen(s["ids"], E)) / some
            z = (ind.sum(0) * torch.logsumexp(l, 1) ** 2).sum() / total
            return {"losses": torch.stack([(share * probs).sum() / full, z]), "counts": None, "probs": probs,
                    "tokens": None}
        rows = ind.sum(0)[:, None]
        a, b = float(s["d_losses"][0]), float(s["d_losses"][1])
        gb = ind.t() @ (a * E / k * s["counts"].double() / some ** 2 / full)
        # the weights' gradient, slot by slot, on the scores
        pick = torch.arange(T, device="cuda")
        chosen = [s["ids"][:, j].long() for j in range(k)]
        den = sum(sc[pick, e] for e in chosen)
        dw = s["d_weights"].double() * SCALE
        mean = sum(dw[:, j] * sc[pick, e] for j, e in enumerate(chosen)) / den
        gw = torch.zeros_like(l)
        for j, e in enumerate(chosen):
            gw[pick, e] += (dw[:, j] - mean) / den if c["renorm"] else dw[:, j]
        if ds_dl is None:
            g = gb + gw
            d = sc * g - sc * (sc * g).sum(1, keepdim=True)
        else:
            tot = sc.sum(1, keepdim=True)
            p = sc / tot
            d = ds_dl * ((gb - (p * gb).sum(1, keepdim=True)) / tot + gw)
        return d + 2 * b / total * rows * torch.logsumexp(l, 1, keepdim=True) * torch.softmax(l, 1)
    d = s["d_logits"].double()
    dx = d @ s["gate"].double()
    if s["dx_in"] is not None:
        dx += s["dx_in"].double()
    return {"dx": dx, "d_gate": d.t().contiguous() @ s["x"].double()}
