"""Oracle of the router's training side in float64: the balance and z losses
with the per-expert counts, their gradient (and the routing weights') to the
logits, and from there to the gate and the hidden states.

Test infrastructure only (see ``oracle/__init__``).  The balance loss is the
product of an expert's share of the assignments and its mean probability,
summed over the experts (Fedus et al., "Switch Transformers", eq. 4 to 6, for
top-k and per sequence as in the DeepSeek-V3 report, "Complementary
Sequence-Wise Auxiliary Loss"); the z loss is the mean squared log-sum-exp of
the logits (Zoph et al., "ST-MoE", eq. 5).  Every gradient is checked against
central differences of the forward functions in the tests.
"""

import numpy as np

from .router import scores

TINY = 1e-20


def members(T, offsets=None, mask=None):
    """The sequence of every row (-1: takes no part) and their number."""
    seq = np.zeros(T, dtype=np.int64)
    n = 1
    if offsets is not None:
        n = len(offsets) - 1
        seq[:] = -1
        for s in range(n):
            seq[offsets[s]:offsets[s + 1]] = s
    if mask is not None:
        seq[np.asarray(mask) == 0] = -1
    return seq, n


def _probabilities(lg, scoring):
    """Scores (a row of -inf scores zero) and p = score / sum."""
    with np.errstate(invalid="ignore"):
        sc = scores(lg, scoring)
    sc = np.where(np.all(lg == -np.inf, axis=1, keepdims=True), 0.0, sc)
    if scoring == "softmax":
        return sc, sc
    return sc, sc / (sc.sum(axis=1, keepdims=True) + TINY)


def _lse(lg):
    m = np.where(np.all(lg == -np.inf, axis=1), 0.0, lg.max(axis=1, initial=-np.inf))
    es = np.exp(lg - m[:, None]).sum(axis=1)
    with np.errstate(divide="ignore"):
        return np.where(es > 0, m + np.log(es), 0.0)


def balance_loss(lg, ids, scoring, offsets=None, mask=None):
    """ids [T, k] without shared slots; ids outside [0, E) do not count."""
    lg = np.asarray(lg, dtype=np.float64)
    T, E = lg.shape
    k = ids.shape[1]
    seq, n = members(T, offsets, mask)
    rows = [np.nonzero(seq == s)[0] for s in range(n)]
    counts = np.zeros((n, E), dtype=np.int64)
    probs = np.zeros((n, E))
    loss, z = 0.0, 0.0
    tokens = np.array([len(r) for r in rows], dtype=np.int64)
    full, total = int((tokens > 0).sum()), int(tokens.sum())
    for s, r in enumerate(rows):
        if not len(r):
            continue
        got = ids[r].reshape(-1)
        got = got[(got >= 0) & (got < E)]
        counts[s] = np.bincount(got, minlength=E)
        probs[s] = _probabilities(lg[r], scoring)[1].mean(axis=0)
        loss += np.sum(E * counts[s] / (k * len(r)) * probs[s])
        z += np.sum(_lse(lg[r]) ** 2)
    return {"losses": np.array([loss / max(full, 1), z / max(total, 1)]), "counts": counts, "probs": probs,
            "tokens": np.concatenate([tokens, [total, full]])}


def weights(lg, ids, scoring, renormalize, scale):
    """The routing weights of given slots (0 for an id outside [0, E))."""
    lg = np.asarray(lg, dtype=np.float64)
    E = lg.shape[1]
    sc, _ = _probabilities(lg, scoring)
    ok = (ids >= 0) & (ids < E)
    sel = np.where(ok, np.take_along_axis(sc, np.where(ok, ids, 0), axis=1), 0.0)
    if renormalize:
        sel = sel / (sel.sum(axis=1, keepdims=True) + TINY)
    return sel * scale


def route_grad(lg, ids, scoring, renormalize, scale, d_weights=None, d_losses=None, counts=None, offsets=None,
               mask=None):
    """(d_logits, magnitude): the gradient and the sum of the magnitudes of
    the terms that it adds up (for error bounds)."""
    lg = np.asarray(lg, dtype=np.float64)
    T, E = lg.shape
    k = ids.shape[1]
    sc, p = _probabilities(lg, scoring)
    seq, n = members(T, offsets, mask)
    tokens = np.array([(seq == s).sum() for s in range(n)])
    gb, beta = np.zeros_like(lg), np.zeros(T)
    if d_losses is not None:
        full, total = max((tokens > 0).sum(), 1), max(tokens.sum(), 1)
        for t in range(T):
            if seq[t] >= 0:
                gb[t] = d_losses[0] * E * counts[seq[t]] / (k * tokens[seq[t]] ** 2 * full)
        beta = np.where(seq >= 0, d_losses[1] * 2.0 / total * _lse(lg), 0.0)
    gw, gw_mag = np.zeros_like(lg), np.zeros_like(lg)
    if d_weights is not None:
        ok = (ids >= 0) & (ids < E)
        at = np.where(ok, ids, 0)
        sel = np.where(ok, np.take_along_axis(sc, at, axis=1), 0.0)
        dw = np.where(ok, d_weights, 0.0) * scale
        ds, ds_mag = dw, np.abs(dw)
        if renormalize:
            den = sel.sum(axis=1, keepdims=True) + TINY
            ds = (dw - (dw * sel).sum(axis=1, keepdims=True) / den) / den
            ds_mag = (np.abs(dw) + (np.abs(dw) * sel).sum(axis=1, keepdims=True) / den) / den
        for j in range(k):
            rows = np.nonzero(ok[:, j])[0]
            gw[rows, at[rows, j]] += ds[rows, j]
            gw_mag[rows, at[rows, j]] += ds_mag[rows, j]
    with np.errstate(invalid="ignore"):
        soft = np.where(np.all(lg == -np.inf, axis=1, keepdims=True), 0.0, scores(lg, "softmax"))
    z, z_mag = beta[:, None] * soft, np.abs(beta)[:, None] * soft
    if scoring == "softmax":
        g, g_mag = gb + gw, np.abs(gb) + gw_mag
        d = p * (g - (p * g).sum(axis=1, keepdims=True))
        mag = p * (g_mag + (p * g_mag).sum(axis=1, keepdims=True))
    else:
        with np.errstate(over="ignore", divide="ignore", invalid="ignore"):
            sig = 1.0 / (1.0 + np.exp(-lg))
            slope = sig * (1.0 / (1.0 + np.exp(lg))) if scoring == "sigmoid" else np.where(sc > 0, sig / (2 * sc), 0.0)
        tot = sc.sum(axis=1, keepdims=True) + TINY
        d = slope * ((gb - (p * gb).sum(axis=1, keepdims=True)) / tot + gw)
        mag = slope * ((np.abs(gb) + (p * np.abs(gb)).sum(axis=1, keepdims=True)) / tot + gw_mag)
    return d + z, mag + z_mag


def gate_grad(x, gate, d_logits, dx_in=None):
    """{"dx", "d_gate"} and the magnitudes "dx_mag", "d_gate_mag"."""
    x, gate, d = (np.asarray(a, dtype=np.float64) for a in (x, gate, d_logits))
    dx, mag = d @ gate, np.abs(d) @ np.abs(gate)
    if dx_in is not None:
        dx = dx + dx_in
        mag = mag + np.abs(dx_in)
    return {"dx": dx, "d_gate": d.T @ x, "dx_mag": mag, "d_gate_mag": np.abs(d).T @ np.abs(x)}
