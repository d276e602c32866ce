"""Python binding of libmoe: same names as the C ABI, torch tensors in and
out.  Argument marshalling only - every step runs in the HIP kernels.

Tensors must be CUDA (HIP) tensors, contiguous, with the dtypes of
include/moe.h: x bf16 [T, H]; gate float32 or bf16 [E, H] (the dtype sets
gate_is_fp32); bias float32 [E] or None;
w13 / w2 in the layout of the weight format (bf16, or uint8 codes plus
float32 (fp8) / uint8 e8m0 (mxfp4) scales).  Work goes onto the current
stream of the tensors' device.  The norm and the router's training side
(rms_norm, rms_norm_grad, balance_loss, route_grad, gate_grad) check shapes,
types and devices and raise ValueError; where they need scratch memory they
take it from torch's allocator per call, so calls on several streams and in
several captured graphs do not meet in it.  Everywhere else the workspace is a zero-initialised byte tensor cached per device
(or passed in); calls that overlap in time must not share one.
"""

import math

import torch

from ._lib import SCORING, STAGE, WFORMAT, MoeError, check, lib

_WS = {}
# Workspaces the cache has outgrown.  They are never freed: a HIP graph
# captured with one keeps its address, and freeing it would let its replays
# write router partials and tile-queue counters into another tensor's memory.
_WS_RETIRED = []


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(device):
    return torch.cuda.current_stream(device).cuda_stream


def workspace(device, nbytes):
    """A zero-filled workspace of at least ``nbytes`` on ``device`` (cached,
    grown on demand; the library leaves its counters at zero after each call,
    so the cached buffer stays valid; an outgrown one is kept alive, not
    freed, since a captured graph may still use it)."""
    device = torch.device(device)
    key = device.index if device.index is not None else torch.cuda.current_device()
    ws = _WS.get(key)
    if ws is None or ws.numel() < nbytes:
        if ws is not None:
            _WS_RETIRED.append(ws)
        ws = torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)
        _WS[key] = ws
    return ws


def _check_cuda(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("libmoe ops take GPU tensors")
            if not t.is_contiguous():
                raise ValueError("libmoe ops take contiguous tensors")


def _gate_is_fp32(gate):
    if gate.dtype == torch.float32:
        return 1
    if gate.dtype == torch.bfloat16:
        return 0
    raise ValueError(f"the gate is float32 or bfloat16, not {gate.dtype}")


def align_max_padded(T, k, E, block_m):
    return int(lib().moe_align_max_padded(T, k, E, block_m))


def align_max_blocks(T, k, E, block_m):
    return int(lib().moe_align_max_blocks(T, k, E, block_m))


def layer_block_m(T, k, E, F, wformat="bf16"):
    return int(lib().moe_layer_block_m(T, E, F, k, WFORMAT[wformat]))


def route(x, gate, bias, k, scoring="softmax", n_group=1, topk_group=1, renormalize=True,
          routed_scale=1.0, return_logits=False, ws=None):
    """moe_route -> (topk_ids int32 [T, k], topk_weights float32 [T, k][, logits])."""
    _check_cuda(x, gate, bias)
    T, H = x.shape
    E = gate.shape[0]
    ids = torch.empty((T, k), dtype=torch.int32, device=x.device)
    w = torch.empty((T, k), dtype=torch.float32, device=x.device)
    logits = torch.empty((T, E), dtype=torch.float32, device=x.device) if return_logits else None
    need = lib().moe_route_workspace_size(T, H, E)
    ws = workspace(x.device, need) if ws is None else ws
    check(lib().moe_route(_ptr(x), _ptr(gate), _gate_is_fp32(gate), _ptr(bias), T, H, E, k, n_group, topk_group,
                          SCORING[scoring], int(bool(renormalize)), float(routed_scale),
                          _ptr(ids), _ptr(w), _ptr(logits), _ptr(ws), ws.numel(), _stream(x.device)),
          "moe_route")
    return (ids, w, logits) if return_logits else (ids, w)


def route_align(x, gate, bias, k, block_m, scoring="softmax", n_group=1, topk_group=1, renormalize=True,
                routed_scale=1.0, ws=None, n_shared=0):
    """moe_route_align -> (topk_ids, topk_weights, sorted_ids, block_expert, num_post_padded [1]);
    with n_shared = 1 the ids / weights have k + 1 slots (slot k: the shared expert E, weight 1)."""
    _check_cuda(x, gate, bias)
    T, H = x.shape
    E = gate.shape[0]
    dev = x.device
    ka, Ea = k + n_shared, E + n_shared
    ids = torch.empty((T, ka), dtype=torch.int32, device=dev)
    w = torch.empty((T, ka), dtype=torch.float32, device=dev)
    sorted_ids = torch.empty(align_max_padded(T, ka, Ea, block_m), dtype=torch.int32, device=dev)
    block_expert = torch.empty(align_max_blocks(T, ka, Ea, block_m), dtype=torch.int32, device=dev)
    npp = torch.empty(1, dtype=torch.int32, device=dev)
    need = lib().moe_route_align_workspace_size(T, H, E, k, n_shared)
    ws = workspace(dev, need) if ws is None else ws
    check(lib().moe_route_align(_ptr(x), _ptr(gate), _gate_is_fp32(gate), _ptr(bias), T, H, E, k, n_shared,
                                n_group, topk_group, SCORING[scoring], int(bool(renormalize)), float(routed_scale),
                                block_m, _ptr(ids), _ptr(w), _ptr(sorted_ids), _ptr(block_expert), _ptr(npp),
                                _ptr(ws), ws.numel(), _stream(dev)), "moe_route_align")
    return ids, w, sorted_ids, block_expert, npp


def align(topk_ids, E, block_m, ws=None):
    """moe_align -> (sorted_ids, block_expert, num_post_padded [1]) on the device."""
    _check_cuda(topk_ids)
    T, k = topk_ids.shape
    dev = topk_ids.device
    sorted_ids = torch.empty(align_max_padded(T, k, E, block_m), dtype=torch.int32, device=dev)
    block_expert = torch.empty(align_max_blocks(T, k, E, block_m), dtype=torch.int32, device=dev)
    npp = torch.empty(1, dtype=torch.int32, device=dev)
    need = lib().moe_align_workspace_size(T, k, E)
    ws = workspace(dev, need) if ws is None else ws
    check(lib().moe_align(_ptr(topk_ids), T, k, E, block_m, _ptr(sorted_ids), _ptr(block_expert), _ptr(npp),
                          _ptr(ws), ws.numel(), _stream(dev)), "moe_align")
    return sorted_ids, block_expert, npp


def _dims(x, w13, w2, wformat):
    T, H = x.shape
    E = w13.shape[0]
    F = w13.shape[1] // 2
    return T, H, E, F


def expert_ffn(x, w13, w2, topk_ids, topk_weights, sorted_ids, block_expert, num_post_padded, block_m,
               wformat="bf16", w13_scale=None, w2_scale=None, ws=None, stages=None, out=None,
               swiglu_limit=math.inf):
    """moe_expert_ffn -> y bf16 [T, H].  ``stages`` (names from
    _lib.STAGE, or an int mask) selects moe_expert_ffn_stages instead."""
    _check_cuda(x, w13, w2, topk_ids, topk_weights, sorted_ids, block_expert, num_post_padded,
                w13_scale, w2_scale)
    T, H, E, F = _dims(x, w13, w2, wformat)
    k = topk_ids.shape[1]
    y = torch.empty((T, H), dtype=torch.bfloat16, device=x.device) if out is None else out
    wf = WFORMAT[wformat]
    need = lib().moe_expert_ffn_workspace_size(T, H, E, F, k, block_m, wf)
    ws = workspace(x.device, need) if ws is None else ws
    args = [_ptr(x), wf, _ptr(w13), _ptr(w13_scale), _ptr(w2), _ptr(w2_scale),
            _ptr(topk_ids), _ptr(topk_weights), _ptr(sorted_ids), _ptr(block_expert),
            _ptr(num_post_padded), T, H, E, F, k, block_m, float(swiglu_limit), _ptr(y), _ptr(ws), ws.numel()]
    if stages is None:
        check(lib().moe_expert_ffn(*args, _stream(x.device)), "moe_expert_ffn")
    else:
        mask = stages if isinstance(stages, int) else sum(STAGE[s] for s in stages)
        check(lib().moe_expert_ffn_stages(*args, mask, _stream(x.device)), "moe_expert_ffn_stages")
    return y


def layer_workspace_size(T, H, E, F, k, block_m=0, wformat="bf16", n_shared=0):
    return int(lib().moe_layer_workspace_size(T, H, E, F, k, n_shared, block_m, WFORMAT[wformat]))


def layer(x, gate, bias, w13, w2, k, scoring="softmax", n_group=1, topk_group=1, renormalize=True,
          routed_scale=1.0, wformat="bf16", w13_scale=None, w2_scale=None, block_m=0, return_routing=False,
          ws=None, out=None, swiglu_limit=math.inf, n_shared=0):
    """moe_layer -> y bf16 [T, H] (and topk ids / weights with return_routing).
    With n_shared = 1, w13 / w2 (and scales) hold the gate's E experts plus
    the shared expert last."""
    _check_cuda(x, gate, bias, w13, w2, w13_scale, w2_scale)
    T, H, Ew, F = _dims(x, w13, w2, wformat)
    E = gate.shape[0]
    if Ew != E + n_shared:
        raise ValueError(f"w13 holds {Ew} experts, the gate {E} and n_shared = {n_shared}")
    y = torch.empty((T, H), dtype=torch.bfloat16, device=x.device) if out is None else out
    ids = w = None
    if return_routing:
        ids = torch.empty((T, k + n_shared), dtype=torch.int32, device=x.device)
        w = torch.empty((T, k + n_shared), dtype=torch.float32, device=x.device)
    wf = WFORMAT[wformat]
    need = lib().moe_layer_workspace_size(T, H, E, F, k, n_shared, block_m, wf)
    ws = workspace(x.device, need) if ws is None else ws
    check(lib().moe_layer(_ptr(x), _ptr(gate), _gate_is_fp32(gate), _ptr(bias), wf, _ptr(w13), _ptr(w13_scale),
                          _ptr(w2), _ptr(w2_scale), T, H, E, F, k, n_shared, n_group, topk_group, SCORING[scoring],
                          int(bool(renormalize)), float(routed_scale), block_m, float(swiglu_limit), _ptr(y),
                          _ptr(ids), _ptr(w),
                          _ptr(ws), ws.numel(), _stream(x.device)), "moe_layer")
    return (y, ids, w) if return_routing else y


def layer_noalloc(x, gate, bias, w13, w2, k, scoring="softmax", n_group=1, topk_group=1, renormalize=True,
                  routed_scale=1.0, wformat="bf16", w13_scale=None, w2_scale=None, block_m=0,
                  return_routing=False, out=None, swiglu_limit=math.inf, n_shared=0):
    """moe_layer_noalloc: moe_layer on the library's own scratch array (no
    workspace; the outputs are still the caller's tensors, allocated here
    unless ``out`` is given)."""
    _check_cuda(x, gate, bias, w13, w2, w13_scale, w2_scale, out)
    T, H, Ew, F = _dims(x, w13, w2, wformat)
    E = gate.shape[0]
    if Ew != E + n_shared:
        raise ValueError(f"w13 holds {Ew} experts, the gate {E} and n_shared = {n_shared}")
    y = torch.empty((T, H), dtype=torch.bfloat16, device=x.device) if out is None else out
    ids = w = None
    if return_routing:
        ids = torch.empty((T, k + n_shared), dtype=torch.int32, device=x.device)
        w = torch.empty((T, k + n_shared), dtype=torch.float32, device=x.device)
    check(lib().moe_layer_noalloc(_ptr(x), _ptr(gate), _gate_is_fp32(gate), _ptr(bias), WFORMAT[wformat],
                                  _ptr(w13), _ptr(w13_scale), _ptr(w2), _ptr(w2_scale), T, H, E, F, k, n_shared,
                                  n_group, topk_group, SCORING[scoring], int(bool(renormalize)),
                                  float(routed_scale), block_m, float(swiglu_limit), _ptr(y), _ptr(ids), _ptr(w),
                                  _stream(x.device)),
          "moe_layer_noalloc")
    return (y, ids, w) if return_routing else y


# ---------------------------------------------------------------------------
# the norm in front of the layer, and the router's training side

# A decode-sized call is mostly host time, so what every call asks of torch
# goes the short way: these queries of torch._C take 0.1 us each, building a
# torch.cuda.Stream for its handle 1.9 us.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_TYPE_IS_FP32 = {torch.float32: 1, torch.bfloat16: 0}


def _tensor(name, t, dtype, shape, index):
    """Checks one argument: its type, shape, device (by its index) and
    layout."""
    if t.dtype == dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return
    if not t.is_cuda or t.get_device() != index:
        raise ValueError(f"{name}: libmoe ops take GPU tensors of one device, not {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has type {t.dtype}, not {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    raise ValueError(f"{name}: libmoe ops take contiguous tensors")


def _gpu(name, t, dims):
    """The device index of a call's first argument, a GPU tensor of ``dims``
    dimensions."""
    if not t.is_cuda:
        raise ValueError(f"{name}: libmoe ops take GPU tensors, not {t.device}")
    if t.dim() != dims:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {dims} dimensions")
    return t.get_device()


def _is_fp32(name, t):
    """1 for a float32 tensor, 0 for a bfloat16 one."""
    f = _TYPE_IS_FP32.get(t.dtype)
    if f is None:
        raise ValueError(f"{name} is float32 or bfloat16, not {t.dtype}")
    return f


def _call(name, index, *args):
    """One library call on the current stream of a device, with that device
    current while the kernels are launched."""
    fn = getattr(lib(), name)
    if _current_device() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status:
        raise MoeError(status, name)


def rms_norm(x, weight, residual=None, eps=1e-6, quant=None, y=None, h=None, q=None, s=None, with_y=True):
    """moe_rms_norm -> (y, h), or (y, h, q, s) with ``quant``.

    y bf16 [T, H]: the norm of x + residual (None with quant and
    ``with_y=False``); h: x + residual in the residual's type (None without
    a residual: it is x).  ``quant`` "fp8" or "mxfp4": also the activations
    of those expert formats, q uint8 [T, H] (e4m3 codes) and s float32
    [T, H/128] or uint8 [T, H/32] (e8m0).  Outputs are allocated unless
    given; h may be the residual (in place)."""
    dev = _gpu("x", x, 2)
    shape = x.shape
    T, H = shape
    _tensor("x", x, torch.bfloat16, shape, dev)
    wf = _is_fp32("weight", weight)
    _tensor("weight", weight, weight.dtype, (H,), dev)
    if quant not in (None, "fp8", "mxfp4"):
        raise ValueError(f"quant is None, 'fp8' or 'mxfp4', not {quant!r}")
    rf = 0
    if residual is not None:
        rf = _is_fp32("residual", residual)
        _tensor("residual", residual, residual.dtype, shape, dev)
        if h is None:
            h = torch.empty_like(residual)
        else:
            _tensor("h", h, residual.dtype, shape, dev)
    elif h is not None:
        raise ValueError("h without a residual is x")
    if y is not None:
        _tensor("y", y, torch.bfloat16, shape, dev)
    elif with_y or quant is None:
        y = torch.empty_like(x)
    if quant is None:
        if q is not None or s is not None:
            raise ValueError("q and s are outputs of a quantised norm")
        qf = 0
    else:
        qf = WFORMAT[quant]
        group, st = (128, torch.float32) if quant == "fp8" else (32, torch.uint8)
        if H % group:
            raise ValueError(f"H = {H} is not a multiple of the {quant} group of {group}")
        if q is None:
            q = torch.empty((T, H), dtype=torch.uint8, device=dev)
        else:
            _tensor("q", q, torch.uint8, shape, dev)
        if s is None:
            s = torch.empty((T, H // group), dtype=st, device=dev)
        else:
            _tensor("s", s, st, (T, H // group), dev)
    _call("moe_rms_norm", dev, x.data_ptr(), _ptr(residual), rf, weight.data_ptr(), wf, T, H, eps, qf,
          _ptr(h), _ptr(y), _ptr(q), _ptr(s))
    return (y, h) if quant is None else (y, h, q, s)


def rms_norm_grad(dy, h, weight, eps=1e-6, dh=None, dx=None, with_weight=True):
    """moe_rms_norm_grad -> (dx, d_weight): the gradients of x (and of the
    residual) in h's type and of the weight in float32 (None without
    ``with_weight``).  ``h``: the forward call's h, or its x where it had no
    residual; ``dh``: the gradient that reaches h from elsewhere."""
    dev = _gpu("dy", dy, 2)
    T, H = dy.shape
    _tensor("dy", dy, torch.bfloat16, (T, H), dev)
    hf, wf = _is_fp32("h", h), _is_fp32("weight", weight)
    _tensor("h", h, h.dtype, (T, H), dev)
    _tensor("weight", weight, weight.dtype, (H,), dev)
    if dh is not None:
        _tensor("dh", dh, h.dtype, (T, H), dev)
    if dx is None:
        dx = torch.empty_like(h)
    else:
        _tensor("dx", dx, h.dtype, (T, H), dev)
    dw = ws = None
    need = 0
    if with_weight:
        dw = torch.empty(H, dtype=torch.float32, device=dev)
        need = lib().moe_rms_norm_grad_workspace_size(T, H)
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    _call("moe_rms_norm_grad", dev, dy.data_ptr(), _ptr(dh), h.data_ptr(), hf, weight.data_ptr(), wf, T, H, eps,
          dx.data_ptr(), _ptr(dw), _ptr(ws), need)
    return dx, dw


def _router_args(logits, topk_ids, n_shared, seq_offsets, token_mask):
    """Checks what balance_loss and route_grad share; (T, E, k, sequences,
    device index)."""
    dev = _gpu("logits", logits, 2)
    _gpu("topk_ids", topk_ids, 2)
    T, E = logits.shape
    _tensor("logits", logits, torch.float32, (T, E), dev)
    _tensor("topk_ids", topk_ids, torch.int32, (T, topk_ids.shape[1]), dev)
    n_seq = 1
    if seq_offsets is not None:
        if seq_offsets.dim() != 1 or seq_offsets.shape[0] < 2:
            raise ValueError("seq_offsets holds the sequences' starts and the last one's end")
        n_seq = seq_offsets.shape[0] - 1
        _tensor("seq_offsets", seq_offsets, torch.int32, (n_seq + 1,), dev)
    if token_mask is not None:
        _tensor("token_mask", token_mask, torch.bool if token_mask.dtype == torch.bool else torch.uint8, (T,), dev)
    return T, E, topk_ids.shape[1] - n_shared, n_seq, dev


def balance_loss(logits, topk_ids, scoring="softmax", seq_offsets=None, token_mask=None, n_shared=0):
    """moe_balance_loss -> (losses float32 [2]: balance and z loss, counts
    int32 [S, E], probs float32 [S, E], tokens int32 [S + 2]).

    ``seq_offsets`` int32 [S + 1] on the GPU cuts the rows into sequences
    (default: all rows are one); ``token_mask`` uint8 or bool [T] leaves out
    the rows where it is 0.  counts and tokens go to route_grad."""
    T, E, k, S, dev = _router_args(logits, topk_ids, n_shared, seq_offsets, token_mask)
    losses = torch.empty(2, dtype=torch.float32, device=dev)
    counts = torch.empty((S, E), dtype=torch.int32, device=dev)
    probs = torch.empty((S, E), dtype=torch.float32, device=dev)
    tokens = torch.empty(S + 2, dtype=torch.int32, device=dev)
    need = lib().moe_balance_loss_workspace_size(T, E, S)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _call("moe_balance_loss", dev, logits.data_ptr(), topk_ids.data_ptr(), _ptr(token_mask), _ptr(seq_offsets), T, E, k,
          n_shared, S, SCORING[scoring], losses.data_ptr(), counts.data_ptr(), probs.data_ptr(), tokens.data_ptr(),
          _ptr(ws), need)
    return losses, counts, probs, tokens


def route_grad(logits, topk_ids, scoring="softmax", renormalize=True, routed_scale=1.0, d_weights=None, d_losses=None,
               counts=None, tokens=None, seq_offsets=None, token_mask=None, n_shared=0, d_logits=None):
    """moe_route_grad -> d_logits float32 [T, E], from ``d_weights`` (float32
    [T, k], the gradient of the routing weights) and / or ``d_losses``
    (float32 [2] on the GPU, the gradient of balance_loss's losses, with its
    counts and tokens)."""
    T, E, k, S, dev = _router_args(logits, topk_ids, n_shared, seq_offsets, token_mask)
    if d_weights is None and d_losses is None:
        raise ValueError("route_grad takes d_weights, d_losses or both")
    if d_weights is not None:
        _tensor("d_weights", d_weights, torch.float32, (T, k + n_shared), dev)
    if d_losses is not None:
        if counts is None or tokens is None:
            raise ValueError("d_losses goes with balance_loss's counts and tokens")
        _tensor("d_losses", d_losses, torch.float32, (2,), dev)
        _tensor("counts", counts, torch.int32, (S, E), dev)
        _tensor("tokens", tokens, torch.int32, (S + 2,), dev)
    if d_logits is None:
        d_logits = torch.empty_like(logits)
    else:
        _tensor("d_logits", d_logits, torch.float32, (T, E), dev)
    _call("moe_route_grad", dev, logits.data_ptr(), topk_ids.data_ptr(), _ptr(token_mask), _ptr(seq_offsets), T, E, k,
          n_shared, S, SCORING[scoring], int(bool(renormalize)), routed_scale, _ptr(d_weights), _ptr(d_losses),
          _ptr(counts), _ptr(tokens), d_logits.data_ptr())
    return d_logits


def gate_grad(x, gate, d_logits, dx_in=None, dx=None, with_dx=True, with_gate=True):
    """moe_gate_grad -> (dx bf16 [T, H], d_gate float32 [E, H]): dx =
    d_logits gate (+ dx_in), d_gate = d_logits^T x; None for the one that
    is not wanted.  dx may be dx_in (in place)."""
    dev = _gpu("x", x, 2)
    _gpu("gate", gate, 2)
    T, H = x.shape
    E = gate.shape[0]
    _tensor("x", x, torch.bfloat16, (T, H), dev)
    gf = _is_fp32("gate", gate)
    _tensor("gate", gate, gate.dtype, (E, H), dev)
    _tensor("d_logits", d_logits, torch.float32, (T, E), dev)
    if not with_dx and (dx is not None or dx_in is not None):
        raise ValueError("dx and dx_in without with_dx")
    if dx_in is not None:
        _tensor("dx_in", dx_in, torch.bfloat16, (T, H), dev)
    if dx is not None:
        _tensor("dx", dx, torch.bfloat16, (T, H), dev)
    elif with_dx:
        dx = torch.empty_like(x)
    d_gate = torch.empty((E, H), dtype=torch.float32, device=dev) if with_gate else None
    need = lib().moe_gate_grad_workspace_size(T, H, E)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    _call("moe_gate_grad", dev, x.data_ptr(), gate.data_ptr(), gf, d_logits.data_ptr(), _ptr(dx_in), T, H, E,
          _ptr(dx), _ptr(d_gate), ws.data_ptr(), need)
    return dx, d_gate


def norm_layer_workspace_size(T, H, E, F, k, block_m=0, wformat="bf16", n_shared=0):
    return int(lib().moe_norm_layer_workspace_size(T, H, E, F, k, n_shared, block_m, WFORMAT[wformat]))


def norm_layer(x, norm_weight, gate, bias, w13, w2, k, residual=None, eps=1e-6, scoring="softmax", n_group=1,
               topk_group=1, renormalize=True, routed_scale=1.0, wformat="bf16", w13_scale=None, w2_scale=None,
               block_m=0, return_routing=False, ws=None, out=None, h=None, swiglu_limit=math.inf, n_shared=0):
    """moe_norm_layer -> (y bf16 [T, H], h) (and topk ids / weights with
    return_routing): the layer on the norm of x + residual; h is that sum in
    the residual's type (None without one).  Other arguments as layer."""
    _check_cuda(x, gate, bias, w13, w2, w13_scale, w2_scale, out, ws)
    T, H, Ew, F = _dims(x, w13, w2, wformat)
    E = gate.shape[0]
    dev = _gpu("x", x, 2)
    if Ew != E + n_shared:
        raise ValueError(f"w13 holds {Ew} experts, the gate {E} and n_shared = {n_shared}")
    _tensor("x", x, torch.bfloat16, (T, H), dev)
    nf = _is_fp32("norm_weight", norm_weight)
    _tensor("norm_weight", norm_weight, norm_weight.dtype, (H,), dev)
    rf = 0
    if residual is not None:
        rf = _is_fp32("residual", residual)
        _tensor("residual", residual, residual.dtype, (T, H), dev)
        if h is None:
            h = torch.empty_like(residual)
        else:
            _tensor("h", h, residual.dtype, (T, H), dev)
    elif h is not None:
        raise ValueError("h without a residual is x")
    if out is not None:
        _tensor("out", out, torch.bfloat16, (T, H), dev)
    y = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if out is None else out
    ids = w = None
    if return_routing:
        ids = torch.empty((T, k + n_shared), dtype=torch.int32, device=dev)
        w = torch.empty((T, k + n_shared), dtype=torch.float32, device=dev)
    wf = WFORMAT[wformat]
    need = lib().moe_norm_layer_workspace_size(T, H, E, F, k, n_shared, block_m, wf)
    ws = workspace(dev, need) if ws is None else ws
    _call("moe_norm_layer", dev, x.data_ptr(), _ptr(residual), rf, norm_weight.data_ptr(), nf, eps,
          _ptr(gate), _gate_is_fp32(gate), _ptr(bias), wf, _ptr(w13),
          _ptr(w13_scale), _ptr(w2), _ptr(w2_scale), T, H, E, F, k, n_shared, n_group, topk_group, SCORING[scoring],
          int(bool(renormalize)), float(routed_scale), block_m, float(swiglu_limit), _ptr(h), _ptr(y), _ptr(ids),
          _ptr(w), _ptr(ws), ws.numel())
    return (y, h, ids, w) if return_routing else (y, h)


def debug_error(ws):
    """Synchronises and returns (and clears) the sticky alignment error bits."""
    return int(lib().moe_debug_error(_ptr(ws), _stream(ws.device)))


def probe_empty(device="cuda"):
    check(lib().moe_probe_empty(_stream(torch.device(device))), "moe_probe_empty")


def probe_mfma(kind, accs, grid, iters, sink=None, device="cuda"):
    """Enqueues the matrix-core issue-rate probe (kind: 0 bf16 16x16x32,
    1 bf16 32x32x16, 2 e4m3 x e4m3, 3 e4m3 x e2m1, 4 e2m1 x e2m1)."""
    dev = torch.device(device)
    if sink is None:
        sink = torch.empty(int(lib().moe_probe_mfma_sink_len(grid)), dtype=torch.float32, device=dev)
    check(lib().moe_probe_mfma(kind, accs, grid, iters, _ptr(sink), _stream(dev)), "moe_probe_mfma")
    return sink


def probe_read(t, sink=None):
    """Reads every byte of ``t`` once (the bare weight-read kernel)."""
    nbytes = t.numel() * t.element_size()
    if sink is None:
        sink = torch.empty(int(lib().moe_probe_read_sink_len(nbytes)), dtype=torch.float32, device=t.device)
    check(lib().moe_probe_read(_ptr(t), nbytes, _ptr(sink), _stream(t.device)), "moe_probe_read")
    return sink
