"""Bindings of include/kda_linear.h and include/kda_norm.h: linear attention with one decay
per head, and the norms round an attention block. Argument checks and marshalling only;
everything runs in libkda.so, on the tensors' device and its current stream. Nothing is
recorded for autograd: a tensor that requires grad is refused while gradients are recorded,
and taken under torch.no_grad() and inside an autograd.Function.
"""
import ctypes
import functools

import torch

from ._binding import KDA_BF16, KDA_F32, _require, check, lib

DECAY_TOKEN, DECAY_HEAD = 0, 1
NORMS = {"rms": 0, "l2": 1}
GATE_ACTS = {"sigmoid": 0, "silu": 1}

_c_int, _vp = ctypes.c_int, ctypes.c_void_p


class LinearArgs(ctypes.Structure):
    _fields_ = [("B", _c_int), ("T", _c_int), ("H", _c_int), ("K", _c_int), ("V", _c_int), ("N", _c_int),
                ("Hk", _c_int), ("dtype", _c_int), ("decay", _c_int), ("scale", ctypes.c_float)]


class NormArgs(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("D", _c_int), ("dtype", _c_int), ("res_dtype", _c_int), ("norm", _c_int),
                ("gate_act", _c_int), ("scale", ctypes.c_float), ("eps", ctypes.c_float)]


_READY = None


def _lib():
    """The library with the signatures of these entry points."""
    global _READY
    if _READY is None:
        L = lib()
        la, na, size = ctypes.POINTER(LinearArgs), ctypes.POINTER(NormArgs), ctypes.c_size_t
        L.kda_linear_chunk_workspace_bytes.argtypes = [la]
        L.kda_linear_chunk_workspace_bytes.restype = size
        L.kda_linear_chunk_fwd.argtypes = [la] + [_vp] * 9 + [size, _vp]
        L.kda_linear_chunk_bwd_workspace_bytes.argtypes = [la]
        L.kda_linear_chunk_bwd_workspace_bytes.restype = size
        L.kda_linear_chunk_bwd.argtypes = [la] + [_vp] * 14 + [size, _vp]
        L.kda_linear_recurrent_fwd.argtypes = [la] + [_vp] * 9
        L.kda_block_norm_fwd.argtypes = [na] + [_vp] * 9
        L.kda_block_norm_bwd_workspace_bytes.argtypes = [na]
        L.kda_block_norm_bwd_workspace_bytes.restype = size
        L.kda_block_norm_bwd.argtypes = [na] + [_vp] * 15 + [size, _vp]
        for f in (L.kda_linear_chunk_fwd, L.kda_linear_chunk_bwd, L.kda_linear_recurrent_fwd, L.kda_block_norm_fwd,
                  L.kda_block_norm_bwd):
            f.restype = _c_int
        _READY = L
    return _READY


def _refuse(name, t, shape, dtype, device):
    if t.shape != shape or t.dtype != dtype:
        raise ValueError("%s must be %s %s, got %s %s" % (name, dtype, list(shape), t.dtype, list(t.shape)))
    if device < 0 or t.get_device() != device:
        raise ValueError("%s must be on %s" % (name, "a GPU" if device < 0 else "cuda:%d" % device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    raise RuntimeError("%s requires grad: this op records no gradients; call it under torch.no_grad() or inside an "
                       "autograd.Function, and its _bwd for them" % name)


def _tensor(name, t, shape, dtype, device):
    """A tensor's pointer, after its checks; None for None. device: the GPU's index, -1 for none."""
    if t is None:
        return None
    if (t.shape != shape or t.dtype is not dtype or device < 0 or t.get_device() != device
            or (t.requires_grad and torch.is_grad_enabled()) or not t.is_contiguous()):
        _refuse(name, t, shape, dtype, device)
    return t.data_ptr()


# PyTorch's own cheap forms of the public calls, which a build without a GPU does not have
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)


def _on_device(f):
    """Runs f with its first tensor's device current: workspace sizes and launches go by it."""
    first = f.__code__.co_varnames[0]

    @functools.wraps(f)
    def g(*args, **kw):
        x = args[0] if args else kw.get(first)
        i = x.get_device() if isinstance(x, torch.Tensor) else -1
        if i < 0 or i == _current_device():
            return f(*args, **kw)
        with torch.cuda.device(i):
            return f(*args, **kw)

    return g


def _launch(device, entry, *args):
    """One entry point on the device's current stream (its handle read without building a
    Stream object, which costs as much as the launch of a single-token step)."""
    status = entry(*args, _current_stream(device))
    if status:
        check(status)


def _attn_args(q, k, v, g, h0, cu_seqlens, scale):
    """The argument block, the slots, and the inputs' pointers."""
    _require(q.dim() == 4 and v.dim() == 4 and g.dim() in (1, 3), "q, k must be [B, T, Hk, K], v [B, T, H, V], "
             "g [B, T, H] or [H]")
    B, T, Hk, K = q.shape
    H, V = v.shape[2], v.shape[3]
    _require(v.shape[:2] == q.shape[:2] and Hk > 0 and H % Hk == 0,
             "v must be [B, T, H, V] with H a multiple of q's heads Hk")
    _require(q.dtype in (torch.bfloat16, torch.float32), "q, k, v must share dtype bf16 or fp32")
    # the library takes 0 for "not given", so what would round to it is refused too
    c_scale = 0.0 if scale is None else ctypes.c_float(scale).value
    _require(scale is None or 0.0 < c_scale < float("inf"), "scale must be a positive fp32 number")
    dev, N = q.get_device(), B
    if cu_seqlens is not None:
        _require(B == 1, "packed inputs (cu_seqlens) need batch 1")
        _require(cu_seqlens.dim() == 1 and cu_seqlens.numel() > 0, "cu_seqlens must be int32 [N+1]")
        N = cu_seqlens.numel() - 1
    head = g.dim() == 1
    ptrs = (_tensor("q", q, q.shape, q.dtype, dev), _tensor("k", k, q.shape, q.dtype, dev),
            _tensor("v", v, v.shape, q.dtype, dev), _tensor("g", g, (H,) if head else (B, T, H), torch.float32, dev),
            _tensor("initial_state", h0, (N, H, K, V), torch.float32, dev),
            _tensor("cu_seqlens", cu_seqlens, (N + 1,), torch.int32, dev))
    a = LinearArgs(B, T, H, K, V, N, 0 if Hk == H else Hk, KDA_BF16 if q.dtype == torch.bfloat16 else KDA_F32,
                   DECAY_HEAD if head else DECAY_TOKEN, c_scale)
    return a, N, dev, ptrs


def _workspace(workspace, need, device):
    """(pointer, bytes, tensor to keep) of a workspace of `need` bytes, the caller's or a new one."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = torch.empty((need,), dtype=torch.uint8, device="cuda:%d" % device)
    _require(workspace.dtype == torch.uint8 and workspace.dim() == 1 and workspace.numel() >= need,
             "workspace must be a 1-D uint8 tensor of at least %d bytes" % need)
    return _tensor("workspace", workspace, workspace.shape, torch.uint8, device), workspace.numel(), workspace


def _outputs(q, v, N, dev, out, final_state, want_state):
    o = torch.empty_like(v) if out is None else out
    B, T, H, V = v.shape
    shape = (N, H, q.shape[3], V)
    ht = torch.empty(shape, dtype=torch.float32, device=q.device) if final_state is None and want_state else final_state
    return o, ht, _tensor("out", o, v.shape, q.dtype, dev), _tensor("final_state", ht, shape, torch.float32, dev)


@_on_device
def chunk_linear_attn(q, k, v, g, initial_state=None, *, cu_seqlens=None, output_final_state=False, scale=None,
                      final_state=None, out=None, workspace=None):
    """Chunked linear attention with one decay per head. Returns (o, ht); ht is None unless requested.

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t,  scale 1/sqrt(K) unless given (> 0).
    q, k are [B, T, Hk, K], v [B, T, H, V] (bf16 or fp32, H a multiple of Hk); g is the fp32
    natural-log decay, g <= 0: [B, T, H], or [H] for one fixed decay per head. -inf resets the
    state. ``initial_state`` is fp32 [N, H, K, V]; ``final_state`` may preallocate the final
    state, including ``initial_state`` itself for an update in place. Packed batches pass
    ``cu_seqlens`` (int32 [N+1]); rows outside it are left as they are in ``out``.
    ``out`` must not overlap an input. ``workspace`` may pass a uint8 tensor of
    ``linear_workspace_bytes``, reused from call to call (calls or captured graphs that share one
    must not run at once); otherwise each call allocates what it needs.
    """
    a, N, dev, (pq, pk, pv, pg, ph, pc) = _attn_args(q, k, v, g, initial_state, cu_seqlens, scale)
    o, ht, po, pt = _outputs(q, v, N, dev, out, final_state, output_final_state)
    L = _lib()
    pw, nw, _keep = _workspace(workspace, int(L.kda_linear_chunk_workspace_bytes(ctypes.byref(a))), dev)
    _launch(dev, L.kda_linear_chunk_fwd, ctypes.byref(a), pq, pk, pv, pg, ph, pc, po, pt, pw, nw)
    return o, ht


@_on_device
def recurrent_linear_attn(q, k, v, g, initial_state=None, *, cu_seqlens=None, output_final_state=False, scale=None,
                          final_state=None, out=None):
    """``chunk_linear_attn`` token by token, for decoding: one kernel that holds the state in
    registers. ``final_state=initial_state`` updates the state in place. Returns (o, ht)."""
    a, N, dev, (pq, pk, pv, pg, ph, pc) = _attn_args(q, k, v, g, initial_state, cu_seqlens, scale)
    o, ht, po, pt = _outputs(q, v, N, dev, out, final_state, output_final_state)
    _launch(dev, _lib().kda_linear_recurrent_fwd, ctypes.byref(a), pq, pk, pv, pg, ph, pc, po, pt)
    return o, ht


@_on_device
def chunk_linear_attn_bwd(q, k, v, g, do, initial_state=None, *, dht=None, cu_seqlens=None, scale=None,
                          workspace=None):
    """Gradients of sum(do * o) + sum(dht * ht) for ``chunk_linear_attn``.

    Returns a dict: dq, dk (q's dtype, summed over the value heads that share a q/k head), dv, dg
    (fp32, shaped as g) and dh0 (fp32 [N, H, K, V]). Nothing of the forward needs to be kept.
    Packed: gradients of rows outside cu_seqlens are not written.
    """
    a, N, dev, (pq, pk, pv, pg, ph, pc) = _attn_args(q, k, v, g, initial_state, cu_seqlens, scale)
    state = (N, v.shape[2], q.shape[3], v.shape[3])
    pdo = _tensor("do", do, v.shape, q.dtype, dev)
    pdht = _tensor("dht", dht, state, torch.float32, dev)
    L = _lib()
    pw, nw, _keep = _workspace(workspace, int(L.kda_linear_chunk_bwd_workspace_bytes(ctypes.byref(a))), dev)
    got = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v), dg=torch.empty_like(g),
               dh0=torch.empty(state, dtype=torch.float32, device=q.device))
    _launch(dev, L.kda_linear_chunk_bwd, ctypes.byref(a), pq, pk, pv, pg, ph, pc, pdo, pdht, got["dq"].data_ptr(),
            got["dk"].data_ptr(), got["dv"].data_ptr(), got["dg"].data_ptr(), got["dh0"].data_ptr(), pw, nw)
    return got


@_on_device
def linear_workspace_bytes(q, k, v, g, *, slots=None, backward=False):
    """Workspace bytes of ``chunk_linear_attn`` (or of its backward) for tensors like these;
    ``slots`` is the number of packed sequences (default: the batch, unpacked)."""
    B, T, Hk, K = q.shape
    H, V = v.shape[2], v.shape[3]
    a = LinearArgs(B, T, H, K, V, B if slots is None else int(slots), 0 if Hk == H else Hk,
                   KDA_BF16 if q.dtype == torch.bfloat16 else KDA_F32, DECAY_HEAD if g.dim() == 1 else DECAY_TOKEN, 0.0)
    L = _lib()
    f = L.kda_linear_chunk_bwd_workspace_bytes if backward else L.kda_linear_chunk_workspace_bytes
    return int(f(ctypes.byref(a)))


def _norm_args(x, weight, gate, gate_act, residual, scale, next_weight, eps, norm):
    """The argument block and the inputs' pointers of a block norm."""
    _require(x.dim() >= 1 and x.shape[-1] > 0, "x must have rows of at least one value")
    _require(x.dtype in (torch.bfloat16, torch.float32), "x must be bf16 or fp32")
    _require(norm in NORMS, "norm must be one of %s" % sorted(NORMS))
    _require(gate_act in GATE_ACTS, "gate_act must be one of %s" % sorted(GATE_ACTS))
    D, dev = x.shape[-1], x.get_device()
    bf16 = x.dtype == torch.bfloat16
    res = x.dtype
    if residual is not None:
        res = residual.dtype
        _require(res in (x.dtype, torch.float32), "residual must be fp32 or of x's dtype")
    vec = isinstance(scale, torch.Tensor)
    ptrs = (_tensor("x", x, x.shape, x.dtype, dev), _tensor("weight", weight, (D,), torch.float32, dev),
            _tensor("gate", gate, x.shape, x.dtype, dev), _tensor("residual", residual, x.shape, res, dev),
            _tensor("scale", scale, (D,), torch.float32, dev) if vec else None,
            _tensor("next_weight", next_weight, (D,), torch.float32, dev))
    a = NormArgs(x.numel() // D, D, KDA_BF16 if bf16 else KDA_F32,
                 KDA_BF16 if res == torch.bfloat16 else KDA_F32, NORMS[norm], GATE_ACTS[gate_act],
                 1.0 if scale is None or vec else float(scale), float(eps))
    return a, ptrs, res, vec


@_on_device
def block_norm(x, weight=None, *, gate=None, gate_act="sigmoid", residual=None, scale=None, next_weight=None,
               next_norm=None, eps=1e-6, norm="rms", out=None, next_out=None):
    """The norm after a block with its gate, residual branch and the norm before the next block.

        n = weight x / sqrt(mean(x^2) + eps);  y = residual + scale n act(gate)
        z = next_weight y / sqrt(mean(y^2) + eps)

    over the last axis of x. Returns y, or (y, z) with ``next_weight`` or ``next_norm=True``. Every
    part but the first norm is optional; ``norm="l2"`` takes the sum in place of the mean (what
    ``chunk_kda`` expects of its q and k rows). x and gate are bf16 or fp32; weights are fp32 [D];
    ``scale`` is a number or fp32 [D]; ``residual`` (and y) may be fp32 beside bf16 x. ``out`` may
    be ``residual`` itself. z comes from y before y is rounded.
    """
    nxt = next_weight is not None if next_norm is None else bool(next_norm)
    _require(nxt or next_weight is None, "next_weight needs the next norm")
    _require(nxt or next_out is None, "next_out needs the next norm")
    a, (px, pw, pg, pr, ps, pn), res, _ = _norm_args(x, weight, gate, gate_act, residual, scale, next_weight, eps, norm)
    y = torch.empty_like(x, dtype=res) if out is None else out
    dev = x.get_device()
    py = _tensor("out", y, x.shape, res, dev)
    z = pz = None
    if nxt:
        z = torch.empty_like(x) if next_out is None else next_out
        pz = _tensor("next_out", z, x.shape, x.dtype, dev)
    _launch(dev, _lib().kda_block_norm_fwd, ctypes.byref(a), px, pw, pg, pr, ps, pn, py, pz)
    return (y, z) if nxt else y


@_on_device
def block_norm_bwd(x, dy, weight=None, *, dz=None, gate=None, gate_act="sigmoid", residual=None, scale=None,
                   next_weight=None, eps=1e-6, norm="rms", workspace=None):
    """Gradients of sum(dy * y) + sum(dz * z) for ``block_norm``; dy may be None beside dz.

    Returns a dict: dx, and for what was passed dweight, dgate, dresidual, dscale (of a tensor
    scale) and dnext_weight; None for the rest. Weights' gradients are fp32.
    """
    _require(dy is not None or dz is not None, "dy or dz must be given")
    _require(next_weight is None or dz is not None, "next_weight needs dz")
    a, (px, pw, pg, pr, ps, pn), res, vec = _norm_args(x, weight, gate, gate_act, residual, scale, next_weight, eps,
                                                      norm)
    dev = x.get_device()
    pdy, pdz = _tensor("dy", dy, x.shape, res, dev), _tensor("dz", dz, x.shape, x.dtype, dev)
    L = _lib()
    params = weight is not None or vec or next_weight is not None
    pws, nws, _keep = _workspace(workspace, int(L.kda_block_norm_bwd_workspace_bytes(ctypes.byref(a))) if params else 0,
                                 dev)
    like = lambda t: None if t is None else torch.empty_like(t)  # noqa: E731
    got = dict(dx=torch.empty_like(x), dweight=like(weight), dgate=like(gate), dresidual=like(residual),
               dscale=like(scale) if vec else None, dnext_weight=like(next_weight))
    ptr = {n: None if t is None else t.data_ptr() for n, t in got.items()}
    _launch(dev, L.kda_block_norm_bwd, ctypes.byref(a), px, pw, pg, pr, ps, pn, pdy, pdz, ptr["dx"], ptr["dgate"],
            ptr["dresidual"], ptr["dweight"], ptr["dscale"], ptr["dnext_weight"], pws, nws)
    return got
