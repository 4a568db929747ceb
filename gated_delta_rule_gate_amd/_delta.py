"""Bindings of include/kda_delta.h and include/kda_rope.h: the gated delta rule with one decay
per head, and the norm of query and key rows with their rotation by position. Argument checks and
marshalling only; everything runs in libkda.so, on the tensors' device and its current stream.
Nothing is recorded for autograd: a tensor that requires grad is refused while gradients are
recorded, and taken under torch.no_grad() and inside an autograd.Function.
"""
import ctypes

import torch

from ._binding import KDA_BF16, KDA_F32, _require, lib
from ._linear import _launch, _on_device, _outputs, _refuse, _tensor, _workspace

QK_NORMS = {"rms": 0, "l2": 1, "none": 2}
PAIRS = {"half": 0, "adjacent": 1}

_c_int, _vp, _i64 = ctypes.c_int, ctypes.c_void_p, ctypes.c_int64


class DeltaArgs(ctypes.Structure):
    _fields_ = [("B", _c_int), ("T", _c_int), ("H", _c_int), ("K", _c_int), ("V", _c_int), ("N", _c_int),
                ("Hk", _c_int), ("dtype", _c_int), ("scale", ctypes.c_float)]


class QkArgs(ctypes.Structure):
    _fields_ = [("tokens", _i64), ("H", _c_int), ("Hk", _c_int), ("D", _c_int), ("rot", _c_int), ("dtype", _c_int),
                ("norm", _c_int), ("pairs", _c_int), ("axes", _c_int), ("sections", _c_int * 4), ("spread", _c_int),
                ("eps", ctypes.c_float), ("q_stride", _i64), ("k_stride", _i64), ("qo_stride", _i64),
                ("ko_stride", _i64)]


_READY = None


def _lib():
    """The library with the signatures of these entry points."""
    global _READY
    if _READY is None:
        L = lib()
        da, qa, size = ctypes.POINTER(DeltaArgs), ctypes.POINTER(QkArgs), ctypes.c_size_t
        L.kda_delta_chunk_workspace_bytes.argtypes = [da]
        L.kda_delta_chunk_workspace_bytes.restype = size
        L.kda_delta_chunk_fwd.argtypes = [da] + [_vp] * 10 + [size, _vp]
        L.kda_delta_chunk_bwd_workspace_bytes.argtypes = [da]
        L.kda_delta_chunk_bwd_workspace_bytes.restype = size
        L.kda_delta_chunk_bwd.argtypes = [da] + [_vp] * 16 + [size, _vp]
        L.kda_delta_recurrent_fwd.argtypes = [da] + [_vp] * 10
        L.kda_qk_norm_rope_fwd.argtypes = [qa] + [_vp] * 9
        L.kda_qk_norm_rope_bwd_workspace_bytes.argtypes = [qa]
        L.kda_qk_norm_rope_bwd_workspace_bytes.restype = size
        L.kda_qk_norm_rope_bwd.argtypes = [qa] + [_vp] * 13 + [size, _vp]
        for f in (L.kda_delta_chunk_fwd, L.kda_delta_chunk_bwd, L.kda_delta_recurrent_fwd, L.kda_qk_norm_rope_fwd,
                  L.kda_qk_norm_rope_bwd):
            f.restype = _c_int
        _READY = L
    return _READY


def _delta_args(q, k, v, g, beta, h0, cu_seqlens, scale):
    """The argument block, the slots, and the inputs' pointers."""
    _require(q.dim() == 4 and v.dim() == 4, "q, k must be [B, T, Hk, K], v [B, T, H, V]")
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
    ptrs = (_tensor("q", q, q.shape, q.dtype, dev), _tensor("k", k, q.shape, q.dtype, dev),
            _tensor("v", v, v.shape, q.dtype, dev), _tensor("g", g, (B, T, H), torch.float32, dev),
            _tensor("beta", beta, (B, T, H), torch.float32, dev),
            _tensor("initial_state", h0, (N, H, K, V), torch.float32, dev),
            _tensor("cu_seqlens", cu_seqlens, (N + 1,), torch.int32, dev))
    a = DeltaArgs(B, T, H, K, V, N, 0 if Hk == H else Hk, KDA_BF16 if q.dtype == torch.bfloat16 else KDA_F32, c_scale)
    return a, N, dev, ptrs


@_on_device
def chunk_gated_delta(q, k, v, g, beta, initial_state=None, *, cu_seqlens=None, output_final_state=False, scale=None,
                      final_state=None, out=None, workspace=None):
    """Chunked gated delta rule with one decay per head. Returns (o, ht); ht is None unless requested.

    S'_t = exp(g_t) S_{t-1},  u_t = beta_t (v_t - S'_t^T k_t),  S_t = S'_t + k_t u_t^T,
    o_t = scale S_t^T q_t,  scale 1/sqrt(K) unless given (> 0).
    q, k are [B, T, Hk, K], v [B, T, H, V] (bf16 or fp32, H a multiple of Hk), k's rows
    l2-normalised (``qk_norm_rope(..., norm="l2")``); g is the fp32 natural-log decay [B, T, H],
    g <= 0, or None for the plain delta rule; -inf resets the state. beta is fp32 [B, T, H],
    post-sigmoid. ``initial_state`` is fp32 [N, H, K, V]; ``final_state`` may preallocate the final
    state, including ``initial_state`` itself for an update in place. Packed batches pass
    ``cu_seqlens`` (int32 [N+1]); rows outside it are left as they are in ``out``.
    ``out`` must not overlap an input. ``workspace`` may pass a uint8 tensor of
    ``gated_delta_workspace_bytes``, reused from call to call (calls or captured graphs that share
    one must not run at once); otherwise each call allocates what it needs.
    """
    a, N, dev, (pq, pk, pv, pg, pb, ph, pc) = _delta_args(q, k, v, g, beta, initial_state, cu_seqlens, scale)
    o, ht, po, pt = _outputs(q, v, N, dev, out, final_state, output_final_state)
    L = _lib()
    pw, nw, _keep = _workspace(workspace, int(L.kda_delta_chunk_workspace_bytes(ctypes.byref(a))), dev)
    _launch(dev, L.kda_delta_chunk_fwd, ctypes.byref(a), pq, pk, pv, pg, pb, ph, pc, po, pt, pw, nw)
    return o, ht


@_on_device
def recurrent_gated_delta(q, k, v, g, beta, initial_state=None, *, cu_seqlens=None, output_final_state=False, scale=None,
                          final_state=None, out=None):
    """``chunk_gated_delta`` token by token, for decoding: one kernel that holds the state in
    registers. ``final_state=initial_state`` updates the state in place. Returns (o, ht)."""
    a, N, dev, (pq, pk, pv, pg, pb, ph, pc) = _delta_args(q, k, v, g, beta, initial_state, cu_seqlens, scale)
    o, ht, po, pt = _outputs(q, v, N, dev, out, final_state, output_final_state)
    _launch(dev, _lib().kda_delta_recurrent_fwd, ctypes.byref(a), pq, pk, pv, pg, pb, ph, pc, po, pt)
    return o, ht


@_on_device
def chunk_gated_delta_bwd(q, k, v, g, beta, do, initial_state=None, *, dht=None, cu_seqlens=None, scale=None,
                          workspace=None):
    """Gradients of sum(do * o) + sum(dht * ht) for ``chunk_gated_delta``.

    Returns a dict: dq, dk (q's dtype, summed over the value heads that share a q/k head), dv, dg
    (fp32 [B, T, H]; None without g), dbeta (fp32 [B, T, H]) and dh0 (fp32 [N, H, K, V]). Nothing of
    the forward needs to be kept; the states of every chunk pass through the workspace. Packed:
    gradients of rows outside cu_seqlens are not written.
    """
    a, N, dev, (pq, pk, pv, pg, pb, ph, pc) = _delta_args(q, k, v, g, beta, initial_state, cu_seqlens, scale)
    state = (N, v.shape[2], q.shape[3], v.shape[3])
    pdo = _tensor("do", do, v.shape, q.dtype, dev)
    pdht = _tensor("dht", dht, state, torch.float32, dev)
    L = _lib()
    pw, nw, _keep = _workspace(workspace, int(L.kda_delta_chunk_bwd_workspace_bytes(ctypes.byref(a))), dev)
    got = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
               dg=None if g is None else torch.empty_like(g), dbeta=torch.empty_like(beta),
               dh0=torch.empty(state, dtype=torch.float32, device=q.device))
    ptr = {n: None if t is None else t.data_ptr() for n, t in got.items()}
    _launch(dev, L.kda_delta_chunk_bwd, ctypes.byref(a), pq, pk, pv, pg, pb, ph, pc, pdo, pdht, ptr["dq"], ptr["dk"],
            ptr["dv"], ptr["dg"], ptr["dbeta"], ptr["dh0"], pw, nw)
    return got


@_on_device
def gated_delta_workspace_bytes(q, k, v, *, slots=None, backward=False):
    """Workspace bytes of ``chunk_gated_delta`` (or of its backward) for tensors like these;
    ``slots`` is the number of packed sequences (default: the batch, unpacked)."""
    B, T, Hk, K = q.shape
    H, V = v.shape[2], v.shape[3]
    a = DeltaArgs(B, T, H, K, V, B if slots is None else int(slots), 0 if Hk == H else Hk,
                  KDA_BF16 if q.dtype == torch.bfloat16 else KDA_F32, 0.0)
    L = _lib()
    f = L.kda_delta_chunk_bwd_workspace_bytes if backward else L.kda_delta_chunk_workspace_bytes
    return int(f(ctypes.byref(a)))


def _heads(name, t, shape, dtype, device):
    """(pointer, elements from a token's rows to the next's) of a [B, T, heads, D] tensor whose
    tokens may lie apart: a part of a fused projection."""
    if t.is_contiguous():
        return _tensor(name, t, shape, dtype, device), 0
    if t.shape != shape or t.dtype is not dtype or device < 0 or t.get_device() != device:
        _refuse(name, t, shape, dtype, device)
    B, T, H, D = shape
    s = t.stride()
    step = s[1] if T > 1 else s[0]
    if (s[3] != 1 and D > 1) or (s[2] != D and H > 1) or (B > 1 and s[0] != T * step) or step < H * D or step % 8:
        raise ValueError("%s must have contiguous [heads, channels] rows at one stride from token to token, "
                         "a multiple of 8 elements" % name)
    if t.requires_grad and torch.is_grad_enabled():
        raise RuntimeError("%s requires grad: this op records no gradients; call it under torch.no_grad() or inside "
                           "an autograd.Function, and its _bwd for them" % name)
    return t.data_ptr(), step


def _qk_args(q, k, q_weight, k_weight, positions, inv_freq, sections, spread, pairs, norm, eps):
    """The argument block and the inputs' pointers."""
    _require(q.dim() == 4 and k.dim() == 4 and q.shape[:2] == k.shape[:2] and q.shape[3] == k.shape[3],
             "q must be [B, T, H, D], k [B, T, Hk, D]")
    _require(q.dtype in (torch.bfloat16, torch.float32) and k.dtype is q.dtype, "q and k must share dtype bf16 or fp32")
    if norm not in QK_NORMS or pairs not in PAIRS:
        _require(norm in QK_NORMS, "norm must be one of %s" % sorted(QK_NORMS))
        _require(False, "pairs must be one of %s" % sorted(PAIRS))
    _require((positions is None) == (inv_freq is None), "positions and inv_freq come together")
    B, T, H, D = q.shape
    Hk, dev = k.shape[2], q.get_device()
    axes = 1 if sections is None else len(sections)
    _require(1 <= axes <= 4, "sections must name one to four axes")
    rot = 0
    if inv_freq is not None:
        _require(inv_freq.dim() == 1, "inv_freq must be fp32 [rot / 2]")
        rot = 2 * inv_freq.numel()
        _require(sections is None or sum(sections) == rot // 2, "sections must sum to the number of frequencies")
    (pq, sq), (pk, sk) = _heads("q", q, q.shape, q.dtype, dev), _heads("k", k, k.shape, q.dtype, dev)
    shape = (B, T) if sections is None else (axes, B, T)
    ptrs = (pq, pk, _tensor("q_weight", q_weight, (D,), torch.float32, dev),
            _tensor("k_weight", k_weight, (D,), torch.float32, dev),
            _tensor("positions", positions, shape, torch.int32, dev),
            _tensor("inv_freq", inv_freq, (rot // 2,), torch.float32, dev))
    sec = (_c_int * 4)(*(sections if sections is not None and axes > 1 else ()))
    a = QkArgs(B * T, H, Hk, D, rot, KDA_BF16 if q.dtype == torch.bfloat16 else KDA_F32, QK_NORMS[norm], PAIRS[pairs],
               axes, sec, int(bool(spread)), float(eps), sq, sk, 0, 0)
    return a, dev, ptrs


@_on_device
def qk_norm_rope(q, k, q_weight=None, k_weight=None, *, positions=None, inv_freq=None, sections=None, spread=False,
                 pairs="half", norm="rms", eps=1e-6, q_out=None, k_out=None):
    """The norm of every head's query and key row, and their rotation by position, in one pass.

    Per row x of D channels: n = weight x / sqrt(mean(x^2) + eps) (``norm="l2"``: the sum in place of
    the mean, what ``chunk_kda`` and ``chunk_gated_delta`` expect; ``"none"``: no norm), then the
    first 2 len(inv_freq) channels turn, pair by pair, by position * inv_freq[i]. A pair is channels
    i and i + len(inv_freq) (``pairs="half"``) or 2i and 2i + 1 (``"adjacent"``). q is [B, T, H, D],
    k [B, T, Hk, D], bf16 or fp32; their tokens may lie apart (parts of a fused projection). Weights
    are fp32 [D], inv_freq fp32, positions int32 [B, T].

    With ``sections`` (one to four numbers of frequencies) positions are [axes, B, T], for instance
    time, height and width, and every frequency reads one axis: neighbours in the axes' order, or with
    ``spread`` axis a >= 1 frequencies a, a + axes, a + 2 axes, ... (sections[a] of them), axis 0 the others.
    Angles are formed in fp64. Returns (q', k'); ``q_out`` and ``k_out`` may be q and k themselves.
    """
    a, dev, (pq, pk, pwq, pwk, pp, pf) = _qk_args(q, k, q_weight, k_weight, positions, inv_freq, sections, spread,
                                                  pairs, norm, eps)
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        po = q_out.data_ptr()
    else:
        po, a.qo_stride = _heads("q_out", q_out, q.shape, q.dtype, dev)
    if k_out is None:
        k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
        pko = k_out.data_ptr()
    else:
        pko, a.ko_stride = _heads("k_out", k_out, k.shape, q.dtype, dev)
    _launch(dev, _lib().kda_qk_norm_rope_fwd, ctypes.byref(a), pq, pk, pwq, pwk, pp, pf, po, pko)
    return q_out, k_out


@_on_device
def qk_norm_rope_bwd(q, k, dq_out, dk_out, q_weight=None, k_weight=None, *, positions=None, inv_freq=None,
                     sections=None, spread=False, pairs="half", norm="rms", eps=1e-6, workspace=None):
    """Gradients of sum(dq_out * q') + sum(dk_out * k') for ``qk_norm_rope``.

    Returns a dict: dq, dk, and for the weights that were passed dq_weight and dk_weight (fp32);
    None for the rest.
    """
    a, dev, (pq, pk, pwq, pwk, pp, pf) = _qk_args(q, k, q_weight, k_weight, positions, inv_freq, sections, spread,
                                                  pairs, norm, eps)
    pdq, a.qo_stride = _heads("dq_out", dq_out, q.shape, q.dtype, dev)
    pdk, a.ko_stride = _heads("dk_out", dk_out, k.shape, q.dtype, dev)
    L = _lib()
    need = 0
    if q_weight is not None or k_weight is not None:
        need = int(L.kda_qk_norm_rope_bwd_workspace_bytes(ctypes.byref(a)))
    pw, nw, _keep = _workspace(workspace, need, dev)
    like = lambda t: None if t is None else torch.empty_like(t)  # noqa: E731
    got = dict(dq=torch.empty_like(q, memory_format=torch.contiguous_format),
               dk=torch.empty_like(k, memory_format=torch.contiguous_format), dq_weight=like(q_weight),
               dk_weight=like(k_weight))
    ptr = {n: None if t is None else t.data_ptr() for n, t in got.items()}
    _launch(dev, L.kda_qk_norm_rope_bwd, ctypes.byref(a), pq, pk, pwq, pwk, pp, pf, pdq, pdk, ptr["dq"], ptr["dk"],
            ptr["dq_weight"], ptr["dk_weight"], pw, nw)
    return got
