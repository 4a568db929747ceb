"""Plain 64-bit references of linear attention with one decay per head and of the block norm,
straight from their definitions (token by token; gradients by differentiating that), with the
size of the terms behind every value, which the tests' tolerances count roundings of."""
import torch

ULP32 = 2.0 ** -24  # largest relative rounding of one fp32 operation
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # finfo.eps / 2: one rounding to the type


def slots_of(B, T, cu):
    off = [n * T for n in range(B + 1)] if cu is None else [int(x) for x in cu]
    return list(zip(off, off[1:]))


def attn(q, k, v, g, h0, cu=None, scale=None):
    """(o, ht) in float64. q, k [B, T, Hk, K], v [B, T, H, V], g [B, T, H] or [H]; all float64.
    Rows outside cu are zero."""
    B, T, Hk, K = q.shape
    H, V = v.shape[2], v.shape[3]
    rep = H // Hk
    scale = K ** -0.5 if scale is None else scale
    qf, kf = (x.reshape(B * T, Hk, K).repeat_interleave(rep, 1) for x in (q, k))
    vf = v.reshape(B * T, H, V)
    gf = g.reshape(B * T, H) if g.dim() == 3 else g.expand(B * T, H)
    a = torch.exp(gf)
    rows, states = {}, []
    for n, (lo, hi) in enumerate(slots_of(B, T, cu)):
        S = h0[n] if h0 is not None else torch.zeros(H, K, V, dtype=torch.float64)
        for t in range(lo, hi):
            S = a[t][:, None, None] * S + kf[t][:, :, None] * vf[t][:, None, :]
            rows[t] = scale * (qf[t][:, :, None] * S).sum(1)
        states.append(S)
    zero = torch.zeros(H, V, dtype=torch.float64)
    o = torch.stack([rows.get(t, zero) for t in range(B * T)]) if B * T else torch.zeros(0, H, V, dtype=torch.float64)
    ht = torch.stack(states) if states else torch.zeros(0, H, K, V, dtype=torch.float64)
    return o.reshape(B, T, H, V), ht


def attn_grads(q, k, v, g, h0, do, dht, cu=None, scale=None):
    """dq, dk, dv, dg, dh0 in float64, by differentiating attn()."""
    N = len(slots_of(q.shape[0], q.shape[1], cu))
    h0 = h0 if h0 is not None else torch.zeros(N, v.shape[2], q.shape[3], v.shape[3], dtype=torch.float64)
    ins = [x.clone().requires_grad_(True) for x in (q, k, v, g, h0)]
    o, ht = attn(*ins, cu=cu, scale=scale)
    L = (o * do).sum() + ((ht * dht).sum() if dht is not None else 0.0)
    got = torch.autograd.grad(L, ins, allow_unused=True)
    return [torch.zeros_like(x) if d is None else d for x, d in zip(ins, got)]


def attn_sizes(q, k, v, g, h0, cu=None, scale=None):
    """Sums of the absolute terms behind o and ht."""
    return attn(q.abs(), k.abs(), v.abs(), g, None if h0 is None else h0.abs(), cu, scale)


def grad_sizes(q, k, v, g, h0, do, dht, cu=None, scale=None):
    """Sums of the absolute terms behind dq, dk, dv, dg and dh0. dg is a sum over the rest of the
    sequence of the terms of q.dq and k.dk, and of <ht, dht>."""
    ab = lambda x: None if x is None else x.abs()  # noqa: E731
    dq, dk, dv, _, dh0 = attn_grads(q.abs(), k.abs(), v.abs(), g, ab(h0), do.abs(), ab(dht), cu, scale)
    B, T, Hk, K = q.shape
    H = v.shape[2]
    # the parts of each value head: of shared heads no more than their sum
    per = lambda x: x.reshape(B * T, Hk, K).repeat_interleave(H // Hk, 1)  # noqa: E731
    terms = (per(q.abs()) * per(dq) + per(k.abs()) * per(dk)).sum(-1)
    ends = torch.zeros(len(slots_of(B, T, cu)), H, dtype=torch.float64)
    if dht is not None:
        _, ht = attn_sizes(q, k, v, g, h0, cu, scale)
        ends = (ht * dht.abs()).sum((-1, -2))
    dg = torch.zeros(B * T, H, dtype=torch.float64)
    for n, (lo, hi) in enumerate(slots_of(B, T, cu)):
        dg[lo:hi] = terms[lo:hi].flip(0).cumsum(0).flip(0) + ends[n]
    dg = dg.reshape(B, T, H) if g.dim() == 3 else dg.sum(0)
    return dq, dk, dv, dg, dh0


def roundings(K, V, T):
    """fp32 roundings on the way of one term into a sum of the chunked form, at most: products over K
    and V, two sums over a chunk of 64, each chunk's state update, the parts of its operands."""
    return K + V + 2 * 64 + 4 * (T // 32 + 1) + 64


def norm(x, weight, gate, act, residual, scale, next_weight, nxt, eps, kind):
    """[y, z] (or [y]) in float64."""
    D = x.shape[-1]
    ss = (x * x).sum(-1, keepdim=True) / (D if kind == "rms" else 1)
    y = x / torch.sqrt(ss + eps)
    if weight is not None:
        y = y * weight
    if gate is not None:
        y = y * torch.sigmoid(gate) * (gate if act == "silu" else 1.0)
    y = y * scale
    if residual is not None:
        y = y + residual
    if not nxt:
        return [y]
    z = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
    return [y, z if next_weight is None else z * next_weight]
