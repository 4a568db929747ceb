"""Plain 64-bit references of the gated delta rule with one decay per head, and of the query/key norm
with rotation, straight from their definitions (token by token; gradients by differentiating that), and
the bounds that the tests of the delta rule count roundings of.

Bounds. With rows k of norm one and beta in [0, 1], a step S -> (I - beta k k^T) e^g S enlarges nothing, so
a rounding of relative size e made on the way to the state stays below e times the largest state (and
written row) so far, M, for good. Every quantity is a product of such a state (M), of its gradient (M'),
and of rows: |o_t| <= scale |q_t| M, |du_t| <= |k_t| M', |dq_t| <= scale |d_o,t| M and so on, norms of rows.
A result that passes n fp32 roundings is off by at most n 2^-24 times that product, row by row in the
2-norm; bf16 results add one rounding, and o what two bf16 parts of state, scores and u leave out."""
import torch

ULP32 = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
LEFT_OUT = {torch.bfloat16: 3 * 2.0 ** -16, torch.float32: 0.0}  # two bf16 parts hold 16 bits


def slots_of(B, T, cu):
    off = [n * T for n in range(B + 1)] if cu is None else [int(x) for x in cu]
    return list(zip(off, off[1:]))


def roundings(K, V, T):
    """At most, of one term: products over K and V, sums over a chunk, its solve (whose condition is taken
    as 4), the operands' parts; and as many again for every chunk that the state passed."""
    return 4 * (K + V + 200) * (T // 64 + 1)


def walk(q, k, v, g, beta, h0, cu=None, scale=None):
    """(o, ht, S' of every token, u) in float64; q, k [B, T, Hk, K], v [B, T, H, V], g [B, T, H] or None.
    Rows outside cu are zero."""
    B, T, Hk, K = q.shape
    H, V = v.shape[2], v.shape[3]
    scale = K ** -0.5 if scale is None else scale
    qf, kf = (x.reshape(B * T, Hk, K).repeat_interleave(H // Hk, 1) for x in (q, k))
    vf, bf = v.reshape(B * T, H, V), beta.reshape(B * T, H)
    a = torch.exp(g.reshape(B * T, H)) if g is not None else torch.ones(B * T, H, dtype=torch.float64)
    rows, states, before, us = {}, [], {}, {}
    for n, (lo, hi) in enumerate(slots_of(B, T, cu)):
        S = h0[n] if h0 is not None else torch.zeros(H, K, V, dtype=torch.float64)
        for t in range(lo, hi):
            S = a[t][:, None, None] * S
            before[t] = S
            u = us[t] = bf[t][:, None] * (vf[t] - (S * kf[t][:, :, None]).sum(1))
            S = S + kf[t][:, :, None] * u[:, None, :]
            rows[t] = scale * (qf[t][:, :, None] * S).sum(1)
        states.append(S)
    zero = torch.zeros(H, V, dtype=torch.float64)
    o = torch.stack([rows.get(t, zero) for t in range(B * T)]) if B * T else torch.zeros(0, H, V, dtype=torch.float64)
    ht = torch.stack(states) if states else torch.zeros(0, H, K, V, dtype=torch.float64)
    return o.reshape(B, T, H, V), ht, before, us


def delta(*args, **kw):
    return walk(*args, **kw)[:2]


def grads(q, k, v, g, beta, h0, do, dht, cu=None, scale=None):
    """dq, dk, dv, dg, dbeta, dh0 in float64, by differentiating walk(); dg zeros without g."""
    N = len(slots_of(q.shape[0], q.shape[1], cu))
    h0 = h0 if h0 is not None else torch.zeros(N, v.shape[2], q.shape[3], v.shape[3], dtype=torch.float64)
    g = torch.zeros_like(beta) if g is None else g
    ins = [x.clone().requires_grad_(True) for x in (q, k, v, g, beta, h0)]
    o, ht = delta(*ins, cu=cu, scale=scale)
    L = (o * do).sum() + ((ht * dht).sum() if dht is not None else 0.0)
    got = torch.autograd.grad(L, ins, allow_unused=True)
    return [torch.zeros_like(x) if d is None else d for x, d in zip(ins, got)]


def sizes(q, k, v, g, beta, h0, cu=None, scale=None, do=None, dht=None):
    """Bounds of the terms behind every row of o and behind ht, [B, T, H] and [N, H]; with do the same of dq, dk, dv,
    dg, dbeta, dh0."""
    B, T, Hk, K = q.shape
    H = v.shape[2]
    scale = K ** -0.5 if scale is None else scale
    _, ht, before, us = walk(q, k, v, g, beta, h0, cu, scale)
    per = lambda x: x.reshape(B * T, Hk, K).repeat_interleave(H // Hk, 1)  # noqa: E731
    norm = lambda x: x.reshape(B * T, H, -1).norm(dim=-1)  # noqa: E731
    qn, kn, vn = per(q).norm(dim=-1), per(k).norm(dim=-1), norm(v)
    zero = torch.zeros(H, dtype=torch.float64)
    M, last = torch.zeros(B * T, H, dtype=torch.float64), []
    for n, (lo, hi) in enumerate(slots_of(B, T, cu)):
        m = h0[n].flatten(1).norm(dim=-1) if h0 is not None else zero
        for t in range(lo, hi):
            m = torch.maximum(m, before[t].flatten(1).norm(dim=-1)) + 0.0
            m = torch.maximum(m, vn[t] + us[t].norm(dim=-1))
            M[t] = m
        last.append(m)
    MT = torch.stack(last) if last else torch.zeros(0, H, dtype=torch.float64)
    shape = lambda x: x.reshape(B, T, H)  # noqa: E731
    out = [shape(scale * qn * M), MT]
    if do is None:
        return out
    a = torch.exp(g.reshape(B * T, H)) if g is not None else torch.ones(B * T, H, dtype=torch.float64)
    qf, kf, df, bf = per(q), per(k), do.reshape(B * T, H, -1), beta.reshape(B * T, H)
    D, first, dun = torch.zeros(B * T, H, dtype=torch.float64), [], torch.zeros(B * T, H, dtype=torch.float64)
    for n, (lo, hi) in enumerate(slots_of(B, T, cu)):
        G = dht[n] if dht is not None else torch.zeros_like(ht[n])
        m = G.flatten(1).norm(dim=-1)
        for t in range(hi - 1, lo - 1, -1):
            G = G + scale * qf[t][:, :, None] * df[t][:, None, :]
            m = torch.maximum(m, G.flatten(1).norm(dim=-1))
            D[t] = m
            du = (G * kf[t][:, :, None]).sum(1)
            dun[t] = du.norm(dim=-1)
            G = a[t][:, None, None] * (G - kf[t][:, :, None] * (bf[t][:, None] * du)[:, None, :])
        first.append(m)
    un = torch.stack([us[t].norm(dim=-1) if t in us else zero for t in range(B * T)]) if B * T else D
    dq = scale * norm(do) * M
    dk = un * D + bf * dun * M + kn * M * D  # the last: u and du are off by the states' errors
    terms = qn * dq + kn * dk
    dg = torch.zeros_like(terms)
    for lo, hi in slots_of(B, T, cu):  # sums over the rest of the chunk, and <S, dS> behind it
        c = terms[lo:hi]
        w = torch.cat([c.cumsum(0), torch.zeros(0, H, dtype=torch.float64)])
        tail = torch.cat([w[63:], w[-1:].expand(min(63, hi - lo), H)])[: hi - lo] if hi > lo else w
        dg[lo:hi] = tail - w + c + M[lo:hi].max(0).values * D[lo:hi] if hi > lo else w
    share = lambda x: x.reshape(B, T, Hk, H // Hk).sum(-1)  # noqa: E731
    return out + [share(dq), share(dk), shape(bf * kn * D), shape(dg), shape(dun * vn + kn * D * vn + kn * kn * M * D),
                  torch.stack(first) if first else MT]


def qk_rope(x, weight, norm, eps, pos, freq, axis, pairs):
    """One tensor's rows in float64: x [B, T, heads, D], pos [axes, B, T] or None, axis: of every frequency."""
    D = x.shape[-1]
    if norm != "none":
        ss = (x * x).sum(-1, keepdim=True) / (D if norm == "rms" else 1)
        x = x / torch.sqrt(ss + eps)
    if weight is not None:
        x = x * weight
    if pos is None:
        return x
    half = freq.numel()
    t = torch.stack([pos[axis[i]].double() * freq[i].double() for i in range(half)], -1)[:, :, None] if half else None
    if not half:
        return x
    a = [i if pairs == "half" else 2 * i for i in range(half)]
    b = [i + half if pairs == "half" else 2 * i + 1 for i in range(half)]
    y = x.clone()
    y[..., a] = x[..., a] * torch.cos(t) - x[..., b] * torch.sin(t)
    y[..., b] = x[..., b] * torch.cos(t) + x[..., a] * torch.sin(t)
    return y


def axes_of(half, sections, spread):
    """The axis that every frequency reads."""
    if sections is None:
        return [0] * half
    if not spread:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    out = [0] * half
    for a in range(1, len(sections)):
        for j in range(sections[a]):
            out[a + j * len(sections)] = a
    return out
