"""Bounds in the 2-norm of one sequence and head, tight enough that a part left out, a wrong sign or a lost term of one
row cannot pass (delta_ref.py's hold for every single value, and are far wider).

Roundings are of either sign, so n of them add up to sqrt(n) 2^-24 of the terms; and the terms of a contraction over
K or V values lie in all directions, so a product of a state of 2-norm M with a row x is of the size |x| M / sqrt(K).
With M the largest state so far as far as the decays since have left it (roundings decay alike), M' the same of the
states' gradients from the end, u what is written and du its gradient, the terms and what the errors of the states add
to them are, in the 2-norm of a row:
    o      scale |q| M / sqrt(K)                 ht     M
    dq     scale |do| M / sqrt(V)                dh0    M'
    du     |k| M' / sqrt(K)                      dv     beta du
    dk     (|u| M' + beta |du| M) / sqrt(V) + |k| M M' / sqrt(K V)
    dbeta  (|du| |v| + |k| M' |v| / sqrt(K)) / sqrt(V) + |k|^2 M M' / (K sqrt(V))
    dg     the root of the sum of (|q| dq + |k| dk)^2 / K over the rest of the chunk, and M M' / sqrt(K V)
A result passes sums over K, over V and over a chunk's 64 tokens, and the state brings as many for every chunk it has
passed: n = (K + V + 64) (1 + T / 64). Terms that are not quite alike are allowed for by a factor of four."""
import torch

import delta_ref as ref


def slot_sums(x, B, T, cu):
    """Root of the sums over every sequence's tokens of the squares of x [B T, H]."""
    return torch.stack([x[lo:hi].square().sum(0).sqrt() for lo, hi in ref.slots_of(B, T, cu)])


def bounds(q, k, v, g, beta, h0, cu=None, scale=None, do=None, dht=None):
    """What the errors of o, ht, and with do of dq, dk, dv, dg, dbeta and dh0 stay below before a rounding to the
    outputs' type, in the 2-norm of every sequence and head [N, H] (dq and dk: [N, Hk])."""
    B, T, Hk, K = q.shape
    H, V = v.shape[2:]
    scale = K ** -0.5 if scale is None else scale
    _, ht, before, us = ref.walk(q, k, v, g, beta, h0, cu, scale)
    per = lambda x: x.reshape(B * T, Hk, K).repeat_interleave(H // Hk, 1)  # noqa: E731
    qf, kf, vf, bf = per(q), per(k), v.reshape(B * T, H, V), beta.reshape(B * T, H)
    qn, kn, vn = qf.norm(dim=-1), kf.norm(dim=-1), vf.norm(dim=-1)
    a = torch.exp(g.reshape(B * T, H)) if g is not None else torch.ones(B * T, H, dtype=torch.float64)
    slots = ref.slots_of(B, T, cu)
    zeros = lambda: torch.zeros(B * T, H, dtype=torch.float64)  # noqa: E731
    M, D, dun, un, n = zeros(), zeros(), zeros(), zeros(), torch.ones(len(slots), dtype=torch.float64)
    last, first = torch.zeros(len(slots), H, dtype=torch.float64), torch.zeros(len(slots), H, dtype=torch.float64)
    for i, (lo, hi) in enumerate(slots):
        n[i] = (K + V + 64) * (1 + (hi - lo) / 64)
        m = h0[i].flatten(1).norm(dim=-1) if h0 is not None else torch.zeros(H, dtype=torch.float64)
        for t in range(lo, hi):
            un[t] = us[t].norm(dim=-1)
            m = M[t] = torch.maximum(torch.maximum(a[t] * m, before[t].flatten(1).norm(dim=-1)), un[t] * kn[t])
        last[i] = torch.maximum(m, ht[i].flatten(1).norm(dim=-1))
        if do is None:
            continue
        G = dht[i] if dht is not None else torch.zeros_like(ht[i])
        m = G.flatten(1).norm(dim=-1)
        for t in range(hi - 1, lo - 1, -1):
            G = G + scale * qf[t][:, :, None] * do.reshape(B * T, H, V)[t][:, None, :]
            m = D[t] = torch.maximum(m, G.flatten(1).norm(dim=-1))
            du = (G * kf[t][:, :, None]).sum(1)
            dun[t] = du.norm(dim=-1)
            m = a[t] * m
            G = a[t][:, None, None] * (G - kf[t][:, :, None] * (bf[t][:, None] * du)[:, None, :])
        first[i] = m
    e = 4 * ref.ULP32 * n.sqrt()[:, None]
    rows = lambda x: e * slot_sums(x, B, T, cu)  # noqa: E731
    out = dict(o=rows(scale * qn * M / K ** 0.5), ht=e * last)
    if do is None:
        return out
    dq = scale * do.reshape(B * T, H, V).norm(dim=-1) * M / V ** 0.5
    dk = (un * D + bf * dun * M) / V ** 0.5 + kn * M * D / (K * V) ** 0.5
    dg = zeros()
    terms = ((qn * dq + kn * dk) ** 2) / K
    for lo, hi in slots:
        for c in range(lo, hi, 64):
            rest = terms[c:min(c + 64, hi)]
            dg[c:min(c + 64, hi)] = rest.flip(0).cumsum(0).flip(0).sqrt()
    share = lambda x: rows(x).reshape(len(slots), Hk, H // Hk).square().sum(-1).sqrt()  # noqa: E731
    out.update(dq=share(dq), dk=share(dk), dv=rows(bf * (dun + kn * D / K ** 0.5)), dg=rows(dg + M * D / (K * V) ** 0.5),
               dbeta=rows((dun * vn + kn * D * vn / K ** 0.5) / V ** 0.5 + kn * kn * M * D / (K * V ** 0.5)), dh0=e * first)
    return out


def exceeded(got, want, bound, B, T, cu=None, states=False):
    """(How many times the bound the largest error of a sequence and head is, the largest bound relative to the
    values). got's type says how it was rounded."""
    off, own = got.detach().cpu().double() - want, want
    if states:
        off, own = off.flatten(2).norm(dim=-1), own.flatten(2).norm(dim=-1)
    else:
        off, own = (slot_sums(x.reshape(B * T, x.shape[2], -1).norm(dim=-1), B, T, cu) for x in (off, own))
    assert torch.isfinite(off).all()
    most = bound + ref.HALF[got.dtype] * own
    some = most > 0
    assert (off[~some] == 0).all()
    if not some.any():
        return 0.0, 0.0
    return (off[some] / most[some]).max().item(), (most[some] / own[some].clamp_min(1e-300)).max().item()


NAMES = ("o", "ht", "dq", "dk", "dv", "dg", "dbeta", "dh0")


def reference(ins, do, dht, cu=None, scale=None):
    """All of NAMES in 64 bits."""
    o, ht = ref.delta(*ins, cu=cu, scale=scale)
    return dict(zip(NAMES, [o, ht] + ref.grads(*ins, do, dht, cu=cu, scale=scale)))


IN = ("q", "k", "v", "g", "beta", "h0")


def step_of(which, ins, want, seed=9):
    """A direction with as much of the gradient in it as of a random one: along it the loss changes by far more than
    its errors, and a gradient that is wrong in any part shows."""
    gen = torch.Generator().manual_seed(seed)
    r = torch.randn(want.shape, generator=gen, dtype=torch.float64)
    return ((r / r.norm() + want / want.norm()) * 2.0).float()


def check_differences(which, ins, do, dht, loss, gradient):
    """The gradient along a direction against central differences of the loss and against 64 bits. ins: float64
    inputs by name (those of IN); loss(x): the loss with input `which` replaced by x (fp32); gradient: of it.

    An error of o of norm b changes the loss by at most b |do|; that of the gradient, along d, by at most b |d|.
    q, v and h0 enter the loss linearly: differences are the gradient. k, beta and g bend it: the same differences
    of the definition in 64 bits say by how much."""
    args = [ins[x] for x in IN]
    want = reference(args, do, dht)["d" + which]
    d = step_of(which, ins, want)
    x = ins[which].float()
    b = bounds(*args, do=do, dht=dht)
    noise = (b["o"].norm() * do.norm() + b["ht"].norm() * dht.norm()).item()
    off = (b["d" + which].norm() * d.double().norm()).item()
    at = (want * d.double()).sum().item()
    along = (gradient.detach().cpu().double() * d.double()).sum().item()
    h = 1.0 if which in ("q", "v", "h0") else 1 / 8
    plus, minus = x + h * d, x - h * d

    def exact(y):
        o, ht = ref.delta(*[y.double() if n == which else ins[n] for n in IN])
        return ((o * do).sum() + (ht * dht).sum()).item()

    # what is stepped by is what the fp32 sums are
    real = ((plus.double() - minus.double()) * want).sum().item() / (2 * h)
    true, mine = (exact(plus) - exact(minus)) / (2 * h), (loss(plus) - loss(minus)) / (2 * h)
    if which in ("q", "v", "h0"):
        assert abs(true - real) <= 1e-9 * abs(real)
    # (errors of both losses; states are larger by the step: twice)
    tol = 2 * noise / h
    assert tol <= 0.01 * abs(at) and off <= 0.01 * abs(at), (which, tol, off, at)
    assert abs(true - at) <= 0.2 * abs(at), (which, true, at)  # the step is small beside the bend
    assert abs(mine - true) <= tol, (which, mine, true, tol)
    assert abs(along - at) <= off, (which, along, at, off)
    assert abs(along - mine) <= off + tol + abs(true - at), (which, along, mine)
