"""Cases, plain forms and calls of the gated delta rule and the query/key norm with rotation.

The gated delta rule with one decay per head (K x V state S, g <= 0 natural-log decay):

    S'_t = exp(g_t) S_{t-1},   u_t = beta_t (v_t - S'_t^T k_t),   S_t = S'_t + k_t u_t^T,   o_t = scale S_t^T q_t

as a chunked forward over prompts ("prefill"), its gradient ("train"), and the recurrence over a few
tokens with the state updated in place ("decode"). The query/key norm takes every head's row of q and
k to weight x / sqrt(mean(x^2) + eps) (or the sum: l2) and turns its channel pairs by angles
position * frequency, a frequency reading one of up to four position axes, forward ("rope") and
backward ("rope_train").
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
DEV = "cuda"
CHUNK = 64  # rows per chunk of the plain form
EPS = 1e-6
THETA = 1e6


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def _delta(op, name, b, t, h, k, v, dtype="bf16", hk=0, slots=0, states=True, cut=0, decay=True):
    return dict(name=name, op=op, b=b, t=t, h=h, hk=hk or h, k=k, v=v, dtype=dtype, slots=slots, states=states, cut=cut,
                decay=decay)


def _rope(op, name, b, t, h, hk, d, rot, dtype="bf16", norm="rms", axes=1, spread=False, pairs="half", fused=False):
    return dict(name=name, op=op, b=b, t=t, h=h, hk=hk, d=d, rot=rot, dtype=dtype, norm=norm, axes=axes, spread=spread,
                pairs=pairs, fused=fused)


def listed():
    return [
        # a serving prefill that fills the card: four prompts of 4096 tokens, 64 heads of width 128, states carried
        _delta("prefill", "delta prefill b4 t4096 h64 d128", 4, 4096, 64, 128, 128),
        # one long document on few heads, from an empty state
        _delta("prefill", "delta prefill b1 t32768 h16 d128", 1, 32768, 16, 128, 128, states=False),
        # prompts of mixed lengths packed into one batch, one slot empty, q and k heads shared by pairs of value heads
        _delta("prefill", "delta prefill packed t15872", 1, 15872, 32, 128, 128, hk=16, slots=10, cut=5),
        # a small model in full precision, a length that is no multiple of anything, unequal odd widths, no decay
        _delta("prefill", "delta prefill fp32 b2 t1000", 2, 1000, 8, 72, 40, dtype="fp32", decay=False),
        # a training step's gradient at the sizes of a mid-sized model
        _delta("train", "delta train b4 t2048 h32 d128", 4, 2048, 32, 128, 128, states=False),
        # a packed training batch with shared q/k heads, carried states and unequal widths
        _delta("train", "delta train packed t4999", 1, 4999, 16, 64, 128, hk=8, slots=7, cut=9),
        # a full decode batch: 256 sequences, one token each
        _delta("decode", "delta decode 256x1 h64 d128", 256, 1, 64, 128, 128),
        # one user, one token: the latency of a single step
        _delta("decode", "delta decode 1x1 h16 d128", 1, 1, 16, 128, 128),
        # the prompt pass of a layer of 32 query and 8 key heads, views of one fused projection
        _rope("rope", "rope b4 t4096 h32/8 d128", 4, 4096, 32, 8, 128, 128, fused=True),
        # a decode step of images and text: three position axes spread over the frequencies
        _rope("rope", "rope 64x1 h32/8 d128 3 axes", 64, 1, 32, 8, 128, 128, axes=3, spread=True),
        # the gradient of that prompt pass, weights included
        _rope("rope_train", "rope grad b4 t4096 h32/8 d128", 4, 4096, 32, 8, 128, 128),
        # an image encoder's heads of width 72 in full precision, positions by row and column, an odd number of patches
        _rope("rope_train", "rope grad fp32 t1037 d72", 1, 1037, 16, 16, 72, 72, dtype="fp32", axes=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "train", "train", "decode", "rope", "rope_train"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("rope", "rope_train"):
        d = rng.choice([64, 128, 256, 8 * rng.randint(1, 64)])
        rot = rng.choice([d, d, 8 * rng.randint(0, d // 8)])
        hk = _log(rng, 1, 16)
        h = hk * rng.choice([1, 1, 2, 3, 4, 7])
        b = rng.choice([1, 1, 2, 5])
        t = _log(rng, 1, max(2, (1 << 26) // (b * (h + hk) * d)))
        axes = rng.choice([1, 1, 2, 3, 4]) if rot >= 32 else 1
        return dict(op=op, b=b, t=t, h=h, hk=hk, d=d, rot=rot, dtype=dtype, norm=rng.choice(["rms", "rms", "l2", "none"]),
                    axes=axes, spread=axes > 1 and rng.random() < 0.5, pairs=rng.choice(["half", "half", "adjacent"]),
                    fused=rng.random() < 0.4)
    hk = rng.choice([1, 2, 3, 4, 5, 8, 16])
    h = hk * rng.choice([1, 1, 1, 2, 3])
    k, v = (8 * rng.randint(1, 32) for _ in range(2))
    if rng.random() < 0.5:
        k = v = rng.choice([64, 128, 256])
    most = (1 << 30) // (3 if op == "train" else 1) // (4 if dtype == "fp32" else 1)  # of token-heads times K times V
    decay = rng.random() < 0.85
    if op == "decode":
        b, t = _log(rng, 1, 256), rng.choice([1, 1, 1, 2, 4])
        b = max(1, min(b, most // (h * k * v)))
        return dict(op=op, b=b, t=t, h=h, hk=hk, k=k, v=v, dtype=dtype, slots=0, states=True, cut=0, decay=decay)
    tokens = max(64, min(16384, 8 * most // (h * k * v)))
    t = _log(rng, 1, tokens)
    packed = rng.random() < 0.4
    b = 1 if packed else max(1, min(rng.choice([1, 2, 3, 4]), tokens // t))
    return dict(op=op, b=b, t=t, h=h, hk=hk, k=k, v=v, dtype=dtype, slots=rng.randint(1, 12) if packed else 0,
                states=rng.random() < 0.7, cut=rng.randrange(1 << 16), decay=decay)


def _offsets(case):
    """Offsets of a packed case: lengths cut at random places, so that some are short, some long and some empty."""
    rng = random.Random(case["cut"])
    cuts = sorted(rng.randint(0, case["t"]) for _ in range(case["slots"] - 1))
    if len(cuts) > 2:
        cuts[1] = cuts[0]  # an empty slot
    return [0] + cuts + [case["t"]]


def _slots(case):
    return case["slots"] or case["b"]


def _sections(case):
    """Frequencies of each axis: the later axes a share each, the first what is left."""
    half, a = case["rot"] // 2, case["axes"]
    return [half - (a - 1) * (half // a)] + [half // a] * (a - 1)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    rows = case["b"] * case["t"]
    if case["op"] in ("rope", "rope_train"):
        n = rows * (case["h"] + case["hk"]) * case["d"]
        pos = 4 * rows * case["axes"] if case["rot"] else 0
        if case["op"] == "rope":
            return {"bytes": 2 * n * e + pos, "flops": 8 * n}
        return {"bytes": 3 * n * e + pos, "flops": 18 * n}
    n = _slots(case)
    kk, vv = rows * case["hk"] * case["k"] * e, rows * case["h"] * case["v"] * e
    state = n * case["h"] * case["k"] * case["v"] * 4
    g = rows * case["h"] * 4 * (2 if case["decay"] else 1)  # g and beta
    steps = rows * case["h"] * case["k"] * case["v"]
    if case["op"] == "train":  # q, k, v, do, g, beta and the states in; dq, dk, dv, dg, dbeta and dh0 out
        return {"bytes": 4 * kk + 3 * vv + 2 * g + state * (3 if case["states"] else 1), "flops": 16 * steps}
    return {"bytes": 2 * kk + 2 * vv + g + state * (2 if case["states"] else 1), "flops": 6 * steps}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, dtype=torch.float32, mul=1.0):
        return (torch.randn(*shape, device=DEV, generator=gen) * mul).to(dtype)

    if case["op"] in ("rope", "rope_train"):
        return _prepare_rope(case, randn, gen, dt)
    b, t, h, hk, k, v = (case[x] for x in ("b", "t", "h", "hk", "k", "v"))
    n = _slots(case)

    def unit(*shape):  # rows of norm one, as the layer's l2 norm leaves them
        x = randn(*shape)
        return (x * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS)).to(dt)

    s = dict(case=case, q=unit(b, t, hk, k), k=unit(b, t, hk, k), v=randn(b, t, h, v, dtype=dt))
    # a rate per head times a softplus of each token's input; write strengths by a sigmoid
    rate = torch.exp(randn(h) - 1.5)
    s["g"] = -rate * torch.log1p(torch.exp(randn(b, t, h))) if case["decay"] else None
    s["beta"] = 1 / (1 + torch.exp(-randn(b, t, h)))
    s["h0"] = randn(n, h, k, v, mul=0.5) if case["states"] else None
    s["cu"] = torch.tensor(_offsets(case), dtype=torch.int32, device=DEV) if case["slots"] else None
    # the plain form's gather of a packed batch into rows of one sequence each
    if case["slots"]:
        off = torch.tensor(_offsets(case), device=DEV)
        lens = off[1:] - off[:-1]
        at = torch.arange(int(lens.max()), device=DEV)
        s["inside"] = at[None, :] < lens[:, None]
        s["from"] = torch.where(s["inside"], off[:-1, None] + at[None, :], torch.zeros_like(at)[None, :])
        s["slot"] = torch.repeat_interleave(torch.arange(n, device=DEV), lens)
        s["place"] = torch.arange(t, device=DEV) - off[s["slot"]]
    if case["op"] == "train":
        s["do"] = randn(b, t, h, v, dtype=dt)
        s["dht"] = randn(n, h, k, v, mul=0.5) if case["states"] else None
    return s


def _prepare_rope(case, randn, gen, dt):
    b, t, h, hk, d, rot = (case[x] for x in ("b", "t", "h", "hk", "d", "rot"))
    if case["fused"]:  # q, k and v of one projection
        qkv = randn(b, t, (h + 2 * hk) * d, dtype=dt)
        q, k = qkv[..., : h * d].unflatten(-1, (h, d)), qkv[..., h * d: (h + hk) * d].unflatten(-1, (hk, d))
    else:
        q, k = randn(b, t, h, d, dtype=dt), randn(b, t, hk, d, dtype=dt)
    w = case["norm"] != "none"
    s = dict(case=case, q=q, k=k, q_weight=1 + randn(d, mul=0.1) if w else None, k_weight=1 + randn(d, mul=0.1) if w else None)
    s["pos"] = s["freq"] = s["sections"] = None
    if rot:
        # text counts on to the end of a long context; images count rows and columns
        base = torch.randint(0, 1 << 17, (b, 1), device=DEV, generator=gen)
        axes = [base + torch.arange(t, device=DEV)]
        axes += [torch.randint(0, 256, (b, t), device=DEV, generator=gen) for _ in range(case["axes"] - 1)]
        s["pos"] = (torch.stack(axes) if case["axes"] > 1 else axes[0]).to(torch.int32).contiguous()
        s["freq"] = THETA ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float32) / rot)
        s["sections"] = _sections(case) if case["axes"] > 1 else None
    if case["op"] == "rope_train":
        s["dq"], s["dk"] = randn(b, t, h, d, dtype=dt), randn(b, t, hk, d, dtype=dt)
    return s


# ---------------------------------------------------------------------------------------------
# plain forms: the gated delta rule
# ---------------------------------------------------------------------------------------------
def _rows(s, x, heads):
    """[B, T, heads, ...] -> [slots, H, chunks, rows, width] in fp32: one row of chunks per sequence and head."""
    case = s["case"]
    if case["slots"]:
        x = torch.where(s["inside"][:, :, None, None], x[0][s["from"]], torch.zeros((), dtype=x.dtype, device=x.device))
    x = x.to(torch.float64 if x.dtype == torch.float64 else torch.float32).transpose(1, 2)
    if heads != case["h"]:
        x = x.repeat_interleave(case["h"] // heads, dim=1)
    n, h, t, w = x.shape
    c = CHUNK
    while c // 2 >= max(t, 1):
        c //= 2
    nc = max(1, -(-t // c))
    x = torch.nn.functional.pad(x, (0, 0, 0, nc * c - t))
    return x.reshape(n, h, nc, c, w).contiguous()


def _tokens(s, x, heads, dtype):
    """The way back: [slots, H, chunks, rows, width] -> [B, T, heads, width], summed over the heads that share one."""
    case = s["case"]
    n, h, nc, c, w = x.shape
    x = x.reshape(n, h, nc * c, w)
    if heads != h:
        x = x.reshape(n, heads, h // heads, nc * c, w).sum(2)
    x = x.transpose(1, 2)
    x = x[s["slot"], s["place"]][None] if case["slots"] else x[:, : case["t"]]
    return x.to(dtype).contiguous()


def _t(x):
    return x.transpose(-1, -2).contiguous()


def _inverse(a):
    """(I + a)^-1 of strictly lower triangular blocks a, from the inverses of halves, quarters and so on."""
    c = a.shape[-1]
    t = torch.eye(c, dtype=a.dtype, device=a.device).expand_as(a).contiguous()
    n = 1
    while n < c:
        blocks = lambda x: x.unflatten(-1, (c // (2 * n), 2 * n)).unflatten(-3, (c // (2 * n), 2 * n)).diagonal(  # noqa: E731
            dim1=-4, dim2=-2).movedim(-1, -3)  # views of the diagonal blocks of 2 n rows
        at, ax = blocks(t), blocks(a)
        low = at[..., n:, n:].contiguous() @ ax[..., n:, :n].contiguous() @ at[..., :n, :n].contiguous()
        at[..., n:, :n] = -low
        n *= 2
    return t


def _parts(s):
    """What both directions need of every chunk: operands, decays and the inverse."""
    case = s["case"]
    q, k, v = _rows(s, s["q"], case["hk"]), _rows(s, s["k"], case["hk"]), _rows(s, s["v"], case["h"])
    beta = _rows(s, s["beta"][..., None], case["h"])
    g = s["g"].double() if s["g"] is not None else torch.zeros_like(s["beta"], dtype=torch.float64)
    b = _rows(s, g[..., None], case["h"])[..., 0].cumsum(-1)  # within each chunk up to and with every token
    c = b.shape[-1]
    i = torch.arange(c, device=b.device)
    d = torch.exp(torch.clamp(b[..., :, None] - b[..., None, :], max=0.0)).float()
    incl = torch.where(i[:, None] >= i[None, :], d, torch.zeros_like(d))
    strict = torch.where(i[:, None] > i[None, :], d, torch.zeros_like(d))
    head, tail = torch.exp(b).float()[..., None], torch.exp(b[..., -1:] - b).float()[..., None]
    whole = torch.exp(b[..., -1]).float()[..., None, None]
    inv = _inverse(beta * strict * (k @ _t(k)))
    first = s["h0"]
    if first is None:
        first = torch.zeros(_slots(case), case["h"], case["k"], case["v"], device=DEV)
    return q, k, v, beta, incl, strict, head, tail, whole, inv, first


def _walk(k, v, beta, head, tail, whole, inv, st):
    """u of every chunk, the state before every chunk, and the last."""
    us, sts = torch.empty_like(v), []
    kh, kt = k * head, _t(k * tail)
    for c in range(k.shape[2]):
        sts.append(st)
        us[:, :, c] = inv[:, :, c] @ (beta[:, :, c] * (v[:, :, c] - kh[:, :, c] @ st))
        st = whole[:, :, c] * st + kt[:, :, c] @ us[:, :, c]
    return us, torch.stack(sts, 2), st


def _plain_delta(s):
    case = s["case"]
    q, k, v, beta, incl, _, head, tail, whole, inv, first = _parts(s)
    u, st, last = _walk(k, v, beta, head, tail, whole, inv, first)
    o = ((q * head) @ st + (incl * (q @ _t(k))) @ u) * case["k"] ** -0.5
    return _tokens(s, o, case["h"], s["v"].dtype), last


def _plain_step(s):
    """A few tokens, one after another, on the state in place."""
    case, st, out = s["case"], s["h0"], []
    rep = case["h"] // case["hk"]
    for t in range(case["t"]):
        q, k = (s[x][:, t].float().repeat_interleave(rep, 1)[:, :, :, None] for x in ("q", "k"))
        if s["g"] is not None:
            st.mul_(torch.exp(s["g"][:, t])[..., None, None])
        u = s["beta"][:, t, :, None] * (s["v"][:, t].float() - (st * k).sum(-2))
        st.add_(k * u[:, :, None, :])
        out.append((st * q).sum(-2) * case["k"] ** -0.5)
    return torch.stack(out, 1).to(s["v"].dtype), st


def _plain_delta_grad(s):
    case = s["case"]
    q, k, v, beta, incl, strict, head, tail, whole, inv, first = _parts(s)
    u, st, _ = _walk(k, v, beta, head, tail, whole, inv, first)
    do = _rows(s, s["do"], case["h"]) * case["k"] ** -0.5
    p = incl * (q @ _t(k))
    # the gradients of the states after each chunk, and of u before beta, from the end
    ds = s["dht"] if s["dht"] is not None else torch.zeros_like(first)
    du, dsts = torch.empty_like(u), []
    near, kt, qh, kh, back = _t(p) @ do, k * tail, _t(q * head), _t(k * head), _t(inv)
    for c in range(k.shape[2] - 1, -1, -1):
        dsts.append(ds)
        du[:, :, c] = back[:, :, c] @ (near[:, :, c] + kt[:, :, c] @ ds)
        ds = whole[:, :, c] * ds + qh[:, :, c] @ do[:, :, c] - kh[:, :, c] @ (beta[:, :, c] * du[:, :, c])
    dst = torch.stack(dsts[::-1], 2)
    dv = beta * du
    x, y = do @ _t(u), dv @ _t(u)
    dq_far, w_far, y_far = head * (do @ _t(st)), head * (du @ _t(st)), tail * (u @ _t(dst))
    dq = dq_far + (incl * x) @ k
    w = w_far + (strict * (du @ _t(u))) @ k  # S'_t du_t
    dk = y_far + _t(incl * x) @ q - _t(strict * y) @ k - beta * w
    dbeta = (du * v).sum(-1, keepdim=True) - (k * w).sum(-1, keepdim=True)
    # a decay scales every pair that it lies between: pairs inside the chunk, those with a state, and state with state
    m = (p * x - strict * (k @ _t(k)) * y).double()
    far, f = ((q * dq_far).double() - (beta * k * w_far).double()).sum(-1), (k * y_far).double().sum(-1)
    z = m.sum(-1) - m.sum(-2) + far - f
    dg = z.flip(-1).cumsum(-1).flip(-1) + f.sum(-1, keepdim=True) + (
        whole[..., 0].double() * (st.double() * dst.double()).sum((-1, -2))[..., None])
    kt = s["q"].dtype
    got = [_tokens(s, dq, case["hk"], kt), _tokens(s, dk, case["hk"], kt), _tokens(s, dv, case["h"], kt),
           _tokens(s, dbeta, case["h"], torch.float32)[..., 0].contiguous(), ds]
    if s["g"] is not None:
        got.append(_tokens(s, dg[..., None], case["h"], torch.float32)[..., 0].contiguous())
    return got


# ---------------------------------------------------------------------------------------------
# plain forms: the norm with rotation
# ---------------------------------------------------------------------------------------------
def _axis_of(case):
    """The position axis that each frequency reads."""
    sec, half = _sections(case), case["rot"] // 2
    i = torch.arange(half, device=DEV)
    if not case["spread"]:
        return torch.repeat_interleave(torch.arange(case["axes"], device=DEV), torch.tensor(sec, device=DEV))
    a = i % case["axes"]
    return torch.where(i < case["axes"] * torch.tensor(sec, device=DEV)[a], a, torch.zeros_like(a))


def _angles(s):
    """cos and sin of every token's angles, [B, T, 1, rot / 2]."""
    pos = s["pos"] if s["case"]["axes"] > 1 else s["pos"][None]
    a = (pos.double()[_axis_of(s["case"])].movedim(0, -1) * s["freq"].double())[:, :, None]
    return torch.cos(a).float(), torch.sin(a).float()


def _turn(s, x, back=False):
    rot = s["case"]["rot"]
    if not rot:
        return x
    c, n = _angles(s)
    n = -n if back else n
    r = x[..., :rot]
    if s["case"]["pairs"] == "half":
        a, b = r[..., : rot // 2], r[..., rot // 2:]
        r = torch.cat([a * c - b * n, b * c + a * n], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    return torch.cat([r, x[..., rot:]], -1)


def _normed(s, x):
    """(x / norm, 1 / norm) of every row, in fp32."""
    x, norm = x.float(), s["case"]["norm"]
    if norm == "none":
        return x, None
    ss = (x * x).sum(-1, keepdim=True)
    rho = torch.rsqrt((ss / x.shape[-1] if norm == "rms" else ss) + EPS)
    return x * rho, rho


def _plain_rope(s):
    got = []
    for n in ("q", "k"):
        x, _ = _normed(s, s[n])
        w = s[n + "_weight"]
        got.append(_turn(s, x if w is None else x * w).to(s[n].dtype).contiguous())
    return got


def _plain_rope_grad(s):
    got = {}
    for n in ("q", "k"):
        xn, rho = _normed(s, s[n])
        d, w = _turn(s, s["d" + n].float(), back=True), s[n + "_weight"]
        if w is not None:
            got["d%s_weight" % n] = (d * xn).double().sum((0, 1, 2)).float()
            d = d * w
        if rho is not None:
            dot = (d * xn).sum(-1, keepdim=True)
            d = rho * (d - xn * (dot / xn.shape[-1] if s["case"]["norm"] == "rms" else dot))
        got["d" + n] = d.to(s[n].dtype).contiguous()
    return got


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def run(s):
    case = s["case"]
    if case["op"] == "prefill":
        if own:
            from gated_delta_rule_gate_amd import chunk_gated_delta

            return chunk_gated_delta(s["q"], s["k"], s["v"], s["g"], s["beta"], s["h0"], cu_seqlens=s["cu"],
                                     output_final_state=True)
        return _plain_delta(s)
    if case["op"] == "decode":  # the state is updated in place
        if own:
            from gated_delta_rule_gate_amd import recurrent_gated_delta

            return recurrent_gated_delta(s["q"], s["k"], s["v"], s["g"], s["beta"], s["h0"], final_state=s["h0"])
        return _plain_step(s)
    if case["op"] == "train":
        if own:
            from gated_delta_rule_gate_amd import chunk_gated_delta_bwd

            got = chunk_gated_delta_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"], s["h0"], dht=s["dht"],
                                        cu_seqlens=s["cu"])
            return [got[x] for x in ("dq", "dk", "dv", "dbeta", "dh0", "dg") if got[x] is not None]
        return _plain_delta_grad(s)
    options = dict(positions=s["pos"], inv_freq=s["freq"], sections=s["sections"], spread=case["spread"],
                   pairs=case["pairs"], norm=case["norm"], eps=EPS)
    if case["op"] == "rope":
        if own:
            from gated_delta_rule_gate_amd import qk_norm_rope

            return list(qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], **options))
        return _plain_rope(s)
    if own:
        from gated_delta_rule_gate_amd import qk_norm_rope_bwd

        got = qk_norm_rope_bwd(s["q"], s["k"], s["dq"], s["dk"], s["q_weight"], s["k_weight"], **options)
        return {x: t for x, t in got.items() if t is not None}
    return _plain_rope_grad(s)


# ---------------------------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_rope(s) if case["op"] in ("rope", "rope_train") else _exact_delta(s)


def _exact_delta(s):
    """Token by token, every sequence in a row of its own, rows past a sequence's end without effect."""
    case = s["case"]
    off = _offsets(case) if case["slots"] else [i * case["t"] for i in range(case["b"] + 1)]
    lens = [b - a for a, b in zip(off, off[1:])]
    n, h, most = len(lens), case["h"], max(lens + [1])
    rep = h // case["hk"]

    def rows(x):
        x = x.reshape(-1, *x.shape[2:])
        out = torch.zeros(n, most, *x.shape[1:], dtype=torch.float64, device=x.device)
        for i, (a, l) in enumerate(zip(off, lens)):
            out[i, :l] = x[a:a + l].double()
        return out

    def back(x):
        x = torch.cat([x[i, :l] for i, l in enumerate(lens)])
        return x.reshape(case["b"], case["t"], *x.shape[1:])

    q, k = (rows(s[x]).repeat_interleave(rep, 2) for x in ("q", "k"))
    v, beta = rows(s["v"]), rows(s["beta"])
    a = torch.exp(rows(s["g"])) if s["g"] is not None else torch.ones_like(beta)
    c = case["k"] ** -0.5

    def start():
        if s["h0"] is not None:
            return s["h0"].double().clone()
        return torch.zeros(n, h, case["k"], case["v"], dtype=torch.float64, device=DEV)

    st, o, miss = start(), torch.zeros_like(v), torch.zeros_like(v)
    for t in range(most):
        st.mul_(a[:, t, :, None, None])
        miss[:, t] = v[:, t] - (k[:, t, :, None, :] @ st)[..., 0, :]
        st.addcmul_(k[:, t, :, :, None], (beta[:, t, :, None] * miss[:, t])[:, :, None, :])
        if case["op"] != "train":
            o[:, t] = c * (q[:, t, :, None, :] @ st)[..., 0, :]
    if case["op"] != "train":
        return back(o), st
    do, u = rows(s["do"]) * c, beta[..., None] * miss
    ds = s["dht"].double().clone() if s["dht"] is not None else torch.zeros_like(st)
    after = (st * ds).sum((-1, -2))  # what a scale of the last state would change
    du, y = torch.zeros_like(v), torch.zeros_like(k)
    for t in range(most - 1, -1, -1):
        ds.addcmul_(q[:, t, :, :, None], do[:, t, :, None, :])
        du[:, t] = (k[:, t, :, None, :] @ ds)[..., 0, :]
        y[:, t] = (ds @ u[:, t, :, :, None])[..., 0]
        ds.addcmul_(k[:, t, :, :, None], (-beta[:, t, :, None] * du[:, t])[:, :, None, :])
        ds.mul_(a[:, t, :, None, None])
    st, dq, w = start(), torch.zeros_like(k), torch.zeros_like(k)
    for t in range(most):
        st.mul_(a[:, t, :, None, None])
        w[:, t] = (st @ (beta[:, t, :, None] * du[:, t])[..., None])[..., 0]
        st.addcmul_(k[:, t, :, :, None], u[:, t, :, None, :])
        dq[:, t] = (st @ do[:, t, :, :, None])[..., 0]
    share = lambda x: back(x.reshape(n, most, case["hk"], rep, case["k"]).sum(3))  # noqa: E731
    got = [share(dq), share(y - w), back(beta[..., None] * du), back((du * miss).sum(-1)), ds]
    if s["g"] is not None:  # a token's decay scales all that comes later of what came before it
        x = (q * dq).sum(-1) - (k * (y + w)).sum(-1)
        inside = torch.arange(most, device=DEV)[None, :] < torch.tensor(lens, device=DEV)[:, None]
        got.append(back(x.flip(1).cumsum(1).flip(1) + after[:, None] * inside[..., None]))
    return got


def _exact_rope(s):
    case = s["case"]
    train, rot = case["op"] == "rope_train", case["rot"]
    outs, got = [], {}
    for n in ("q", "k"):
        x = s[n].double().detach().requires_grad_(train)
        w = s[n + "_weight"]
        w = w.double().detach().requires_grad_(train) if w is not None else None
        with torch.enable_grad() if train else torch.no_grad():
            r = x
            if case["norm"] != "none":
                m = torch.sum(x ** 2, -1, keepdim=True)
                r = x / torch.sqrt((m / case["d"] if case["norm"] == "rms" else m) + EPS)
            r = r if w is None else r * w
            if rot:  # each pair is a complex number, turned by e^(i angle)
                first, second = (r[..., : rot // 2], r[..., rot // 2: rot]) if case["pairs"] == "half" else (
                    r[..., 0:rot:2], r[..., 1:rot:2])
                pos = s["pos"].reshape(-1, case["b"], case["t"]).double()
                freq, sec, ang = s["freq"].double(), _sections(case), []
                for i in range(rot // 2):
                    if case["spread"]:
                        ax = i % case["axes"] if i < case["axes"] * sec[i % case["axes"]] else 0
                    else:
                        ax = next(a for a in range(case["axes"]) if i < sum(sec[: a + 1]))
                    ang.append(pos[ax] * freq[i])
                ang = torch.stack(ang, -1)[:, :, None]
                z = torch.complex(first, second) * torch.polar(torch.ones_like(ang), ang)
                both = [z.real, z.imag]
                turned = torch.cat(both, -1) if case["pairs"] == "half" else torch.stack(both, -1).flatten(-2)
                r = torch.cat([turned, r[..., rot:]], -1)
        if not train:
            outs.append(r)
            continue
        leaves = [x] + ([w] if w is not None else [])
        d = torch.autograd.grad(r, leaves, s["d" + n].double())
        got["d" + n] = d[0]
        if w is not None:
            got["d%s_weight" % n] = d[1]
    return got if train else outs
