"""Cases, plain forms and calls of the linear attention and block norm operators.

Linear attention with one decay per head (K x V state S, g <= 0 natural-log decay):

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,        o_t = scale S_t^T q_t

as a chunked forward over prompts ("prefill"), its gradient ("train"), and the recurrence over a
few tokens with the state updated in place ("decode"). The block norm is what surrounds such a
layer: a norm of its output rows with weight and gate, the residual branch with its scale, and
the norm before the next block, forward and backward.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
DEV = "cuda"
CHUNK = 64  # rows per chunk of the plain form


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def _attn(op, name, b, t, h, k, v, dtype="bf16", hk=0, decay="token", slots=0, states=True, cut=0):
    return dict(name=name, op=op, b=b, t=t, h=h, hk=hk or h, k=k, v=v, dtype=dtype, decay=decay, slots=slots,
                states=states, cut=cut)


def _norm(op, name, rows, d, dtype="bf16", res="none", gate="none", scale="none", nxt=False):
    return dict(name=name, op=op, rows=rows, d=d, dtype=dtype, res=res, gate=gate, scale=scale, nxt=nxt)


def listed():
    return [
        # a serving prefill that fills the card: four prompts of 4096 tokens, 64 heads of width 128, states carried
        _attn("prefill", "prefill b4 t4096 h64 d128", 4, 4096, 64, 128, 128),
        # one long document on few heads, with the fixed decay per head of retention layers
        _attn("prefill", "prefill b1 t32768 h16 d128", 1, 32768, 16, 128, 128, decay="head", states=False),
        # prompts of mixed lengths packed into one batch, two slots empty, q and k heads shared by pairs of value heads
        _attn("prefill", "prefill packed t15872 h32/16", 1, 15872, 32, 128, 128, hk=16, slots=10, cut=5),
        # a small model in full precision, a length that is no multiple of anything, unequal odd widths
        _attn("prefill", "prefill fp32 b2 t1000 h8 k72v40", 2, 1000, 8, 72, 40, dtype="fp32"),
        # a training step's gradient at the sizes of a mid-sized model
        _attn("train", "train b4 t2048 h32 d128", 4, 2048, 32, 128, 128, states=False),
        # a packed training batch with shared q/k heads, carried states and unequal widths
        _attn("train", "train packed t4999 h16/8 k64v128", 1, 4999, 16, 64, 128, hk=8, slots=7, cut=9),
        # a full decode batch: 256 sequences, one token each
        _attn("decode", "decode 256x1 h64 d128", 256, 1, 64, 128, 128),
        # one user, one token: the latency of a single step
        _attn("decode", "decode 1x1 h16 d128", 1, 1, 16, 128, 128),
        # the per-head output norm with its sigmoid gate, over the first case's outputs
        _norm("norm", "norm 1048576x128 sigmoid gate", 1048576, 128, gate="sigmoid"),
        # residual stream in fp32: norm after the block, residual, norm before the next block; decode-sized batch
        _norm("norm", "norm 77x2304 residual, next", 77, 2304, res="fp32", nxt=True),
        # the gradient of the per-head output norm with a SiLU gate
        _norm("norm_train", "norm grad 262144x128 silu gate", 262144, 128, gate="silu"),
        # the gradient of a whole residual branch with a scale per channel and the next block's norm
        _norm("norm_train", "norm grad 8192x4096 residual", 8192, 4096, res="bf16", gate="sigmoid", scale="channel", nxt=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "train", "train", "decode", "norm", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("norm", "norm_train"):
        d = 8 * _log(rng, 1, 1024)
        res = rng.choice(["none", "same", "fp32"])
        return dict(op=op, rows=_log(rng, 1, max(2, min(1 << 20, (1 << 25) // d))), d=d, dtype=dtype,
                    res=dtype if res == "same" else res, gate=rng.choice(["none", "sigmoid", "silu"]),
                    scale=rng.choice(["none", "number", "channel"]), nxt=rng.random() < 0.5)
    hk = rng.choice([1, 2, 3, 4, 5, 8, 16])
    h = hk * rng.choice([1, 1, 1, 2, 3])
    k, v = (8 * rng.randint(1, 32) for _ in range(2))
    if rng.random() < 0.5:
        k = v = rng.choice([64, 128, 256])
    most = (1 << 30) // (3 if op == "train" else 1) // (4 if dtype == "fp32" else 1)  # of token-heads times K times V
    if op == "decode":
        b, t = _log(rng, 1, 256), rng.choice([1, 1, 1, 2, 4])
        b = max(1, min(b, most // (h * k * v)))
        return dict(op=op, b=b, t=t, h=h, hk=hk, k=k, v=v, dtype=dtype, decay=rng.choice(["head", "token"]), slots=0,
                    states=True, cut=0)
    tokens = max(64, min(16384, 8 * most // (h * k * v)))
    t = _log(rng, 1, tokens)
    packed = rng.random() < 0.4
    b = 1 if packed else max(1, min(rng.choice([1, 2, 3, 4]), tokens // t))
    return dict(op=op, b=b, t=t, h=h, hk=hk, k=k, v=v, dtype=dtype, decay=rng.choice(["head", "token"]),
                slots=rng.randint(1, 12) if packed else 0, states=rng.random() < 0.7, cut=rng.randrange(1 << 16))


def _offsets(case):
    """Offsets of a packed case: lengths cut at random places, so that some are short, some long and some empty."""
    rng = random.Random(case["cut"])
    cuts = sorted(rng.randint(0, case["t"]) for _ in range(case["slots"] - 1))
    if len(cuts) > 2:
        cuts[1] = cuts[0]  # an empty slot
    return [0] + cuts + [case["t"]]


def _slots(case):
    return case["slots"] or case["b"]


def work(case):
    if case["op"] in ("norm", "norm_train"):
        n, e = case["rows"] * case["d"], 2 if case["dtype"] == "bf16" else 4
        r = {"none": 0, "bf16": 2, "fp32": 4}[case["res"]]
        gate = e if case["gate"] != "none" else 0
        if case["op"] == "norm":  # x, gate, residual in; the sum and the next block's input out
            return {"bytes": n * (e + gate + r + (r or e) + (e if case["nxt"] else 0)), "flops": 12 * n}
        # x, gate, residual and the outputs' gradients in; the inputs' gradients out
        need_r = r if case["nxt"] else 0
        return {"bytes": n * (2 * e + 2 * gate + need_r + r + (r or e) + (e if case["nxt"] else 0)), "flops": 30 * n}
    e = 2 if case["dtype"] == "bf16" else 4
    rows, n = case["b"] * case["t"], _slots(case)
    kk, vv = rows * case["hk"] * case["k"] * e, rows * case["h"] * case["v"] * e
    state = n * case["h"] * case["k"] * case["v"] * 4
    g = rows * case["h"] * 4 if case["decay"] == "token" else case["h"] * 4
    steps = rows * case["h"] * case["k"] * case["v"]
    if case["op"] == "train":  # q, k, v, do and the states in; dq, dk, dv, dg and dh0 out
        return {"bytes": 4 * kk + 3 * vv + 2 * g + state * (3 if case["states"] else 1), "flops": 10 * steps}
    return {"bytes": 2 * kk + 2 * vv + g + state * (2 if case["states"] else 1), "flops": 4 * steps}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, dtype=torch.float32, mul=1.0):
        return (torch.randn(*shape, device=DEV, generator=gen) * mul).to(dtype)

    if case["op"] in ("norm", "norm_train"):
        rows, d = case["rows"], case["d"]
        rt = DTYPES.get(case["res"])
        s = dict(case=case, x=randn(rows, d, dtype=dt), weight=1 + randn(d, mul=0.1),
                 gate=randn(rows, d, dtype=dt) if case["gate"] != "none" else None,
                 residual=randn(rows, d, dtype=rt, mul=2.0) if rt else None,
                 scale={"none": None, "number": 0.5, "channel": 0.5 + randn(d, mul=0.1)}[case["scale"]],
                 next_weight=1 + randn(d, mul=0.1) if case["nxt"] else None)
        if case["op"] == "norm_train":
            s["dy"] = randn(rows, d, dtype=rt or dt)
            s["dz"] = randn(rows, d, dtype=dt) if case["nxt"] else None
        return s

    b, t, h, hk, k, v = (case[x] for x in ("b", "t", "h", "hk", "k", "v"))
    n = _slots(case)
    s = dict(case=case, q=randn(b, t, hk, k, dtype=dt), k=randn(b, t, hk, k, dtype=dt, mul=k ** -0.5),
             v=randn(b, t, h, v, dtype=dt))
    if case["decay"] == "head":  # fixed decays, memories of 32 to 8192 tokens spread over the heads
        s["g"] = torch.log1p(-torch.exp2(-5 - 8 * torch.rand(h, device=DEV, generator=gen)))
    else:  # a rate per head times a softplus of each token's input
        rate = torch.exp(randn(h) - 1.5)
        s["g"] = -rate * torch.log1p(torch.exp(randn(b, t, h)))
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


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------
def _rows(s, x, heads):
    """[B, T, heads, ...] -> fp32 [slots, H, chunks, CHUNK, width]: one row of chunks per sequence and head."""
    case = s["case"]
    if case["slots"]:
        x = torch.where(s["inside"][:, :, None, None], x[0][s["from"]], torch.zeros((), dtype=x.dtype, device=x.device))
    x = x.to(torch.float64 if x.dtype == torch.float64 else torch.float32).transpose(1, 2)
    if heads != case["h"]:
        x = x.repeat_interleave(case["h"] // heads, dim=1)
    n, h, t, w = x.shape
    c = min(CHUNK, max(t, 1))
    nc = max(1, -(-t // c))
    x = torch.nn.functional.pad(x, (0, 0, 0, nc * c - t))
    return x.reshape(n, h, nc, c, w).contiguous()


def _tokens(s, x, heads, dtype):
    """The way back: [slots, H, chunks, CHUNK, width] -> [B, T, heads, width], summed over the heads that share one."""
    case = s["case"]
    n, h, nc, c, w = x.shape
    x = x.reshape(n, h, nc * c, w)
    if heads != h:
        x = x.reshape(n, heads, h // heads, nc * c, w).sum(2)
    x = x.transpose(1, 2)
    x = x[s["slot"], s["place"]][None] if case["slots"] else x[:, : case["t"]]
    return x.to(dtype).contiguous()


def _decays(s):
    """Sums of the decays, in 64 bits: within each chunk up to and with every token, and over whole chunks."""
    case = s["case"]
    g = s["g"]
    if case["decay"] == "head":
        g = g[None, None, :].expand(case["b"], case["t"], case["h"])
    b = _rows(s, g.double()[..., None].contiguous(), case["h"])[..., 0].cumsum(-1)  # [n, h, nc, c]
    over = torch.cat([torch.zeros_like(b[..., :1, -1]), b[..., -1].cumsum(-1)], -1)  # [n, h, nc + 1]
    return b, over


def _tri(m, keep):
    return torch.where(keep, m, torch.zeros((), dtype=m.dtype, device=m.device))


def _chunk_states(kv, over, first):
    """The state before every chunk and after the last: sums of the chunks' own parts kv, decayed."""
    n, h, nc, k, v = kv.shape
    if nc == 1:
        last = kv if first is None else torch.exp(over[..., 1:]).float()[..., None, None] * first[:, :, None] + kv
        return torch.cat([torch.zeros_like(kv) if first is None else first[:, :, None], last], 2)
    d = over[..., :, None] - over[..., None, 1:]  # [n, h, nc + 1, nc]
    row, col = torch.arange(nc + 1, device=kv.device)[:, None], torch.arange(nc, device=kv.device)[None, :]
    d = _tri(torch.exp(torch.clamp(d, max=0.0)), row > col).float()
    st = (d @ kv.reshape(n, h, nc, k * v)).reshape(n, h, nc + 1, k, v)
    if first is not None:
        st = st + torch.exp(over).float()[..., None, None] * first[:, :, None]
    return st


def _scores(b):
    """Decay from token s to token r of each chunk, zero for later s."""
    c = b.shape[-1]
    i = torch.arange(c, device=b.device)
    keep = i[:, None] >= i[None, :]
    return _tri(torch.exp(torch.clamp(b[..., :, None] - b[..., None, :], max=0.0)), keep).float()


def _scale(case):
    return case["k"] ** -0.5


def _plain_attn(s):
    case = s["case"]
    q, k, v = _rows(s, s["q"], case["hk"]), _rows(s, s["k"], case["hk"]), _rows(s, s["v"], case["h"])
    b, over = _decays(s)
    tail = torch.exp(b[..., -1:] - b).float()[..., None]
    st = _chunk_states((k * tail).transpose(-1, -2).contiguous() @ v, over, s["h0"])
    p = (q @ k.transpose(-1, -2).contiguous()) * _scores(b)
    o = p @ v + torch.exp(b).float()[..., None] * (q @ st[:, :, :-1])
    return _tokens(s, o * _scale(case), case["h"], s["v"].dtype), st[:, :, -1].contiguous()


def _plain_attn_grad(s):
    case = s["case"]
    q, k, v = _rows(s, s["q"], case["hk"]), _rows(s, s["k"], case["hk"]), _rows(s, s["v"], case["h"])
    do = _rows(s, s["do"], case["h"]) * _scale(case)
    b, over = _decays(s)
    head, tail = torch.exp(b).float()[..., None], torch.exp(b[..., -1:] - b).float()[..., None]
    whole = torch.exp(b[..., -1]).float()
    t = lambda x: x.transpose(-1, -2).contiguous()  # noqa: E731
    st = _chunk_states(t(k * tail) @ v, over, s["h0"])
    # gradients of the states after each chunk: the same sum, run from the end
    back = (over[..., -1:] - over).flip(-1)
    dst = _chunk_states((t(q * head) @ do).flip(2), back, s["dht"]).flip(2)
    h, dh = st[:, :, :-1], dst[:, :, 1:]
    w = _scores(b)
    p, dp = (q @ t(k)) * w, (do @ t(v)) * w
    dq_far, dk_far = head * (do @ t(h)), tail * (v @ t(dh))
    dq, dk = dp @ k + dq_far, t(dp) @ q + dk_far
    dv = t(p) @ do + tail * (k @ dh)
    # a decay scales every pair that it lies between: pairs inside the chunk, those with a state, and state with state
    m = (p * (do @ t(v))).double()
    e, f = (q.double() * dq_far.double()).sum(-1), (k.double() * dk_far.double()).sum(-1)
    x = m.sum(-1) - m.sum(-2) + e - f
    dg = x.flip(-1).cumsum(-1).flip(-1) + f.sum(-1, keepdim=True) + (
        whole.double() * (h.double() * dh.double()).sum((-1, -2)))[..., None]
    dg = _tokens(s, dg[..., None], case["h"], torch.float64)[..., 0]
    dg = dg.sum((0, 1)).float() if case["decay"] == "head" else dg.float()
    kt = s["q"].dtype
    return (_tokens(s, dq, case["hk"], kt), _tokens(s, dk, case["hk"], kt), _tokens(s, dv, case["h"], kt), dg,
            dst[:, :, 0].contiguous())


def _act(kind, g):
    sig = 1 / (1 + torch.exp(-g))
    return sig if kind == "sigmoid" else g * sig


def _act_grad(kind, g):
    sig = 1 / (1 + torch.exp(-g))
    return sig * (1 - sig) if kind == "sigmoid" else sig * (1 + g * (1 - sig))


EPS = 1e-6


def _norm_parts(s, f):
    """The operator's intermediates with every tensor taken by f."""
    x, case = f(s["x"]), s["case"]
    rho = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xn = x * rho
    n = xn * f(s["weight"])
    gate = f(s["gate"]) if s["gate"] is not None else None
    y = n * _act(case["gate"], gate) if gate is not None else n
    c = 1.0 if s["scale"] is None else s["scale"] if isinstance(s["scale"], float) else f(s["scale"])
    r = y * c + (f(s["residual"]) if s["residual"] is not None else 0)
    rho2 = torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
    return x, rho, xn, n, gate, y, c, r, rho2


def _norm_out(s, f):
    r, rho2 = _norm_parts(s, f)[-2:]
    outs = [r]
    if s["next_weight"] is not None:
        outs.append(r * rho2 * f(s["next_weight"]))
    return outs


def _plain_norm(s):
    outs = _norm_out(s, torch.Tensor.float)
    rt = s["residual"].dtype if s["residual"] is not None else s["x"].dtype
    return [outs[0].to(rt)] + [z.to(s["x"].dtype) for z in outs[1:]]


def _plain_norm_grad(s):
    f = torch.Tensor.float
    x, rho, xn, n, gate, y, c, r, rho2 = _norm_parts(s, f)
    total = lambda t: t.double().sum(0).float()  # noqa: E731
    got = {}
    dr = f(s["dy"])
    if s["next_weight"] is not None:
        dz, rn = f(s["dz"]), r * rho2
        got["dnext_weight"] = total(dz * rn)
        dz = dz * f(s["next_weight"])
        dr = dr + rho2 * (dz - rn * (dz * rn).mean(-1, keepdim=True))
    if s["residual"] is not None:
        got["dresidual"] = dr.to(s["residual"].dtype)
    if isinstance(s["scale"], torch.Tensor):
        got["dscale"] = total(dr * y)
    dn = dr * c
    if gate is not None:
        got["dgate"] = (dn * n * _act_grad(s["case"]["gate"], gate)).to(s["gate"].dtype)
        dn = dn * _act(s["case"]["gate"], gate)
    got["dweight"] = total(dn * xn)
    dn = dn * f(s["weight"])
    got["dx"] = (rho * (dn - xn * (dn * xn).mean(-1, keepdim=True))).to(s["x"].dtype)
    return got


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def run(s):
    case = s["case"]
    if case["op"] == "prefill":
        if own:
            from gated_delta_rule_gate_amd import chunk_linear_attn

            return chunk_linear_attn(s["q"], s["k"], s["v"], s["g"], s["h0"], cu_seqlens=s["cu"], output_final_state=True)
        return _plain_attn(s)
    if case["op"] == "decode":  # the state is updated in place
        if own:
            from gated_delta_rule_gate_amd import recurrent_linear_attn

            return recurrent_linear_attn(s["q"], s["k"], s["v"], s["g"], s["h0"], final_state=s["h0"])
        o, ht = _plain_attn(s)
        s["h0"].copy_(ht)
        return o, s["h0"]
    if case["op"] == "train":
        if own:
            from gated_delta_rule_gate_amd import chunk_linear_attn_bwd

            got = chunk_linear_attn_bwd(s["q"], s["k"], s["v"], s["g"], s["do"], s["h0"], dht=s["dht"], cu_seqlens=s["cu"])
            return tuple(got[x] for x in ("dq", "dk", "dv", "dg", "dh0"))
        return _plain_attn_grad(s)
    options = dict(gate=s["gate"], residual=s["residual"], scale=s["scale"], next_weight=s["next_weight"], eps=EPS)
    if s["gate"] is not None:
        options["gate_act"] = case["gate"]
    if case["op"] == "norm":
        if own:
            from gated_delta_rule_gate_amd import block_norm

            got = block_norm(s["x"], s["weight"], **options)
            return list(got) if isinstance(got, tuple) else [got]
        return _plain_norm(s)
    if own:
        from gated_delta_rule_gate_amd import block_norm_bwd

        got = block_norm_bwd(s["x"], s["dy"], s["weight"], dz=s["dz"], **options)
        return {x: t for x, t in got.items() if t is not None}
    return _plain_norm_grad(s)


# ---------------------------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm_train"):
        return _exact_norm(s)
    # token by token, every sequence in a row of its own, rows past a sequence's end without effect
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

    def back(x, dtype=None):
        x = torch.cat([x[i, :l] for i, l in enumerate(lens)])
        return x.reshape(case["b"], case["t"], *x.shape[1:])

    q, k = (rows(s[x]).repeat_interleave(rep, 2) for x in ("q", "k"))
    v = rows(s["v"])
    g = s["g"].double()
    g = rows(g if g.dim() == 3 else g.expand(case["b"], case["t"], h))
    a = torch.exp(g)
    st = s["h0"].double().clone() if s["h0"] is not None else torch.zeros(n, h, case["k"], case["v"], dtype=torch.float64, device=DEV)
    c = case["k"] ** -0.5
    train = case["op"] == "train"
    do = rows(s["do"]) * c if train else None
    out = torch.zeros_like(q if train else v)
    for t in range(most):
        st.mul_(a[:, t, :, None, None]).addcmul_(k[:, t, :, :, None], v[:, t, :, None, :])
        if train:  # dq_t = S_t do_t
            out[:, t] = (st @ do[:, t, :, :, None])[..., 0]
        else:
            out[:, t] = c * (q[:, t, :, None, :] @ st)[..., 0, :]
    if not train:
        return back(out), st
    dq, dk, dv = out, torch.zeros_like(k), torch.zeros_like(v)
    ds = s["dht"].double().clone() if s["dht"] is not None else torch.zeros_like(st)
    after = (st * ds).sum((-1, -2))  # what a scale of the last state would change
    for t in range(most - 1, -1, -1):
        ds.addcmul_(q[:, t, :, :, None], do[:, t, :, None, :])
        dk[:, t] = (ds @ v[:, t, :, :, None])[..., 0]
        dv[:, t] = (k[:, t, :, None, :] @ ds)[..., 0, :]
        ds.mul_(a[:, t, :, None, None])
    # a token's decay scales all that comes later of what came before it
    x = (q * dq).sum(-1) - (k * dk).sum(-1)
    inside = torch.arange(most, device=DEV)[None, :] < torch.tensor(lens, device=DEV)[:, None]
    dg = back(x.flip(1).cumsum(1).flip(1) + after[:, None] * inside[..., None])
    if case["decay"] == "head":
        dg = dg.sum((0, 1))
    share = lambda x: back(x.reshape(n, most, case["hk"], rep, case["k"]).sum(3))  # noqa: E731
    return share(dq), share(dk), back(dv), dg, ds


def _exact_norm(s):
    case = s["case"]
    names = ["x", "weight"] + [x for x in ("gate", "residual", "scale", "next_weight") if isinstance(s[x], torch.Tensor)]
    train = case["op"] == "norm_train"
    t = {x: s[x].double().detach().requires_grad_(train) for x in names}
    with torch.enable_grad() if train else torch.no_grad():
        y = t["x"] / torch.sqrt(torch.sum(t["x"] ** 2, -1, keepdim=True) / case["d"] + EPS) * t["weight"]
        if "gate" in t:
            y = y * torch.sigmoid(t["gate"]) * (t["gate"] if case["gate"] == "silu" else 1.0)
        y = y * (t["scale"] if "scale" in t else s["scale"] or 1.0)
        if "residual" in t:
            y = y + t["residual"]
        outs = [y]
        if "next_weight" in t:
            outs.append(y / torch.sqrt(torch.sum(y ** 2, -1, keepdim=True) / case["d"] + EPS) * t["next_weight"])
    if not train:
        return outs
    grads = [s["dy"].double()] + ([s["dz"].double()] if case["nxt"] else [])
    got = torch.autograd.grad(outs, [t[x] for x in names], grads)
    return {"d" + x: g for x, g in zip(names, got)}
