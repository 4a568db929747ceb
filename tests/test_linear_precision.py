"""How exact linear attention's results are, norm by norm, beside the worst cases that the other tests
bound: fp32 results (every output of fp32 calls; states, dg and dh0 of bf16 calls) carry fp32 rounding,
and bf16 rows the one rounding to bf16.

A term passes at most n roundings of 2^-24 (linear_ref.roundings), which are independent of each other,
so a result's error has a norm of about sqrt(n / 3) 2^-24 of the result's own: the limit is
sqrt(n) 2^-24, 1.1e-6 to 1.8e-6 here. dg is a sum whose terms cancel: its limit is that of its terms'
norm (dg_terms). bf16 rows may be off by that and by 2^-16 for each of the two
operands that enter them as two bf16 parts, beside the error of the best bf16 rows. The tests on the CPU
plant the losses that the worst cases let through in the 64-bit definition, and find them outside."""
import pytest
import torch

import linear_ref as ref
from kda_testlib import need_gpu
from test_gpu_linear import dev, f64, inputs64, make

BF16, FP32 = torch.bfloat16, torch.float32
SHAPES = [
    # B, T, H, Hk, K, V, lens
    (1, 60, 2, 2, 64, 64, None),
    (2, 150, 2, 1, 64, 64, None),
    (2, 65, 4, 2, 40, 200, None),
    (1, 130, 2, 1, 256, 128, None),
    (1, 700, 2, 2, 128, 64, [300, 0, 400]),
    (1, 4999, 2, 2, 64, 64, None),  # in segments
]
_id = lambda c: "b%dt%dh%d-%dk%dv%d" % c[:6]  # noqa: E731


def limit(K, V, T):
    return ref.roundings(K, V, T) ** 0.5 * ref.ULP32


def off(got, want):
    return ((f64(got) - want).norm() / want.norm()).item()


def rows_limit(want, K, V, T):
    """Of bf16 rows: the best that bf16 can hold, and what two parts leave out."""
    return off(want.to(BF16), want) + 2 * 2.0 ** -16 + limit(K, V, T)


def dg_terms(args, do, dht, cu=None, stretch=256):
    """The 2-norm of the terms that come together in each dg, [B, T, H]: from <h, dh> at one end of a
    stretch of tokens and the products of q.dq and k.dk between it and t, on the side where that is less."""
    q, k, v, g, h0 = args
    B, T, Hk, K = q.shape
    H = v.shape[2]
    q, k = (x.repeat_interleave(H // Hk, 2) for x in (q, k))
    dq, dk = ref.attn_grads(q, k, v, g, h0, do, dht, cu=cu)[:2]
    flat = lambda x: x.reshape(B * T, *x.shape[2:])  # noqa: E731
    dots = flat(((q * dq) ** 2).sum(-1) + ((k * dk) ** 2).sum(-1))
    q, k, v, a, do = flat(q), flat(k), flat(v), flat(g).exp()[..., None, None], flat(do) * K ** -0.5
    out = torch.zeros(B * T, H, dtype=torch.float64)
    for n, (lo, hi) in enumerate(ref.slots_of(B, T, cu)):
        cuts = list(range(lo, hi, stretch)) + [hi]
        S, G, at, ends = h0[n], dht[n], {lo: h0[n]}, {}
        for t in range(lo, hi):
            S = a[t] * S + k[t][:, :, None] * v[t][:, None, :]
            if t + 1 in cuts:
                at[t + 1] = S
        for t in range(hi, lo - 1, -1):
            if t in at:
                ends[t] = ((at[t] * G) ** 2).sum((-1, -2))
            if t > lo:
                G = a[t - 1] * (G + q[t - 1][:, :, None] * do[t - 1][:, None, :])
        for x, y in zip(cuts, cuts[1:]):
            back = ends[y] + dots[x:y].flip(0).cumsum(0).flip(0)
            fore = ends[x] + dots[x:y].cumsum(0) - dots[x:y]
            out[x:y] = torch.minimum(back, fore)
    return out.sqrt().reshape(B, T, H)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=_id)
def test_errors(shape, dtype):
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_linear_attn, chunk_linear_attn_bwd

    B, T, H, Hk, K, V, lens = shape
    d = make(B, T, H, Hk, K, V, dtype, "token", lens, seed=60)
    g, args, do, dht = dev(d), inputs64(d), f64(d["do"]), f64(d["dht"])
    o, ht = chunk_linear_attn(g["q"], g["k"], g["v"], g["g"], g["h0"], cu_seqlens=g["cu"], output_final_state=True)
    got = chunk_linear_attn_bwd(g["q"], g["k"], g["v"], g["g"], g["do"], g["h0"], dht=g["dht"], cu_seqlens=g["cu"])
    names = ("o", "ht", "dq", "dk", "dv", "dg", "dh0")
    want = ref.attn(*args, cu=d["cu"]) + tuple(ref.attn_grads(*args, do, dht, cu=d["cu"]))
    for n, w in zip(names, want):
        x = dict(got, o=o, ht=ht)[n]
        most = limit(K, V, T) if x.dtype == FP32 else rows_limit(w, K, V, T)
        if n == "dg":
            most *= (dg_terms(args, do, dht, d["cu"]).norm() / w.norm()).item()
        assert off(x, w) <= most, (n, off(x, w), most)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T", [200, 256, 257, 290, 700])
def test_a_large_final_gradient_stays_at_the_end(T, dtype):
    """Decays of e^-1 and a final state's gradient of 1e4: 60 tokens before the end nothing is left of it,
    and dg there is as exact as without it. (Carried over them, its rounding alone would be 1e-3.)"""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_linear_attn_bwd

    d = make(1, T, 2, 2, 64, 64, dtype, "token", seed=62)
    d["g"], d["dht"] = torch.full_like(d["g"], -1.0), 1e4 * d["dht"]
    g, args, do, dht = dev(d), inputs64(d), f64(d["do"]), f64(d["dht"])
    got = chunk_linear_attn_bwd(g["q"], g["k"], g["v"], g["g"], g["do"], g["h0"], dht=g["dht"])["dg"]
    want, size = ref.attn_grads(*args, do, dht)[3], dg_terms(args, do, dht)
    early = f64(got)[:, :T - 60] - want[:, :T - 60]
    most = limit(64, 64, T) * size[:, :T - 60].norm()
    assert size[:, :T - 60].max() < 1e3 and early.norm() <= most, (early.norm().item(), most.item())
    late = f64(got)[:, T - 60:] - want[:, T - 60:]
    assert late.norm() <= limit(64, 64, T) * size[:, T - 60:].norm()


@pytest.mark.gpu
def test_recurrence_errors():
    need_gpu()
    from gated_delta_rule_gate_amd import recurrent_linear_attn

    d = make(3, 70, 2, 1, 64, 64, FP32, "token", seed=61)
    g, want = dev(d), ref.attn(*inputs64(d))
    for x, w in zip(recurrent_linear_attn(g["q"], g["k"], g["v"], g["g"], g["h0"], output_final_state=True), want):
        assert off(x, w) <= limit(64, 64, 70), (off(x, w), limit(64, 64, 70))


def parts(x, n):
    """x as a sum of n bf16 parts."""
    rest, s = x.float(), torch.zeros_like(x)
    for _ in range(n):
        p = rest.to(BF16).float()
        rest, s = rest - p, s + p.double()
    return s


@pytest.mark.parametrize("shape", SHAPES[:3], ids=_id)
def test_two_parts_of_an_input_are_seen(shape):
    """fp32 inputs taken as two bf16 parts in place of three: outside the limit, one input alone."""
    B, T, H, Hk, K, V, _ = shape
    d = make(B, T, H, Hk, K, V, FP32, "token", seed=60)
    args, do, dht = inputs64(d), f64(d["do"]), f64(d["dht"])
    want = ref.attn(*args) + tuple(ref.attn_grads(*args, do, dht))
    assert off(parts(args[0], 3), args[0]) < limit(K, V, T) / 4
    reach = {0: (0, 3, 4, 6), 1: (0, 1, 2, 4), 2: (0, 1, 2, 3)}  # of q, k, v among o, ht, dq, dk, dv, dg, dh0
    for i, outs in reach.items():
        a = list(args)
        a[i] = parts(a[i], 2)
        lost = ref.attn(*a) + tuple(ref.attn_grads(*a, do, dht))
        for j in outs:
            assert off(lost[j], want[j]) > 1.25 * limit(K, V, T), (i, j)


def _chunk(d):
    """The chunked form of a batch of one chunk without an initial state: decays, scores, operands by head."""
    q, k, v, g, _ = inputs64(d)
    q, k, v, b = q[0].transpose(0, 1), k[0].transpose(0, 1), v[0].transpose(0, 1), g[0].cumsum(0).transpose(0, 1)
    return q, k, v, b, (q @ k.mT) * torch.exp(b[:, :, None] - b[:, None, :]).tril() * q.shape[-1] ** -0.5


def test_two_parts_of_the_decayed_rows_are_seen():
    """The rows of the state update, decayed, as two bf16 parts: outside the limit of a bf16 call's state."""
    d = make(1, 60, 2, 2, 64, 64, BF16, "token", states=False, seed=60)
    _, k, v, b, _ = _chunk(d)
    w = torch.exp(b[:, -1:] - b)[..., None] * v
    want = ref.attn(*inputs64(d))[1][0]
    assert off(k.mT @ w, want) < 1e-12
    assert off(k.mT @ parts(w, 3), want) < limit(64, 64, 60) / 4
    assert off(k.mT @ parts(w, 2), want) > 1.25 * limit(64, 64, 60)


def test_one_part_of_the_scores_is_seen():
    """Scores as one bf16 part: outside the limit of bf16 rows."""
    d = make(1, 60, 2, 2, 64, 64, BF16, "token", states=False, seed=60)
    _, _, v, _, s = _chunk(d)
    want = ref.attn(*inputs64(d))[0][0].transpose(0, 1)
    most = rows_limit(want, 64, 64, 60)
    assert off((parts(s, 2) @ v).to(BF16), want) < most
    assert off((parts(s, 1) @ v).to(BF16), want) > 1.25 * most
