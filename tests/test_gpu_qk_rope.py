"""The norm of query and key rows with rotation by position on the GPU against 64 bits: types, widths, partial
rotation, both pair layouts, one to four position axes, parts of a fused projection, far positions, gradients.

Tolerances count roundings: of a row of D values, D + 16 fp32 ones for its norm and dots, 8 for weights, angles
(the sine and cosine are off by two ulp and an angle in turns by 2^-25 of a turn: 2 pi 2^-25 < 4 2^-24) and
products, relative to the row's largest terms; a result adds one rounding to its type."""
import numpy as np
import pytest
import torch

import delta_ref as ref
from kda_testlib import need_gpu

BF16, FP32 = torch.bfloat16, torch.float32
pytestmark = pytest.mark.gpu

CASES = [
    # B, T, H, Hk, D, rot, norm, pairs, sections, spread, fused
    (1, 1, 1, 1, 8, 8, "rms", "half", None, False, False),
    (2, 3, 2, 1, 64, 64, "rms", "half", None, False, True),
    (1, 5, 3, 3, 72, 72, "rms", "half", (18, 18), False, False),
    (2, 7, 4, 2, 128, 128, "rms", "half", (24, 20, 20), True, True),
    (1, 9, 4, 2, 128, 128, "l2", "adjacent", (16, 24, 24), False, False),
    (3, 4, 7, 1, 80, 40, "rms", "adjacent", None, False, False),
    (1, 33, 5, 2, 256, 64, "rms", "half", None, False, True),
    (1, 17, 2, 2, 512, 512, "none", "half", (64, 64, 64, 64), True, False),
    (1, 11, 2, 1, 504, 504, "rms", "adjacent", None, False, False),
    (1, 700, 12, 3, 96, 48, "l2", "half", (8, 8, 8), True, False),
    (2, 650, 1, 1, 128, 0, "l2", "half", None, False, False),
    (1, 40, 70, 5, 16, 8, "rms", "half", (4,), False, False),
    (1, 3000, 9, 2, 64, 56, "none", "adjacent", (0, 14, 14), False, False),
    (1, 130, 48, 16, 40, 24, "rms", "half", (12, 0), True, True),
]


def _id(c):
    return "b%dt%dh%d-%dd%dr%d-%s-%s" % c[:8] + ("" if c[8] is None else "-%daxes" % len(c[8])) + ("-spread" if c[9] else "")


def make(case, dtype, seed=0, far=1 << 17):
    B, T, H, Hk, D, rot, norm, pairs, sections, spread, fused = case
    r = np.random.Generator(np.random.PCG64(seed + 31 * T + D))
    f = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32))  # noqa: E731
    if fused:
        qkv = f(B, T, (H + 2 * Hk) * D).to(dtype).cuda()
        q, k = qkv[..., :H * D].unflatten(-1, (H, D)), qkv[..., H * D:(H + Hk) * D].unflatten(-1, (Hk, D))
    else:
        q, k = f(B, T, H, D).to(dtype).cuda(), f(B, T, Hk, D).to(dtype).cuda()
    d = dict(q=q, k=k, wq=1 + 0.2 * f(D), wk=1 + 0.2 * f(D), dq=f(B, T, H, D).to(dtype), dk=f(B, T, Hk, D).to(dtype))
    d["pos"] = d["freq"] = None
    if rot:
        shape = (B, T) if sections is None else (len(sections), B, T)
        d["pos"] = torch.from_numpy(r.integers(-far, far, shape).astype(np.int32))
        d["freq"] = (1e4 ** (-torch.arange(0, rot, 2) / rot)).float()
    g = {x: t if t is None or t.is_cuda else t.cuda() for x, t in d.items()}
    kw = dict(positions=g["pos"], inv_freq=g["freq"], sections=sections, spread=spread, pairs=pairs, norm=norm)
    return g, kw


def want_of(g, kw, x, w, eps=1e-6):
    half = 0 if kw["inv_freq"] is None else kw["inv_freq"].numel()
    pos = None if kw["positions"] is None else kw["positions"].cpu().reshape(-1, *x.shape[:2])
    freq = None if kw["inv_freq"] is None else kw["inv_freq"].cpu()
    return ref.qk_rope(x, w, kw["norm"], eps, pos, freq, ref.axes_of(half, kw["sections"], kw["spread"]), kw["pairs"])


def within(got, want, size, dtype, n, what):
    got = got.detach().cpu().double()
    assert got.shape == want.shape and torch.isfinite(got).all(), what
    off, tol = (got - want).abs(), ref.HALF[dtype] * want.abs() + n * ref.ULP32 * size
    worst = (off / tol.clamp_min(1e-300)).max().item()
    assert (off <= tol).all(), "%s: off by %.3g times the tolerance" % (what, worst)


def f64(x):
    return x.detach().cpu().double()


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("case", CASES, ids=_id)
def test_forward(case, dtype):
    need_gpu()
    from gated_delta_rule_gate_amd import qk_norm_rope

    g, kw = make(case, dtype)
    D = case[4]
    for weights in ((g["wq"], g["wk"]), (None, g["wk"])):
        got = qk_norm_rope(g["q"], g["k"], *weights, **kw)
        for name, y, x, w in zip(("q", "k"), got, (g["q"], g["k"]), weights):
            want = want_of(g, kw, f64(x), None if w is None else f64(w))
            big = want.abs().amax(-1, keepdim=True)  # a turned pair's terms
            assert y.is_contiguous() and y.dtype == dtype
            within(y, want, big * 2, dtype, D + 24, name)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("case", CASES, ids=_id)
def test_backward(case, dtype):
    need_gpu()
    from gated_delta_rule_gate_amd import qk_norm_rope_bwd

    g, kw = make(case, dtype, seed=1)
    B, T, H, Hk, D = case[:5]
    got = qk_norm_rope_bwd(g["q"], g["k"], g["dq"], g["dk"], g["wq"], g["wk"], **kw)
    for name, x, w, dy in (("q", g["q"], g["wq"], g["dq"]), ("k", g["k"], g["wk"], g["dk"])):
        x64, w64 = f64(x).requires_grad_(True), f64(w).requires_grad_(True)
        y = want_of(g, kw, x64, w64)
        dx, dw = torch.autograd.grad((y * f64(dy)).sum(), (x64, w64))
        # |dx| <= 2 |rho w dy|: the terms of a row, by its largest channels; a dot's terms add up over D
        X = f64(x)
        ss = (X * X).sum(-1, keepdim=True) / (D if kw["norm"] == "rms" else 1)
        rho = 1 / torch.sqrt(ss + 1e-6) if kw["norm"] != "none" else torch.ones_like(ss)
        top = rho * f64(dy).abs().amax(-1, keepdim=True) * 2 * f64(w).abs().max()
        xn = X * rho
        dot = (xn.abs().sum(-1, keepdim=True) / (D if kw["norm"] == "rms" else 1)) * top
        size = top + xn.abs() * dot if kw["norm"] != "none" else top
        within(got["d" + name], dx, size, dtype, D + 32, "d" + name)
        rows = (2 * f64(dy).abs().amax(-1, keepdim=True) * xn.abs()).flatten(0, 2).sum(0)
        # a lane's rows one after another, then lanes, waves and workgroups
        within(got["d%s_weight" % name], dw, rows, FP32, D + 32 + B * T * x.shape[2], "weight of " + name)


def test_gradient_against_differences():
    """y is linear in the weight: L(w + d) - L(w - d) = 2 <dw, d>; in x along a direction d by central
    differences of h, whose own error of the 64-bit definition is taken off."""
    need_gpu()
    from gated_delta_rule_gate_amd import qk_norm_rope, qk_norm_rope_bwd

    g, kw = make(CASES[3], FP32, seed=3)
    g["q"], g["k"] = g["q"].contiguous(), g["k"].contiguous()
    got = qk_norm_rope_bwd(g["q"], g["k"], g["dq"], g["dk"], g["wq"], g["wk"], **kw)

    def loss(q, w):
        y, _ = qk_norm_rope(q, g["k"], w, g["wk"], **kw)
        return (y.double() * g["dq"].double()).sum().item()

    def exact(q, w):
        return (want_of(g, kw, f64(q), f64(w)) * f64(g["dq"])).sum().item()

    size = (want_of(g, kw, f64(g["q"]), f64(g["wq"])).abs() * f64(g["dq"]).abs()).sum().item()
    noise = 2 * 160 * ref.ULP32 * size
    dw = torch.randn_like(g["wq"])
    along = (got["dq_weight"].double() * dw.double()).sum().item()
    assert abs((loss(g["q"], g["wq"] + dw) - loss(g["q"], g["wq"] - dw)) / 2 - along) <= 4 * noise
    h, dx = 1 / 64, torch.randn_like(g["q"])
    plus, minus = g["q"] + h * dx, g["q"] - h * dx
    mine, true = (loss(plus, g["wq"]) - loss(minus, g["wq"])) / (2 * h), (exact(plus, g["wq"]) - exact(minus, g["wq"])) / (2 * h)
    assert abs(mine - true) <= noise / h
    at = (got["dq"].double() * dx.double()).sum().item()
    assert abs(true - at) <= 0.02 * abs(at) + 0.02 * got["dq"].norm().item() * dx.norm().item() ** 0.5


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_far_positions(dtype):
    """Angles of positions up to 2^31 - 1 with a frequency of one: the turns are reduced in fp64, whose product
    is off by 2^-53 of 2^31 / 2 pi turns: 2^-25 of a turn."""
    need_gpu()
    from gated_delta_rule_gate_amd import qk_norm_rope

    case = (1, 64, 2, 2, 32, 32, "none", "half", None, False, False)
    g, kw = make(case, dtype)
    kw["positions"] = torch.arange(64, dtype=torch.int32).reshape(1, 64).cuda() * 33333331 + (2 ** 31 - 1 - 63 * 33333331)
    assert kw["positions"].max().item() == 2 ** 31 - 1
    got, _ = qk_norm_rope(g["q"], g["k"], **kw)
    x = f64(g["q"])
    # the oracle's own angle: exact products of integers and a power of two or of an fp32 frequency's 24 bits,
    # reduced by whole turns in 64 bits of mantissa
    ang = np.asarray(f64(kw["positions"])[0][:, None].numpy(), np.longdouble) * np.asarray(f64(kw["inv_freq"]).numpy(), np.longdouble)
    two_pi = np.longdouble("6.28318530717958647692528676655900577")
    turns = ang / two_pi
    ang = torch.from_numpy(((turns - np.rint(turns)) * two_pi).astype(np.float64))[None, :, None]
    a, b = x[..., :16], x[..., 16:]
    want = torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)
    size = (a.abs() + b.abs()).repeat(1, 1, 1, 2)
    within(got, want, size, dtype, 24, "far")


def test_outputs_in_place_and_in_a_projection():
    """The outputs over the inputs, contiguous and as parts of a fused projection whose values stay."""
    need_gpu()
    from gated_delta_rule_gate_amd import qk_norm_rope, qk_norm_rope_bwd

    for case in (CASES[3], CASES[4], CASES[6]):
        g, kw = make(case, BF16, seed=4)
        want = qk_norm_rope(g["q"], g["k"], g["wq"], g["wk"], **kw)
        base = g["q"]._base.clone() if g["q"]._base is not None else None
        back = qk_norm_rope_bwd(g["q"], g["k"], g["dq"], g["dk"], g["wq"], g["wk"], **kw)
        got = qk_norm_rope(g["q"], g["k"], g["wq"], g["wk"], q_out=g["q"], k_out=g["k"], **kw)
        assert got[0] is g["q"] and all(torch.equal(a, b) for a, b in zip(got, want))
        if base is not None:
            n = (case[2] + case[3]) * case[4]
            assert torch.equal(g["q"]._base[..., n:], base[..., n:])
        g2, kw = make(case, BF16, seed=4)  # gradients of the outputs as parts of a projection
        wide = torch.zeros(*g2["dq"].shape[:2], (case[2] + case[3]) * case[4], dtype=BF16, device="cuda")
        dq, dk = wide[..., :case[2] * case[4]].unflatten(-1, g2["dq"].shape[2:]), wide[..., case[2] * case[4]:].unflatten(-1, g2["dk"].shape[2:])
        dq.copy_(g2["dq"]), dk.copy_(g2["dk"])
        again = qk_norm_rope_bwd(g2["q"], g2["k"], dq, dk, g2["wq"], g2["wk"], **kw)
        assert all(torch.equal(back[x], again[x]) for x in back)


def test_rows_of_zeros_and_non_finite_rows():
    """A row of zeros stays zeros; a NaN or an infinity stays in its row, forward and backward (but for the weights)."""
    need_gpu()
    from gated_delta_rule_gate_amd import qk_norm_rope, qk_norm_rope_bwd

    g, kw = make(CASES[9], BF16, seed=5)
    g["q"][0, 3, 2] = 0
    y, yk = qk_norm_rope(g["q"], g["k"], g["wq"], g["wk"], **kw)
    assert (y[0, 3, 2] == 0).all()
    b = qk_norm_rope_bwd(g["q"], g["k"], g["dq"], g["dk"], g["wq"], g["wk"], **kw)
    q2 = g["q"].clone()
    q2[0, 5, 1, 7], q2[0, 6, 4, 90] = float("nan"), float("inf")
    y2, yk2 = qk_norm_rope(q2, g["k"], g["wq"], g["wk"], **kw)
    b2 = qk_norm_rope_bwd(q2, g["k"], g["dq"], g["dk"], g["wq"], g["wk"], **kw)
    for x, x2 in ((y, y2), (b["dq"], b2["dq"])):
        hit = ~torch.isfinite(x2).all(-1)
        assert hit[0, 5, 1] and hit[0, 6, 4] and hit.sum() == 2
        assert torch.equal(x[~hit], x2[~hit])
    assert torch.equal(yk, yk2) and torch.equal(b["dk"], b2["dk"]) and torch.equal(b["dk_weight"], b2["dk_weight"])


def test_no_tokens():
    need_gpu()
    from gated_delta_rule_gate_amd import qk_norm_rope, qk_norm_rope_bwd

    q, k, w = torch.empty(2, 0, 4, 64, device="cuda"), torch.empty(2, 0, 2, 64, device="cuda"), torch.ones(64, device="cuda")
    y, z = qk_norm_rope(q, k, w, w)
    assert y.shape == q.shape and z.shape == k.shape
    got = qk_norm_rope_bwd(q, k, q, k, w, w)
    assert (got["dq_weight"] == 0).all() and (got["dk_weight"] == 0).all()


def test_l2_rows_feed_the_delta_rule():
    """Norm and rotation, the delta rule, and back: the operators as a layer calls them, against one 64-bit graph."""
    need_gpu()
    from gated_delta_rule_gate_amd import (block_norm, block_norm_bwd, chunk_gated_delta, chunk_gated_delta_bwd,
                                           qk_norm_rope, qk_norm_rope_bwd)

    B, T, H, Hk, D = 1, 100, 4, 2, 64
    gen = np.random.Generator(np.random.PCG64(8))
    f = lambda *s: torch.from_numpy(gen.standard_normal(s).astype(np.float32))  # noqa: E731
    qkv = f(B, T, (2 * Hk + H) * D)
    pos, freq = torch.arange(T, dtype=torch.int32).reshape(1, T), (1e4 ** (-torch.arange(0, 32, 2) / 32)).float()
    g, beta, w, z, dy = -f(B, T, H).abs() * 0.2, torch.sigmoid(f(B, T, H)), 1 + 0.1 * f(D), f(B, T, H, D), f(B, T, H, D)
    d = [x.cuda() for x in (qkv, pos, freq, g, beta, w, z, dy)]

    def parts(x):
        return [x[..., a * D:b * D].unflatten(-1, (b - a, D)) for a, b in ((0, Hk), (Hk, 2 * Hk), (2 * Hk, 2 * Hk + H))]

    q, k, v = parts(d[0])
    v = v.contiguous()
    kw = dict(positions=d[1], inv_freq=d[2], norm="l2")
    qn, kn = qk_norm_rope(q, k, **kw)
    o, _ = chunk_gated_delta(qn, kn, v, d[3], d[4])
    y = block_norm(o, d[5], gate=d[6], gate_act="silu")
    b = block_norm_bwd(o, d[7], d[5], gate=d[6], gate_act="silu")
    c = chunk_gated_delta_bwd(qn, kn, v, d[3], d[4], b["dx"])
    r = qk_norm_rope_bwd(q, k, c["dq"], c["dk"], **kw)

    leaf = [x.double().clone().requires_grad_(True) for x in (qkv, g, beta)]
    q6, k6, v6 = parts(leaf[0])
    turn = lambda x: ref.qk_rope(x, None, "l2", 1e-6, pos[None], freq, [0] * 16, "half")  # noqa: E731
    o6, _ = ref.delta(turn(q6), turn(k6), v6, leaf[1], leaf[2], None)
    n6 = o6 / torch.sqrt((o6 * o6).mean(-1, keepdim=True) + 1e-6) * w.double()
    y6 = n6 * z.double() * torch.sigmoid(z.double())
    want = torch.autograd.grad((y6 * dy.double()).sum(), leaf)
    got = torch.cat([r["dq"].flatten(2), r["dk"].flatten(2), c["dv"].flatten(2)], -1)
    # fp32 throughout: each of the six stages leaves at most its roundings (about 4 (64 + 64 + 200) 2 for the two
    # chunks) of terms that the output norm, by its small rows, makes larger: taken as 2^10 in the 2-norm
    tol = 2624 * ref.ULP32 * 2.0 ** 3
    for name, a, e in (("y", y, y6), ("dqkv", got, want[0]), ("dg", c["dg"], want[1]), ("dbeta", c["dbeta"], want[2])):
        off = ((f64(a) - e.detach()).norm() / e.norm()).item()
        assert off <= tol, (name, off, tol)


@pytest.mark.parametrize("case", [CASES[3], CASES[9]], ids=_id)
def test_graph_replays(case):
    need_gpu()
    from gated_delta_rule_gate_amd import qk_norm_rope, qk_norm_rope_bwd

    g, kw = make(case, BF16, seed=6)

    def step():
        return list(qk_norm_rope(g["q"], g["k"], g["wq"], g["wk"], **kw)) + list(
            qk_norm_rope_bwd(g["q"], g["k"], g["dq"], g["dk"], g["wq"], g["wk"], **kw).values())

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(3):
        g["dq"].mul_(1.5)
        kw["positions"].add_(7)
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_long_offsets():
    """Rows whose offsets pass 32 bits."""
    need_gpu()
    from gated_delta_rule_gate_amd import qk_norm_rope, qk_norm_rope_bwd

    T, H, D = 140000, 120, 128  # 2.15e9 elements
    q = torch.zeros(1, T, H, D, dtype=BF16, device="cuda")
    q[:, -3:] = torch.randn(1, 3, H, D, device="cuda").to(BF16)
    k, w = torch.zeros(1, T, 1, D, dtype=BF16, device="cuda"), torch.ones(D, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda").reshape(1, T)
    freq = (1e4 ** (-torch.arange(0, D, 2) / D)).float().cuda()
    one = [x[:, -3:].contiguous() for x in (q, k, pos)]
    y, _ = qk_norm_rope(q, k, w, w, positions=pos, inv_freq=freq)
    y1, _ = qk_norm_rope(one[0], one[1], w, w, positions=one[2], inv_freq=freq)
    assert torch.equal(y[:, -3:], y1)
    got = qk_norm_rope_bwd(q, k, q, k, w, w, positions=pos, inv_freq=freq)
    want = qk_norm_rope_bwd(one[0], one[1], one[0], one[1], w, w, positions=one[2], inv_freq=freq)
    assert torch.equal(got["dq"][:, -3:], want["dq"])
