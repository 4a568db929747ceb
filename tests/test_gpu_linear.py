"""Linear attention with one decay per head on the GPU against the 64-bit token recurrence:
the chunked forward, its gradient and the recurrence, over types, widths, shared q/k heads,
lengths round the chunk, packed batches, segments, resets, and what stays untouched.

Tolerances count roundings: a sum of terms of total size `m` that passes n fp32 roundings is off by
at most n 2^-24 m; bf16 results add one rounding, and where scores and state enter a bf16 output as
two bf16 parts, what those leave out: 2^-16 of each, times m."""
import numpy as np
import pytest
import torch

import linear_ref as ref
from kda_testlib import need_gpu

pytestmark = pytest.mark.gpu


def make(B, T, H, Hk, K, V, dtype, decay, lens=None, states=True, seed=0, strength=1.0):
    r = np.random.Generator(np.random.PCG64(seed + 1000 * T + 7 * K + V))
    f = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32))  # noqa: E731
    N = B if lens is None else len(lens)
    d = dict(q=f(B, T, Hk, K).to(dtype), k=(f(B, T, Hk, K) * K ** -0.5).to(dtype), v=f(B, T, H, V).to(dtype))
    d["g"] = -strength * (f(H).abs() * 0.2 if decay == "head" else f(B, T, H).abs() * 0.3)
    d["h0"] = f(N, H, K, V) if states else None
    d["cu"] = None if lens is None else torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
    d["do"] = f(B, T, H, V).to(dtype)
    d["dht"] = f(N, H, K, V) if states else None
    return d


def dev(d):
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def f64(x):
    return None if x is None else x.detach().cpu().double()


def inputs64(d):
    return [f64(d[x]) for x in ("q", "k", "v", "g", "h0")]


def within(got, want, size, dtype, n, what, parts=0.0):
    """|got - want| <= one rounding to dtype + (n 2^-24 + parts) of the terms' size."""
    got, want = f64(got), f64(want)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), what
    tol = ref.HALF[dtype] * want.abs() + (n * ref.ULP32 + parts) * size * 1.01
    off = (got - want).abs()
    worst = (off / tol.clamp_min(1e-300)).max().item() if off.numel() else 0.0
    assert (off <= tol).all(), "%s: off by %.3g times the tolerance" % (what, worst)


PARTS = {torch.bfloat16: 2 * 2.0 ** -16, torch.float32: 0.0}
SHAPES = [
    # B, T, H, Hk, K, V, lens
    (1, 1, 1, 1, 8, 8, None),
    (2, 15, 3, 3, 64, 64, None),
    (1, 63, 2, 1, 128, 128, None),
    (2, 64, 2, 2, 128, 64, None),
    (1, 65, 2, 2, 40, 200, None),
    (1, 130, 3, 1, 256, 256, None),
    (1, 97, 2, 2, 136, 72, None),
    (3, 257, 4, 2, 64, 128, None),
    (1, 300, 2, 1, 128, 128, [0, 64, 1, 0, 130, 0]),
    (1, 400, 2, 2, 72, 40, [33, 300]),
    (1, 1500, 2, 2, 64, 64, None),
    (2, 1090, 2, 1, 40, 136, None),
    (1, 1700, 2, 1, 128, 136, [3, 1100, 0, 520, 60]),
]


def _id(c):
    return "b%dt%dh%d-%dk%dv%d%s" % (c[:6] + ("-packed" if c[6] else "",))


@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=_id)
def test_forward(shape, dtype, decay):
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_linear_attn

    B, T, H, Hk, K, V, lens = shape
    d = make(B, T, H, Hk, K, V, dtype, decay, lens, states=T != 97)
    g = dev(d)
    out = torch.full((B, T, H, V), 7.0, dtype=dtype, device="cuda")
    o, ht = chunk_linear_attn(g["q"], g["k"], g["v"], g["g"], g["h0"], cu_seqlens=g["cu"], output_final_state=True, out=out)
    want, size = ref.attn(*inputs64(d), cu=d["cu"]), ref.attn_sizes(*inputs64(d), cu=d["cu"])
    end = T if lens is None else sum(lens)
    n = ref.roundings(K, V, T)
    within(o[:, :end], want[0][:, :end], size[0][:, :end], dtype, n, "o", PARTS[dtype])
    within(ht, want[1], size[1], torch.float32, n, "ht")
    assert (o[:, end:] == 7.0).all(), "rows behind the last sequence were written"
    if lens:
        for i, l in enumerate(lens):
            if l == 0:
                assert torch.equal(ht[i], g["h0"][i])


@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=_id)
def test_backward(shape, dtype, decay):
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_linear_attn_bwd

    B, T, H, Hk, K, V, lens = shape
    d = make(B, T, H, Hk, K, V, dtype, decay, lens, states=T != 97, seed=1)
    g = dev(d)
    got = chunk_linear_attn_bwd(g["q"], g["k"], g["v"], g["g"], g["do"], g["h0"], dht=g["dht"], cu_seqlens=g["cu"])
    end = T if lens is None else sum(lens)
    do = f64(d["do"]).clone()
    do[:, end:] = 0
    want = ref.attn_grads(*inputs64(d), do, f64(d["dht"]), cu=d["cu"])
    size = ref.grad_sizes(*inputs64(d), do, f64(d["dht"]), cu=d["cu"])
    n = ref.roundings(K, V, T) + H // Hk
    for i, name in enumerate(("dq", "dk", "dv")):
        parts = PARTS[dtype] if name == "dv" else 0.0
        within(got[name][:, :end], want[i][:, :end], size[i][:, :end], dtype, n, name, parts)
    cut = (lambda x: x[:, :end]) if decay == "token" else (lambda x: x)
    within(cut(got["dg"]), cut(want[3]), cut(size[3]), torch.float32, n, "dg")
    within(got["dh0"], want[4], size[4], torch.float32, n, "dh0")


@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", [
    (1, 1, 1, 1, 8, 8, None), (5, 1, 4, 2, 128, 128, None), (300, 1, 4, 4, 128, 128, None), (2, 3, 3, 1, 72, 40, None),
    (2, 4, 2, 2, 256, 256, None), (3, 17, 2, 2, 64, 200, None), (1, 12, 3, 3, 136, 64, [1, 0, 5, 3]),
    (600, 1, 1, 1, 256, 256, None),
], ids=_id)
def test_recurrent(shape, dtype, decay):
    need_gpu()
    from gated_delta_rule_gate_amd import recurrent_linear_attn

    B, T, H, Hk, K, V, lens = shape
    d = make(B, T, H, Hk, K, V, dtype, decay, lens, seed=2)
    g = dev(d)
    out = torch.full((B, T, H, V), 7.0, dtype=dtype, device="cuda")
    o, ht = recurrent_linear_attn(g["q"], g["k"], g["v"], g["g"], g["h0"], cu_seqlens=g["cu"], output_final_state=True,
                                  out=out)
    want, size = ref.attn(*inputs64(d), cu=d["cu"]), ref.attn_sizes(*inputs64(d), cu=d["cu"])
    end = T if lens is None else sum(lens)
    n = ref.roundings(K, V, T)
    within(o[:, :end], want[0][:, :end], size[0][:, :end], dtype, n, "o")
    within(ht, want[1], size[1], torch.float32, n, "ht")
    assert (o[:, end:] == 7.0).all()
    # in place
    o2, h2 = recurrent_linear_attn(g["q"], g["k"], g["v"], g["g"], g["h0"], cu_seqlens=g["cu"], final_state=g["h0"])
    assert h2 is g["h0"] and torch.equal(h2, ht) and torch.equal(o2[:, :end], o[:, :end])


@pytest.mark.parametrize("T", [200, 1600])
def test_in_place_state(T):
    """The final state written over the initial one, with and without segments."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_linear_attn

    g = dev(make(1, T, 2, 2, 128, 128, torch.bfloat16, "head", seed=3, strength=0.1))
    o, ht = chunk_linear_attn(g["q"], g["k"], g["v"], g["g"], g["h0"], output_final_state=True)
    o2, h2 = chunk_linear_attn(g["q"], g["k"], g["v"], g["g"], g["h0"], final_state=g["h0"])
    assert torch.equal(o, o2) and torch.equal(ht, h2)


def test_no_tokens():
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_linear_attn, chunk_linear_attn_bwd, recurrent_linear_attn

    g = dev(make(2, 0, 2, 2, 64, 64, torch.bfloat16, "token", seed=4))
    for f in (chunk_linear_attn, recurrent_linear_attn):
        o, ht = f(g["q"], g["k"], g["v"], g["g"], g["h0"], output_final_state=True)
        assert o.shape == (2, 0, 2, 64) and torch.equal(ht, g["h0"])
    got = chunk_linear_attn_bwd(g["q"], g["k"], g["v"], g["g"], g["do"], g["h0"], dht=g["dht"])
    assert torch.equal(got["dh0"], g["dht"])
    h = dev(make(2, 0, 2, 2, 64, 64, torch.bfloat16, "head", seed=4))
    assert (chunk_linear_attn_bwd(h["q"], h["k"], h["v"], h["g"], h["do"], h["h0"], dht=h["dht"])["dg"] == 0).all()


@pytest.mark.parametrize("lens", [[], [0, 0, 0], [0, 0, 0, 5]], ids=["none", "empty", "last"])
def test_slots_without_tokens(lens):
    """Packed batches of no slot, of empty slots only, and of empty slots before a short one."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_linear_attn, chunk_linear_attn_bwd, recurrent_linear_attn

    T = 40
    d = make(1, T, 4, 2, 64, 64, torch.bfloat16, "head", lens=lens, seed=40)
    d["cu"] = torch.tensor([3] + [3 + sum(lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32)
    g = dev(d)
    for f in (chunk_linear_attn, recurrent_linear_attn):
        out = torch.full_like(g["v"], 7.0)
        _, ht = f(g["q"], g["k"], g["v"], g["g"], g["h0"], cu_seqlens=g["cu"], output_final_state=True, out=out)
        assert all(torch.equal(ht[i], g["h0"][i]) for i, l in enumerate(lens) if l == 0)
        assert (out[:, :3] == 7.0).all() and (out[:, 3 + sum(lens):] == 7.0).all()
        assert torch.isfinite(out).all()
    got = chunk_linear_attn_bwd(g["q"], g["k"], g["v"], g["g"], g["do"], g["h0"], dht=g["dht"], cu_seqlens=g["cu"])
    assert all(torch.equal(got["dh0"][i], g["dht"][i]) for i, l in enumerate(lens) if l == 0)
    assert torch.isfinite(got["dg"]).all() and (sum(lens) > 0 or (got["dg"] == 0).all())


def test_many_heads_and_slots():
    """More (sequence, head) pairs than compute units, slots shorter and longer than a chunk, shared heads."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_linear_attn, chunk_linear_attn_bwd

    lens = [1, 70, 0, 33, 64, 128, 7, 100, 3, 17]
    d = make(1, sum(lens) + 2, 48, 16, 64, 72, torch.bfloat16, "token", lens=lens, seed=41)
    g = dev(d)
    o, ht = chunk_linear_attn(g["q"], g["k"], g["v"], g["g"], g["h0"], cu_seqlens=g["cu"], output_final_state=True)
    end, n = sum(lens), ref.roundings(64, 72, 128)
    want, size = ref.attn(*inputs64(d), cu=d["cu"]), ref.attn_sizes(*inputs64(d), cu=d["cu"])
    within(o[:, :end], want[0][:, :end], size[0][:, :end], torch.bfloat16, n, "o", PARTS[torch.bfloat16])
    within(ht, want[1], size[1], torch.float32, n, "ht")
    do = f64(d["do"]).clone()
    do[:, end:] = 0
    got = chunk_linear_attn_bwd(g["q"], g["k"], g["v"], g["g"], g["do"], g["h0"], dht=g["dht"], cu_seqlens=g["cu"])
    want, size = (f(*inputs64(d), do, f64(d["dht"]), cu=d["cu"]) for f in (ref.attn_grads, ref.grad_sizes))
    for i, name in enumerate(("dq", "dk", "dv", "dg")):
        t = torch.float32 if name == "dg" else torch.bfloat16
        within(got[name][:, :end], want[i][:, :end], size[i][:, :end], t, n + 3, name, PARTS[t] if name == "dv" else 0.0)
    within(got["dh0"], want[4], size[4], torch.float32, n, "dh0")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_resets_and_strong_decays(dtype):
    """-inf, decays far below fp32's range, zero decays, and weak ones next to them in one chunk."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_linear_attn, chunk_linear_attn_bwd, recurrent_linear_attn

    d = make(1, 150, 2, 2, 64, 64, dtype, "token", seed=5, strength=0.2)
    d["g"][0, ::7] = -float("inf")
    d["g"][0, 3::11] = -1e4
    d["g"][0, 5::9] = -90.0
    d["g"][0, 40:50] = 0.0
    d["g"][0, 140:] = -float("inf")
    g = dev(d)
    args = inputs64(d)
    want, size = ref.attn(*args), ref.attn_sizes(*args)
    n = ref.roundings(64, 64, 150)
    for f in (chunk_linear_attn, recurrent_linear_attn):
        o, ht = f(g["q"], g["k"], g["v"], g["g"], g["h0"], output_final_state=True)
        within(o, want[0], size[0], dtype, n, "o", PARTS[dtype])
        within(ht, want[1], size[1], torch.float32, n, "ht")
    got = chunk_linear_attn_bwd(g["q"], g["k"], g["v"], g["g"], g["do"], g["h0"], dht=g["dht"])
    do, dht = f64(d["do"]), f64(d["dht"])
    args[3] = args[3].clamp_min(-1e5)  # the derivative at -inf is the limit: zero
    want, size = ref.attn_grads(*args, do, dht), ref.grad_sizes(*args, do, dht)
    for i, name in enumerate(("dq", "dk", "dv", "dg", "dh0")):
        t = torch.float32 if name in ("dg", "dh0") else dtype
        within(got[name], want[i], size[i], t, n, name, PARTS[dtype] if name == "dv" else 0.0)


def test_non_finite_stays_in_its_head_and_chunk():
    """A NaN reaches its own head from its chunk's start on: not earlier chunks, other heads or sequences."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_linear_attn

    g = dev(make(1, 400, 2, 2, 64, 64, torch.bfloat16, "token", lens=[130, 270], seed=6))
    o, ht = chunk_linear_attn(g["q"], g["k"], g["v"], g["g"], g["h0"], cu_seqlens=g["cu"], output_final_state=True)
    for name in ("v", "k", "q", "g"):
        b = {x: None if t is None else t.clone() for x, t in g.items()}
        b[name][0, 130 + 70, 1] = float("nan")
        o2, h2 = chunk_linear_attn(b["q"], b["k"], b["v"], b["g"], b["h0"], cu_seqlens=b["cu"], output_final_state=True)
        assert torch.equal(o[:, :130], o2[:, :130]) and torch.equal(o[:, :, 0], o2[:, :, 0]), name
        assert torch.equal(o[0, 130:194, 1], o2[0, 130:194, 1]), name
        assert not torch.isfinite(o2[0, 200, 1]).any(), name
        assert torch.equal(ht[0], h2[0]) and torch.equal(ht[1, 0], h2[1, 0]), name


def test_rows_outside_the_offsets():
    """Rows before the first offset and behind the last are neither read nor written, gradients included."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_linear_attn, lib
    from gated_delta_rule_gate_amd import _linear

    d = make(1, 300, 4, 2, 64, 64, torch.bfloat16, "token", lens=[70, 100], seed=7)
    d["cu"] += 20
    for x in ("q", "k", "v", "g", "do"):
        d[x][0, :20] = float("nan")
        d[x][0, 190:] = float("nan")
    g = dev(d)
    out = torch.full_like(g["v"], 7.0)
    o, _ = chunk_linear_attn(g["q"], g["k"], g["v"], g["g"], g["h0"], cu_seqlens=g["cu"], out=out)
    inner = [x[:, 20:190] if i < 4 else x for i, x in enumerate(inputs64(d))]
    want = ref.attn(*inner, cu=d["cu"] - 20)
    size = ref.attn_sizes(*inner, cu=d["cu"] - 20)
    within(o[:, 20:190], want[0], size[0], torch.bfloat16, ref.roundings(64, 64, 300), "o", PARTS[torch.bfloat16])
    assert (o[:, :20] == 7.0).all() and (o[:, 190:] == 7.0).all()
    # the C entry, with gradients that hold a mark
    a, _, i, (pq, pk, pv, pg, ph, pc) = _linear._attn_args(g["q"], g["k"], g["v"], g["g"], g["h0"], g["cu"], None)
    marks = [torch.full_like(g[x], 7.0) for x in ("q", "k", "v", "g")]
    need = lib().kda_linear_chunk_bwd_workspace_bytes(a)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN everywhere
    _linear._launch(i, lib().kda_linear_chunk_bwd, a, pq, pk, pv, pg, ph, pc, g["do"].data_ptr(),
                    g["dht"].data_ptr(), *[m.data_ptr() for m in marks], None, ws.data_ptr(), need)
    for m in marks:
        assert (m[:, :20] == 7.0).all() and (m[:, 190:] == 7.0).all()
        assert torch.isfinite(m[:, 20:190]).all()


@pytest.mark.parametrize("which", ["q", "k", "v", "h0"])
def test_gradient_against_differences(which):
    """o and ht are linear in each of q, k, v, h0 alone: L(x + d) - L(x - d) = 2 <dx, d> up to rounding."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_linear_attn, chunk_linear_attn_bwd

    d = make(1, 150, 2, 1, 72, 40, torch.float32, "token", seed=8)
    g = dev(d)
    step = torch.from_numpy(np.random.Generator(np.random.PCG64(9)).standard_normal(tuple(d[which].shape)).astype(np.float32))

    def loss(sign):
        m = dict(g, **{which: (g[which] + sign * step.cuda())})
        o, ht = chunk_linear_attn(m["q"], m["k"], m["v"], m["g"], m["h0"], output_final_state=True)
        return ((o.double() * m["do"].double()).sum() + (ht.double() * m["dht"].double()).sum()).item()

    got = chunk_linear_attn_bwd(g["q"], g["k"], g["v"], g["g"], g["do"], g["h0"], dht=g["dht"])["d" + which]
    diff, along = loss(1) - loss(-1), 2 * (got.double() * step.cuda().double()).sum().item()
    args = [x.abs() if i != 3 else x for i, x in enumerate(inputs64(d))]
    at = ("q", "k", "v", None, "h0").index(which)
    args[at] = args[at] + step.abs().double()
    so, sh = ref.attn(*args)
    size = (so * f64(d["do"]).abs()).sum() + (sh * f64(d["dht"]).abs()).sum()
    # both losses' roundings and the gradient's; x + d itself is rounded once
    tol = (4 * ref.roundings(72, 40, 150) + 4) * ref.ULP32 * size.item()
    assert abs(diff - along) <= tol, (diff, along, tol)


def test_decay_gradient_against_differences():
    """L is a + b e^x in one token's decay x: a central difference is off by h^2 / 6 of its own size."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_linear_attn, chunk_linear_attn_bwd

    d = make(1, 100, 2, 2, 64, 64, torch.float32, "token", seed=10)
    g = dev(d)
    dg = chunk_linear_attn_bwd(g["q"], g["k"], g["v"], g["g"], g["do"], g["h0"], dht=g["dht"])["dg"]
    args = inputs64(d)
    so, sh = ref.attn_sizes(*args)
    size = ((so * f64(d["do"]).abs()).sum() + (sh * f64(d["dht"]).abs()).sum()).item()
    h = 2.0 ** -4
    for t, head in ((0, 0), (37, 1), (64, 0), (99, 1)):
        def loss(sign):
            x = g["g"].clone()
            x[0, t, head] += sign * h
            o, ht = chunk_linear_attn(g["q"], g["k"], g["v"], x, g["h0"], output_final_state=True)
            return ((o.double() * g["do"].double()).sum() + (ht.double() * g["dht"].double()).sum()).item()

        diff, want = (loss(1) - loss(-1)) / (2 * h), dg[0, t, head].item()
        n = ref.roundings(64, 64, 100)
        # h itself is off by a rounding of x +- h, at most |x| + h
        tol = h * h / 6 * 1.01 * abs(want) + n * ref.ULP32 * size * (1 + 1 / h) * 1.01
        assert abs(diff - want) <= tol, (t, head, diff, want, tol)


def test_long_offsets():
    """A packed batch whose token offsets times heads and widths pass 32 bits."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_linear_attn

    H, K, T = 64, 128, 300000  # 2.46e9 elements a tensor
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.empty(1, T, H, K, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    lens = [T - 100, 100]
    for x in (q, k, v):
        x[:, -164:] = torch.randn(1, 164, H, K, device="cuda", generator=gen).to(torch.bfloat16)
    g = torch.full((H,), -0.1, device="cuda")
    cu = torch.tensor([0, T - 100, T], dtype=torch.int32, device="cuda")
    cu2 = torch.tensor([T - 100, T - 100, T], dtype=torch.int32, device="cuda")
    out = torch.empty_like(v)
    for x in (q, k, v):  # the rest of the first sequence does not matter: keep it finite
        x[:, :-164] = 0
    o, ht = chunk_linear_attn(q, k, v, g, cu_seqlens=cu, output_final_state=True, out=out)
    tail = [x[:, -100:].contiguous() for x in (q, k, v)]
    o1, h1 = chunk_linear_attn(*tail, g, output_final_state=True)
    within(o[:, -100:], o1, torch.zeros(()), torch.bfloat16, 0, "tail")
    assert torch.equal(ht[1], h1[0])
    o.zero_()
    o2, _ = chunk_linear_attn(q, k, v, g, cu_seqlens=cu2, out=out)
    assert torch.equal(o2[:, -100:], o1)


@pytest.mark.parametrize("T", [130, 1500])
def test_graph_replays(T):
    """Captured forward, gradient and recurrence; replays with new inputs and offsets equal eager calls."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_linear_attn, chunk_linear_attn_bwd, recurrent_linear_attn

    g = dev(make(1, T, 2, 1, 64, 64, torch.bfloat16, "token", lens=[T // 3, T - T // 3], seed=11))

    def step():
        o, ht = chunk_linear_attn(g["q"], g["k"], g["v"], g["g"], g["h0"], cu_seqlens=g["cu"], output_final_state=True)
        b = chunk_linear_attn_bwd(g["q"], g["k"], g["v"], g["g"], g["do"], g["h0"], dht=g["dht"], cu_seqlens=g["cu"])
        r = recurrent_linear_attn(g["q"][:, :1].contiguous(), g["k"][:, :1].contiguous(), g["v"][:, :1].contiguous(),
                                  g["g"][:, :1].contiguous(), ht[:1].contiguous())
        return [o, ht] + [b[x] for x in ("dq", "dk", "dv", "dg", "dh0")] + [r[0]]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for turn in range(3):
        g["v"].copy_(torch.randn_like(g["v"], dtype=torch.float32).to(torch.bfloat16))
        g["cu"].copy_(torch.tensor([0, 10 + 40 * turn, T], dtype=torch.int32))
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(held, want):
            assert torch.equal(x, y)


def test_two_graphs_and_an_eager_call():
    """Graphs captured from the same inputs, each with its own workspace, replayed one after the other and
    between eager calls."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_linear_attn, chunk_linear_attn_bwd

    g = dev(make(1, 1300, 2, 2, 64, 128, torch.bfloat16, "head", seed=30))
    fwd = lambda: list(chunk_linear_attn(g["q"], g["k"], g["v"], g["g"], g["h0"], output_final_state=True))  # noqa: E731
    bwd = lambda: list(chunk_linear_attn_bwd(g["q"], g["k"], g["v"], g["g"], g["do"], g["h0"],  # noqa: E731
                                             dht=g["dht"]).values())
    fwd(), bwd()
    torch.cuda.synchronize()
    graphs = []
    for f in (fwd, bwd):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = f()
        graphs.append((graph, held, f))
    for _ in range(3):
        g["k"].mul_(1.25)
        for graph, held, f in graphs + graphs[::-1]:
            want = f()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_two_streams_with_workspaces_of_their_own():
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_linear_attn, linear_workspace_bytes

    sets = [dev(make(1, 2000, 2, 2, 128, 128, torch.bfloat16, "token", seed=20 + i)) for i in range(2)]
    want = [chunk_linear_attn(g["q"], g["k"], g["v"], g["g"], g["h0"], output_final_state=True) for g in sets]
    ws = [torch.empty(max(256, linear_workspace_bytes(g["q"], g["k"], g["v"], g["g"])),
                      dtype=torch.uint8, device="cuda") for g in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for g, s, w in zip(sets, streams, ws):
        with torch.cuda.stream(s):
            got.append(chunk_linear_attn(g["q"], g["k"], g["v"], g["g"], g["h0"], output_final_state=True, workspace=w))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_prompt_then_tokens():
    """A prompt through the chunked form, then tokens one by one on the state it left: the whole sequence."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_linear_attn, recurrent_linear_attn

    d = make(2, 90, 2, 1, 64, 64, torch.float32, "token", seed=12)
    g = dev(d)
    cut = lambda a, b: [g[x][:, a:b].contiguous() for x in ("q", "k", "v", "g")]  # noqa: E731
    o, state = chunk_linear_attn(*cut(0, 80), g["h0"], output_final_state=True)
    rows = [o]
    for t in range(80, 90):
        o, _ = recurrent_linear_attn(*cut(t, t + 1), state, final_state=state)
        rows.append(o)
    want, size = ref.attn(*inputs64(d)), ref.attn_sizes(*inputs64(d))
    n = ref.roundings(64, 64, 90) + 10 * 3
    within(torch.cat(rows, 1), want[0], size[0], torch.float32, n, "o")
    within(state, want[1], size[1], torch.float32, n, "state")


# Shapes whose kernels the ones above do not reach: with more than 32 (sequence, head) pairs fp32 goes by 128
# columns, and with more than 128 (segment, head) pairs the state pass does too.
MANY_HEADS = [
    # B, T, H, Hk, K, V, lens, in segments
    (1, 150, 40, 20, 128, 128, None, False),
    (2, 97, 24, 8, 64, 72, None, False),
    (1, 150, 48, 16, 72, 40, None, False),
    (1, 200, 36, 36, 128, 72, [70, 0, 33, 90], False),
    (1, 1100, 48, 16, 72, 72, None, True),
    (1, 1100, 80, 80, 40, 72, None, True),
    (1, 2600, 48, 48, 72, 24, [1500, 0, 1060], True),
    (1, 1100, 48, 24, 136, 72, None, "bf16"),  # fp32 has two column blocks, and pairs enough
]


def on_gpu64(d):
    """The 64-bit reference's arguments, on the GPU: (q, k, v, g, h0), do without rows outside, dht."""
    up = lambda x: d[x].cuda().double()  # noqa: E731
    return [up(x) for x in ("q", "k", "v", "g", "h0")], up("do"), up("dht")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", MANY_HEADS, ids=_id)
def test_many_heads(shape, dtype):
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_linear_attn, chunk_linear_attn_bwd, linear_workspace_bytes

    B, T, H, Hk, K, V, lens, cut = shape
    d = make(B, T, H, Hk, K, V, dtype, "head" if H == 40 else "token", lens, seed=70)
    g = dev(d)
    need = linear_workspace_bytes(g["q"], g["k"], g["v"], g["g"], slots=None if lens is None else len(lens))
    assert (need > 0) == (dtype == torch.bfloat16 if cut == "bf16" else cut)
    end = T if lens is None else sum(lens)
    args, do, dht = on_gpu64(d)
    do[:, end:] = 0
    n = ref.roundings(K, V, T) + H // Hk
    o, ht = chunk_linear_attn(g["q"], g["k"], g["v"], g["g"], g["h0"], cu_seqlens=g["cu"], output_final_state=True)
    got = chunk_linear_attn_bwd(g["q"], g["k"], g["v"], g["g"], g["do"], g["h0"], dht=g["dht"], cu_seqlens=g["cu"])
    with torch.device("cuda"):
        want = [*ref.attn(*args, cu=d["cu"]), *ref.attn_grads(*args, do, dht, cu=d["cu"])]
        size = [*ref.attn_sizes(*args, cu=d["cu"]), *ref.grad_sizes(*args, do, dht, cu=d["cu"])]
    for name, w, s in zip(("o", "ht", "dq", "dk", "dv", "dg", "dh0"), want, size):
        x = dict(got, o=o, ht=ht)[name]
        rows = name in ("o", "dq", "dk", "dv") or (name == "dg" and x.dim() == 3)
        c = (lambda t: t[:, :end]) if rows else (lambda t: t)
        within(c(x), c(w), c(s).cpu(), x.dtype, n, name, PARTS[dtype] if name in ("o", "dv") else 0.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", [
    # 512 and more (sequence, head, 128 columns): blocks of 128 columns, over several tokens and partial widths
    (130, 3, 4, 2, 72, 136, None), (256, 2, 2, 1, 128, 128, None), (130, 2, 4, 4, 200, 256, None),
    (520, 1, 1, 1, 40, 72, None), (256, 2, 2, 2, 256, 128, None), (1, 215, 4, 1, 64, 128, [i % 4 for i in range(140)]),
    (1, 100, 16, 16, 136, 40, [0, 7, 1, 2] * 9),
], ids=_id)
def test_recurrent_with_many_sequences(shape, dtype):
    need_gpu()
    from gated_delta_rule_gate_amd import recurrent_linear_attn

    B, T, H, Hk, K, V, lens = shape
    assert (B if lens is None else len(lens)) * H * -(-V // 128) >= 512
    d = make(B, T, H, Hk, K, V, dtype, "token", lens, seed=71)
    g = dev(d)
    out = torch.full((B, T, H, V), 7.0, dtype=dtype, device="cuda")
    o, ht = recurrent_linear_attn(g["q"], g["k"], g["v"], g["g"], g["h0"], cu_seqlens=g["cu"], output_final_state=True,
                                  out=out)
    args = on_gpu64(d)[0]
    with torch.device("cuda"):
        want, size = ref.attn(*args, cu=d["cu"]), ref.attn_sizes(*args, cu=d["cu"])
    end, n = T if lens is None else sum(lens), ref.roundings(K, V, T)
    within(o[:, :end], want[0][:, :end], size[0][:, :end].cpu(), dtype, n, "o")
    within(ht, want[1], size[1].cpu(), torch.float32, n, "ht")
    assert (o[:, end:] == 7.0).all()
    recurrent_linear_attn(g["q"], g["k"], g["v"], g["g"], g["h0"], cu_seqlens=g["cu"], final_state=g["h0"])
    assert torch.equal(g["h0"], ht)


@pytest.mark.parametrize("lens", [None, [1500, 0, 1, 599]], ids=["dense", "packed"])
def test_calls_repeat_themselves(lens):
    """The same call gives the same bits, whatever lay in the memory that it takes."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_linear_attn, chunk_linear_attn_bwd

    g = dev(make(1, 2100, 8, 4, 64, 128, torch.bfloat16, "token", lens, seed=72))

    def call():
        dirty = [torch.full((n,), float("nan"), device="cuda") for n in (1 << 16, 1 << 20, 1 << 23)]
        del dirty
        o, ht = chunk_linear_attn(g["q"], g["k"], g["v"], g["g"], g["h0"], cu_seqlens=g["cu"], output_final_state=True)
        b = chunk_linear_attn_bwd(g["q"], g["k"], g["v"], g["g"], g["do"], g["h0"], dht=g["dht"], cu_seqlens=g["cu"])
        return [o, ht] + list(b.values())

    first = call()
    assert all(torch.isfinite(x).all() for x in first)
    for _ in range(4):
        assert all(torch.equal(a, b) for a, b in zip(first, call()))
