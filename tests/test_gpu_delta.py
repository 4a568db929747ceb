"""The gated delta rule with one decay per head on the GPU against the 64-bit token recurrence: the chunked
forward, its gradient and the recurrence, over types, widths, shared q/k heads, lengths round the chunk,
packed batches, resets, repeated keys, and what stays untouched. Tolerances: delta_ref.py."""
import numpy as np
import pytest
import torch

import delta_ref as ref
from kda_testlib import need_gpu

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


def make(B, T, H, Hk, K, V, dtype, lens=None, states=True, seed=0, strength=1.0, decay=True):
    r = np.random.Generator(np.random.PCG64(seed + 1000 * T + 7 * K + V))
    f = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32))  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True) * 0.99  # noqa: E731  rounding to bf16 keeps it below one
    N = B if lens is None else len(lens)
    d = dict(q=unit(f(B, T, Hk, K)).to(dtype), k=unit(f(B, T, Hk, K)).to(dtype), v=f(B, T, H, V).to(dtype))
    d["g"] = -strength * f(B, T, H).abs() * 0.3 if decay else None
    d["beta"] = torch.sigmoid(f(B, T, H))
    d["h0"] = f(N, H, K, V) if states else None
    d["cu"] = None if lens is None else torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
    d["do"] = f(B, T, H, V).to(dtype)
    d["dht"] = f(N, H, K, V) if states else None
    return d


def dev(d):
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def f64(x):
    return None if x is None else x.detach().cpu().double()


IN = ("q", "k", "v", "g", "beta", "h0")


def inputs64(d):
    return [f64(d[x]) for x in IN]


def on(g, f, *more, **kw):
    return f(*[g[x] for x in IN[:5]], *more, g["h0"], cu_seqlens=g["cu"], **kw)


def within(got, want, size, dtype, n, what, left_out=0.0):
    """2-norms over the last axis (or, of states, the last two): |got - want| <= a rounding to dtype + (n 2^-24 +
    left_out) size."""
    got, want = f64(got), f64(want)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), what
    off, own = got - want, want
    while off.dim() > size.dim():
        off, own = off.norm(dim=-1), own.norm(dim=-1)
    tol = ref.HALF[dtype] * own.abs() + (n * ref.ULP32 + left_out) * size * 1.01
    worst = (off.abs() / tol.clamp_min(1e-300)).max().item() if off.numel() else 0.0
    assert (off.abs() <= tol).all(), "%s: off by %.3g times the tolerance" % (what, worst)


SHAPES = [
    # B, T, H, Hk, K, V, lens
    (1, 1, 1, 1, 8, 8, None),
    (2, 15, 3, 3, 64, 64, None),
    (1, 31, 1, 1, 256, 8, None),
    (1, 33, 2, 1, 8, 256, None),
    (1, 63, 2, 1, 128, 128, None),
    (2, 64, 2, 2, 128, 64, None),
    (1, 65, 2, 2, 40, 200, None),
    (1, 130, 3, 1, 256, 256, None),
    (1, 97, 2, 2, 136, 72, None),
    (3, 257, 4, 2, 64, 128, None),
    (1, 300, 2, 1, 128, 128, [0, 64, 1, 0, 130, 0]),
    (1, 400, 2, 2, 72, 40, [33, 300]),
    (1, 333, 2, 2, 256, 136, [5, 0, 200, 64, 32]),
    (2, 520, 2, 1, 40, 136, None),
]


def _id(c):
    return "b%dt%dh%d-%dk%dv%d%s" % (c[:6] + ("-packed" if c[6] else "",))


def check_forward(d, f, out):
    g = dev(d)
    B, T, H, V = d["v"].shape
    K, dtype = d["q"].shape[3], d["v"].dtype
    o, ht = on(g, f, output_final_state=True, out=out)
    want, size = ref.delta(*inputs64(d), cu=d["cu"]), ref.sizes(*inputs64(d), cu=d["cu"])
    n, inside = ref.roundings(K, V, T), torch.zeros(T, dtype=torch.bool)
    for lo, hi in ([(0, T)] if d["cu"] is None else ref.slots_of(B, T, d["cu"])):
        inside[lo:hi] = True
    within(o[:, inside], want[0][:, inside], size[0][:, inside], dtype, n, "o", ref.LEFT_OUT[dtype])
    within(ht, want[1], size[1], FP32, n, "ht")
    return o, ht, inside


@pytest.mark.parametrize("decay", [True, False], ids=["decay", "plain"])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=_id)
def test_forward(shape, dtype, decay):
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta

    B, T, H, Hk, K, V, lens = shape
    d = make(B, T, H, Hk, K, V, dtype, lens, states=T != 97, decay=decay)
    out = torch.full((B, T, H, V), 7.0, dtype=dtype, device="cuda")
    o, ht, inside = check_forward(d, chunk_gated_delta, out)
    assert (o[:, ~inside] == 7.0).all(), "rows behind the last sequence were written"
    if lens:
        for i, l in enumerate(lens):
            if l == 0:
                assert torch.equal(ht[i].cpu(), d["h0"][i])


LONG = [  # cut into segments: few heads, several times as many chunks
    (1, 1500, 2, 2, 64, 64, None),
    (2, 1090, 2, 1, 40, 136, None),
    (1, 1700, 2, 1, 128, 136, [3, 1100, 0, 520, 60]),
    (1, 1300, 2, 1, 256, 72, None),
    (1, 2100, 1, 1, 128, 128, [64, 1984, 52]),
]


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", LONG, ids=_id)
def test_long_forward(shape, dtype):
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta

    B, T, H, Hk, K, V, lens = shape
    # weak decays: a segment's map matters to the next
    d = make(B, T, H, Hk, K, V, dtype, lens, seed=80, strength=0.01)
    out = torch.full((B, T, H, V), 7.0, dtype=dtype, device="cuda")
    o, ht, inside = check_forward(d, chunk_gated_delta, out)
    assert (o[:, ~inside] == 7.0).all()
    g = dev(d)  # in place
    o2, h2 = on(g, chunk_gated_delta, final_state=g["h0"])
    assert torch.equal(o2[:, inside], o[:, inside]) and torch.equal(h2, ht)


def check_backward(d, scale=None):
    from gated_delta_rule_gate_amd import chunk_gated_delta_bwd

    g = dev(d)
    B, T, Hk, K = d["q"].shape
    H, V = d["v"].shape[2:]
    dtype = d["v"].dtype
    got = on(g, chunk_gated_delta_bwd, g["do"], dht=g["dht"], scale=scale)
    inside = torch.zeros(T, dtype=torch.bool)
    for lo, hi in ([(0, T)] if d["cu"] is None else ref.slots_of(B, T, d["cu"])):
        inside[lo:hi] = True
    do = f64(d["do"]).clone()
    do[:, ~inside] = 0
    want = ref.grads(*inputs64(d), do, f64(d["dht"]), cu=d["cu"], scale=scale)
    size = ref.sizes(*inputs64(d), cu=d["cu"], do=do, dht=f64(d["dht"]), scale=scale)[2:]
    n = ref.roundings(K, V, T) + H // Hk
    for i, name in enumerate(("dq", "dk", "dv", "dg", "dbeta")):
        if got[name] is None:
            assert name == "dg" and d["g"] is None
            continue
        t = FP32 if name in ("dg", "dbeta") else dtype
        within(got[name][:, inside], want[i][:, inside], size[i][:, inside], t, n, name)
    within(got["dh0"], want[5], size[5], FP32, n, "dh0")
    return got


@pytest.mark.parametrize("decay", [True, False], ids=["decay", "plain"])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=_id)
def test_backward(shape, dtype, decay):
    need_gpu()
    B, T, H, Hk, K, V, lens = shape
    check_backward(make(B, T, H, Hk, K, V, dtype, lens, states=T != 97, seed=1, decay=decay))


def test_scale():
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta, recurrent_gated_delta

    d = make(1, 70, 2, 2, 64, 64, FP32, seed=50)
    g = dev(d)
    want, size = ref.delta(*inputs64(d), scale=0.7), ref.sizes(*inputs64(d), scale=0.7)
    for f in (chunk_gated_delta, recurrent_gated_delta):
        within(on(g, f, scale=0.7)[0], want[0], size[0], FP32, ref.roundings(64, 64, 70), "o")
    check_backward(d, scale=0.7)


@pytest.mark.parametrize("decay", [True, False], ids=["decay", "plain"])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", [
    (1, 1, 1, 1, 8, 8, None), (5, 1, 4, 2, 128, 128, None), (300, 1, 4, 4, 128, 128, None), (2, 3, 3, 1, 72, 40, None),
    (2, 4, 2, 2, 256, 256, None), (3, 17, 2, 2, 64, 200, None), (1, 12, 3, 3, 136, 64, [1, 0, 5, 3]),
    (600, 1, 1, 1, 256, 256, None),
], ids=_id)
def test_recurrent(shape, dtype, decay):
    need_gpu()
    from gated_delta_rule_gate_amd import recurrent_gated_delta

    B, T, H, Hk, K, V, lens = shape
    d = make(B, T, H, Hk, K, V, dtype, lens, seed=2, decay=decay)
    out = torch.full((B, T, H, V), 7.0, dtype=dtype, device="cuda")
    o, ht, inside = check_forward(d, recurrent_gated_delta, out)
    assert (o[:, ~inside] == 7.0).all()
    g = dev(d)  # in place
    o2, h2 = on(g, recurrent_gated_delta, final_state=g["h0"])
    assert h2 is g["h0"] and torch.equal(h2, ht) and torch.equal(o2[:, inside], o[:, inside])


@pytest.mark.parametrize("T", [200, 1600])
def test_in_place_state(T):
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta

    g = dev(make(1, T, 2, 2, 128, 128, BF16, seed=3, strength=0.1))
    o, ht = on(g, chunk_gated_delta, output_final_state=True)
    o2, h2 = on(g, chunk_gated_delta, final_state=g["h0"])
    assert torch.equal(o, o2) and torch.equal(ht, h2)


def test_no_tokens():
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta, chunk_gated_delta_bwd, recurrent_gated_delta

    g = dev(make(2, 0, 2, 2, 64, 64, BF16, seed=4))
    for f in (chunk_gated_delta, recurrent_gated_delta):
        o, ht = on(g, f, output_final_state=True)
        assert o.shape == (2, 0, 2, 64) and torch.equal(ht, g["h0"])
    got = on(g, chunk_gated_delta_bwd, g["do"], dht=g["dht"])
    assert torch.equal(got["dh0"], g["dht"])


@pytest.mark.parametrize("lens", [[], [0, 0, 0], [0, 0, 0, 5]], ids=["none", "empty", "last"])
def test_slots_without_tokens(lens):
    """Packed batches of no slot, of empty slots only, and of empty slots before a short one."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta, chunk_gated_delta_bwd, recurrent_gated_delta

    T = 40
    d = make(1, T, 4, 2, 64, 64, BF16, lens=lens, seed=40)
    d["cu"] = torch.tensor([3] + [3 + sum(lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32)
    g = dev(d)
    for f in (chunk_gated_delta, recurrent_gated_delta):
        out = torch.full_like(g["v"], 7.0)
        _, ht = on(g, f, output_final_state=True, out=out)
        assert all(torch.equal(ht[i], g["h0"][i]) for i, l in enumerate(lens) if l == 0)
        assert (out[:, :3] == 7.0).all() and (out[:, 3 + sum(lens):] == 7.0).all()
        assert torch.isfinite(out).all()
    got = on(g, chunk_gated_delta_bwd, g["do"], dht=g["dht"])
    assert all(torch.equal(got["dh0"][i], g["dht"][i]) for i, l in enumerate(lens) if l == 0)


def test_many_heads_and_slots():
    """More (sequence, head) pairs than compute units, slots shorter and longer than a chunk, shared heads."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta

    lens = [1, 70, 0, 33, 64, 128, 7, 100, 3, 17]
    d = make(1, sum(lens) + 2, 48, 16, 64, 72, BF16, lens=lens, seed=41)
    check_forward(d, chunk_gated_delta, None)
    check_backward(d)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_resets_and_strong_decays(dtype):
    """-inf, decays far below fp32's range, zero decays, and weak ones next to them in one chunk."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta, recurrent_gated_delta

    d = make(1, 150, 2, 2, 64, 64, dtype, seed=5, strength=0.2)
    d["g"][0, ::7] = -float("inf")
    d["g"][0, 3::11] = -1e4
    d["g"][0, 5::9] = -90.0
    d["g"][0, 40:50] = 0.0
    d["g"][0, 140:] = -float("inf")
    for f in (chunk_gated_delta, recurrent_gated_delta):
        check_forward(d, f, None)
    from gated_delta_rule_gate_amd import chunk_gated_delta_bwd

    g = dev(d)
    got = on(g, chunk_gated_delta_bwd, g["do"], dht=g["dht"])
    d["g"] = d["g"].clamp_min(-1e5)  # the derivative at -inf is the limit: zero
    same = check_backward(d)
    assert all(torch.equal(got[x], same[x]) for x in got)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T", [64, 200])
def test_one_key_again_and_again(T, dtype):
    """beta 1, no decay, a key that never changes: every token replaces what the one before wrote, and the
    chunk's system has ones all below its diagonal. S_t = S_0 - k k^T S_0 + k v_t^T for unit k."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta

    d = make(1, T, 1, 1, 64, 64, dtype, seed=6, decay=False)
    k = torch.zeros(64)
    k[[3, 10, 11, 40]] = torch.tensor([0.5, -0.5, 0.5, 0.5])  # norm one in either type
    d["k"][:] = k.to(dtype)
    d["beta"][:] = 1.0
    o, ht, _ = check_forward(d, chunk_gated_delta, None)
    h0, kk = f64(d["h0"])[0, 0], k.double()
    want = h0 - kk[:, None] * (kk @ h0)[None] + kk[:, None] * f64(d["v"])[0, -1, 0][None]
    within(ht[0, 0], want, torch.tensor(h0.norm().item() + 10.0, dtype=torch.float64), FP32, ref.roundings(64, 64, T), "ht")
    check_backward(d)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_tokens_that_write_nothing(dtype):
    """beta 0 leaves the state as the decay leaves it; v gets no gradient there, beta does."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta, recurrent_gated_delta

    d = make(1, 140, 2, 1, 72, 64, dtype, seed=7)
    d["beta"][0, ::3] = 0.0
    d["beta"][0, 64:128, 1] = 0.0
    for f in (chunk_gated_delta, recurrent_gated_delta):
        check_forward(d, f, None)
    got = check_backward(d)
    assert (got["dv"][0, ::3] == 0).all() and (got["dv"][0, 64:128, 1] == 0).all()
    assert (got["dbeta"][0, ::3].abs() > 0).all()


def test_non_finite_stays_in_its_head_and_chunk():
    """A NaN reaches its own head from its chunk's start on: not earlier chunks, other heads or sequences."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta, chunk_gated_delta_bwd

    g = dev(make(1, 400, 2, 2, 64, 64, BF16, lens=[130, 270], seed=6))
    o, ht = on(g, chunk_gated_delta, output_final_state=True)
    grad = on(g, chunk_gated_delta_bwd, g["do"], dht=g["dht"])
    for name in ("v", "k", "q", "g", "beta"):
        b = {x: None if t is None else t.clone() for x, t in g.items()}
        b[name][0, 130 + 70, 1] = float("nan")
        o2, h2 = on(b, chunk_gated_delta, output_final_state=True)
        assert torch.equal(o[:, :130], o2[:, :130]) and torch.equal(o[:, :, 0], o2[:, :, 0]), name
        assert torch.equal(o[0, 130:194, 1], o2[0, 130:194, 1]), name
        assert not torch.isfinite(o2[0, 200, 1]).any(), name
        assert torch.equal(ht[0], h2[0]) and torch.equal(ht[1, 0], h2[1, 0]), name
        grad2 = on(b, chunk_gated_delta_bwd, b["do"], dht=b["dht"])
        for x in ("dq", "dk", "dv", "dg", "dbeta"):
            assert torch.equal(grad[x][:, :130], grad2[x][:, :130]), (name, x)
            assert torch.equal(grad[x][:, :, 0], grad2[x][:, :, 0]), (name, x)


def test_rows_outside_the_offsets():
    """Rows before the first offset and behind the last are neither read nor written, gradients included."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta, lib
    from gated_delta_rule_gate_amd import _delta, _linear

    d = make(1, 300, 4, 2, 64, 64, BF16, lens=[70, 100], seed=7)
    d["cu"] += 20
    for x in ("q", "k", "v", "g", "beta", "do"):
        d[x][0, :20] = float("nan")
        d[x][0, 190:] = float("nan")
    g = dev(d)
    out = torch.full_like(g["v"], 7.0)
    o, _ = on(g, chunk_gated_delta, out=out)
    inner = [x[:, 20:190] if i < 5 else x for i, x in enumerate(inputs64(d))]
    want, size = ref.delta(*inner, cu=d["cu"] - 20), ref.sizes(*inner, cu=d["cu"] - 20)
    within(o[:, 20:190], want[0], size[0], BF16, ref.roundings(64, 64, 300), "o", ref.LEFT_OUT[BF16])
    assert (o[:, :20] == 7.0).all() and (o[:, 190:] == 7.0).all()
    # the C entry, with gradients that hold a mark and a workspace of NaN
    a, _, i, ptrs = _delta._delta_args(*[g[x] for x in IN], g["cu"], None)
    marks = [torch.full_like(g[x], 7.0) for x in ("q", "k", "v", "g", "beta")]
    need = lib().kda_delta_chunk_bwd_workspace_bytes(a)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    _linear._launch(i, lib().kda_delta_chunk_bwd, a, *ptrs, g["do"].data_ptr(), g["dht"].data_ptr(),
                    *[m.data_ptr() for m in marks], None, ws.data_ptr(), need)
    for m in marks:
        assert (m[:, :20] == 7.0).all() and (m[:, 190:] == 7.0).all()
        assert torch.isfinite(m[:, 20:190]).all()


@pytest.mark.parametrize("which", ["q", "v", "h0", "k", "beta", "g"])
def test_gradient_against_differences(which):
    """Central differences along a random direction. In q, v and h0 alone the loss is linear; in k, beta and g
    it is smooth, and a step h leaves h^2 times the third derivative: two steps, extrapolated, leave h^4."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta, chunk_gated_delta_bwd

    d = make(1, 150, 2, 1, 72, 40, FP32, seed=8)
    g = dev(d)
    step = torch.from_numpy(np.random.Generator(np.random.PCG64(9)).standard_normal(tuple(d[which].shape)).astype(np.float32))
    step = step / step.norm() * 4.0

    def loss(sign):
        # in 64 bits the steps are exact: x + h d rounded once, and the difference taken from what was rounded
        m = dict(g, **{which: (g[which] + sign * step.cuda())})
        o, ht = on(m, chunk_gated_delta, output_final_state=True)
        return ((o.double() * m["do"].double()).sum() + (ht.double() * m["dht"].double()).sum()).item()

    got = on(g, chunk_gated_delta_bwd, g["do"], dht=g["dht"])["d" + which]
    along = (got.double() * step.cuda().double()).sum().item()
    so, sh = ref.sizes(*inputs64(d))
    size = (so * f64(d["do"]).norm(dim=-1)).sum().item() + (sh * f64(d["dht"]).flatten(2).norm(dim=-1)).sum().item()
    noise = 3 * ref.roundings(72, 40, 150) * ref.ULP32 * size
    if which in ("q", "v", "h0"):
        assert abs((loss(1) - loss(-1)) / 2 - along) <= noise
        return
    # the same differences of the 64-bit definition say what the steps themselves leave
    h = 1 / 8

    def exact(sign):
        args = dict(zip(IN, inputs64(d)))
        args[which] = f64(g[which] + sign * step.cuda())
        o, ht = ref.delta(*[args[x] for x in IN])
        return ((o * f64(d["do"])).sum() + (ht * f64(d["dht"])).sum()).item()

    mine, true = (loss(h) - loss(-h)) / (2 * h), (exact(h) - exact(-h)) / (2 * h)
    assert abs(mine - true) <= noise / h
    want = ref.grads(*inputs64(d), f64(d["do"]), f64(d["dht"]))[IN.index(which)]
    at = (want * step.double()).sum().item()
    assert abs(true - at) <= 0.05 * abs(at) + 0.05 * want.norm().item()  # the definition's own step error is small
    assert abs(along - at) <= noise


def test_long_offsets():
    """Offsets that pass 32 bits: token offsets times heads and widths in a packed batch, forward and backward."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta, chunk_gated_delta_bwd

    H, K, V, T = 128, 8, 128, 135000  # 2.2e9 elements of v
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k = (torch.zeros(1, T, 1, K, dtype=BF16, device="cuda") for _ in range(2))
    v, do = (torch.zeros(1, T, H, V, dtype=BF16, device="cuda") for _ in range(2))
    for x in (q, k, v, do):
        x[:, -164:] = (torch.randn(1, 164, *x.shape[2:], device="cuda", generator=gen) * 0.3).to(BF16)
    g = torch.full((1, T, H), -0.1, device="cuda")
    beta = torch.full((1, T, H), 0.5, device="cuda")
    cu = torch.tensor([0, T - 100, T], dtype=torch.int32, device="cuda")
    o, ht = chunk_gated_delta(q, k, v, g, beta, cu_seqlens=cu, output_final_state=True)
    tail = [x[:, -100:].contiguous() for x in (q, k, v, g, beta)]
    o1, h1 = chunk_gated_delta(*tail, output_final_state=True)
    assert torch.equal(o[:, -100:], o1) and torch.equal(ht[1], h1[0])
    got = chunk_gated_delta_bwd(q, k, v, g, beta, do, cu_seqlens=cu)
    want = chunk_gated_delta_bwd(*tail, do[:, -100:].contiguous())
    for x in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(got[x][:, -100:], want[x]), x
    assert torch.equal(got["dh0"][1], want["dh0"][0])


def test_long_state_offsets():
    """States whose offsets pass 32 bits, updated in place token by token."""
    need_gpu()
    from gated_delta_rule_gate_amd import recurrent_gated_delta

    N, H, K = 1025, 32, 256  # 2.15e9 elements
    gen = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (torch.randn(N, 1, H, K, device="cuda", generator=gen).mul_(0.06).to(BF16) for _ in range(3))
    g, beta = -torch.rand(N, 1, H, device="cuda", generator=gen), torch.rand(N, 1, H, device="cuda", generator=gen)
    h = torch.empty(N, H, K, K, device="cuda")
    h[-2:] = torch.randn(2, H, K, K, device="cuda", generator=gen)
    h[:-2] = 0
    alone = h[-1:].clone()
    o, _ = recurrent_gated_delta(q, k, v, g, beta, h, final_state=h)
    o1, h1 = recurrent_gated_delta(*[x[-1:].contiguous() for x in (q, k, v, g, beta)], alone, output_final_state=True)
    # one sequence runs by 32 columns, all of them by 128: sums over K in another order
    size = 0.06 * 16 * (alone.norm() + 1.0).double().cpu()
    assert ((o[-1].double() - o1[0].double()).abs().cpu() <= ref.HALF[BF16] * 2 * o1[0].double().abs().cpu() + 600 * ref.ULP32 * size).all()
    assert ((h[-1] - h1[0]).abs().cpu() <= 600 * ref.ULP32 * size).all()


@pytest.mark.parametrize("T", [130, 1500])
def test_graph_replays(T):
    """Captured forward, gradient and recurrence; replays with new inputs and offsets equal eager calls."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta, chunk_gated_delta_bwd, recurrent_gated_delta

    g = dev(make(1, T, 2, 1, 64, 64, BF16, lens=[T // 3, T - T // 3], seed=11))

    def step():
        o, ht = on(g, chunk_gated_delta, output_final_state=True)
        b = on(g, chunk_gated_delta_bwd, g["do"], dht=g["dht"])
        r = recurrent_gated_delta(*[g[x][:, :1].contiguous() for x in IN[:5]], ht[:1].contiguous())
        return [o, ht] + list(b.values()) + [r[0]]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for turn in range(3):
        g["v"].copy_(torch.randn_like(g["v"], dtype=FP32).to(BF16))
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
    from gated_delta_rule_gate_amd import chunk_gated_delta, chunk_gated_delta_bwd

    g = dev(make(1, 1300, 2, 2, 64, 128, BF16, seed=30))
    fwd = lambda: list(on(g, chunk_gated_delta, output_final_state=True))  # noqa: E731
    bwd = lambda: list(on(g, chunk_gated_delta_bwd, g["do"], dht=g["dht"]).values())  # noqa: E731
    fwd(), bwd()
    torch.cuda.synchronize()
    graphs = []
    for f in (fwd, bwd):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = f()
        graphs.append((graph, held, f))
    for _ in range(3):
        g["v"].mul_(1.25)
        for graph, held, f in graphs + graphs[::-1]:
            want = f()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_two_streams_with_workspaces_of_their_own():
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta, chunk_gated_delta_bwd, gated_delta_workspace_bytes

    sets = [dev(make(1, 2000, 2, 2, 128, 128, BF16, seed=20 + i)) for i in range(2)]
    runs = [lambda g, w: list(on(g, chunk_gated_delta, output_final_state=True, workspace=w)),
            lambda g, w: list(on(g, chunk_gated_delta_bwd, g["do"], dht=g["dht"], workspace=w).values())]
    for back, run in enumerate(runs):
        want = [run(g, None) for g in sets]
        ws = [torch.empty(gated_delta_workspace_bytes(g["q"], g["k"], g["v"], backward=bool(back)), dtype=torch.uint8,
                          device="cuda") for g in sets]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in sets]
        got = []
        for g, s, w in zip(sets, streams, ws):
            with torch.cuda.stream(s):
                got.append(run(g, w))
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for a, b in zip(got, want) for x, y in zip(a, b))


def test_prompt_then_tokens():
    """A prompt through the chunked form, then tokens one by one on the state it left: the whole sequence."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta, recurrent_gated_delta

    d = make(2, 133, 4, 2, 128, 64, BF16, seed=12)
    g = dev(d)
    cut = lambda lo, hi: [g[x][:, lo:hi].contiguous() for x in IN[:5]]  # noqa: E731
    o, st = chunk_gated_delta(*cut(0, 128), g["h0"], output_final_state=True)
    rows = [o]
    for t in range(128, 133):
        rows.append(recurrent_gated_delta(*cut(t, t + 1), st, final_state=st)[0])
    want, size = ref.delta(*inputs64(d)), ref.sizes(*inputs64(d))
    n = ref.roundings(128, 64, 133)
    within(torch.cat(rows, 1), want[0], size[0], BF16, n, "o", ref.LEFT_OUT[BF16])
    within(st, want[1], size[1], FP32, n, "state")


@pytest.mark.parametrize("lens", [None, [700, 0, 123, 300]], ids=["dense", "packed"])
def test_calls_repeat_themselves(lens):
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta, chunk_gated_delta_bwd

    T = 1123
    g = dev(make(1, T, 6, 3, 128, 128, BF16, lens=lens, seed=60))
    one = lambda: list(on(g, chunk_gated_delta, output_final_state=True)) + list(  # noqa: E731
        on(g, chunk_gated_delta_bwd, g["do"], dht=g["dht"]).values())
    first = one()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, one()))


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(1, 700, 4, 2, 128, 128, None), (1, 500, 2, 2, 256, 64, [300, 200]), (2, 333, 3, 3, 64, 256, None)],
                         ids=_id)
def test_errors(shape, dtype):
    """Errors as fp32's, in the 2-norm of a whole tensor: roundings of either sign add up by their squares, so
    n of them leave sqrt(n) 2^-24 of the terms. A part of 8 bits left out would leave 2^-16 or more. The terms
    behind a result are taken as four times its norm (K, V and a chunk's 64 rows make n; dg, a difference of
    two such sums, as sixteen times)."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta, chunk_gated_delta_bwd

    B, T, H, Hk, K, V, lens = shape
    d = make(B, T, H, Hk, K, V, dtype, lens, seed=70)
    g, do, dht = dev(d), f64(d["do"]), f64(d["dht"])
    o, ht = on(g, chunk_gated_delta, output_final_state=True)
    got = dict(on(g, chunk_gated_delta_bwd, g["do"], dht=g["dht"]), o=o, ht=ht)
    want = dict(zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), ref.grads(*inputs64(d), do, dht, cu=d["cu"])))
    want.update(zip(("o", "ht"), ref.delta(*inputs64(d), cu=d["cu"])))
    for name, w in want.items():
        off = ((f64(got[name]) - w).norm() / w.norm()).item()
        most = (K + V + 64) ** 0.5 * ref.ULP32 * (16 if name == "dg" else 4)
        if got[name].dtype == BF16:  # one rounding, evenly spread over half a step: 1/sqrt(3) of the largest
            most += ref.HALF[BF16] / 3 ** 0.5
        assert off <= most, (name, off, most)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_first_decay_of_a_sequence_from_zero(dtype):
    """It scales a state of zeros: its gradient is zero, not what rounding leaves of the sums. Decays of sequences
    with a start state, and all later ones, have one."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta_bwd

    lens = [1, 70, 0, 1, 2]
    d = make(1, sum(lens), 3, 3, 64, 64, dtype, lens=lens, states=False)
    at = [0, 1, 71, 72]
    dg = on(dev(d), chunk_gated_delta_bwd, dev(d)["do"])["dg"].cpu()
    assert (dg[0, at] == 0).all()
    rest = [i for i in range(sum(lens)) if i not in at]
    assert (dg[0, rest] != 0).all()
    d["h0"] = torch.ones(len(lens), 3, 64, 64)
    dg = on(dev(d), chunk_gated_delta_bwd, dev(d)["do"])["dg"].cpu()
    assert (dg[0, at] != 0).all()


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("lens", [None, [100, 1500, 0, 400]], ids=["dense", "packed"])
def test_long_heads_of_every_decay(lens, dtype):
    """Heads side by side whose segments leave all of the state before them, some of it, nothing, and a head that
    is reset here and there."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta

    d = make(1, 2000, 4, 2, 64, 72, dtype, lens, seed=81, strength=1.0)
    d["g"] *= torch.tensor([0.0, 0.01, 3.0, 0.02])
    d["g"][0, 333::500, 3] = -float("inf")
    o, ht, inside = check_forward(d, chunk_gated_delta, None)
    g = dev(d)
    o2, h2 = on(g, chunk_gated_delta, final_state=g["h0"])
    assert torch.equal(o2[:, inside], o[:, inside]) and torch.equal(h2, ht)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_long_rows_hold_up_the_decays(dtype):
    """One key of norm 2 and beta 0.9: a step takes the state's part along it times 1 - 3.6, and decays of 1 / 2.6
    leave it as it is for good, though they sum to far under what counts as zero.

    Bound. Along the key a step's size is one, across it less, so roundings add up as with short rows; but a
    written row is |k| |u|, |u| <= |v| + |k| M, and an entry of the chunk's inverse at most 3.6 instead of one:
    sizes times 16."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta

    d = make(1, 1500, 2, 2, 8, 64, dtype, seed=82)
    d["k"][:] = 0
    d["k"][..., 3] = 2.0
    d["q"][:] = 0
    d["q"][..., 3] = 1.0
    d["beta"][:] = 0.9
    d["g"][:] = -float(np.log(2.6))
    d["v"] *= 0.01  # so that the start still counts at the end
    g = dev(d)
    o, ht = on(g, chunk_gated_delta, output_final_state=True)
    want, size = ref.delta(*inputs64(d)), ref.sizes(*inputs64(d))
    assert want[1][0, :, 3].norm() > 0.2 * d["h0"][0, :, 3].norm()
    n = ref.roundings(8, 64, 1500)
    within(o, want[0], 16 * size[0], dtype, n, "o", ref.LEFT_OUT[dtype])
    within(ht, want[1], 16 * size[1], FP32, n, "ht")


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("K", [8, 72, 136, 192, 200, 256])
def test_chunks_of_one_row(K, dtype):
    """Every width of key rows with a last chunk of one token, alone in its sequence or not."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta

    d = make(1, 98, 2, 1, K, 24, dtype, lens=[65, 33], seed=83)
    check_forward(d, chunk_gated_delta, None)
    check_backward(d)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_long_backward(dtype):
    """Many chunks, on heads that forget nothing, a little, and all of it."""
    need_gpu()
    d = make(1, 1100, 3, 3, 64, 40, dtype, seed=84, strength=1.0)
    d["g"] *= torch.tensor([0.0, 0.01, 3.0])
    check_backward(d)
