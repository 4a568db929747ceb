"""The block norm (norm, gate, residual and scale, next norm) and its gradients on the GPU against
the 64-bit definition, differentiated, over row widths, types and every combination of its parts.

Tolerances count fp32 roundings: a row's statistic is a sum of D squares (D + 8 roundings of its
relative size, halved by the root), an activation is off by a few more; every value then passes
about a dozen products. The terms' sizes come with the reference."""
import itertools

import numpy as np
import pytest
import torch

import linear_ref as ref
from kda_testlib import need_gpu

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


def make(rows, D, dtype, res, gate, scale, nxt, weights=True, seed=0):
    r = np.random.Generator(np.random.PCG64(seed + D + rows))
    f = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32))  # noqa: E731
    rt = res if res is not None else dtype
    return dict(x=f(rows, D).to(dtype), weight=1 + 0.1 * f(D) if weights else None,
                gate=f(rows, D).to(dtype) if gate else None,
                residual=f(rows, D).to(res) if res is not None else None,
                scale=0.5 + 0.1 * f(D) if scale == "channel" else scale,
                next_weight=1 + 0.1 * f(D) if nxt and weights else None,
                dy=f(rows, D).to(rt), dz=f(rows, D).to(dtype) if nxt else None)


def on(d, dev="cuda"):
    return {k: v.to(dev) if isinstance(v, torch.Tensor) else v for k, v in d.items()}


NAMES = ("x", "weight", "gate", "residual", "scale", "next_weight")


def reference(d, act, nxt, eps, kind):
    """Outputs and gradients by name in float64, and the sizes of the terms behind the gradients."""
    t = {k: d[k].double().requires_grad_(True) for k in NAMES if isinstance(d[k], torch.Tensor)}
    g = lambda k: t.get(k)  # noqa: E731
    scale = t["scale"] if "scale" in t else (1.0 if d["scale"] is None else d["scale"])
    outs = ref.norm(t["x"], g("weight"), g("gate"), act, g("residual"), scale, g("next_weight"), nxt, eps, kind)
    grads = torch.autograd.grad(sum((o * d[n].double()).sum() for o, n in zip(outs, ("dy", "dz")) if d[n] is not None),
                                list(t.values()))
    return [o.detach() for o in outs], dict(zip(("d" + k for k in t), grads))


def sizes(d, act, nxt, eps, kind):
    """Sums of the absolute terms behind each gradient, by the formulas of the backward."""
    D = d["x"].shape[-1]
    a = lambda k: d[k].double().abs() if isinstance(d[k], torch.Tensor) else 1.0  # noqa: E731
    x, w, w2 = a("x"), a("weight"), a("next_weight")
    c = a("scale") if isinstance(d["scale"], torch.Tensor) else abs(1.0 if d["scale"] is None else d["scale"])
    m = D if kind == "rms" else 1
    rho = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / m + eps)
    gate = d["gate"].double() if d["gate"] is not None else None
    sig = torch.sigmoid(gate) if gate is not None else 1.0
    actv = sig * (gate.abs() if act == "silu" else 1.0) if gate is not None else 1.0
    dact = (sig * (1 + gate.abs()) if act == "silu" else sig) if gate is not None else 0.0
    n = x * rho * w
    y = a("residual") * (1.0 if d["residual"] is not None else 0.0) + c * n * actv
    t = a("dy") if d["dy"] is not None else torch.zeros_like(x)
    out = {}
    if nxt:
        real = reference(d, act, nxt, eps, kind)[0][0]
        rho2 = 1 / torch.sqrt((real * real).mean(-1, keepdim=True) + eps)
        dz = a("dz")
        out["dnext_weight"] = (dz * y * rho2).sum(0)
        t = t + rho2 * (dz * w2 + y * rho2 ** 2 * (w2 * dz * y).mean(-1, keepdim=True))
    out["dresidual"] = t
    out["dscale"] = (t * n * actv).sum(0)
    out["dgate"] = t * c * n * dact
    dn = t * c * actv
    out["dweight"] = (dn * x * rho).sum(0)
    out["dx"] = rho * (w * dn + x * rho ** 2 * (w * dn * x).sum(-1, keepdim=True) / m)
    return out, (y, y * (rho2 if nxt else 1.0) * w2)


def check(got, want, size, dtype, n, what):
    got, want = got.detach().cpu().double(), want
    assert got.shape == want.shape and torch.isfinite(got).all(), what
    tol = ref.HALF[dtype] * want.abs() + n * ref.ULP32 * size * 1.01
    off = (got - want).abs()
    assert (off <= tol).all(), "%s: off by %.3g times the tolerance" % (what, (off / tol.clamp_min(1e-300)).max())


def count(D, rows, nxt):
    """Roundings: a statistic over D values (twice with the next norm), about 32 products, a sum over rows."""
    return (D + 32) * (2 if nxt else 1) + 32


def run_both(d, act, nxt, eps=1e-6, kind="rms"):
    from gated_delta_rule_gate_amd import block_norm, block_norm_bwd

    g = on(d)
    kw = dict(gate=g["gate"], gate_act=act, residual=g["residual"], scale=g["scale"], next_weight=g["next_weight"],
              eps=eps, norm=kind)
    rows, D = d["x"].shape
    outs = block_norm(g["x"], g["weight"], next_norm=nxt, **kw)
    outs = list(outs) if nxt else [outs]
    want, grads = reference(d, act, nxt, eps, kind)
    size, osize = sizes(d, act, nxt, eps, kind)
    n = count(D, rows, nxt)
    rt = d["residual"].dtype if d["residual"] is not None else d["x"].dtype
    for o, w, s, t in zip(outs, want, osize, (rt, d["x"].dtype)):
        check(o, w, s, t, n, "y or z")
    got = block_norm_bwd(g["x"], g["dy"], g["weight"], dz=g["dz"], **kw)
    for name, w in grads.items():
        t = got[name].dtype
        extra = rows if name in ("dweight", "dscale", "dnext_weight") else 0
        check(got[name], w, size[name], t, n + extra, name)
    assert {k for k, v in got.items() if v is not None} == set(grads)
    return outs, got


@pytest.mark.parametrize("D", [8, 16, 24, 40, 64, 128, 200, 256, 512, 520, 1024, 1032, 2048, 2056, 4096, 5000, 8192, 8200,
                               16384])
def test_widths(D):
    need_gpu()
    d = make(37, D, BF16, FP32, True, "channel", True)
    run_both(d, "silu", True)


@pytest.mark.parametrize("dtype,res", [(BF16, None), (BF16, BF16), (BF16, FP32), (FP32, None), (FP32, FP32)])
@pytest.mark.parametrize("gate,scale,nxt", list(itertools.product([False, True], [None, 0.25, "channel"], [False, True])))
def test_parts(dtype, res, gate, scale, nxt):
    need_gpu()
    act = "silu" if scale == 0.25 else "sigmoid"
    run_both(make(19, 128, dtype, res, gate, scale, nxt), act, nxt)


@pytest.mark.parametrize("kind", ["rms", "l2"])
@pytest.mark.parametrize("rows,D", [(1, 64), (5, 72), (3, 4096), (3000, 128), (70001, 8), (1200, 2056)])
def test_rows_without_weights(rows, D, kind):
    need_gpu()
    run_both(make(rows, D, FP32, None, True, None, True, weights=False), "sigmoid", True, eps=1e-5, kind=kind)


@pytest.mark.parametrize("dtype,res", [(BF16, None), (BF16, BF16), (BF16, FP32), (FP32, FP32)])
def test_no_rows(dtype, res):
    """A batch without rows: empty outputs, and weights' gradients of zero."""
    need_gpu()
    from gated_delta_rule_gate_amd import block_norm, block_norm_bwd

    d = on(make(0, 136, dtype, res, True, "channel", True))
    common = dict(weight=d["weight"], gate=d["gate"], residual=d["residual"], scale=d["scale"],
                  next_weight=d["next_weight"])
    y, z = block_norm(d["x"], **common)
    assert y.shape == z.shape == (0, 136) and y.dtype == (res or dtype) and z.dtype == dtype
    # a workspace of NaN: every part that is summed has to be written
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
    got = block_norm_bwd(d["x"], d["dy"], dz=d["dz"], workspace=ws, **common)
    assert got["dx"].shape == (0, 136)
    for n in ("dweight", "dscale", "dnext_weight"):
        assert got[n].shape == (136,) and not got[n].any(), n


def test_only_the_next_gradient():
    """dy may be left out beside dz."""
    need_gpu()
    from gated_delta_rule_gate_amd import block_norm_bwd

    d = make(40, 256, BF16, BF16, False, None, True)
    d["dy"] = None
    want = reference(d, "sigmoid", True, 1e-6, "rms")[1]
    size = sizes(d, "sigmoid", True, 1e-6, "rms")[0]
    g = on(d)
    got = block_norm_bwd(g["x"], None, g["weight"], dz=g["dz"], residual=g["residual"], next_weight=g["next_weight"])
    for name, w in want.items():
        check(got[name], w, size[name], got[name].dtype, count(256, 40, True) + 40, name)


def test_zero_rows_and_zero_values():
    need_gpu()
    from gated_delta_rule_gate_amd import block_norm, block_norm_bwd

    x = torch.zeros(0, 64, dtype=BF16, device="cuda")
    w = torch.ones(64, device="cuda")
    assert block_norm(x, w).shape == (0, 64)
    got = block_norm_bwd(x, x, w)
    assert got["dx"].shape == (0, 64) and (got["dweight"] == 0).all()
    x = torch.zeros(5, 64, dtype=BF16, device="cuda")
    y, z = block_norm(x, w, next_norm=True)
    assert (y == 0).all() and (z == 0).all()


def test_in_place_residual():
    need_gpu()
    from gated_delta_rule_gate_amd import block_norm

    g = on(make(33, 2304, BF16, FP32, False, 0.5, True))
    kw = dict(scale=0.5, next_weight=g["next_weight"])
    y, z = block_norm(g["x"], g["weight"], residual=g["residual"], **kw)
    y2, z2 = block_norm(g["x"], g["weight"], residual=g["residual"], out=g["residual"], **kw)
    assert y2 is g["residual"] and torch.equal(y, y2) and torch.equal(z, z2)


def test_one_row_does_not_touch_another():
    """NaN in one row stays there."""
    need_gpu()
    from gated_delta_rule_gate_amd import block_norm

    for D in (40, 128, 1024, 4096):
        g = on(make(33, D, BF16, None, True, None, False))
        y = block_norm(g["x"], g["weight"], gate=g["gate"])
        g["x"][7, 3] = float("nan")
        y2 = block_norm(g["x"], g["weight"], gate=g["gate"])
        keep = torch.arange(33, device="cuda") != 7
        assert torch.equal(y[keep], y2[keep]) and torch.isnan(y2[7]).all()


def test_graph_replays():
    need_gpu()
    from gated_delta_rule_gate_amd import block_norm, block_norm_bwd

    g = on(make(300, 1032, BF16, BF16, True, "channel", True))
    kw = dict(gate=g["gate"], residual=g["residual"], scale=g["scale"], next_weight=g["next_weight"])

    def step():
        y, z = block_norm(g["x"], g["weight"], **kw)
        b = block_norm_bwd(g["x"], g["dy"], g["weight"], dz=g["dz"], **kw)
        return [y, z] + [b[k] for k in sorted(b)]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(3):
        g["x"].copy_(torch.randn(300, 1032, device="cuda").to(BF16))
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_gradient_against_differences():
    """Along a direction d, L(x + h d) - L(x - h d) over 2h differs from <dx, d> by h^2 / 6 of L's third
    derivative and the losses' rounding over h. The third derivative along d is taken from the 64-bit
    definition by differentiating three times, at its largest over the step."""
    need_gpu()
    from gated_delta_rule_gate_amd import block_norm, block_norm_bwd

    d = make(6, 64, FP32, FP32, True, "channel", True, seed=3)
    g = on(d)
    kw = dict(gate_act="silu", gate=g["gate"], residual=g["residual"], scale=g["scale"], next_weight=g["next_weight"])
    got = block_norm_bwd(g["x"], g["dy"], g["weight"], dz=g["dz"], **kw)
    h = 2.0 ** -7
    for which in ("x", "gate", "residual"):
        step = torch.from_numpy(np.random.Generator(np.random.PCG64(4)).standard_normal((6, 64)).astype(np.float32))

        def loss(s):
            m = dict(g, **{which: g[which] + s * h * step.cuda()})
            y, z = block_norm(m["x"], m["weight"], **dict(kw, gate=m["gate"], residual=m["residual"]))
            return ((y.double() * m["dy"].double()).sum() + (z.double() * m["dz"].double()).sum()).item()

        def third(at):
            u = torch.tensor(at, dtype=torch.float64, requires_grad=True)
            m = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in d.items()}
            m[which] = m[which] + u * step.double()
            y, z = ref.norm(m["x"], m["weight"], m["gate"], "silu", m["residual"], m["scale"], m["next_weight"], True,
                            1e-6, "rms")
            L = (y * m["dy"]).sum() + (z * m["dz"]).sum()
            for _ in range(3):
                (L,) = torch.autograd.grad(L, u, create_graph=True)
            return abs(L.item())

        cubic = 2 * max(third(i * h / 4) for i in range(-4, 5))  # twice the largest of nine points
        (sy, sz) = sizes(d, "silu", True, 1e-6, "rms")[1]
        size = ((sy * d["dy"].double().abs()).sum() + (sz * d["dz"].double().abs()).sum()).item()
        gsize = (sizes(d, "silu", True, 1e-6, "rms")[0]["d" + which] * step.double().abs()).sum().item()
        n = count(64, 6, True)
        tol = h * h / 6 * cubic + n * ref.ULP32 * (1.1 * size / h + gsize)
        diff = (loss(1) - loss(-1)) / (2 * h)
        along = (got["d" + which].double() * step.cuda().double()).sum().item()
        assert abs(diff - along) <= tol, (which, diff, along, tol)


def test_layer_as_used():
    """A run of the operators as a layer calls them: l2-normalised q and k rows, linear attention (and KDA
    on the same rows), the gated output norm, the residual stream with the next norm, against 64 bits."""
    need_gpu()
    from gated_delta_rule_gate_amd import block_norm, chunk_kda, chunk_linear_attn

    B, T, H, K = 2, 70, 2, 64
    r = np.random.Generator(np.random.PCG64(5))
    f = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32))  # noqa: E731
    q, k, v, gate = (f(B, T, H, K) for _ in range(4))
    g, w, w1, w2, x = -0.3 * f(B, T, H).abs(), 1 + 0.1 * f(K), 1 + 0.1 * f(H * K), 1 + 0.1 * f(H * K), f(B, T, H * K)
    c = lambda t: t.cuda()  # noqa: E731
    qn, kn = block_norm(c(q), norm="l2"), block_norm(c(k), norm="l2")
    o, _ = chunk_linear_attn(qn, kn, c(v), c(g))
    n = block_norm(o, c(w), gate=c(gate))
    y, z = block_norm(n.view(B, T, H * K), c(w1), residual=c(x), scale=0.5, next_weight=c(w2))
    d = lambda t: t.double()  # noqa: E731
    qr, kr = (ref.norm(d(t), None, None, "sigmoid", None, 1.0, None, False, 1e-6, "l2")[0] for t in (q, k))
    orf, _ = ref.attn(qr, kr, d(v), d(g), None)
    nr = ref.norm(orf, d(w), d(gate), "sigmoid", None, 1.0, None, False, 1e-6, "rms")[0]
    yr, zr = ref.norm(nr.reshape(B, T, H * K), d(w1), None, "sigmoid", d(x), 0.5, d(w2), True, 1e-6, "rms")
    # attention rows whose terms cancel are small beside them: their norm takes that relative error on
    osize, _ = ref.attn_sizes(qr, kr, d(v), d(g), None)
    rel = (ref.roundings(K, K, T) + 3 * (K + 40)) * ref.ULP32 * osize.norm(dim=-1) / orf.norm(dim=-1)
    worst = rel.max().item() + 3 * count(H * K, 1, True) * ref.ULP32
    for got, want in ((y, yr), (z, zr)):
        off = (got.cpu().double() - want).norm(dim=-1)
        assert (off <= 4 * worst * (nr.reshape(B, T, H * K).norm(dim=-1) + want.norm(dim=-1))).all()
    # the same rows through KDA: the norms feed it as they feed linear attention
    A, dt = torch.zeros(H, device="cuda"), torch.zeros(H, K, device="cuda")
    ok, _ = chunk_kda(qn, kn, c(v), c(f(B, T, H, K)), torch.sigmoid(c(f(B, T, H))), A_log=A, dt_bias=dt)
    assert torch.isfinite(block_norm(ok, c(w), gate=c(gate))).all()


@pytest.mark.parametrize("nxt", [False, True])
@pytest.mark.parametrize("rows,D", [(5, 8), (37, 8), (5, 128), (37, 128), (5, 512), (37, 512), (3, 520)])
def test_without_eps(rows, D, nxt):
    """eps = 0: the places past the last row in a workgroup of several rows hold zeros, whose norm is no
    number; they enter no sum."""
    need_gpu()
    for kind in ("rms", "l2"):
        run_both(make(rows, D, BF16, FP32, True, "channel", nxt), "silu", nxt, eps=0.0, kind=kind)


def test_infinite_gate_in_the_last_row():
    """An infinite gate makes its own column's sums infinite and leaves the others finite: what stands past
    the last row in a workgroup of several rows enters no sum."""
    need_gpu()
    from gated_delta_rule_gate_amd import block_norm_bwd

    d = make(5, 128, FP32, None, True, "channel", False)
    d["gate"][4, 9] = float("inf")
    g = on(d)
    got = block_norm_bwd(g["x"], g["dy"], g["weight"], gate=g["gate"], gate_act="silu", scale=g["scale"])
    for n in ("dweight", "dscale"):
        assert torch.isinf(got[n][9]), n
        assert torch.isfinite(torch.cat([got[n][:9], got[n][10:]])).all(), n


def test_more_rows_than_a_launch_has_workgroups():
    """A launch's threads are counted in 32 bits: 2^25 rows of a 128-thread workgroup each go through twice."""
    need_gpu()
    from gated_delta_rule_gate_amd import block_norm

    D, most = 520, (2 ** 32 - 1) // 128
    rows = most + 70
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 90e9:
        pytest.skip("needs 70 GB of GPU memory")
    x = torch.empty(rows, D, dtype=BF16, device="cuda").fill_(0.5)
    y = torch.empty_like(x).fill_(float("nan"))
    w = torch.from_numpy(np.random.Generator(np.random.PCG64(8)).standard_normal(D).astype(np.float32)).cuda()
    at = [0, 1, 69, 70, most - 1, most, most + 1, rows - 1]
    own = torch.from_numpy(np.random.Generator(np.random.PCG64(9)).standard_normal((len(at), D)).astype(np.float32))
    own = own.to(BF16).cuda()
    for i, r in zip(at, own):
        x[i].copy_(r)
    block_norm(x, w, out=y)
    assert torch.equal(torch.stack([y[i] for i in at]), block_norm(own, w))
    rest = block_norm(torch.full((1, D), 0.5, dtype=BF16, device="cuda"), w)
    other = sum((y[i:i + (1 << 22)] != rest).any(-1).sum().item() for i in range(0, rows, 1 << 22))
    assert other == len(at)
    del x, y
    torch.cuda.empty_cache()


def walk_of(rows, D):
    """(rows of a workgroup at a time, the most rows that one of its lanes adds up)."""
    lanes = 1
    while lanes < 512 and lanes * 8 < D:
        lanes *= 2
    at_once = max(1, 256 // lanes) if lanes < 128 else 1
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    blocks = min(-(-rows // at_once), cus * (1 if D > 4096 else 1024 // lanes if D > 512 else 4))
    return at_once, -(-rows // (blocks * at_once))


@pytest.mark.parametrize("rows,D,dtype,res", [
    (300007, 8, BF16, FP32), (40001, 64, FP32, FP32), (16421, 128, BF16, BF16), (9001, 512, BF16, FP32),
    (1500, 1032, BF16, BF16), (1100, 4096, BF16, FP32), (700, 8192, BF16, BF16), (600, 8200, FP32, FP32),
    (300, 16384, BF16, FP32),
])
@pytest.mark.parametrize("nxt", [False, True])
def test_workgroups_that_walk_their_rows(rows, D, dtype, res, nxt):
    """More rows than the workgroups hold at once: each walks several groups of rows, with parameter sums
    over all of them and over more workgroups than are added at a time. A sum passes a rounding for every
    row that its lane adds, and one for each lane that holds the column; over workgroups it is fp64. Leaving
    out one workgroup's rows of one step is outside the tolerance."""
    need_gpu()
    from gated_delta_rule_gate_amd import block_norm, block_norm_bwd

    d = on(make(rows, D, dtype, res, True, "channel", nxt))
    kw = dict(gate=d["gate"], gate_act="silu", residual=d["residual"], scale=d["scale"], next_weight=d["next_weight"])
    want, grads = reference(d, "silu", nxt, 1e-6, "rms")
    size, osize = sizes(d, "silu", nxt, 1e-6, "rms")
    n = count(D, rows, nxt)
    outs = block_norm(d["x"], d["weight"], next_norm=nxt, **kw)
    for o, w, s, t in zip(outs if nxt else [outs], want, osize, (res, dtype)):
        check(o, w.cpu(), s.cpu(), t, n, "y or z")
    got = block_norm_bwd(d["x"], d["dy"], d["weight"], dz=d["dz"], **kw)
    at_once, steps = walk_of(rows, D)
    assert steps > 1
    cut = slice(rows // 2, rows // 2 + at_once)
    part = {k: v[cut] if k in ("x", "gate", "residual", "dy", "dz") and v is not None else v for k, v in d.items()}
    lost = reference(part, "silu", nxt, 1e-6, "rms")[1]
    for name, w in grads.items():
        extra = steps + at_once if name in ("dweight", "dscale", "dnext_weight") else 0
        check(got[name], w.cpu(), size[name].cpu(), got[name].dtype, n + extra, name)
        if extra:
            with pytest.raises(AssertionError, match="times the tolerance"):
                check(got[name], (w - lost[name]).cpu(), size[name].cpu(), got[name].dtype, n + extra, name)
