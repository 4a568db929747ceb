"""What the gated delta rule and the query/key norm refuse, without a GPU: status codes of the C entry points
before any launch, workspace queries, and the Python checks."""
import ctypes
import os

import pytest
import torch

FAKE = ctypes.c_void_p(0x100000)  # aligned, never dereferenced: every call here is refused before a launch
ODD = ctypes.c_void_p(0x100008)
BIG = 1 << 50


@pytest.fixture(scope="module")
def L():
    from gated_delta_rule_gate_amd import _binding, _delta, build

    if not os.path.exists(_binding.LIB_PATH):
        build.build()
    return _delta._lib()


def dl(**kw):
    from gated_delta_rule_gate_amd._delta import DeltaArgs

    a = DeltaArgs(1, 64, 2, 128, 128, 1, 0, 0, 0.0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def qk(**kw):
    from gated_delta_rule_gate_amd._delta import QkArgs

    a = QkArgs(4, 4, 2, 128, 64, 0, 0, 0, 1, (ctypes.c_int * 4)(), 0, 1e-6, 0, 0, 0, 0)
    for k, v in kw.items():
        setattr(a, k, (ctypes.c_int * 4)(*v) if k == "sections" else v)
    return a


def fwd(L, a, p=None, ws=FAKE, n=BIG):
    return L.kda_delta_chunk_fwd(a, *(p or [FAKE] * 5 + [None, None, FAKE, None]), ws, n, None)


def rec(L, a, p=None):
    return L.kda_delta_recurrent_fwd(a, *(p or [FAKE] * 5 + [None, None, FAKE, None]), None)


def bwd(L, a, p=None, grads=None, ws=FAKE, n=BIG):
    return L.kda_delta_chunk_bwd(a, *(p or [FAKE] * 5 + [None, None, FAKE, None]), *(grads or [FAKE] * 5 + [None]), ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), 3), (dict(K=44), 8), (dict(V=264), 8), (dict(K=0), 2), (dict(B=2), 2), (dict(H=0), 2),
    (dict(H=4097), 2), (dict(H=3, Hk=2), 2), (dict(Hk=-1), 2), (dict(T=-1), 2), (dict(N=-1), 2),
])
def test_delta_arguments(L, kw, code):
    a = dl(**kw)
    assert rec(L, a) == code and fwd(L, a) == code and bwd(L, a) == code
    if "B" not in kw:  # N != B is a packed query's right
        assert L.kda_delta_chunk_workspace_bytes(a) == 0 and L.kda_delta_chunk_bwd_workspace_bytes(a) == 0


def test_delta_pointers(L):
    a, good = dl(), [FAKE] * 5 + [None, None, FAKE, None]
    for f in (fwd, rec, bwd):
        for i in (0, 1, 2, 4, 7):  # g (3) may be missing
            p = list(good)
            p[i] = None
            assert f(L, a, p) == 1, (f, i)
        for i in (0, 1, 2, 3, 4, 5, 7, 8):
            p = list(good)
            p[i] = ODD
            assert f(L, a, p) == 6, (f, i)
        assert f(L, None) == 1
        assert f(L, dl(B=2, N=2), [FAKE] * 5 + [None, FAKE, FAKE, None]) == 2  # packed needs one batch
    for i in range(5):
        p = [FAKE] * 5 + [None]
        p[i] = None
        assert bwd(L, a, None, p) == 1, i
        p[i] = ODD
        assert bwd(L, a, None, p) == 6, i
    # without g its gradient is not asked for: what is missing is the workspace
    p = list(good)
    p[3] = None
    assert bwd(L, a, p, [FAKE] * 3 + [None, FAKE, None], None, 0) == 7


def test_delta_workspaces(L):
    a = dl(T=300)
    for query, call in ((L.kda_delta_chunk_workspace_bytes, lambda ws, n: fwd(L, a, None, ws, n)),
                        (L.kda_delta_chunk_bwd_workspace_bytes, lambda ws, n: bwd(L, a, None, None, ws, n))):
        need = query(a)
        assert need > 0 and query(dl(T=0)) == 0
        assert call(None, need) == 7 and call(FAKE, need - 1) == 7
        assert call(ctypes.c_void_p(0x100010), need) == 6


@pytest.mark.parametrize("sizes,chunked,taken", [
    (dict(B=1366, N=1366, H=4096), True, dict(B=1365, N=1365, H=4096)),        # 128 columns: 768 threads
    (dict(B=2048, N=2048, H=4096, V=64), True, dict(B=2047, N=2047, H=4096, V=64)),  # 64 columns: 512 threads
    (dict(B=4096, N=4096, H=4096), False, dict(B=4095, N=4095, H=4096)),       # the recurrence: 256 threads
])
def test_more_workgroups_than_a_launch_takes(L, sizes, chunked, taken):
    """Refused before the first launch, so that no output is written by half; one sequence fewer is taken, and
    the missing workspace is what is wrong."""
    a = dl(T=1, **sizes)
    if not chunked:
        assert rec(L, a) == 8
        return
    assert fwd(L, a) == 8 and bwd(L, a) == 8
    assert fwd(L, dl(T=1, **taken), None, None, 0) == 7


def test_long_batches_that_a_launch_does_not_take(L):
    # the chunks' passes: one workgroup a chunk and head
    assert fwd(L, dl(T=1 << 30, H=4096, Hk=4096), None, None, 0) == 8
    assert bwd(L, dl(T=1 << 30, H=1024), None, None, None, 0) == 8
    assert bwd(L, dl(T=1 << 24, H=8, Hk=4, K=256, V=8), None, None, None, 0) == 8  # the shared heads' sum
    assert bwd(L, dl(T=(1 << 24) - 1, H=8, Hk=4, K=256, V=8), None, None, None, 0) == 7


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), 2), (dict(H=0), 2), (dict(Hk=0), 2), (dict(D=0), 2), (dict(rot=-8), 2), (dict(rot=136), 2),
    (dict(axes=0), 2), (dict(axes=5), 2), (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2), (dict(dtype=2), 3),
    (dict(norm=3), 5), (dict(pairs=2), 5), (dict(D=100, rot=0), 8), (dict(D=520), 8), (dict(rot=20), 8),
    (dict(q_stride=504), 2), (dict(k_stride=8), 2), (dict(q_stride=516), 2), (dict(qo_stride=-512), 2),
    (dict(ko_stride=(1 << 31) + 8), 2),
    (dict(axes=2, sections=(16, 15, 0, 0)), 2), (dict(axes=2, sections=(33, -1, 0, 0)), 2),
    (dict(axes=3, sections=(8, 8, 16, 0), spread=1), 2),  # 2 + 3 * 15 is no frequency of 32
    (dict(axes=2, sections=(16, 8, 8, 0)), 2),
])
def test_qk_arguments(L, kw, code):
    a = qk(**kw)
    assert L.kda_qk_norm_rope_fwd(a, *[FAKE] * 8, None) == code
    assert L.kda_qk_norm_rope_bwd(a, *[FAKE] * 12, FAKE, BIG, None) == code
    assert L.kda_qk_norm_rope_bwd_workspace_bytes(a) == 0


def test_qk_pointers(L):
    a, p = qk(), [FAKE] * 8
    assert L.kda_qk_norm_rope_fwd(None, *p, None) == 1
    for i in (0, 1, 4, 5, 6, 7):
        x = list(p)
        x[i] = None
        assert L.kda_qk_norm_rope_fwd(a, *x, None) == 1, i
    for i in (0, 1, 6, 7):
        x = list(p)
        x[i] = ODD
        assert L.kda_qk_norm_rope_fwd(a, *x, None) == 6, i
    p = [FAKE] * 10 + [None, None]
    for i in (0, 1, 4, 5, 6, 7, 8, 9):
        x = list(p)
        x[i] = None
        assert L.kda_qk_norm_rope_bwd(a, *x, None, 0, None) == 1, i
    for i in (0, 1, 6, 7, 8, 9):
        x = list(p)
        x[i] = ODD
        assert L.kda_qk_norm_rope_bwd(a, *x, None, 0, None) == 6, i
    need = L.kda_qk_norm_rope_bwd_workspace_bytes(a)
    for ws, n, code in ((None, need, 7), (FAKE, need - 1, 7), (ODD, need, 6)):
        assert L.kda_qk_norm_rope_bwd(a, *p[:10], FAKE, None, ws, n, None) == code


def test_python_checks():
    from gated_delta_rule_gate_amd import (chunk_gated_delta, chunk_gated_delta_bwd, qk_norm_rope, qk_norm_rope_bwd,
                                           recurrent_gated_delta)

    q, g = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 4, 2)
    for f, do in ((chunk_gated_delta, ()), (recurrent_gated_delta, ()), (chunk_gated_delta_bwd, (q,))):
        with pytest.raises(ValueError, match="must be on"):
            f(q, q, q, g, g, *do)
        with pytest.raises(ValueError, match="must be on"):
            f(q, q, q, None, g, *do)
        with pytest.raises(ValueError, match="multiple of q's heads"):
            f(q, q, torch.zeros(1, 4, 3, 64, dtype=torch.bfloat16), g, g, *do)
        with pytest.raises(ValueError, match="dtype"):
            f(q.half(), q.half(), q.half(), g, g, *do)
        with pytest.raises(ValueError, match="need batch 1"):
            f(q.expand(2, 4, 2, 64), q, q.expand(2, 4, 2, 64), g, g, *do, cu_seqlens=torch.zeros(3, dtype=torch.int32))
        for scale in (0, -0.125, 1e-60, float("nan"), float("inf"), 1e60):
            with pytest.raises(ValueError, match="scale must be"):
                f(q, q, q, g, g, *do, scale=scale)
        with pytest.raises(TypeError, match="missing"):
            f()
    f, pos = torch.ones(16), torch.zeros(1, 4, dtype=torch.int32)
    for kw, text in ((dict(), "must be on"), (dict(norm="mean"), "norm must be"), (dict(pairs="third"), "pairs must be"),
                     (dict(positions=pos), "come together"), (dict(inv_freq=f), "come together"),
                     (dict(positions=pos, inv_freq=f, sections=(8, 9)), "sum to"),
                     (dict(positions=pos, inv_freq=f, sections=(4, 4, 4, 2, 2)), "one to four"),
                     (dict(positions=pos, inv_freq=f, sections=()), "one to four")):
        with pytest.raises(ValueError, match=text):
            qk_norm_rope(q, q, **kw)
        with pytest.raises(ValueError, match=text):
            qk_norm_rope_bwd(q, q, q, q, **kw)
    with pytest.raises(ValueError, match="Hk, D"):
        qk_norm_rope(q, q[..., :32])
    with pytest.raises(ValueError, match="share dtype"):
        qk_norm_rope(q, q.float())
    with pytest.raises(TypeError, match="missing"):
        qk_norm_rope()


def test_workspace_queries():
    from gated_delta_rule_gate_amd import gated_delta_workspace_bytes

    q, v = torch.zeros(1, 100, 2, 64), torch.zeros(1, 100, 4, 32)
    one, back = gated_delta_workspace_bytes(q, q, v), gated_delta_workspace_bytes(q, q, v, backward=True)
    assert 0 < one < back and gated_delta_workspace_bytes(q, q, v, slots=9) > one


@pytest.mark.gpu
def test_python_checks_on_the_device():
    from kda_testlib import need_gpu

    need_gpu()
    from gated_delta_rule_gate_amd import KdaError, chunk_gated_delta, chunk_gated_delta_bwd, qk_norm_rope

    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16, device="cuda")
    g, h = torch.zeros(1, 4, 2, device="cuda"), torch.zeros(1, 2, 64, 64, device="cuda")
    bad = [
        dict(k=q[:, :3]), dict(v=q.float()), dict(g=g.double()), dict(g=g[:, :, :1]), dict(beta=g.bfloat16()),
        dict(beta=g.cpu()), dict(initial_state=h.bfloat16()), dict(initial_state=h[:, :1]), dict(q=q.transpose(1, 2)),
        dict(final_state=h[:, :, :32]), dict(out=q.float()), dict(cu_seqlens=torch.zeros(2, device="cuda")),
        dict(workspace=torch.zeros(4, dtype=torch.uint8, device="cuda")), dict(beta=g.transpose(1, 2).contiguous().transpose(1, 2)),
    ]
    for kw in bad:
        a = dict(dict(q=q, k=q, v=q, g=g, beta=g), **kw)
        with pytest.raises(ValueError):
            chunk_gated_delta(**a)
    with pytest.raises(KdaError):  # a width that is no multiple of eight
        w = torch.zeros(1, 4, 2, 60, dtype=torch.bfloat16, device="cuda")
        chunk_gated_delta(w, w, w, g, g)
    with pytest.raises(ValueError):
        chunk_gated_delta_bwd(q, q, q, g, g, q.float())
    wide = torch.zeros(2, 4, 5 * 64, dtype=torch.bfloat16, device="cuda")
    part = wide[..., :128].unflatten(-1, (2, 64))
    for x in (part.transpose(1, 2), part[:, ::2], part.flip(2)[..., ::2], wide[..., 1:129].unflatten(-1, (2, 64))):
        if x.shape == part.shape and x.data_ptr() % 16:
            with pytest.raises(KdaError):  # rows that begin between vectors
                qk_norm_rope(x, x)
        elif x.shape[1] == 2 and x.stride(0) == 2 * x.stride(1):
            qk_norm_rope(x, x)  # every other token is one stride too
        else:
            with pytest.raises(ValueError):
                qk_norm_rope(x, x)
    odd = torch.zeros(1, 4, 132, dtype=torch.bfloat16, device="cuda")[..., :128].unflatten(-1, (2, 64))
    with pytest.raises(ValueError, match="multiple of 8"):
        qk_norm_rope(odd, odd)


@pytest.mark.gpu
def test_gradients_that_are_not_recorded():
    """Leaves are taken where no gradient is recorded and refused where one would be lost."""
    from kda_testlib import need_gpu

    need_gpu()
    from gated_delta_rule_gate_amd import (chunk_gated_delta, chunk_gated_delta_bwd, qk_norm_rope, qk_norm_rope_bwd,
                                           recurrent_gated_delta)

    q = torch.randn(1, 4, 2, 64, device="cuda").bfloat16()
    wide = torch.randn(1, 4, 256, device="cuda").bfloat16()
    g, w = -torch.rand(1, 4, 2, device="cuda"), torch.ones(64, device="cuda")

    def calls(q, w, g, wide):
        d, part = q.detach(), wide[..., :128].unflatten(-1, (2, 64))
        return [lambda: chunk_gated_delta(q, d, d, g, -g), lambda: recurrent_gated_delta(d, d, d, g, -g),
                lambda: chunk_gated_delta_bwd(q, d, d, g, -g, d), lambda: qk_norm_rope(d, d, w, w),
                lambda: qk_norm_rope(part, d), lambda: qk_norm_rope_bwd(d, d, d, d, w, w)]

    flat = lambda r: [t for t in (r.values() if isinstance(r, dict) else r) if t is not None]  # noqa: E731
    leaves = [t.clone().requires_grad_(True) for t in (q, w, g, wide)]
    for plain, call in zip(calls(q, w, g, wide), calls(*leaves)):
        want = flat(plain())
        with pytest.raises(RuntimeError, match="requires grad.*no_grad"):
            call()
        for mode in (torch.no_grad, torch.inference_mode):
            with mode():
                got = flat(call())
            assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))
