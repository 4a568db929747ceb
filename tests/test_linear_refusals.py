"""What linear attention and the block norm refuse, without a GPU: status codes of the C entry points
before any launch, workspace queries, and the Python checks."""
import ctypes
import os

import pytest
import torch

FAKE = ctypes.c_void_p(0x100000)  # aligned, never dereferenced: every call here is refused before a launch


@pytest.fixture(scope="module")
def L():
    from gated_delta_rule_gate_amd import _binding, _linear, build

    if not os.path.exists(_binding.LIB_PATH):
        build.build()
    return _linear._lib()


def lin(**kw):
    from gated_delta_rule_gate_amd._linear import LinearArgs

    a = LinearArgs(1, 64, 2, 128, 128, 1, 0, 0, 0, 0.0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def nrm(**kw):
    from gated_delta_rule_gate_amd._linear import NormArgs

    a = NormArgs(4, 128, 0, 0, 0, 0, 1.0, 1e-6)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BAD = [
    (dict(dtype=7), 3), (dict(decay=2), 5), (dict(K=44), 8), (dict(V=264), 8), (dict(K=0), 2), (dict(B=2), 2),
    (dict(H=0), 2), (dict(H=4097), 2), (dict(H=3, Hk=2), 2), (dict(Hk=-1), 2), (dict(T=-1), 2), (dict(N=-1), 2),
]


@pytest.mark.parametrize("kw,code", BAD)
def test_linear_arguments(L, kw, code):
    a = lin(**kw)
    assert L.kda_linear_recurrent_fwd(a, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None, None) == code
    assert L.kda_linear_chunk_fwd(a, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None, FAKE, 1 << 40, None) == code
    assert L.kda_linear_chunk_bwd(a, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None, FAKE, FAKE, FAKE, FAKE, None, FAKE,
                                  1 << 40, None) == code
    if "B" not in kw:  # N != B is a packed query's right
        assert L.kda_linear_chunk_workspace_bytes(a) == 0 and L.kda_linear_chunk_bwd_workspace_bytes(a) == 0


def test_linear_pointers(L):
    a, odd = lin(), ctypes.c_void_p(0x100004)
    for i in (0, 1, 2, 3, 6):
        p = [FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None]
        p[i] = None
        assert L.kda_linear_recurrent_fwd(a, *p, None) == 1, i
        assert L.kda_linear_chunk_fwd(a, *p, FAKE, 1 << 40, None) == 1, i
    for i in (0, 1, 2, 3, 4, 6, 7):
        p = [FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None]
        p[i] = odd
        assert L.kda_linear_recurrent_fwd(a, *p, None) == 6, i
        assert L.kda_linear_chunk_fwd(a, *p, FAKE, 1 << 40, None) == 6, i
    for i in range(4):  # dq, dk, dv, dg are required
        p = [FAKE] * 4
        p[i] = None
        assert L.kda_linear_chunk_bwd(a, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None, *p, None, FAKE, 1 << 40,
                                      None) == 1
    assert L.kda_linear_recurrent_fwd(None, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None, None) == 1
    assert L.kda_linear_chunk_fwd(lin(B=2, N=2), FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE, None, FAKE, 1 << 40, None) == 2


def test_linear_workspaces(L):
    a = lin(T=8192, H=2)
    need = L.kda_linear_chunk_workspace_bytes(a)
    assert need > 0  # two heads: the sequence is cut into segments
    for ws, n in ((None, need), (FAKE, need - 1)):
        assert L.kda_linear_chunk_fwd(a, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None, ws, n, None) == 7
    assert L.kda_linear_chunk_fwd(a, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None, ctypes.c_void_p(0x100010), need,
                                  None) == 6
    assert L.kda_linear_chunk_workspace_bytes(lin(T=64)) == 0
    need = L.kda_linear_chunk_bwd_workspace_bytes(a)
    for ws, n in ((None, need), (FAKE, need - 1)):
        assert L.kda_linear_chunk_bwd(a, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None, FAKE, FAKE, FAKE, FAKE, None, ws,
                                      n, None) == 7


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 2), (dict(D=0), 2), (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2), (dict(dtype=2), 3),
    (dict(dtype=1, res_dtype=0), 3), (dict(res_dtype=1), 3), (dict(norm=2), 5), (dict(gate_act=2), 5), (dict(D=100), 8),
    (dict(D=16392), 8),
])
def test_norm_arguments(L, kw, code):
    a = nrm(**kw)
    assert L.kda_block_norm_fwd(a, FAKE, None, None, None, None, None, FAKE, None, None) == code
    assert L.kda_block_norm_bwd(a, FAKE, None, None, None, None, None, FAKE, None, FAKE, None, None, None, None, None,
                                FAKE, 1 << 40, None) == code


def test_norm_pointers(L):
    a, odd = nrm(), ctypes.c_void_p(0x100008)
    assert L.kda_block_norm_fwd(a, None, None, None, None, None, None, FAKE, None, None) == 1
    assert L.kda_block_norm_fwd(a, FAKE, None, None, None, None, None, None, None, None) == 1
    for i in range(8):
        p = [FAKE, None, None, None, None, None, FAKE, None]
        p[i] = odd
        assert L.kda_block_norm_fwd(a, *p, None) == 6
    bwd = lambda dy, dz, dx, gate=None, dgate=None, dw=None, ws=FAKE, n=1 << 40: L.kda_block_norm_bwd(  # noqa: E731
        a, FAKE, None, gate, None, None, None, dy, dz, dx, dgate, None, dw, None, None, ws, n, None)
    assert bwd(None, None, FAKE) == 1 and bwd(FAKE, None, None) == 1 and bwd(FAKE, None, FAKE, gate=FAKE) == 1
    assert bwd(FAKE, None, FAKE, dw=FAKE, ws=None) == 7 and bwd(FAKE, None, FAKE, dw=FAKE, n=16) == 7


def test_norm_gradient_of_a_next_weight_needs_dz(L):
    a = nrm()
    assert L.kda_block_norm_bwd(a, FAKE, None, None, None, None, None, FAKE, None, FAKE, None, None, None, None, FAKE,
                                FAKE, 1 << 40, None) == 1


def test_python_checks():
    from gated_delta_rule_gate_amd import block_norm, block_norm_bwd, chunk_linear_attn, recurrent_linear_attn

    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    g = torch.zeros(1, 4, 2)
    for f in (chunk_linear_attn, recurrent_linear_attn):
        with pytest.raises(ValueError, match="must be on"):
            f(q, q, q, g)
        with pytest.raises(ValueError, match="multiple of q's heads"):
            f(q, q, torch.zeros(1, 4, 3, 64, dtype=torch.bfloat16), g)
        with pytest.raises(ValueError, match="dtype"):
            f(q.half(), q.half(), q.half(), g)
        with pytest.raises(ValueError, match="need batch 1"):
            f(q.expand(2, 4, 2, 64), q, q.expand(2, 4, 2, 64), g, cu_seqlens=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="must be on"):
        block_norm(q)
    with pytest.raises(ValueError, match="norm must be"):
        block_norm(q, norm="mean")
    with pytest.raises(ValueError, match="gate_act"):
        block_norm(q, gate_act="tanh")
    with pytest.raises(ValueError, match="residual"):
        block_norm(q.float(), residual=q)
    with pytest.raises(ValueError, match="next_weight"):
        block_norm(q, next_weight=torch.ones(64), next_norm=False)
    with pytest.raises(ValueError, match="dy or dz"):
        block_norm_bwd(q, None)


@pytest.mark.parametrize("scale", [0, 0.0, -0.125, 1e-60, float("nan"), float("inf"), 1e60])
def test_scales(scale):
    from gated_delta_rule_gate_amd import chunk_linear_attn, chunk_linear_attn_bwd, recurrent_linear_attn

    q, g = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 4, 2)
    for f, do in ((chunk_linear_attn, ()), (recurrent_linear_attn, ()), (chunk_linear_attn_bwd, (q,))):
        with pytest.raises(ValueError, match="scale must be"):
            f(q, q, q, g, *do, scale=scale)


def test_tensors_by_keyword():
    """Every argument can be named, the first too; one that is left out is named in the error."""
    from gated_delta_rule_gate_amd import (block_norm, block_norm_bwd, chunk_linear_attn, chunk_linear_attn_bwd,
                                           linear_workspace_bytes, recurrent_linear_attn)

    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    t = dict(q=q, k=q, v=q, g=torch.zeros(1, 4, 2))
    for f, kw in ((chunk_linear_attn, t), (recurrent_linear_attn, t), (chunk_linear_attn_bwd, dict(t, do=q)),
                  (block_norm, dict(x=q)), (block_norm_bwd, dict(x=q, dy=q))):
        with pytest.raises(ValueError, match="must be on a GPU"):
            f(**kw)
        with pytest.raises(TypeError, match="missing"):
            f()
    assert linear_workspace_bytes(**t) == linear_workspace_bytes(*t.values())


@pytest.mark.gpu
def test_python_checks_on_the_device():
    from kda_testlib import need_gpu

    need_gpu()
    from gated_delta_rule_gate_amd import KdaError, block_norm, chunk_linear_attn, chunk_linear_attn_bwd

    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(1, 4, 2, device="cuda")
    with pytest.raises(RuntimeError, match="requires grad"):
        chunk_linear_attn(q.clone().requires_grad_(True), q, q, g)
    with pytest.raises(ValueError, match="g must be"):
        chunk_linear_attn(q, q, q, g.double())
    with pytest.raises(ValueError, match="contiguous"):
        chunk_linear_attn(q.transpose(1, 2).contiguous().transpose(1, 2), q, q, g)
    with pytest.raises(ValueError, match="out must be"):
        chunk_linear_attn(q, q, q, g, out=q.float())
    with pytest.raises(ValueError, match="final_state"):
        chunk_linear_attn(q, q, q, g, final_state=torch.zeros(1, 2, 64, 32, device="cuda"))
    with pytest.raises(ValueError, match="cu_seqlens must be"):
        chunk_linear_attn(q, q, q, g, cu_seqlens=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="workspace"):
        chunk_linear_attn_bwd(q, q, q, g, q, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(KdaError, match="UNSUPPORTED"):
        z = torch.zeros(1, 4, 2, 12, dtype=torch.bfloat16, device="cuda")
        chunk_linear_attn(z, z, q, g)
    with pytest.raises(KdaError, match="UNSUPPORTED"):
        block_norm(torch.zeros(3, 12, device="cuda"))


@pytest.mark.parametrize("sizes,wide", [
    # (sequence, head) pairs times threads of a workgroup: 2^32 and more than a launch counts
    (dict(B=4096, N=4096, H=4096), False),             # the recurrence: 256 threads
    (dict(B=2048, N=2048, H=4096, K=64, V=64), True),  # chunked by 64 columns: 512 threads
    (dict(B=1366, N=1366, H=4096), True),              # by 128 columns: 768
    (dict(B=683, N=683, H=4096, V=256), True),
    (dict(N=2048, H=4096, K=64, V=64), True),          # packed
])
def test_more_workgroups_than_a_launch_takes(L, sizes, wide):
    """Refused before the first launch, so that no output is written by half."""
    a = lin(T=1, **sizes)
    cu = FAKE if a.B != a.N else None
    if wide:
        assert L.kda_linear_chunk_fwd(a, FAKE, FAKE, FAKE, FAKE, None, cu, FAKE, None, FAKE, 1 << 50, None) == 8
        assert L.kda_linear_chunk_bwd(a, FAKE, FAKE, FAKE, FAKE, None, cu, FAKE, None, FAKE, FAKE, FAKE, FAKE, None, FAKE,
                                      1 << 50, None) == 8
    else:
        assert L.kda_linear_recurrent_fwd(a, FAKE, FAKE, FAKE, FAKE, None, cu, FAKE, None, None) == 8


def test_the_largest_launches_are_not_refused(L):
    """One pair of a sequence fewer: the sizes are taken, and the missing workspace is what is wrong."""
    for kw in (dict(B=2047, N=2047, H=4096, K=64, V=64), dict(B=1365, N=1365, H=4096)):
        a = lin(T=1, **kw)
        assert L.kda_linear_chunk_bwd(a, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None, FAKE, FAKE, FAKE, FAKE, None,
                                      None, 0, None) == 7
    # shared heads: their gradients' sum, 2^32 pieces of four values
    big = lin(B=1, N=1, T=1 << 24, H=8, Hk=4, K=256, V=8)
    assert L.kda_linear_chunk_bwd(big, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None, FAKE, FAKE, FAKE, FAKE, None, None,
                                  0, None) == 8
    big.T -= 1
    assert L.kda_linear_chunk_bwd(big, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None, FAKE, FAKE, FAKE, FAKE, None, None,
                                  0, None) == 7


def test_import_without_gpu_bindings():
    """A PyTorch build without a GPU imports the package; calls are refused for their tensors' device."""
    import subprocess
    import sys

    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import gated_delta_rule_gate_amd as p
q = torch.zeros(1, 4, 2, 64)
try:
    p.chunk_linear_attn(q, q, q, torch.zeros(2))
except ValueError as e:
    assert "must be on a GPU" in str(e), e
else:
    raise AssertionError("not refused")
print("imported", p.linear_workspace_bytes(q, q, q, torch.zeros(2)))
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=root, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("imported"), r.stderr[-2000:]


def _calls(q, w, g):
    """Every entry point, on inputs of which any may require a gradient."""
    from gated_delta_rule_gate_amd import (block_norm, block_norm_bwd, chunk_linear_attn, chunk_linear_attn_bwd,
                                           recurrent_linear_attn)

    d = q.detach()
    return dict(chunk=lambda: chunk_linear_attn(q, d, d, g), recurrent=lambda: recurrent_linear_attn(q, d, d, g),
                chunk_bwd=lambda: chunk_linear_attn_bwd(q, d, d, g, d), norm=lambda: block_norm(d, w),
                norm_bwd=lambda: block_norm_bwd(d, d, w))


@pytest.mark.gpu
def test_gradients_that_are_not_recorded():
    """Parameters are taken as they are where no gradient is recorded (no_grad, inference mode, inside an
    autograd.Function) and refused where one would be lost, naming the way out."""
    from kda_testlib import need_gpu

    need_gpu()
    plain = (torch.randn(1, 4, 2, 64, device="cuda").bfloat16(), torch.randn(64, device="cuda"),
             -torch.rand(1, 4, 2, device="cuda"))
    leaves = tuple(t.clone().requires_grad_(True) for t in plain)
    flat = lambda r: [t for t in (r.values() if isinstance(r, dict) else r if isinstance(r, tuple) else [r])  # noqa: E731
                      if t is not None]
    for name, want in _calls(*plain).items():
        want, call = flat(want()), _calls(*leaves)[name]
        with pytest.raises(RuntimeError, match="requires grad.*no_grad"):
            call()
        for mode in (torch.no_grad, torch.inference_mode):
            with mode():
                got = flat(call())
            assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want)), name
            assert not any(t.requires_grad for t in got)


@pytest.mark.gpu
def test_inside_an_autograd_function():
    """The forward and its _bwd as a user's autograd.Function calls them."""
    from kda_testlib import need_gpu

    need_gpu()
    from gated_delta_rule_gate_amd import block_norm, block_norm_bwd

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight):
            ctx.save_for_backward(x, weight)
            return block_norm(x, weight)

        @staticmethod
        def backward(ctx, dy):
            x, weight = ctx.saved_tensors
            got = block_norm_bwd(x, dy.contiguous(), weight)
            return got["dx"], got["dweight"]

    x, w = (torch.randn(*s, device="cuda").requires_grad_(True) for s in ((5, 64), (64,)))
    dy = torch.randn(5, 64, device="cuda")
    (Norm.apply(x, w) * dy).sum().backward()
    want = block_norm_bwd(x.detach(), dy, w.detach())
    assert torch.equal(x.grad, want["dx"]) and torch.equal(w.grad, want["dweight"])


def test_a_next_output_needs_the_next_norm():
    from gated_delta_rule_gate_amd import block_norm

    x = torch.zeros(3, 64)
    for kw in (dict(), dict(next_norm=False)):
        with pytest.raises(ValueError, match="next_out needs the next norm"):
            block_norm(x, next_out=torch.zeros(3, 64), **kw)
