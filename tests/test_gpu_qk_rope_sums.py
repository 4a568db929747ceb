"""The weights' gradients of the norm with rotation, sums over all rows, as exact as their sums are: by the 2-norm of all
channels, in batches whose workgroups take one token group or several.

A channel's gradient is a sum over rows of dn x rho. Roundings are of either sign: what n of them leave of every term,
and the sums of a lane's at most 64 rows (each off by 2^-24 of the sum so far), add up to (64 + n)^1/2 2^-24 of the
root of the terms' squares. n = D + 64: the norm's sum over D, angles, turns and products. A factor of four as in
delta_norms.py. A row that is left out is a whole term."""
import pytest
import torch

import delta_ref as ref
from kda_testlib import need_gpu
from test_gpu_qk_rope import BF16, FP32, _id, f64, make, want_of

CASES = [
    (1, 40000, 2, 1, 64, 64, "rms", "half", None, False, False),  # 1250 groups of 32 tokens for 1024 workgroups
    (1, 5000, 1, 1, 512, 0, "rms", "half", None, False, False),   # 1250 groups of four tokens
    (1, 3000, 9, 2, 64, 56, "none", "adjacent", (0, 14, 14), False, False),
    (1, 700, 12, 3, 96, 48, "l2", "half", (8, 8, 8), True, False),
    (1, 130, 48, 16, 40, 24, "rms", "half", (12, 0), True, True),
]


def gradient_and_bound(g, kw, name):
    """dw in 64 bits, its bound, and the terms of every row."""
    x, w, dy = f64(g[name]), f64(g["w" + name]), f64(g["d" + name])
    D = x.shape[-1]
    # per row: the derivative of dy . y in the row's own copy of the weight
    own = w.expand(*x.shape).clone().requires_grad_(True)
    terms, = torch.autograd.grad((want_of(g, kw, x, own) * dy).sum(), own)
    terms = terms.reshape(-1, D)
    return terms.sum(0), 4 * (64 + D + 64) ** 0.5 * ref.ULP32 * terms.norm().item(), terms


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("case", CASES, ids=_id)
def test_weights_gradients(case, dtype):
    need_gpu()
    from gated_delta_rule_gate_amd import qk_norm_rope_bwd

    g, kw = make(case, dtype, seed=7)
    got = qk_norm_rope_bwd(g["q"], g["k"], g["dq"], g["dk"], g["wq"], g["wk"], **kw)
    for name in ("q", "k"):
        want, most, _ = gradient_and_bound(g, kw, name)
        off = (f64(got["d%s_weight" % name]) - want).norm().item()
        print("%s %.3g of %.3g, values %.3g" % (name, off, most, want.norm().item()), end=" ")
        assert off <= most, (name, off, most)


@pytest.mark.parametrize("case", CASES[2:], ids=_id)
def test_a_lost_row_is_seen(case):
    """On the CPU: sums in 32 bits over rows stay within the bound, without one of the rows they do not."""
    from unittest import mock

    with mock.patch.object(torch.Tensor, "cuda", lambda x: x):
        g, kw = make(case, FP32, seed=7)
    for name in ("q", "k"):
        want, most, terms = gradient_and_bound(g, kw, name)
        part = terms.float().reshape(-1, 10, terms.shape[-1])
        lanes = part[:, 0].clone()
        for i in range(1, 10):
            lanes += part[:, i]
        assert (lanes.double().sum(0) - want).norm().item() <= most
        assert (want - terms[-1] - want).norm().item() > 10 * most
        assert most < 1e-4 * want.norm().item()
