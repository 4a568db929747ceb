"""How exact the gated delta rule's results are on the GPU, by criteria that a bf16 part left out, a wrong sign or
a lost term cannot pass."""
import pytest
import torch

import delta_ref as ref
from kda_testlib import need_gpu
from test_gpu_delta import BF16, FP32, IN, _id, dev, f64, inputs64, make, on

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [
    (2, 500, 4, 2, 128, 128, None), (1, 1500, 2, 2, 128, 136, None), (3, 257, 4, 4, 64, 64, None), (2, 300, 3, 3, 256, 72, None),
    (1, 900, 4, 4, 72, 128, [3, 500, 0, 397]), (200, 33, 2, 2, 128, 128, None),
], ids=_id)
def test_bf16_outputs_round_an_fp32_result(shape):
    """o of a bf16 call is the value of an fp32 one, rounded once. Where the 64-bit value lies nearer to the border
    between two bf16 values than the fp32 result is off, the rounding may go the other way: a share of places that
    grows with the size of the error. The fp32 call on the same values shows what share fp32 errors make; the
    bf16 call's sums are up to twice as long (chunks of 64 tokens for 32), so its errors are at most 2 of
    the fp32 call's, taken as 3, and the counts scatter by their roots. Operands of 16 bits have errors ten
    times as large and more."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta

    B, T, H, Hk, K, V, lens = shape
    d = make(B, T, H, Hk, K, V, BF16, lens, seed=90)
    want = ref.delta(*inputs64(d), cu=d["cu"])[0].to(BF16)
    g = dev(d)
    o = on(g, chunk_gated_delta)[0]
    o32 = on(dict(g, **{x: g[x].float() for x in ("q", "k", "v")}), chunk_gated_delta)[0].to(BF16)
    wrong, wrong32 = (int((x.cpu() != want).sum()) for x in (o, o32))
    print("of %d outputs %d, fp32 rounded %d" % (want.numel(), wrong, wrong32))
    assert wrong <= 3 * wrong32 + 5 * (3 * wrong32) ** 0.5 + 5
