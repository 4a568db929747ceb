"""How exact the rotation's sines and cosines are on the GPU: pairs (1, 0) without a norm come out as cosine and sine."""
import numpy as np
import pytest
import torch

from kda_testlib import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("far", [1 << 10, 1 << 17, 1 << 30])
def test_sines_and_cosines(far):
    """In fp32. What is left of an angle when whole quarters of a turn are taken off in 64 bits is at most an eighth of a
    turn, and rounding it to 32 bits leaves 2 pi 2^-28, evenly spread: 1.4e-8 in the mean square, of which the slopes of
    sine and cosine pass on half. Sines and cosines good to a unit of the last place (2^-24 in the upper half of their
    range), errors spread over half of it either way, leave 1.7e-8. Together 2.0e-8; 2.8e-8 are allowed. With the remainder
    of a whole turn, up to a half, in 32 bits the angles alone would leave 4.1e-8, and all together 3.3e-8 and more.

    The angle itself is a product of 31 and 24 bits, then one with 1 / 2 pi (itself rounded): three roundings in 64 bits of
    2^-53 of an angle of at most 6.2 far, together 3e-10 at 2^17 and 2e-6 at 2^30."""
    need_gpu()
    from gated_delta_rule_gate_amd import qk_norm_rope

    T, D = 4096, 128
    r = np.random.Generator(np.random.PCG64(far))
    pos = torch.from_numpy(r.integers(-far, far, (1, T)).astype(np.int32))
    freq = (1e4 ** (-torch.arange(0, D, 2) / D)).float()
    freq[:8] = torch.tensor([1.0, 0.3, 0.7, 1.9, 3.1, 0.01, 6.2, 0.9])  # of all phases however near the position
    x = torch.zeros(1, T, 1, D)
    x[..., : D // 2] = 1.0
    y, _ = qk_norm_rope(x.cuda(), x.cuda(), positions=pos.cuda(), inv_freq=freq.cuda(), norm="none")
    y = y.cpu().double()
    ang = np.asarray(pos.numpy()[0][:, None], np.longdouble) * np.asarray(freq.double().numpy(), np.longdouble)
    two_pi = np.longdouble("6.28318530717958647692528676655900577")
    turns = ang / two_pi
    ang = torch.from_numpy(((turns - np.rint(turns)) * two_pi).astype(np.float64))[None, :, None]
    used = ang.abs().amax(dim=1).flatten() > 3.0  # frequencies that pass through all phases
    assert used.sum() >= 8
    for name, got, want in (("cos", y[..., : D // 2], ang.cos()), ("sin", y[..., D // 2:], ang.sin())):
        off = (got - want)[..., used]
        print("%s %.3g at most %.3g" % (name, off.square().mean().sqrt().item(), off.abs().max().item()), end=" ")
        assert off.square().mean().sqrt().item() <= 2.8e-8 + 3 * 2.0 ** -53 * 6.2 * far
