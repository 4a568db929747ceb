"""The bounds of delta_norms.py on the CPU: an evaluation of the definition in 32 bits stays far below them, and
mistakes planted in the 64-bit results do not."""
import pytest
import torch

import delta_norms as norms
import delta_ref as ref
from test_gpu_delta import FP32, _id, f64, inputs64, make

CASES = [
    (2, 15, 3, 3, 64, 64, None), (1, 65, 2, 2, 40, 200, None), (1, 98, 2, 1, 136, 24, [65, 33]), (1, 130, 3, 1, 256, 256, None),
    (1, 400, 2, 2, 72, 40, [33, 300]), (1, 300, 2, 2, 64, 128, None),
]


def _all(d):
    B, T = d["q"].shape[:2]
    do = f64(d["do"]).clone()
    if d["cu"] is not None:
        do[:, int(d["cu"][-1]):] = 0
    dht = f64(d["dht"])
    return (do, dht, norms.bounds(*inputs64(d), cu=d["cu"], do=do, dht=dht),
            norms.reference(inputs64(d), do, dht, cu=d["cu"]))


def _ratio(name, got, want, bound, d):
    B, T = d["q"].shape[:2]
    return norms.exceeded(got, want[name], bound[name], B, T, d["cu"], states=name in ("ht", "dh0"))


@pytest.mark.parametrize("shape", CASES, ids=_id)
def test_32_bits_stay_below(shape):
    d = make(*shape[:6], FP32, shape[6], seed=1)
    do, dht, bound, want = _all(d)
    # the recurrence and its derivative, every step in 32 bits
    ins = [x.float() for x in inputs64(d)]
    got = norms.reference(ins, do.float(), dht.float(), cu=d["cu"])
    for name in norms.NAMES:
        over, most = _ratio(name, got[name].float(), want, bound, d)
        assert over <= 0.5 and most <= 1e-3, (name, over, most)


@pytest.mark.parametrize("shape", CASES, ids=_id)
@pytest.mark.parametrize("name", norms.NAMES)
def test_planted_mistakes(name, shape):
    """Zeros, the other sign, a last row (of a state: the last row of the last head) that lacks a hundredth, all of it larger by
    2^-10."""
    d = make(*shape[:6], FP32, shape[6], seed=1)
    _, _, bound, want = _all(d)
    w = want[name]
    last = int(d["cu"][-1]) - 1 if d["cu"] is not None else -1
    tail = w.clone()
    if name in ("ht", "dh0"):
        tail[-1, -1, -1] *= 0.99
    else:
        tail[-1, last] *= 0.99
    for wrong in (torch.zeros_like(w), -w, tail, w * (1 + 2.0 ** -10)):
        over, _ = _ratio(name, wrong.float(), want, bound, d)
        assert over > 1.0, (name, over)


@pytest.mark.parametrize("which", norms.IN)
def test_differences_see_a_wrong_gradient(which):
    d = make(1, 150, 2, 1, 72, 40, FP32, seed=8)
    ins, do, dht = dict(zip(norms.IN, inputs64(d))), f64(d["do"]), f64(d["dht"])
    want = norms.reference([ins[x] for x in norms.IN], do, dht)["d" + which]

    def loss(x, sign=1.0):
        o, ht = ref.delta(*[x.double() if n == which else ins[n] for n in norms.IN])
        return sign * ((o.float().double() * do).sum() + (ht.float().double() * dht).sum()).item()

    norms.check_differences(which, ins, do, dht, loss, want.float())
    for wrong in (torch.zeros_like(want), -want, want * 1.02):
        with pytest.raises(AssertionError):
            norms.check_differences(which, ins, do, dht, loss, wrong.float())
    with pytest.raises(AssertionError):
        norms.check_differences(which, ins, do, dht, lambda x: loss(x, 0.98), want.float())
