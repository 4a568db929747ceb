"""How exact the gated delta rule's results are on the GPU, by criteria that a bf16 part left out, a wrong sign or
a lost term cannot pass."""
import math

import pytest
import torch

import delta_norms as norms
import delta_ref as ref
from kda_testlib import need_gpu
from test_gpu_delta import BF16, FP32, IN, LONG, SHAPES, _id, dev, f64, inputs64, make, on

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


def check_norms(d, backward=True):
    """Every result's error, in the 2-norm of each sequence and head, below delta_norms.bounds."""
    from gated_delta_rule_gate_amd import chunk_gated_delta, chunk_gated_delta_bwd

    B, T = d["q"].shape[:2]
    g, cu, end = dev(d), d["cu"], T if d["cu"] is None else int(d["cu"][-1])
    o, ht = on(g, chunk_gated_delta, output_final_state=True)
    got, do, dht = dict(o=o, ht=ht), None, f64(d["dht"])
    if backward:
        got.update(on(g, chunk_gated_delta_bwd, g["do"], dht=g["dht"]))
        do = f64(d["do"]).clone()
        do[:, end:] = 0
        want = norms.reference(inputs64(d), do, dht, cu=cu)
    else:
        want = dict(zip(norms.NAMES, ref.delta(*inputs64(d), cu=cu)))
    bound = norms.bounds(*inputs64(d), cu=cu, do=do, dht=dht)
    for name in norms.NAMES if backward else norms.NAMES[:2]:
        if name == "dg" and d["g"] is None:
            continue
        states = name in ("ht", "dh0")
        over, most = norms.exceeded(got[name], want[name], bound[name], B, T, cu, states=states)
        print("%s %.2f of %.0e" % (name, over, most), end=" ")
        assert over <= 1.0, (name, over, most)


@pytest.mark.parametrize("decay", [True, False], ids=["decay", "plain"])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=_id)
def test_norms(shape, dtype, decay):
    need_gpu()
    check_norms(make(*shape[:6], dtype, shape[6], states=shape[1] != 97, seed=91, decay=decay))


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("K", [8, 72, 136, 192, 200, 256])
def test_norms_of_chunks_of_one_row(K, dtype):
    need_gpu()
    check_norms(make(1, 98, 2, 1, K, 24, dtype, lens=[65, 33], seed=92))


def test_norms_of_many_heads_and_slots():
    need_gpu()
    lens = [1, 70, 0, 33, 64, 128, 7, 100, 3, 17]
    check_norms(make(1, sum(lens) + 2, 48, 16, 64, 72, BF16, lens=lens, seed=93))


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_norms_where_tokens_write_nothing(dtype):
    need_gpu()
    d = make(1, 140, 2, 1, 72, 64, dtype, seed=94)
    d["beta"][0, ::3] = 0.0
    d["beta"][0, 64:128, 1] = 0.0
    check_norms(d)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_norms_of_long_gradients(dtype):
    """Many chunks, on heads that forget nothing, a little, and all of it."""
    need_gpu()
    d = make(1, 1100, 3, 3, 64, 40, dtype, seed=95)
    d["g"] *= torch.tensor([0.0, 0.01, 3.0])
    check_norms(d)


@pytest.mark.parametrize("decay", [0.01, None], ids=["weak", "plain"])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", LONG + [(2, 2600, 2, 1, 40, 136, None)], ids=_id)
def test_norms_of_long_forwards(shape, dtype, decay):
    """Cut into segments, whose maps matter to the next."""
    need_gpu()
    check_norms(make(*shape[:6], dtype, shape[6], seed=96, strength=decay or 0.0, decay=decay is not None), backward=False)


@pytest.mark.parametrize("which", norms.IN)
def test_gradient_against_close_differences(which):
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta, chunk_gated_delta_bwd

    d = make(1, 150, 2, 1, 72, 40, FP32, seed=8)
    g, do, dht = dev(d), f64(d["do"]), f64(d["dht"])

    def loss(x):
        o, ht = on(dict(g, **{which: x.cuda()}), chunk_gated_delta, output_final_state=True)
        return ((f64(o) * do).sum() + (f64(ht) * dht).sum()).item()

    norms.check_differences(which, dict(zip(IN, inputs64(d))), do, dht, loss,
                            on(g, chunk_gated_delta_bwd, g["do"], dht=g["dht"])["d" + which])


def _still(K, V, dtype, seed):
    """40 chunks of tokens that write nothing and leave all as it is."""
    d = make(1, 2560, 1, 1, K, V, dtype, seed=seed)
    d["g"][:] = 0.0
    d["beta"][:] = 0.0
    return d


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("K", [64, 128, 256])
def test_segments_hand_states_over_as_they_are(K, dtype):
    """Every segment's map is the identity: the chain's products with it, of the state in three parts, leave all 24
    bits of it. Two parts would leave 16."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta

    g = dev(_still(K, 136, dtype, 97))
    for gate in (g["g"], None):
        _, ht = on(dict(g, g=gate), chunk_gated_delta, output_final_state=True)
        assert torch.equal(ht, g["h0"])


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("K", [64, 128, 256])
def test_maps_of_segments_are_whole(K, dtype):
    """One chunk in the middle writes, all others leave the state as it is; the state at the start has a one in every
    column. What comes out is then the map of that chunk's segment, and the same as of the chunk alone: the map's
    three parts hold all of its bits.

    Chunks of 32 tokens (fp32, and 256 channels) make segments of a multiple of 32: of 5 chunks, a border lies at
    11 x 160 = 1760 = 64 x 27 + 32, in the middle of the 64 tokens of chunk 27. Two maps are multiplied there, by a
    sum over K rounded otherwise than the walk's: columns of norm one are off by no more than delta_norms.bounds of
    either, each 4 (K + K + 64)^1/2 2^-24. Of the five places at most two can lie so."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta

    d = _still(K, K, dtype, 98)
    d["h0"][:] = torch.eye(K)
    d["v"][:] = 0.0
    whole, small = {}, dtype == FP32 or K > 128
    for c in (3, 13, 20, 27, 39):
        part = slice(64 * c, 64 * c + 64)
        e = dict(d, beta=torch.zeros_like(d["beta"]), g=torch.zeros_like(d["g"]))
        e["beta"][:, part] = 0.7
        e["g"][:, part] = -0.01
        g = dev(e)
        for gate in (g["g"], None):
            _, ht = on(dict(g, g=gate), chunk_gated_delta, output_final_state=True)
            alone = [g[x][:, part].contiguous() for x in ("q", "k", "v")] + [None if gate is None else gate[:, part].contiguous(),
                                                                            g["beta"][:, part].contiguous(), g["h0"]]
            _, want = chunk_gated_delta(*alone, output_final_state=True)
            assert not torch.equal(want, g["h0"])
            off = (ht - want).norm(dim=-2).max().item()
            assert off == 0.0 or small and off <= 8 * (2 * K + 64) ** 0.5 * ref.ULP32, (c, gate is None, off)
            whole[gate is None] = whole.get(gate is None, 0) + (off == 0.0)
    assert all(n >= 3 for n in whole.values()), whole


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("K", [64, 128, 256])
def test_maps_times_states(K, dtype):
    """One token decays the state, all others leave it as it is: the map of its segment is a multiple of the identity,
    and each value of what comes out the product of two numbers of three parts. The decay is off by 2.4 2^-24 (its
    exponent's rounding and an exponential good to one unit of the last place), its product with a state by 1, the
    products of parts that are left out by 2 (both of at most 2^-24), the sum of the others by 2: below 9 2^-24 = 2^-20.8.
    Without the product of the two second parts, here both of 0.8 2^-8 and more, 2^-17.3 would be missing."""
    need_gpu()
    from gated_delta_rule_gate_amd import chunk_gated_delta

    gen = torch.Generator().manual_seed(99)
    for token in (200, 900, 1300, 1700):
        d = _still(K, 64, dtype, 99)
        d["g"][:, token] = math.log(0.5 * (1 + 0.95 * 2.0 ** -8))
        sign = torch.randint(0, 2, d["h0"].shape, generator=gen) * 2 - 1
        d["h0"] = sign * (1 + (torch.randint(0, 64, d["h0"].shape, generator=gen) + 0.4 + 0.1 * torch.rand(d["h0"].shape, generator=gen)) / 128)
        g = dev(d)
        _, ht = on(g, chunk_gated_delta, output_final_state=True)
        want = f64(d["h0"]) * torch.exp(f64(d["g"]).sum())
        off = ((f64(ht) - want) / want).abs().max().item()
        assert off <= 9 * ref.ULP32, off / ref.ULP32
