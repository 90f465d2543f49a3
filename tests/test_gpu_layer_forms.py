"""GPU tests of forms of the layer calls that the sizes in test_gpu_layer.py do not reach, with that file's
layer, 64-bit reference and tolerances."""
import math

import pytest
import torch

import heterogeneous_adapters_sgmv_b200 as L
from tests.test_gpu_layer import BF, Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available()
    L._load()


def test_bgmv_layer_with_the_workspace_of_a_larger_batch():
    """The scaled intermediate has more parts in smaller batches; one workspace serves all."""
    big = Layer(1024, 2048, 136, (16, 40), seed=41)
    assert big.table.workspace_bytes(512) <= big.ws.numel()
    for T in (512, 130, 1):
        m = Layer(T, 2048, 136, (16, 40), seed=42, act="silu")
        ids = m.ids()
        big.ws.fill_(255)
        m.check(m.bgmv(ids, ws=big.ws), ids, "%d tokens" % T)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "gelu"])
def test_activations_keep_their_relative_accuracy_in_the_lower_tail(act):
    """One bf16 z an output column, from 0 down to where the results pass below 2^-126 of z.  Of the result: one
    rounding (2^-8); the exponential, 2 + 1.17 |u| steps of 2^-23 of an argument |u| <= 88 with four roundings of
    2^-24 in it, and the quotient (2 steps): 2^-14 in all; the normal distribution function is within 5 steps.
    What is flushed is below |z| 2^-126."""
    z = torch.cat([-torch.linspace(0, 12, 300), -torch.logspace(1, math.log10(95), 212)]).to(BF)
    m = Layer(2, 64, 512, (8,), seed=43, act=act)
    m.x.zero_()
    m.x[:, 5] = 1
    m.W.zero_()
    m.W[:, 5] = z.cuda()
    d = z.double()
    want = {"silu": d * torch.special.expit(d), "gelu": d / 2 * torch.special.erfc(-d * math.sqrt(0.5)),
            "gelu_tanh": d * torch.special.expit(2 * math.sqrt(2 / math.pi) * (d + 0.044715 * d ** 3))}[act]
    floor = (d.abs() + 1) * 2.0 ** -126
    tol = (2.0 ** -8 + 2.0 ** -14) * want.abs() + floor
    assert (want.abs() > 2 * floor).sum() > {"silu": 500, "gelu": 320, "gelu_tanh": 245}[act]   # not all floor
    ids = torch.full((2,), -1, dtype=torch.int32)
    for y in (m.bgmv(ids).clone(), m.sgmv(m.segments([0], []))):
        got = y[0].cpu().double()
        bad = ~((got - want).abs() <= tol)
        assert not bad.any(), (d[bad][0].item(), got[bad][0].item(), want[bad][0].item())
