"""GPU tests of forms of the layer calls that the sizes in test_gpu_layer.py do not reach, with that file's
layer, 64-bit reference and tolerances."""
import math

import pytest
import torch

import heterogeneous_adapters_sgmv_b200 as L
from tests.test_gpu_layer import BF, Layer, _ids_of

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


# (tokens, h, o): the ring of the weight pass goes round at least twice with k split over 1, 2, 4 and 8 CTAs, one and
# two to an SM; the partial sums land beside the ring and in it; the scaled intermediate comes in one to four parts.
# test_layer_shape.py holds that these sizes do so.
ROUNDS = [(1, 1032, 15240), (120, 648, 9480), (40, 520, 19208), (40, 2120, 4616), (390, 1352, 1032), (512, 840, 2312),
          (70, 840, 9480), (40, 3784, 2056), (1030, 2248, 136), (1, 2760, 5128), (63, 1736, 5128), (129, 3528, 72),
          (40, 3528, 2312), (63, 3528, 2312), (33, 4104, 136), (256, 3080, 2056), (512, 1160, 2312),
          (129, 4616, 72), (40, 4360, 2056)]


@pytest.mark.parametrize("ranks", [(16, 40, 8), (128, 5, 64)])
@pytest.mark.parametrize("T,h,o", ROUNDS)
def test_bgmv_layer_long_rings(T, h, o, ranks):
    m = Layer(T, h, o, ranks, seed=44, bias=True, act="silu", mul=True, residual=True, pad=8)
    ids = m.ids()
    m.check(m.bgmv(ids), ids, "ids")
    first = m.y.clone()
    none = torch.full((T,), -1, dtype=torch.int32)
    m.check(m.bgmv(None), none, "no ids")
    assert torch.equal(m.bgmv(ids), first)


def _cut(T, step):
    ptr = [3]
    while ptr[-1] + step < T - 2:
        ptr.append(ptr[-1] + step)
    return ptr, [s % 3 for s in range(len(ptr) - 1)]


# more tiles than pairs of CTAs, so that each pair uses its accumulators, operand tiles and barriers again: 198
# wide tiles, 180 narrow ones (the narrower width where it ends sooner); k axes of one, two and four k-blocks; a
# few segments a tile and ten
@pytest.mark.parametrize("bias,mul,residual", [(True, True, True), (False, True, True), (False, False, True),
                                               (True, True, False), (False, False, False)])
@pytest.mark.parametrize("h,step", [(64, 300), (72, 25), (200, 150)])
@pytest.mark.parametrize("o", [8200, 3720])
def test_sgmv_layer_several_tiles_a_pair(o, h, step, bias, mul, residual):
    T = 1400
    m = Layer(T, h, o, (64, 16, 8), seed=45, act="silu", bias=bias, mul=mul, residual=residual, pad=8)
    ptr, adapters = _cut(T, step)
    m.check(m.sgmv(m.segments(ptr, adapters)), _ids_of(T, ptr, adapters))
    first = m.y.clone()
    assert torch.equal(m.sgmv(m.segments(ptr, adapters)), first)


def test_layers_of_clusters_on_three_streams():
    """Small layers whose clusters share the device: two streams of the per-token form and one of the segment form,
    many calls in flight at once, each with its own workspace."""
    a = Layer(161, 72, 128, (16, 8), seed=46, act="silu")
    b = Layer(250, 264, 1032, (16, 8), seed=47, residual=True)
    c = Layer(300, 512, 264, (64, 16), seed=48, act="gelu")
    ids = [a.ids().cuda(), b.ids().cuda()]
    seg = c.segments([0, 130, 300], [1, 0])

    def call(m, i, y, stream=None):
        if m is c:
            m.sgmv(seg, y=y, stream=stream)
        else:
            L.lora_bgmv_layer(m.table.handle, ids[i], m.T, m.x, m.h, m.W, m.h, m.epilogue(), y, m.o, 0, m.ws,
                              m.ws.numel(), stream)
        return y

    layers = (a, b, c)
    want = [call(m, i, torch.empty_like(m.y)) for i, m in enumerate(layers)]
    a.check(want[0], ids[0].cpu())
    streams = [torch.cuda.Stream() for _ in layers]
    outs = [[torch.zeros_like(m.y) for _ in range(40)] for m in layers]
    torch.cuda.synchronize()
    for k in range(40):
        for i, m in enumerate(layers):
            call(m, i, outs[i][k], streams[i])
    torch.cuda.synchronize()
    for i, m in enumerate(layers):
        assert all(torch.equal(y, want[i]) for y in outs[i])
        assert L.lora_get_status(m.table.handle) == (0, 0)


@pytest.mark.parametrize("with_ids", [False, True])
def test_bgmv_layer_takes_weights_written_just_before(with_ids):
    m = Layer(5, 1024, 2056, (16, 8), seed=49, bias=True)
    ids = m.ids(bare=0.0) if with_ids else None
    d = ids.cuda() if with_ids else None
    both = [(m.W.clone(), m.bias.clone()), (m.W * 2, m.bias * -1)]

    def call(y):
        L.lora_bgmv_layer(m.table.handle, d, m.T, m.x, m.h, m.W, m.h, m.epilogue(), y, m.o, 0, m.ws, m.ws.numel())
        return y

    want, outs = [], []
    for W, bias in both:
        m.W.copy_(W)
        m.bias.copy_(bias)
        torch.cuda.synchronize()
        want.append(call(torch.empty_like(m.y)))
        torch.cuda.synchronize()
    for k in range(40):
        m.bias.copy_(both[k % 2][1])
        m.W.copy_(both[k % 2][0])
        outs.append(call(torch.empty_like(m.y)))
    torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])
    assert all(torch.equal(y, want[k % 2]) for k, y in enumerate(outs))
