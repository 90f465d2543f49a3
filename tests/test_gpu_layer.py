"""GPU tests of the whole-layer calls lora_bgmv_layer and lora_sgmv_layer against a plain 64-bit
form of their definition,

    z = x W^T + s_i B_i A_i x (+ bias),   y = act(z) * mul + residual,

one adapter at a time on the CPU.  Tolerance per output, derived from the arithmetic:
  * one rounding to bf16: 2^-8 of the result;
  * z: at most h products summed in fp32 with at most a step (2^-23) lost per addition, and the
    adapter's intermediate kept to 2^-17 (bf16 hi + lo) or better, against the sums of the absolute
    products; 1.13 is the largest slope of the activations;
  * the activation itself: fast exponential and division, 2^-18 of |z|.
The last two pass through mul.
"""
import math

import pytest
import torch

import heterogeneous_adapters_sgmv_b200 as L
from tests.gpu_util import kernels_launched, option

pytestmark = pytest.mark.gpu

ACT = {"none": L.LORA_ACT_NONE, "relu": L.LORA_ACT_RELU, "gelu": L.LORA_ACT_GELU, "gelu_tanh": L.LORA_ACT_GELU_TANH,
       "silu": L.LORA_ACT_SILU}
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available()
    L._load()


class Layer:
    """A seeded layer with its adapters; operands may sit in wider buffers (pad columns)."""

    def __init__(self, T, h, o, ranks, seed=0, bias=False, mul=False, residual=False, act="none", pad=0, y_off=0):
        g = torch.Generator().manual_seed(1000 * seed + T + 7 * h + 13 * o)
        self.T, self.h, self.o, self.ranks, self.act, self.y_off = T, h, o, list(ranks), act, y_off
        self.gen = g

        def rnd(rows, cols, scale=1.0):
            wide = (torch.randn(rows, cols + pad, generator=g) * scale).to(BF).cuda()
            return wide[:, :cols]

        self.x, self.W = rnd(T, h), rnd(o, h, h ** -0.5)
        self.A = [(torch.randn(r, h, generator=g) * h ** -0.5).to(BF).cuda() for r in self.ranks]
        self.B = [(torch.randn(o, r, generator=g) * 0.14).to(BF).cuda() for r in self.ranks]
        self.scales = [2.0 / (1 + i % 3) for i in range(len(self.ranks))]
        self.bias = torch.randn(o, generator=g).to(BF).cuda() if bias else None
        self.mul = rnd(T, o) if mul else None
        self.residual = rnd(T, o, 2.0) if residual else None
        self.y = torch.full((T, o + pad + y_off), 7.0, dtype=BF, device="cuda")
        self.table = L.AdapterTable(self.A, self.B, self.ranks, self.scales, h, o, L.LORA_BF16)
        # a workspace that starts as NaN: nothing may depend on what it held
        self.ws = torch.full((self.table.workspace_bytes(T),), 255, dtype=torch.uint8, device="cuda")

    def epilogue(self):
        return L.make_epilogue(bias=self.bias, act=ACT[self.act], mul=self.mul,
                               ldmul=self.mul.stride(0) if self.mul is not None else 0, residual=self.residual,
                               ldres=self.residual.stride(0) if self.residual is not None else 0)

    def ids(self, bare=0.2):
        ids = torch.randint(0, len(self.ranks), (self.T,), generator=self.gen, dtype=torch.int32)
        ids[torch.rand(self.T, generator=self.gen) < bare] = -1
        return ids

    def bgmv(self, ids, y=None, epi=None, ws=None, stream=None):
        y = self.y if y is None else y
        ws = self.ws if ws is None else ws
        d = ids.cuda() if ids is not None else None
        L.lora_bgmv_layer(self.table.handle, d, self.T, self.x, self.x.stride(0), self.W, self.W.stride(0),
                          epi or self.epilogue(), y, y.stride(0), self.y_off, ws, ws.numel(), stream)
        return y

    def segments(self, ptr, adapters):
        dev = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in (ptr, adapters or [0], [len(adapters)])]
        self._segs = dev
        return L.make_segments(None, dev[0], dev[1], dev[2], self.T, len(adapters))

    def sgmv(self, seg, y=None, epi=None, stream=None):
        y = self.y if y is None else y
        L.lora_sgmv_layer(self.table.handle, seg, self.x, self.x.stride(0), self.W, self.W.stride(0),
                          epi or self.epilogue(), y, y.stride(0), self.y_off, self.ws, self.ws.numel(), stream)
        return y

    def reference(self, ids):
        """(y, tolerance) in 64 bits on the CPU."""
        d = lambda t: t.cpu().double()
        x, W = d(self.x), d(self.W)
        z, size = x @ W.t(), x.abs() @ W.abs().t()
        hi_lo = torch.zeros_like(z)
        for i in set(ids.tolist()) - {-1}:
            rows = torch.nonzero(ids == i).flatten()
            A, B, s = d(self.A[i]), d(self.B[i]), self.scales[i]
            z[rows] += s * (x[rows] @ A.t()) @ B.t()
            size[rows] += s * (x[rows].abs() @ A.abs().t()) @ B.abs().t()
            hi_lo[rows] += s * (x[rows] @ A.t()).abs() @ B.abs().t()
        if self.bias is not None:
            z, size = z + d(self.bias), size + d(self.bias).abs()
        off = 1.13 * ((self.h + 130) * 2.0 ** -23 * size + 2.0 ** -17 * hi_lo) + 2.0 ** -18 * z.abs()
        a = {"none": lambda t: t, "relu": lambda t: t.clamp(min=0), "gelu": lambda t: t * torch.special.ndtr(t),
             "gelu_tanh": lambda t: t / 2 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3))),
             "silu": lambda t: t * torch.sigmoid(t)}[self.act](z)
        if self.mul is not None:
            a, off = a * d(self.mul), off * d(self.mul).abs()
        if self.residual is not None:
            a = a + d(self.residual)
        return a, off + 2.0 ** -8 * a.abs() + 1e-30

    def check(self, y, ids, what=""):
        torch.cuda.synchronize()
        ref, tol = self.reference(ids)
        got = y[:, self.y_off:self.y_off + self.o].cpu().double()
        bad = ~((got - ref).abs() <= tol)
        if bad.any():
            i = tuple(int(v) for v in torch.nonzero(bad)[0])
            raise AssertionError("%s: %d of %d outputs off, first at %s: %r, wanted %r +- %r" % (
                what, int(bad.sum()), bad.numel(), i, got[i].item(), ref[i].item(), tol[i].item()))
        # nothing beside the slice is written
        assert (y[:, :self.y_off] == 7.0).all() and (y[:, self.y_off + self.o:] == 7.0).all()
        assert L.lora_get_status(self.table.handle) == (0, 0)


# ------------------------------------------------------------------------------- per-token ids

# sizes around the tiles: 16 tokens an MMA column step, 256 a tile; 128 rows of W a tile; 64 a k-block;
# few W tiles and a long k axis split k over 8 CTAs, a short one over none
@pytest.mark.parametrize("T,h,o", [(1, 8, 8), (1, 4096, 8), (2, 64, 128), (15, 72, 136), (16, 512, 128),
                                   (17, 1000, 264), (33, 200, 1032), (64, 1096, 1000), (130, 128, 520),
                                   (177, 320, 256), (256, 640, 128), (257, 328, 392), (515, 256, 144),
                                   # several token tiles, whose rounded-up size the shares of a cluster of 2, 4
                                   # and 8 have to cover
                                   (260, 128, 264), (261, 304, 136), (777, 128, 64), (521, 520, 72), (389, 192, 72)])
def test_bgmv_layer_sizes(T, h, o):
    m = Layer(T, h, o, (16, 3, 128, 8, 20), seed=1, bias=True, act="silu", mul=True, residual=True)
    ids = m.ids()
    m.check(m.bgmv(ids), ids, "ids")
    none = torch.full((T,), -1, dtype=torch.int32)
    m.check(m.bgmv(None), none, "no ids")
    m.check(m.bgmv(none), none, "ids of -1")


# more than 64 tokens on one CTA of an SM (16 epilogue warps), with k split over 1, 2, 4 and 8 CTAs; from 192
# tokens on tiles of at most 128; more row tiles than the device runs clusters of 8, and of 4
@pytest.mark.parametrize("T,h,o", [(65, 64, 72), (67, 128, 136), (79, 256, 200), (101, 520, 264), (128, 64, 4616),
                                   (191, 136, 128), (192, 136, 128), (250, 264, 72), (253, 640, 136), (287, 72, 64),
                                   (288, 72, 64), (386, 200, 136), (70, 520, 2048), (5, 520, 2056), (3, 264, 4616)])
def test_bgmv_layer_wide_epilogues_and_clusters(T, h, o):
    m = Layer(T, h, o, (128, 5, 16, 64, 40), seed=30, bias=True, act="gelu", mul=True, residual=True, pad=8)
    ids = m.ids()
    m.check(m.bgmv(ids), ids, "ids")
    bad = ids.clone()
    bad[T // 2:] = 5                               # an adapter that is not there: its rows are left alone
    m.y.fill_(7.0)
    m.bgmv(bad)
    torch.cuda.synchronize()
    assert (m.y[T // 2:] == 7.0).all()
    assert L.lora_get_status(m.table.handle) == (L.LORA_ERR_DEVICE_STATUS, L.LORA_STATUS_BAD_ID)
    none = torch.full((T,), -1, dtype=torch.int32)
    m.check(m.bgmv(none), none, "ids of -1")
    m.check(m.bgmv(None), none, "no ids")


# tables of one rank and of several: multiples of 8 up to 64, 64 alone and 128 (the rows of a warp read as one
# block), others (rows that begin and end inside 16 bytes)
@pytest.mark.parametrize("ranks", [(8, 64, 24), (64,), (128, 64), (128, 16, 48), (1,), (3, 2), (7, 9, 15), (60, 12),
                                   (127, 121), (125, 64, 8, 128)])
@pytest.mark.parametrize("T,h,o", [(3, 72, 8), (18, 264, 1032), (45, 64, 40), (45, 136, 19208), (99, 128, 264)])
def test_bgmv_layer_ranks(T, h, o, ranks):
    m = Layer(T, h, o, ranks, seed=31, act="silu", mul=True)
    ids = m.ids(bare=0.1)
    m.check(m.bgmv(ids), ids)


@pytest.mark.parametrize("T", [3, 40, 90])
@pytest.mark.parametrize("ranks", [(64, 128), (5, 12), (8, 40)])
def test_bgmv_layer_keeps_rows_of_an_adapter_apart(T, ranks):
    """A row of B that is not finite reaches its own output column and no other."""
    m = Layer(T, 136, 264, ranks, seed=32)
    for B in m.B:
        B[[0, 37, 263]] = float("nan")
    ids = m.ids(bare=0.0)
    y = m.bgmv(ids)
    torch.cuda.synchronize()
    nan = torch.zeros(264, dtype=torch.bool, device="cuda")
    nan[[0, 37, 263]] = True
    assert y[:, nan].isnan().all() and y[:, ~nan].isfinite().all()
    for B in m.B:
        B[[0, 37, 263]] = 0.0
    m.check(m.bgmv(ids), ids)


@pytest.mark.parametrize("act", sorted(ACT))
@pytest.mark.parametrize("bias,mul,residual", [(False, False, False), (True, False, False), (False, True, False),
                                               (False, False, True), (True, True, True)])
def test_bgmv_layer_epilogues(act, bias, mul, residual):
    m = Layer(21, 136, 152, (16, 1, 9), seed=2, act=act, bias=bias, mul=mul, residual=residual, pad=24, y_off=16)
    ids = m.ids()
    m.check(m.bgmv(ids), ids, act)


def test_bgmv_layer_without_epilogue():
    m = Layer(5, 264, 264, (8,), seed=3)
    ids = m.ids()
    L.lora_bgmv_layer(m.table.handle, ids.cuda(), m.T, m.x, m.h, m.W, m.h, None, m.y, m.o, 0, m.ws, m.ws.numel())
    m.check(m.y, ids)


def test_bgmv_layer_in_place():
    """y holds the residual (or the gate) and takes the result."""
    for name in ("residual", "mul"):
        m = Layer(40, 512, 384, (16, 64), seed=4, act="gelu", **{name: True})
        ids = m.ids()
        y = getattr(m, name).clone()
        epi = L.make_epilogue(act=ACT["gelu"], **({"residual": y, "ldres": m.o} if name == "residual" else
                                                  {"mul": y, "ldmul": m.o}))
        m.check(m.bgmv(ids, y=y, epi=epi), ids, name)


def test_bgmv_layer_bad_ids_leave_their_rows():
    m = Layer(20, 256, 256, (16, 8), seed=5, residual=True)
    ids = m.ids(bare=0.1)
    bad = ids.clone()
    bad[3], bad[11], bad[19] = 2, -2, 2 ** 31 - 1
    y = m.bgmv(bad)
    rc, word = L.lora_get_status(m.table.handle)
    assert rc == L.LORA_ERR_DEVICE_STATUS and word == L.LORA_STATUS_BAD_ID
    rows = torch.tensor([3, 11, 19], device="cuda")
    assert (y[rows] == 7.0).all()
    ref, tol = m.reference(ids)
    keep = torch.tensor([i for i in range(20) if i not in (3, 11, 19)])
    assert ((y.cpu().double() - ref).abs() <= tol)[keep].all()


def test_bgmv_layer_rows_do_not_mix():
    """A token of infinities or NaN spoils its own row only; so does an adapter of NaN."""
    m = Layer(19, 256, 384, (16, 16), seed=6, act="silu", residual=True)
    ids = torch.tensor([i % 2 for i in range(19)], dtype=torch.int32)
    clean = m.bgmv(ids).clone()
    m.x[4] = float("nan")
    m.x[7] = float("inf")
    m.residual[9] = float("inf")
    y = m.bgmv(ids, y=torch.empty_like(m.y))
    same = [i for i in range(19) if i not in (4, 7, 9)]
    assert torch.equal(y[same], clean[same])
    assert y[4].isnan().all() and (y[9] == float("inf")).all() and not y[7].isfinite().any()
    m = Layer(19, 256, 384, (16, 16), seed=6, act="silu", residual=True)
    m.A[1].fill_(float("nan"))
    y = m.bgmv(ids, y=torch.empty_like(m.y))
    assert torch.equal(y[0::2], clean[0::2]) and y[1::2].isnan().all()


def test_relu_keeps_nan_and_large_values():
    m = Layer(4, 64, 64, (8,), seed=7, act="relu")
    m.x[1] = float("nan")
    assert m.bgmv(None)[1].isnan().all()
    for act in ("silu", "gelu", "gelu_tanh"):   # far out the activations are 0 and z
        m = Layer(2, 64, 64, (8,), seed=7, act=act)
        m.x.fill_(0)
        m.x[:, 0] = 1
        m.W.fill_(0)
        m.W[:32, 0], m.W[32:, 0] = 1e30, -1e30
        y = m.bgmv(None)
        assert (y[:, :32] == m.W[0, 0]).all() and (y[:, 32:] == 0).all()


def test_bgmv_layer_same_bits_each_run_and_without_programmatic_launch():
    m = Layer(64, 2048, 512, (16, 64, 8), seed=8, act="silu", mul=True)
    ids = m.ids()
    a = m.bgmv(ids).clone()
    for _ in range(5):
        assert torch.equal(m.bgmv(ids), a)
    with option("pdl", 0):
        assert torch.equal(m.bgmv(ids), a)
    names = kernels_launched(lambda: m.bgmv(ids))
    assert names == {"layer_shrink_kernel", "layer_stream_kernel"}
    assert kernels_launched(lambda: m.bgmv(None)) == {"layer_stream_kernel"}


@pytest.mark.parametrize("T,h,o", [(192, 128, 264), (257, 264, 136), (600, 72, 1032)])
def test_bgmv_layer_without_adapters_in_large_batches(T, h, o):
    """Without ids large batches take the tiles of the segment form; a table of any ranks will do."""
    m = Layer(T, h, o, (3, 128), seed=9, act="silu", mul=True, residual=True, pad=8, y_off=16)
    none = torch.full((T,), -1, dtype=torch.int32)
    assert kernels_launched(lambda: m.bgmv(None)) == {"layer_gemm_kernel"}
    m.check(m.y, none)


# ------------------------------------------------------------------------------- segments

def _ids_of(T, ptr, adapters):
    ids = torch.full((T,), -1, dtype=torch.int32)
    for s, a in enumerate(adapters):
        ids[ptr[s]:ptr[s + 1]] = a
    return ids


# row tiles are 256 tokens wide wherever the segments lie: segments inside one tile, across several, empty
# ones, rows before the first and behind the last
@pytest.mark.parametrize("T,h,o,ptr", [
    (1, 64, 8, [0, 1]), (5, 8, 264, [0, 5]), (256, 128, 256, [0, 256]), (512, 512, 512, [0, 128, 512]),
    (300, 1000, 136, [20, 20, 120, 250, 257, 290]), (777, 264, 520, [0, 1, 2, 300, 301, 700, 777]),
    (1030, 192, 768, [5, 255, 256, 258, 1020, 1030]), (129, 64, 64, [129, 129])])
def test_sgmv_layer_segments(T, h, o, ptr):
    m = Layer(T, h, o, (64, 16, 8, 40), seed=11, bias=True, act="gelu_tanh", mul=True, residual=True)
    adapters = [(3 * s) % 4 for s in range(len(ptr) - 1)]
    m.check(m.sgmv(m.segments(ptr, adapters)), _ids_of(T, ptr, adapters))


def test_sgmv_layer_many_short_segments():
    T = 611
    m = Layer(T, 128, 264, (8, 16, 64), seed=12, residual=True)
    ptr, s = [3], 0
    while ptr[-1] < T - 4:
        ptr.append(ptr[-1] + 1 + s % 3)
        s += 1
    adapters = [i % 3 for i in range(len(ptr) - 1)]
    assert len(adapters) > 250
    m.check(m.sgmv(m.segments(ptr, adapters)), _ids_of(T, ptr, adapters))


@pytest.mark.parametrize("act", sorted(ACT))
@pytest.mark.parametrize("bias,mul,residual", [(False, False, False), (True, False, False), (False, True, False),
                                               (False, False, True), (True, True, True)])
def test_sgmv_layer_epilogues(act, bias, mul, residual):
    m = Layer(290, 136, 296, (16, 64), seed=13, act=act, bias=bias, mul=mul, residual=residual, pad=24, y_off=8)
    ptr = [10, 130, 280]
    m.check(m.sgmv(m.segments(ptr, [1, 0])), _ids_of(290, ptr, [1, 0]), act)


def test_sgmv_layer_no_segments_and_in_place():
    m = Layer(270, 256, 264, (16,), seed=14, act="relu", residual=True)
    none = torch.full((270,), -1, dtype=torch.int32)
    m.check(m.sgmv(m.segments([0], [])), none, "no segments")
    y = m.residual.clone()
    epi = L.make_epilogue(act=ACT["relu"], residual=y, ldres=m.o)
    m.check(m.sgmv(m.segments([0, 270], [0]), y=y, epi=epi), torch.zeros(270, dtype=torch.int32), "in place")


def test_sgmv_layer_more_tiles_than_pairs():
    """Each pair of CTAs runs several tiles, so both accumulators are used again."""
    T, o = 1400, 8200
    m = Layer(T, 72, o, (16, 32), seed=15, act="silu", mul=True)
    ptr = [0, 100, 800, 1399]
    m.check(m.sgmv(m.segments(ptr, [0, 1, 0])), _ids_of(T, ptr, [0, 1, 0]))


def test_sgmv_layer_reports_bad_segments():
    m = Layer(300, 128, 128, (16, 8), seed=16)
    y = m.sgmv(m.segments([0, 100, 200, 300], [0, 7, 1]))
    rc, word = L.lora_get_status(m.table.handle)
    assert rc == L.LORA_ERR_DEVICE_STATUS and word == L.LORA_STATUS_BAD_SEGMENT
    m.check(y, _ids_of(300, [0, 100, 200, 300], [0, -1, 1]), "rows of the unknown adapter get the base product")


def test_sgmv_layer_agrees_with_the_base_call():
    """Without an epilogue it computes what lora_sgmv_base does, and so does the per-token form."""
    T, h, o = 512, 1024, 768
    m = Layer(T, h, o, (64, 16), seed=17)
    ptr = [0, 256, 512]
    seg = m.segments(ptr, [0, 1])
    ids = _ids_of(T, ptr, [0, 1])
    base = torch.empty_like(m.y)
    L.lora_sgmv_base(m.table.handle, seg, m.x, h, m.W, h, base, o, 0, False, m.ws, m.ws.numel())
    for y in (base, m.sgmv(seg).clone(), m.bgmv(ids).clone()):
        m.y = y
        m.check(y, ids)


# ------------------------------------------------------------------------------- together

def test_layers_captured_and_on_two_streams():
    """One graph of both forms, replayed with new inputs, beside eager calls with their own workspace
    on another stream."""
    a = Layer(33, 256, 512, (16, 8), seed=21, act="silu", residual=True)
    b = Layer(300, 512, 256, (64, 16), seed=22, act="gelu", bias=True)
    ids = a.ids()
    ids_d = ids.cuda()
    ptr, ads = [0, 130, 300], [1, 0]
    seg = b.segments(ptr, ads)
    other = Layer(48, 640, 384, (16,), seed=23, mul=True)
    o_ids = other.ids()
    o_want = other.bgmv(o_ids).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def both():
        L.lora_bgmv_layer(a.table.handle, ids_d, a.T, a.x, a.h, a.W, a.h, a.epilogue(), a.y, a.o, 0, a.ws, a.ws.numel())
        b.sgmv(seg)

    with torch.cuda.stream(s):
        both()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        both()
    for k in range(3):
        a.x.copy_(torch.randn(a.T, a.h, generator=a.gen).to(BF))
        b.x.copy_(torch.randn(b.T, b.h, generator=b.gen).to(BF))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        got = other.bgmv(o_ids, y=torch.empty_like(other.y))
        torch.cuda.synchronize()
        assert torch.equal(got, o_want)
        a.check(a.y, ids, "replay %d" % k)
        b.check(b.y, _ids_of(300, ptr, ads), "replay %d" % k)


def test_layer_refuses_a_short_workspace_and_another_device():
    m = Layer(9, 64, 64, (8,), seed=24)
    with pytest.raises(L.LoraError) as e:
        L.lora_bgmv_layer(m.table.handle, m.ids().cuda(), 9, m.x, 64, m.W, 64, None, m.y, 64, 0, m.ws, 64)
    assert e.value.code == L.LORA_ERR_WORKSPACE
    assert (m.y == 7.0).all()


@pytest.mark.parametrize("bit,T,form", [(8, 5, "bgmv"), (8, 70, "bgmv"), (8, 300, "bgmv"), (16, 300, "sgmv")])
def test_layer_wait_runs_out_then_recovers(bit, T, form):
    """A stage that is armed and never loaded: with the bound at 20 ms the waits on it run out, the status
    word says so, and the next call on the same table runs as if nothing had been."""
    m = Layer(T, 1024, 392, (16, 8), seed=25, act="silu", mul=True, residual=True)
    ptr, ads = [0, T // 2, T], [0, 1]
    ids = _ids_of(T, ptr, ads)
    call = (lambda: m.bgmv(ids)) if form == "bgmv" else (lambda: m.sgmv(m.segments(ptr, ads)))
    with option("wait_limit_ns", 20_000_000), option("inject_stall", bit):
        call()
        torch.cuda.synchronize()
    rc, word = L.lora_get_status(m.table.handle)
    assert rc == L.LORA_ERR_TIMEOUT and word == L.LORA_STATUS_TIMEOUT
    call()
    m.check(m.y, ids, "after a timeout")
