"""GPU tests of the norms around a block (lora_norm_before, lora_norm_after) against a plain 64-bit
form of their definition on the CPU.

Tolerance per output, derived from the arithmetic.  A sum over a row passes at most 48 additions per
value (32 in a thread, 10 levels of shuffles, the rest to spare), so a mean or a mean square is within
48 half steps (2^-24) of its terms' absolute mean, and the reciprocal root halves that and adds a few
steps: a normalised value is within 64 * 2^-24 of (|x| + mean |x|) / sqrt(var + eps), times its gain.
The products and sums behind it add three half steps each.  The norm of a rounded-off r passes its
input's error on, divided by its own root.  Then one rounding to the output's type (2^-8 for bf16, 2^-24
for fp32)."""
import pytest
import torch

import heterogeneous_adapters_sgmv_b200 as L
from tests.gpu_util import kernels_launched, option

pytestmark = pytest.mark.gpu

TYPES = {"bf16": (torch.bfloat16, L.LORA_BF16, 2.0 ** -8), "f32": (torch.float32, L.LORA_F32, 2.0 ** -24)}
KIND = {"rms": L.LORA_NORM_RMS, "layer": L.LORA_NORM_LAYER}
GATE = {"none": L.LORA_GATE_NONE, "adapter": L.LORA_GATE_ADAPTER, "token": L.LORA_GATE_TOKEN}
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available()
    L._load()


class Norms:
    def __init__(self, T, d, dtype="bf16", n=5, seed=0, pad=0):
        self.E, self.code, self.half = TYPES[dtype]
        self.T, self.d, self.n, self.pad = T, d, n, pad
        self.g = torch.Generator().manual_seed(100 * seed + T + 3 * d)
        w = torch.zeros(8 * d, dtype=self.E, device="cuda")
        self.table = L.AdapterTable([w] * n, [w] * n, [8] * n, [1.0] * n, d, d, self.code, keep=w)

    def rnd(self, rows, scale=1.0, mean=0.0):
        wide = (torch.randn(rows, self.d + self.pad, generator=self.g) * scale + mean).to(self.E).cuda()
        return wide[:, :self.d]

    def out(self):
        return torch.full((self.T, self.d + self.pad), 7.0, dtype=self.E, device="cuda")[:, :self.d]

    def ids(self):
        ids = torch.randint(-1, self.n, (self.T,), generator=self.g, dtype=torch.int32)
        return ids

    def norm(self, kind, rows=1, shift=True, gain=True, eps=1e-5):
        w = dict(kind=kind, eps=eps, gain=self.rnd(rows, 0.3, 1.0) if gain else None,
                 shift=self.rnd(rows, 0.5) if shift else None)
        ld = 0 if rows == 1 else self.d + self.pad
        w["arg"] = L.make_norm(KIND[kind], eps, gain=w["gain"], shift=w["shift"], ld=ld)
        return w


def rows_of(w, ids, T):
    if w is None:
        return None
    w = w.cpu().double()
    return w.expand(T, -1) if w.shape[0] == 1 else w[(ids + 1).long()]


def norm_ref(x, off, w, ids):
    """N(x) in 64 bits, and how far fp32 may be off where x itself is off by `off`."""
    T = x.shape[0]
    g = rows_of(w["gain"], ids, T)
    b = rows_of(w["shift"], ids, T)
    mean = x.mean(1, keepdim=True) if w["kind"] == "layer" else torch.zeros(T, 1).double()
    c = x - mean
    inv = 1 / (c.square().mean(1, keepdim=True) + w["eps"]).sqrt()
    y = c * inv
    size = (x.abs() + x.abs().mean(1, keepdim=True)) * inv
    o = 64 * U * size + (off + off.mean(1, keepdim=True)) * inv + y.abs() * (c.abs() * off).mean(1, keepdim=True) * inv ** 2
    if g is not None:
        y, o = y * g, (o + 3 * U * y.abs()) * g.abs()
    if b is not None:
        y = y + b
        o = o + 3 * U * (y.abs() + b.abs())
    return y, o


def close(got, ref, off, half, what):
    torch.cuda.synchronize()
    got = got.cpu().double()
    tol = off + half * ref.abs() + 1e-30
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        i = tuple(int(v) for v in torch.nonzero(bad)[0])
        raise AssertionError("%s: %d of %d off, first at %s: %r, wanted %r +- %r" % (
            what, int(bad.sum()), bad.numel(), i, got[i].item(), ref[i].item(), tol[i].item()))


# widths around what a block of each size holds, and the widest
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1, 8), (3, 64), (5, 256), (2, 264), (7, 512), (33, 1000), (9, 1032), (4, 2048),
                                 (3, 2056), (300, 4096), (2, 5120), (5, 8192), (3, 8200), (2, 16384)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_before(dtype, T, d, kind):
    m = Norms(T, d, dtype, pad=16)
    x = m.rnd(T, 3.0, 0.5)
    ids = m.ids()
    zero = torch.zeros(T, m.d).double()
    for rows, the_ids, shift, gain in ((1, None, True, True), (1 + m.n, ids, False, True), (1 + m.n, ids, True, True),
                                       (1 + m.n, None, False, True), (1, ids, False, False)):
        w = m.norm(kind, rows, shift, gain)
        h = m.out()
        L.lora_norm_before(m.table.handle, the_ids.cuda() if the_ids is not None else None, T, d, x, x.stride(0),
                           w["arg"], h, h.stride(0))
        ref, off = norm_ref(x.cpu().double(), zero, w, the_ids if the_ids is not None else torch.full((T,), -1))
        close(h, ref, off, m.half, "%s rows %d" % (kind, rows))
        assert (h._base[:, d:] == 7.0).all()
    assert L.lora_get_status(m.table.handle) == (0, 0)


@pytest.mark.parametrize("dtype,T,d", [("bf16", 1, 4096), ("bf16", 37, 1000), ("f32", 18, 520), ("bf16", 3, 16384),
                                       ("f32", 2, 16384)])
@pytest.mark.parametrize("kind", ["none", "rms", "layer"])
@pytest.mark.parametrize("nxt", ["none", "rms", "layer"])
@pytest.mark.parametrize("gate", ["none", "adapter", "token"])
def test_norm_after(dtype, T, d, kind, nxt, gate):
    m = Norms(T, d, dtype, seed=2, pad=8)
    z, res = m.rnd(T, 2.0, 0.3), m.rnd(T, 4.0, -0.2)
    ids = m.ids()
    w = m.norm(kind, 1 + m.n) if kind != "none" else None
    w2 = m.norm(nxt, 1 + m.n, shift=False) if nxt != "none" else None
    gt = None if gate == "none" else m.rnd(T if gate == "token" else 1 + m.n, 0.5, 0.5)
    a, c = 0.75, -1.5
    for with_res in (True, False):
        arg = L.make_residual(residual=res if with_res else None, ldres=res.stride(0), gate=gt,
                              ldgate=gt.stride(0) if gt is not None else 0, gate_kind=GATE[gate], res_scale=a,
                              branch_scale=c)
        r, h = m.out(), m.out()
        L.lora_norm_after(m.table.handle, ids.cuda(), T, d, z, z.stride(0), w and w["arg"], arg, r, r.stride(0),
                          w2 and w2["arg"], h if w2 else None, h.stride(0))
        u, off = z.cpu().double(), torch.zeros(T, d).double()
        if w:
            u, off = norm_ref(u, off, w, ids)
        if gt is not None:
            gg = gt.cpu().double() if gate == "token" else rows_of(gt, ids, T)
            u, off = u * gg, off * gg.abs()
        part = a * res.cpu().double() if with_res else torch.zeros(T, d).double()
        ref = part + c * u
        off = abs(c) * (off + 3 * U * u.abs()) + 3 * U * (part.abs() + ref.abs())
        close(r, ref, off, m.half, "r")
        assert (r._base[:, d:] == 7.0).all() and (h._base[:, d:] == 7.0).all()
        if w2:
            ref2, off2 = norm_ref(ref, off, w2, ids)
            close(h, ref2, off2, m.half, "h")
            only = m.out()      # h alone, without r
            L.lora_norm_after(m.table.handle, ids.cuda(), T, d, z, z.stride(0), w and w["arg"], arg, None, 0,
                              w2["arg"], only, only.stride(0))
            assert torch.equal(only, h)
    assert L.lora_get_status(m.table.handle) == (0, 0)


def test_norms_in_place():
    m = Norms(9, 1024, seed=3)
    w, w2, ids = m.norm("layer", 6), m.norm("rms", 6), m.ids().cuda()
    x, res = m.rnd(9), m.rnd(9)
    h = m.out()
    L.lora_norm_before(m.table.handle, ids, 9, 1024, x, 1024, w["arg"], h, 1024)
    y = x.clone()
    L.lora_norm_before(m.table.handle, ids, 9, 1024, y, 1024, w["arg"], y, 1024)
    assert torch.equal(h, y)
    r, h = m.out(), m.out()
    L.lora_norm_after(m.table.handle, ids, 9, 1024, x, 1024, w["arg"], L.make_residual(res, 1024), r, 1024, w2["arg"],
                      h, 1024)
    z, s = x.clone(), res.clone()   # the residual stream and the block's output take the results
    L.lora_norm_after(m.table.handle, ids, 9, 1024, z, 1024, w["arg"], L.make_residual(s, 1024), s, 1024, w2["arg"], z,
                      1024)
    assert torch.equal(s, r) and torch.equal(z, h)


def test_norms_bad_ids_leave_their_rows():
    m = Norms(12, 256, seed=4)
    w = m.norm("rms", 6)
    x = m.rnd(12)
    ids = m.ids()
    good, bad = m.out(), m.out()
    L.lora_norm_before(m.table.handle, ids.cuda(), 12, 256, x, 256, w["arg"], good, 256)
    ids[2], ids[7] = 5, -7
    L.lora_norm_before(m.table.handle, ids.cuda(), 12, 256, x, 256, w["arg"], bad, 256)
    assert L.lora_get_status(m.table.handle) == (L.LORA_ERR_DEVICE_STATUS, L.LORA_STATUS_BAD_ID)
    keep = [i for i in range(12) if i not in (2, 7)]
    assert (bad[[2, 7]] == 7.0).all() and torch.equal(bad[keep], good[keep])
    r = m.out()
    L.lora_norm_after(m.table.handle, ids.cuda(), 12, 256, x, 256, w["arg"], L.make_residual(), r, 256)
    assert L.lora_get_status(m.table.handle) == (L.LORA_ERR_DEVICE_STATUS, L.LORA_STATUS_BAD_ID)
    assert (r[[2, 7]] == 7.0).all() and not (r[keep] == 7.0).all()


def test_norm_rows_with_nothing_in_them():
    """A row of zeros gives the shift; constant rows have no variance; infinities stay in their row."""
    m = Norms(4, 512, "f32", seed=5)
    x = m.rnd(4)
    x[0] = 0
    x[1] = 1000.25
    x[2] = float("inf")
    for kind in ("rms", "layer"):
        w = m.norm(kind)
        h = m.out()
        L.lora_norm_before(m.table.handle, None, 4, 512, x, 512, w["arg"], h, 512)
        assert torch.equal(h[0], w["shift"][0])
        if kind == "layer":
            assert torch.equal(h[1], w["shift"][0])
        assert not h[2].isfinite().any()
        ref, off = norm_ref(x[3:].cpu().double(), torch.zeros(1, 512).double(), w, torch.tensor([-1]))
        close(h[3:], ref, off, m.half, kind)


def test_layer_norm_of_a_large_mean():
    """The variance is taken from centred values: a mean 2000 times the spread costs no more than the
    centring does."""
    m = Norms(6, 4096, "f32", seed=6)
    x = m.rnd(6, 1.0, 2000.0)
    w = m.norm("layer")
    h = m.out()
    L.lora_norm_before(m.table.handle, None, 6, 4096, x, 4096, w["arg"], h, 4096)
    ref, off = norm_ref(x.cpu().double(), torch.zeros(6, 4096).double(), w, torch.full((6,), -1))
    close(h, ref, off, m.half, "large mean")


# many rows: persistent blocks with a ring in shared memory, whose depth falls with the width (four rows of
# the narrow ones; where not even two fit, as of the widest rows in 32 bits with their weights, a block takes
# one row); the last blocks get fewer rows than the first
@pytest.mark.parametrize("dtype,T,d", [("bf16", 4001, 64), ("bf16", 1777, 1032), ("bf16", 2500, 2048),
                                       ("bf16", 3003, 4096), ("bf16", 1800, 8200), ("bf16", 1777, 16384),
                                       ("f32", 1901, 520), ("f32", 1777, 4096), ("f32", 1776, 16384)])
def test_norms_of_many_rows(dtype, T, d):
    m = Norms(T, d, dtype, seed=7, pad=8)
    x, res = m.rnd(T, 2.0, 0.3), m.rnd(T, 3.0)
    ids = m.ids()
    zero = torch.zeros(T, d).double()
    w, w2 = m.norm("layer", 1 + m.n), m.norm("rms", 1)
    h = m.out()
    names = kernels_launched(lambda: L.lora_norm_before(m.table.handle, ids.cuda(), T, d, x, x.stride(0), w["arg"], h,
                                                        h.stride(0)))
    assert names == {"ring_norm_kernel" if d * x.element_size() < 65536 else "block_norm_kernel"}
    ref, off = norm_ref(x.cpu().double(), zero, w, ids)
    close(h, ref, off, m.half, "before")
    gate = m.rnd(T, 0.5, 0.5)
    arg = L.make_residual(residual=res, ldres=res.stride(0), gate=gate, ldgate=gate.stride(0), gate_kind=L.LORA_GATE_TOKEN,
                          res_scale=0.5, branch_scale=2.0)
    r, h2 = m.out(), m.out()
    bad = ids.clone()
    bad[::97] = m.n
    L.lora_norm_after(m.table.handle, bad.cuda(), T, d, x, x.stride(0), w["arg"], arg, r, r.stride(0), w2["arg"], h2,
                      h2.stride(0))
    assert L.lora_get_status(m.table.handle) == (L.LORA_ERR_DEVICE_STATUS, L.LORA_STATUS_BAD_ID)
    g = gate.cpu().double()
    u, off = ref * g * 2.0, off * g.abs() * 2.0
    part = 0.5 * res.cpu().double()
    off = off + 6 * U * u.abs() + 3 * U * (part.abs() + (part + u).abs())
    ref2, off2 = norm_ref(part + u, off, w2, ids)
    for got, want, o in ((r, part + u, off), (h2, ref2, off2)):
        assert (got[::97] == 7.0).all()
        keep = torch.arange(T) % 97 != 0
        close(got[keep.cuda()], want[keep], o[keep], m.half, "after")
    assert (r._base[:, d:] == 7.0).all() and (h._base[:, d:] == 7.0).all()


def test_norm_rows_in_place_ahead_of_the_ring():
    """Rows are read ahead of the block that writes them in place."""
    T, d = 5000, 1024
    m = Norms(T, d, seed=8)
    w, w2, ids = m.norm("rms", 6), m.norm("layer", 6), m.ids().cuda()
    z, s = m.rnd(T), m.rnd(T)
    r, h = m.out(), m.out()
    L.lora_norm_after(m.table.handle, ids, T, d, z, d, w["arg"], L.make_residual(s, d), r, d, w2["arg"], h, d)
    L.lora_norm_after(m.table.handle, ids, T, d, z, d, w["arg"], L.make_residual(s, d), s, d, w2["arg"], z, d)
    assert torch.equal(s, r) and torch.equal(z, h)


def test_norm_wait_runs_out_then_recovers():
    m = Norms(3000, 512, seed=9)
    w, x = m.norm("rms"), m.rnd(3000)
    good, h = m.out(), m.out()
    L.lora_norm_before(m.table.handle, None, 3000, 512, x, 512, w["arg"], good, 512)
    with option("wait_limit_ns", 20_000_000), option("inject_stall", 32):
        L.lora_norm_before(m.table.handle, None, 3000, 512, x, 512, w["arg"], h, 512)
        torch.cuda.synchronize()
    assert L.lora_get_status(m.table.handle) == (L.LORA_ERR_TIMEOUT, L.LORA_STATUS_TIMEOUT)
    assert (h == 7.0).all()
    L.lora_norm_before(m.table.handle, None, 3000, 512, x, 512, w["arg"], h, 512)
    assert torch.equal(h, good)


# ------------------------------------------------------------------------------- together

def test_a_block_of_norms_and_layers():
    """norm before -> gated MLP with adapters -> norm after, as a served block runs them, in the per-token
    form and in the segment form, eagerly and from a graph; the two forms agree with the 64-bit block."""
    T, d, f, n = 272, 512, 1024, 3
    g = torch.Generator().manual_seed(9)
    bf = lambda *s, k=1.0, m=0.0: (torch.randn(*s, generator=g) * k + m).to(torch.bfloat16).cuda()
    x = bf(T, d)
    W = {"up": bf(f, d, k=d ** -0.5), "gate": bf(f, d, k=d ** -0.5), "down": bf(d, f, k=f ** -0.5)}
    tabs, AB = {}, {}
    for name, (hi, ho) in {"up": (d, f), "gate": (d, f), "down": (f, d)}.items():
        A = [bf(16, hi, k=hi ** -0.5) for _ in range(n)]
        B = [bf(ho, 16, k=0.1) for _ in range(n)]
        AB[name] = (A, B)
        tabs[name] = L.AdapterTable(A, B, [16] * n, [2.0] * n, hi, ho, L.LORA_BF16)
    gains, gains2, gate = bf(1 + n, d, k=0.2, m=1.0), bf(1 + n, d, k=0.2, m=1.0), bf(1 + n, d, k=0.3, m=0.6)
    nb = L.make_norm(L.LORA_NORM_RMS, 1e-6, gain=gains, ld=d)
    na = L.make_norm(L.LORA_NORM_RMS, 1e-6, gain=gains2, ld=d)
    ptr, ads = [0, 100, 100, 260], [2, 0, 1]
    ids = torch.full((T,), -1, dtype=torch.int32)
    for s, a in enumerate(ads):
        ids[ptr[s]:ptr[s + 1]] = a
    ids_d = ids.cuda()
    dev = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in (ptr, ads, [3])]
    seg = L.make_segments(None, dev[0], dev[1], dev[2], T, 3)
    ws = torch.empty(max(t.workspace_bytes(T) for t in tabs.values()), dtype=torch.uint8, device="cuda")
    buf = {k: torch.empty(T, c, dtype=torch.bfloat16, device="cuda") for k, c in
           (("h", d), ("up", f), ("act", f), ("down", d), ("r", d), ("h2", d))}

    def layer(form, name, src, epi, dst):
        t = tabs[name]
        args = (src, t.h, W[name], t.h, epi, dst, t.o, 0, ws, ws.numel())
        if form == "ids":
            L.lora_bgmv_layer(t.handle, ids_d, T, *args)
        else:
            L.lora_sgmv_layer(t.handle, seg, *args)

    def block(form):
        L.lora_norm_before(tabs["up"].handle, ids_d, T, d, x, d, nb, buf["h"], d)
        layer(form, "up", buf["h"], None, buf["up"])
        layer(form, "gate", buf["h"], L.make_epilogue(act=L.LORA_ACT_SILU, mul=buf["up"], ldmul=f), buf["act"])
        layer(form, "down", buf["act"], None, buf["down"])
        L.lora_norm_after(tabs["down"].handle, ids_d, T, d, buf["down"], d, na,
                          L.make_residual(x, d, gate, d, L.LORA_GATE_ADAPTER, 1.0, 0.5), buf["r"], d, nb, buf["h2"], d)

    # the block in 64 bits, with the stored tensors rounded where the calls store them
    dd = lambda t: t.cpu().double()
    rd = lambda t: t.to(torch.bfloat16).double()
    pick = lambda w: dd(w)[(ids + 1).long()]
    rms = lambda v: v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt()

    def lin(v, name):
        z = v @ dd(W[name]).t()
        for i in range(n):
            rows = torch.nonzero(ids == i).flatten()
            z[rows] += 2.0 * (v[rows] @ dd(AB[name][0][i]).t()) @ dd(AB[name][1][i]).t()
        return z

    h = rd(rms(dd(x)) * pick(gains))
    up, gt = rd(lin(h, "up")), lin(h, "gate")
    down = rd(lin(rd(gt * torch.sigmoid(gt) * up), "down"))
    r = dd(x) + 0.5 * pick(gate) * (rms(down) * pick(gains2))
    h2 = rms(r) * pick(gains)
    for form in ("ids", "segments"):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            block(form)
        torch.cuda.synchronize()
        eager = {k: v.clone() for k, v in buf.items()}
        # Each stored tensor may fall on the other side of a rounding (2^-8 of it); through a product of
        # random signs such steps add up as sqrt(h) * (2^-8 |v|) |w|, i.e. 2^-8 of the output's spread.
        # Four roundings lie before r and five before h2: 2^-8 * 5 of the spread, and six standard
        # deviations of it over the outputs.
        for got, ref, k in ((eager["r"], r, 4), (eager["h2"], h2, 5)):
            assert (dd(got) - ref).abs().max() <= 6 * k * 2.0 ** -8 * ref.std(), form
        for v in buf.values():
            v.fill_(-3.0)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            block(form)
        with torch.cuda.stream(s):
            gr.replay()
        torch.cuda.synchronize()
        for k, v in eager.items():
            assert torch.equal(buf[k], v), (form, k)
        with option("pdl", 0):
            block(form)
        torch.cuda.synchronize()
        for k, v in eager.items():
            assert torch.equal(buf[k], v), (form, k)
    assert kernels_launched(lambda: block("ids")) == {"block_norm_kernel", "layer_shrink_kernel", "layer_stream_kernel"}
    for t in tabs.values():
        assert L.lora_get_status(t.handle) == (0, 0)


# a few rows an SM: blocks of the ring that get one row and two; one row fewer, and each row has a block of its own
@pytest.mark.parametrize("dtype,per_sm,extra,d", [("bf16", 4, 0, 64), ("bf16", 4, 1, 4096), ("bf16", 4, -1, 4096),
                                                  ("bf16", 6, 5, 8200), ("bf16", 4, 0, 2048), ("f32", 5, 3, 520),
                                                  ("f32", 4, 0, 4096)])
def test_norm_after_with_a_few_rows_an_sm(dtype, per_sm, extra, d):
    T = per_sm * torch.cuda.get_device_properties(0).multi_processor_count + extra
    m = Norms(T, d, dtype, seed=8)
    x, res = m.rnd(T, 2.0, 0.3), m.rnd(T, 3.0)
    ids = m.ids()
    w, w2 = m.norm("layer", 1 + m.n), m.norm("rms", 1)
    arg = L.make_residual(residual=res, ldres=res.stride(0), res_scale=0.5, branch_scale=2.0)
    r, h = m.out(), m.out()
    names = kernels_launched(lambda: L.lora_norm_after(m.table.handle, ids.cuda(), T, d, x, x.stride(0), w["arg"], arg, r,
                                                       r.stride(0), w2["arg"], h, h.stride(0)))
    assert names == {"block_norm_kernel" if extra < 0 else "ring_norm_kernel"}
    u, off = norm_ref(x.cpu().double(), torch.zeros(T, d).double(), w, ids)
    u, off = 2.0 * u, 2.0 * off
    part = 0.5 * res.cpu().double()
    off = off + 6 * U * u.abs() + 3 * U * (part.abs() + (part + u).abs())
    ref2, off2 = norm_ref(part + u, off, w2, ids)
    close(r, part + u, off, m.half, "r")
    close(h, ref2, off2, m.half, "h")
