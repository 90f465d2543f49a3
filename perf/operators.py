"""What is measured of the operators around a served block: the layer product with its adapter
term, bias, activation, gate product and residual (``lora_bgmv_layer`` for per-token adapter
ids, ``lora_sgmv_layer`` for contiguous segments), and the norms before and after a block with
their per-adapter gains, gate and residual scale (``lora_norm_before``, ``lora_norm_after``).

``run`` computes the plain form with elementary torch operations in 32 bits; with ``own`` set it
makes the calls that a user makes of the framework.  ``exact`` gives the definition in 64 bits.
"""
import math
import random

import torch

own = False

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # The attention output projection for a single token (one chat, latency counts).
        {"name": "layer one token", "op": "bgmv_layer", "T": 1, "h": 4096, "o": 4096, "n": 32, "ranks": "16",
         "zipf": 0.0, "bare": 0.0, "bias": False, "act": "none", "mul": False, "residual": True},
        # The gated half of an MLP in a decode batch, one request per token.
        {"name": "layer decode gate", "op": "bgmv_layer", "T": 64, "h": 4096, "o": 14336, "n": 32, "ranks": "16",
         "zipf": 0.0, "bare": 0.0, "bias": False, "act": "silu", "mul": True, "residual": False},
        # The way back down in a large decode batch with adapters of many ranks, a few of them popular.
        {"name": "layer decode down", "op": "bgmv_layer", "T": 256, "h": 14336, "o": 4096, "n": 128,
         "ranks": "8,16,32,64", "zipf": 1.0, "bare": 0.0, "bias": False, "act": "none", "mul": False,
         "residual": True},
        # Odd sizes throughout: ranks of no round size, a third of the tokens without an adapter.
        {"name": "layer decode odd", "op": "bgmv_layer", "T": 37, "h": 1096, "o": 1000, "n": 11, "ranks": "3,8,20,128",
         "zipf": 0.0, "bare": 0.33, "bias": True, "act": "gelu", "mul": False, "residual": True},
        # Prompts of eight tenants through the gated half of an MLP: the largest case.
        {"name": "layer prompts gate", "op": "sgmv_layer", "T": 4096, "h": 4096, "o": 14336, "n": 8, "ranks": "64",
         "segs": 8, "ragged": False, "bias": False, "act": "silu", "mul": True, "residual": False},
        # Prompts of any length through the small key/value projection, some without an adapter.
        {"name": "layer prompts ragged", "op": "sgmv_layer", "T": 1531, "h": 4096, "o": 1024, "n": 7,
         "ranks": "8,16,32,64", "segs": 9, "ragged": True, "bias": True, "act": "none", "mul": False,
         "residual": False},
        # Prompts on the way back down, into the residual stream.
        {"name": "layer prompts down", "op": "sgmv_layer", "T": 2048, "h": 14336, "o": 4096, "n": 4, "ranks": "16,64",
         "segs": 4, "ragged": True, "bias": False, "act": "none", "mul": False, "residual": True},
        # The norm before a block for a single token.
        {"name": "norm before one token", "op": "norm_before", "dtype": "bf16", "T": 1, "d": 4096, "n": 32,
         "kind": "rms", "per_adapter": True, "shift": False},
        # The norm before a block over a batch of prompts, gains chosen by each token's adapter.
        {"name": "norm before prompts", "op": "norm_before", "dtype": "bf16", "T": 4096, "d": 4096, "n": 8,
         "kind": "rms", "per_adapter": True, "shift": False},
        # A decode batch: norm after the block, adapter gate, residual, and the next block's norm.
        {"name": "norm after decode", "op": "norm_after", "dtype": "bf16", "T": 64, "d": 4096, "n": 32, "kind": "rms",
         "next": "rms", "per_adapter": True, "shift": False, "gate": "adapter"},
        # Prompts, with a gate per token and a scaled residual.
        {"name": "norm after prompts", "op": "norm_after", "dtype": "bf16", "T": 4096, "d": 4096, "n": 8,
         "kind": "rms", "next": "rms", "per_adapter": False, "shift": False, "gate": "token"},
        # Odd sizes in 32 bits: layer norm with shifts around the residual sum.
        {"name": "norm after odd", "op": "norm_after", "dtype": "f32", "T": 517, "d": 1000, "n": 5, "kind": "none",
         "next": "layer", "per_adapter": True, "shift": True, "gate": "none"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _eighths(rng, lo, hi):
    return max(lo, min(hi, _log(rng, lo, hi) // 8 * 8))


def draw(rng):
    op = rng.choice(("bgmv_layer", "sgmv_layer", "norm_before", "norm_after"))
    if op in ("bgmv_layer", "sgmv_layer"):
        h = _eighths(rng, 256, 14336)
        o = _eighths(rng, 256, min(14336, 4096 * 14336 // h))
        case = {"op": op, "T": 0, "h": h, "o": o}
        if op == "bgmv_layer":
            case["T"] = _log(rng, 1, 512)
            case["n"] = _log(rng, 1, 96)
            case["ranks"] = rng.choice(("16", "64", "8,16,32,64", "5,128", "1,9,24"))
            case["zipf"] = rng.choice((0.0, 0.8, 1.0))
            case["bare"] = rng.choice((0.0, 0.0, 0.25))
        else:
            # no more products and no more bytes than the largest listed case
            most = min(4096 * 4096 * 14336 // (h * o), (1 << 27) // (h + 3 * o))
            case["T"] = max(1, min(_log(rng, 129, 6000), most))
            case["n"] = rng.randint(1, 12)
            case["ranks"] = rng.choice(("16", "64", "8,16,32,64", "24,40"))
            case["segs"] = rng.randint(1, min(16, case["T"]))
            case["ragged"] = rng.random() < 0.75
        case["bias"] = rng.random() < 0.5
        case["act"] = rng.choice(ACTS)
        case["mul"] = rng.random() < 0.4
        case["residual"] = rng.random() < 0.5
        return case
    dtype = rng.choice(("bf16", "bf16", "f32"))
    case = {"op": op, "dtype": dtype, "T": _log(rng, 1, 8192), "d": _eighths(rng, 64, 16384), "n": rng.randint(1, 40)}
    case["T"] = max(1, min(case["T"], (1 << (25 if dtype == "bf16" else 24)) // case["d"]))
    case["kind"] = rng.choice(("rms", "rms", "layer") if op == "norm_before" else ("rms", "layer", "none"))
    if op == "norm_after":
        case["next"] = rng.choice(("rms", "layer", "none"))
        case["gate"] = rng.choice(("none", "adapter", "token"))
    case["per_adapter"] = rng.random() < 0.6
    case["shift"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------------------------- inputs


def _ranks(case):
    r = [int(v) for v in case["ranks"].split(",")]
    return [r[i % len(r)] for i in range(case["n"])]


def _segments(case):
    """Row bounds of the segments and the adapter of each; ragged ones leave rows before and
    after them without an adapter."""
    T, S, n = case["T"], case["segs"], case["n"]
    if not case["ragged"]:
        cuts = [T * s // S for s in range(S + 1)]
    else:
        rng = random.Random(1000 * T + S)
        cuts = sorted(rng.randint(0, T) for _ in range(S + 1))
    return cuts, [s % n for s in range(S)]


def _ids(case, gen):
    """Adapter of each token: uniform, or Zipf with a share of tokens without one (-1)."""
    n, T = case["n"], case["T"]
    p = torch.arange(1, n + 1, dtype=torch.float64) ** -case.get("zipf", 0.0)
    ids = torch.multinomial(p, T, replacement=True, generator=gen).int()
    bare = case.get("bare", 0.0)
    if bare:
        ids[torch.rand(T, generator=gen) < bare] = -1
    return ids


def prepare(case, seed):
    cpu = torch.Generator().manual_seed(seed)
    gen = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, mean=0.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale + mean).to(dtype)

    return (_prepare_layer if case["op"].endswith("layer") else _prepare_norm)(case, cpu, normal)


def _prepare_layer(case, cpu, normal):
    T, h, o = case["T"], case["h"], case["o"]
    ranks = _ranks(case)
    st = {"case": case, "ranks": ranks, "scales": [16.0 / r for r in ranks], "x": normal(T, h),
          "W": normal(o, h, scale=h ** -0.5),
          # A_i [r_i, h] and B_i [o, r_i] of all adapters, one behind the other
          "A": normal(sum(ranks), h, scale=h ** -0.5), "B": normal(o * sum(ranks), scale=0.02 ** 0.5),
          "bias": normal(o) if case["bias"] else None, "mul": normal(T, o) if case["mul"] else None,
          "residual": normal(T, o) if case["residual"] else None}
    if case["op"] == "sgmv_layer":
        cuts, adapters = _segments(case)
        ids = torch.full((T,), -1, dtype=torch.int32)
        for s, a in enumerate(adapters):
            ids[cuts[s]:cuts[s + 1]] = a
        st["bounds"] = torch.tensor(cuts, dtype=torch.int32, device="cuda")
        st["adapters"] = torch.tensor(adapters, dtype=torch.int32, device="cuda")
        st["count"] = torch.tensor([len(adapters)], dtype=torch.int32, device="cuda")
    else:
        ids = _ids(case, cpu)
    st["ids"] = ids.cuda()
    if own:
        import heterogeneous_adapters_sgmv_b200 as L
        a0, b0, first = st["A"].data_ptr(), st["B"].data_ptr(), [sum(ranks[:i]) for i in range(len(ranks))]
        st["table"] = L.AdapterTable([a0 + 2 * h * f for f in first], [b0 + 2 * o * f for f in first], ranks,
                                     st["scales"], h, o, L.LORA_BF16, keep=(st["A"], st["B"]))
        st["ws"] = torch.empty(st["table"].workspace_bytes(T), dtype=torch.uint8, device="cuda")
        st["y"] = torch.empty(T, o, dtype=torch.bfloat16, device="cuda")
        act = {"none": L.LORA_ACT_NONE, "relu": L.LORA_ACT_RELU, "gelu": L.LORA_ACT_GELU,
               "gelu_tanh": L.LORA_ACT_GELU_TANH, "silu": L.LORA_ACT_SILU}[case["act"]]
        st["epilogue"] = L.make_epilogue(bias=st["bias"], act=act, mul=st["mul"], ldmul=o, residual=st["residual"],
                                         ldres=o)
        if case["op"] == "sgmv_layer":
            longest = max(b - a for a, b in zip(cuts, cuts[1:]))
            st["segments"] = L.make_segments(None, st["bounds"], st["adapters"], st["count"], T, len(adapters), longest)
    else:
        st["owner"] = torch.repeat_interleave(torch.arange(len(ranks)), torch.tensor(ranks)).cuda()
        st["row_scale"] = torch.repeat_interleave(torch.tensor(st["scales"]), torch.tensor(ranks)).cuda()
    return st


def _prepare_norm(case, cpu, normal):
    T, d, n, E = case["T"], case["d"], case["n"], TYPES[case["dtype"]]
    rows = 1 + n if case["per_adapter"] else 1

    def weights(kind):
        if kind == "none":
            return None
        return {"kind": kind, "eps": 1e-5, "gain": normal(rows, d, scale=0.2, mean=1.0, dtype=E),
                "shift": normal(rows, d, scale=0.2, dtype=E) if case["shift"] else None}

    # a residual stream is wide, with a mean, and its rows differ in size
    size = normal(T, 1, dtype=torch.float32).exp()
    st = {"case": case, "x": (normal(T, d, mean=0.3, dtype=torch.float32) * size).to(E),
          "ids": (_ids(dict(case, bare=0.2), cpu)).cuda(), "norm": weights(case["kind"])}
    if case["op"] == "norm_after":
        st["residual"] = normal(T, d, scale=2.0, dtype=E)
        st["next"] = weights(case["next"])
        gate_rows = {"none": 0, "adapter": 1 + n, "token": T}[case["gate"]]
        st["gate"] = normal(gate_rows, d, scale=0.5, mean=0.5, dtype=E) if gate_rows else None
        st["res_scale"], st["branch_scale"] = 0.875, 1.25
    if own:
        import heterogeneous_adapters_sgmv_b200 as L
        t = L.LORA_BF16 if case["dtype"] == "bf16" else L.LORA_F32
        # the adapters of the projection that the norm stands beside
        wts = [normal(8 * d, scale=d ** -0.5, dtype=E), normal(8 * d, scale=0.02 ** 0.5, dtype=E)]
        st["table"] = L.AdapterTable([wts[0]] * n, [wts[1]] * n, [8] * n, [2.0] * n, d, d, t, keep=wts)

        def struct(w):
            if w is None:
                return None
            kind = {"rms": L.LORA_NORM_RMS, "layer": L.LORA_NORM_LAYER}[w["kind"]]
            return L.make_norm(kind, w["eps"], gain=w["gain"], shift=w["shift"], ld=d if case["per_adapter"] else 0)

        st["norm_arg"] = struct(st["norm"])
        st["h"] = torch.empty(T, d, dtype=E, device="cuda")
        if case["op"] == "norm_after":
            st["next_arg"] = struct(st["next"])
            st["r"] = torch.empty(T, d, dtype=E, device="cuda")
            kind = {"none": L.LORA_GATE_NONE, "adapter": L.LORA_GATE_ADAPTER, "token": L.LORA_GATE_TOKEN}[case["gate"]]
            st["residual_arg"] = L.make_residual(residual=st["residual"], ldres=d, gate=st["gate"], ldgate=d,
                                                 gate_kind=kind, res_scale=st["res_scale"],
                                                 branch_scale=st["branch_scale"])
    return st


# ------------------------------------------------------------------------------- the calls


def run(st):
    case = st["case"]
    if own:
        return _own(st)
    return {"bgmv_layer": _plain_layer, "sgmv_layer": _plain_layer, "norm_before": _plain_before,
            "norm_after": _plain_after}[case["op"]](st)


def _own(st):
    import heterogeneous_adapters_sgmv_b200 as L
    case = st["case"]
    table = st["table"].handle
    if case["op"] in ("bgmv_layer", "sgmv_layer"):
        T, h, o = case["T"], case["h"], case["o"]
        if case["op"] == "bgmv_layer":
            L.lora_bgmv_layer(table, st["ids"], T, st["x"], h, st["W"], h, st["epilogue"], st["y"], o, 0, st["ws"],
                              st["ws"].numel())
        else:
            L.lora_sgmv_layer(table, st["segments"], st["x"], h, st["W"], h, st["epilogue"], st["y"], o, 0, st["ws"],
                              st["ws"].numel())
        return st["y"]
    T, d = case["T"], case["d"]
    if case["op"] == "norm_before":
        L.lora_norm_before(table, st["ids"], T, d, st["x"], d, st["norm_arg"], st["h"], d)
        return st["h"]
    if st["next_arg"] is None:
        L.lora_norm_after(table, st["ids"], T, d, st["x"], d, st["norm_arg"], st["residual_arg"], st["r"], d, None,
                          None, 0)
        return st["r"]
    L.lora_norm_after(table, st["ids"], T, d, st["x"], d, st["norm_arg"], st["residual_arg"], st["r"], d,
                      st["next_arg"], st["h"], d)
    return st["r"], st["h"]


def _plain_layer(st):
    """The adapters' A_i stacked into one tall matrix: every token meets every adapter, and all but
    its own are masked out before the stacked B_i."""
    case, o, ranks = st["case"], st["case"]["o"], st["ranks"]
    x = st["x"].float()
    v = x @ st["A"].float().t()
    v = torch.where(st["ids"][:, None] == st["owner"][None, :], v * st["row_scale"], 0.0)
    B = torch.cat([b.view(o, r) for b, r in zip(st["B"].split([o * r for r in ranks]), ranks)], 1).float()
    z = x @ st["W"].float().t() + v @ B.t()
    if st["bias"] is not None:
        z = z + st["bias"].float()
    if case["act"] == "relu":
        z = torch.where(z < 0, 0.0, z)
    elif case["act"] == "gelu":
        z = 0.5 * z * torch.special.erfc(z * -math.sqrt(0.5))
    elif case["act"] == "gelu_tanh":
        z = z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    elif case["act"] == "silu":
        z = z / (1 + torch.exp(-z))
    if st["mul"] is not None:
        z = z * st["mul"].float()
    if st["residual"] is not None:
        z = z + st["residual"].float()
    return z.to(st["x"].dtype)


def _plain_rows(w, st):
    """Each token's row of a weight: row 0 without an adapter, row 1 + i with adapter i."""
    return w[(st["ids"] + 1).long()].float() if w.shape[0] > 1 else w.float()


def _plain_norm(x, w, st):
    if w is None:
        return x
    if w["kind"] == "layer":
        x = x - x.mean(1, keepdim=True)
    x = x * torch.rsqrt((x * x).mean(1, keepdim=True) + w["eps"]) * _plain_rows(w["gain"], st)
    return x if w["shift"] is None else x + _plain_rows(w["shift"], st)


def _plain_before(st):
    return _plain_norm(st["x"].float(), st["norm"], st).to(st["x"].dtype)


def _plain_after(st):
    E = st["x"].dtype
    u = _plain_norm(st["x"].float(), st["norm"], st) * st["branch_scale"]
    if st["case"]["gate"] == "adapter":
        u = u * _plain_rows(st["gate"], st)
    elif st["case"]["gate"] == "token":
        u = u * st["gate"].float()
    r = st["residual"].float() * st["res_scale"] + u
    if st["next"] is None:
        return r.to(E)
    return r.to(E), _plain_norm(r, st["next"], st).to(E)


# ------------------------------------------------------------------------------- in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].endswith("layer"):
        return _exact_layer(st)
    x, ids = st["x"].double(), st["ids"].tolist()
    u = _exact_norm(x, st["norm"], ids)
    if case["op"] == "norm_before":
        return u
    gate = st["gate"]
    if gate is not None:
        u = u * (gate.double() if case["gate"] == "token" else _exact_rows(gate, ids))
    r = st["res_scale"] * st["residual"].double() + st["branch_scale"] * u
    return r if st["next"] is None else (r, _exact_norm(r, st["next"], ids))


def _exact_layer(st):
    case, h, o = st["case"], st["case"]["h"], st["case"]["o"]
    x, ids = st["x"].double(), st["ids"].long()
    z = torch.mm(x, st["W"].double().t())
    first = 0
    for i, r in enumerate(st["ranks"]):
        rows = torch.nonzero(ids == i).flatten()
        if rows.numel():
            A = st["A"][first:first + r].double()
            B = st["B"][o * first:o * (first + r)].view(o, r).double()
            z[rows] += st["scales"][i] * torch.mm(torch.mm(x[rows], A.t()), B.t())
        first += r
    if st["bias"] is not None:
        z += st["bias"].double()
    act = case["act"]
    if act == "relu":
        z = z.clamp(min=0)
    elif act == "gelu":
        z = z * torch.special.ndtr(z)
    elif act == "gelu_tanh":
        z = z / 2 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    elif act == "silu":
        z = z * torch.sigmoid(z)
    if st["mul"] is not None:
        z = z * st["mul"].double()
    if st["residual"] is not None:
        z = z + st["residual"].double()
    return z


def _exact_rows(w, ids):
    if w.shape[0] == 1:
        return w.double().expand(len(ids), -1)
    return torch.index_select(w.double(), 0, torch.tensor([1 + i for i in ids], device=w.device))


def _exact_norm(x, w, ids):
    if w is None:
        return x
    mean = x.sum(1, keepdim=True) / x.shape[1] if w["kind"] == "layer" else 0.0
    c = x - mean
    y = c / torch.sqrt(torch.sum(c ** 2, 1, keepdim=True) / x.shape[1] + w["eps"]) * _exact_rows(w["gain"], ids)
    return y if w["shift"] is None else y + _exact_rows(w["shift"], ids)


# ------------------------------------------------------------------------------- the floor


def _touched(case):
    """Expected rank sums: (of the distinct adapters that a batch meets, of its tokens)."""
    ranks = _ranks(case)
    if case["op"] == "sgmv_layer":
        cuts, adapters = _segments(case)
        lens = [b - a for a, b in zip(cuts, cuts[1:])]
        met = {a for a, l in zip(adapters, lens) if l > 0}
        return sum(ranks[a] for a in met), sum(ranks[a] * l for a, l in zip(adapters, lens))
    T, n = case["T"], case["n"]
    p = [(i + 1.0) ** -case["zipf"] for i in range(n)]
    p = [(1 - case["bare"]) * v / sum(p) for v in p]
    return (sum(r * (1 - (1 - q) ** T) for r, q in zip(ranks, p)), T * sum(r * q for r, q in zip(ranks, p)))


def work(case):
    T = case["T"]
    if case["op"].endswith("layer"):
        h, o = case["h"], case["o"]
        distinct, tokens = _touched(case)
        values = h * o + T * h + T * o * (1 + case["mul"] + case["residual"]) + o * case["bias"] + distinct * (h + o)
        return {"bytes": 2 * values, "flops": 2 * T * h * o + 2 * tokens * (h + o)}
    d, size = case["d"], 2 if case["dtype"] == "bf16" else 4
    rows = 1 + min(case["n"], T) if case["per_adapter"] else 1
    if case["op"] == "norm_before":
        norms, planes, gate = 1, 2, 0
    else:
        norms = (case["kind"] != "none") + (case["next"] != "none")
        planes = 3 + (case["next"] != "none") + (case["gate"] == "token")
        gate = 1 + min(case["n"], T) if case["gate"] == "adapter" else 0
    values = planes * T * d + (norms * rows * (1 + case["shift"]) + gate) * d
    return {"bytes": size * values, "flops": T * d * (4 * norms + planes)}
