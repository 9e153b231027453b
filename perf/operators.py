"""Cases of the operators around the token exchange: the norm that makes its rows, and
the experts' matrix products on the rows that it delivers.

Each case is one call as a mixture-of-experts layer makes it.  `run` computes it in plain
torch operations in float32 (own = False) or through the library's entry points (own =
True).  Sizes are those of the repository's workloads (decode, prefill, top-8, edge,
tiny); the experts' inner width, which no workload has, is 1024 or 2048.

8-bit rows ("mx8"): n e4m3 elements, then n/32 scale bytes (E8M0, a power of two for each
32 elements), padded to a multiple of 16 bytes.  4-bit weights ("mx4"): two E2M1 elements
a byte, the even one in the low half, with the same scales in an array of their own.
"""
import math

import torch

own = False

F32, BF16, MX8, MX4 = 0, 1, 2, 3
KIND = {"f32": F32, "bf16": BF16, "mx8": MX8, "mx4": MX4}
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ---- cases ---------------------------------------------------------------------------

def _norm(name, rows, hidden, dtype, residual, y, y8):
    c = {"op": "norm", "rows": rows, "hidden": hidden, "dtype": dtype, "residual": residual, "y": y, "y8": y8}
    return {"name": name, **c} if name else c


def _experts(name, ranks, epr, rows, cap, k, n, kinds, swiglu, routing):
    """rows: all ranks' rows together; cap: rows of a rank's slice; n: the weights' rows for each
    expert (with swiglu gate and up, so n / 2 columns come out)."""
    i, w, o = kinds.split(":")
    c = {"op": "matmul4" if w == "mx4" else "matmul", "ranks": ranks, "epr": epr, "rows": rows, "cap": cap, "k": k,
         "n": n, "in": i, "w": w, "out": o, "swiglu": swiglu, "routing": routing}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one token of a decode step on its way into the layer: both kinds of output
        _norm("norm_one_token", 1, 5120, "bf16", True, True, True),
        # an odd width and row count in float32, as in a small test model
        _norm("norm_f32_odd", 1027, 2047, "f32", True, True, False),
        # prefill, 8 ranks x 8192 tokens: residual kept, 8-bit rows for the dispatch
        _norm("norm_prefill_mx8", 65536, 5120, "bf16", True, False, True),
        # the tiny workload's experts, float32, an odd inner width
        _experts("experts_tiny_f32", 4, 2, 512, 512, 128, 2 * 77, "f32:f32:f32", True, "uniform"),
        # decode, 8 ranks x 128 tokens, top-1 over 128 experts, Zipf routing: gate and up
        _experts("experts_decode_bf16", 8, 16, 1024, 1024, 5120, 4096, "bf16:bf16:bf16", True, "zipf1.1"),
        # edge, 64 ranks x 16 tokens, top-2: the down product; 40 % of the rows on one rank
        _experts("experts_edge_down_bf16", 64, 1, 2048, 1024, 1024, 2048, "bf16:bf16:bf16", False, "edge"),
        # prefill, 8 ranks x 8192 tokens, top-1 over 128 experts: gate and up
        _experts("experts_prefill_bf16", 8, 16, 65536, 65536, 5120, 4096, "bf16:bf16:bf16", True, "zipf1.2"),
        # the same in 8 bits, 8-bit rows out for the down product
        _experts("experts_prefill_mx8", 8, 16, 65536, 65536, 5120, 4096, "mx8:mx8:mx8", True, "zipf1.2"),
        # one token's one expert in a decode step of a single user, 4-bit weights
        _experts("experts4_one_token", 8, 16, 1, 1, 5120, 4096, "bf16:mx4:bf16", True, "uniform"),
        # decode, 8 ranks x 128 tokens: gate and up, 4-bit weights
        _experts("experts4_decode_bf16", 8, 16, 1024, 1024, 5120, 4096, "bf16:mx4:bf16", True, "zipf1.1"),
        # top-8 decode, 16 ranks x 16 tokens over 256 experts: 8 rows an expert, 8-bit rows
        _experts("experts4_top8_decode_mx8", 16, 16, 2048, 2048, 7168, 4096, "mx8:mx4:mx8", True, "uniform"),
        # top-8 prefill, 16 ranks x 2048 tokens: the down product, 1024 rows an expert
        _experts("experts4_top8_prefill_mx8", 16, 16, 262144, 32768, 2048, 7168, "mx8:mx4:bf16", False, "uniform"),
    ]


def _log(rng, a, b):
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    if rng.random() < 0.3:
        dtype = rng.choice(["bf16", "bf16", "f32"])
        rows, y8 = _log(rng, 1, 65536), dtype == "bf16" and rng.random() < 0.6
        hidden = 32 * _log(rng, 1, 224) if y8 or rng.random() < 0.5 else _log(rng, 1, 7168)
        return _norm(None, rows, hidden, dtype, rng.random() < 0.7, not y8 or rng.random() < 0.5, y8)
    kinds = rng.choice(["f32:f32:f32", "bf16:bf16:bf16", "bf16:bf16:bf16", "mx8:mx8:bf16", "mx8:mx8:mx8", "bf16:mx4:bf16",
                        "bf16:mx4:bf16", "mx8:mx4:bf16", "mx8:mx4:mx8"])
    swiglu = rng.random() < 0.5
    ranks, epr = rng.choice([(8, 16), (16, 16), (64, 1), (4, 2), (1, 8), (3, 5), (1, 1)])
    block = 32 if "mx" in kinds else rng.choice([1, 2, 8, 32])
    k = block * max(1, _log(rng, 64, 7168) // block)
    out = 32 if kinds.endswith("mx8") else rng.choice([1, 2, 16, 32])
    n = out * max(1, _log(rng, 64, 4096) // (out * (2 if swiglu else 1))) * (2 if swiglu else 1)
    rows = _log(rng, 1, 16384)
    # a slice holds every row (the largest that a routing can need), or just over the mean: then rows are dropped
    cap = rows if rng.random() < 0.8 else max(1, rows // ranks + rows // (8 * ranks))
    return _experts(None, ranks, epr, rows, cap, k, n, kinds, swiglu, rng.choice(["uniform", "zipf1.1", "edge"]))


# ---- inputs --------------------------------------------------------------------------

def _row_bytes(n):
    return (n + n // 32 + 15) // 16 * 16


def _gen(seed, which):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 16 + which)
    return g


def _pow2(e):
    """2^e in float32 for whole e in [-126, 127], exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _to_mx8(v):
    """float32 [rows][n] -> (e4m3 elements as bytes, scale bytes): the scale is the smallest power
    of two that keeps the largest of its 32 elements within 448."""
    b = v.reshape(v.shape[0], -1, 32)
    a = b.abs().amax(dim=2)
    m, e = torch.frexp(a)                         # a = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = (e - 9 + (m > 0.875)).clamp(min=-127)
    e = torch.where(a > 0, e, torch.full_like(e, -127))
    bad = ~torch.isfinite(a)
    # times 2^-e in two halves: 2^127 and 2^-118 are both reached
    h = torch.div(-e, 2, rounding_mode="floor")
    q = (b * _pow2(h)[:, :, None] * _pow2(-e - h)[:, :, None]).to(torch.float8_e4m3fn)
    q = q.view(torch.uint8).masked_fill(bad[:, :, None], 127)
    s = (e + 127).to(torch.uint8).masked_fill(bad, 255)
    return q.reshape(v.shape), s


def _offsets(case, seed):
    """Group starts [ranks][epr + 1] of rows routed to experts (int32, host): what the receive side knows."""
    g = torch.Generator()
    g.manual_seed(seed * 16 + 7)
    e = case["ranks"] * case["epr"]
    if case["routing"].startswith("zipf"):
        p = 1.0 / torch.arange(1, e + 1, dtype=torch.float64) ** float(case["routing"][4:])
        p = p[torch.randperm(e, generator=g)]
    elif case["routing"] == "edge":               # a quarter receive nothing, one receives 40 %
        p = torch.ones(e, dtype=torch.float64)
        at = torch.randperm(e, generator=g)
        p[at[: e // 4]] = 0
        rest = float(p.sum()) - 1
        if rest > 0:
            p[at[-1]] = rest * 2 / 3
    else:
        p = torch.ones(e, dtype=torch.float64)
    to = torch.multinomial(p, case["rows"], replacement=True, generator=g)
    counts = torch.bincount(to, minlength=e).reshape(case["ranks"], case["epr"])
    off = torch.zeros((case["ranks"], case["epr"] + 1), dtype=torch.int64)
    off[:, 1:] = counts.cumsum(1)
    return off.to(torch.int32)


def _random_rows(shape, kind, g, scale=1.0):
    """A tensor of N(0, scale^2) of the row type, made in slices of the first dimension."""
    n = shape[-1]
    out = torch.empty(shape[:-1] + ((_row_bytes(n),) if kind == "mx8" else (n,)), device="cuda",
                      dtype=torch.uint8 if kind == "mx8" else TORCH[kind])
    for part in out.reshape(-1, out.shape[-1]).split(1 << 16):
        v = torch.randn((part.shape[0], n), device="cuda", generator=g)
        if kind == "mx8":
            q, s = _to_mx8(v * scale)
            part[:, :n] = q
            part[:, n:n + n // 32] = s
            part[:, n + n // 32:] = 0
        else:
            part.copy_(v * scale)
    return out


def prepare(case, seed):
    if case["op"] == "norm":
        rows, h, t = case["rows"], case["hidden"], TORCH[case["dtype"]]
        s = {"case": case,
             "x": torch.randn((rows, h), device="cuda", generator=_gen(seed, 0)).to(t),
             "residual": torch.randn((rows, h), device="cuda", generator=_gen(seed, 1)).mul_(4).to(t) if case["residual"] else None,
             "weight": (1 + 0.1 * torch.randn(h, device="cuda", generator=_gen(seed, 2))).to(t),
             "residual_out": torch.zeros((rows, h), device="cuda", dtype=t) if case["residual"] else None,
             "y": torch.zeros((rows, h), device="cuda", dtype=t) if case["y"] else None,
             "y8": torch.zeros((rows, _row_bytes(h)), device="cuda", dtype=torch.uint8) if case["y8"] else None}
        return s
    r, epr, cap, k, n = case["ranks"], case["epr"], case["cap"], case["k"], case["n"]
    e, width = r * epr, case["n"] // 2 if case["swiglu"] else case["n"]
    off = _offsets(case, seed)
    rows = torch.zeros((r, cap, _row_bytes(k) if case["in"] == "mx8" else k), device="cuda",
                       dtype=torch.uint8 if case["in"] == "mx8" else TORCH[case["in"]])
    g = _gen(seed, 0)
    for d in range(r):                            # rows behind a slice's last one stay zero
        m = int(off[d, -1].clamp(max=cap))
        if m:
            rows[d, :m] = _random_rows((m, k), case["in"], g)
    g = _gen(seed, 1)
    sd, scales = k ** -0.5, None
    if case["w"] == "mx4":
        w = torch.randint(0, 256, (e, n, k // 2), device="cuda", generator=g, dtype=torch.uint8)
        scales = torch.randint(118, 121, (e, n, k // 32), device="cuda", generator=g, dtype=torch.uint8)
    elif case["w"] == "mx8":
        p = _random_rows((e, n, k), "mx8", g, sd)
        w, scales = p[..., :k].contiguous(), p[..., k:k + k // 32].contiguous()
    else:
        w = _random_rows((e, n, k), case["w"], g, sd)
    o = case["out"]
    return {"case": case, "rows": rows, "offsets": off.cuda(), "weight": w, "scales": scales,
            "out": torch.zeros((r, cap, _row_bytes(width) if o == "mx8" else width), device="cuda",
                               dtype=torch.uint8 if o == "mx8" else TORCH[o]),
            "status": torch.zeros(1, dtype=torch.int32, device="cuda")}


# ---- the plain forms and the library's calls -----------------------------------------

def _parts(rows, n):
    """8-bit rows as the values that they hold: elements and scales (views)."""
    return [rows[..., :n].view(torch.float8_e4m3fn), rows[..., n:n + n // 32].view(torch.float8_e8m0fnu)]


def _plain_rows(v, kind, out):
    """Rounds float32 rows into rows of `out` of the given type."""
    if kind == "mx8":
        n = v.shape[-1]
        out[:, :n], out[:, n:n + n // 32] = _to_mx8(v)
    else:
        out.copy_(v)


def _plain_values(rows, kind, k):
    """Rows of any type in float32."""
    if kind != "mx8":
        return rows.float()
    s = _pow2(rows[:, k:k + k // 32].to(torch.int32) - 127)
    return (rows[:, :k].view(torch.float8_e4m3fn).float().reshape(rows.shape[0], -1, 32) * s[:, :, None]).reshape(-1, k)


def _plain_weight(w, scales, kind, k):
    """One expert's weights [n][k] in float32."""
    if kind in TORCH:
        return w.float()
    s = _pow2(scales.to(torch.int32) - 127)[:, :, None]
    if kind == "mx8":
        v = w.view(torch.float8_e4m3fn).float()
    else:
        v = torch.tensor(E2M1, device=w.device)[torch.stack((w & 15, w >> 4), dim=-1).to(torch.int32)]
    return (v.reshape(w.shape[0], -1, 32) * s).reshape(w.shape[0], k)


def _run_norm(s):
    c = s["case"]
    if own:
        from moe_alltoallv_resident_amd import a2av
        a2av.rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"], residual_out=s["residual_out"], y=s["y"], y8=s["y8"])
    else:
        v = s["x"].float()
        if c["residual"]:
            v = v + s["residual"].float()
            s["residual_out"].copy_(v)
        v = v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
        if c["y"]:
            s["y"].copy_(v)
        if c["y8"]:
            _plain_rows(v, "mx8", s["y8"])
    return [s["residual_out"], s["y"], _parts(s["y8"], c["hidden"]) if c["y8"] else None]


def _run_experts(s):
    c = s["case"]
    width = c["n"] // 2 if c["swiglu"] else c["n"]
    if own:
        from moe_alltoallv_resident_amd import a2av
        a2av.expert_matmul(s["rows"], s["offsets"], s["weight"], s["out"], s["status"], weight_scales=s["scales"],
                           in_dtype=KIND[c["in"]], weight_dtype=KIND[c["w"]], out_dtype=KIND[c["out"]],
                           activation=a2av.ACT_SWIGLU if c["swiglu"] else a2av.ACT_NONE)
    else:
        # eager torch has no product over ragged groups: their sizes go to the host, and each group that
        # has rows is one product
        starts = s["offsets"].clamp(max=c["cap"]).tolist()
        for e in range(c["ranks"] * c["epr"]):
            d, le = divmod(e, c["epr"])
            a, b = starts[d][le], starts[d][le + 1]
            if a == b:
                continue
            w = _plain_weight(s["weight"][e], None if s["scales"] is None else s["scales"][e], c["w"], c["k"])
            v = _plain_values(s["rows"][d, a:b], c["in"], c["k"]) @ w.t()
            if c["swiglu"]:
                gate, up = v[:, :width], v[:, width:]
                v = gate / (1 + torch.exp(-gate)) * up
            _plain_rows(v, c["out"], s["out"][d, a:b])
    return _parts(s["out"], width) if c["out"] == "mx8" else s["out"]


def run(state):
    return _run_norm(state) if state["case"]["op"] == "norm" else _run_experts(state)


def work(case):
    size = {"f32": 4, "bf16": 2, "mx8": 1 + 1 / 32, "mx4": 0.5 + 1 / 32}
    if case["op"] == "norm":
        e, n = size[case["dtype"]], case["rows"] * case["hidden"]
        b = n * (e * (1 + 2 * case["residual"] + case["y"]) + size["mx8"] * case["y8"]) + e * case["hidden"]
        return {"bytes": b, "flops": 5 * n}
    off = _offsets(case, 0).clamp(max=case["cap"])   # the groups that have rows vary a little with the seed
    counts = off[:, 1:] - off[:, :-1]
    rows, active = int(counts.sum()), int((counts > 0).sum())
    width = case["n"] // 2 if case["swiglu"] else case["n"]
    b = (rows * (case["k"] * size[case["in"]] + width * size[case["out"]]) + active * case["n"] * case["k"] * size[case["w"]]
         + 4 * off.numel())
    return {"bytes": b, "flops": 2 * rows * case["n"] * case["k"]}


# ---- the definitions in 64 bits ------------------------------------------------------

def _exact_mx8(v):
    """Elements (not rounded) and scales of float64 rows."""
    a = v.unflatten(1, (-1, 32)).abs().amax(dim=2)
    e = torch.ceil(torch.log2(a / 448)).clamp(min=-127)
    e = torch.where(a / torch.exp2(e) > 448, e + 1, e)     # log2 may round past a whole number
    e = torch.where(a / torch.exp2(e - 1) <= 448, e - 1, e).clamp(min=-127)
    return v / torch.exp2(e).repeat_interleave(32, dim=1), torch.exp2(e)


def _exact_unpack(elements, scales):
    return elements * torch.exp2(scales.double() - 127).repeat_interleave(32, dim=-1)


def _exact_norm(case, s):
    v = s["x"].double()
    if case["residual"]:
        v = v + s["residual"].double()
    y = v / torch.sqrt(v.square().sum(dim=1, keepdim=True) / case["hidden"] + EPS) * s["weight"].double()
    return [v if case["residual"] else None, y if case["y"] else None, list(_exact_mx8(y)) if case["y8"] else None]


def _exact_experts(case, s):
    k, n, cap, epr = case["k"], case["n"], case["cap"], case["epr"]
    width = n // 2 if case["swiglu"] else n
    mx = case["out"] == "mx8"
    out = [torch.zeros((case["ranks"], cap, width), dtype=torch.float64, device="cuda")]
    if mx:
        # a row that is not written holds zero bytes: the scale 2^-127
        out.append(torch.full((case["ranks"], cap, width // 32), 2.0 ** -127, dtype=torch.float64, device="cuda"))
    off = s["offsets"].cpu().numpy()
    table = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    for d in range(case["ranks"]):
        for le in range(epr):
            lo, hi = min(int(off[d, le]), cap), min(int(off[d, le + 1]), cap)
            if lo >= hi:
                continue
            e = d * epr + le
            w = s["weight"][e]
            if case["w"] == "mx4":
                v = torch.empty((n, k), dtype=torch.float64, device="cuda")
                v[:, 0::2], v[:, 1::2] = table[(w % 16).long()], table[(w // 16).long()]
                w = _exact_unpack(v, s["scales"][e])
            elif case["w"] == "mx8":
                w = _exact_unpack(w.view(torch.float8_e4m3fn).double(), s["scales"][e])
            else:
                w = w.double()
            for at in range(lo, hi, 8192):
                to = min(hi, at + 8192)
                x = s["rows"][d, at:to]
                if case["in"] == "mx8":
                    x = _exact_unpack(x[:, :k].view(torch.float8_e4m3fn).double(), x[:, k:k + k // 32])
                v = torch.mm(x.double(), w.t())
                if case["swiglu"]:
                    v = v[:, :width] * torch.sigmoid(v[:, :width]) * v[:, width:]
                if mx:
                    out[0][d, at:to], out[1][d, at:to] = _exact_mx8(v)
                else:
                    out[0][d, at:to] = v
    return out if mx else out[0]


def exact(case, seed):
    if case["op"] != "norm" and 2 * case["rows"] * case["n"] * case["k"] > 2e13:
        return None
    s = prepare(case, seed)
    return _exact_norm(case, s) if case["op"] == "norm" else _exact_experts(case, s)
