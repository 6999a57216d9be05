"""Cases for the operators around the routed experts: tokens sorted by expert and
back with their gradients, the norms before and after the block with its gate and
residual scale, and the microscaled 4-bit (MXFP4) quantisation and grouped product.

Sizes are those of this repository's workloads (hidden 7168, expert width 2048, 32
experts, top-8 of 4096 tokens; the Zipf(1.2) routing over 28 of 32 experts), of its
tiny configuration, and generic odd ones. `run` computes the plain form in f32, or
calls the framework where `own` is true.
"""
import math

import torch

own = False

EPS = 1e-6
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------------ cases
def listed():
    return [
        # one token of a serving loop on its way to its eight experts: latency
        {"name": "dispatch_one_token", "kind": "dispatch", "T": 1, "k": 8, "E": 32, "H": 7168,
         "dtype": "bf16", "keep": 1.0},
        # a training batch: 4096 tokens, top-8 of 32 experts
        {"name": "dispatch_batch", "kind": "dispatch", "T": 4096, "k": 8, "E": 32, "H": 7168,
         "dtype": "bf16", "keep": 1.0},
        # the way back on one expert-parallel rank that holds a part of the experts
        {"name": "combine_part", "kind": "combine", "T": 4093, "k": 8, "E": 32, "H": 4096,
         "dtype": "bf16", "keep": 0.75},
        # both gradients of a training batch: of the weighted sum and of the sorted copy
        {"name": "route_backward_batch", "kind": "route_bwd", "T": 4096, "k": 8, "E": 32,
         "H": 7168, "dtype": "bf16", "keep": 1.0},
        # the norms between two blocks for a handful of decoded tokens: latency
        {"name": "norms_decode", "kind": "norm_fwd", "T": 7, "H": 7168, "dtype": "bf16",
         "parts": "both", "gate": "channel", "sigmoid": False},
        # a training batch, the block's output under a learned gate per token
        {"name": "norms_batch", "kind": "norm_fwd", "T": 4096, "H": 7168, "dtype": "bf16",
         "parts": "both", "gate": "token", "sigmoid": True},
        # its backward pass
        {"name": "norms_backward_batch", "kind": "norm_bwd", "T": 4096, "H": 7168,
         "dtype": "bf16", "parts": "both", "gate": "token", "sigmoid": True},
        # an f32 residual stream of odd length with a gate for every value
        {"name": "norms_backward_odd_f32", "kind": "norm_bwd", "T": 5003, "H": 1544,
         "dtype": "f32", "parts": "both", "gate": "full", "sigmoid": True},
        # 4-bit weights, one token in eight experts: bound by the weights' bytes
        {"name": "mxfp4_wi_one_token", "kind": "mxfp4", "M": 8, "K": 7168, "N": 4096, "E": 32,
         "routing": "spread", "silu": True},
        # the balanced step's first product with SwiGLU, 1024 rows for each expert
        {"name": "mxfp4_wi_balanced", "kind": "mxfp4", "M": 32768, "K": 7168, "N": 4096, "E": 32,
         "routing": "balanced", "silu": True},
        # the second product under a skewed router (some experts have no rows)
        {"name": "mxfp4_wo_skewed", "kind": "mxfp4", "M": 32768, "K": 2048, "N": 7168, "E": 32,
         "routing": "zipf", "silu": False},
        # expert weights brought to 4 bits and read back (loading, or simulated in training)
        {"name": "mxfp4_weights", "kind": "mxfp4_weights", "E": 8, "K": 7168, "N": 4096},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _multiple(rng, lo, hi, step):
    while True:
        n = max(1, int(round(_log(rng, lo, hi) / step))) * step
        if n != 3072 and lo <= n <= hi:
            return n


def draw(rng):
    kind = rng.choice(["dispatch", "combine", "route_bwd", "norm_fwd", "norm_bwd", "mxfp4",
                       "mxfp4", "mxfp4_weights"])
    if kind in ("dispatch", "combine", "route_bwd"):
        return {"kind": kind, "T": _log(rng, 1, 4096), "k": rng.randint(1, 8),
                "E": rng.choice([8, 17, 32, 61, 128, 256]), "H": _multiple(rng, 256, 7168, 8),
                "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "keep": rng.choice([1.0, 1.0, 0.75, 0.25])}
    if kind in ("norm_fwd", "norm_bwd"):
        H = _multiple(rng, 128, 8192, 8)
        T = _log(rng, 1, min(16384, 4096 * 7168 // H))
        return {"kind": kind, "T": T, "H": H, "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "parts": rng.choice(["both", "both", "pre", "post"]),
                "gate": rng.choice(["none", "token", "channel", "full"]),
                "sigmoid": rng.choice([False, True])}
    if kind == "mxfp4":
        return {"kind": kind, "M": _log(rng, 1, 32768), "K": _multiple(rng, 256, 7168, 32),
                "N": _multiple(rng, 256, 4096, 32), "E": rng.choice([4, 8, 17, 32]),
                "routing": rng.choice(["balanced", "zipf", "spread"]),
                "silu": rng.choice([False, True])}
    return {"kind": kind, "E": rng.randint(1, 8), "K": _multiple(rng, 128, 7168, 32),
            "N": _multiple(rng, 128, 4096, 16)}


def _rows_of(c):
    """Rows of the sorted buffer: room for the kept slots of an expert-parallel rank."""
    return c["T"] * c["k"]


def _sizes(c):
    """Group sizes before the seed permutes them."""
    M, E = c["M"], c["E"]
    if c["routing"] == "balanced":
        w = [1.0] * E
    elif c["routing"] == "zipf":
        full = max(1, E * 7 // 8)
        w = [(r + 1) ** -1.2 for r in range(full)] + [0.0] * (E - full)
    else:  # every row to an expert of its own, as far as there are any, at most eight experts
        full = min(E, 8)
        w = [1.0] * full + [0.0] * (E - full)
    raw = [M * x / sum(w) for x in w]
    n = [int(x) for x in raw]
    order = sorted(range(E), key=lambda i: n[i] - raw[i])
    for i in order[:M - sum(n)]:
        n[i] += 1
    return n


# ---------------------------------------------------------------------- prepare
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _gate_shape(c):
    return {"none": None, "token": (c["T"],), "channel": (c["H"],),
            "full": (c["T"], c["H"])}[c["gate"]]


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": dict(c)}
    if c["kind"] in ("dispatch", "combine", "route_bwd"):
        T, k, E, H, dt = c["T"], c["k"], c["E"], c["H"], DT[c["dtype"]]
        M = _rows_of(c)
        # a router's choice: distinct experts for each token, some experts in more demand
        score = torch.randn(T, E, generator=g, device="cuda") + \
            torch.randn(E, generator=g, device="cuda") * 0.5
        ids = torch.topk(score, k, dim=1).indices.to(torch.int32)
        if c["keep"] < 1.0:  # slots whose expert another rank holds
            away = torch.rand(T, k, generator=g, device="cuda") >= c["keep"]
            ids = torch.where(away, torch.full_like(ids, -1), ids)
        s["ids"] = ids.contiguous()
        s["M"] = M
        if c["kind"] == "dispatch":
            s["x"] = _normal(g, T, H, dtype=dt)
            s["rows"] = torch.zeros(M, H, dtype=dt, device="cuda")
            return s
        s["slot_row"], s["row_slot"] = _sort_plain(s["ids"], E, M)[1:]
        w = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), dim=1)
        s["weights"] = w.contiguous()
        s["y"] = _normal(g, M, H, dtype=dt)
        if c["kind"] == "route_bwd":
            s["dout"] = _normal(g, T, H, scale=0.01, dtype=dt)
            s["drows_in"] = _normal(g, M, H, scale=0.01, dtype=dt)
            s["drows"] = torch.zeros(M, H, dtype=dt, device="cuda")
        return s
    if c["kind"] in ("norm_fwd", "norm_bwd"):
        T, H, dt = c["T"], c["H"], DT[c["dtype"]]
        post, pre = c["parts"] in ("both", "post"), c["parts"] in ("both", "pre")
        s["residual_scale"], s["branch_scale"] = 1.0, 0.7071
        s["x"] = _normal(g, T, H, scale=2.0, dtype=dt)
        s["y"] = _normal(g, T, H, scale=0.3, dtype=dt) if post else None
        s["w_post"] = 1.0 + _normal(g, H, scale=0.2) if post else None
        s["w_pre"] = 1.0 + _normal(g, H, scale=0.2) if pre else None
        shape = _gate_shape(c) if post else None
        s["gate"] = None
        if shape is not None:
            s["gate"] = _normal(g, *shape, dtype=dt if c["gate"] == "full" else torch.float32)
        s["sigmoid"] = bool(c["sigmoid"]) and s["gate"] is not None
        if c["kind"] == "norm_bwd":
            r, _, s["rstd_post"], s["rstd_pre"] = _norm_plain(s)
            s["r"] = r if post else s["x"]
            s["dr"] = _normal(g, T, H, scale=0.01, dtype=dt)
            s["dh"] = _normal(g, T, H, scale=0.01, dtype=dt) if pre else None
        return s
    if c["kind"] == "mxfp4":
        M, K, N, E = c["M"], c["K"], c["N"], c["E"]
        perm = torch.randperm(E, generator=g, device="cuda").tolist()
        n = _sizes(c)
        s["sizes"] = [n[i] for i in perm]
        s["group_sizes"] = torch.tensor(s["sizes"], dtype=torch.int32, device="cuda")
        x = torch.randn(M, K, generator=g, device="cuda")
        big = torch.rand(M, 1, generator=g, device="cuda") < 0.001
        s["x"] = torch.where(big, x * 50, x).to(torch.bfloat16)
        codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(E, (K + 127) // 128, N, 4, dtype=torch.uint8, device="cuda")
        for e in range(E):
            w = (torch.randn(N, K, generator=g, device="cuda") * 0.02).to(torch.bfloat16)
            codes[e], scales[e] = _pack(*_quantize_plain(w.float()))
        s["codes"], s["scales"] = codes, scales
        s["out"] = torch.zeros(M, N // 2 if c["silu"] else N, dtype=torch.bfloat16, device="cuda")
        return s
    E, K, N = c["E"], c["K"], c["N"]
    w = _normal(g, E, K, N, scale=0.02)
    outlier = torch.rand(E, K, 1, generator=g, device="cuda") < 0.002
    s["w"] = torch.where(outlier, w * 30, w).to(torch.bfloat16)
    return s


# ------------------------------------------------------------------ plain forms
def _sort_plain(ids, E, M):
    key = ids.reshape(-1).long()
    key = torch.where((key < 0) | (key >= E), torch.full_like(key, E), key)
    n = key.numel()
    order = torch.argsort(key, stable=True)
    count = torch.zeros(E + 1, dtype=torch.long, device=key.device)
    count.scatter_add_(0, key, torch.ones_like(key))
    end = torch.cumsum(count[:E], 0).clamp(max=M)
    sizes = torch.diff(end, prepend=torch.zeros_like(end[:1]))
    place = torch.empty_like(key)
    place[order] = torch.arange(n, device=key.device)
    slot_row = torch.where((key < E) & (place < M), place, torch.full_like(place, -1))
    row_slot = torch.full((M,), -1, dtype=torch.long, device=key.device)
    m = min(n, M)
    row_slot[:m] = torch.where(key[order[:m]] < E, order[:m], torch.full_like(order[:m], -1))
    i32 = torch.int32
    return sizes.to(i32), slot_row.reshape(ids.shape).to(i32), row_slot.to(i32)


def _by_token(rows, slot_row):
    """rows [M, H] as f32 [T, k, H], zero where a slot has no row."""
    at = slot_row.long()
    v = rows[at.clamp(min=0)].float()
    return v * (at >= 0).unsqueeze(-1)


def _combine_plain(rows, slot_row, weights):
    v = _by_token(rows, slot_row)
    if weights is not None:
        v = v * weights.unsqueeze(-1)
    return v.sum(1).to(rows.dtype)


def _combine_bwd_plain(dout, rows, slot_row, row_slot, weights):
    k = slot_row.shape[1]
    dweights = (_by_token(rows, slot_row) * dout.float().unsqueeze(1)).sum(-1)
    slot = row_slot.long().clamp(min=0)
    drows = weights.reshape(-1)[slot].unsqueeze(1) * dout[slot // k].float()
    drows = torch.where((row_slot >= 0).unsqueeze(1), drows, torch.zeros_like(drows))
    return drows.to(rows.dtype), dweights


def _gate_value(s):
    if s["gate"] is None:
        return None
    v = s["gate"].float()
    if s["sigmoid"]:
        v = 1.0 / (1.0 + torch.exp(-v))
    return v.unsqueeze(1) if s["case"]["gate"] == "token" else v


def _norm_plain(s):
    x = s["x"].float()
    rstd_post = rstd_pre = h = None
    r = x
    if s["y"] is not None:
        y = s["y"].float()
        rstd_post = 1.0 / torch.sqrt((y * y).mean(1) + EPS)
        b = y * rstd_post.unsqueeze(1) * s["w_post"]
        g = _gate_value(s)
        if g is not None:
            b = b * g
        r = s["residual_scale"] * x + s["branch_scale"] * b
    if s["w_pre"] is not None:
        rstd_pre = 1.0 / torch.sqrt((r * r).mean(1) + EPS)
        h = (r * rstd_pre.unsqueeze(1) * s["w_pre"]).to(s["x"].dtype)
    return (r.to(s["x"].dtype) if s["y"] is not None else None), h, rstd_post, rstd_pre


def _norm_bwd_plain(s):
    dt = s["x"].dtype
    d = s["dr"].float()
    dw_pre = dy = dw_post = dgate = None
    if s["w_pre"] is not None:
        rh = s["r"].float() * s["rstd_pre"].unsqueeze(1)
        dh = s["dh"].float()
        dw_pre = (dh * rh).sum(0)
        u = dh * s["w_pre"]
        d = d + s["rstd_pre"].unsqueeze(1) * (u - rh * (u * rh).mean(1, keepdim=True))
    if s["y"] is None:
        return d.to(dt), dy, dw_post, dw_pre, dgate
    yh = s["y"].float() * s["rstd_post"].unsqueeze(1)
    db = s["branch_scale"] * d
    dn = db
    g = _gate_value(s)
    if g is not None:
        dn = db * g
        dg = db * yh * s["w_post"]
        if s["sigmoid"]:
            dg = dg * (g * (1.0 - g))
        kind = s["case"]["gate"]
        dgate = dg.sum(1) if kind == "token" else dg.sum(0) if kind == "channel" else dg.to(dt)
    dw_post = (dn * yh).sum(0)
    u = dn * s["w_post"]
    dy = s["rstd_post"].unsqueeze(1) * (u - yh * (u * yh).mean(1, keepdim=True))
    return (s["residual_scale"] * d).to(dt), dy.to(dt), dw_post, dw_pre, dgate


def _pow2(biased):
    """2^(biased - 127) in f32, from its bits (torch.ldexp's powers may be rounded)."""
    b = biased.to(torch.int32)
    return torch.where(b > 0, b << 23, torch.full_like(b, 1 << 22)).view(torch.float32)


def _quantize_plain(v):
    """f32 [..., K] -> e2m1 codes u8 [..., K] and biased exponents u8 [..., K/32]."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    amax = b.abs().amax(-1)
    # floor(log2(amax)) is the exponent field of the f32 value
    e = ((amax.view(torch.int32) >> 23) - 127 - 2).clamp(min=-127)
    a = (b * _pow2(127 - e).unsqueeze(-1)).abs()
    # the grid 0, .5, 1, 1.5, 2, 3, 4, 6: ties go to the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) +
            (a >= 3.5) + (a > 5.0))
    code = code + 8 * torch.signbit(b).to(torch.uint8)
    return code.reshape(v.shape), (e + 127).to(torch.uint8)


def _pack(code, exponent):
    """Codes two a byte (the even one low), exponents [N, K/32] as [K/128, N, 4]."""
    N, nb = exponent.shape
    pad = torch.zeros(N, -(-nb // 4) * 4, dtype=torch.uint8, device=code.device)
    pad[:, :nb] = exponent
    return code[:, 0::2] | (code[:, 1::2] << 4), \
        pad.reshape(N, -1, 4).permute(1, 0, 2).contiguous()


def _grid(device, dtype):
    t = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=device, dtype=dtype)
    return torch.cat([t, -t])


def _values(code, exponent):
    """Codes and biased exponents as the f32 values that they stand for."""
    v = _grid(code.device, torch.float32)[code.long()]
    return v * _pow2(exponent).repeat_interleave(32, dim=-1)


def _unpack(codes, scales):
    """One expert's weights [N, K] as codes and exponents [N, K/32]."""
    N, half = codes.shape
    code = torch.stack([codes & 15, codes >> 4], -1).reshape(N, 2 * half)
    return code, scales.permute(1, 0, 2).reshape(N, -1)[:, :2 * half // 32]


def _mxfp4_plain(s):
    c = s["case"]
    parts = []
    xs = torch.split(s["x"], s["sizes"])
    for e in range(c["E"]):
        if s["sizes"][e] == 0:
            continue
        a = _values(*_quantize_plain(xs[e].float()))
        y = a @ _values(*_unpack(s["codes"][e], s["scales"][e])).t()
        if c["silu"]:
            gate, up = y.chunk(2, dim=1)
            y = gate / (1.0 + torch.exp(-gate)) * up
        parts.append(y)
    return torch.cat(parts).to(torch.bfloat16)


def run(state):
    s, c = state, state["case"]
    kind = c["kind"]
    if own:
        return _run_own(s, c, kind)
    if kind == "dispatch":
        sizes, slot_row, row_slot = _sort_plain(s["ids"], c["E"], s["M"])
        rows = s["x"][row_slot.long().clamp(min=0) // c["k"]]
        rows = torch.where((row_slot >= 0).unsqueeze(1), rows, torch.zeros_like(rows))
        return {"group_sizes": sizes, "slot_row": slot_row, "row_slot": row_slot, "rows": rows}
    if kind == "combine":
        return {"out": _combine_plain(s["y"], s["slot_row"], s["weights"])}
    if kind == "route_bwd":
        drows, dweights = _combine_bwd_plain(s["dout"], s["y"], s["slot_row"], s["row_slot"],
                                             s["weights"])
        return {"drows": drows, "dweights": dweights,
                "dx": _combine_plain(s["drows_in"], s["slot_row"], None)}
    if kind == "norm_fwd":
        return list(_norm_plain(s))
    if kind == "norm_bwd":
        return list(_norm_bwd_plain(s))
    if kind == "mxfp4":
        return _mxfp4_plain(s)
    w = s["w"].transpose(1, 2).float()
    return _values(*_quantize_plain(w)).to(torch.bfloat16)


def _run_own(s, c, kind):
    from fp8_moe_routed_gb300 import binding as fb
    if kind == "dispatch":
        rows, sizes, slot_row, row_slot = fb.dispatch_tokens(s["x"], s["ids"], c["E"], s["M"],
                                                             out=s["rows"])
        return {"group_sizes": sizes, "slot_row": slot_row, "row_slot": row_slot, "rows": rows}
    if kind == "combine":
        return {"out": fb.combine_tokens(s["y"], s["slot_row"], s["weights"])}
    if kind == "route_bwd":
        drows, dweights = fb.combine_tokens_bwd(s["dout"], s["y"], s["slot_row"], s["weights"],
                                                out=s["drows"])
        return {"drows": drows, "dweights": dweights,
                "dx": fb.dispatch_tokens_bwd(s["drows_in"], s["slot_row"])}
    if kind == "norm_fwd":
        return list(fb.norm_fwd(s["x"], s["y"], s["w_post"], s["w_pre"], gate=s["gate"],
                                gate_kind=None if s["gate"] is None else c["gate"],
                                sigmoid=s["sigmoid"], residual_scale=s["residual_scale"],
                                branch_scale=s["branch_scale"], eps=EPS))
    if kind == "norm_bwd":
        return list(fb.norm_bwd(s["dr"], s["dh"], s["r"], s["y"], s["w_post"], s["w_pre"],
                                s["rstd_post"], s["rstd_pre"], gate=s["gate"],
                                gate_kind=None if s["gate"] is None else c["gate"],
                                sigmoid=s["sigmoid"], residual_scale=s["residual_scale"],
                                branch_scale=s["branch_scale"]))
    if kind == "mxfp4":
        f = fb.gmm_silu_mxfp4_fwd if c["silu"] else fb.gmm_mxfp4_fwd
        return f(s["x"], s["codes"], s["scales"], s["group_sizes"], out=s["out"])
    codes, scales = fb.mxfp4_quantize_weights(s["w"])
    return fb.mxfp4_dequantize(codes, scales)


# ------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["kind"] in ("dispatch", "combine", "route_bwd"):
        T, k, H, b, M = c["T"], c["k"], c["H"], BYTES[c["dtype"]], _rows_of(c)
        n = T * k * c["keep"]
        if c["kind"] == "dispatch":
            return {"bytes": T * H * b + n * H * b + 8 * T * k + 4 * M + 4 * c["E"], "flops": 0}
        if c["kind"] == "combine":
            return {"bytes": n * H * b + T * H * b + 8 * T * k, "flops": 2 * n * H}
        return {"bytes": 2 * T * H * b + 3 * n * H * b + 16 * T * k, "flops": 4 * n * H}
    if c["kind"] in ("norm_fwd", "norm_bwd"):
        T, H, b = c["T"], c["H"], BYTES[c["dtype"]]
        post, pre = c["parts"] in ("both", "post"), c["parts"] in ("both", "pre")
        if c["kind"] == "norm_fwd":
            n = 1 + 2 * post + pre + (post and c["gate"] == "full")
            return {"bytes": n * T * H * b + 4 * T * (post + pre) + 4 * H * (post + pre),
                    "flops": T * H * (7 * post + 4 * pre)}
        n = 2 + 2 * post + 2 * pre + 2 * (post and c["gate"] == "full")
        return {"bytes": n * T * H * b + 4 * T * (post + pre) + 8 * H * (post + pre),
                "flops": T * H * (14 * post + 11 * pre)}
    if c["kind"] == "mxfp4":
        M, K, N = c["M"], c["K"], c["N"]
        used = sum(1 for n in _sizes(c) if n)
        return {"bytes": 2 * M * K + used * N * (K // 2 + K // 32) +
                2 * M * (N // 2 if c["silu"] else N), "flops": 2 * M * K * N}
    n = c["E"] * c["K"] * c["N"]
    return {"bytes": 2 * n + 2 * n, "flops": 0}


# ------------------------------------------------------------------------ exact
def _d(t):
    return None if t is None else t.double()


def _exact_mxfp4_operand(v):
    """Definition in 64 bits: block scale 2^(floor(log2 amax) - 2), nearest grid value
    with ties to the even code, found by distance."""
    b = v.double().reshape(*v.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    mant, ex = torch.frexp(amax)
    ex = torch.where(mant == 0, torch.full_like(ex, -127), (ex - 3).clamp(min=-127))
    scale = ((ex.long() + 1023) << 52).view(torch.float64)
    a = (b / scale).abs()
    grid = _grid(v.device, torch.float64)[:8]
    best = torch.zeros_like(a)
    gap = a.clone()
    for i in (2, 4, 6, 1, 3, 5, 7):  # even codes first: an odd one has to be nearer
        near = (a - grid[i]).abs()
        take = near < gap
        best = torch.where(take, grid[i], best)
        gap = torch.where(take, near, gap)
    return (torch.copysign(best, b) * scale).reshape(v.shape)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["kind"] == "dispatch":
        # whole numbers and copies: each kept row, found from its slot
        place = _sort_plain(s["ids"], c["E"], s["M"])[1].reshape(-1).long()
        kept = torch.nonzero(place >= 0).reshape(-1)
        rows = torch.zeros(s["M"], c["H"], dtype=torch.float64, device="cuda")
        rows[place[kept]] = s["x"].double()[kept // c["k"]]
        return {"group_sizes": None, "slot_row": None, "row_slot": None, "rows": rows}
    if c["kind"] in ("combine", "route_bwd"):
        T, k = s["ids"].shape
        at = s["slot_row"].reshape(-1).long()
        kept = torch.nonzero(at >= 0).reshape(-1)
        token = kept // k

        def back(rows, weights):
            total = torch.zeros(T, c["H"], dtype=torch.float64, device="cuda")
            v = rows[at[kept]].double()
            if weights is not None:
                v = v * weights.reshape(-1)[kept].double().unsqueeze(1)
            return total.index_add_(0, token, v)

        if c["kind"] == "combine":
            return {"out": back(s["y"], s["weights"])}
        w = s["weights"].reshape(-1)[kept].double()
        d = s["dout"].double()[token]
        drows = torch.zeros(s["M"], c["H"], dtype=torch.float64, device="cuda")
        drows[at[kept]] = w.unsqueeze(1) * d
        dweights = torch.zeros(T * k, dtype=torch.float64, device="cuda")
        dweights[kept] = (s["y"][at[kept]].double() * d).sum(1)
        return {"drows": drows, "dweights": dweights.reshape(T, k),
                "dx": back(s["drows_in"], None)}
    if c["kind"] == "norm_fwd":
        x, y, gate = _d(s["x"]), _d(s["y"]), _d(s["gate"])
        r, rp, rq, h = x, None, None, None
        if y is not None:
            rp = (y.square().mean(1) + EPS).rsqrt()
            g = 1.0
            if gate is not None:
                g = torch.sigmoid(gate) if s["sigmoid"] else gate
                g = g[:, None] if c["gate"] == "token" else g
            r = s["residual_scale"] * x + s["branch_scale"] * g * (y * rp[:, None] *
                                                                  _d(s["w_post"]))
        if s["w_pre"] is not None:
            rq = (r.square().mean(1) + EPS).rsqrt()
            h = r * rq[:, None] * _d(s["w_pre"])
        return [r if y is not None else None, h, rp, rq]
    if c["kind"] == "norm_bwd":
        # the saved rstd are inputs here; a row's gradient through them is the projection
        D = _d(s["dr"])
        H = c["H"]
        dw_pre = None
        if s["w_pre"] is not None:
            rh = _d(s["r"]) * _d(s["rstd_pre"])[:, None]
            u = _d(s["dh"]) * _d(s["w_pre"])
            dot = torch.einsum("th,th->t", u, rh) / H
            D = D + _d(s["rstd_pre"])[:, None] * (u - rh * dot[:, None])
            dw_pre = torch.einsum("th,th->h", _d(s["dh"]), rh)
        if s["y"] is None:
            return [D, None, None, dw_pre, None]
        yh = _d(s["y"]) * _d(s["rstd_post"])[:, None]
        bD = s["branch_scale"] * D
        n = yh * _d(s["w_post"])
        g, slope, dgate = torch.ones((), dtype=torch.float64, device="cuda"), 1.0, None
        if s["gate"] is not None:
            z = _d(s["gate"])
            z = z[:, None] if c["gate"] == "token" else z
            g = torch.sigmoid(z) if s["sigmoid"] else z
            slope = g * (1 - g) if s["sigmoid"] else 1.0
            dgate = bD * n * slope
            if c["gate"] == "token":
                dgate = dgate.sum(1)
            elif c["gate"] == "channel":
                dgate = dgate.sum(0)
        dn = bD * g
        u = dn * _d(s["w_post"])
        dot = torch.einsum("th,th->t", u, yh) / H
        dy = _d(s["rstd_post"])[:, None] * (u - yh * dot[:, None])
        return [s["residual_scale"] * D, dy, torch.einsum("th,th->h", dn, yh), dw_pre, dgate]
    if c["kind"] == "mxfp4":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        grid = _grid("cuda", torch.float64)
        row = 0
        for e, n in enumerate(s["sizes"]):
            if not n:
                continue
            code = s["codes"][e]
            w = torch.empty(c["N"], c["K"], dtype=torch.float64, device="cuda")
            w[:, 0::2] = grid[(code % 16).long()]
            w[:, 1::2] = grid[(code // 16).long()]
            ex = s["scales"][e].transpose(0, 1).reshape(c["N"], -1)[:, :c["K"] // 32]
            power = ((ex.long() - 127 + 1023) << 52).view(torch.float64)
            w = w.reshape(c["N"], -1, 32) * power[:, :, None]
            w = w.reshape(c["N"], c["K"])
            y = _exact_mxfp4_operand(s["x"][row:row + n]) @ w.T
            if c["silu"]:
                half = c["N"] // 2
                y = torch.nn.functional.silu(y[:, :half]) * y[:, half:]
            out[row:row + n] = y
            row += n
        return out
    return torch.stack([_exact_mxfp4_operand(w.T.contiguous()) for w in s["w"]])
