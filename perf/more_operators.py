"""Cases for the operators around a training step of the routed experts: the router's
choice of experts with its weights, the balance loss with the experts' counts, the
gradients of both, and the AdamW step that turns gradients into the next weights (with
states in 32 or 8 bits, a bf16 copy, or the experts' 8-bit codes).

Sizes are those of this repository's workloads (hidden 7168, expert width 2048, top-8 of
4096 tokens), of its expert counts, and generic odd ones. `run` computes the plain form,
or calls the framework where `own` is true.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
BLOCK = 128  # values of an 8-bit state that share a scale
BETA1, BETA2, EPS, DECAY, LR = 0.9, 0.999, 1e-8, 0.1, 3e-4


# ------------------------------------------------------------------------ cases
def listed():
    return [
        # one token of a serving loop chooses its experts: latency
        {"name": "router_one_token", "kind": "router", "T": 1, "E": 256, "k": 8, "dtype": "f32",
         "score": "sigmoid", "bias": True, "normalize": True, "balance": False, "B": 1, "pad": 0},
        # a training batch of ragged sequences: choice, weights, counts and loss per sequence
        {"name": "router_batch", "kind": "router", "T": 4096, "E": 256, "k": 8, "dtype": "f32",
         "score": "sigmoid", "bias": True, "normalize": True, "balance": True, "B": 5, "pad": 0},
        # a large batch as one sequence, bf16 logits, the classic softmax router
        {"name": "router_large", "kind": "router", "T": 65536, "E": 128, "k": 8, "dtype": "bf16",
         "score": "softmax", "bias": False, "normalize": False, "balance": True, "B": 1, "pad": 0},
        # counts and loss of choices that were made elsewhere: an odd number of experts
        {"name": "balance_odd", "kind": "balance", "T": 5003, "E": 61, "k": 6, "dtype": "f32",
         "score": "softmax", "bias": False, "normalize": True, "balance": True, "B": 7, "pad": 300},
        # the same for many experts and a large batch
        {"name": "balance_large", "kind": "balance", "T": 32768, "E": 512, "k": 8, "dtype": "f32",
         "score": "sigmoid", "bias": False, "normalize": True, "balance": True, "B": 8, "pad": 0},
        # the gradient of both into the logits of a training batch
        {"name": "router_backward_batch", "kind": "router_bwd", "T": 4096, "E": 256, "k": 8,
         "dtype": "f32", "score": "sigmoid", "bias": True, "normalize": True, "balance": True,
         "B": 5, "pad": 0},
        # of a large padded batch with bf16 logits
        {"name": "router_backward_large", "kind": "router_bwd", "T": 65536, "E": 128, "k": 8,
         "dtype": "bf16", "score": "softmax", "bias": False, "normalize": False, "balance": True,
         "B": 17, "pad": 1000},
        # the small parameters of a block (norms, router bias, odd ones): latency
        {"name": "adamw_small", "kind": "adamw", "tensors": 9, "total": 40000, "bits": 32,
         "gtype": "f32", "copy": False, "on_device": False},
        # many parameters of odd sizes in bf16 with f32 masters; step and rate on the device
        {"name": "adamw_many", "kind": "adamw", "tensors": 300, "total": 60000000, "bits": 32,
         "gtype": "bf16", "copy": True, "on_device": True},
        # the same with 8-bit states and f32 gradients
        {"name": "adamw_many_8bit", "kind": "adamw", "tensors": 300, "total": 60000000, "bits": 8,
         "gtype": "f32", "copy": True, "on_device": False},
        # the experts' weights of a block, from gradients to the next forward's 8-bit codes
        {"name": "adamw_experts", "kind": "adamw_codes", "E": 8, "K": 7168, "F": 2048, "bits": 32},
        # the same with 8-bit states
        {"name": "adamw_experts_8bit", "kind": "adamw_codes", "E": 8, "K": 7168, "F": 2048,
         "bits": 8},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["router", "router", "balance", "router_bwd", "router_bwd", "adamw",
                       "adamw", "adamw_codes"])
    if kind in ("router", "balance", "router_bwd"):
        E = rng.choice([8, 17, 32, 61, 64, 128, 160, 256, 384, 512, 1000])
        T = _log(rng, 1, min(65536, 32768 * 512 // E))
        balance = kind != "router" or rng.random() < 0.6
        return {"kind": kind, "T": T, "E": E, "k": rng.randint(1, 8),
                "dtype": rng.choice(["bf16", "f32"]), "score": rng.choice(["softmax", "sigmoid"]),
                "bias": kind == "router" and rng.random() < 0.5,
                "normalize": rng.random() < 0.7, "balance": balance,
                "B": min(T, _log(rng, 1, 64)), "pad": rng.choice([0, 0, T // 9])}
    if kind == "adamw":
        return {"kind": kind, "tensors": _log(rng, 1, 400), "total": _log(rng, 5000, 60000000),
                "bits": rng.choice([8, 32]), "gtype": rng.choice(["bf16", "f32"]),
                "copy": rng.random() < 0.5, "on_device": rng.random() < 0.3}
    return {"kind": kind, "E": rng.randint(1, 8), "K": 32 * _log(rng, 4, 224),
            "F": 16 * _log(rng, 4, 128), "bits": rng.choice([8, 32])}


def _offsets(c):
    """Where the sequences of a batch begin and end: ragged, the padding behind the last."""
    used, B = c["T"] - c["pad"], c["B"]
    w = [1.0 + (i * 7919 % 13) / 4 for i in range(B)]
    at, done = [0], 0.0
    for x in w:
        done += x
        at.append(int(round(used * done / sum(w))))
    return at


def _counts(c):
    """Numbers of values of the tensors of an adamw case: from one value to many, mostly odd."""
    n, total = c["tensors"], c["total"]
    w = [((i * 2654435761) % 997 + 1) ** 3 for i in range(n)]
    out = [max(1, int(total * x / sum(w))) for x in w]
    out[0] = max(1, out[0] + total - sum(out))
    return out


# ---------------------------------------------------------------------- prepare
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _states(s, g, n, bits, blocks=None):
    """First and second moments as a running program has them."""
    s["m"] = _normal(g, n, scale=3e-4)
    s["v"] = (_normal(g, n, scale=1e-3).square_() + 1e-8 * torch.rand(n, generator=g, device="cuda"))
    if bits == 8:
        zero = torch.zeros((), dtype=torch.int32, device="cuda")
        s["m"], s["m_scale"] = _encode(s["m"], zero, blocks, False)
        s["v"], s["v_scale"] = _encode(torch.sqrt(s["v"]), zero, blocks, True)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": dict(c)}
    if c["kind"] in ("router", "balance", "router_bwd"):
        T, E, k = c["T"], c["E"], c["k"]
        # some experts in more demand, logits of a trained router's spread
        x = torch.randn(T, E, generator=g, device="cuda") * 1.5 + \
            torch.randn(E, generator=g, device="cuda") * 0.5
        s["logits"] = x.to(DT[c["dtype"]])
        s["bias"] = _normal(g, E, scale=0.05) if c["bias"] else None
        at = torch.tensor(_offsets(c), dtype=torch.int32, device="cuda")
        s["offsets"] = at if c["B"] > 1 or c["pad"] else None
        s["scale"] = 2.5 if c["normalize"] else 1.0
        if c["kind"] != "router":
            s["ids"], _ = _choose_plain(s, c)
        if c["kind"] == "router_bwd":
            s["slope"] = _balance_plain(s, c, s["ids"])[2]
            s["dweights"] = _normal(g, T, k, scale=0.1)
            s["dloss"] = 0.001 * T * (1.0 + torch.rand(c["B"], generator=g, device="cuda"))
        return s
    s["step"], s["seed"] = 1000 + int(seed) % 7, int(seed) % 1000
    if c["kind"] == "adamw":
        sizes = _counts(c)
        n = sum(sizes)
        s["sizes"] = sizes
        s["p"] = _normal(g, n, scale=0.02)
        s["g"] = _normal(g, n, scale=1e-3, dtype=DT[c["gtype"]])
        blocks = None
        if c["bits"] == 8:
            per = torch.tensor(sizes, device="cuda")
            first = torch.cumsum(per, 0) - per
            each = -(-per // BLOCK)
            which = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), per)
            s["at"] = torch.arange(n, device="cuda") - first[which]
            s["which"] = which
            blocks = (torch.cumsum(each, 0) - each)[which] + s["at"] // BLOCK
            blocks = s["blocks"] = (blocks, sum(-(-x // BLOCK) for x in sizes))
        _states(s, g, n, c["bits"], blocks)
        s["copy"] = torch.zeros(n, dtype=torch.bfloat16, device="cuda") if c["copy"] else None
        if c["on_device"]:
            s["step_dev"] = torch.tensor([s["step"]], dtype=torch.int64, device="cuda")
            s["lr_dev"] = torch.tensor([LR], dtype=torch.float32, device="cuda")
        return s
    shapes = _expert_shapes(c)
    for name, shape in zip(("wi", "wo"), shapes):
        n = math.prod(shape)
        t = s[name] = {"shape": shape}
        t["p"] = _normal(g, n, scale=0.02)
        t["g"] = _normal(g, n, scale=1e-3)
        _states(t, g, n, c["bits"])
        t["codes"] = torch.zeros(shape, dtype=torch.uint8, device="cuda")
        t["scale"] = torch.zeros(shape[0], shape[2], device="cuda")
    s["grad_scale"] = torch.tensor([0.37], device="cuda")
    return s


def _expert_shapes(c):
    return (c["E"], c["K"], 2 * c["F"]), (c["E"], c["F"], c["K"])


# ------------------------------------------------------- plain forms: the router
def _sequence(s, c):
    """The sequence of each token, B for those behind the last one."""
    t = torch.arange(c["T"], device="cuda")
    if s["offsets"] is None:
        return torch.zeros_like(t)
    return torch.searchsorted(s["offsets"][1:].long(), t, right=True)


def _scores(x, c):
    if c["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _choose_plain(s, c):
    """ids and weights. The order is settled in 64 bits: two values may lie closer than 32 tell."""
    x = s["logits"].double()
    if s["bias"] is not None:
        x = _scores(x, c) + s["bias"].double()
    ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    w = torch.gather(_scores(s["logits"].float(), c), 1, ids)
    if c["normalize"]:
        w = w / w.sum(1, keepdim=True)
    w = w * s["scale"]
    if s["offsets"] is not None:
        inside = (_sequence(s, c) < c["B"]).unsqueeze(1)
        ids = torch.where(inside, ids, torch.full_like(ids, -1))
        w = torch.where(inside, w, torch.zeros_like(w))
    return ids.to(torch.int32), w


def _balance_plain(s, c, ids):
    """counts [B, E], loss [B], slope [B, E] (the loss's derivative by a token's share)."""
    B, E = c["B"], c["E"]
    seq = _sequence(s, c)
    share = _scores(s["logits"].float(), c)
    share = share / share.sum(1, keepdim=True)
    total = torch.zeros(B + 1, E, dtype=torch.float64, device="cuda")
    total.index_add_(0, seq, share.double())
    key = seq.unsqueeze(1) * E + ids.long()
    key = torch.where(ids >= 0, key, torch.full_like(key, B * E)).reshape(-1)
    counts = torch.zeros((B + 1) * E, dtype=torch.int64, device="cuda")
    counts.scatter_add_(0, key, torch.ones_like(key))
    counts = counts.reshape(B + 1, E)[:B]
    n = torch.zeros(B + 1, dtype=torch.int64, device="cuda")
    n.scatter_add_(0, seq, torch.ones_like(seq))
    chosen = counts.sum(1, keepdim=True).double()
    slope = E * counts.double() / (chosen * n[:B].unsqueeze(1).double()).clamp(min=1)
    loss = (slope * total[:B]).sum(1)
    return counts.to(torch.int32), loss.float(), slope.float()


def _router_bwd_plain(s, c):
    x = s["logits"].float()
    score = _scores(x, c)
    share = score / score.sum(1, keepdim=True)
    rate = 1.0 / (1.0 + torch.exp(x)) if c["score"] == "sigmoid" else torch.ones_like(x)
    ids = s["ids"].long()
    inside = (ids[:, :1] >= 0).float()
    ids = ids.clamp(min=0)
    dw = s["dweights"] * inside * s["scale"]
    w = torch.gather(score, 1, ids)
    if c["normalize"]:
        w = w / w.sum(1, keepdim=True)
        dw = dw - (dw * w).sum(1, keepdim=True)
    elif c["score"] == "softmax":
        # the scores that are not chosen share in the sum
        all_dw = torch.zeros_like(x).scatter_(1, ids, dw)
        dw = dw - (all_dw * score).sum(1, keepdim=True)
        dx = -score * (all_dw * score).sum(1, keepdim=True)
        dx.scatter_(1, ids, dw * w)
    if c["normalize"] or c["score"] == "sigmoid":
        dx = torch.zeros_like(x).scatter_(1, ids, dw * w * torch.gather(rate, 1, ids))
    seq = _sequence(s, c).clamp(max=c["B"] - 1)
    d = s["dloss"][seq].unsqueeze(1) * s["slope"][seq] * inside
    dx = dx + share * (d - (d * share).sum(1, keepdim=True)) * rate
    return dx.to(s["logits"].dtype)


# ---------------------------------------------------- plain forms: the optimiser
def _random(at, which, step, seed):
    """32 random bits of a value, from its place: multiplications by the odd numbers next to
    the fractions of the golden ratio and of the roots of 2, 3 and 5, with shifts between them."""
    mask = 0xFFFFFFFF
    key = (seed + 0x6A09E667 * step + 0xBB67AE85 * which) & mask
    x = ((at & mask) * 0x9E3779B9 + (at >> 32) * 0x3C6EF373 + key) & mask
    x = ((x ^ (x >> 16)) * 0xBB67AE85) & mask
    x = ((x ^ (x >> 15)) * 0x6A09E667) & mask
    return x ^ (x >> 16)


def _blocks_max(a, blocks):
    """The largest of each block, and a function that gives every value its block's. blocks:
    the block of every value and their number, or None for whole blocks in order."""
    if blocks is None:
        top = a.reshape(-1, BLOCK).amax(1)
        return top, lambda t: t.unsqueeze(1).expand(-1, BLOCK).reshape(-1)
    at, count = blocks
    top = torch.zeros(count, device="cuda").scatter_reduce_(0, at, a, "amax")
    return top, lambda t: t[at]


def _encode(x, random16, blocks, never_zero):
    """x as e4m3 codes with one scale for BLOCK values: x / scale is rounded up where its
    lower bits and the random ones overflow (the value times 2^-120 has the code's bits
    on top)."""
    top, spread = _blocks_max(x.abs(), blocks)
    scale = top * torch.full_like(top, 1.0 / 448)
    scale = torch.where(scale < 2.0 ** -126, torch.zeros_like(scale), scale)
    inverse = torch.where(scale > 0, torch.ones_like(scale) / scale, torch.zeros_like(scale))
    y = (x.abs() * spread(inverse)) * 2.0 ** -120
    code = ((y.view(torch.int32) + (random16 << 4) + 8) >> 20).clamp(max=0x7E)
    if never_zero:
        code = torch.where((x > 0) & (spread(scale) > 0), code.clamp(min=1), code)
    else:
        code = code + 128 * torch.signbit(x).to(torch.int32)
    return code.to(torch.uint8), scale


def _decode(codes, scale, blocks):
    value = codes.view(torch.float8_e4m3fn).float()
    if blocks is None:
        return (value.reshape(-1, BLOCK) * scale.unsqueeze(1)).reshape(-1)
    return value * scale[blocks[0]]


def _rates(s, c):
    """(1 - lr wd, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)), from 64 bits."""
    if c.get("on_device"):
        t, lr = s["step_dev"].double(), s["lr_dev"].double()
        return ((1 - lr * DECAY).float(), (lr / (1 - BETA1 ** t)).float(),
                (1 / torch.sqrt(1 - BETA2 ** t)).float())
    t = s["step"]
    return 1 - LR * DECAY, LR / (1 - BETA1 ** t), 1 / math.sqrt(1 - BETA2 ** t)


def _moments(p, g, m, v, rates):
    """The step itself: every product and sum rounded by itself."""
    keep, rate, root = rates
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + (g * (1 - BETA2)) * g
    r = torch.sqrt(v)
    return p * keep - (m / (r * root + EPS)) * rate, m, v, r


def _adamw_plain(t, g, rates, step, seed, bits, at, which, blocks):
    """One step on the flat values of t, in place."""
    m, v = t["m"], t["v"]
    if bits == 8:
        m = _decode(m, t["m_scale"], blocks)
        v = _decode(v, t["v_scale"], blocks)
        v = v * v
    p, m, v, r = _moments(t["p"], g, m, v, rates)
    t["p"].copy_(p)
    if bits == 32:
        t["m"].copy_(m)
        t["v"].copy_(v)
        return
    random = _random(at, which, step, seed)
    new = _encode(m, (random & 0xFFFF).to(torch.int32), blocks, False)
    t["m"].copy_(new[0])
    t["m_scale"].copy_(new[1])
    new = _encode(r, (random >> 16).to(torch.int32), blocks, True)
    t["v"].copy_(new[0])
    t["v_scale"].copy_(new[1])


def _experts_plain(t, s, c, which):
    at = torch.arange(t["p"].numel(), device="cuda") if c["bits"] == 8 else None
    _adamw_plain(t, t["g"] * s["grad_scale"], _rates(s, c), s["step"], s["seed"], c["bits"], at,
                 which, None)
    p = t["p"].reshape(t["shape"])
    top = p.abs().amax(1).clamp(min=1e-12)
    t["scale"].copy_(top / torch.full_like(top, 448.0))
    q = (p / t["scale"].unsqueeze(1)).to(torch.float8_e4m3fn)
    t["codes"].copy_(q.view(torch.uint8))


def _told(t):
    """A tensor's new values and states; 8-bit ones as the numbers that their codes are."""
    out = {"p": t["p"], "m": t["m"], "v": t["v"]}
    if "m_scale" in t:
        out |= {"m": t["m"].view(torch.float8_e4m3fn), "m_scale": t["m_scale"],
                "v": t["v"].view(torch.float8_e4m3fn), "v_scale": t["v_scale"]}
    return out


def run(state):
    s, c = state, state["case"]
    kind = c["kind"]
    if own:
        return _run_own(s, c, kind)
    if kind == "router":
        ids, w = _choose_plain(s, c)
        out = {"ids": ids, "weights": w}
        if c["balance"]:
            out["counts"], out["loss"], out["slope"] = _balance_plain(s, c, ids)
        return out
    if kind == "balance":
        counts, loss, slope = _balance_plain(s, c, s["ids"])
        return {"counts": counts, "loss": loss, "slope": slope}
    if kind == "router_bwd":
        return {"dlogits": _router_bwd_plain(s, c)}
    s["step"] += 1
    if kind == "adamw":
        if c["on_device"]:
            s["step_dev"] += 1
        _adamw_plain(s, s["g"].float(), _rates(s, c), s["step"], s["seed"], c["bits"], s.get("at"),
                     s.get("which"), s.get("blocks"))
        out = _told(s)
        if c["copy"]:
            out["copy"] = s["copy"].copy_(s["p"])
        return out
    _experts_plain(s["wi"], s, c, 0)
    _experts_plain(s["wo"], s, c, 1)
    return _experts_told(s)


def _experts_told(s):
    out = {"wi": _told(s["wi"]), "wo": _told(s["wo"])}
    out["wi"] |= {"codes": s["wi"]["codes"].view(torch.float8_e4m3fn), "scale": s["wi"]["scale"]}
    out["wo"] |= {"codes": s["wo"]["codes"].view(torch.float8_e4m3fn), "scale": s["wo"]["scale"]}
    return out


def _run_own(s, c, kind):
    from fp8_moe_routed_gb300 import binding as fb
    if kind == "router":
        ids, w, counts, loss, slope = fb.router_fwd(
            s["logits"], c["k"], score=c["score"], bias=s["bias"], normalize=c["normalize"],
            weight_scale=s["scale"], balance=c["balance"], seq_offsets=s["offsets"])
        out = {"ids": ids, "weights": w}
        if c["balance"]:
            out |= {"counts": counts, "loss": loss, "slope": slope}
        return out
    if kind == "balance":
        counts, loss, slope = fb.balance_fwd(s["logits"], s["ids"], score=c["score"],
                                             seq_offsets=s["offsets"])
        return {"counts": counts, "loss": loss, "slope": slope}
    if kind == "router_bwd":
        return {"dlogits": fb.router_bwd(
            s["dweights"], s["logits"], s["ids"], score=c["score"], normalize=c["normalize"],
            weight_scale=s["scale"], dloss=s["dloss"], slope=s["slope"],
            seq_offsets=s["offsets"])}
    s["step"] += 1
    if "plan" not in s:  # what a program makes once, with its parameters and their states
        s["plan"], s["grads"] = _plan(fb, s, c)
    if kind == "adamw":
        if c["on_device"]:
            s["step_dev"] += 1
        fb.adamw_step(s["plan"], s["grads"], step=s["step_dev"] if c["on_device"] else s["step"],
                      lr=s["lr_dev"] if c["on_device"] else LR, beta1=BETA1, beta2=BETA2, eps=EPS,
                      seed=s["seed"])
        out = _told(s)
        if c["copy"]:
            out["copy"] = s["copy"]
        return out
    fb.adamw_step(s["plan"], s["grads"], step=s["step"], lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS,
                  grad_scale=s["grad_scale"], seed=s["seed"])
    return _experts_told(s)


def _plan(fb, s, c):
    if c["kind"] == "adamw":
        def parts(t, sizes):
            return None if t is None else list(torch.split(t, sizes))
        n, nb = s["sizes"], [-(-x // BLOCK) for x in s["sizes"]]
        plan = fb.AdamwPlan(parts(s["p"], n), parts(s["m"], n), parts(s["v"], n),
                            m_scales=parts(s.get("m_scale"), nb),
                            v_scales=parts(s.get("v_scale"), nb), copies=parts(s["copy"], n),
                            weight_decay=DECAY)
        return plan, parts(s["g"], n)
    ts = [s["wi"], s["wo"]]
    scales = {k: [t[k[:-1]] for t in ts] for k in ("m_scales", "v_scales")} if c["bits"] == 8 else {}
    plan = fb.AdamwPlan([t["p"].view(t["shape"]) for t in ts], [t["m"].view(t["shape"]) for t in ts],
                        [t["v"].view(t["shape"]) for t in ts], codes=[t["codes"] for t in ts],
                        code_scales=[t["scale"] for t in ts], weight_decay=DECAY, **scales)
    return plan, [t["g"].view(t["shape"]) for t in ts]


# ------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["kind"] in ("router", "balance", "router_bwd"):
        T, E, k, b = c["T"], c["E"], c["k"], BYTES[c["dtype"]]
        per_seq = (8 * E + 4) * c["B"] if c["balance"] else 0
        if c["kind"] == "router":
            return {"bytes": T * E * b + 8 * T * k + 4 * E * c["bias"] + per_seq,
                    "flops": T * E * (4 + 3 * c["balance"])}
        if c["kind"] == "balance":
            return {"bytes": T * E * b + 4 * T * k + per_seq, "flops": 6 * T * E}
        return {"bytes": 2 * T * E * b + 8 * T * k + 4 * (E + 1) * c["B"], "flops": 11 * T * E}
    if c["kind"] == "adamw":
        n = sum(_counts(c))
        states = 16 if c["bits"] == 32 else 4 + 16 / BLOCK
        return {"bytes": n * (8 + BYTES[c["gtype"]] + states + 2 * c["copy"]), "flops": 15 * n}
    shapes = _expert_shapes(c)
    n = sum(math.prod(x) for x in shapes)
    states = 16 if c["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": n * (8 + 4 + states + 1) + sum(4 * x[0] * x[2] for x in shapes),
            "flops": 18 * n}


# ------------------------------------------------------------------------ exact
def _exact_share(x, c):
    if c["score"] == "sigmoid":
        score = torch.sigmoid(x)
        return score, score / score.sum(1, keepdim=True)
    score = torch.softmax(x, 1)
    return score, score


def _nearest_e4m3(x):
    """The nearest e4m3 number, ties to the even one, found by the spacing at x."""
    _, e = torch.frexp(x.abs().clamp(min=2.0 ** -6))
    step = torch.ldexp(torch.ones_like(x), e - 4)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_adamw(t, c, g, which_rates):
    keep, rate, root = which_rates
    m, v = t["m"], t["v"]
    eight = c["bits"] == 8
    if eight:
        per = t["blocks"][0] if "blocks" in t else \
            torch.arange(t["p"].numel(), device="cuda") // BLOCK
        m = m.view(torch.float8_e4m3fn).double() * t["m_scale"].double()[per]
        v = (v.view(torch.float8_e4m3fn).double() * t["v_scale"].double()[per]).square()
    m = torch.lerp(g, m.double(), BETA1)
    v = torch.lerp(g * g, v.double(), BETA2)
    p = t["p"].double() * keep - rate * m / (root * v.sqrt() + EPS)
    if not eight:
        return {"p": p, "m": m, "v": v}
    # the codes are rounded by chance: only their scales have a value of their own
    def top(a):
        out = torch.zeros(int(per[-1]) + 1, dtype=torch.float64, device="cuda")
        return out.scatter_reduce_(0, per, a.abs(), "amax") / 448
    return {"p": p, "m": None, "m_scale": top(m), "v": None, "v_scale": top(v.sqrt())}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["kind"] in ("router", "balance", "router_bwd"):
        T, E, B = c["T"], c["E"], c["B"]
        x = s["logits"].double()
        score, share = _exact_share(x, c)
        at = _offsets(c) if s["offsets"] is not None else [0, T]
        if c["kind"] == "router_bwd":
            # by the chain of its parts: through the weights, the scores' shares, the scores
            x.requires_grad_(True)
            score, share = _exact_share(x, c)
            used = at[-1]
            w = torch.gather(score[:used], 1, s["ids"][:used].long())
            if c["normalize"]:
                w = w / w.sum(1, keepdim=True)
            total = (w * s["dweights"][:used].double()).sum() * s["scale"]
            for b in range(B):
                part = share[at[b]:at[b + 1]].sum(0)
                total = total + s["dloss"][b].double() * (part * s["slope"][b].double()).sum()
            return {"dlogits": torch.autograd.grad(total, x)[0]}
        out = {}
        if c["kind"] == "router":
            rank = x if s["bias"] is None else score + s["bias"].double()
            ids = torch.argsort(rank, dim=1, descending=True, stable=True)[:, :c["k"]]
            w = torch.gather(score, 1, ids)
            if c["normalize"]:
                w = w / w.sum(1, keepdim=True)
            w[at[-1]:] = 0
            out = {"ids": None, "weights": w * s["scale"]}
            if not c["balance"]:
                return out
        else:
            ids = s["ids"].long()
        loss, slope = [], []
        for b in range(B):
            n = at[b + 1] - at[b]
            counts = torch.bincount(ids[at[b]:at[b + 1]].reshape(-1), minlength=E).double()
            d = counts * (E / max(1, n * n * c["k"]))
            slope.append(d)
            loss.append(torch.dot(d, share[at[b]:at[b + 1]].sum(0)))
        return out | {"counts": None, "loss": torch.stack(loss), "slope": torch.stack(slope)}
    t, lr = s["step"] + 1, LR
    if c.get("on_device"):
        lr = s["lr_dev"].item()
    rates = 1 - lr * DECAY, lr / (1 - BETA1 ** t), (1 - BETA2 ** t) ** -0.5
    if c["kind"] == "adamw":
        out = _exact_adamw(s, c, s["g"].double(), rates)
        if c["copy"]:
            out["copy"] = out["p"]
        return out
    out = {}
    for name in ("wi", "wo"):
        w = s[name]
        r = _exact_adamw(w, c, w["g"].double() * s["grad_scale"].double(), rates)
        p = r["p"].reshape(w["shape"])
        r["scale"] = p.abs().amax(1) / 448
        r["codes"] = _nearest_e4m3(p / r["scale"].unsqueeze(1))
        out[name] = r
    return out
