"""Plain 64-bit forms of the operators around the routed experts, for the tests:
tokens sorted by expert and back, the norms around a block, MXFP4. Written from the
definitions in include/fp8moe.h; nothing here calls the library."""
import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


# ------------------------------------------------------------------------ tokens
def sort_tokens(ids, E, M):
    """(group_sizes, slot_row, row_slot) by Python's stable sort; lists."""
    flat = ids.reshape(-1).tolist()
    kept = sorted((s for s, e in enumerate(flat) if 0 <= e < E), key=lambda s: flat[s])[:M]
    slot_row = [-1] * len(flat)
    for row, s in enumerate(kept):
        slot_row[s] = row
    sizes = [0] * E
    for s in kept:
        sizes[flat[s]] += 1
    return sizes, slot_row, kept + [-1] * (M - len(kept))


def combine(rows, slot_row, weights=None):
    T, k = slot_row.shape
    out = torch.zeros(T, rows.shape[1], dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            r = int(slot_row[t, j])
            if 0 <= r < rows.shape[0]:
                w = 1.0 if weights is None else float(weights[t, j])
                out[t] += w * rows[r].double()
    return out


def combine_bwd(dout, rows, slot_row, weights):
    T, k = slot_row.shape
    drows = torch.zeros(rows.shape, dtype=torch.float64)
    dw = torch.zeros(T, k, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            r = int(slot_row[t, j])
            if 0 <= r < rows.shape[0]:
                drows[r] = float(weights[t, j]) * dout[t].double()
                dw[t, j] = (dout[t].double() * rows[r].double()).sum()
    return drows, dw


# ------------------------------------------------------------------------- norms
def gate_value(gate, kind, sigmoid):
    if gate is None:
        return 1.0
    g = torch.sigmoid(gate) if sigmoid else gate
    return g[:, None] if kind == "token" else g


def norm_fwd(x, y, w_post, w_pre, gate, kind, sigmoid, a, b, eps):
    """float64 in, float64 out; differentiable."""
    r = x
    if w_post is not None:
        n = w_post * y / torch.sqrt(y.square().mean(1, keepdim=True) + eps)
        r = a * x + b * gate_value(gate, kind, sigmoid) * n
    h = None
    if w_pre is not None:
        h = w_pre * r / torch.sqrt(r.square().mean(1, keepdim=True) + eps)
    return r, h


# ------------------------------------------------------------------------- MXFP4
def mx_quantize(v):
    """float64 [..., K] -> codes uint8 [..., K], scale bytes uint8 [..., K/32]."""
    b = v.double().reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    amax = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    safe = torch.where(bad | (amax == 0), torch.ones_like(amax), amax)
    e = torch.frexp(safe)[1].long() - 1 - 2            # floor(log2 amax) - 2
    e = torch.where(amax == 0, torch.full_like(e, -127), e).clamp(min=-127)
    q = (b / torch.ldexp(torch.ones_like(amax), e)[..., None]).abs()
    q = torch.where(bad[..., None], torch.zeros_like(q), q)
    dist = (q[..., None] - E2M1).abs()
    near = dist.amin(-1, keepdim=True)
    tied = dist == near                                # one code, or two neighbours
    even = torch.arange(8) % 2 == 0
    code = torch.where(tied.sum(-1) > 1, (tied & even).long().argmax(-1),
                       tied.long().argmax(-1))
    code = torch.where(q > 6.0, torch.full_like(code, 7), code)
    sign = torch.signbit(b) & ~bad[..., None]
    byte = torch.where(bad, torch.full_like(e, 255), e + 127)
    return (code + 8 * sign.long()).to(torch.uint8).reshape(v.shape), byte.to(torch.uint8)


def mx_values(codes, byte):
    """float64 values of codes [..., K] with scale bytes [..., K/32]."""
    v = torch.cat([E2M1, -E2M1])[codes.long()]
    v = v.reshape(*codes.shape[:-1], codes.shape[-1] // 32, 32)
    s = torch.ldexp(torch.ones(byte.shape, dtype=torch.float64), byte.long() - 127)
    s = torch.where(byte == 255, torch.full_like(s, float("nan")), s)
    return (v * s[..., None]).reshape(codes.shape)


def mx_pack(codes, byte):
    """[R, K] codes and [R, K/32] bytes in the library's layout: [R, K/2], [K/128, R, 4]."""
    R, nb = byte.shape
    words = (nb + 3) // 4
    s = torch.zeros(R, words * 4, dtype=torch.uint8)
    s[:, :nb] = byte
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous(), \
        s.reshape(R, words, 4).permute(1, 0, 2).contiguous()


def mx_product(x, codes, byte, sizes, silu):
    """x float [M, K] quantised by rows, codes [E, N, K], byte [E, N, K/32]."""
    M, N = x.shape[0], codes.shape[1]
    out = torch.zeros(M, N // 2 if silu else N, dtype=torch.float64)
    row = 0
    for e, n in enumerate(sizes):
        y = mx_values(*mx_quantize(x[row:row + n])) @ mx_values(codes[e], byte[e]).T
        if silu:
            g, u = y[:, :N // 2], y[:, N // 2:]
            y = g / (1 + torch.exp(-g)) * u
        out[row:row + n] = y
        row += n
    return out


# -------------------------------------------------------------------- tolerances
def check_f32(got, ref, what=""):
    """Results of f32 sums. A sum here is a chain of at most 160 additions of exact or
    once-rounded terms joined by trees, a result a few operations more: about
    160 * 2^-24 = 1e-5 of the typical term sum, taken as the larger of the result and
    the results' rms."""
    g, r = got.detach().cpu().double(), ref.detach().cpu().double()
    assert g.shape == r.shape, (what, g.shape, r.shape)
    assert torch.isfinite(g).all(), f"{what}: non-finite"
    if r.numel() == 0:
        return
    rms = r.square().mean().sqrt()
    bad = (g - r).abs() > 1e-5 * torch.maximum(r.abs(), rms)
    assert not bad.any(), (what, int(bad.sum()), float((g - r).abs().max()), float(rms))


def check_rows(got, ref, what=""):
    """Results in their rows' type: f32 as check_f32; bf16 within one bf16 step of the
    64-bit value (half a step for the rounding, the f32 error below the rest), and for
    values far below the rms within the f32 error of the sums that made them."""
    if got.dtype == torch.float32:
        return check_f32(got, ref, what)
    g, r = got.detach().cpu().double(), ref.detach().cpu().double()
    assert g.shape == r.shape, (what, g.shape, r.shape)
    assert torch.isfinite(g).all(), f"{what}: non-finite"
    if r.numel() == 0:
        return
    step = torch.pow(2.0, torch.floor(torch.log2(r.abs().clamp_min(2.0 ** -126))) - 7)
    bad = (g - r).abs() > step + 1e-5 * r.square().mean().sqrt()
    assert not bad.any(), (what, int(bad.sum()), float((g - r).abs().max()))
