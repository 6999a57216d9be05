"""Plain 64-bit forms of the router, the balance loss and the AdamW step, on the CPU."""
import math

import numpy as np
import torch

INF = float("inf")


# ------------------------------------------------------------------------------ router
def scores(x, score):
    """64-bit scores and the tokens' shares of a [T, E] tensor; rows of -inf give zeros. The
    shares are taken on the scale of the row's largest score, as exact arithmetic has them."""
    if score == "softmax":
        s = torch.softmax(x, 1)
        dead = (x == -INF).all(1, keepdim=True)
        return torch.where(dead, torch.zeros_like(s), s), torch.where(dead, torch.zeros_like(s), s)
    log_s = -torch.nn.functional.softplus(-x)
    dead = (x == -INF).all(1, keepdim=True)
    p = torch.softmax(log_s, 1)
    return torch.sigmoid(x), torch.where(dead, torch.zeros_like(p), p)


def choose(x, k, score, bias):
    """ids [T, k] in 64 bits: largest first, ties to the lowest, -inf never."""
    c = x if bias is None else scores(x, score)[0] + bias
    c = torch.where(x == -INF, torch.full_like(c, -INF), c)
    ids = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :k]
    return torch.where(torch.gather(c, 1, ids) == -INF, torch.full_like(ids, -1), ids)


def weights(x, ids, score, normalize, scale):
    """f64 [T, k] for given ids (-1: 0); differentiable."""
    on = (ids >= 0) & (ids < x.shape[1])
    at = torch.where(on, ids, torch.zeros_like(ids)).long()
    if not normalize:
        s = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)
        return torch.where(on, scale * torch.gather(s, 1, at), torch.zeros(()).double())
    log_s = x if score == "softmax" else -torch.nn.functional.softplus(-x)
    z = torch.where(on, torch.gather(log_s, 1, at), torch.tensor(-1e300, dtype=torch.float64))
    return torch.where(on, scale * torch.softmax(z, 1), torch.zeros(()).double())


def sequences(T, offsets):
    """The sequence of each token, -1 outside."""
    seq = torch.full((T,), -1, dtype=torch.long)
    if offsets is None:
        return torch.zeros(T, dtype=torch.long)
    for b in range(len(offsets) - 1):
        seq[offsets[b]:offsets[b + 1]] = b
    return seq


def balance(x, ids, score, offsets):
    """(counts [B, E], loss [B], slope [B, E]) of given choices; the loss is differentiable."""
    T, E = x.shape
    B = 1 if offsets is None else len(offsets) - 1
    seq = sequences(T, offsets)
    if score == "softmax":
        p = torch.softmax(x, 1)
    else:
        p = torch.softmax(-torch.nn.functional.softplus(-x), 1)
    valid = (ids >= 0) & (ids < E)
    counts = torch.zeros(B, E, dtype=torch.int64)
    slope, loss = torch.zeros(B, E, dtype=torch.float64), []
    for b in range(B):
        rows = torch.nonzero((seq == b) & valid.any(1)).reshape(-1)
        counts[b] = torch.bincount(ids[rows][valid[rows]].long(), minlength=E)
        C, n = int(counts[b].sum()), len(rows)
        if C:
            slope[b] = E * counts[b].double() / (float(C) * n)
        live = (x[rows] != -INF).any(1)
        loss.append((slope[b] * p[rows][live].sum(0)).sum())
    return counts, torch.stack(loss), slope


# ------------------------------------------------------------------------------- AdamW
F = np.float32


def random_bits(n, which, step, seed, first=0):
    """The hash behind the 8-bit moments' rounding, from its description."""
    with np.errstate(over="ignore"):
        i = np.arange(first, first + n, dtype=np.uint64)
        key = np.uint32((seed + 0x6A09E667 * step + 0xBB67AE85 * which) & 0xFFFFFFFF)
        x = (i & np.uint64(0xFFFFFFFF)).astype(np.uint32) * np.uint32(0x9E3779B9)
        x = x + (i >> np.uint64(32)).astype(np.uint32) * np.uint32(0x3C6EF373) + key
        x = (x ^ (x >> np.uint32(16))) * np.uint32(0xBB67AE85)
        x = (x ^ (x >> np.uint32(15))) * np.uint32(0x6A09E667)
        return x ^ (x >> np.uint32(16))


E4M3 = np.array([(-1.0 if c & 128 else 1.0) *
                 ((c & 7) * 2.0 ** -9 if not c & 0x78 else
                  (1 + (c & 7) / 8) * 2.0 ** (((c >> 3) & 15) - 7)) for c in range(256)])
E4M3[0x7F] = E4M3[0xFF] = np.nan
MAGNITUDES = E4M3[:0x7F]                       # ascending


def decode(codes, scale):
    """f32 values of codes u8 [n]: one rounding of code * scale."""
    per = np.repeat(scale, 128)[:len(codes)]
    with np.errstate(invalid="ignore"):
        return E4M3[codes].astype(F) * per


def encode(x, random16, never_zero):
    """Codes and scales of f32 values by the description: the magnitude over the scale, cut to
    the 20 bits below the code's, goes up with the probability of what is cut (16 random bits,
    taken in the middle of their step), found here from the neighbouring codes' values."""
    n = len(x)
    blocks = -(-n // 128)
    pad = np.zeros(blocks * 128, F)
    pad[:n] = np.abs(x)
    scale = pad.reshape(blocks, 128).max(1) * F(1.0 / 448)
    scale[scale < F(2.0 ** -126)] = 0
    with np.errstate(divide="ignore"):
        inverse = np.where(scale > 0, F(1) / scale, F(0))
    per = np.repeat(inverse, 128)[:n]
    y = np.abs(x) * per                                      # f32
    # what the format's grid below 2^-149 * 2^120 cannot hold is rounded away first
    y = np.rint(y.astype(np.float64) * 2.0 ** 29) * 2.0 ** -29 * (y < 2.0 ** -6) + \
        y.astype(np.float64) * (y >= 2.0 ** -6)
    low = np.clip(np.searchsorted(MAGNITUDES, y, side="right") - 1, 0, 0x7E)
    gap = np.where(low < 0x7E, MAGNITUDES[np.minimum(low + 1, 0x7E)] - MAGNITUDES[low], 32.0)
    part = (y - MAGNITUDES[low]) / gap                       # [0, 1)
    up = part * 2.0 ** 20 + random16.astype(np.float64) * 16 + 8 >= 2.0 ** 20
    code = np.minimum(low + up, 0x7E)
    if never_zero:
        code = np.where((code == 0) & (x > 0) & (np.repeat(scale, 128)[:n] > 0), 1, code)
    else:
        code = code | np.where(np.signbit(x), 128, 0)
    return code.astype(np.uint8), scale


def rates(step, lr, beta1, beta2):
    return F(lr / (1.0 - math.pow(beta1, step))), F(1.0 / math.sqrt(1.0 - math.pow(beta2, step)))


def adamw(p, g, m, v, step, lr, beta1, beta2, eps, decay, grad_scale=None):
    """One step in f32 with every operation rounded by itself: (p, m, v, sqrt(v))."""
    rate, root = rates(step, lr, beta1, beta2)
    if grad_scale is not None:
        g = g * F(grad_scale)
    m = m * F(beta1) + g * F(1.0 - beta1)
    v = v * F(beta2) + (g * F(1.0 - beta2)) * g
    r = np.sqrt(v)
    p = p * F(1.0 - lr * decay) - (m / (r * root + F(eps))) * rate
    return p, m, v, r


def adamw_64(p, g, m, v, step, lr, beta1, beta2, eps, decay, grad_scale=None):
    """The formula in 64 bits, and the magnitudes that its roundings are relative to."""
    p, g, m, v = (np.asarray(t, np.float64) for t in (p, g, m, v))
    if grad_scale is not None:
        g = g * grad_scale
    m1 = beta1 * m + (1 - beta1) * g
    v1 = beta2 * v + (1 - beta2) * g * g
    den = np.sqrt(v1) / math.sqrt(1 - beta2 ** step) + eps
    size = np.abs(beta1 * m) + np.abs((1 - beta1) * g)
    update = lr / (1 - beta1 ** step) / den
    return (p * (1 - lr * decay) - update * m1, m1, v1,
            np.abs(p) + update * size, size)
