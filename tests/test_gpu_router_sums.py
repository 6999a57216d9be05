"""The balance loss's sums: that no token is lost at the ends of chunks, groups and sequences, and
the range of sizes in which the kernel of eight lanes a token begins (4096 tokens)."""
import pytest
import torch

import train_reference as ref
from fp8_moe_routed_gb300 import binding as fb
from test_gpu_router import BF16, F32, U, check_backward, check_forward, cut, draw, offsets_cuda, width

pytestmark = pytest.mark.gpu


def up(a, b):
    return -(-a // b)


def additions(T, E, k, biased, B):
    """How many additions a share passes on its way into the loss: its lane's tokens, lanes and
    warps of a CTA, the parts that a thread joins, the threads of a column, the CTAs of a
    sequence, and the sum over the experts."""
    groups = T >= 4096 and E <= 128 and k <= 8 and not biased
    if groups:
        chunk = min(256, max(32, up(T // 304, 32) * 32))
        inner = chunk // 32 + 2 + 8
    else:
        chunk = min(128, max(8, up(T // 608, 8) * 8))
        inner = chunk // 8 + 8
    columns = 32
    while columns < E:
        columns *= 2
    parts, threads = up(T, chunk), 1024 // columns
    ctas = 8 if parts // B > 64 else 1
    return inner + up(parts + 1, threads * ctas) + threads + ctas + 10


def check_loss(x, k, biased, ids, score, offsets, counts, loss, slope):
    """A share is within 60 + 2 width units of 2^-24 (an exponential, its argument's rounding, a
    sum of at most 37 terms, a reciprocal), its slope within 8; then a product and the sums."""
    T, E = x.shape
    B = 1 if offsets is None else len(offsets) - 1
    want = ref.balance(x.double(), ids, score, offsets)
    assert torch.equal(counts.cpu().long(), want[0])
    assert ((slope.double().cpu() - want[2]).abs() <= 8 * U * want[2]).all()
    tol = (60 + 2 * width(x.float()) + 9 + additions(T, E, k, biased, B)) * U
    off = (loss.double().cpu() - want[1]).abs() / want[1].clamp(min=1e-30)
    assert (off <= tol).all(), (float(off.max()), tol)
    return want[1]


# tokens, experts, sequences: the kernel of eight lanes from its smallest chunks on with every
# remainder by four and by chunks, and the kernel of a warp
TAILS = [(4096, 128, 1), (4097, 64, 3), (4098, 32, 2), (4099, 61, 1), (4127, 128, 5), (4129, 8, 40),
         (10003, 100, 7), (16385, 128, 1), (17001, 31, 9), (30050, 128, 2),
         (1, 8, 1), (9, 256, 1), (1001, 300, 3), (4095, 128, 4), (5003, 512, 2)]


@pytest.mark.parametrize("T,E,B", TAILS)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_tokens_at_the_ends_count(T, E, B, dtype, score):
    """Every token chose expert 1, but only the first and the last three of a sequence have their
    share there: each of these is a quarter of the sequence's loss or more."""
    offsets = None if B == 1 else cut(T, B, T, T // 50)
    spans = list(zip(offsets, offsets[1:])) if offsets else [(0, T)]
    ends = sorted({t for a, b in spans for t in [a, *range(max(a, b - 3), b)] if a <= t < b})
    x = torch.full((T, E), -20.0)
    x[:, 0] = 10.0
    x[ends, 0], x[ends, 1] = -20.0, 10.0
    x = x.to(dtype)
    ids = torch.full((T, 1), 1, dtype=torch.int32)
    fb.read_status()
    got = fb.balance_fwd(x.cuda(), ids.cuda(), score=score, seq_offsets=offsets_cuda(offsets))
    assert fb.read_status() == 0
    want = check_loss(x, 1, False, ids.long(), score, offsets, *got)
    # the loss is made of the ends: E / n for each of a sequence's
    for (a, b), loss in zip(spans, want.tolist()):
        mine = sum(a <= t < b for t in ends)
        assert a == b or abs(loss * (b - a) / E - mine) < 0.01


SIZES = [(4095, 128, 8, F32, "softmax", True, 3, 0), (4096, 128, 8, BF16, "softmax", False, 0, 0),
         (4096, 8, 2, F32, "sigmoid", True, 5, 100), (4097, 64, 8, F32, "softmax", True, 1, 0),
         (4097, 61, 5, BF16, "sigmoid", True, 4, 7), (4111, 17, 1, F32, "softmax", False, 60, 1),
         (8191, 100, 7, BF16, "softmax", True, 2, 0), (9001, 128, 8, F32, "sigmoid", False, 17, 33),
         (9728, 32, 3, BF16, "sigmoid", True, 0, 0), (11999, 127, 8, F32, "softmax", True, 6, 500)]


@pytest.mark.parametrize("T,E,k,dtype,score,normalize,B,pad", SIZES)
def test_where_eight_lanes_a_token_begin(T, E, k, dtype, score, normalize, B, pad):
    """Choice, weights, balance loss and gradient on both sides of the limit and in its smallest
    chunks, with the loss to within its own roundings: a lost token is 1 / T of it, ten times that."""
    x = draw(T, E, T + E, dtype)
    offsets = cut(T, B, T, pad) if B else None
    got = check_forward(x, k, score, None, normalize, 2.5, offsets)
    check_loss(x, k, False, got[0].cpu().long(), score, offsets, *got[2:])
    check_backward(x, k, score, normalize, 2.5, offsets)


@pytest.mark.parametrize("T,E,k,score,biased", [
    (65536, 128, 8, "softmax", False), (16390, 100, 8, "sigmoid", True),
    (20011, 256, 8, "sigmoid", True), (4099, 256, 8, "sigmoid", True), (5000, 1024, 2, "softmax", False)])
def test_large_batches_lose_no_token(T, E, k, score, biased):
    x = draw(T, E, T, F32, spread=1.0)
    bias = torch.randn(E, generator=torch.Generator().manual_seed(E)) * 0.05 if biased else None
    got = fb.router_fwd(x.cuda(), k, score=score, bias=None if bias is None else bias.cuda(),
                        balance=True)
    check_loss(x, k, biased, got[0].cpu().long(), score, None, *got[2:])
