"""The router's choice, the balance loss and their gradient against 64-bit forms, on the GPU."""
import math

import pytest
import torch

import train_reference as ref
from fp8_moe_routed_gb300 import binding as fb

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
INF = float("inf")
U = 2.0 ** -24                        # half a step of f32


def draw(T, E, seed, dtype, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, E, generator=g) * spread + torch.randn(E, generator=g) * 0.5
    return x.to(dtype)


def cut(T, B, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    at = sorted(torch.randint(0, T - pad + 1, (B - 1,), generator=g).tolist())
    return [0] + at + [T - pad]


def offsets_cuda(offsets):
    return None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")


def width(x):
    """The largest distance of a row's finite logits: an exponential's argument is rounded to
    half a step of it, which its value has as a relative error."""
    f = x[torch.isfinite(x)]
    return float(f.max() - f.min()) if f.numel() else 0.0


def check_forward(x, k, score, bias, normalize, scale, offsets, balance=True):
    """A whole forward against 64 bits; returns what the gradient takes."""
    T, E = x.shape
    dev = x.cuda()
    fb.read_status()
    got = fb.router_fwd(dev, k, score=score, bias=None if bias is None else bias.cuda(),
                        normalize=normalize, weight_scale=scale, balance=balance,
                        seq_offsets=offsets_cuda(offsets))
    assert fb.read_status() == 0
    ids, w = got[0].cpu(), got[1].double().cpu()
    x64 = x.double()
    want = ref.choose(x64, k, score, None if bias is None else bias.double())
    seq = ref.sequences(T, offsets)
    want[seq < 0] = -1
    assert torch.equal(ids.long(), want)
    want_w = ref.weights(x64, want, score, normalize, scale)
    # a score: an exponential (2 units, its argument's rounding), a sum, a reciprocal, a product;
    # the sum of the chosen or of the row: at most 37 additions of positive terms; a quotient,
    # the scale: below 2 (8 + width) + 40 units of 2^-24
    tol = (60 + 2 * width(x.float())) * U
    assert ((w - want_w).abs() <= tol * want_w.abs() + 1e-37).all(), float((w - want_w).abs().max())
    if balance:
        check_balance(x, want, score, offsets, *got[2:])
    return got


def check_balance(x, ids, score, offsets, counts, loss, slope):
    T = x.shape[0]
    want_counts, want_loss, want_slope = ref.balance(x.double(), ids, score, offsets)
    assert torch.equal(counts.cpu().long(), want_counts)
    # count, E, C and n as f32, a product and two quotients
    assert ((slope.double().cpu() - want_slope).abs() <= 8 * U * want_slope).all()
    # positive terms: a share as above, and at most T / 8 + 200 additions on the way of any of them
    tol = (60 + 2 * width(x.float()) + T / 8 + 200) * U
    assert ((loss.double().cpu() - want_loss).abs() <= tol * want_loss + 1e-37).all()


# T, E, k, type, score, bias, normalize, sequences (0: none given), padding
FORWARD = [
    (1, 1, 1, F32, "softmax", False, True, 0, 0), (1, 256, 8, F32, "sigmoid", True, True, 0, 0),
    (1, 1024, 32, BF16, "softmax", False, False, 0, 0), (7, 2, 2, BF16, "sigmoid", False, True, 3, 0),
    (33, 8, 8, F32, "softmax", True, False, 2, 5), (100, 17, 4, BF16, "softmax", False, True, 5, 10),
    (129, 32, 3, F32, "sigmoid", True, False, 1, 0), (257, 61, 6, F32, "softmax", False, False, 9, 1),
    (64, 64, 8, BF16, "softmax", True, True, 64, 0), (1000, 65, 8, F32, "sigmoid", False, True, 4, 0),
    (513, 100, 5, BF16, "sigmoid", True, True, 2, 100), (1001, 128, 8, BF16, "softmax", False, False, 1, 0),
    (2500, 160, 8, F32, "sigmoid", True, True, 3, 77), (777, 254, 7, BF16, "sigmoid", False, False, 20, 0),
    (4099, 256, 8, F32, "sigmoid", True, True, 5, 3), (300, 384, 8, F32, "softmax", False, True, 2, 0),
    (301, 511, 9, BF16, "softmax", False, True, 2, 0), (600, 512, 8, F32, "sigmoid", True, False, 0, 0),
    (99, 1000, 10, F32, "softmax", True, True, 4, 9), (64, 1023, 32, F32, "sigmoid", False, True, 1, 0),
    (5000, 1024, 2, BF16, "softmax", False, False, 3, 0),
    # from 16384 tokens on, at most 128 experts, at most 8 chosen: eight lanes a token
    (16384, 8, 8, F32, "softmax", False, True, 3, 0), (16385, 31, 3, F32, "sigmoid", True, True, 7, 5),
    (17001, 61, 6, BF16, "sigmoid", False, False, 0, 0), (16900, 128, 8, BF16, "softmax", False, False, 5, 77),
    (16399, 160, 5, F32, "softmax", True, False, 300, 0), (20011, 256, 8, F32, "sigmoid", True, True, 4, 11),
    (16500, 255, 1, BF16, "softmax", False, True, 1, 0), (16390, 257, 8, F32, "sigmoid", False, True, 2, 0),
    (16401, 64, 9, BF16, "softmax", False, True, 2, 0), (16390, 100, 8, F32, "sigmoid", True, True, 3, 9),
    (16500, 127, 7, F32, "softmax", True, True, 2, 0), (16385, 128, 8, F32, "sigmoid", False, False, 40, 0),
]


@pytest.mark.parametrize("T,E,k,dtype,score,biased,normalize,B,pad", FORWARD)
def test_choice_weights_and_balance(T, E, k, dtype, score, biased, normalize, B, pad):
    x = draw(T, E, T + E, dtype)
    bias = torch.randn(E, generator=torch.Generator().manual_seed(E)) * 0.05 if biased else None
    offsets = cut(T, B, T, pad) if B else None
    first = check_forward(x, k, score, bias, normalize, 2.5, offsets)
    # without the loss, and once more: the same bits
    b = None if bias is None else bias.cuda()
    plain = fb.router_fwd(x.cuda(), k, score=score, bias=b, normalize=normalize, weight_scale=2.5,
                          seq_offsets=offsets_cuda(offsets))
    again = fb.router_fwd(x.cuda(), k, score=score, bias=b, normalize=normalize, weight_scale=2.5,
                          seq_offsets=offsets_cuda(offsets), balance=True)
    assert torch.equal(plain[0], first[0]) and torch.equal(plain[1], first[1])
    assert plain[2:] == (None, None, None)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    # the loss of these choices, handed in
    counts, loss, slope = fb.balance_fwd(x.cuda(), first[0], score=score,
                                         seq_offsets=offsets_cuda(offsets))
    assert torch.equal(counts, first[2]) and torch.equal(slope, first[4])
    check_balance(x, first[0].cpu().long(), score, offsets, counts, loss, slope)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E", [8, 61, 256, 1024])
def test_ties_go_to_the_lowest_expert(score, biased, E):
    """Equal logits everywhere; few distinct values; equal ones next to the border."""
    k = min(8, E)
    bias = torch.zeros(E) if biased else None
    for x in (torch.zeros(9, E), torch.full((3, E), -4.25), draw(65, E, 3, F32).round(),
              torch.where(torch.arange(E) % 3 == 1, 1.0, -0.0).repeat(5, 1)):
        check_forward(x, k, score, bias, True, 1.0, None)


@pytest.mark.parametrize("biased", [False, True])
def test_values_that_f32_hardly_tells_apart(biased):
    """Neighbouring f32 logits; sigmoids that agree in f32; scores that differ by less than their
    error: the order is that of the exact values."""
    E, k = 64, 6
    base = torch.nextafter(torch.tensor(2.0), torch.tensor(3.0))
    step = torch.arange(E).float() * 2.0 ** -22
    g = torch.Generator().manual_seed(1)
    rows = [(2.0 + step)[torch.randperm(E, generator=g)] for _ in range(20)]
    rows += [(20.0 + torch.arange(E) * 0.01)[torch.randperm(E, generator=g)] for _ in range(20)]
    rows += [torch.where(torch.arange(E) < 40, base, torch.tensor(2.0))]
    x = torch.stack(rows)
    bias = torch.zeros(E) if biased else None
    check_forward(x, k, "sigmoid", bias, True, 1.0, None)
    if biased:
        # biases that undo the scores up to a rounding of f32
        s = torch.sigmoid(x[0].double())
        check_forward(x[:1].repeat(3, 1), k, "sigmoid", (1.0 - s).float(), True, 1.0, None)
        check_forward(x, k, "softmax", (torch.randn(E, generator=g) * 2.0 ** -24), True, 1.0, None)


def test_masked_experts_and_rows():
    """Experts at -inf are not chosen: fewer than topk, or none at all, which also leaves the
    token out of the balance sums."""
    x = draw(40, 33, 5, F32)
    x[0, 3:] = -INF
    x[1] = -INF
    x[2, :32] = -INF
    x[7::5, ::2] = -INF
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.randn(33)):
            ids, w, counts, loss, slope = check_forward(x, 8, score, bias, True, 2.0, None)
            assert ids[1].tolist() == [-1] * 8 and w[1].tolist() == [0.0] * 8
            assert sorted(ids[0].tolist())[:5] == [-1] * 5
            dl = fb.router_bwd(torch.randn(40, 8, device="cuda"), x.cuda(), ids, score=score,
                               dloss=torch.ones(1, device="cuda"), slope=slope)
            assert torch.isfinite(dl).all() and (dl[1] == 0).all()
            assert (dl.cpu()[x == -INF] == 0).all()
    # an expert whose bias is -inf is out, too
    bias = torch.zeros(33)
    bias[5] = -INF
    ids = fb.router_fwd(x.cuda(), 8, score="sigmoid", bias=bias.cuda())[0]
    assert not (ids == 5).any()


@pytest.mark.parametrize("shift", [-300.0, -60.0, 60.0, 300.0])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_far_logits(shift, dtype):
    """Scores that all round to zero or to one in f32 have weights, shares and gradients."""
    x = (draw(20, 40, 2, F32) + shift).to(dtype)
    _, _, _, _, slope = check_forward(x, 4, "sigmoid", None, True, 1.0, None)
    check_forward(x, 4, "softmax", None, False, 1.0, None)
    check_backward(x, 4, "sigmoid", True, 1.0, None)
    check_backward(x, 4, "softmax", False, 1.0, None)


def test_nan_spoils_its_token_alone():
    x = draw(9, 48, 8, F32)
    x[4, 7] = float("nan")
    x[6] = float("nan")
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.zeros(48)):
            ids, w, *_ = fb.router_fwd(x.cuda(), 5, score=score,
                                       bias=None if bias is None else bias.cuda())
            clean = [i for i in range(9) if i not in (4, 6)]
            want = ref.choose(x[clean].double(), 5, score, None)
            assert torch.equal(ids.cpu()[clean].long(), want) and torch.isfinite(w[clean]).all()
            assert torch.isnan(w[4]).any() and torch.isnan(w[6]).all()
            for t in (4, 6):                   # still experts of the range, each once
                assert len(set(ids[t].tolist())) == 5 and 0 <= min(ids[t].tolist())
                assert max(ids[t].tolist()) < 48


def test_no_tokens_and_empty_sequences():
    x = torch.empty(0, 24, device="cuda")
    ids, w, counts, loss, slope = fb.router_fwd(x, 3, balance=True)
    assert ids.shape == w.shape == (0, 3)
    assert not counts.any() and loss.tolist() == [0.0] and not slope.any()
    off = torch.tensor([0, 0, 0], dtype=torch.int32, device="cuda")
    counts, loss, slope = fb.balance_fwd(x, ids, seq_offsets=off)
    assert counts.shape == (2, 24) and loss.tolist() == [0.0, 0.0] and not slope.any()
    assert fb.router_bwd(w, x, ids).shape == (0, 24)
    check_forward(draw(50, 24, 1, F32), 3, "softmax", None, True, 1.0, [0, 0, 20, 20, 20, 50, 50])
    check_forward(draw(50, 24, 1, F32), 3, "softmax", None, True, 1.0, [10, 10, 11, 45])
    check_forward(draw(50, 24, 1, F32), 3, "softmax", None, True, 1.0, [50, 50])


def test_bad_offsets_are_reported():
    x = draw(50, 24, 1, F32).cuda()
    for bad in ([0, 60], [-5, 50], [0, 30, 20, 50], [2 ** 31 - 1, -2 ** 31], [70, 80, 90]):
        fb.read_status()
        ids, *_ = fb.router_fwd(x, 3, balance=True, seq_offsets=offsets_cuda(bad))
        assert fb.read_status() == fb.STATUS_BAD_OFFSETS
        assert int(ids.max()) < 24 and int(ids.min()) >= -1


def test_given_choices():
    """Ids outside the range are no choices; one that occurs twice counts twice."""
    T, E = 70, 20
    x = draw(T, E, 4, BF16)
    ids = torch.randint(0, E, (T, 4), generator=torch.Generator().manual_seed(2)).to(torch.int32)
    ids[3] = -1
    ids[5, 1:] = -7
    ids[6] = ids[6, 0]
    ids[8, 2] = ids[8, 3] = ids[8, 0]
    fb.read_status()
    out = fb.balance_fwd(x.cuda(), ids.cuda(), score="sigmoid")
    assert fb.read_status() == 0
    check_balance(x, ids.long(), "sigmoid", None, *out)
    for normalize in (True, False):
        for score in ("softmax", "sigmoid"):
            check_backward(x, 4, score, normalize, 1.5, None, ids=ids)
    ids[9, 0] = E
    ids[10, 3] = 2 ** 31 - 1
    out = fb.balance_fwd(x.cuda(), ids.cuda(), score="sigmoid")
    assert fb.read_status() == fb.STATUS_BAD_EXPERT
    check_balance(x, ids.long(), "sigmoid", None, *out)
    check_backward(x, 4, "softmax", True, 1.5, None, ids=ids)
    assert fb.read_status() == fb.STATUS_BAD_EXPERT


def reference_total(x, ids, score, normalize, scale, offsets, dw, dloss, slope):
    """What the gradient is of: weights with dw, shares with the given slope."""
    E = x.shape[1]
    seq = ref.sequences(x.shape[0], offsets)
    valid = ((ids >= 0) & (ids < E)).any(1) & (seq >= 0) & (x != -INF).any(1)
    rows = torch.nonzero(valid).reshape(-1)
    total = torch.zeros((), dtype=torch.float64)
    if dw is not None:
        total = total + (ref.weights(x[rows], ids[rows], score, normalize, scale) * dw[rows]).sum()
    if dloss is not None:
        z = x[rows] if score == "softmax" else -torch.nn.functional.softplus(-x[rows])
        total = total + (torch.softmax(z, 1) * (dloss[:, None] * slope)[seq[rows]]).sum()
    return total


def check_backward(x, k, score, normalize, scale, offsets, ids=None, parts="both"):
    T, E = x.shape
    B = 1 if offsets is None else len(offsets) - 1
    g = torch.Generator().manual_seed(T + k)
    dev, off = x.cuda(), offsets_cuda(offsets)
    if ids is None:
        ids = fb.router_fwd(dev, k, score=score, normalize=normalize, seq_offsets=off)[0].cpu()
    dw = torch.randn(T, k, generator=g) if parts != "loss" else None
    dloss = torch.rand(B, generator=g) * T if parts != "weights" else None
    slope = torch.rand(B, E, generator=g) * 2 / T if parts != "weights" else None
    to = lambda t: None if t is None else t.cuda()  # noqa: E731
    got = fb.router_bwd(to(dw), dev, ids.cuda(), score=score, normalize=normalize,
                        weight_scale=scale, dloss=to(dloss), slope=to(slope), seq_offsets=off)
    assert got.dtype == x.dtype
    d64 = [None if t is None else t.double() for t in (dw, dloss, slope)]
    x64 = x.double().requires_grad_()
    total = reference_total(x64, ids.long(), score, normalize, scale, offsets, *d64)
    want = torch.autograd.grad(total, x64)[0] if total.requires_grad else torch.zeros_like(x64)
    want = torch.nan_to_num(want)
    # every term is a product of factors with the forward's errors, in sums whose roundings are
    # relative to the terms' magnitudes: q (w (|dw| + sum |dw| w) + p (|D| + sum |D| p))
    x64 = x64.detach()
    q = torch.sigmoid(-x64) if score == "sigmoid" else torch.ones_like(x64)
    p = ref.scores(x64, score)[1]
    D = torch.zeros_like(x64)
    if dloss is not None:
        D = (d64[1][:, None] * d64[2])[ref.sequences(T, offsets).clamp(min=0)].abs()
    size = torch.zeros_like(x64)
    if dw is not None:
        on = (ids >= 0) & (ids < E)
        at = torch.where(on, ids, torch.zeros_like(ids)).long()
        a = torch.where(on, (scale * d64[0]).abs(), torch.zeros(()).double())
        if normalize:
            w = ref.weights(x64, ids.long(), score, True, 1.0)
            size.scatter_add_(1, at, w * (a + (a * w).sum(1, keepdim=True)))
        elif score == "softmax":
            D = D.scatter_add(1, at, a)
        else:
            size.scatter_add_(1, at, a * torch.gather(torch.sigmoid(x64), 1, at))
    size = q * (size + p * (D + (D * p).sum(1, keepdim=True)))
    tol = (120 + 4 * width(x.float())) * U * size + torch.finfo(x.dtype).eps / 2 * want.abs()
    err = (got.double().cpu() - want).abs()
    assert (err <= tol + 1e-37).all(), float((err / (tol + 1e-37)).max())
    return got


@pytest.mark.parametrize("T,E,k,dtype,score,biased,normalize,B,pad", FORWARD)
def test_gradient(T, E, k, dtype, score, biased, normalize, B, pad):
    x = draw(T, E, T + E, dtype)
    offsets = cut(T, B, T, pad) if B else None
    both = check_backward(x, k, score, normalize, 2.5, offsets)
    check_backward(x, k, score, normalize, 2.5, offsets, parts="weights")
    check_backward(x, k, score, normalize, 2.5, offsets, parts="loss")
    if offsets is not None and offsets[-1] < T:
        assert (both[offsets[-1]:] == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_against_differences(score, normalize):
    """Central differences of the 64-bit forward at the call's own counts (h^2 = 1e-8 of the third
    derivative, which is of the size of the gradient, and 1e-16 / h)."""
    T, E, k, h = 6, 10, 3, 1e-4
    offsets = [0, 2, 6]
    x = draw(T, E, 11, F32)
    ids, _, _, _, slope = fb.router_fwd(x.cuda(), k, score=score, normalize=normalize, balance=True,
                                        seq_offsets=offsets_cuda(offsets))
    dw, dloss = torch.randn(T, k), torch.tensor([3.0, 5.0])
    got = fb.router_bwd(dw.cuda(), x.cuda(), ids, score=score, normalize=normalize,
                        dloss=dloss.cuda(), slope=slope, seq_offsets=offsets_cuda(offsets)).cpu()
    args = (ids.cpu().long(), score, normalize, 1.0, offsets, dw.double(), dloss.double(),
            slope.cpu().double())
    for t in range(T):
        for e in range(E):
            up, down = x.double(), x.double()
            up[t, e] += h
            down[t, e] -= h
            d = (reference_total(up, *args) - reference_total(down, *args)) / (2 * h)
            assert abs(float(d) - float(got[t, e])) <= 2e-6


def test_many_tokens_are_chosen_as_few_are():
    """The rows on which a choice can go wrong, few and repeated in a large batch, which other
    kernels take: the same experts, weights and gradients to a few roundings."""
    E, k = 96, 6
    g = torch.Generator().manual_seed(5)
    rows = [torch.zeros(4, E), draw(60, E, 3, F32).round(), draw(60, E, 4, F32), draw(30, E, 5, BF16).float(),
            (2.0 + torch.arange(E) * 2.0 ** -22)[torch.randperm(E, generator=g)][None],
            (20.0 + torch.arange(E) * 0.01)[torch.randperm(E, generator=g)][None],
            draw(20, E, 6, F32) - 200, draw(20, E, 7, F32) * 1e-5]
    x = torch.cat(rows)
    x[9, 2:] = -INF
    x[10] = -INF
    x[11, 3] = float("nan")
    x[12, ::3] = -INF
    T = x.shape[0]
    many = -(-16400 // T)
    for dtype in (F32, BF16):
        few = x.to(dtype).cuda()
        lots = few.repeat(many, 1)
        for score in ("softmax", "sigmoid"):
            for bias in (None, torch.zeros(E).cuda(), (torch.randn(E, generator=g) * 0.05).cuda()):
                for normalize in (True, False):
                    a = fb.router_fwd(few, k, score=score, bias=bias, normalize=normalize)
                    b = fb.router_fwd(lots, k, score=score, bias=bias, normalize=normalize)
                    sound = ~torch.isnan(x).any(1)
                    ids = b[0].view(many, T, k)
                    assert torch.equal(ids[:, sound], a[0][sound].expand(many, -1, -1))
                    torch.testing.assert_close(b[1].view(many, T, k), a[1].expand(many, -1, -1),
                                               rtol=4e-6, atol=1e-37, equal_nan=True)
                    if bias is not None:
                        continue
                    dw = torch.randn(T, k, generator=g).cuda()
                    slope = torch.rand(1, E, generator=g).cuda()
                    dl = torch.ones(1, device="cuda")
                    d = fb.router_bwd(dw, few, a[0], score=score, normalize=normalize, dloss=dl,
                                      slope=slope)
                    e = fb.router_bwd(dw.repeat(many, 1), lots, a[0].repeat(many, 1), score=score,
                                      normalize=normalize, dloss=dl, slope=slope)
                    # sums in another order: of 96 terms, relative to the row's largest
                    top = d.float().abs().amax(1, keepdim=True)
                    tol = 200 * U * top + torch.finfo(dtype).eps * d.float().abs()
                    off = (e.view(many, T, E).float() - d.float()).abs()
                    assert (off <= tol)[:, sound].all()


def test_captured_and_on_streams():
    """A captured forward and backward follow their inputs when they are replayed; two streams
    with workspaces of their own do not meet."""
    T, E, k = 300, 96, 4
    xs = [draw(T, E, s, F32).cuda() for s in range(4)]
    want = [fb.router_fwd(x, k, score="sigmoid", balance=True) for x in xs]
    dw, dl = torch.randn(T, k, device="cuda"), torch.ones(1, device="cuda")
    want_d = [fb.router_bwd(dw, x, w[0], score="sigmoid", dloss=dl, slope=w[4])
              for x, w in zip(xs, want)]
    x = xs[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fb.router_fwd(x, k, score="sigmoid", balance=True)
        d = fb.router_bwd(dw, x, out[0], score="sigmoid", dloss=dl, slope=out[4])
    for i in (2, 1, 3):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i])) and torch.equal(d, want_d[i])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(4):
        with torch.cuda.stream(streams[i % 2]):
            got.append(fb.router_fwd(xs[i], k, score="sigmoid", balance=True))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_rows_past_two_to_the_31_values():
    """Logits of more than 2^31 values: the last rows are as they are alone."""
    T, E = 2 ** 22 + 40, 512
    x = torch.zeros(T, E, dtype=BF16, device="cuda")
    tail = draw(40, E, 9, BF16).cuda()
    x[-40:] = tail
    ids, w, counts, loss, slope = fb.router_fwd(x, 4, balance=True)
    alone = fb.router_fwd(tail, 4)
    assert torch.equal(ids[-40:], alone[0]) and torch.equal(w[-40:], alone[1])
    assert int(counts.sum()) == 4 * T and int(counts[0, 0]) >= T - 40
    d = fb.router_bwd(w, x, ids, dloss=torch.zeros(1, device="cuda"), slope=slope)
    alone_d = fb.router_bwd(w[-40:].contiguous(), tail, alone[0])
    assert torch.equal(d[-40:], alone_d)
