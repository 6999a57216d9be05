"""The norms' gate behind a sigmoid, over logits where it or one minus it vanishes, on the
GPU against 64-bit values."""
import pytest
import torch

from fp8_moe_routed_gb300 import binding as fb

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32

# exp(-|z|) from one down to f32's smallest normal values
LOGITS = [0.0, 0.1, 1.0, 3.0, 5.0, 8.0, 10.0, 12.0, 14.0, 15.5, 17.0, 20.0, 30.0, 45.0, 60.0, 80.0]
H, B = 128, 0.7
KINDS = [(k, t) for t in (F32, BF16) for k in ("token", "channel", "full")]


def make(kind, dtype):
    """Inputs of one sign, so that no sum cancels, and in 64 bits: the logit of every element,
    the normalised y and t = exp(-|z|)."""
    z1 = torch.tensor(LOGITS + [-z for z in LOGITS])
    T = z1.numel() if kind == "token" else 5
    gate = z1 if kind == "token" else z1.repeat(H // z1.numel())
    if kind == "full":
        gate = gate.expand(T, H).to(dtype).contiguous()
    z = (gate[:, None] if kind == "token" else gate).expand(T, H).double()
    g = torch.Generator().manual_seed(2)
    y, dr = ((1 + torch.rand(T, H, generator=g)).to(dtype) for _ in range(2))
    w = 1 + torch.rand(H, generator=g)
    yh = y.double() * y.double().square().mean(1, keepdim=True).rsqrt()
    kw = dict(gate=gate.cuda(), gate_kind=kind, sigmoid=True, branch_scale=B)
    return y, dr, w, yh, z, torch.exp(-z.abs()), kw


def worst(have, want):
    return float(((have.cpu().double() - want).abs() / want.abs()).max())


@pytest.mark.parametrize("kind,dtype", KINDS)
def test_value(kind, dtype):
    """r = b g w yh with x = 0. In steps of 2^-24: the sigmoid 11 (an exponential within 7, an
    addition, a reciprocal within 2, a product), rstd 13 (half the error of a sum of 128
    squares in chains of 8 and trees of 5, a reciprocal root of two units), the other products
    5: 29, or 1.7e-6; 2e-6 is asked. bf16: one of its steps, half of it the rounding."""
    y, _, w, yh, z, t, kw = make(kind, dtype)
    g = torch.where(z >= 0, 1 / (1 + t), t / (1 + t))
    r = fb.norm_fwd(torch.zeros_like(y).cuda(), y.cuda(), w.cuda(), None, eps=0.0, **kw)[0]
    off = worst(r, B * g * w.double() * yh)
    assert off <= (2e-6 if dtype == F32 else 2.0 ** -8), off


def ends():
    """Logits of one row each: open, closed, NaN, the last ones above zero, a half."""
    z = torch.tensor([float("inf"), float("-inf"), 1e30, -1e30, float("nan"), -87.7, -104.0, 0.0])
    return z, z[:, None].expand(8, H).contiguous()


@pytest.mark.parametrize("kind", ["token", "full"])
def test_value_at_the_ends(kind):
    """Huge logits open or close the gate, NaN stays alone, small gates are not cut to zero."""
    z, full = ends()
    x, y, w = torch.zeros(8, H), torch.ones(8, H), torch.ones(H)
    r = fb.norm_fwd(x.cuda(), y.cuda(), w.cuda(), None, gate=(full if kind == "full" else z).cuda(),
                    gate_kind=kind, sigmoid=True, eps=0.0)[0].cpu()
    assert (r[0] == 1).all() and (r[1] == 0).all() and (r[2] == 1).all() and (r[3] == 0).all()
    assert torch.isnan(r[4]).all() and (r[7] == 0.5).all()
    assert ((r[5] > 8e-39) & (r[5] < 9e-39)).all() and (r[6] < 1e-44).all()


@pytest.mark.parametrize("kind,dtype", KINDS)
def test_slope(kind, dtype):
    """dgate = b dr w yh g (1 - g), summed over what shares a logit. The steps of test_value
    with 3 more for the slope's second factor, and up to 16 for the sum: 48, or 2.9e-6; 3e-6
    is asked.
    bf16 for a gate per element alone, the other gates and their gradients are f32."""
    y, dr, w, yh, z, t, kw = make(kind, dtype)
    rp = fb.norm_fwd(torch.zeros_like(y).cuda(), y.cuda(), w.cuda(), None, eps=0.0, **kw)[2]
    dgate = fb.norm_bwd(dr.cuda(), None, None, y.cuda(), w.cuda(), None, rp, None, **kw)[4]
    want = B * dr.double() * w.double() * yh * t / (1 + t) ** 2
    want = {"token": want.sum(1), "channel": want.sum(0), "full": want}[kind]
    off = worst(dgate, want)
    assert off <= (2.0 ** -8 if dgate.dtype == BF16 else 3e-6), off


@pytest.mark.parametrize("kind", ["token", "full"])
def test_slope_at_the_ends(kind):
    z, full = ends()
    dr, y, w = torch.ones(8, H), torch.ones(8, H), torch.ones(H)
    gate = (full if kind == "full" else z).cuda()
    dgate = fb.norm_bwd(dr.cuda(), None, None, y.cuda(), w.cuda(), None, torch.ones(8, device="cuda"),
                        None, gate=gate, gate_kind=kind, sigmoid=True)[4].cpu()
    n = H if kind == "token" else 1
    assert (dgate[:4] == 0).all() and torch.isnan(dgate[4]).all()
    assert ((dgate[5] > n * 8e-39) & (dgate[5] < n * 9e-39)).all() and (dgate[6] < n * 1e-44).all()
    assert (dgate[7] == n * 0.25).all()


@pytest.mark.parametrize("kind", ["token", "channel", "full"])
def test_bf16_rows_at_the_ends(kind):
    """The same in bf16 rows, whose gates per element and channel take the fast exponential:
    beyond f32's smallest normal value a gate may be zero, but nothing is infinite or NaN."""
    z, full = ends()
    n = H // 8
    gate = {"token": z, "channel": z.repeat_interleave(n), "full": full.to(BF16)}[kind].cuda()
    T = 8 if kind == "token" else 3 if kind == "channel" else 8
    y, dr = (torch.ones(T, H, dtype=BF16) for _ in range(2))
    w = torch.ones(H)
    kw = dict(gate=gate, gate_kind=kind, sigmoid=True)
    r = fb.norm_fwd(torch.zeros_like(y).cuda(), y.cuda(), w.cuda(), None, eps=0.0, **kw)[0].cpu().float()
    dgate = fb.norm_bwd(dr.cuda(), None, None, y.cuda(), w.cuda(), None, torch.ones(T, device="cuda"),
                        None, **kw)[4].cpu().float()
    if kind == "channel":
        r, dgate = r[0].reshape(8, n), dgate.reshape(8, n)
    terms = {"token": H, "channel": T, "full": 1}[kind]
    for i, want in enumerate([1.0, 0.0, 1.0, 0.0]):
        assert (r[i] == want).all() and (dgate[i] == 0).all()
    assert torch.isnan(r[4]).all() and torch.isnan(dgate[4]).all()
    assert ((r[5:7] >= 0) & (r[5:7] < 1e-38)).all() and (r[7] == 0.5).all()
    assert ((dgate[5:7] >= 0) & (dgate[5:7] < terms * 1e-38)).all()
    assert (dgate[7] == terms * 0.25).all()
