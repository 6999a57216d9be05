"""The norms' gradient for rows far from unit scale, on the GPU against 64-bit forms: every
row whose sum of squares f32 can hold has the precision of a row of ones."""
import pytest
import torch

import layer_reference as ref
from fp8_moe_routed_gb300 import binding as fb

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def gradients(d, kind, sigmoid, a, b):
    """64-bit gradients by the formulas of the definition, from the saved f32 rstd."""
    v = {k: None if t is None else t.double() for k, t in d.items()}
    rh = v["r"] * v["rstd_pre"][:, None]
    u = v["w_pre"] * v["dh"]
    D = v["rstd_pre"][:, None] * (u - rh * (u * rh).mean(1, keepdim=True))
    if v["dr"] is not None:
        D = D + v["dr"]
    out = {"dw_pre": (v["dh"] * rh).sum(0)}
    if v["y"] is None:
        return {"dx": D, **out}
    yh = v["y"] * v["rstd_post"][:, None]
    g = ref.gate_value(v["gate"], kind, sigmoid)
    dn = b * D * g
    t = v["w_post"] * dn
    dG = b * D * v["w_post"] * yh * (g * (1 - g) if sigmoid else 1.0)
    out["dy"] = v["rstd_post"][:, None] * (t - yh * (t * yh).mean(1, keepdim=True))
    out["dw_post"] = (dn * yh).sum(0)
    out["dgate"] = {None: None, "token": dG.sum(1), "channel": dG.sum(0), "full": dG}[kind]
    return {"dx": a * D, **out}


# rms of r and of y (None: no block output): the smallest with eps = 0, as the forward takes them
SCALES = [(1e-17, None), (1e-15, None), (1e15, None), (1e17, None), (1e-15, 1e-15), (1e-17, 1.0),
          (1.0, 1e-17), (1e15, 1.0), (1.0, 1e17), (1e17, 1e17), (1e-17, 1e17)]


@pytest.mark.parametrize("gate,sigmoid", [(None, False), ("token", True), ("channel", True),
                                          ("full", True)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rms_r,rms_y", SCALES)
def test_backward(rms_r, rms_y, dtype, gate, sigmoid):
    if rms_y is None and gate is not None:
        pytest.skip("a gate belongs to a block output")
    T, H, a, b = 37, 128, 0.9, 0.7
    g = torch.Generator().manual_seed(1)
    post = rms_y is not None
    d = {"dr": None, "dh": torch.randn(T, H, generator=g).to(dtype),
         "r": (rms_r * torch.randn(T, H, generator=g)).to(dtype),
         "w_pre": 1 + 0.3 * torch.randn(H, generator=g),
         "y": (rms_y * torch.randn(T, H, generator=g)).to(dtype) if post else None,
         "w_post": 1 + 0.3 * torch.randn(H, generator=g) if post else None, "gate": None}
    shape = {None: None, "token": (T,), "channel": (H,), "full": (T, H)}[gate]
    if shape is not None:
        d["gate"] = torch.randn(*shape, generator=g).to(dtype if gate == "full" else F32)
    for row, rstd in (("r", "rstd_pre"), ("y", "rstd_post")):
        t = d[row]
        d[rstd] = None if t is None else t.double().square().mean(1).rsqrt().float()
    want = gradients(d, gate, sigmoid, a if post else 1.0, b)
    c = {k: None if t is None else t.cuda() for k, t in d.items()}
    got = fb.norm_bwd(None, c["dh"], c["r"], c["y"], c["w_post"], c["w_pre"], c["rstd_post"],
                      c["rstd_pre"], gate=c["gate"], gate_kind=gate, sigmoid=sigmoid,
                      residual_scale=a, branch_scale=b)
    # the relative bounds of ref.check_f32 hold at any scale: both sides are multiplied by the
    # reference's largest power of two, exactly, so that the squares of the rms stay in range
    for name, have in zip(("dx", "dy", "dw_post", "dw_pre", "dgate"), got):
        if have is None:
            assert want.get(name) is None
            continue
        w = want[name]
        p = float(2.0 ** -torch.frexp(w.abs().max())[1].double())
        unit = have.double() * p
        assert torch.isfinite(unit).all(), name
        (check_rows if have.dtype == BF16 else ref.check_f32)(unit, w * p, name)


def check_rows(got, want, what):
    """ref.check_rows on scaled values: bf16's step is relative, so it scales with them."""
    g, w = got.cpu(), want
    step = torch.pow(2.0, torch.floor(torch.log2(w.abs().clamp_min(2.0 ** -126))) - 7)
    bad = (g - w).abs() > step + 1e-5 * w.square().mean().sqrt()
    assert not bad.any(), (what, int(bad.sum()), float((g - w).abs().max()))
