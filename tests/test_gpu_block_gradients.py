"""The block example's gradients on seeded inputs: every step against its 64-bit form on the
inputs that the step had, and the whole against a 64-bit block with bounds from the rounding
of the 8-bit products' activations."""
import pytest
import torch

import layer_reference as ref
from fp8_moe_routed_gb300 import binding as fb
from fp8_moe_routed_gb300 import moe_block as mb
from test_gpu_moe_block import dequantized8, reference_block

pytestmark = pytest.mark.gpu

H, F, E = 256, 128, 8
# Rounding to e4m3 (3 mantissa bits) is off by a factor's 2^-4 at most and 2.6 % in the rms.
# A row of the experts' outputs has it twice over, in the two products' activations, the first
# time through both factors of the SwiGLU: sqrt(3) * 2.6 % < 5 %. Its gradient comes back
# through a norm of such a row: another 5 %.
ROW, DOUT = 0.05, 0.05


def setup(T, topk):
    p, _, x, h, ids, weights = mb.example(T=T, H=H, F=F, E=E, topk=topk, seed=10 + T)
    g = torch.Generator().manual_seed(T)
    dr, dh = (torch.randn(T, H, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    r, h_next, saved = mb.forward(p, x, h, ids, weights)
    return p, x, h, ids, weights, dr, dh, r, h_next, saved, mb.backward(p, saved, dr, dh)


CASES = [(1, 4), (1, 1), (2, 8), (40, 3), (129, 2)]


@pytest.mark.parametrize("T,topk", CASES)
def test_steps(T, topk):
    """The router's weights' gradient and the norms' on the values that went into them."""
    p, x, h, ids, weights, dr, dh, r, _, s, grads = setup(T, topk)
    dx, dout, dw_post, dw_pre, dgate = fb.norm_bwd(
        dr, dh, s["r"], s["out"], p.w_post, p.w_pre, s["rstd_post"], s["rstd_pre"], **p.norms())
    for name, v in (("dx", dx), ("dw_post", dw_post), ("dw_pre", dw_pre), ("dgate", dgate)):
        assert torch.equal(grads[name], v)
    want_rows, want = ref.combine_bwd(dout.cpu(), s["y"].cpu(), s["slot_row"].cpu(),
                                      weights.cpu())
    # f32 sums of H terms, against the terms' size: a dot product may cancel
    size = (dout.cpu().double().abs()[:, None, :]
            * s["y"].cpu().double().abs()[s["slot_row"].cpu().long()]).sum(-1)
    assert ((grads["dweights"].cpu().double() - want).abs() <= 1e-5 * size).all()
    drows, _ = fb.combine_tokens_bwd(dout, s["y"], s["slot_row"], weights)
    ref.check_rows(drows, want_rows, "drows")
    # the norms' parameters, from the formulas in 64 bits
    d = {k: v.double().cpu() for k, v in (("dr", dr), ("dh", dh), ("r", s["r"]), ("y", s["out"]),
                                         ("w", p.w_post), ("v", p.w_pre), ("z", p.gate))}
    rq, rp = (s[k].double().cpu()[:, None] for k in ("rstd_pre", "rstd_post"))
    rh, yh, u = d["r"] * rq, d["y"] * rp, d["v"] * d["dh"]
    D = d["dr"] + rq * (u - rh * (u * rh).mean(1, keepdim=True))
    gate = torch.sigmoid(d["z"])
    ref.check_f32(dw_pre, (d["dh"] * rh).sum(0), "dw_pre")
    ref.check_f32(dw_post, (D * gate * yh).sum(0), "dw_post")
    ref.check_f32(dgate, (D * d["w"] * yh).sum(0) * gate * (1 - gate), "dgate")


@pytest.mark.parametrize("T,topk", CASES)
def test_whole_block(T, topk):
    p, x, h, ids, weights, dr, dh, r, h_next, s, grads = setup(T, topk)
    leaf = [t.double().cpu().requires_grad_() for t in
            (x, h, weights, p.w_post, p.w_pre, p.gate)]
    wi, wo = dequantized8(p.wi).requires_grad_(), dequantized8(p.wo).requires_grad_()
    q = mb.Params(p.wi, p.wo, leaf[3], leaf[4], None, p.residual_scale, p.branch_scale, p.eps)
    out = experts(leaf[1], ids.cpu(), leaf[2], wi, wo)
    out.retain_grad()
    want_r, want_h = ref.norm_fwd(leaf[0], out, leaf[3], leaf[4], leaf[5], "channel", True,
                                  q.residual_scale, q.branch_scale, q.eps)
    with torch.no_grad():      # the same block as the one that the other tests compare with
        r2, h2 = reference_block(*[t.detach() for t in leaf[:2]], ids.cpu(), leaf[2].detach(),
                                 wi.detach(), wo.detach(), p)
        assert torch.allclose(r2, want_r) and torch.allclose(h2, want_h)
    ((want_r * dr.double().cpu()).sum() + (want_h * dh.double().cpu()).sum()).backward()
    # A router weight's gradient is <dout, row>, a sum of H terms that may cancel to nothing.
    # Its error is <dout's, row> + <dout, row's>: H terms of either sign, sqrt(H) below the
    # product of the norms; six deviations of that.
    with torch.no_grad():
        rows = torch.stack([torch.stack([experts(leaf[1][t:t + 1], ids[t:t + 1, j:j + 1].cpu(),
                                                 torch.ones(1, 1, dtype=torch.float64), wi, wo)[0]
                                         for j in range(topk)]) for t in range(T)])
        size = out.grad.norm(dim=1)[:, None] * rows.norm(dim=2)
    bound = 6 * (ROW + DOUT) * size / H ** 0.5
    off = (grads["dweights"].double().cpu() - leaf[2].grad).abs()
    assert (off <= bound).all(), float((off / bound).max())
    # sums over tokens of products with a row's value: that value's error, per row
    for name, at in (("dw_post", 3), ("dw_pre", 4), ("dgate", 5)):
        have, want = grads[name].double().cpu(), leaf[at].grad
        assert (have - want).norm() <= 2 * (ROW + DOUT) * want.norm(), name


def experts(h, ids, weights, wi, wo):
    """The weighted sum of the experts' outputs, 64 bits."""
    out = []
    for t in range(ids.shape[0]):
        o = 0
        for j in range(ids.shape[1]):
            gu = h[t] @ wi[int(ids[t, j])]
            o = o + weights[t, j] * ((torch.nn.functional.silu(gu[:F]) * gu[F:]) @ wo[int(ids[t, j])])
        out.append(o)
    return torch.stack(out)
