"""The block example: its calls in the order of their use, against 64-bit forms of the
whole block, and its gradients against differences of those."""
import pytest
import torch

import layer_reference as ref
from fp8_moe_routed_gb300 import binding as fb
from fp8_moe_routed_gb300 import moe_block as mb

pytestmark = pytest.mark.gpu


def reference_block(x, h, ids, weights, wi, wo, p, w=None):
    """64-bit block on plain weights [E, H, 2F], [E, F, H]; differentiable."""
    T, k = ids.shape
    F = wo.shape[1]
    out = []
    for t in range(T):
        o = 0
        for j in range(k):
            e = int(ids[t, j])
            gu = h[t] @ wi[e]
            o = o + weights[t, j] * ((torch.nn.functional.silu(gu[:F]) * gu[F:]) @ wo[e])
        out.append(o)
    out = torch.stack(out)
    gate = None if p.gate is None else p.gate.double().cpu()
    return ref.norm_fwd(x, out, p.w_post.double().cpu(), p.w_pre.double().cpu(), gate, "channel", True,
                        p.residual_scale, p.branch_scale, p.eps)


def dequantized8(pair):
    return fb.dequantize_fp8_codes(*pair).double().cpu()


def dequantized4(pair):
    return fb.mxfp4_dequantize(*pair).double().cpu().transpose(1, 2)


def close(a, b, rel, what):
    """Relative 2-norm difference: the products round their activations to 3 mantissa bits
    (8-bit, about 2.5 % a factor) or to one (4-bit, about 10 %), twice in the block."""
    a, b = a.double().cpu(), b.double().cpu()
    d = float((a - b).norm() / b.norm())
    assert d <= rel, (what, d)


@pytest.mark.parametrize("T,topk", [(40, 3), (1, 4)])
def test_block_and_gradients(T, topk):
    p8, p4, x, h, ids, weights = mb.example(T=T, H=256, F=128, E=8, topk=topk, seed=T)
    fb.read_status()
    r, h_next, saved = mb.forward(p8, x, h, ids, weights)
    r4, h4 = mb.serve(p4, x, h, ids, weights)
    dr, dh = torch.randn_like(r), torch.randn_like(r)
    grads = mb.backward(p8, saved, dr, dh)
    assert fb.read_status() == 0

    xs = [t.double().cpu() for t in (x, h, weights)]
    for t in xs:
        t.requires_grad_()
    wi, wo = dequantized8(p8.wi).requires_grad_(), dequantized8(p8.wo).requires_grad_()
    want_r, want_h = reference_block(xs[0], xs[1], ids.cpu(), xs[2], wi, wo, p8)
    close(r, want_r.detach(), 0.05, "r")
    close(h_next, want_h.detach(), 0.05, "h")
    ((want_r * dr.double().cpu()).sum() + (want_h * dh.double().cpu()).sum()).backward()
    close(grads["dx"], xs[0].grad, 0.05, "dx")
    close(grads["dh"], xs[1].grad, 0.15, "dh")
    close(grads["dweights"], xs[2].grad, 0.15, "dweights")
    close(grads["dwi"], wi.grad, 0.15, "dwi")
    close(grads["dwo"], wo.grad, 0.15, "dwo")

    want_r4, want_h4 = reference_block(*[t.detach() for t in (xs[0], xs[1])], ids.cpu(), xs[2].detach(),
                                       dequantized4(p4.wi), dequantized4(p4.wo), p4)
    close(r4, want_r4, 0.2, "r4")
    close(h4, want_h4, 0.2, "h4")


def test_serve_is_the_composition_of_its_calls():
    _, p, x, h, ids, weights = mb.example(T=77, H=512, F=256, E=16, topk=4, seed=1)
    r, h_next = mb.serve(p, x, h, ids, weights)
    gs, slot_row, row_slot = fb.sort_tokens(ids, 16)
    rows = h[row_slot.long() // 4]
    act = fb.gmm_silu_mxfp4_fwd(rows, *p.wi, gs)
    y = fb.gmm_mxfp4_fwd(act, *p.wo, gs)
    out = fb.combine_tokens(y, slot_row, weights)
    r2, h2, _, _ = fb.norm_fwd(x, out, p.w_post, p.w_pre, gate=p.gate, gate_kind="channel",
                               sigmoid=True)
    assert torch.equal(r, r2) and torch.equal(h_next, h2)
    # one token alone gives the bits it has in the batch
    one_r, one_h = mb.serve(p, x[5:6], h[5:6], ids[5:6], weights[5:6])
    assert torch.equal(one_r, r[5:6]) and torch.equal(one_h, h_next[5:6])


def test_runs_as_a_module(capsys):
    mb.main()
    assert "cosine" in capsys.readouterr().out
