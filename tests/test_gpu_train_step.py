"""The block's training step: router, experts, norms and optimiser in the order of their use."""
import numpy as np
import pytest
import torch

import train_reference as ref
from fp8_moe_routed_gb300 import binding as fb
from fp8_moe_routed_gb300 import moe_block as mb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("T,offsets", [(70, None), (70, [0, 25, 60]), (1, None)])
def test_step_is_the_composition_of_its_calls(bits, T, offsets):
    """Twice: the same results from the same calls made one by one, and new weights that are the
    optimiser's for the step's gradients; the next forward takes the codes that it left."""
    p, router, trainer, x, h = mb.training_example(T=T, H=256, F=128, E=8, topk=3, bits=bits)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    wi = trainer.plan.params[0]
    for step in (1, 2):
        dr, dh_next = torch.randn_like(x), torch.randn_like(x)
        before = wi.clone()
        codes = p.wi[0].clone(), p.wi[1].clone()
        m, v = trainer.m[0].clone(), trainer.v[0].clone()
        ms = vs = None
        if bits == 8:
            ms, vs = trainer.scales[0][0].clone(), trainer.scales[1][0].clone()

        logits = h.float() @ router.w
        ids, weights, counts, loss, slope = fb.router_fwd(logits, 3, score="sigmoid",
                                                          bias=router.bias, balance=True,
                                                          seq_offsets=off)
        fb.read_status()
        r, h_next, saved = mb.forward(p, x, h, ids, weights)
        grads = mb.backward(p, saved, dr, dh_next)
        dlogits = fb.router_bwd(grads["dweights"], logits, ids, score="sigmoid", slope=slope,
                                dloss=torch.full_like(loss, router.balance), seq_offsets=off)
        got = mb.train_step(p, router, trainer, x, h, dr, dh_next, lr=1e-3, seq_offsets=off)
        assert fb.read_status() == 0
        assert torch.equal(got[0], r) and torch.equal(got[1], h_next) and torch.equal(got[2], loss)
        assert torch.equal(got[3]["dwi"], grads["dwi"])
        want = h.float().t() @ dlogits
        torch.testing.assert_close(got[3]["dw_router"], want)
        if offsets is not None:                   # padding tokens pass the block by
            assert (ids[offsets[-1]:] == -1).all() and (saved["out"][offsets[-1]:] == 0).all()

        # the new weights, and their codes
        flat = lambda t: t.cpu().numpy().reshape(-1)  # noqa: E731
        if bits == 32:
            m0, v0 = flat(m), flat(v)
        else:
            m0 = ref.decode(flat(m), flat(ms))
            v0 = np.square(ref.decode(flat(v), flat(vs)))
        new = ref.adamw(flat(before), flat(grads["dwi"]), m0, v0, step, 1e-3, 0.9, 0.999, 1e-8, 0.1)
        assert np.array_equal(flat(wi), new[0])
        top = wi.abs().amax(1).clamp(min=1e-12)
        scale = top / torch.full_like(top, 448.0)
        q = (wi / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        assert torch.equal(p.wi[1], scale) and torch.equal(p.wi[0], q)
        assert not torch.equal(p.wi[0], codes[0])


def test_router_gradient_through_the_block():
    """The router's weights: their gradient against 64-bit autograd of weights and balance loss for
    the block's own dweights (three terms a token and the balance's, f32 products of 256)."""
    p, router, trainer, x, h = mb.training_example(T=50, H=256, F=128, E=8, topk=3)
    router.balance = 0.5
    ids, weights, chosen = mb.choose(router, h)
    dweights = torch.randn_like(weights)
    dh, dw = mb.choose_backward(router, chosen, dweights)
    w, hh = router.w.double().cpu().requires_grad_(), h.double().cpu().requires_grad_()
    logits = hh @ w
    total = (ref.weights(logits, ids.cpu().long(), "sigmoid", True, 1.0) * dweights.double().cpu()).sum()
    total = total + 0.5 * ref.balance(logits, ids.cpu().long(), "sigmoid", None)[1].sum()
    want = torch.autograd.grad(total, [w, hh])
    for got, v in ((dw, want[0]), (dh, want[1])):
        # library products in f32 (or their tensor-core form): 2^-11 a factor at worst
        assert float((got.double().cpu() - v).norm() / v.norm()) <= 2e-3


def test_bits_are_checked():
    with pytest.raises(ValueError):
        mb.training_example(T=4, H=256, F=128, E=4, topk=2, bits=16)
