"""The block's trainer around a step that is refused, and around weights that were replaced."""
import pytest
import torch

from fp8_moe_routed_gb300 import binding as fb
from fp8_moe_routed_gb300 import moe_block as mb


class Plan:
    """In place of the optimiser's: a machine without a GPU has no plan."""

    def __init__(self, params, m, v, **kw):
        self.params = params


@pytest.fixture
def made(monkeypatch):
    E, H, F = 2, 16, 16
    monkeypatch.setattr(fb, "AdamwPlan", Plan)
    calls = []
    monkeypatch.setattr(fb, "adamw_step", lambda plan, grads, **kw: calls.append(kw["step"]))
    wi, wo = torch.randn(E, H, 2 * F), torch.randn(E, F, H)
    p = mb.Params(mb.fp8_weight(wi), mb.fp8_weight(wo), w_post=torch.ones(H), w_pre=torch.ones(H),
                  gate=torch.zeros(H))
    router = mb.Router(torch.randn(H, E), 1, bias=torch.zeros(E))
    trainer = mb.Trainer(p, router, wi, wo)
    return p, router, trainer, {k: None for k in trainer.names}, calls


def test_a_refused_step_is_not_counted(made, monkeypatch):
    """The next one has its number: the corrections by 1 - beta^t and the random bits are those of
    the steps that were made."""
    _, _, trainer, grads, calls = made
    trainer.step(grads, lr=1e-3)

    def refuse(*args, **kw):
        raise ValueError("refused")

    with monkeypatch.context() as mp:
        mp.setattr(fb, "adamw_step", refuse)
        with pytest.raises(ValueError, match="refused"):
            trainer.step(grads, lr=1e-3)
    with pytest.raises(KeyError):
        trainer.step({}, lr=1e-3)
    assert trainer.steps == 1
    trainer.step(grads, lr=1e-3)
    assert calls == [1, 2] and trainer.steps == 2


@pytest.mark.parametrize("name", ["wi", "wo", "w_post", "w_pre", "gate", "router"])
def test_replaced_weights_are_refused(made, name):
    """Weights that the block takes from now on and that the trainer does not hold would stay as
    they are while it steps others."""
    p, router, trainer, grads, calls = made
    if name == "router":
        router.w = router.w.clone()
    elif name in ("wi", "wo"):
        setattr(p, name, mb.fp8_weight(torch.randn(getattr(p, name)[0].shape)))
    else:
        setattr(p, name, getattr(p, name).clone())
    with pytest.raises(ValueError, match="replaced"):
        trainer.step(grads, lr=1e-3)
    assert trainer.steps == 0 and not calls


def test_a_gate_that_is_gone_is_refused(made):
    p, router, trainer, grads, calls = made
    p.gate = None
    with pytest.raises(ValueError, match="gate was replaced"):
        trainer.step(grads, lr=1e-3)
    assert not calls


def test_the_same_weights_in_a_new_pair(made):
    """A pair is only a pair: its tensors are what counts, and a bias of the choice is no weight."""
    p, router, trainer, grads, calls = made
    p.wi = (p.wi[0], p.wi[1])
    router.bias = torch.ones_like(router.bias)
    trainer.step(grads, lr=1e-3)
    assert calls == [1]
