"""What a plan of the AdamW step notices: memory that a tensor of its list no longer has."""
import pytest
import torch

from fp8_moe_routed_gb300 import binding as fb

pytestmark = pytest.mark.gpu

E, K, N = 2, 32, 128


def tensors():
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    u = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    return dict(p=f(E, K, N), m=u(E, K, N), v=u(E, K, N), m_scales=f(E * K * N // 128),
                v_scales=f(E * K * N // 128),
                copies=torch.zeros(E, K, N, dtype=torch.bfloat16, device="cuda"),
                codes=u(E, K, N), code_scales=f(E, N))


def plan_of(t):
    other = torch.ones(5, device="cuda")          # a second param, without codes and copy
    one = lambda k: [t[k], None]  # noqa: E731
    m, v = torch.zeros(5, device="cuda"), torch.zeros(5, device="cuda")
    return fb.AdamwPlan([t["p"], other], [t["m"], m], [t["v"], v], m_scales=one("m_scales"),
                        v_scales=one("v_scales"), copies=one("copies"), codes=one("codes"),
                        code_scales=one("code_scales"))


def grads():
    return [torch.ones(E, K, N, device="cuda"), torch.ones(5, device="cuda")]


@pytest.mark.parametrize("name", ["p", "m", "v", "m_scales", "v_scales", "copies", "codes",
                                  "code_scales"])
@pytest.mark.parametrize("how", ["data", "set", "grown"])
def test_memory_that_was_replaced_is_refused(name, how):
    """A tensor that has other memory than the plan knows (a loaded state, a grown one) is named
    before anything is launched: neither the old memory nor the new is written."""
    t = tensors()
    plan = plan_of(t)
    fb.adamw_step(plan, grads(), step=1, lr=1e-3)
    other = t[name].clone()
    if how == "data":
        t[name].data = other
    elif how == "set":
        t[name].set_(other)
    else:
        old = t[name].data_ptr()
        t[name].resize_(1 << 22).zero_()
        if t[name].data_ptr() == old:             # grown in its place: it has the plan's memory
            pytest.skip("the memory was grown in place")
    torch.cuda.synchronize()
    before = {k: x.clone() for k, x in t.items()}
    with pytest.raises(ValueError, match="storage"):
        fb.adamw_step(plan, grads(), step=2, lr=1e-3)
    with pytest.raises(ValueError, match="storage"):
        fb.adamw_step(plan, [grads()[0], None], step=2, lr=1e-3)
    for k, x in t.items():
        assert torch.equal(x, before[k]), k
