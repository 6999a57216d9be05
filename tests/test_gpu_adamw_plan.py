"""What a plan of the AdamW step notices: memory that a tensor of its list no longer has; and what
autograd notices of a step."""
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


def test_autograd_sees_that_weights_changed():
    """A weight, copy or codes that a backward pass still needs: the pass ends in an error, as it
    does after any other change in place, not in the gradient of other weights."""
    t = tensors()
    plan = plan_of(t)
    p = t["p"].requires_grad_()
    x = torch.randn(K, N, device="cuda", requires_grad=True)

    class Scaled(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            ctx.save_for_backward(w)
            return x * w.float()[0]

        @staticmethod
        def backward(ctx, d):
            w, = ctx.saved_tensors
            return d * w.float()[0], None

    for make in (lambda: (x * p[0]).sum(), lambda: Scaled.apply(x, t["copies"]).sum(),
                 lambda: Scaled.apply(x, t["codes"]).sum(),
                 lambda: Scaled.apply(x[0], t["code_scales"]).sum()):
        loss = make()
        fb.adamw_step(plan, grads(), step=1, lr=1e-3)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
        make().backward()                          # and a new pass is fine


def test_what_a_step_leaves_alone_keeps_its_version():
    """A param without a gradient is not changed, and a refused step changes nothing."""
    t = tensors()
    plan = plan_of(t)
    before = {k: x._version for k, x in t.items()}
    fb.adamw_step(plan, [None, grads()[1]], step=1, lr=1e-3)
    with pytest.raises(ValueError):
        fb.adamw_step(plan, grads()[:1], step=1, lr=1e-3)
    with pytest.raises(fb.Fp8MoeError):
        fb.adamw_step(plan, grads(), step=0, lr=1e-3)
    assert {k: x._version for k, x in t.items()} == before
    fb.adamw_step(plan, [grads()[0], None], step=1, lr=1e-3)
    assert all(t[k]._version > before[k] for k in ("p", "copies", "codes", "code_scales"))


def test_parts_of_one_buffer():
    """Params that are views of one tensor share its version; a step in inference mode has none."""
    flat = torch.ones(30, device="cuda", requires_grad=True)
    with torch.no_grad():
        parts = list(torch.split(flat, [10, 20]))
    zeros = lambda: [torch.zeros(n, device="cuda") for n in (10, 20)]  # noqa: E731
    plan = fb.AdamwPlan(parts, zeros(), zeros())
    loss = (flat * flat).sum()
    before = flat._version
    fb.adamw_step(plan, zeros(), step=1, lr=1e-3)
    assert flat._version == before + 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        p = torch.ones(10, device="cuda")
        plan = fb.AdamwPlan([p], [torch.zeros_like(p)], [torch.zeros_like(p)], weight_decay=0.5)
        fb.adamw_step(plan, [torch.zeros_like(p)], step=1, lr=1.0)
        assert p.tolist() == [0.5] * 10
    fb.adamw_step(plan, [torch.zeros(10, device="cuda")], step=2, lr=1.0)
    assert p.tolist() == [0.25] * 10
