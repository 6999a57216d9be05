"""What the router's and the optimiser's calls refuse, before any launch."""
import ctypes

import pytest
import torch

from fp8_moe_routed_gb300 import binding as fb

P = ctypes.c_void_p
EINVAL, EALIGN, EWORKSPACE = -1, -2, -3


def fwd(logits=16, T=10, E=8, type=1, score=0, bias=None, topk=2, normalize=1, offsets=None, B=1,
        ids=16, weights=16, counts=16, loss=16, slope=16, ws=256, wsb=10 ** 9):
    return fb.load().fp8moe_router_fwd(P(logits), T, E, type, score, P(bias), topk, normalize, 1.0,
                                       P(offsets), B, P(ids), P(weights), P(counts), P(loss),
                                       P(slope), P(ws), wsb, None)


def balance(logits=16, ids=16, T=10, E=8, type=1, score=0, topk=2, offsets=None, B=1, counts=16,
            loss=16, slope=16, ws=256, wsb=10 ** 9):
    return fb.load().fp8moe_balance_fwd(P(logits), P(ids), T, E, type, score, topk, P(offsets), B,
                                        P(counts), P(loss), P(slope), P(ws), wsb, None)


def bwd(dweights=16, logits=16, ids=16, T=10, E=8, type=1, score=0, topk=2, normalize=1, dloss=16,
        slope=16, offsets=None, B=1, out=16):
    return fb.load().fp8moe_router_bwd(P(dweights), P(logits), P(ids), T, E, type, score, topk,
                                       normalize, 1.0, P(dloss), P(slope), P(offsets), B, P(out),
                                       None)


@pytest.mark.parametrize("call", [fwd, balance, bwd])
def test_sizes_and_kinds(call):
    for bad in (dict(E=0), dict(E=1025), dict(topk=0), dict(topk=33, E=64), dict(topk=9), dict(T=-1),
                dict(T=2 ** 31), dict(T=2 ** 30, topk=2), dict(type=2), dict(type=-1), dict(score=2),
                dict(score=-1), dict(B=0, offsets=16), dict(B=2), dict(logits=None),
                dict(ids=None)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(logits=8), dict(ids=2), dict(offsets=2)):
        assert call(**bad) == EALIGN, bad


def test_forward():
    assert fwd(normalize=2) == EINVAL and fwd(weights=None) == EINVAL
    assert fwd(counts=None) == EINVAL and fwd(loss=None) == EINVAL and fwd(slope=None) == EINVAL
    assert fwd(ws=None) == EWORKSPACE and fwd(wsb=64) == EWORKSPACE and fwd(ws=128) == EALIGN
    assert fwd(bias=2) == EALIGN and fwd(weights=2) == EALIGN and fwd(slope=2) == EALIGN
    none = dict(counts=None, loss=None, slope=None, ws=None, wsb=0)
    assert fwd(T=0, **none) == 0 and fwd(T=0, logits=None, ids=None, weights=None, **none) == 0


def test_balance_and_gradient():
    assert balance(counts=None) == EINVAL and balance(slope=None) == EINVAL
    assert balance(ws=None) == EWORKSPACE and balance(wsb=64) == EWORKSPACE
    assert bwd(normalize=-1) == EINVAL and bwd(out=None) == EINVAL
    assert bwd(dloss=None) == EINVAL and bwd(slope=None) == EINVAL
    assert bwd(slope=4) == EALIGN and bwd(out=8) == EALIGN and bwd(dweights=2) == EALIGN
    assert bwd(T=0) == 0


def test_balance_workspace():
    """A part for each chunk of tokens and each sequence: shares and counts of every expert, and
    a number of tokens."""
    for T, B, E in ((0, 1, 8), (1, 1, 1), (4096, 5, 256), (65536, 1, 128)):
        chunk = min(128, max(8, -(-(T // 608) // 8) * 8))
        slots = -(-T // chunk) + B
        up = lambda n: -(-n // 256) * 256  # noqa: E731
        assert fb.workspace_size(fb.OP_BALANCE, T, 0, B, E) == 2 * up(4 * slots * E) + up(4 * slots)


# ------------------------------------------------------------------------------- AdamW
def tensor(**kw):
    d = dict(p=16, g=16, m=16, v=16, n=100, g_type=1, state_bits=32)
    d.update({k: 0 if v is None else v for k, v in kw.items()})
    return fb._AdamwTensor(**d)


def step(*tensors, count=None, step=1, step_dev=None, lr=1e-3, lr_dev=None, beta1=0.9, beta2=0.999,
         eps=1e-8, grad_scale=None, ws=256, wsb=10 ** 9):
    table = (fb._AdamwTensor * max(1, len(tensors)))(*tensors)
    return fb.load().fp8moe_adamw_step(table, len(tensors) if count is None else count, step,
                                       P(step_dev), lr, P(lr_dev), beta1, beta2, eps, P(grad_scale),
                                       0, P(ws), wsb, None)


def test_adamw_numbers():
    for bad in (dict(step=0), dict(step=-3), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0),
                dict(beta1=float("nan")), dict(lr=float("nan")), dict(eps=float("nan"))):
        assert step(tensor(), **bad) == EINVAL, bad
    for bad in (dict(step_dev=4), dict(lr_dev=2), dict(grad_scale=2)):
        assert step(tensor(), **bad) == EALIGN, bad
    assert step(count=-1) == EINVAL
    assert fb.load().fp8moe_adamw_step(None, 1, 1, None, 1e-3, None, 0.9, 0.999, 1e-8, None, 0, None,
                                       0, None) == EINVAL
    assert step() == 0 and step(tensor(n=0, p=None)) == 0          # nothing to do
    assert step(tensor(), step_dev=16, ws=None) == EWORKSPACE
    assert step(tensor(), lr_dev=16, wsb=100) == EWORKSPACE
    assert step(tensor(), lr_dev=16, ws=64) == EALIGN


def test_adamw_tensors():
    codes = dict(codes=16, code_scale=16, n=2 * 32 * 48, K=32, N=48)
    for bad in (dict(n=-1), dict(n=2 ** 43), dict(p=None), dict(g=None), dict(m=None), dict(v=None),
                dict(g_type=2), dict(state_bits=16), dict(state_bits=8), dict(m_scale=16),
                dict(state_bits=8, m_scale=16), dict(weight_decay=float("nan")), dict(codes=16),
                dict(code_scale=16), {**codes, "n": 2 * 32 * 48 + 1}, {**codes, "K": 0},
                {**codes, "n": 2000 * 32 * 48}, {**codes, "n": 2 ** 21 * 64, "K": 2 ** 22, "N": 32},
                {**codes, "K": 2 ** 40, "N": 2 ** 40}):
        assert step(tensor(), tensor(**bad)) == EINVAL, bad
    for bad in (dict(p=2), dict(g=2), dict(m=2), dict(v=2), dict(copy=1),
                dict(g=1, g_type=0), dict(state_bits=8, m_scale=2, v_scale=16),
                {**codes, "code_scale": 2}, {**codes, "n": 40 * 48, "K": 40},
                {**codes, "n": 32 * 40, "N": 40}):
        assert step(tensor(), tensor(**bad)) == EALIGN, bad
    assert step(tensor(**codes), ws=None) == EWORKSPACE
    assert step(tensor(**codes), wsb=256 + 4 * (2 * 48 + 2) - 1) == EWORKSPACE


def test_adamw_workspace():
    def size(*tensors, on_device=0):
        table = (fb._AdamwTensor * max(1, len(tensors)))(*tensors)
        return fb.load().fp8moe_adamw_workspace_size(table, len(tensors), on_device)
    assert size() == 0 and size(tensor()) == 0 and size(tensor(), on_device=1) == 256
    codes = dict(codes=16, code_scale=16, n=2 * 32 * 48, K=32, N=48)
    assert size(tensor(**codes)) == 256 + 512
    assert size(tensor(**codes), tensor(**codes), on_device=1) == 256 + 1024
    # what the step refuses needs none
    assert size(tensor(**{**codes, "K": 2 ** 32, "N": 2 ** 32})) == 0
    assert size(tensor(**{**codes, "n": -5})) == 0 and size(tensor(**{**codes, "K": 0})) == 0


def test_python_side_refuses_what_is_no_cuda_tensor():
    x, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: fb.router_fwd(x, 2), lambda: fb.balance_fwd(x, ids),
                 lambda: fb.router_bwd(None, x, ids), lambda: fb.AdamwPlan([x], [x], [x])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        fb.router_fwd(x.double(), 2)
    with pytest.raises(TypeError):
        fb.router_fwd([1.0], 2)
    with pytest.raises(ValueError, match="one entry"):
        fb.AdamwPlan([x], [], [])


@pytest.mark.gpu
def test_python_side_refuses():
    x = torch.zeros(4, 8, device="cuda")
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    for call in (lambda: fb.router_fwd(x, 2, score="relu"), lambda: fb.router_fwd(x.t(), 2),
                 lambda: fb.router_fwd(x, 0), lambda: fb.router_fwd(x[0], 2),
                 lambda: fb.router_fwd(x, 2, bias=f(9)),
                 lambda: fb.router_fwd(x, 2, seq_offsets=off[:1]),
                 lambda: fb.router_fwd(x, 2, bias=torch.zeros(8)),
                 lambda: fb.balance_fwd(x, ids[:3].contiguous()),
                 lambda: fb.router_bwd(f(4, 3), x, ids), lambda: fb.router_bwd(None, x, ids, dloss=f(1)),
                 lambda: fb.router_bwd(None, x, ids, dloss=f(2), slope=f(1, 8)),
                 lambda: fb.router_bwd(None, x, ids, out=f(4, 9))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        fb.router_fwd(x, 2, seq_offsets=off.long())
    with pytest.raises(fb.Fp8MoeError, match="EINVAL"):
        fb.router_fwd(x, 9)
    with pytest.raises(fb.Fp8MoeError, match="EALIGN"):
        fb.router_fwd(f(100)[1:33].view(4, 8), 2)
    with pytest.raises(fb.Fp8MoeError, match="EWORKSPACE"):
        fb.router_fwd(x, 2, balance=True, workspace=f(8))
    # plans
    u = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    p, m, v = f(10), f(10), f(10)
    for call in (lambda: fb.AdamwPlan([p], [m], [p]), lambda: fb.AdamwPlan([p, p], [m, m], [v, v]),
                 lambda: fb.AdamwPlan([p], [m], [f(11)]),
                 lambda: fb.AdamwPlan([p], [u(10)], [u(10)], m_scales=[f(1)]),
                 lambda: fb.AdamwPlan([p], [u(10)], [u(10)], m_scales=[f(2)], v_scales=[f(2)]),
                 lambda: fb.AdamwPlan([p], [m], [v], codes=[u(10)], code_scales=[f(1)]),
                 lambda: fb.AdamwPlan([p], [m], [v], weight_decay=[0.1, 0.2]),
                 lambda: fb.AdamwPlan([p], [m], [v], copies=[None, None])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        fb.AdamwPlan([p.double()], [m], [v])
    with pytest.raises(TypeError):
        fb.AdamwPlan([p], [m], [v], copies=[f(10)])
    plan = fb.AdamwPlan([p], [m], [v])
    for call in (lambda: fb.adamw_step(plan, [], 1, 1e-3), lambda: fb.adamw_step(plan, [f(9)], 1, 1e-3),
                 lambda: fb.adamw_step(plan, [f(20)[::2]], 1, 1e-3),
                 lambda: fb.adamw_step(plan, [torch.zeros(10)], 1, 1e-3),
                 lambda: fb.adamw_step(plan, [f(10)], 1, 1e-3, grad_scale=f(2))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        fb.adamw_step(plan, [f(10).half()], 1, 1e-3)
    with pytest.raises(TypeError):
        fb.adamw_step(plan, [f(10)], torch.zeros(1, device="cuda"), 1e-3)
    with pytest.raises(fb.Fp8MoeError, match="EINVAL"):
        fb.adamw_step(plan, [f(10)], 0, 1e-3)
    p.data = f(10)
    with pytest.raises(ValueError, match="storage"):
        fb.adamw_step(plan, [f(10)], 1, 1e-3)
