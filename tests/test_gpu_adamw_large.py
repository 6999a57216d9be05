"""The AdamW step where places need more than 32 bits: the values at the far end are as they are in
a small tensor, in every array."""
import numpy as np
import pytest
import torch

import train_reference as ref
from fp8_moe_routed_gb300 import binding as fb

pytestmark = pytest.mark.gpu

F = np.float32
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.999, eps=1e-8)
DECAY = 0.1
BF16, U8 = torch.bfloat16, torch.uint8


@pytest.fixture(autouse=True)
def _memory():
    yield
    torch.cuda.empty_cache()


def tail(n, seed):
    rng = np.random.default_rng(seed)
    g = torch.from_numpy((rng.standard_normal(n) * 1e-2).astype(F)).to(BF16)
    return (rng.standard_normal(n) * 0.02).astype(F), g.float().numpy()


def cuda(a, dtype=None):
    t = torch.from_numpy(a).cuda()
    return t if dtype is None else t.to(dtype)


def equal(t, a):
    return np.array_equal(t.float().cpu().numpy().reshape(-1) if t.dtype == BF16
                          else t.cpu().numpy().reshape(-1), a)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_tensor(bits):
    n = 2 ** 32 + 300
    first = 2 ** 32 - 4096                           # whole blocks of an 8-bit moment from here on
    state = torch.float32 if bits == 32 else U8
    p = torch.zeros(n, device="cuda")
    g, copy = (torch.zeros(n, dtype=BF16, device="cuda") for _ in range(2))
    m, v = (torch.zeros(n, dtype=state, device="cuda") for _ in range(2))
    scales = [None if bits == 32 else [torch.zeros(fb.adamw_blocks(n), device="cuda")]
              for _ in range(2)]
    p0, g0 = tail(n - first, 1)
    p[first:], g[first:] = cuda(p0), cuda(g0, BF16)
    plan = fb.AdamwPlan([p], [m], [v], m_scales=scales[0], v_scales=scales[1], copies=[copy],
                        weight_decay=DECAY)
    fb.adamw_step(plan, [g], step=2, seed=3, **HYPER)
    zero = np.zeros(n - first, F)
    new, m1, v1, r = ref.adamw(p0, g0, zero, zero, 2, decay=DECAY, **HYPER)
    assert equal(p[first:], new)
    assert equal(copy[first:], torch.from_numpy(new).to(BF16).float().numpy())
    if bits == 32:
        assert equal(m[first:], m1) and equal(v[first:], v1)
    else:
        chance = ref.random_bits(n - first, 0, 2, 3, first=first)
        for t, scale, x, bits16, never in ((m, scales[0], m1, chance & np.uint32(0xFFFF), False),
                                           (v, scales[1], r, chance >> np.uint32(16), True)):
            codes, per = ref.encode(x, bits16, never)
            assert equal(t[first:], codes) and equal(scale[0][first // 128:], per)
            assert not scale[0][:first // 128].any()
    for t in (p, m, v, copy):
        assert not t[:first].any()


@pytest.mark.parametrize("bits", [32, 8])
def test_weights_with_codes(bits):
    """The last of 17 experts of 2^28 weights against the same expert alone."""
    E, K, N = 17, 2 ** 14, 2 ** 14
    state = torch.float32 if bits == 32 else U8
    gen = torch.Generator(device="cuda").manual_seed(1)

    def made(E):
        z = lambda dtype, *s: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
        t = dict(p=z(torch.float32, E, K, N), g=z(BF16, E, K, N), m=z(state, E, K, N),
                 v=z(state, E, K, N), codes=z(U8, E, K, N), scale=z(torch.float32, E, N))
        if bits == 8:
            t.update(ms=z(torch.float32, E * K * N // 128), vs=z(torch.float32, E * K * N // 128))
        return t

    def step(t):
        one = lambda k: [t[k]] if k in t else None  # noqa: E731
        plan = fb.AdamwPlan([t["p"]], [t["m"]], [t["v"]], m_scales=one("ms"), v_scales=one("vs"),
                            codes=[t["codes"]], code_scales=[t["scale"]], weight_decay=DECAY)
        fb.adamw_step(plan, [t["g"]], step=2, seed=3, **HYPER)

    few, many = made(1), made(E)
    few["p"].normal_(0, 0.02, generator=gen)
    few["g"].normal_(0, 0.01, generator=gen)
    p0, g0 = (few[k].view(-1)[-4096:].float().cpu().numpy() for k in "pg")
    many["p"][-1:], many["g"][-1:] = few["p"], few["g"]
    step(few)
    step(many)
    for k in ("p", "codes", "scale") + (("m", "v") if bits == 32 else ()):
        assert torch.equal(many[k][-1:], few[k]), k
        if k != "scale":
            assert not many[k][:-1].any(), k
    assert (many["scale"][:-1].cpu() == torch.tensor(1e-12) / torch.tensor(448.0)).all()
    if bits == 32:
        return
    blocks = K * N // 128
    for k in ("ms", "vs"):
        assert torch.equal(many[k][-blocks:], few[k]) and not many[k][:-blocks].any(), k
    # the codes are rounded by chance, from their places
    zero = np.zeros(4096, F)
    _, m1, _, r = ref.adamw(p0, g0, zero, zero, 2, decay=DECAY, **HYPER)
    chance = ref.random_bits(4096, 0, 2, 3, first=E * K * N - 4096)
    for k, x, bits16, never in (("m", m1, chance & np.uint32(0xFFFF), False),
                                ("v", r, chance >> np.uint32(16), True)):
        assert equal(many[k].view(-1)[-4096:], ref.encode(x, bits16, never)[0]), k
