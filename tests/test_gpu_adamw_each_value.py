"""The AdamW step of a value depends on that value alone: not on its neighbours, nor on where its
tensor lies in memory; and far from one, its root and quotient are as f32 rounds them."""
import numpy as np
import pytest
import torch

import train_reference as ref
from fp8_moe_routed_gb300 import binding as fb

pytestmark = pytest.mark.gpu

F = np.float32
HYPER = dict(lr=1.0, beta1=0.9, beta2=0.999, eps=1e-8)


def shifted(t, by):
    """t at `by` values behind a boundary of 512 bytes."""
    room = torch.empty(t.numel() + by, dtype=t.dtype, device="cuda")
    room[by:] = t
    return room[by:]


def new_weights(placement, g, m, v, ms=None, vs=None):
    """One step of weights of zero, without decay: what comes out is -rate * quotient."""
    by = dict(zip("pgmv", placement))
    p = shifted(torch.zeros_like(g), by["p"])
    g, m, v = shifted(g, by["g"]), shifted(m, by["m"]), shifted(v, by["v"])
    ms, vs = (None if s is None else [s.clone()] for s in (ms, vs))
    plan = fb.AdamwPlan([p], [m], [v], m_scales=ms, v_scales=vs)
    fb.adamw_step(plan, [g], step=7, **HYPER)
    return p, m, v


def differ(a, b):
    """Values whose bits differ."""
    word = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return int((a.view(word) != b.view(word)).sum())


@pytest.mark.parametrize("bits", [32, 8])
def test_one_result_wherever_a_tensor_lies(bits):
    """First moments from 2^-125 up (gradients that stopped), every eighth second moment zero: the
    values around it are the same on 16 bytes, at odd addresses, and in blocks that begin
    elsewhere, whatever shares a thread's work with them there."""
    n = 2 ** 26
    gen = torch.Generator(device="cuda").manual_seed(3)
    draw = lambda n: torch.rand(n, generator=gen, device="cuda")  # noqa: E731
    zero = torch.arange(n, device="cuda", dtype=torch.int32) % 8 == 3
    g = torch.zeros(n, device="cuda")
    if bits == 32:
        m = torch.exp2(draw(n) * 115 - 125)
        v = draw(n).mul_(1e-4).masked_fill_(zero, 0.0)
        scales = (None, None)
    else:
        codes = lambda: torch.randint(1, 0x7E, (n,), generator=gen, device="cuda",  # noqa: E731
                                      dtype=torch.uint8)
        m, v = codes(), codes().masked_fill_(zero, 0)
        scales = (torch.exp2(draw(n // 128) * 100 - 125), draw(n // 128) * 1e-5 + 1e-6)
    # 8-bit moments take wide accesses from their first value on or nowhere
    places = [(0, 0, 0, 0), (0, 1, 0, 0)] + ([(1, 1, 1, 1)] if bits == 32 else [])
    first = new_weights(places[0], g, m, v, *scales)
    for place in places[1:]:
        other = new_weights(place, g, m, v, *scales)
        for name, a, b in zip("pmv", first, other):
            assert differ(a, b) == 0, (place, name, differ(a, b))


def step_of(m, v, g=None, step=1000, on_device=False, **hyper):
    """New weights and moments of weights of zero, on the GPU and by the reference."""
    n = len(m)
    h = {**HYPER, **hyper}
    g = np.zeros(n, F) if g is None else g
    t = [torch.from_numpy(a.copy()).cuda() for a in (np.zeros(n, F), g, m, v)]
    plan = fb.AdamwPlan([t[0]], [t[2]], [t[3]])
    at = torch.tensor([step], device="cuda") if on_device else step
    fb.adamw_step(plan, [t[1]], step=at, **h)
    with np.errstate(all="ignore"):
        want = ref.adamw(np.zeros(n, F), g, m, v, step, decay=0.0, **h)
    return [x.cpu().numpy() for x in (t[0], t[2], t[3])], want


def off(got, want):
    return int((~((got == want) | (np.isnan(got) & np.isnan(want)))).sum())


def test_small_first_moments():
    """A gradient that stopped: m falls by 0.9 a step, v by 0.999, so that m comes below 2^-100
    while v is an ordinary number. One quotient (or root) in 2^22 may be rounded the other way:
    0.13 expected of 2^18 quotients and as many roots; five by chance are less likely than 1e-6."""
    n = 2 ** 18
    rng = np.random.default_rng(1)
    m = (np.exp2(rng.uniform(-130, -100, n)) * rng.choice([-1, 1], n)).astype(F)
    v = np.square(rng.uniform(1e-4, 1e-2, n)).astype(F)
    got, want = step_of(m, v, lr=1e20)
    assert off(got[0], want[0]) <= 4 and off(got[1], want[1]) == off(got[2], want[2]) == 0


@pytest.mark.parametrize("eps", [2.0 ** 21, 1e10, 1e30, 1.5e38])
def test_large_eps(eps):
    """Quotients by any eps that f32 holds."""
    n = 2 ** 12
    rng = np.random.default_rng(2)
    m = (rng.standard_normal(n) * min(eps, 1e36)).astype(F)
    v = np.square(rng.uniform(1e-4, 1e-2, n)).astype(F)
    got, want = step_of(m, v, eps=eps)
    assert off(got[0], want[0]) == 0


@pytest.mark.parametrize("on_device", [False, True])
@pytest.mark.parametrize("hyper", [dict(lr=1e-30), dict(lr=0.0), dict(lr=-3e-4), dict(lr=1e30),
                                   dict(beta1=0.0), dict(beta2=0.0), dict(eps=0.0),
                                   dict(beta2=1 - 2.0 ** -40, step=1), dict(beta1=1 - 2.0 ** -20, step=1)])
def test_rates_at_their_ends(hyper, on_device):
    """Rates that vanish or are huge, factors of a moment's correction at the ends of their range."""
    n = 2 ** 12
    rng = np.random.default_rng(4)
    m, g = (rng.standard_normal(n) * 1e-3).astype(F), (rng.standard_normal(n) * 1e-2).astype(F)
    v = np.square(rng.uniform(1e-4, 1e-2, n)).astype(F)
    got, want = step_of(m, v, g, on_device=on_device, **hyper)
    # a power in 64 bits, within two units of itself on the GPU, is the whole of 1 - b^t's error
    if on_device and "step" in hyper:
        rel = 4 * 2.0 ** -53 / (1 - hyper.get("beta1", hyper.get("beta2"))) + 8 * 2.0 ** -24
        assert (np.abs(got[0] - want[0]) <= rel * np.abs(want[0])).all()
    else:
        assert off(got[0], want[0]) == 0
    assert off(got[1], want[1]) == off(got[2], want[2]) == 0


def test_a_correction_without_end():
    """A beta2 whose power is 1 to 64 bits, or next to it: finite weights, whatever pow() says."""
    m, v = np.full(256, 1e-3, F), np.full(256, 1e-4, F)
    for on_device in (False, True):
        got, _ = step_of(m, v, on_device=on_device, step=1, beta2=1 - 2.0 ** -53)
        assert np.isfinite(got[0]).all()


def test_far_values_among_ordinary_ones():
    """Infinite, huge, tiny, zero and NaN moments, each beside ordinary values: every one as f32
    has it, and the values beside them as they are without them."""
    n = 4096
    rng = np.random.default_rng(3)
    m, g = (rng.standard_normal(n) * 1e-3).astype(F), (rng.standard_normal(n) * 1e-2).astype(F)
    v = np.square(rng.uniform(1e-4, 1e-2, n)).astype(F)
    plain, _ = step_of(m, v, g)
    far_m = [np.inf, -np.inf, 3e38, 1e30, 1e12, 2.0 ** -149, 1e-40, -1e-30, 0.0, -0.0, np.nan]
    far_v = [np.inf, 3e38, 1e37, 1e20, 1e11, 2.0 ** -149, 1e-40, 1e-31, 0.0, np.nan, -1e-3]
    far = np.zeros(n, bool)
    for j, x in enumerate(far_m):
        m[7 + 37 * j] = x
        far[7 + 37 * j] = True
    for j, x in enumerate(far_v):
        v[1029 + 37 * j] = x
        far[1029 + 37 * j] = True
    for j, x in enumerate(far_m):
        for i, y in enumerate(far_v):
            at = 2048 + 16 * (j * len(far_v) + i)
            m[at], v[at], far[at] = x, y, True
    g[far] = 0.0
    got, want = step_of(m, v, g)
    for a, b in zip(got, want):
        assert off(a[far], b[far]) == 0, [(m[i], v[i], x, y) for i, x, y in
                                          zip(np.nonzero(far)[0], a[far], b[far])
                                          if not (x == y or (np.isnan(x) and np.isnan(y)))]
    for a, b in zip(got, plain):
        assert np.array_equal(a[~far], b[~far])
