"""The AdamW step: bit for bit against f32 operations rounded one by one, and against the formula
in 64 bits, on the GPU."""
import threading

import numpy as np
import pytest
import torch

import train_reference as ref
from fp8_moe_routed_gb300 import binding as fb

pytestmark = pytest.mark.gpu

F = np.float32
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.999, eps=1e-8)
DECAY = 0.1


def numbers(n, seed, scale):
    return (np.random.default_rng(seed).standard_normal(n) * scale).astype(F)


class Tensor:
    """One tensor of a step, here and on the GPU. shift: values between a 512-byte boundary and
    the tensor's first."""

    def __init__(self, n, bits=32, gtype="f32", copy=False, shape=None, codes=False, shift=0, seed=0,
                 zero=False):
        self.n, self.bits, self.shape = n, bits, shape or (n,)
        self.p, self.m = numbers(n, seed, 0.02), numbers(n, seed + 1, 1e-3)
        self.g = numbers(n, seed + 2, 1e-2)
        if gtype == "bf16":
            self.g = torch.from_numpy(self.g).bfloat16().float().numpy()
        self.v = np.square(numbers(n, seed + 3, 1e-2))
        if zero:
            self.m[:], self.v[:] = 0, 0
        self.m_scale = self.v_scale = None
        if bits == 8:
            none = np.zeros(n, np.uint32)
            self.m, self.m_scale = ref.encode(self.m, none, False)
            self.v, self.v_scale = ref.encode(np.sqrt(self.v), none, True)

        def put(a, dtype=None):
            if a is None:
                return None
            t = torch.from_numpy(a)
            t = t if dtype is None else t.to(dtype)
            room = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")
            room[shift:] = t.cuda()
            return room[shift:].view(self.shape if t.numel() == n else t.shape)

        self.d = {k: put(getattr(self, k)) for k in ("p", "m", "v", "m_scale", "v_scale")}
        self.d["g"] = put(self.g, torch.bfloat16 if gtype == "bf16" else None)
        self.d["copy"] = put(np.zeros(n, F), torch.bfloat16) if copy else None
        self.d["codes"] = put(np.zeros(n, np.uint8)) if codes else None
        self.d["scale"] = torch.zeros(self.shape[0], self.shape[2], device="cuda") if codes else None

    def step(self, which, step, seed=0, grad_scale=None, decay=DECAY):
        m, v = self.m, self.v
        if self.bits == 8:
            m, v = ref.decode(m, self.m_scale), ref.decode(v, self.v_scale)
            v = v * v
        self.p, m, v, r = ref.adamw(self.p, self.g, m, v, step, decay=decay, grad_scale=grad_scale,
                                    **HYPER)
        if self.bits == 32:
            self.m, self.v = m, v
            return
        bits = ref.random_bits(self.n, which, step, seed)
        self.m, self.m_scale = ref.encode(m, bits & np.uint32(0xFFFF), False)
        self.v, self.v_scale = ref.encode(r, bits >> np.uint32(16), True)

    def check(self):
        for k in ("p", "m", "v", "m_scale", "v_scale"):
            if self.d[k] is None:
                continue
            got = self.d[k].cpu().numpy().reshape(-1)
            want = getattr(self, k)
            same = np.array_equal(got, want, equal_nan=got.dtype.kind == "f")
            assert same, (k, self.n, int((got != want).sum()))
        if self.d["copy"] is not None:
            assert torch.equal(self.d["copy"].cpu().reshape(-1), torch.from_numpy(self.p).bfloat16())
        if self.d["codes"] is not None:
            p = torch.from_numpy(self.p).view(self.shape)
            top = p.abs().amax(1).clamp(min=1e-12)
            scale = top / torch.full_like(top, 448.0)
            assert torch.equal(self.d["scale"].cpu(), scale)
            q = (p / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
            assert torch.equal(self.d["codes"].cpu(), q)


def plan_of(ts, decay=DECAY):
    col = lambda k: [t.d[k] for t in ts]  # noqa: E731
    return fb.AdamwPlan(col("p"), col("m"), col("v"), m_scales=col("m_scale"),
                        v_scales=col("v_scale"), copies=col("copy"), codes=col("codes"),
                        code_scales=col("scale"), weight_decay=decay)


def grads_of(ts):
    return [t.d["g"] for t in ts]


def run(ts, steps=(1, 2), seed=0, grad_scale=None):
    plan = plan_of(ts)
    gs = None if grad_scale is None else torch.tensor([grad_scale], device="cuda")
    for s in steps:
        fb.adamw_step(plan, grads_of(ts), step=s, seed=seed, grad_scale=gs, **HYPER)
        for i, t in enumerate(ts):
            t.step(i, s, seed, grad_scale)
        for t in ts:
            t.check()


SIZES = [1, 2, 3, 4, 5, 31, 127, 128, 129, 255, 256, 1000, 4095, 4096, 4097, 8192, 12345, 40001]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gtype", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_sizes_and_alignments(bits, gtype, shift):
    """Every size alone and all in one call: 16-byte aligned, on odd values, in between."""
    ts = [Tensor(n, bits, gtype, copy=i % 2 == 0, shift=shift, seed=10 * i)
          for i, n in enumerate(SIZES)]
    run(ts, steps=(1, 2, 1000), seed=7)
    run([Tensor(4100, bits, gtype, copy=True, shift=shift, seed=3)], steps=(5,), grad_scale=0.3)


def test_kinds_mixed_in_one_call():
    ts = [Tensor(5000, 32, "f32", seed=1), Tensor(5000, 8, "bf16", copy=True, seed=2),
          Tensor(2 * 32 * 128, 8, "f32", shape=(2, 32, 128), codes=True, seed=3),
          Tensor(2 * 48 * 80, 32, "bf16", shape=(2, 48, 80), codes=True, copy=True, seed=4),
          Tensor(7, 8, "f32", shift=1, seed=5), Tensor(0, 32, seed=6)]
    run(ts, steps=(3, 4), seed=123456789, grad_scale=1.7)


def test_more_tensors_than_a_launch_takes():
    ts = [Tensor(1 + 37 * i % 500, 8 if i % 3 == 0 else 32, seed=i) for i in range(600)]
    run(ts, steps=(2,))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("E,K,N", [(1, 16, 16), (2, 144, 128), (3, 128, 272), (1, 272, 384),
                                   (5, 16, 640), (1, 1040, 144), (2, 256, 2048)])
@pytest.mark.parametrize("shift", [0, 1])
def test_codes(bits, E, K, N, shift):
    """The weights' 8-bit codes and channel scales: whole and partial tiles, with 8-bit blocks that
    cross rows (N no multiple of 128), and off the 16-byte boundary."""
    t = Tensor(E * K * N, bits, shape=(E, K, N), codes=True, shift=shift, seed=K + N)
    t.p.reshape(E, K, N)[0, :, N // 2] = 0          # a channel of zeros, but for its update
    t.d["p"].copy_(torch.from_numpy(t.p).view(E, K, N))
    run([t], steps=(1, 2))


def test_codes_of_zero_channels_and_nan():
    E, K, N = 1, 32, 16
    t = Tensor(E * K * N, shape=(E, K, N), codes=True, zero=True)
    w = t.d["p"]
    w.zero_()
    w[0, 3, 5] = float("nan")
    w[0, 4, 6] = float("inf")
    t.d["g"].zero_()
    fb.adamw_step(plan_of([t]), grads_of([t]), step=1, **HYPER)
    scale, codes = t.d["scale"][0], t.d["codes"][0]
    tiny = torch.tensor(1e-12).div(torch.tensor(448.0))
    keep = [c for c in range(N) if c not in (5, 6)]
    assert (scale[keep].cpu() == tiny).all() and not codes[:, keep].any()
    assert torch.isnan(scale[5]) and (codes[:, 5] == 0x7F).all() and torch.isinf(scale[6])
    assert codes[4, 6] == 0x7F and not codes[5:, 6].any()


@pytest.mark.parametrize("bits", [32, 8])
def test_against_the_formula(bits):
    """64 bits. m and v: two products and a sum, each rounded (an error of 2^-24 of each term's
    size, and of the sum); p: besides, the quotient, root and rates: below 12 of these."""
    t = Tensor(20000, bits, seed=9)
    m, v = t.m, t.v
    if bits == 8:
        m = ref.decode(m, t.m_scale).astype(np.float64)
        v = np.square(ref.decode(v, t.v_scale).astype(np.float64))
    want = ref.adamw_64(t.p, t.g, m, v, 17, decay=DECAY, **HYPER)
    fb.adamw_step(plan_of([t]), grads_of([t]), step=17, **HYPER)
    U = 2.0 ** -24
    p = t.d["p"].double().cpu().numpy()
    assert (np.abs(p - want[0]) <= 14 * U * want[3]).all()
    if bits == 32:
        assert (np.abs(t.d["m"].double().cpu().numpy() - want[1]) <= 4 * U * want[4]).all()
        assert (np.abs(t.d["v"].double().cpu().numpy() - want[2]) <= 6 * U * want[2]).all()


def test_eight_bit_moments_keep_their_mean():
    """Rounded by chance, the moments' error over many seeds is without a bias: the mean of S
    draws is within 6 deviations of sqrt(gap^2 / 4 / S), and never outside the two codes."""
    n, S = 1024, 400
    t = Tensor(n, 8, seed=4)
    start = {k: t.d[k].clone() for k in ("m", "v", "m_scale", "v_scale", "p")}
    old_m = ref.decode(t.m, t.m_scale)
    old_r = ref.decode(t.v, t.v_scale)
    _, m, _, r = ref.adamw(t.p, t.g, old_m, old_r * old_r, 10, decay=DECAY, **HYPER)
    plan = plan_of([t])
    sums = {"m": np.zeros(n), "v": np.zeros(n)}
    for seed in range(S):
        for k, x in start.items():
            t.d[k].copy_(x)
        fb.adamw_step(plan, grads_of([t]), step=10, seed=seed, **HYPER)
        for k in sums:
            codes = t.d[k].cpu().numpy()
            sums[k] += ref.E4M3[codes] * np.repeat(t.d[k + "_scale"].cpu().numpy(), 128)
    for k, true in (("m", m), ("v", r)):
        scale = np.repeat(t.d[k + "_scale"].cpu().numpy(), 128).astype(np.float64)
        x = np.abs(true.astype(np.float64)) / scale
        gap = scale * np.maximum(2.0 ** -9, 2.0 ** (np.floor(np.log2(np.maximum(x, 1e-30))) - 3))
        off = np.abs(sums[k] / S - true)
        if k == "v":                                # rounded up where zero would be: not unbiased
            off = off[x >= 2.0 ** -9]
            gap = gap[x >= 2.0 ** -9]
        assert (off <= 6 * gap / 2 / S ** 0.5 + 1e-4 * gap).all()


def test_small_changes_are_not_lost_in_eight_bits():
    """A gradient that stops: both moments fade by their rates although a step changes them by
    less than half a code's spacing (v by 0.1 %): after 1500 steps sqrt(v) is at 0.999^750 = 0.47
    of its value. A mean over 4096 values whose codes walk with steps of up to an eighth."""
    n = 4096
    p, g = torch.zeros(n, device="cuda"), torch.ones(n, device="cuda")
    g += torch.rand(n, device="cuda")
    u8 = lambda: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    f = lambda: torch.zeros(n // 128, device="cuda")  # noqa: E731
    m, v, ms, vs = u8(), u8(), f(), f()
    plan = fb.AdamwPlan([p], [m], [v], m_scales=[ms], v_scales=[vs])
    value = lambda c, s: (c.view(torch.float8_e4m3fn).float().view(-1, 128) * s[:, None])  # noqa
    fb.adamw_step(plan, [g], step=1, **HYPER)
    first = value(v, vs).double().mean()
    zero = torch.zeros(n, device="cuda")
    for s in range(2, 1502):
        fb.adamw_step(plan, [zero], step=s, **HYPER)
    got = float(value(v, vs).double().mean() / first)
    assert abs(got - 0.999 ** 750) <= 0.06 * 0.47
    assert float(value(m, ms).abs().max()) <= 1e-6      # 0.9^1500 of it is nothing


def test_second_moments_never_become_zero():
    """Next to a large one in its block a small second moment keeps the smallest code."""
    n = 128
    t = Tensor(n, 8, zero=True)
    g = torch.full((n,), 1e-9, device="cuda")
    g[0] = 1.0
    g[5] = 0.0
    plan = plan_of([t])
    for s in range(1, 6):
        fb.adamw_step(plan, [g], step=s, **HYPER)
    codes = t.d["v"].cpu().tolist()
    assert codes[5] == 0 and codes[0] == 0x7E and all(c == 1 for c in codes[6:])
    assert torch.isfinite(t.d["p"]).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_infinite_and_nan_gradients(bits):
    """They spoil their own value at once; 8-bit moments of their block in the next step; nothing
    else."""
    t = Tensor(1000, bits, seed=2)
    keep = t.d["g"].clone()
    t.d["g"][300] = float("nan")
    t.d["g"][700] = float("inf")
    plan = plan_of([t])
    fb.adamw_step(plan, grads_of([t]), step=3, **HYPER)
    good = torch.ones(1000, dtype=torch.bool)
    good[[300, 700]] = False
    assert torch.isfinite(t.d["p"]).cpu().equal(good)
    t.d["g"].copy_(keep)
    fb.adamw_step(plan, grads_of([t]), step=4, **HYPER)
    if bits == 8:
        good[256:384] = False
        good[640:768] = False
        assert not torch.isfinite(t.d["p"])[256:384].any()
    assert torch.isfinite(t.d["p"]).cpu()[good].all()


def test_extreme_values():
    """Moments below the scales' range are zero; huge and tiny gradients stay in line with f32."""
    for scale in (1e-38, 1e-30, 1e-20, 1e-18, 1e-17, 1e-16, 1e-15, 1e-14, 1e-13, 1e9, 1e15, 1e18):
        for bits in (32, 8):
            t = Tensor(2000, bits, zero=True)
            t.g = numbers(2000, 5, 1) * F(scale)
            t.d["g"].copy_(torch.from_numpy(t.g))
            run([t], steps=(1, 2))


def test_params_without_a_gradient_stay():
    ts = [Tensor(300, b, copy=True, seed=b) for b in (32, 8)]
    before = [{k: x.clone() for k, x in t.d.items() if x is not None} for t in ts]
    fb.adamw_step(plan_of(ts), [None, None], step=1, **HYPER)
    other = Tensor(300, 8, seed=50)
    plan = plan_of(ts + [other])
    fb.adamw_step(plan, [None, None, other.d["g"]], step=1, **HYPER)
    for t, b in zip(ts, before):
        for k, x in b.items():
            assert torch.equal(t.d[k], x), k
    other.step(2, 1)                # its number in the call counts the ones without
    other.check()
    # and with them again
    fb.adamw_step(plan, grads_of(ts) + [None], step=2, **HYPER)
    for i, t in enumerate(ts):
        t.step(i, 2)
        t.check()


def test_two_threads_step_one_plan():
    """Each thread has the gradients of every other param: a call's gradients stay its own."""
    ts = [Tensor(50 + i, 8 if i % 4 > 1 else 32, seed=i) for i in range(64)]
    plan, steps, errors = plan_of(ts), range(1, 21), []
    torch.cuda.synchronize()

    def work(half):
        try:
            grads = [t.d["g"] if i % 2 == half else None for i, t in enumerate(ts)]
            for s in steps:
                fb.adamw_step(plan, grads, step=s, **HYPER)
        except Exception as e:                  # noqa: BLE001 - shown by the assertion below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(half,)) for half in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for i, t in enumerate(ts):
        for s in steps:
            t.step(i, s)
        t.check()


def test_weight_decay_of_each():
    ts = [Tensor(200, seed=i) for i in range(3)]
    decays = [0.0, 0.5, 0.01]
    fb.adamw_step(plan_of(ts, decays), grads_of(ts), step=4, **HYPER)
    for i, t in enumerate(ts):
        t.step(i, 4, decay=decays[i])
        t.check()


def test_step_and_rate_on_the_device_captured():
    """A captured step follows the step number, the rate, the gradient's scale and the gradients
    that it finds; a workspace of its own makes two graphs independent."""
    ts = [[Tensor(5000, 8, "bf16", copy=True, seed=1 + i),
           Tensor(2 * 64 * 128, 32, shape=(2, 64, 128), codes=True, seed=2 + i)] for i in range(2)]
    graphs = []
    for group in ts:
        step = torch.zeros(1, dtype=torch.int64, device="cuda")
        lr = torch.zeros(1, device="cuda")
        gs = torch.ones(1, device="cuda")
        plan = plan_of(group)
        hyper = {**HYPER, "lr": lr}
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step += 1
            fb.adamw_step(plan, grads_of(group), step=step, grad_scale=gs, seed=5, **hyper)
        graphs.append((graph, step, lr, gs))
    for s in (1, 2, 3):
        for (graph, _, lr, gs), group in zip(graphs, ts):
            lr.fill_(HYPER["lr"] * s)
            gs.fill_(0.5 * s)
            graph.replay()
    torch.cuda.synchronize()
    for group in ts:
        for s in (1, 2, 3):
            rate = float(F(HYPER["lr"] * s))
            for i, t in enumerate(group):
                with pytest.MonkeyPatch.context() as mp:
                    mp.setitem(HYPER, "lr", rate)
                    t.step(i, s, 5, 0.5 * s)
        for t in group:
            t.check()


def test_on_a_side_stream():
    a, b = Tensor(100000, 8, seed=1), Tensor(100000, 32, seed=2)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in (1, 2, 3):
        for t, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                fb.adamw_step(plan_of([t]), grads_of([t]), step=s, **HYPER)
    torch.cuda.synchronize()
    for t in (a, b):
        for s in (1, 2, 3):
            t.step(0, s)
        t.check()


def test_more_than_two_to_the_32_values():
    """Places past 32 bits, in both mappings: the last values are as the reference has them."""
    n = 2 ** 32 + 300
    p = torch.zeros(n, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    ms, vs = (torch.zeros(fb.adamw_blocks(n), device="cuda") for _ in range(2))
    first = 2 ** 32 - 4096                           # whole blocks from here on
    t = Tensor(n - first, 8, "bf16", zero=True, seed=1)
    p[first:], g[first:] = t.d["p"], t.d["g"]
    plan = fb.AdamwPlan([p], [m], [v], m_scales=[ms], v_scales=[vs], weight_decay=DECAY)
    fb.adamw_step(plan, [g], step=2, seed=3, **HYPER)
    _, mm, _, r = ref.adamw(t.p, t.g, np.zeros(t.n, F), np.zeros(t.n, F), 2, decay=DECAY, **HYPER)
    bits = ref.random_bits(t.n, 0, 2, 3, first=first)
    codes, scale = ref.encode(mm, bits & np.uint32(0xFFFF), False)
    assert np.array_equal(m[first:].cpu().numpy(), codes)
    assert np.array_equal(ms[first // 128:].cpu().numpy(), scale)
    codes, scale = ref.encode(r, bits >> np.uint32(16), True)
    assert np.array_equal(v[first:].cpu().numpy(), codes)
    assert not m[:first].any() and not p[:first].any()
