"""The norms around a block, forward and backward, against 64-bit forms on the GPU."""
import pytest
import torch

import layer_reference as ref
from fp8_moe_routed_gb300 import binding as fb

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


def make(T, H, dtype, parts, gate, seed):
    g = torch.Generator().manual_seed(seed)
    post, pre = parts != "pre", parts != "post"
    d = {"x": torch.randn(T, H, generator=g).to(dtype), "y": None, "w_post": None, "w_pre": None,
         "gate": None}
    if post:
        d["y"] = (torch.randn(T, H, generator=g) * 0.3).to(dtype)
        d["w_post"] = 1 + 0.3 * torch.randn(H, generator=g)
        shape = {None: None, "token": (T,), "channel": (H,), "full": (T, H)}[gate]
        if shape is not None:
            d["gate"] = torch.randn(*shape, generator=g).to(dtype if gate == "full" else F32)
    if pre:
        d["w_pre"] = 1 + 0.3 * torch.randn(H, generator=g)
    d["dr"] = torch.randn(T, H, generator=g).to(dtype)
    d["dh"] = torch.randn(T, H, generator=g).to(dtype) if pre else None
    return d


def cuda(v):
    return None if v is None else v.cuda()


def dbl(v):
    return None if v is None else v.double()


def scales(d):
    return (0.9, 0.7) if d["y"] is not None else (1.0, 1.0)


def forward(d, kind, sigmoid):
    a, b = scales(d)
    return fb.norm_fwd(cuda(d["x"]), cuda(d["y"]), cuda(d["w_post"]), cuda(d["w_pre"]),
                       gate=cuda(d["gate"]), gate_kind=kind, sigmoid=sigmoid, residual_scale=a,
                       branch_scale=b, eps=EPS)


def reference(d, kind, sigmoid):
    a, b = scales(d)
    return ref.norm_fwd(dbl(d["x"]), dbl(d["y"]), dbl(d["w_post"]), dbl(d["w_pre"]),
                        dbl(d["gate"]), kind, sigmoid, a, b, EPS)


CASES = [  # T, H, type, parts, gate, sigmoid
    (1, 7168, BF16, "both", "channel", False), (7, 7168, BF16, "both", "token", True),
    (200, 8, BF16, "both", "full", True), (1000, 128, BF16, "both", None, False),
    (333, 520, BF16, "both", "channel", True), (19, 8192, BF16, "both", "full", False),
    (5, 16384, BF16, "both", "token", False), (311, 1544, F32, "both", "full", True),
    (40, 4, F32, "both", "channel", True), (170, 8192, F32, "both", "token", False),
    (321, 2056, F32, "both", None, False), (450, 1032, BF16, "pre", None, False),
    (33, 7168, F32, "pre", None, False), (450, 1032, BF16, "post", "token", False),
    (160, 776, F32, "post", "channel", True), (3, 4104, BF16, "post", None, False),
    (600, 2048, F32, "both", "token", True), (400, 16384, BF16, "both", "full", True),
    (330, 8192, F32, "both", "full", False), (310, 16384, BF16, "both", "channel", False),
]


@pytest.mark.parametrize("T,H,dtype,parts,gate,sigmoid", CASES)
def test_forward(T, H, dtype, parts, gate, sigmoid):
    d = make(T, H, dtype, parts, gate, seed=T + H)
    r, h, rstd_post, rstd_pre = forward(d, gate, sigmoid)
    want_r, want_h = reference(d, gate, sigmoid)
    if parts == "pre":
        assert r is None and rstd_post is None
    else:
        ref.check_rows(r, want_r, "r")
        ref.check_f32(rstd_post, 1 / torch.sqrt(dbl(d["y"]).square().mean(1) + EPS), "rstd_post")
    if parts == "post":
        assert h is None and rstd_pre is None
    else:
        ref.check_rows(h, want_h, "h")
        ref.check_f32(rstd_pre, 1 / torch.sqrt(want_r.square().mean(1) + EPS), "rstd_pre")


def gradients(d, kind, sigmoid, r):
    """64-bit gradients by the definition's derivative. For bf16 rows the backward's
    inputs are the rounded r, so h is taken as a function of that r."""
    a, b = scales(d)
    leaves = {k: dbl(d[k]).requires_grad_() for k in ("x", "y", "w_post", "w_pre", "gate")
              if d[k] is not None}
    get = leaves.get
    out = ref.norm_fwd(get("x"), get("y"), get("w_post"), None if get("y") is not None else
                       get("w_pre"), get("gate"), kind, sigmoid, a, b, EPS)
    if get("y") is None:
        loss = (out[1] * dbl(d["dh"])).sum() + (out[0] * dbl(d["dr"])).sum()
        loss.backward()
        return {k: v.grad for k, v in leaves.items()}
    D = dbl(d["dr"])
    if get("w_pre") is not None:
        rr = dbl(r.cpu()).requires_grad_()
        h = ref.norm_fwd(rr, None, None, get("w_pre"), None, None, False, 1, 1, EPS)[1]
        (h * dbl(d["dh"])).sum().backward()
        D = D + rr.grad
    (out[0] * D).sum().backward()
    return {k: v.grad for k, v in leaves.items()}


@pytest.mark.parametrize("T,H,dtype,parts,gate,sigmoid", CASES)
def test_backward(T, H, dtype, parts, gate, sigmoid):
    d = make(T, H, dtype, parts, gate, seed=T + 2 * H)
    a, b = scales(d)
    r, _, rstd_post, _ = forward(d, gate, sigmoid)
    rin = r if r is not None else cuda(d["x"])
    # rstd of the r that the backward reads (the forward's is of r before rounding)
    rstd_pre = None
    if d["w_pre"] is not None:
        rstd_pre = (1 / torch.sqrt(rin.double().square().mean(1) + EPS)).float()
    got = fb.norm_bwd(cuda(d["dr"]), cuda(d["dh"]), rin, cuda(d["y"]), cuda(d["w_post"]),
                      cuda(d["w_pre"]), rstd_post, rstd_pre, gate=cuda(d["gate"]), gate_kind=gate,
                      sigmoid=sigmoid, residual_scale=a, branch_scale=b)
    want = gradients(d, gate, sigmoid, rin)
    for name, g in zip(("x", "y", "w_post", "w_pre", "gate"), got):
        if name in want:
            check = ref.check_rows if g.dim() == 2 else ref.check_f32
            check(g, want[name], "d" + name)
        else:
            assert g is None


@pytest.mark.parametrize("gate,sigmoid", [(None, False), ("token", True), ("channel", True),
                                          ("full", False)])
def test_backward_against_differences(gate, sigmoid):
    """Directional central differences of the 64-bit forward against f32 gradients."""
    T, H = 37, 264
    d = make(T, H, F32, "both", gate, seed=9)
    a, b = scales(d)
    r, _, rstd_post, rstd_pre = forward(d, gate, sigmoid)
    got = fb.norm_bwd(cuda(d["dr"]), cuda(d["dh"]), r, cuda(d["y"]), cuda(d["w_post"]),
                      cuda(d["w_pre"]), rstd_post, rstd_pre, gate=cuda(d["gate"]), gate_kind=gate,
                      sigmoid=sigmoid, residual_scale=a, branch_scale=b)
    g = torch.Generator().manual_seed(4)
    for name, grad in zip(("x", "y", "w_post", "w_pre", "gate"), got):
        if d[name] is None:
            continue
        v = torch.randn(d[name].shape, generator=g).double()
        v = v / v.norm()
        ends = []
        for s in (1e-5, -1e-5):
            moved = dict(d)
            moved[name] = dbl(d[name]) + s * v
            rr, h = ref.norm_fwd(dbl(moved["x"]), dbl(moved["y"]), dbl(moved["w_post"]),
                                 dbl(moved["w_pre"]), dbl(moved["gate"]), gate, sigmoid, a, b, EPS)
            ends.append((rr * dbl(d["dr"])).sum() + (h * dbl(d["dh"])).sum())
        slope = (ends[0] - ends[1]) / 2e-5
        have = (grad.cpu().double() * v).sum()
        # f32 gradients: 1e-5 of the terms; differences: step^2 and 2^-52 * |L| / step
        tol = 1e-5 * (grad.cpu().double() * v).abs().sum() + 1e-6 * max(1.0, abs(float(slope)))
        assert abs(have - slope) <= tol, (name, float(have), float(slope))


def test_backward_without_stream_gradient():
    """dr = None is a zero gradient."""
    d = make(50, 256, F32, "both", "token", seed=2)
    r, _, rp, rq = forward(d, "token", False)
    args = (r, cuda(d["y"]), cuda(d["w_post"]), cuda(d["w_pre"]), rp, rq)
    kw = dict(gate=cuda(d["gate"]), gate_kind="token", residual_scale=0.9, branch_scale=0.7)
    one = fb.norm_bwd(None, cuda(d["dh"]), *args, **kw)
    two = fb.norm_bwd(torch.zeros_like(r), cuda(d["dh"]), *args, **kw)
    for p, q in zip(one, two):
        assert torch.equal(p, q)


def test_rows_do_not_touch_each_other():
    """A row of NaN or infinity stays alone; a zero row gives rstd = 1/sqrt(eps) and zeros."""
    x = torch.randn(64, 512).to(BF16)
    y = torch.randn(64, 512).to(BF16)
    x[5], y[9], x[20], y[20] = float("nan"), float("inf"), 0.0, 0.0
    w = torch.ones(512)
    r, h, rp, rq = fb.norm_fwd(x.cuda(), y.cuda(), w.cuda(), w.cuda(), eps=EPS)
    keep = [i for i in range(64) if i not in (5, 9)]
    assert torch.isfinite(r[keep]).all() and torch.isfinite(h[keep]).all()
    assert torch.isnan(h[5]).all() and torch.isnan(h[9]).all()
    assert (h[20] == 0).all() and abs(float(rp[20]) - 1000.0) < 0.01


def test_no_rows_and_repeats():
    e = torch.empty(0, 64, dtype=BF16, device="cuda")
    w = torch.ones(64, device="cuda")
    z = torch.empty(0, device="cuda")
    r, h, _, _ = fb.norm_fwd(e, e, w, w)
    assert r.shape == h.shape == (0, 64)
    got = fb.norm_bwd(e, e, e, e, w, w, z, z, gate=w, gate_kind="channel")
    assert (got[2] == 0).all() and (got[3] == 0).all() and (got[4] == 0).all()
    # the same bits from run to run
    d = make(3000, 1024, BF16, "both", "channel", seed=1)
    r, _, rp, rq = forward(d, "channel", True)
    run = lambda: fb.norm_bwd(cuda(d["dr"]), cuda(d["dh"]), r, cuda(d["y"]), cuda(d["w_post"]),
                              cuda(d["w_pre"]), rp, rq, gate=cuda(d["gate"]),
                              gate_kind="channel", sigmoid=True)
    for p, q in zip(run(), run()):
        assert torch.equal(p, q)
    assert fb.read_status() == 0


def test_refusals():
    x = torch.zeros(4, 64, dtype=BF16, device="cuda")
    w = torch.ones(64, device="cuda")
    t = torch.ones(4, device="cuda")
    with pytest.raises(TypeError):
        fb.norm_fwd(x.half(), None, None, w)
    with pytest.raises(TypeError):
        fb.norm_fwd(x, None, None, w.to(BF16))
    with pytest.raises(ValueError):
        fb.norm_fwd(x, x, None, w)                         # y without its weight
    with pytest.raises(ValueError):
        fb.norm_fwd(x, x[:, :32], w, w)
    with pytest.raises(ValueError):
        fb.norm_fwd(x, x, w, w, gate=t)                    # kind not named
    with pytest.raises(ValueError):
        fb.norm_fwd(x, x, w, w, gate=t, gate_kind="channel")
    with pytest.raises(ValueError):
        fb.norm_fwd(x, None, None, w, gate=t, gate_kind="token")
    with pytest.raises(fb.Fp8MoeError, match="EINVAL"):
        fb.norm_fwd(x)                                     # nothing to do
    for eps in (-1e-6, float("nan")):
        with pytest.raises(fb.Fp8MoeError, match="EINVAL"):
            fb.norm_fwd(x, None, None, w, eps=eps)
    with pytest.raises(fb.Fp8MoeError, match="EALIGN"):
        fb.norm_fwd(torch.zeros(4, 12, dtype=BF16, device="cuda"), None, None,
                    torch.ones(12, device="cuda"))
    with pytest.raises(fb.Fp8MoeError, match="EINVAL"):
        fb.norm_fwd(torch.zeros(1, 16392, dtype=BF16, device="cuda"), None, None,
                    torch.ones(16392, device="cuda"))
    with pytest.raises(ValueError):
        fb.norm_bwd(None, None, x, None, None, w, None, t)
    with pytest.raises(ValueError):
        fb.norm_bwd(x, x, None, None, None, w, None, t)    # r missing
    with pytest.raises(fb.Fp8MoeError, match="EWORKSPACE"):
        fb.norm_bwd(x, x, x, None, None, w, None, t,
                    workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
