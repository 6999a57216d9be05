"""One mixture-of-experts block around the routed experts, from the library's calls:

    ids, weights = the router's choice for the normalised tokens h   (the caller's)
    rows         = h sorted by expert                                 dispatch_tokens
    y            = the experts' SwiGLU MLP on the rows                the grouped products
    out          = the weighted sum of each token's rows              combine_tokens
    r, h'        = residual sum with the norms after and before       norm_fwd

`forward` and `backward` are the training pass on 8-bit weights, `serve` the block on
4-bit weights. `choose` and `choose_backward` are the router in front of it with its balance
loss (router_fwd, router_bwd), and `Trainer` holds the f32 weights and their moments and turns
the gradients into the next weights, the experts' as 8-bit codes (adamw_step); `train_step` is
all of them together. Run as a module for a small demonstration on a GPU:

    python -m fp8_moe_routed_gb300.moe_block
"""
from __future__ import annotations

import dataclasses
from typing import Any, Optional

import torch

from . import binding as fb


@dataclasses.dataclass
class Params:
    """Weights of a block: `wi` [E, H, 2F] and `wo` [E, F, H] as (codes, scales) pairs,
    8-bit (codes and per-channel scales) or 4-bit (mxfp4_quantize_weights), the norms'
    f32 weights, and a gate of the block's output (None, or f32 logits per channel)."""
    wi: tuple
    wo: tuple
    w_post: torch.Tensor
    w_pre: torch.Tensor
    gate: Optional[torch.Tensor] = None
    residual_scale: float = 1.0
    branch_scale: float = 1.0
    eps: float = 1e-6

    def norms(self) -> dict:
        return dict(gate=self.gate, gate_kind=None if self.gate is None else "channel",
                    sigmoid=self.gate is not None, residual_scale=self.residual_scale,
                    branch_scale=self.branch_scale)


def route(h: torch.Tensor, w_router: torch.Tensor, topk: int):
    """A plain router: softmax over the chosen logits. ids int32 [T, topk], weights f32."""
    logits = h.float() @ w_router.float()
    top = torch.topk(logits, topk, dim=1)
    return top.indices.to(torch.int32).contiguous(), torch.softmax(top.values, dim=1).contiguous()


@dataclasses.dataclass
class Router:
    """Weights f32 [H, E] of the logits, an optional bias of the choice (f32 [E]), and the
    factor of the balance loss (of each sequence) in the total."""
    w: torch.Tensor
    topk: int
    score: str = "softmax"
    bias: Optional[torch.Tensor] = None
    weight_scale: float = 1.0
    balance: float = 1e-3

    def options(self) -> dict:
        return dict(score=self.score, weight_scale=self.weight_scale)


def choose(router: Router, h, seq_offsets=None):
    """The router's choice for the normalised tokens h [T, H]: (ids, weights, saved), with the
    balance loss of each sequence and the experts' counts in saved."""
    logits = h.float() @ router.w
    ids, weights, counts, loss, slope = fb.router_fwd(
        logits, router.topk, bias=router.bias, balance=True, seq_offsets=seq_offsets,
        **router.options())
    saved: dict[str, Any] = dict(h=h, logits=logits, ids=ids, counts=counts, loss=loss, slope=slope,
                                 seq_offsets=seq_offsets)
    return ids, weights, saved


def choose_backward(router: Router, saved: dict, dweights):
    """Gradients for dweights (of the router's weights) and the balance loss's own: (dh, dw)."""
    dloss = torch.full_like(saved["loss"], router.balance)
    dlogits = fb.router_bwd(dweights, saved["logits"], saved["ids"], dloss=dloss,
                            slope=saved["slope"], seq_offsets=saved["seq_offsets"],
                            **router.options())
    return dlogits @ router.w.t(), saved["h"].float().t() @ dlogits


def forward(p: Params, x, h, ids, weights):
    """x: residual stream, h: its norm (both bf16 [T, H]). Returns (r, h_next, saved)."""
    num_experts = p.wi[0].shape[0]
    rows, gs, slot_row, _ = fb.dispatch_tokens(h, ids, num_experts)
    gu = fb.gmm_fp8_fwd(rows, *p.wi, gs)
    g, u = gu.float().chunk(2, dim=1)
    act = (g * torch.sigmoid(g) * u).to(torch.bfloat16)
    y = fb.gmm_fp8_fwd(act, *p.wo, gs)
    out = fb.combine_tokens(y, slot_row, weights)
    r, h_next, rstd_post, rstd_pre = fb.norm_fwd(x, out, p.w_post, p.w_pre, eps=p.eps, **p.norms())
    saved: dict[str, Any] = dict(rows=rows, gs=gs, slot_row=slot_row, gu=gu, act=act, y=y, out=out,
                                 r=r, rstd_post=rstd_post, rstd_pre=rstd_pre, weights=weights)
    return r, h_next, saved


def backward(p: Params, saved: dict, dr, dh_next):
    """Gradients for dr (of r) and dh_next (of h_next): a dict with dx, dh (of the two
    inputs), dweights (of the router's weights) and those of the parameters."""
    s = saved
    dx, dout, dw_post, dw_pre, dgate = fb.norm_bwd(
        dr, dh_next, s["r"], s["out"], p.w_post, p.w_pre, s["rstd_post"], s["rstd_pre"], **p.norms())
    dy, dweights = fb.combine_tokens_bwd(dout, s["y"], s["slot_row"], s["weights"])
    dwo = fb.tgmm_drhs_quant(s["act"], dy, s["gs"])
    dgu = fb.gmm_dlhs_dswiglu_fp8(dy, *p.wo, s["gu"], s["gs"])
    dwi = fb.tgmm_drhs_quant(s["rows"], dgu, s["gs"])
    drows = fb.gmm_dlhs_fp8(dgu, *p.wi, s["gs"])
    dh = fb.dispatch_tokens_bwd(drows, s["slot_row"])
    return dict(dx=dx, dh=dh, dweights=dweights, dwi=dwi, dwo=dwo, dw_post=dw_post, dw_pre=dw_pre,
                dgate=dgate)


class Trainer:
    """The f32 weights behind a block and its router, with their moments in 32 or 8 bits. wi
    [E, H, 2F] and wo [E, F, H] are f32; the block's codes and scales are what they become. The
    experts and the router's weights decay, the norms and the gate do not."""

    def __init__(self, p: Params, router: Router, wi: torch.Tensor, wo: torch.Tensor, bits: int = 32,
                 weight_decay: float = 0.1, seed: int = 0):
        if bits not in (8, 32):
            raise ValueError(f"bits must be 8 or 32, got {bits}")
        self.names = ["dwi", "dwo", "dw_router", "dw_post", "dw_pre"]
        params = [wi, wo, router.w, p.w_post, p.w_pre]
        if p.gate is not None:
            self.names.append("dgate")
            params.append(p.gate)
        n = len(params)
        dtype = torch.uint8 if bits == 8 else torch.float32
        self.m = [torch.zeros(t.shape, dtype=dtype, device=t.device) for t in params]
        self.v = [torch.zeros_like(t) for t in self.m]
        scales = [[torch.zeros(fb.adamw_blocks(t.numel()), device=t.device) for t in params]
                  for _ in range(2)] if bits == 8 else [None, None]
        none = [None] * (n - 2)
        self.plan = fb.AdamwPlan(params, self.m, self.v, m_scales=scales[0], v_scales=scales[1],
                                 codes=[p.wi[0], p.wo[0]] + none,
                                 code_scales=[p.wi[1], p.wo[1]] + none,
                                 weight_decay=[weight_decay] * 3 + [0.0] * (n - 3))
        self.scales, self.seed, self.steps = scales, seed, 0
        self.p, self.router, self.held = p, router, self._weights(p, router)

    @staticmethod
    def _weights(p: Params, router: Router) -> dict:
        """What the block and its router take, by name."""
        return {"wi": p.wi[0], "the scales of wi": p.wi[1], "wo": p.wo[0],
                "the scales of wo": p.wo[1], "w_post": p.w_post, "w_pre": p.w_pre, "gate": p.gate,
                "the router's w": router.w}

    def step(self, grads: dict, lr: float, grad_scale=None) -> None:
        """One AdamW step for the gradients of backward and choose_backward. A step that is refused
        is not counted; one is refused if the block or its router have other weights than at the
        start, as they would stay as they are."""
        for name, t in self._weights(self.p, self.router).items():
            if t is not self.held[name]:
                raise ValueError(f"{name} was replaced: make a new Trainer")
        fb.adamw_step(self.plan, [grads[k] for k in self.names], step=self.steps + 1, lr=lr,
                      grad_scale=grad_scale, seed=self.seed)
        self.steps += 1


def train_step(p: Params, router: Router, trainer: Trainer, x, h, dr, dh_next, lr: float,
               seq_offsets=None):
    """The whole step for x, h and the gradients of its two results, dr and dh_next: forward,
    backward and new weights. Returns (r, h_next, losses, grads); grads["dh"] has the router's
    part, too."""
    ids, weights, chosen = choose(router, h, seq_offsets)
    r, h_next, saved = forward(p, x, h, ids, weights)
    grads = backward(p, saved, dr, dh_next)
    dh, grads["dw_router"] = choose_backward(router, chosen, grads["dweights"])
    grads["dh"] = grads["dh"].float() + dh
    trainer.step(grads, lr)
    return r, h_next, chosen["loss"], grads


def serve(p: Params, x, h, ids, weights):
    """The block on 4-bit weights: (r, h_next)."""
    num_experts = p.wi[0].shape[0]
    rows, gs, slot_row, _ = fb.dispatch_tokens(h, ids, num_experts)
    act = fb.gmm_silu_mxfp4_fwd(rows, *p.wi, gs)
    y = fb.gmm_mxfp4_fwd(act, *p.wo, gs)
    out = fb.combine_tokens(y, slot_row, weights)
    r, h_next, _, _ = fb.norm_fwd(x, out, p.w_post, p.w_pre, eps=p.eps, **p.norms())
    return r, h_next


def fp8_weight(w: torch.Tensor) -> tuple:
    """bf16 or f32 [E, K, N] as e4m3 codes and per-channel scales (input preparation)."""
    w = w.float()
    scale = (w.abs().amax(dim=1) / 448.0).clamp_min(1e-12)
    q = (w / scale[:, None, :]).clamp_(-448.0, 448.0)
    return q.to(torch.float8_e4m3fn).view(torch.uint8), scale.contiguous()


def example(T: int = 1000, H: int = 1024, F: int = 512, E: int = 16, topk: int = 4, seed: int = 0):
    """Random weights and tokens, the same in 8 and in 4 bits: (p8, p4, x, h, ids, weights)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")
    wi = (rand(E, H, 2 * F) * H ** -0.5).to(torch.bfloat16)
    wo = (rand(E, F, H) * F ** -0.5).to(torch.bfloat16)
    common = dict(w_post=1 + 0.1 * rand(H), w_pre=1 + 0.1 * rand(H), gate=rand(H))
    p8 = Params(fp8_weight(wi), fp8_weight(wo), **common)
    p4 = Params(fb.mxfp4_quantize_weights(wi), fb.mxfp4_quantize_weights(wo), **common)
    x = rand(T, H).to(torch.bfloat16)
    _, h, _, _ = fb.norm_fwd(x, w_pre=torch.ones(H, device="cuda"))
    ids, weights = route(h, rand(H, E) * H ** -0.5, topk)
    return p8, p4, x, h, ids, weights


def training_example(T: int = 1000, H: int = 1024, F: int = 512, E: int = 16, topk: int = 4,
                     bits: int = 8, seed: int = 0):
    """A block with a router and a trainer of their own: (p, router, trainer, x, h)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")
    wi, wo = rand(E, H, 2 * F) * H ** -0.5, rand(E, F, H) * F ** -0.5
    p = Params(fp8_weight(wi), fp8_weight(wo), w_post=1 + 0.1 * rand(H), w_pre=1 + 0.1 * rand(H),
               gate=rand(H))
    router = Router(rand(H, E) * H ** -0.5, topk, score="sigmoid", bias=0.01 * rand(E))
    trainer = Trainer(p, router, wi, wo, bits=bits)
    x = rand(T, H).to(torch.bfloat16)
    _, h, _, _ = fb.norm_fwd(x, w_pre=torch.ones(H, device="cuda"))
    return p, router, trainer, x, h


def main() -> None:
    p, router, trainer, x, h = training_example()
    for _ in range(2):
        r, h_next, losses, _ = train_step(p, router, trainer, x, h, 1e-3 * torch.randn_like(x),
                                          1e-3 * torch.randn_like(x), lr=1e-3)
    print(f"{trainer.steps} training steps, moments in 8 bits: balance loss {float(losses[0]):.4f}")
    p8, p4, x, h, ids, weights = example()
    r, h_next, saved = forward(p8, x, h, ids, weights)
    grads = backward(p8, saved, torch.randn_like(r), torch.randn_like(r))
    r4, h4 = serve(p4, x, h, ids, weights)
    one, _ = serve(p4, x[:1], h[:1], ids[:1], weights[:1])
    torch.cuda.synchronize()
    assert fb.read_status() == 0
    sim = torch.nn.functional.cosine_similarity(h_next.float().flatten(), h4.float().flatten(), 0)
    print(f"{x.shape[0]} tokens, {p8.wi[0].shape[0]} experts: 8-bit and 4-bit blocks agree to a "
          f"cosine of {float(sim):.4f}; one token served: {tuple(one.shape)}; gradients: "
          f"{', '.join(k for k in grads)}")


if __name__ == "__main__":
    main()
