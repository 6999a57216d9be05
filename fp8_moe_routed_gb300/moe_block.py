"""One mixture-of-experts block around the routed experts, from the library's calls:

    ids, weights = the router's choice for the normalised tokens h   (the caller's)
    rows         = h sorted by expert                                 dispatch_tokens
    y            = the experts' SwiGLU MLP on the rows                the grouped products
    out          = the weighted sum of each token's rows              combine_tokens
    r, h'        = residual sum with the norms after and before       norm_fwd

`forward` and `backward` are the training step on 8-bit weights, `serve` the block on
4-bit weights. Run as a module for a small demonstration on a GPU:

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


def main() -> None:
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
