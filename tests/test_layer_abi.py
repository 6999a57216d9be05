"""Host-side argument checks of the token, norm and MXFP4 entry points (no GPU: every
refusal comes before any device call), and the 64-bit forms against themselves."""
import ctypes

import pytest
import torch

import layer_reference as ref
from fp8_moe_routed_gb300 import binding as fb

P = ctypes.c_void_p
EINVAL, EALIGN, EWORKSPACE = -1, -2, -3


def test_workspace_sizes():
    M, K = 1000, 7168
    words = M * 56 * 4
    for op in (fb.OP_GMM_MXFP4_FWD, fb.OP_GMM_SILU_MXFP4_FWD):
        assert fb.workspace_size(op, M, K, 4096, 32) == M * K // 2 + words
    assert fb.workspace_size(fb.OP_GMM_MXFP4_FWD, 3, 32, 16, 1) == 256 + 256
    assert fb.workspace_size(fb.OP_NORM_BWD, 4096, K, 0, 0) == 2 * 256 * K * 4
    assert fb.workspace_size(fb.OP_NORM_BWD, 5, K, 0, 0) == 2 * 5 * K * 4
    assert fb.workspace_size(fb.OP_NORM_BWD, 0, K, 0, 0) == 0


def sort(L, ids=16, T=4, k=2, E=8, M=8, gs=16, sr=16, rs=16):
    return L.fp8moe_sort_tokens(P(ids), T, k, E, M, P(gs), P(sr), P(rs), None)


def dispatch(L, x=16, ids=16, T=4, k=2, H=64, ty=0, E=8, M=8, rows=16):
    return L.fp8moe_dispatch_tokens(P(x), P(ids), T, k, H, ty, E, M, P(rows), P(16), P(16), P(16),
                                    None)


def combine(L, rows=16, M=8, H=64, ty=0, sr=16, w=16, T=4, k=2, out=16):
    return L.fp8moe_combine_tokens(P(rows), M, H, ty, P(sr), P(w), T, k, P(out), None)


def combine_bwd(L, dout=16, rows=16, M=8, H=64, ty=0, sr=16, w=16, T=4, k=2, drows=16, dw=16):
    return L.fp8moe_combine_tokens_bwd(P(dout), P(rows), M, H, ty, P(sr), P(w), T, k, P(drows),
                                       P(dw), None)


@pytest.mark.parametrize("call,bad,code", [
    (sort, dict(T=-1), EINVAL), (sort, dict(k=0), EINVAL), (sort, dict(k=33), EINVAL),
    (sort, dict(E=0), EINVAL), (sort, dict(E=1025), EINVAL), (sort, dict(M=-1), EINVAL),
    (sort, dict(M=2 ** 31), EINVAL), (sort, dict(T=2 ** 30, k=2), EINVAL),
    (sort, dict(ids=0), EINVAL), (sort, dict(gs=0), EINVAL), (sort, dict(sr=0), EINVAL),
    (sort, dict(ids=18), EALIGN), (sort, dict(rs=17), EALIGN),
    (dispatch, dict(ty=2), EINVAL), (dispatch, dict(H=0), EINVAL), (dispatch, dict(H=12), EALIGN),
    (dispatch, dict(H=6, ty=1), EALIGN), (dispatch, dict(x=0), EINVAL),
    (dispatch, dict(rows=8), EALIGN), (dispatch, dict(rows=0), EINVAL),
    (combine, dict(ty=-1), EINVAL), (combine, dict(out=0), EINVAL), (combine, dict(rows=0), EINVAL),
    (combine, dict(w=2), EALIGN), (combine, dict(out=24), EALIGN), (combine, dict(T=0), 0),
    (combine_bwd, dict(w=0), EINVAL), (combine_bwd, dict(dw=0), EINVAL),
    (combine_bwd, dict(drows=0), EINVAL), (combine_bwd, dict(dout=20), EALIGN),
    (combine_bwd, dict(T=0), 0),
])
def test_token_refusals(call, bad, code):
    assert call(fb.load(), **bad) == code


def norm_fwd(L, x=16, y=16, T=4, H=64, ty=0, wp=16, wq=16, gate=0, kind=0, sig=0, r=16, h=16,
             rp=16, rq=16):
    return L.fp8moe_norm_fwd(P(x), P(y), T, H, ty, P(wp), P(wq), P(gate), kind, sig, 1.0, 1.0, 1e-6,
                             P(r), P(h), P(rp), P(rq), None)


def norm_bwd(L, dr=16, dh=16, r=16, y=16, T=4, H=64, ty=0, wp=16, wq=16, rp=16, rq=16, gate=0,
             kind=0, sig=0, dx=16, dy=16, dwp=16, dwq=16, dg=0, ws=256, wsb=1 << 30):
    return L.fp8moe_norm_bwd(P(dr), P(dh), P(r), P(y), T, H, ty, P(wp), P(wq), P(rp), P(rq),
                             P(gate), kind, sig, 1.0, 1.0, P(dx), P(dy), P(dwp), P(dwq), P(dg),
                             P(ws), wsb, None)


@pytest.mark.parametrize("call,bad,code", [
    (norm_fwd, dict(T=-1), EINVAL), (norm_fwd, dict(H=0), EINVAL), (norm_fwd, dict(H=20), EALIGN),
    (norm_fwd, dict(H=16392), EINVAL), (norm_fwd, dict(H=8196, ty=1), EINVAL),
    (norm_fwd, dict(ty=3), EINVAL), (norm_fwd, dict(kind=4), EINVAL), (norm_fwd, dict(sig=2), EINVAL),
    (norm_fwd, dict(wp=0, wq=0), EINVAL), (norm_fwd, dict(wp=0), EINVAL),
    (norm_fwd, dict(kind=1), EINVAL), (norm_fwd, dict(gate=16), EINVAL),
    (norm_fwd, dict(y=0), EINVAL), (norm_fwd, dict(h=0), EINVAL), (norm_fwd, dict(rq=0), EINVAL),
    (norm_fwd, dict(kind=2, gate=20), EALIGN), (norm_fwd, dict(kind=1, gate=18), EALIGN),
    (norm_fwd, dict(x=8), EALIGN), (norm_fwd, dict(T=0), 0),
    (norm_bwd, dict(dh=0), EINVAL), (norm_bwd, dict(r=0), EINVAL), (norm_bwd, dict(dx=0), EINVAL),
    (norm_bwd, dict(dy=0), EINVAL), (norm_bwd, dict(dwq=0), EINVAL),
    (norm_bwd, dict(kind=2, gate=16), EINVAL), (norm_bwd, dict(wq=0), EINVAL),
    (norm_bwd, dict(wq=0, dh=0, dr=0), EINVAL), (norm_bwd, dict(ws=0), EWORKSPACE),
    (norm_bwd, dict(wsb=100), EWORKSPACE), (norm_bwd, dict(ws=16), EALIGN),
    (norm_bwd, dict(dy=12), EALIGN),
])
def test_norm_refusals(call, bad, code):
    assert call(fb.load(), **bad) == code


def gmm(L, x=16, M=8, K=64, c=16, s=16, E=2, N=32, gs=16, out=16, ws=256, wsb=1 << 30, silu=False):
    f = L.fp8moe_gmm_silu_mxfp4_fwd if silu else L.fp8moe_gmm_mxfp4_fwd
    return f(P(x), M, K, P(c), P(s), E, N, P(gs), P(out), P(ws), wsb, None)


@pytest.mark.parametrize("bad,code", [
    (dict(K=48), EALIGN), (dict(N=24), EALIGN), (dict(N=16, silu=True), EALIGN),
    (dict(E=0), EINVAL), (dict(M=-1), EINVAL), (dict(M=0), 0), (dict(x=0), EINVAL),
    (dict(s=0), EINVAL), (dict(c=8), EALIGN), (dict(s=8), EALIGN), (dict(ws=0), EWORKSPACE),
    (dict(ws=16), EALIGN), (dict(wsb=64), EWORKSPACE),
])
def test_mxfp4_product_refusals(bad, code):
    assert gmm(fb.load(), **bad) == code


def test_mxfp4_quantiser_refusals():
    L = fb.load()
    assert L.fp8moe_mxfp4_quantize_rows(P(16), 4, 48, P(16), 1, P(16), P(16), None) == EALIGN
    assert L.fp8moe_mxfp4_quantize_rows(P(16), 4, 64, None, 1, P(16), P(16), None) == EINVAL
    assert L.fp8moe_mxfp4_quantize_rows(P(16), 0, 64, None, 1, None, None, None) == 0
    assert L.fp8moe_mxfp4_quantize_weights(P(16), 1, 64, 8, P(16), P(16), None) == EALIGN
    assert L.fp8moe_mxfp4_quantize_weights(None, 1, 64, 16, P(16), P(16), None) == EINVAL
    assert L.fp8moe_mxfp4_dequantize(P(16), P(8), 1, 16, 64, P(16), None) == EALIGN
    assert L.fp8moe_mxfp4_dequantize(P(16), P(16), 1025, 16, 64, P(16), None) == EINVAL


def test_reference_quantiser_by_hand():
    """Values whose codes are known from the format's table."""
    v = torch.zeros(1, 32, dtype=torch.float64)
    v[0, :9] = torch.tensor([6.0, 5.0, 2.5, 1.25, 0.25, -3.5, 0.75, 7.9, -0.2])
    codes, byte = ref.mx_quantize(v)
    assert int(byte) == 127                               # floor(log2 7.9) = 2: X = 1
    assert codes[0, :9].tolist() == [7, 6, 4, 2, 0, 8 + 6, 2, 7, 8]
    assert ref.mx_values(codes, byte)[0, :4].tolist() == [6.0, 4.0, 2.0, 1.0]
    v[0, 0] = float("inf")
    codes, byte = ref.mx_quantize(v)
    assert int(byte) == 255 and int(codes.max()) == 0


def test_reference_sort_by_hand():
    ids = torch.tensor([[2, 0], [0, -1], [1, 2]], dtype=torch.int32)
    assert ref.sort_tokens(ids, 3, 6) == ([2, 1, 2], [3, 0, 1, -1, 2, 4], [1, 2, 4, 0, 5, -1])
    assert ref.sort_tokens(ids, 3, 2) == ([2, 0, 0], [-1, 0, 1, -1, -1, -1], [1, 2])
