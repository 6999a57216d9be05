"""MXFP4 quantisation and the 4-bit grouped product against 64-bit forms on the GPU."""
import pytest
import torch

import layer_reference as ref
from fp8_moe_routed_gb300 import binding as fb
from parity_util import check_bf16

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def sizes_tensor(sizes):
    return torch.tensor(sizes, dtype=torch.int32, device="cuda")


def edge_rows(K):
    """Rows that meet the format's edges: ties, saturation, zeros, subnormals, extremes,
    infinities and NaN, every one in a block of its own."""
    g = torch.Generator().manual_seed(0)
    rows = [torch.randn(K, generator=g), torch.zeros(K), torch.full((K,), -0.0)]
    ties = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.249, 0.2510, 7.0, 7.5]
                        + [-0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -7.9])
    rows += [ties.repeat(K // 20 + 1)[:K] * s for s in (1.0, 2.0 ** -126, 2.0 ** 100, 2.0 ** -130)]
    tiny = torch.randn(K, generator=g) * 2.0 ** -128
    big = torch.randn(K, generator=g).clamp(-1, 1) * 3.3e38
    rows += [tiny, big]
    for bad in (float("nan"), float("inf"), float("-inf")):
        r = torch.randn(K, generator=g)
        r[K // 2] = bad
        rows.append(r)
    return torch.stack(rows).to(BF16)


@pytest.mark.parametrize("K", [32, 96, 128, 416, 1056, 7168])
def test_quantize_rows_bits(K):
    x = edge_rows(K)
    M = x.shape[0]
    gs = sizes_tensor([M - 2, 0, 1])                       # the last row is past the groups
    codes, scales = fb.mxfp4_quantize_rows(x.cuda(), gs)
    want_c, want_s = ref.mx_pack(*ref.mx_quantize(x[:M - 1]))
    nb = K // 32
    assert torch.equal(codes[:M - 1].cpu(), want_c)
    got_s = scales.cpu().permute(1, 0, 2).reshape(M, -1)[:, :nb]
    assert torch.equal(got_s[:M - 1], want_s.permute(1, 0, 2).reshape(M - 1, -1)[:, :nb])
    assert (codes[M - 1] == 0).all() and (got_s[M - 1] == 0).all()


@pytest.mark.parametrize("E,K,N", [(1, 32, 16), (3, 96, 80), (2, 288, 64), (2, 512, 272),
                                   (1, 1056, 144)])
def test_quantize_and_dequantize_weights(E, K, N):
    g = torch.Generator().manual_seed(K)
    w = (torch.randn(E, K, N, generator=g) * torch.exp(3 * torch.randn(E, K, 1, generator=g)))
    w = w.to(BF16)
    w[0, :12, 0] = edge_rows(32)[:, 0]
    codes, scales = fb.mxfp4_quantize_weights(w.cuda())
    back = fb.mxfp4_dequantize(codes, scales)
    for e in range(E):
        c, b = ref.mx_quantize(w[e].T.contiguous())
        want_c, want_s = ref.mx_pack(c, b)
        assert torch.equal(codes[e].cpu(), want_c)
        nb = K // 32
        assert torch.equal(scales[e].cpu().permute(1, 0, 2).reshape(N, -1)[:, :nb], b)
        v = ref.mx_values(c, b).to(BF16)
        assert torch.equal(torch.nan_to_num(back[e].cpu().float(), nan=1.5e30),
                           torch.nan_to_num(v.float(), nan=1.5e30))


def weights(E, K, N, seed):
    """Codes and scale bytes drawn as such: every code, scales over a wide range."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 16, (E, N, K), generator=g, dtype=torch.uint8)
    byte = torch.randint(118, 127, (E, N, K // 32), generator=g, dtype=torch.uint8)
    packed = [ref.mx_pack(codes[e], byte[e]) for e in range(E)]
    pc, ps = (torch.stack([p[i] for p in packed]) for i in (0, 1))
    words = ps.shape[1]
    pad = words * 4 - K // 32
    if pad:                                                # bytes past K/32 mean nothing
        ps[:, -1, :, 4 - pad:] = 255
    return codes, byte, pc, ps


PRODUCTS = [  # group sizes, rows past them, K, N, SwiGLU
    ([1], 0, 32, 16, False), ([1], 0, 32, 32, True), ([0, 0, 3], 2, 64, 48, False),
    ([5, 0, 1], 0, 128, 96, True), ([16, 17, 15], 4, 256, 256, False),
    ([31, 33, 32], 0, 288, 288, True), ([96, 97], 0, 320, 272, False),
    ([207, 208, 209], 7, 512, 512, True), ([416, 417, 1], 0, 544, 528, False),
    ([700, 0, 0, 12], 0, 1056, 160, True), ([64] * 9, 0, 768, 1024, False),
    ([0, 0], 5, 128, 128, False), ([1] * 8 + [0] * 24, 0, 2048, 512, True),
    ([833, 100], 3, 96, 2080, False), ([3] * 130, 0, 352, 80, False),
    ([0] * 700 + [2, 0, 300] + [0] * 321, 5, 64, 48, False),
]


@pytest.mark.parametrize("sizes,extra,K,N,silu", PRODUCTS)
def test_product(sizes, extra, K, N, silu):
    E, T = len(sizes), sum(sizes)
    codes, byte, pc, ps = weights(E, K, N, seed=K + N)
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T + extra, K, generator=g).to(BF16)
    x[T:] = float("nan")                                   # never read
    x[:T][torch.rand(T, generator=g) < 0.05] *= 50
    cols = N // 2 if silu else N
    out = torch.full((T + extra, cols), 3.0, dtype=BF16, device="cuda")
    f = fb.gmm_silu_mxfp4_fwd if silu else fb.gmm_mxfp4_fwd
    fb.read_status()
    got = f(x.cuda(), pc.cuda(), ps.cuda(), sizes_tensor(sizes), out=out)
    assert fb.read_status() == 0
    assert (got[T:] == 3.0).all()
    if T:
        want = ref.mx_product(x[:T].double(), codes, byte, sizes, silu)
        check_bf16(got[:T], want, what=f"{sizes} {K} {N}")


def test_every_scale_byte_pair_and_code():
    """One block per row: codes and scales of both sides enter exactly."""
    g = torch.Generator().manual_seed(2)
    K, N, M = 128, 256, 64
    codes = torch.randint(0, 16, (1, N, K), generator=g, dtype=torch.uint8)
    byte = torch.randint(100, 150, (1, N, K // 32), generator=g, dtype=torch.uint8)
    # each weight row keeps one block, so that its result is one block's sum
    keep = torch.arange(N) % 4
    for n in range(N):
        mask = torch.zeros(K, dtype=torch.bool)
        mask[keep[n] * 32:(keep[n] + 1) * 32] = True
        codes[0, n, ~mask] = 0
    p = ref.mx_pack(codes[0], byte[0])
    x = (torch.randn(M, K, generator=g)
         * torch.exp2(torch.randint(-20, 20, (M, 4), generator=g).float())
         .repeat_interleave(32, dim=1)).to(BF16)
    got = fb.gmm_mxfp4_fwd(x.cuda(), p[0][None].cuda(), p[1][None].cuda(), sizes_tensor([M]))
    want = ref.mx_product(x.double(), codes, byte, [M], False)
    # 32 products of 4-bit values are exact in f32: one rounding to bf16
    assert torch.equal(got.cpu(), want.to(BF16))


def test_bad_rows_and_weights_stay_alone():
    codes, byte, pc, ps = weights(1, 256, 128, seed=1)
    x = torch.randn(40, 256).to(BF16)
    x[7, 3], x[21, 200] = float("nan"), float("inf")
    ps[0, 1, 77, 2] = 255                                  # a NaN scale of weight row 77
    got = fb.gmm_mxfp4_fwd(x.cuda(), pc.cuda(), ps.cuda(), sizes_tensor([40])).cpu()
    nan = torch.isnan(got)
    assert nan[7].all() and nan[21].all() and nan[:, 77].all()
    rest = nan.clone()
    rest[7] = rest[21] = False
    rest[:, 77] = False
    assert not rest.any()


def test_activation_gradient_by_the_dequantized_weight():
    """dlhs = dout x W^T through mxfp4_dequantize and gmm_bf16_fwd."""
    sizes, K, N = [40, 0, 25], 256, 128
    codes, byte, pc, ps = weights(3, K, N, seed=4)
    dout = torch.randn(65, N, generator=torch.Generator().manual_seed(1)).to(BF16)
    w = fb.mxfp4_dequantize(pc.cuda(), ps.cuda())          # [E, N, K]: the product's K is N
    got = fb.gmm_bf16_fwd(dout.cuda(), w, sizes_tensor(sizes), False)
    want, row = torch.zeros(65, K, dtype=torch.float64), 0
    for e, n in enumerate(sizes):
        want[row:row + n] = dout[row:row + n].double() @ ref.mx_values(codes[e], byte[e])
        row += n
    check_bf16(got, want)


def test_clipped_and_negative_groups():
    codes, byte, pc, ps = weights(3, 64, 64, seed=6)
    x = torch.randn(20, 64).to(BF16)
    fb.read_status()
    got = fb.gmm_mxfp4_fwd(x.cuda(), pc.cuda(), ps.cuda(), sizes_tensor([-4, 15, 9]))
    assert fb.read_status() == fb.STATUS_NEGATIVE_GROUP | fb.STATUS_GROUPS_EXCEED_M
    want = ref.mx_product(x.double(), codes, byte, [0, 15, 5], False)
    check_bf16(got, want)


def test_repeats_streams_and_graph():
    codes, byte, pc, ps = weights(4, 512, 256, seed=5)
    x, pc, ps = torch.randn(300, 512).to(BF16).cuda(), pc.cuda(), ps.cuda()
    gs = sizes_tensor([100, 0, 150, 50])
    want = fb.gmm_silu_mxfp4_fwd(x, pc, ps, gs)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        assert torch.equal(fb.gmm_silu_mxfp4_fwd(x, pc, ps, gs), want)
    torch.cuda.current_stream().wait_stream(st)
    out = torch.empty_like(want)
    ws = torch.empty(fb.workspace_size(fb.OP_GMM_SILU_MXFP4_FWD, 300, 512, 256, 4),
                     dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fb.gmm_silu_mxfp4_fwd(x, pc, ps, gs, out=out, workspace=ws)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_refusals():
    x = torch.zeros(8, 64, dtype=BF16, device="cuda")
    c = torch.zeros(2, 32, 32, dtype=torch.uint8, device="cuda")
    s = torch.zeros(2, 1, 32, 4, dtype=torch.uint8, device="cuda")
    gs = sizes_tensor([4, 4])
    with pytest.raises(TypeError):
        fb.gmm_mxfp4_fwd(x.float(), c, s, gs)
    with pytest.raises(ValueError):
        fb.gmm_mxfp4_fwd(x[:, :32].contiguous(), c, s, gs)
    with pytest.raises(ValueError):
        fb.gmm_mxfp4_fwd(x, c, s[:, :, :16].contiguous(), gs)
    with pytest.raises(ValueError):
        fb.gmm_mxfp4_fwd(x, c, s, gs, out=torch.empty(8, 16, dtype=BF16, device="cuda"))
    with pytest.raises(fb.Fp8MoeError, match="EALIGN"):
        fb.mxfp4_quantize_weights(torch.zeros(1, 48, 32, dtype=BF16, device="cuda"))
    with pytest.raises(fb.Fp8MoeError, match="EALIGN"):
        fb.gmm_silu_mxfp4_fwd(x, c[:, :16].contiguous(), s[:, :, :16].contiguous(), gs)
    with pytest.raises(fb.Fp8MoeError, match="EWORKSPACE"):
        fb.gmm_mxfp4_fwd(x, c, s, gs, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
