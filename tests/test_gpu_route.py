"""Tokens sorted by expert and back against plain 64-bit forms, on the GPU."""
import pytest
import torch

import layer_reference as ref
from fp8_moe_routed_gb300 import binding as fb

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def draw_ids(T, k, E, seed, drop=0.0, skew=0.0):
    g = torch.Generator().manual_seed(seed)
    p = torch.exp(torch.randn(E, generator=g) * skew)
    ids = torch.multinomial(p, max(1, T * k), replacement=True, generator=g)[:T * k]
    ids = ids.reshape(T, k).to(torch.int32)
    if drop:
        ids[torch.rand(T, k, generator=g) < drop] = -1
    return ids


# T, topk, E, rows of the buffer past (or short of) the kept slots, share dropped
SORTS = [
    (1, 1, 1, 0, 0.0), (1, 8, 32, 0, 0.0), (3, 5, 7, 9, 0.3), (33, 2, 1024, 0, 0.0),
    (127, 32, 61, 100, 0.1), (1024, 8, 32, 0, 0.0),
    (256, 8, 32, 0, 0.0), (257, 8, 32, 7, 0.1),                # the last size of one CTA, and more
    (1025, 8, 32, 0, 0.5), (4096, 8, 256, 1000, 0.0), (9001, 7, 1024, 0, 0.02),
    (2000, 8, 16, -3000, 0.0), (64, 4, 8, -255, 0.0), (5, 3, 4, 0, 1.0),
]


@pytest.mark.parametrize("T,k,E,extra,drop", SORTS)
def test_sort(T, k, E, extra, drop):
    ids = draw_ids(T, k, E, seed=T + k, drop=drop, skew=1.0)
    M = max(1, T * k + extra)
    fb.read_status()
    gs, slot_row, row_slot = fb.sort_tokens(ids.cuda(), E, M)
    want = ref.sort_tokens(ids, E, M)
    assert gs.cpu().tolist() == want[0]
    assert slot_row.cpu().reshape(-1).tolist() == want[1]
    assert row_slot.cpu().tolist() == want[2]
    kept = int(((ids >= 0) & (ids < E)).sum())
    assert fb.read_status() == (fb.STATUS_GROUPS_EXCEED_M if kept > M else 0)


def test_sort_reports_and_drops_bad_ids():
    ids = torch.tensor([[0, 4], [2 ** 31 - 1, 1], [-1, -2 ** 31]], dtype=torch.int32)
    fb.read_status()
    gs, slot_row, row_slot = fb.sort_tokens(ids.cuda(), 4)
    assert gs.tolist() == [1, 1, 0, 0]
    assert slot_row.tolist() == [[0, -1], [-1, 1], [-1, -1]]
    assert row_slot.tolist() == [0, 3, -1, -1, -1, -1]
    assert fb.read_status() == fb.STATUS_BAD_EXPERT


def test_no_tokens():
    ids = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    x = torch.empty(0, 64, dtype=BF16, device="cuda")
    rows, gs, slot_row, row_slot = fb.dispatch_tokens(x, ids, 5, M=3)
    assert gs.tolist() == [0] * 5 and row_slot.tolist() == [-1] * 3 and slot_row.shape == (0, 4)
    assert fb.combine_tokens(rows, slot_row, torch.empty(0, 4, device="cuda")).shape == (0, 64)
    drows, dw = fb.combine_tokens_bwd(x, rows, slot_row, torch.empty(0, 4, device="cuda"))
    assert drows.shape == (3, 64) and dw.shape == (0, 4)


# T, topk, E, H, type, share dropped
MOVES = [
    (1, 8, 32, 7168, BF16, 0.0), (1, 1, 1, 8, BF16, 0.0), (7, 3, 4, 1000, BF16, 0.3),
    (65, 9, 16, 264, F32, 0.2), (130, 32, 40, 4, F32, 0.0), (33, 8, 8, 2056, BF16, 0.9),
    (1030, 8, 61, 136, BF16, 0.1), (12, 2, 3, 16392, BF16, 0.0),
]


@pytest.mark.parametrize("T,k,E,H,dtype,drop", MOVES)
def test_dispatch_combine_and_gradients(T, k, E, H, dtype, drop):
    g = torch.Generator().manual_seed(T * H)
    ids = draw_ids(T, k, E, seed=H, drop=drop)
    M = T * k + 3
    x = torch.randn(T, H, generator=g).to(dtype)
    w = torch.rand(T, k, generator=g) - 0.3
    rows = torch.full((M, H), 7.0, dtype=dtype, device="cuda")
    got, gs, slot_row, row_slot = fb.dispatch_tokens(x.cuda(), ids.cuda(), E, M, out=rows)
    assert got.data_ptr() == rows.data_ptr()
    sizes, srow, rslot = ref.sort_tokens(ids, E, M)
    assert gs.tolist() == sizes and row_slot.tolist() == rslot
    srow = torch.tensor(srow).reshape(T, k)
    assert torch.equal(slot_row.cpu().long(), srow)
    want = torch.full((M, H), 7.0, dtype=dtype)
    for r, s in enumerate(rslot):
        if s >= 0:
            want[r] = x[s // k]
    assert torch.equal(got.cpu(), want)                     # copies; rows past the last untouched

    # garbage in the rows that no slot names may not reach any sum
    y = torch.randn(M, H, generator=g).to(dtype)
    y[sum(sizes):] = float("nan")
    ref.check_rows(fb.combine_tokens(y.cuda(), slot_row, w.cuda()), ref.combine(y, srow, w), "out")
    ref.check_rows(fb.dispatch_tokens_bwd(y.cuda(), slot_row), ref.combine(y, srow), "dx")
    dout = torch.randn(T, H, generator=g).to(dtype)
    drows = torch.full((M, H), 5.0, dtype=dtype, device="cuda")
    drows, dw = fb.combine_tokens_bwd(dout.cuda(), y.cuda(), slot_row, w.cuda(), out=drows)
    want_rows, want_w = ref.combine_bwd(dout, y, srow, w)
    n = sum(sizes)
    ref.check_rows(drows[:n], want_rows[:n], "drows")
    assert (drows[n:] == 5.0).all()
    ref.check_f32(dw, want_w, "dweights")


def test_gradient_against_differences():
    """d/dp of L = <c, combine(dispatch(x), w)> by central differences in 64 bits."""
    T, k, E, H = 9, 4, 5, 32
    g = torch.Generator().manual_seed(3)
    ids = draw_ids(T, k, E, seed=8, drop=0.2)
    x = torch.randn(T, H, generator=g)
    w = torch.rand(T, k, generator=g)
    c = torch.randn(T, H, generator=g)
    _, _, slot_row, _ = fb.dispatch_tokens(x.cuda(), ids.cuda(), E)
    rows = torch.zeros(T * k, H, device="cuda")
    rows = fb.dispatch_tokens(x.cuda(), ids.cuda(), E, out=rows)[0]
    drows, dw = fb.combine_tokens_bwd(c.cuda(), rows, slot_row, w.cuda(),
                                      out=torch.zeros_like(rows))
    dx = fb.dispatch_tokens_bwd(drows, slot_row)
    live = (ids >= 0).double()

    def loss(x, w):
        return (c.double() * x * (w * live).sum(1, keepdim=True)).sum()

    for p, grad in (("x", dx), ("w", dw)):
        v = torch.randn(x.shape if p == "x" else w.shape, generator=g).double()
        step = 1e-4
        ends = [loss(x.double() + s * v, w.double()) if p == "x" else
                loss(x.double(), w.double() + s * v) for s in (step, -step)]
        slope = (ends[0] - ends[1]) / (2 * step)
        have = (grad.cpu().double() * v).sum()
        # the loss is linear in each; f32 gradients: 1e-5 of the terms' sum
        assert abs(have - slope) <= 1e-5 * (grad.cpu().double() * v).abs().sum()


def test_stale_or_broken_slot_row_stays_in_bounds():
    """Entries past the buffer count as no row."""
    rows = torch.ones(4, 16, device="cuda")
    slot_row = torch.tensor([[0, 4], [2 ** 31 - 1, -5]], dtype=torch.int32, device="cuda")
    out = fb.combine_tokens(rows, slot_row)
    assert out[0].eq(1).all() and out[1].eq(0).all()


def test_offsets_past_32_bits():
    """Rows whose byte and element offsets pass 2^32 (8.6 GB of rows)."""
    H, T, k = 8192, 8, 1
    M = 530_000
    rows = torch.zeros(M, H, dtype=BF16, device="cuda")
    slot_row = torch.tensor([[M - 1 - 3 * t] for t in range(T)], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    v = torch.randn(T, H, generator=g, device="cuda").to(BF16)
    rows[slot_row[:, 0].long()] = v
    assert torch.equal(fb.combine_tokens(rows, slot_row), v)
    w = torch.full((T, k), 2.0, device="cuda")
    drows, dw = fb.combine_tokens_bwd(v, rows, slot_row, w, out=rows)
    assert torch.equal(drows[slot_row[:, 0].long()], v * 2)


def test_another_stream():
    ids = draw_ids(500, 8, 32, seed=5).cuda()
    x = torch.randn(500, 256, device="cuda").to(BF16)
    want = fb.dispatch_tokens(x, ids, 32)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = fb.dispatch_tokens(x, ids, 32)
    torch.cuda.current_stream().wait_stream(st)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_refusals():
    x = torch.zeros(4, 64, dtype=BF16, device="cuda")
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        fb.sort_tokens(ids.long(), 4)
    with pytest.raises(TypeError):
        fb.dispatch_tokens(x.half(), ids, 4)
    with pytest.raises(ValueError):
        fb.dispatch_tokens(x, ids[:3].contiguous(), 4)
    with pytest.raises(ValueError):
        fb.dispatch_tokens(x.t(), ids, 4)
    with pytest.raises(ValueError):
        fb.dispatch_tokens(x, ids, 4, out=torch.empty(3, 64, dtype=BF16, device="cuda"))
    with pytest.raises(fb.Fp8MoeError, match="EALIGN"):
        fb.dispatch_tokens(torch.zeros(4, 12, dtype=BF16, device="cuda"), ids, 4)
    with pytest.raises(fb.Fp8MoeError, match="EINVAL"):
        fb.sort_tokens(ids, 1025)
    with pytest.raises(fb.Fp8MoeError, match="EINVAL"):
        fb.sort_tokens(torch.zeros(2, 33, dtype=torch.int32, device="cuda"), 4)
    rows, _, slot_row, _ = fb.dispatch_tokens(x, ids, 4)
    with pytest.raises(ValueError):
        fb.combine_tokens(rows, slot_row, torch.zeros(4, 3, device="cuda"))
    with pytest.raises(TypeError):
        fb.combine_tokens(rows, slot_row, torch.zeros(4, 2, dtype=BF16, device="cuda"))
    with pytest.raises(TypeError):
        fb.combine_tokens_bwd(x.float(), rows, slot_row, torch.zeros(4, 2, device="cuda"))
