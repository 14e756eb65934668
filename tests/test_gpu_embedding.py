"""Token embedding and its table's gradient through the C ABI, against the plain 64-bit
forms.  The lookup is one FP32 product rounded once, so it is compared bit for bit.  A
gradient element that sums c terms of absolute sum A in FP32 is within (c + 2) 2^-24 A of
the exact sum (one rounding per addition, one for the scale, one for the result), plus half
a BF16 step (2^-8 of the value) where it is stored so."""
import numpy as np
import pytest
import torch

import plain_ops as P
from gpu_common import need_cuda, to_np

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def M():
    need_cuda()
    from token_dispatch_expert_top_gb300 import moe
    return moe


def _ws(M, n=256):
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    M.moe_workspace_init(ws)
    return ws


def _strided(rows, cols, dtype, pad, shift, fill=None):
    """A [rows][cols] view, `pad` elements between rows, starting `shift` elements in."""
    buf = torch.empty(rows * (cols + pad) + shift, dtype=dtype, device="cuda")
    if fill is None:
        buf.normal_()
    else:
        buf.fill_(fill)
    return buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols], buf


@pytest.mark.parametrize("H,pad,shift", [(1, 0, 0), (7, 0, 0), (8, 0, 0), (64, 8, 0), (64, 3, 1), (1409, 0, 0),
                                         (2048, 0, 0), (264, 0, 8), (256, 0, 4)])
@pytest.mark.parametrize("tdt,odt", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
def test_embedding_bitwise(M, H, pad, shift, tdt, odt, idt):
    V, N, scale = 37, 61, 1.3
    table, _ = _strided(V, H, tdt, pad, shift)
    out, buf = _strided(N, H, odt, pad, shift, fill=7.0)
    ids = torch.randint(-1, V, (N,), device="cuda").to(idt)
    ids[0], ids[1], ids[2] = 0, V - 1, -5
    M.moe_embedding(ids, table, out, scale)
    ref = P.embedding(to_np(ids), to_np(table).astype(np.float64), float(np.float32(scale)))
    want = torch.from_numpy(ref.astype(np.float32)).to(odt)
    assert torch.equal(out.cpu(), want)
    out.fill_(7.0)
    assert bool((buf == 7.0).all())                        # nothing between the rows was written


def test_embedding_lengths_and_bad_ids(M):
    table = torch.randn(5, 16, device="cuda")
    ws = _ws(M)
    out = torch.empty(0, 16, device="cuda")
    M.moe_embedding(torch.empty(0, dtype=torch.int32, device="cuda"), table, out, 1.0, ws)
    out = torch.full((1, 16), 9.0, device="cuda")
    M.moe_embedding(torch.tensor([4], device="cuda"), table, out, 1.0, ws)
    assert torch.equal(out[0], table[4]) and M.moe_last_device_status(ws) == M.MOE_OK
    out = torch.full((2, 2, 16), 9.0, device="cuda")       # leading dimensions count as rows
    M.moe_embedding(torch.tensor([[1, 5], [1 << 40, -1]], device="cuda"), table, out, 1.0, ws)
    assert torch.equal(out[0, 0], table[1]) and bool((out.view(4, 16)[1:] == 0).all())
    assert M.moe_last_device_status(ws) == M.MOE_ERR_DEVICE_CHECK
    assert M.moe_last_device_status(ws) == M.MOE_OK


def test_embedding_rows_past_32_bit_offsets(M):
    V, H = 300_001, 7168                                   # 2.15e9 elements
    table = torch.zeros((V, H), dtype=BF16, device="cuda")
    table[V - 1].normal_()
    out = torch.empty((3, H), dtype=BF16, device="cuda")
    M.moe_embedding(torch.tensor([V - 1, 0, V - 1], device="cuda"), table, out)
    assert torch.equal(out[0], table[V - 1]) and torch.equal(out[2], table[V - 1]) and not out[1].any()
    # and the gradient's last row
    ws = _ws(M, M.moe_embedding_workspace_bytes(3, V, H))
    dout = torch.randn((3, H), device="cuda").to(BF16)
    M.moe_embedding_backward(torch.tensor([V - 1, -1, V - 1], device="cuda"), dout, table, 1.0, False, ws)
    assert torch.equal(table[V - 1], (dout[0].float() + dout[2].float()).to(BF16))
    assert not table[:V - 1].any()


def _grad_case(M, ids, V, H, gdt, tdt, scale=1.0, accumulate=False, pad=0, shift=0, N_ws=None):
    N = len(ids)
    dout, _ = _strided(N, H, gdt, pad, shift)
    dtable, buf = _strided(V, H, tdt, pad, shift, fill=3.0)
    ws = _ws(M, M.moe_embedding_workspace_bytes(N, V, H))
    M.moe_embedding_backward(ids, dout, dtable, scale, accumulate, ws)
    assert M.moe_last_device_status(ws) == M.MOE_OK
    g, a, cnt = P.embedding_grad(to_np(ids), to_np(dout).astype(np.float64), V, float(np.float32(scale)))
    ref = g + (3.0 if accumulate else 0.0)
    tol = (cnt[:, None] + 2) * 2.0 ** -24 * (a + np.abs(ref))
    if tdt == BF16:
        tol = tol + 2.0 ** -8 * np.abs(ref)
    got = to_np(dtable).astype(np.float64)
    assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) - tol)
    untouched = cnt == 0
    assert np.all(got[untouched] == (3.0 if accumulate else 0.0))
    again, _ = _strided(V, H, tdt, pad, shift, fill=3.0)
    M.moe_embedding_backward(ids, dout, again, scale, accumulate, ws)
    assert torch.equal(again, dtable)                      # the same bits every time
    dtable.fill_(3.0)
    assert bool((buf == 3.0).all())


@pytest.mark.parametrize("N", [1, 2, 31, 32, 33, 64, 65, 511, 513, 2000])
@pytest.mark.parametrize("V,H", [(1, 5), (3, 64), (1000, 24), (70000, 8)])
def test_embedding_grad_lengths(M, N, V, H):
    """One id for all tokens (runs across many ranges), few ids, many ids."""
    gen = torch.Generator(device="cuda").manual_seed(N)
    ids = torch.randint(-1, V, (N,), device="cuda", generator=gen)
    _grad_case(M, ids, V, H, F32, F32)


@pytest.mark.parametrize("H,pad,shift", [(1, 0, 0), (9, 0, 0), (256, 0, 0), (264, 8, 0), (520, 3, 1), (1409, 0, 0)])
@pytest.mark.parametrize("gdt,tdt", [(F32, F32), (BF16, F32), (BF16, BF16), (F32, BF16)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embedding_grad_layouts(M, H, pad, shift, gdt, tdt, accumulate):
    rng = np.random.default_rng(3)
    ids = rng.zipf(1.4, size=300)
    ids = torch.from_numpy(np.where(ids > 50, -1, ids - 1).astype(np.int32)).cuda()
    _grad_case(M, ids, 50, H, gdt, tdt, scale=-0.7, accumulate=accumulate, pad=pad, shift=shift)


# Up to 1024 tokens take one launch, more are sorted first: the same cases on both sides.
@pytest.mark.parametrize("N", [1000, 1024, 1025, 1500])
@pytest.mark.parametrize("H,pad,shift", [(1, 0, 0), (9, 0, 0), (264, 8, 0), (520, 3, 1), (2056, 0, 0)])
@pytest.mark.parametrize("gdt,tdt,accumulate", [(F32, F32, False), (BF16, F32, True), (BF16, BF16, False)])
def test_embedding_grad_either_way(M, N, H, pad, shift, gdt, tdt, accumulate):
    rng = np.random.default_rng(N)
    ids = rng.zipf(1.4, size=N)
    ids = torch.from_numpy(np.where(ids > 600, -1, ids - 1).astype(np.int32)).cuda()
    _grad_case(M, ids, 600, H, gdt, tdt, scale=1.7, accumulate=accumulate, pad=pad, shift=shift)


@pytest.mark.parametrize("N", [1, 3, 40, 257, 1024, 1100])
@pytest.mark.parametrize("H", [8, 2048, 4103, 4112])
def test_embedding_grad_one_id(M, N, H):
    """One run of every token, whose columns many CTAs share; and two that take turns."""
    _grad_case(M, torch.full((N,), 2, device="cuda"), 3, H, BF16, F32)
    _grad_case(M, torch.arange(N, device="cuda") % 2, 3, H, F32, F32, accumulate=True)


def test_embedding_grad_orders_of_many_tokens(M):
    for ids in (list(range(1200)), list(range(1200))[::-1], [7] * 1024 + [8] * 32 + [9], [5] * 33 + [6] * 999 + [5] * 70,
                [1, 2] * 700, [1199] * 1025, [-1] * 1040):
        _grad_case(M, torch.tensor(ids, device="cuda"), 1200, 40, F32, F32)


def test_embedding_grad_few_tokens_of_a_tall_table(M):
    """More rows than one CTA marks at a time."""
    ids = torch.tensor([0, 4095, 4096, 1_299_999, 5, 5, -3], device="cuda")
    _grad_case(M, ids, 1_300_000, 3, F32, BF16)


def test_embedding_grad_orders(M):
    """Sorted, reversed and interleaved tokens; runs that begin and end on range borders."""
    for ids in (list(range(200)), list(range(200))[::-1], [7] * 32 + [8] * 32 + [9], [5] * 33 + [6] * 31 + [5] * 70,
                [1, 2] * 100, [199] * 65, [-1] * 40):
        _grad_case(M, torch.tensor(ids, device="cuda"), 200, 40, F32, F32)


def test_embedding_grad_empty_and_bad_ids(M):
    dtable = torch.full((4, 8), 2.0, device="cuda")
    ws = _ws(M, M.moe_embedding_workspace_bytes(4, 4, 8))
    none = torch.empty((0, 8), device="cuda")
    M.moe_embedding_backward(torch.empty(0, dtype=torch.int64, device="cuda"), none, dtable, 1.0, True, ws)
    assert bool((dtable == 2.0).all())
    M.moe_embedding_backward(torch.empty(0, dtype=torch.int64, device="cuda"), none, dtable, 1.0, False, ws)
    assert not dtable.any()
    dout = torch.randn(4, 8, device="cuda")
    M.moe_embedding_backward(torch.tensor([4, 1, 1 << 33, -(1 << 40)], device="cuda"), dout, dtable, 1.0, False, ws)
    assert torch.equal(dtable[1], dout[1]) and not dtable[[0, 2, 3]].any()
    assert M.moe_last_device_status(ws) == M.MOE_ERR_DEVICE_CHECK


def test_embedding_grad_is_the_lookups_transpose(M):
    """Differences of the lookup, which is linear: <dout, E(W + D) - E(W)> = <dtable, D>."""
    V, H, N = 90, 48, 500
    gen = torch.Generator(device="cuda").manual_seed(5)
    ids = torch.randint(-1, V, (N,), device="cuda", generator=gen)
    W, D = (torch.randn(V, H, device="cuda", generator=gen) for _ in range(2))
    dout = torch.randn(N, H, device="cuda", generator=gen)
    a, b = torch.empty(N, H, device="cuda"), torch.empty(N, H, device="cuda")
    M.moe_embedding(ids, W + D, a, 2.0)
    M.moe_embedding(ids, W, b, 2.0)
    dtable = torch.empty(V, H, device="cuda")
    M.moe_embedding_backward(ids, dout, dtable, 2.0, False, _ws(M, M.moe_embedding_workspace_bytes(N, V, H)))
    left, right = (dout.double() * (a.double() - b.double())).sum(), (dtable.double() * D.double()).sum()
    # N*H terms of order 2, each off by at most a few 2^-24 of about 4
    assert abs(float(left - right)) <= N * H * 16 * 2.0 ** -24


def test_embedding_on_another_stream(M):
    V, H, N = 500, 512, 3000
    ids = torch.randint(0, V, (N,), device="cuda")
    table, dout = torch.randn(V, H, device="cuda"), torch.randn(N, H, device="cuda")
    out, dtable = torch.empty(N, H, device="cuda"), torch.empty(V, H, device="cuda")
    ws = _ws(M, M.moe_embedding_workspace_bytes(N, V, H))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    M.moe_embedding(ids, table, out, 1.0, ws, side)
    M.moe_embedding_backward(ids, dout, dtable, 1.0, False, ws, side)
    side.synchronize()
    assert torch.equal(out, table[ids])
    ref = torch.zeros(V, H, dtype=torch.float64, device="cuda").index_add_(0, ids, dout.double())
    assert float((dtable.double() - ref).abs().max()) < 64 * 2.0 ** -24 * 64


@pytest.mark.parametrize("longest,N,H", [(8192, 8160, 2048), (1170, 1162, 3584), (2400, 1100, 1409)])
def test_embedding_grad_in_a_longer_batchs_workspace(M, longest, N, H):
    """One workspace for the longest batch serves a shorter one, whose ranges are shorter."""
    V = 700
    gen = torch.Generator(device="cuda").manual_seed(N)
    ids = torch.randint(-1, V, (N,), device="cuda", generator=gen)
    dout = torch.randint(-8, 9, (N, H), device="cuda", generator=gen).float()
    ws = _ws(M, M.moe_embedding_workspace_bytes(longest, V, H))
    dtable = torch.full((V, H), 5.0, device="cuda")
    M.moe_embedding_backward(ids, dout, dtable, 1.0, False, ws)
    ref = torch.zeros((V, H), device="cuda").index_add_(0, ids.clamp(min=0), dout * (ids >= 0).unsqueeze(1))
    assert torch.equal(dtable, ref)                        # whole numbers: exact in any order
    assert M.moe_last_device_status(ws) == M.MOE_OK


def _many_ids(kind, N, V):
    gen = torch.Generator(device="cuda").manual_seed(N)
    n = torch.arange(N, device="cuda")
    if kind == "zipf":
        u = torch.rand(N, generator=gen, device="cuda", dtype=torch.float64)
        return (torch.exp(u * np.log(V + 1.0)).long() - 1).clamp(0, V - 1)
    if kind == "one":
        return torch.full_like(n, 5)
    if kind == "two in turns":                             # owned by the same CTA
        return torch.where(n % 2 == 0, 3, 5)
    if kind == "two in blocks":
        return torch.where(n < N // 2 + 7, 5, 3)
    return torch.randint(-V // 4, V, (N,), generator=gen, device="cuda")     # a fifth of padding


# One sweep of the ordering covers 4096 ids, and a CTA lists 4096 tokens of its own at a time.
@pytest.mark.parametrize("N", [4096, 4097, 8192, 8193, 20000])
@pytest.mark.parametrize("kind", ["zipf", "one", "two in turns", "two in blocks", "padded"])
@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
@pytest.mark.parametrize("V,H,accumulate", [(600, 264, False), (70_000, 24, True)])
def test_embedding_grad_of_many_sweeps(M, N, kind, idt, V, H, accumulate):
    """Sums of whole numbers, which FP32 adds exactly in any order."""
    ids = _many_ids(kind, N, V)
    gen = torch.Generator(device="cuda").manual_seed(H)
    dout = torch.randint(-8, 9, (N, H), device="cuda", generator=gen).float()
    ref = torch.full((V, H), 3.0 if accumulate else 0.0, device="cuda")
    ref.index_add_(0, ids.clamp(min=0), dout * (ids >= 0).unsqueeze(1))
    ws = _ws(M, M.moe_embedding_workspace_bytes(N, V, H))
    for dtype in (F32, BF16):
        dtable = torch.full((V, H), 3.0, device="cuda")
        M.moe_embedding_backward(ids.to(idt), dout.to(dtype), dtable, 1.0, accumulate, ws)
        assert torch.equal(dtable, ref)
    assert M.moe_last_device_status(ws) == M.MOE_OK


@pytest.mark.parametrize("kind", ["one", "two in turns", "zipf"])
def test_embedding_grad_of_many_sweeps_in_fractions(M, kind):
    _grad_case(M, _many_ids(kind, 9001, 300), 300, 40, F32, F32, scale=0.3)
