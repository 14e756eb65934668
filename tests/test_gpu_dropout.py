"""Dropout through the C ABI against the plain form.  Which elements are kept is compared
exactly; a kept element is one FP32 fused multiply-add of a factor rounded to FP32: within
2^-22 of (|x| factor + |residual|), plus half a BF16 step where it is stored so."""
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


def _view(rows, cols, dtype, pad, shift):
    buf = torch.empty(rows * (cols + pad) + shift, dtype=dtype, device="cuda").normal_()
    return buf[shift:].view(rows, cols + pad)[:, :cols]


@pytest.mark.parametrize("rows,cols,pad,shift", [(1, 1, 0, 0), (1, 8, 0, 0), (3, 7, 0, 0), (5, 64, 0, 0),
                                                 (5, 64, 8, 8), (4, 64, 1, 0), (4, 200, 0, 1), (7, 1409, 0, 0),
                                                 (2, 4104, 0, 0)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.999, 1.0])
def test_dropout_matches_plain(M, rows, cols, pad, shift, dtype, residual, p):
    x = _view(rows, cols, dtype, pad, shift)
    res = _view(rows, cols, dtype, pad, shift) if residual else None
    out = torch.full((rows, cols), 7.0, dtype=dtype, device="cuda")
    seed, offset = 0xFEDCBA9876543210, (1 << 40) + 5
    M.moe_dropout(x, out, p, seed, offset, res)
    xf, rf = to_np(x).astype(np.float64), 0.0 if res is None else to_np(res).astype(np.float64)
    thr = round(p * 65536)
    keep = P.dropout_bits(rows, cols, seed, offset) >= thr
    ref = P.dropout(xf, p, seed, offset) + rf
    got = to_np(out).astype(np.float64)
    factor = 65536.0 / (65536 - thr) if thr < 65536 else 0.0
    tol = 2.0 ** -22 * (np.abs(xf) * factor + np.abs(rf)) + (2.0 ** -8 * np.abs(ref) if dtype == BF16 else 0.0)
    assert np.all(np.abs(got - ref) <= tol)
    assert np.array_equal(got[~keep], (rf + np.zeros_like(xf))[~keep])


def test_dropout_gradient_is_the_same_mask(M):
    """Differences: dropout is linear in x, so <g, D(x + d) - D(x)> = <D(g), d>."""
    x, d, g = (torch.randn(33, 520, device="cuda") for _ in range(3))
    a, b, dg = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    res = torch.randn_like(x)
    M.moe_dropout(x + d, a, 0.3, 11, 4, res)
    M.moe_dropout(x, b, 0.3, 11, 4, res)
    M.moe_dropout(g, dg, 0.3, 11, 4)
    left, right = (g.double() * (a.double() - b.double())).sum(), (dg.double() * d.double()).sum()
    assert abs(float(left - right)) <= x.numel() * 16 * 2.0 ** -24
    assert torch.equal(dg == 0, (a - res) - (b - res) == 0) or bool(((dg == 0) == (a == b)).all())


def test_dropout_in_place_and_what_is_dropped(M):
    x = torch.randn(9, 256, device="cuda").to(BF16)
    x[:, ::3] = float("nan")
    x[:, 1::3] = float("inf")
    res = torch.randn(9, 256, device="cuda").to(BF16)
    want = torch.empty_like(x)
    M.moe_dropout(x, want, 0.5, 3, 0, res)
    keep = torch.from_numpy(P.dropout_bits(9, 256, 3, 0) >= 32768).cuda()
    assert torch.equal(want[~keep], res[~keep])            # whatever a dropped element holds
    y = x.clone()
    M.moe_dropout(y, y, 0.5, 3, 0, res)                    # over x
    z = res.clone()
    M.moe_dropout(x, z, 0.5, 3, 0, z)                      # into the residual stream
    for t in (y, z):
        assert torch.equal(t.view(torch.int16), want.view(torch.int16))


def test_dropout_large_and_counters_past_32_bits(M):
    """The element's counter is a 64-bit number: rows past 2^32 counters differ from their
    low 32 bits' (checked through the plain form), and a large matrix keeps the rate."""
    rows, cols = 4096, 4096
    x = torch.ones((rows, cols), dtype=BF16, device="cuda")
    out = torch.empty_like(x)
    M.moe_dropout(x, out, 0.25, 5, 6)
    n, kept = rows * cols, int((out != 0).sum())
    assert abs(kept - 0.75 * n) < 6 * (n * 0.75 * 0.25) ** 0.5     # six standard deviations
    tail = P.dropout_bits(rows, 8, 5, 6)                            # rows of one counter: b = r
    got = torch.empty((rows, 8), dtype=BF16, device="cuda")
    M.moe_dropout(x[:, :8], got, 0.25, 5, 6)
    assert np.array_equal(to_np(got) != 0, tail >= 16384)
    M.moe_dropout(x, x, 0.25, 5, 6, None, torch.cuda.current_stream())
    assert torch.equal(x, out)


@pytest.mark.parametrize("rows,cols,pad,shift", [(33, 520, 0, 0), (33, 521, 3, 1)])
@pytest.mark.parametrize("p", [0.3, 0.9])
def test_forward_and_gradient_keep_the_counters_elements(M, rows, cols, pad, shift, p):
    """Each against the plain form's bits by itself."""
    keep = torch.from_numpy(P.dropout_bits(rows, cols, 11, 4) >= round(p * 65536)).cuda()
    for _ in range(2):                                     # an input, and the gradient of the output
        x = _view(rows, cols, F32, pad, shift).abs_().add_(0.5)
        out = torch.empty((rows, cols), device="cuda")
        M.moe_dropout(x, out, p, 11, 4)
        assert torch.equal(out != 0, keep)


@pytest.mark.parametrize("rows,cols,ld", [(2 ** 32 + 64, 1, 1),             # by columns
                                          (1, 2 ** 35 + 512, 2 ** 35 + 512),  # one long row
                                          (2 ** 32 + 64, 8, 16)])           # groups of a padded matrix
def test_dropout_counters_past_32_bits(M, rows, cols, ld):
    """Elements on both sides of the counter 2^32, in place, against the generator."""
    torch.cuda.empty_cache()
    need = rows * ld * 2
    if torch.cuda.mem_get_info()[0] < need + (8 << 30):
        pytest.skip(f"{need >> 30} GB of device memory are not free")
    x = torch.empty((rows, ld), dtype=BF16, device="cuda")[:, :cols]
    groups = (cols + 7) // 8
    width = min(cols, 8)
    counters = [0, 1, 77, 2 ** 31, 2 ** 32 - 1, *range(2 ** 32, 2 ** 32 + 64)]
    at = [(x[b // groups, b % groups * 8:b % groups * 8 + width], b) for b in counters]
    for part, _ in at:
        part.fill_(1.0)
    seed, offset, p, m = 0x123456789ABCDEF, 3, 0.5, 0xFFFFFFFF
    M.moe_dropout(x, x, p, seed, offset)
    got = torch.stack([part for part, _ in at]).cpu() != 0
    want = []
    for b in counters:
        w = P.philox([b & m, b >> 32, offset, 0], [seed & m, seed >> 32])
        want.append([(w[i // 2] >> 16 * (i % 2) & 0xFFFF) >= 32768 for i in range(width)])
    assert torch.equal(got, torch.tensor(want))
    del x, at, part
    torch.cuda.empty_cache()
