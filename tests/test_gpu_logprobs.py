"""Log probabilities of given tokens, entropy, top alternatives and the gradient through the
C ABI, against the plain 64-bit forms.

Tolerances, derived from the kernel's arithmetic (FP32, a row split over at least 128 lanes):
  - an exponential is off by at most 2^-22 (ex2) + |c d| 2^-23 (its argument, two
    roundings) of itself; weighted by exp(-|c d|) the latter stays below 2^-24 on average;
  - a row's sum adds a lane's V / 128 terms in sequence, then about 16 partial sums:
    eps = (V / 128 + 64) 2^-24 of the sum covers both;
  - logp = c (x - m) - ln S: |c (x - m)| 2^-22 + eps + |logp| 2^-23;
  - entropy = ln S - c t / S: the moment's terms have the same relative errors, so
    (2 + 2 (entropy + 1)) eps;
  - the gradient's p: (eps + (|logp| + |c (x - m)| + 4) 2^-22) p, times the bracket it
    stands in; each product and sum rounds by 2^-23 more; half a BF16 step (2^-8) where it
    is stored so.
Indices are compared exactly."""
import numpy as np
import pytest
import torch

import plain_ops as P
from gpu_common import need_cuda, to_np

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")


@pytest.fixture(scope="module")
def M():
    need_cuda()
    from token_dispatch_expert_top_gb300 import moe
    return moe


def _eps(V):
    return (V / 128 + 64) * 2.0 ** -24


def _close(got, ref, tol):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        stored = ref.astype(np.float32)                    # what passes FP32's range is an infinity in it
        same = got == stored
        assert np.array_equal(np.isfinite(got), np.isfinite(stored))
        assert np.all(same | (np.abs(got - ref) <= tol)), np.nanmax(np.where(same, 0, np.abs(got - ref) - tol))


def _forward(M, x, t, scale, n_top):
    T = x.shape[0]
    f = dict(dtype=F32, device="cuda")
    o = dict(logp=torch.full((T,), 9.0, **f), entropy=torch.full((T,), 9.0, **f), stats=torch.full((T, 2), 9.0, **f),
             top_idx=torch.full((T, n_top), -9, dtype=torch.int32, device="cuda"),
             top_logp=torch.full((T, n_top), 9.0, **f))
    M.moe_token_logprobs(x, t, o["logp"], o["entropy"], o["stats"], o["top_idx"], o["top_logp"], scale)
    return o


def _check(M, x, t, scale=1.0, n_top=5, grad=True):
    """Forward and gradient of the logits x (any strides) and targets t."""
    T, V = x.shape
    n_top = min(n_top, V)
    o = _forward(M, x, t, scale, n_top)
    s = float(np.float32(scale))
    xf, tf = to_np(x).astype(np.float64), to_np(t)
    logp, ent, lp = P.token_logprobs(xf, tf, s)
    eps = _eps(V)
    with np.errstate(invalid="ignore"):
        m = xf.max(1, keepdims=True)
        dist = np.where(np.isneginf(xf), 0.0, np.abs(s * (xf - m)))
    lp_tol = dist * 2.0 ** -22 + eps + np.where(np.isneginf(lp), 0.0, np.abs(lp)) * 2.0 ** -23
    rows = np.arange(T)
    _close(to_np(o["logp"]), logp, lp_tol[rows, np.clip(tf, 0, V - 1)])
    _close(to_np(o["entropy"]), ent, (4 + 2 * ent) * eps)
    if n_top:
        idx = P.top_rows(xf, n_top)
        np.testing.assert_array_equal(to_np(o["top_idx"]), idx)
        _close(to_np(o["top_logp"]), np.take_along_axis(lp, idx, 1), np.take_along_axis(lp_tol, idx, 1))
    if not grad:
        return o
    g = torch.Generator(device="cuda").manual_seed(1)
    gl, gh = torch.randn(T, device="cuda", generator=g), torch.randn(T, device="cuda", generator=g)
    for use_l, use_h in ((True, True), (True, False), (False, True)):
        d = torch.full((T, V), 9.0, dtype=x.dtype, device="cuda")
        M.moe_token_logprobs_backward(x, t if use_l else None, o["stats"], o["entropy"] if use_h else None,
                                      gl if use_l else None, gh if use_h else None, d, scale)
        al = to_np(gl).astype(np.float64) * use_l
        ah = to_np(gh).astype(np.float64) * use_h
        ref = P.token_logprobs_grad(xf, tf, s, al, ah)
        p = np.exp(lp)
        lpf = np.where(np.isneginf(lp), 0.0, lp)
        bracket = np.abs(al)[:, None] + np.abs(ah)[:, None] * (np.abs(lpf) + ent[:, None] + 1)
        p_rel = eps + (np.abs(lpf) + dist + 4) * 2.0 ** -22
        tol = s * (p * bracket * (2 * p_rel + 2.0 ** -21) + np.abs(ah)[:, None] * p * (lp_tol + (4 + 2 * ent)[:, None] * eps)
                   + np.abs(al)[:, None] * 2.0 ** -22 * (p > 0)) + 2.0 ** -23 * np.abs(ref)
        if x.dtype == BF16:
            tol = tol + 2.0 ** -8 * np.abs(ref)
        _close(to_np(d), ref, tol + 1e-37)
    return o


def _logits(T, V, dtype, pad=0, shift=0, seed=0, std=3.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.empty(T * (V + pad) + shift, dtype=dtype, device="cuda").normal_(0, std, generator=gen)
    return buf[shift:].view(T, V + pad)[:, :V]


def _targets(T, V, seed=0, low=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + 77)
    return torch.randint(low, V, (T,), device="cuda", generator=gen)


@pytest.mark.parametrize("V", [1, 2, 7, 8, 31, 33, 255, 256, 257, 1000, 2049, 8191, 50001])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1, 5])
def test_vocabulary_sizes(M, V, dtype, T):
    _check(M, _logits(T, V, dtype, seed=V), _targets(T, V), n_top=20)


@pytest.mark.parametrize("T", [1, 2, 3, 18, 19, 20, 37, 75, 76, 77, 150, 153, 300, 305, 1000])
def test_row_counts(M, T):
    """Every way a row may be split over CTAs gives the same answers."""
    _check(M, _logits(T, 3001, BF16, seed=T), _targets(T, 3001, low=-1), n_top=8, grad=T < 80)


@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (3, 5), (8, 8), (64, 0), (7, 1)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strides_and_alignments(M, pad, shift, dtype):
    _check(M, _logits(6, 1003, dtype, pad, shift), _targets(6, 1003).int(), n_top=32)
    _check(M, _logits(6, 1024, dtype, pad, shift), _targets(6, 1024).int(), n_top=32)


@pytest.mark.parametrize("scale", [1.0, 0.05, 1.25, 7.0, 100.0])
@pytest.mark.parametrize("n_top", [0, 1, 2, 31, 32])
def test_scales_and_top_lengths(M, scale, n_top):
    _check(M, _logits(4, 4099, F32, seed=3), _targets(4, 4099), scale, n_top)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [9, 700])
def test_masks_ties_and_orders(M, dtype, T):
    V = 2500
    x = _logits(T, V, dtype, seed=9)
    t = _targets(T, V, seed=2, low=-1)
    low = torch.finfo(dtype).min
    x[0] = 1.5                                             # all equal: the lowest indices
    x[1] = torch.arange(V, device="cuda").to(dtype) / 64   # ascending (with ties in BF16)
    x[2] = -torch.arange(V, device="cuda").to(dtype) / 64  # descending
    x[3] = -INF                                            # masked throughout
    x[4, 1:] = -INF                                        # one logit left, not always the target
    x[5, ::2] = -INF
    x[6] = low                                             # the lowest value everywhere: uniform
    x[7, 100:] = low                                       # masks of the lowest value
    x[8, ::3], x[8, 1::3] = 0.0, -0.0                      # signed zeros tie
    t[3], t[4], t[5], t[7] = 11, 2000, 0, 1200             # masked targets
    _check(M, x, t.int(), 1.0, 32)
    _check(M, x, t, 0.5, 7)


@pytest.mark.parametrize("T", [1, 40, 700])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_one_logit_left_is_certain(M, T, dtype):
    """A distribution of one token: log probability and entropy exactly 0."""
    V = 3333
    x = torch.full((T, V), -INF, dtype=dtype, device="cuda")
    t = _targets(T, V)
    x[torch.arange(T, device="cuda"), t] = torch.randn(T, device="cuda").mul_(20).to(dtype)
    for scale in (1.0, 0.7, 1.25):
        o = _forward(M, x, t, scale, 3)
        assert not o["logp"].any() and not o["entropy"].any()
        assert torch.equal(o["top_idx"][:, 0].long(), t) and not o["top_logp"][:, 0].any()


@pytest.mark.parametrize("T", [3, 40, 700])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("left", [0, 1, 2, 7, 31, 33, 200])
def test_few_logits_left(M, T, dtype, left):
    """Grammar-masked rows: `left` logits, at the front, at the end, spread, in one run; the
    masked ones fill the list by index."""
    V = 9001
    gen = torch.Generator(device="cuda").manual_seed(left)
    full = _logits(T, V, dtype, seed=left)
    x = torch.full((T, V), -INF, dtype=dtype, device="cuda")
    for r in range(T):
        at = (torch.arange(left, device="cuda"), V - 1 - torch.arange(left, device="cuda"),
              torch.randperm(V, generator=gen, device="cuda")[:left], 4000 + torch.arange(left, device="cuda"))[r % 4]
        x[r, at] = full[r, at]
    for n in (1, 8, 32):
        _check(M, x, _targets(T, V).int(), 1.0, n, grad=T < 10)


def test_extreme_values(M):
    """Logits of up to the largest finite values, both signs; probabilities that underflow."""
    x = torch.zeros((4, 600), device="cuda")
    big = torch.finfo(F32).max
    x[0, 5], x[0, 6] = big, -big
    x[1, :] = -big
    x[1, 9] = big
    x[2, :300] = 200.0
    x[3] = torch.linspace(-1e4, 1e4, 600, device="cuda")
    _check(M, x, torch.tensor([5, 9, 3, 599], device="cuda"), 1.0, 10)


def test_nan_and_infinity_stay_in_their_row(M):
    V = 3000
    x = _logits(4, V, F32, seed=4)
    clean = x.clone()
    x[1, 2000] = float("nan")
    x[2, 7] = INF
    t = _targets(4, V)
    a, b = _forward(M, x, t, 1.0, 8), _forward(M, clean, t, 1.0, 8)
    for k in a:
        assert torch.equal(a[k][[0, 3]], b[k][[0, 3]])
    for r in (1, 2):
        assert torch.isnan(a["logp"][r]) and torch.isnan(a["entropy"][r])
        idx = a["top_idx"][r]
        assert int(idx.min()) >= 0 and int(idx.max()) < V and len(set(idx.tolist())) == 8
    g = torch.randn(4, device="cuda")
    d, e = torch.empty_like(x), torch.empty_like(x)
    M.moe_token_logprobs_backward(x, t, a["stats"], a["entropy"], g, g, d)
    M.moe_token_logprobs_backward(clean, t, b["stats"], b["entropy"], g, g, e)
    assert torch.equal(d[[0, 3]], e[[0, 3]]) and torch.isnan(d[1]).any() and torch.isnan(d[2]).any()


def test_targets_out_of_range(M):
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    M.moe_workspace_init(ws)
    x = _logits(4, 100, F32)
    t = torch.tensor([100, -7, 1 << 40, 99], device="cuda")
    logp, ent, stats = torch.empty(4, device="cuda"), torch.empty(4, device="cuda"), torch.empty(4, 2, device="cuda")
    M.moe_token_logprobs(x, t, logp, ent, stats, scale=1.0, ws=ws)
    assert logp[:3].tolist() == [0.0, 0.0, 0.0] and float(logp[3]) < 0.0
    assert M.moe_last_device_status(ws) == M.MOE_ERR_DEVICE_CHECK
    d = torch.full_like(x, 5.0)
    M.moe_token_logprobs_backward(x, t, stats, None, torch.ones(4, device="cuda"), None, d, ws=ws)
    assert not d[:3].any() and bool((d[3] != 0).all())
    assert M.moe_last_device_status(ws) == M.MOE_ERR_DEVICE_CHECK


def test_gradient_over_the_logits_and_other_streams(M):
    x = _logits(40, 5000, BF16, pad=8, seed=6)
    t = _targets(40, 5000)
    o = _forward(M, x, t, 1.0, 0)
    gl, gh = torch.randn(40, device="cuda"), torch.randn(40, device="cuda")
    d = torch.empty((40, 5000), dtype=BF16, device="cuda")
    M.moe_token_logprobs_backward(x, t, o["stats"], o["entropy"], gl, gh, d)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = x.clone()
    torch.cuda.synchronize()
    M.moe_token_logprobs_backward(y, t, o["stats"], o["entropy"], gl, gh, y, stream=side)
    side.synchronize()
    assert torch.equal(y, d)


def test_gradient_against_differences_of_the_plain_form(M):
    """Directional differences of the plain loss at the kernel's inputs."""
    T, V, scale = 6, 301, 0.8
    x, t = _logits(T, V, F32, seed=8), _targets(T, V, low=-1)
    o = _forward(M, x, t, scale, 0)
    gl, gh = torch.randn(T, device="cuda"), torch.randn(T, device="cuda")
    d = torch.empty_like(x)
    M.moe_token_logprobs_backward(x, t, o["stats"], o["entropy"], gl, gh, d, scale)
    xf, tf, s = to_np(x).astype(np.float64), to_np(t), float(np.float32(scale))
    u = np.random.default_rng(0).standard_normal((T, V))

    def loss(y):
        logp, h, _ = P.token_logprobs(y, tf, s)
        return (to_np(gl).astype(np.float64) * logp).sum() + (to_np(gh).astype(np.float64) * h).sum()

    e = 1e-5
    diff = (loss(xf + e * u) - loss(xf - e * u)) / (2 * e)
    got = (to_np(d).astype(np.float64) * u).sum()
    # the differences are good to about 1e-8; each of the T V elements to about 2^-18 of its
    # size, the sizes adding to at most sum |g| (1 + (entropy + |logp|)) per row
    assert abs(diff - got) < 1e-7 + 2.0 ** -18 * T * 30


def test_rows_past_32_bit_offsets(M):
    T, V = 1100, 2_000_000                                 # 2.2e9 elements
    x = torch.zeros((T, V), dtype=BF16, device="cuda")
    x[T - 1, V - 1] = 9.0
    t = torch.full((T,), V - 1, device="cuda")
    o = _forward(M, x, t, 1.0, 2)
    lse = np.log(np.exp(9.0) + V - 1)
    assert abs(float(o["logp"][T - 1]) - (9.0 - lse)) < 2 * _eps(V) + 2.0 ** -20
    assert o["top_idx"][T - 1].tolist() == [V - 1, 0] and o["top_idx"][0].tolist() == [0, 1]
    ones = torch.ones(T, device="cuda")
    M.moe_token_logprobs_backward(x, t, o["stats"], None, ones, None, x)
    assert abs(float(x[T - 1, V - 1]) - (1 - np.exp(9.0 - lse))) < 2.0 ** -8
    assert abs(float(x[0, 5]) * V + 1) < 2.0 ** -7


@pytest.mark.parametrize("T", [2, 250])
def test_the_largest_vocabulary(M, T):
    """2^22 FP32 logits a row (their last chunk partial at an odd alignment): ties throughout,
    so the top list is looked for the general way, with the most chunks it can have."""
    V = 1 << 22
    buf = torch.zeros(T * (V + 1) + 1, device="cuda")
    x = buf[1:].view(T, V + 1)[:, :V]
    x[:, V - 3] = 2.0
    t = torch.full((T,), V - 3, device="cuda")
    o = _forward(M, x, t, 1.0, 32)
    lse = np.log(np.exp(2.0) + V - 1)
    assert float((o["logp"] - (2.0 - lse)).abs().max()) < 2 * _eps(V) + 2.0 ** -18
    assert bool((o["top_idx"] == torch.tensor([V - 3] + list(range(31)), device="cuda")).all())


def test_same_bits_every_time(M):
    x, t = _logits(64, 40001, BF16, seed=12), _targets(64, 40001)
    a, b = _forward(M, x, t, 1.0, 8), _forward(M, x, t, 1.0, 8)
    assert all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,V", [(4, 3000), (700, 3000), (4, 50001)])
@pytest.mark.parametrize("bad", [float("nan"), INF])
def test_a_row_with_nan_or_infinity_gives_nan_for_masked_tokens_too(M, T, V, dtype, bad):
    """The sum of such a row is no number, so neither is any log probability read off it:
    those of a masked target and of the masked ends of the top list among them."""
    x = _logits(T, V, dtype, seed=4)
    t = _targets(T, V).int()
    x[1] = -INF
    x[1, [7, 1000, 2900]] = torch.tensor([0.5, bad, 1.0], device="cuda", dtype=dtype)
    t[1] = 11                                              # masked
    x[2] = -INF
    x[2, 2000] = bad                                       # nothing else left
    t[2] = 2999
    x[3, ::2] = -INF
    x[3, 5] = bad
    t[3] = 4
    o = _forward(M, x, t, 0.7, 8)
    for r in (1, 2, 3):
        assert torch.isnan(o["logp"][r]) and torch.isnan(o["entropy"][r])
        assert torch.isnan(o["top_logp"][r]).all()
        idx = o["top_idx"][r]
        assert int(idx.min()) >= 0 and int(idx.max()) < V and len(set(idx.tolist())) == 8
    assert bool(torch.isfinite(o["logp"][0])) and bool(torch.isfinite(o["top_logp"][0]).all())


def _far_logits(T, V, scale):
    """Normal FP32 logits that `scale` brings to about 0 .. 13 below a row's largest."""
    gen = torch.Generator(device="cuda").manual_seed(T + V)
    z = torch.rand((T, V), generator=gen, device="cuda", dtype=torch.float64)
    if scale > 1:
        return (2.0 ** -126 * (1 + 4 * z)).float()         # 3e38 of these: 3.5 .. 17.6
    x = ((2 * z - 1) * 3.4e38).float()                     # 1e-38 of these: -3.4 .. 3.4
    x[0, :V // 2] = torch.finfo(F32).max                   # differences that pass FP32's range
    x[0, V // 2:] = -torch.finfo(F32).max
    return x


@pytest.mark.parametrize("scale", [3e38, 2.0 ** 127, 1e-38, 2.0 ** -126])
@pytest.mark.parametrize("T,V", [(3, 600), (3, 50001), (700, 2500)])
def test_scales_at_the_ends_of_fp32(M, T, V, scale):
    """Every positive finite scale is accepted: with the largest, scale log2 e passes FP32's range,
    with the smallest the logits' differences and their sums do."""
    x, t = _far_logits(T, V, scale), _targets(T, V, low=-1)
    _check(M, x, t, scale, 5, grad=T < 10)


@pytest.mark.parametrize("scale", [3e38, 1e-38, 2.0 ** -126])
def test_gradients_at_scales_at_the_ends_of_fp32(M, scale):
    """With gradients that bring the results back into FP32's range."""
    T, V = 6, 901
    x, t = _far_logits(T, V, scale), _targets(T, V)
    x[1] = x[1].min()
    x[1, t[1]] = x[1].abs().max() * 200 if scale > 1 else x[2].max()
    s, back = float(np.float32(scale)), 1e-30 if scale > 1 else 1e30
    o = _forward(M, x, t, scale, 0)
    g = torch.Generator(device="cuda").manual_seed(1)
    gl, gh = (torch.randn(T, device="cuda", generator=g) * back for _ in range(2))
    d = torch.full((T, V), 9.0, device="cuda")
    M.moe_token_logprobs_backward(x, t, o["stats"], o["entropy"], gl, gh, d, scale)
    xf, tf = to_np(x).astype(np.float64), to_np(t)
    al, ah = to_np(gl).astype(np.float64), to_np(gh).astype(np.float64)
    _, ent, lp = P.token_logprobs(xf, tf, s)
    ref, p, eps = P.token_logprobs_grad(xf, tf, s, al, ah), np.exp(lp), _eps(V)
    dist = np.abs(s * (xf - xf.max(1, keepdims=True)))
    lp_tol = dist * 2.0 ** -22 + eps + np.abs(lp) * 2.0 ** -23
    bracket = np.abs(al)[:, None] + np.abs(ah)[:, None] * (np.abs(lp) + ent[:, None] + 1)
    p_rel = eps + (np.abs(lp) + dist + 4) * 2.0 ** -22
    tol = s * (p * bracket * (2 * p_rel + 2.0 ** -21) + np.abs(ah)[:, None] * p * (lp_tol + (4 + 2 * ent)[:, None] * eps)
               + np.abs(al)[:, None] * 2.0 ** -22 * (p > 0)) + 2.0 ** -23 * np.abs(ref)
    _close(to_np(d), ref, tol + 1e-37 * back)


def test_a_certain_token_at_the_largest_scale_has_no_gradient(M):
    """One token that is certain: g_logp (1 - p) is 0, although scale g_logp is past FP32's range."""
    V, scale = 900, 3e38
    x = torch.full((2, V), -4.0, device="cuda")
    x[:, 100] = 4.0
    t = torch.tensor([100, 5], device="cuda")
    o = _forward(M, x, t, scale, 1)
    assert o["logp"].tolist() == [0.0, -INF] and not o["entropy"].any()
    g = torch.full((2,), 10.0, device="cuda")
    d = torch.full((2, V), 9.0, device="cuda")
    M.moe_token_logprobs_backward(x, t, o["stats"], o["entropy"], g, g, d, scale)
    assert not d[0].any()
    want = torch.zeros(V, device="cuda")
    want[5], want[100] = INF, -INF
    assert torch.equal(d[1], want)
