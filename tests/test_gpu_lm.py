"""The operators around the layer, run together as a small language model (lm.py): each
result against plain 64-bit arithmetic on the model's own intermediate tensors.  Tolerances
are the BF16 layer's (2e-2 of a row's largest value): the head's two products round to BF16
once each, as the layer's do."""
import numpy as np
import pytest
import torch

import plain_ops as P
from gpu_common import TOL, need_cuda, row_rel_err, to_np
from token_dispatch_expert_top_gb300 import synth

pytestmark = pytest.mark.gpu


def _f64(t):
    return to_np(t).astype(np.float64)


@pytest.fixture(scope="module")
def lm():
    need_cuda()
    from token_dispatch_expert_top_gb300.layer import MoeLayer
    from token_dispatch_expert_top_gb300.lm import MoeLM
    w = synth.Workload("lm_test", N=128, H=256, I=128, E=8, k=2, S=2, dtype="bf16")
    layer = MoeLayer(w, synth.make_inputs(w), train=True)
    gen = torch.Generator(device="cuda").manual_seed(3)
    table = (torch.randn((301, w.H), generator=gen, device="cuda") / 16).to(torch.bfloat16)
    return MoeLM(layer, table, embed_scale=16.0, dropout=0.2, seed=11)


def _tokens(lm, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.randint(-1, 301, (128,), generator=gen, device="cuda").int()
    targets = torch.randint(-1, 301, (128,), generator=gen, device="cuda").int()
    return ids, targets


def test_forward_and_gradients_against_the_formulas(lm):
    ids, targets = _tokens(lm, 0)
    logp, entropy = (t.clone() for t in lm.forward_train(ids, targets))
    table, i, t = _f64(lm.table), to_np(ids), to_np(targets)
    x0 = P.embedding(i, table, 16.0)
    assert np.array_equal(_f64(lm.x0), x0)                    # a power of two: exact
    y = _f64(lm.layer.out)
    h = P.dropout(y, 0.2, 11, lm.step, x0)
    assert row_rel_err(_f64(lm.h), h).max() < TOL["bf16"]
    logits = _f64(lm.logits)
    assert row_rel_err(logits, _f64(lm.h) @ table.T).max() < TOL["bf16"]
    ref_logp, ref_h, _ = P.token_logprobs(logits, t, 1.0)
    np.testing.assert_allclose(to_np(logp), ref_logp, atol=1e-5)
    np.testing.assert_allclose(to_np(entropy), ref_h, atol=1e-5)

    g = torch.Generator(device="cuda").manual_seed(1)
    gl, gh = torch.randn(128, generator=g, device="cuda"), torch.randn(128, generator=g, device="cuda") * 0.1
    hb = lm.h.clone()
    dtable, rest = lm.backward(gl, gh)
    dlogits = P.token_logprobs_grad(logits, t, 1.0, _f64(gl), _f64(gh))
    assert row_rel_err(_f64(lm.logits), dlogits).max() < TOL["bf16"]
    dl = _f64(lm.logits)
    dh = dl @ table
    assert row_rel_err(_f64(lm.dh), dh).max() < TOL["bf16"]
    assert row_rel_err(_f64(lm.dy), P.dropout(_f64(lm.dh), 0.2, 11, lm.step)).max() < TOL["bf16"]
    dx0 = _f64(lm.dx0)
    assert row_rel_err(dx0, _f64(lm.layer.dx) + _f64(lm.dh)).max() < TOL["bf16"]
    ref, _, _ = P.embedding_grad(i, dx0, 301, 16.0)
    assert row_rel_err(_f64(dtable), ref + dl.T @ _f64(hb)).max() < TOL["bf16"]
    assert len(rest) == 4 and all(torch.isfinite(r).all() for r in rest)
    assert lm.device_status() == 0


def test_score_lists_the_likeliest_tokens(lm):
    ids, targets = _tokens(lm, 5)
    logp, entropy, top_idx, top_logp = lm.score(ids, targets, n_top=4, temperature=0.5)
    x = _f64(lm.logits)
    ref_logp, ref_h, lp = P.token_logprobs(x, to_np(targets), 2.0)
    np.testing.assert_allclose(to_np(logp), ref_logp, atol=2e-5)
    np.testing.assert_allclose(to_np(entropy), ref_h, atol=2e-5)
    idx = P.top_rows(x, 4)
    np.testing.assert_array_equal(to_np(top_idx), idx)
    np.testing.assert_allclose(to_np(top_logp), np.take_along_axis(lp, idx, 1), atol=2e-5)


def test_a_bad_token_is_reported(lm):
    ids, targets = _tokens(lm, 6)
    ids[3] = 301
    lm.score(ids, targets)
    from token_dispatch_expert_top_gb300 import moe as M
    assert lm.device_status() == M.MOE_ERR_DEVICE_CHECK
    assert lm.device_status() == M.MOE_OK


def test_the_example_fits_its_batch():
    need_cuda()
    from token_dispatch_expert_top_gb300 import lm as L
    losses = L.main(steps=10)
    assert losses[-1] < 0.5 * losses[0]


def test_backward_wants_its_own_forward(lm):
    """The logits are overwritten by backward and by score: gradients of them again, or of a
    score's, would be of something else."""
    ids, targets = _tokens(lm, 8)
    g = torch.ones(128, device="cuda")
    lm.forward_train(ids, targets)
    lm.backward(g, weights=False)
    with pytest.raises(RuntimeError):
        lm.backward(g, weights=False)
    lm.forward_train(ids, targets)
    lm.score(ids, targets)
    with pytest.raises(RuntimeError):
        lm.backward(g, weights=False)
    lm.forward_train(ids, targets)
    want = [t.clone() for t in (lm.logits, lm.h)]
    first = lm.backward(g, weights=False)[0].clone()
    lm.score(ids, targets)
    lm.step -= 1                                           # the same dropout again
    lm.forward_train(ids, targets)
    assert torch.equal(lm.logits, want[0]) and torch.equal(lm.h, want[1])
    assert torch.equal(lm.backward(g, weights=False)[0], first)


def test_the_tables_gradient_keeps_its_32_bits(lm):
    """The head's part and the embedding's are sums of FP32 precision, not rounded to BF16 between.
    The head's: products of two BF16 numbers are exact in FP32, and N of them are added, each
    addition off by at most 2^-23 of the absolute sum (2^-24, or twice that where the tensor
    cores cut bits off); the embedding's adds a row per token of the id, the scale's rounding and its
    own addition onto the head's."""
    ids, targets = _tokens(lm, 9)
    gen = torch.Generator(device="cuda").manual_seed(2)
    lm.forward_train(ids, targets)
    h = _f64(lm.h)
    dtable, _ = lm.backward(torch.randn(128, generator=gen, device="cuda"), weights=False)
    dl, dx0, i = _f64(lm.logits), _f64(lm.dx0), to_np(ids)
    emb, emb_abs, count = P.embedding_grad(i, dx0, 301, 16.0)
    ref, size = dl.T @ h + emb, np.abs(dl).T @ np.abs(h) + emb_abs
    tol = (128 + 4 + count[:, None]) * 2.0 ** -23 * size
    assert np.all(np.abs(_f64(dtable) - ref) <= tol)
