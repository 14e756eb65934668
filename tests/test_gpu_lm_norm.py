"""The small language model with norms in front of the layer and the head, and its optimiser
(lm.py): each result against plain 64-bit arithmetic on the model's own intermediate tensors, as
in test_gpu_lm.py.  Tolerances are the BF16 layer's for what is rounded to BF16 on the way, and
those of test_gpu_norm.py and test_gpu_adamw.py for the operators themselves."""
import numpy as np
import pytest
import torch

import plain_ops as P
import plain_train as T
from gpu_common import TOL, need_cuda, row_rel_err, to_np
from token_dispatch_expert_top_gb300 import synth

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _f64(t):
    return to_np(t).astype(np.float64)


def _model(**kw):
    need_cuda()
    from token_dispatch_expert_top_gb300.layer import MoeLayer
    from token_dispatch_expert_top_gb300.lm import MoeLM
    w = synth.Workload("lm_test", N=128, H=256, I=128, E=8, k=2, S=2, dtype="bf16")
    layer = MoeLayer(w, synth.make_inputs(w), train=True)
    gen = torch.Generator(device="cuda").manual_seed(3)
    table = (torch.randn((301, w.H), generator=gen, device="cuda") / 16).to(torch.bfloat16)
    lm = MoeLM(layer, table, embed_scale=16.0, dropout=0.2, seed=11, norm_eps=1e-5, **kw)
    for t in (lm.w_in, lm.w_out):
        t.copy_(torch.rand(w.H, generator=gen, device="cuda") + 0.5)
    ids = torch.randint(-1, 301, (128,), generator=gen, device="cuda").int()
    targets = torch.randint(-1, 301, (128,), generator=gen, device="cuda").int()
    return lm, ids, targets


def test_forward_and_gradients_against_the_formulas():
    lm, ids, targets = _model()
    logp, entropy = (t.clone() for t in lm.forward_train(ids, targets))
    table, i, t = _f64(lm.table), to_np(ids), to_np(targets)
    x0 = P.embedding(i, table, 16.0)
    assert np.array_equal(_f64(lm.x0), x0)                    # a power of two: exact
    n_in, r_in = T.rms_norm(x0, _f64(lm.w_in), 1e-5)          # rows without a token: zeros
    assert np.all(np.abs(_f64(lm.n_in) - n_in) <= (32 * U + 2.0 ** -8) * np.abs(n_in) * (1 + 2 ** -8))
    assert np.all(np.abs(_f64(lm.r_in) - r_in) <= 32 * U * r_in)
    y = _f64(lm.layer.out)
    assert row_rel_err(_f64(lm.h), P.dropout(y, 0.2, 11, lm.step, x0)).max() < TOL["bf16"]
    h = _f64(lm.h)
    n_out, r_out = T.rms_norm(h, _f64(lm.w_out), 1e-5)
    assert np.all(np.abs(_f64(lm.n_out) - n_out) <= (32 * U + 2.0 ** -8) * np.abs(n_out) * (1 + 2 ** -8))
    logits = _f64(lm.logits)
    assert row_rel_err(logits, _f64(lm.n_out) @ table.T).max() < TOL["bf16"]
    ref_logp, ref_h, _ = P.token_logprobs(logits, t, 1.0)
    np.testing.assert_allclose(to_np(logp), ref_logp, atol=1e-5)
    np.testing.assert_allclose(to_np(entropy), ref_h, atol=1e-5)

    g = torch.Generator(device="cuda").manual_seed(1)
    gl = torch.randn(128, generator=g, device="cuda")
    kept = {k: getattr(lm, k).clone() for k in ("h", "n_out", "x0", "r_in", "r_out")}
    dtable, _ = lm.backward(gl)
    dl = _f64(lm.logits)
    assert row_rel_err(dl, P.token_logprobs_grad(logits, t, 1.0, _f64(gl), np.zeros(128))).max() < TOL["bf16"]
    dn = dl @ table                                           # rounded to BF16, then through the norm
    dh, dw_out, _ = T.rms_norm_grad(dn, h, _f64(lm.w_out), _f64(kept["r_out"]), None)
    assert row_rel_err(_f64(lm.dh), dh).max() < TOL["bf16"]
    # dn's rounding, half a step of each term
    terms = (np.abs(dn) * np.abs(h) * _f64(kept["r_out"])[:, None]).sum(0)
    assert np.all(np.abs(_f64(lm.dw_out) - dw_out) <= (2.0 ** -8 + 2.0 ** -12) * terms)
    dx0, dw_in, _ = T.rms_norm_grad(_f64(lm.layer.dx), x0, _f64(lm.w_in), _f64(kept["r_in"]), _f64(lm.dh))
    assert row_rel_err(_f64(lm.dx0), dx0).max() < TOL["bf16"]
    terms = (np.abs(_f64(lm.layer.dx)) * np.abs(x0) * _f64(kept["r_in"])[:, None]).sum(0)
    assert np.all(np.abs(_f64(lm.dw_in) - dw_in) <= 132 * U * terms)
    emb, emb_abs, count = P.embedding_grad(i, _f64(lm.dx0), 301, 16.0)
    n = _f64(kept["n_out"])
    tol = (128 + 4 + count[:, None]) * 2.0 ** -23 * (np.abs(dl).T @ np.abs(n) + emb_abs)
    assert np.all(np.abs(_f64(dtable) - (dl.T @ n + emb)) <= tol)
    assert lm.device_status() == 0


def test_score_is_the_training_forward_without_dropout():
    lm, ids, targets = _model()
    lm.dropout = 0.0
    want = [t.clone() for t in lm.forward_train(ids, targets)]
    logits = lm.logits.clone()
    got = lm.score(ids, targets, n_top=2)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(lm.logits, logits)


@pytest.mark.parametrize("eight_bits", [False, True])
@pytest.mark.parametrize("max_norm", [1e-3, 1e9])
def test_optimiser_steps_the_models_own_weights(eight_bits, max_norm):
    from token_dispatch_expert_top_gb300.lm import LmOptimizer
    lm, ids, targets = _model()
    opt = LmOptimizer(lm, lr=1e-2, max_norm=max_norm, eight_bits=eight_bits, seed=7)
    weights = [(opt.master, lm.dtable, 0.1), (lm.layer.w_router, lm.layer.dw_router, 0.0), (lm.w_in, lm.dw_in, 0.0),
               (lm.w_out, lm.dw_out, 0.0)]
    before = [_f64(p) for p, _, _ in weights]
    lm.forward_train(ids, targets)
    lm.backward(torch.ones(128, device="cuda") / 128, weights=False)
    norm = float(opt.step())
    grads = [_f64(g) for _, g, _ in weights]
    want, f = T.grad_norm(grads, max_norm)
    assert abs(norm - want) <= 30 * U * want and abs(float(opt.factor) - f) <= 32 * U * f
    for (p, _, wd), p0, g in zip(weights, before, grads):
        m, v = T.moments(g, 0.0, 0.0, 0.9, 0.95, f)
        ref, d = T.update(p0, m, v, 1e-2, 0.9, 0.95, 1e-8, wd, 1)
        half = 2.0 ** -8 if p.dtype == torch.bfloat16 else U
        # the first step is lr times m / sqrt(v), both of one gradient, whose factor is off by 62 u
        tol = 3 * U * np.abs(p0) + np.abs(d * m) * 2.0 ** -16 + half * np.abs(ref) * (1 + 2 ** -7)
        assert np.all(np.abs(_f64(p) - ref) <= tol)
    assert torch.equal(lm.table, opt.master.to(torch.bfloat16))    # what the next forward reads
    assert int(opt.number) == 1


def test_optimiser_keeps_out_a_step_that_is_not_finite():
    from token_dispatch_expert_top_gb300.lm import LmOptimizer
    lm, ids, targets = _model()
    opt = LmOptimizer(lm)
    lm.forward_train(ids, targets)
    lm.backward(torch.ones(128, device="cuda"), weights=False)
    lm.dw_in[3] = float("nan")
    before = [t.clone() for t in (opt.master, lm.table, lm.w_in, lm.w_out, lm.layer.w_router)]
    assert not np.isfinite(float(opt.step()))
    assert all(torch.equal(a, b) for a, b in zip(before, (opt.master, lm.table, lm.w_in, lm.w_out, lm.layer.w_router)))
    assert int(opt.number) == 0                               # it is no step that moments have to be corrected for
    lm.forward_train(ids, targets)
    lm.backward(torch.ones(128, device="cuda"), weights=False)
    assert np.isfinite(float(opt.step())) and int(opt.number) == 1
    assert not torch.equal(before[1], lm.table)


def test_steps_below_the_routers_last_place_add_up():
    """64 steps of 1e-5, where half a last place of the router's BF16 weights is 1e-4.  FP32 weights and moments
    round each step: 64 times 3 u of the weight and 2^-16 of the step; then half a step of BF16."""
    from token_dispatch_expert_top_gb300.lm import LmOptimizer
    lm, ids, targets = _model()
    opt = LmOptimizer(lm, lr=1e-5, max_norm=float("inf"))
    lm.forward_train(ids, targets)
    lm.backward(torch.ones(128, device="cuda"), weights=False)
    p = start = _f64(lm.layer.w_router)
    g, m, v = _f64(lm.layer.dw_router), 0.0, 0.0
    for t in range(1, 65):
        opt.step()
        m, v = T.moments(g, m, v, 0.9, 0.95)
        p, _ = T.update(p, m, v, float(np.float32(1e-5)), 0.9, 0.95, 1e-8, 0.0, t)
    tol = 64 * (3 * U * (np.abs(start) + 1e-3) + 1e-5 * 2.0 ** -16) + 2.0 ** -8 * np.abs(p)
    assert np.all(np.abs(_f64(lm.layer.w_router) - p) <= tol * (1 + 2.0 ** -8))
    assert (np.abs(p - start) > 2 * tol).mean() > 0.5          # a router left as it was is out of that


def test_dropout_and_the_rounding_of_moments_take_different_bits():
    """Both default to one seed, and count steps from 1 and element groups from 0."""
    from token_dispatch_expert_top_gb300.lm import LmOptimizer
    lm, ids, targets = _model()
    lm.seed = 0
    opt = LmOptimizer(lm, eight_bits=True)
    lm.forward_train(ids, targets)
    lm.backward(torch.ones(128, device="cuda") / 128, weights=False)
    opt.step()
    n = 8192
    e = opt.tensors.entries[0]
    m, _ = T.moments(_f64(lm.dtable).reshape(-1)[:n], 0.0, 0.0, 0.9, 0.95, float(opt.factor))
    codes, scales = (t.reshape(-1).cpu().numpy().astype(np.int64) for t in opt.tensors._kept[1][:1] + opt.tensors._kept[4][:1])
    assert e.m == opt.tensors._kept[1][0].data_ptr()

    def agreeing(seed):
        return (T.encode(m, scales[:n // 32], T.bits16(n, seed, 1, 0), False) == codes[:n]).mean()

    assert agreeing(opt.seed) >= 0.999 and agreeing(lm.seed) <= 0.9


def test_a_captured_step_is_the_step():
    """Forward, backward and update replayed from one graph, against the same steps called directly."""
    from token_dispatch_expert_top_gb300.lm import LmOptimizer
    results = []
    for captured in (False, True):
        lm, ids, targets = _model()
        lm.dropout = 0.0                                      # (its counter is a number of the call)
        opt = LmOptimizer(lm, eight_bits=True)
        g = torch.ones(128, device="cuda") / 128

        def step():
            lm.forward_train(ids, targets)
            lm.backward(g, weights=False)
            opt.step()

        step()
        torch.cuda.synchronize()
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        for _ in range(3):
            graph.replay() if captured else step()
        results.append([t.clone() for t in (opt.master, lm.table, lm.w_in, lm.layer.w_router, opt.number)])
    assert int(results[0][4]) == 4
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_the_example_with_norms_runs():
    need_cuda()
    from token_dispatch_expert_top_gb300 import lm as L
    losses = L.main(steps=4, adamw=True)
    assert len(losses) == 4 and np.all(np.isfinite(losses))
