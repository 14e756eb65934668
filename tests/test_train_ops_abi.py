"""Refusals of root-mean-square norm, its gradient, the gradient norm and the AdamW step, decided on
the host before any launch, and of their Python entry points."""
import ctypes

import pytest
import torch

from token_dispatch_expert_top_gb300 import moe as M

INV, UNS, WSP, OK = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED, M.MOE_ERR_WORKSPACE, M.MOE_OK
NAN, INF = float("nan"), float("inf")


def _norm(x=64, dt=1, rows=4, cols=64, ldx=64, res=128, ldr=64, sm=192, lds=64, w=256, wdt=0, eps=1e-6, out=320, odt=1,
          ldo=64, codes=384, scales=448, rstd=512):
    return M.lib().moe_rms_norm(x, dt, rows, cols, ldx, res, ldr, sm, lds, w, wdt, eps, out, odt, ldo, codes, scales,
                                rstd, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(x=None), INV), (dict(x=65), INV), (dict(dt=2), INV), (dict(rows=-1), INV), (dict(cols=-1), INV),
    (dict(ldx=63), INV), (dict(res=None), INV), (dict(sm=None), INV), (dict(ldr=63), INV), (dict(lds=63), INV),
    (dict(w=257), INV), (dict(wdt=2), INV), (dict(w=258), INV), (dict(eps=0.0), INV), (dict(eps=NAN), INV),
    (dict(eps=-1.0), INV), (dict(eps=INF), INV), (dict(odt=2), INV), (dict(out=321), INV), (dict(ldo=63), INV),
    (dict(out=322, odt=0), INV), (dict(codes=None), INV), (dict(scales=None), INV), (dict(rstd=514), INV),
    (dict(out=None, codes=None, scales=None), INV), (dict(cols=40), INV), (dict(rows=1 << 31), UNS),
    (dict(cols=(1 << 24) + 32, ldx=1 << 25, ldr=1 << 25, lds=1 << 25, ldo=1 << 25), UNS),
    (dict(sm=64, lds=72), INV), (dict(sm=128, lds=72), INV), (dict(out=64), INV), (dict(out=192), INV),
    (dict(out=128), INV), (dict(res=None, sm=None, out=64, odt=0), INV), (dict(res=None, sm=None, out=64, ldo=72), INV),
    (dict(rows=0, x=None), OK), (dict(cols=0), OK)])
def test_rms_norm_refusals(kw, rc):
    assert _norm(**kw) == rc


def _norm_bwd(dout=64, gdt=1, rows=4, cols=64, ldg=64, s=128, dt=1, lds=64, w=256, wdt=0, rstd=512, dsum=576, ldu=64,
              dx=640, ldx=64, dw=704, acc=0, ws=32, wsb=1 << 20):
    return M.lib().moe_rms_norm_backward(dout, gdt, rows, cols, ldg, s, dt, lds, w, wdt, rstd, dsum, ldu, dx, ldx, dw,
                                         acc, ws, wsb, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(dout=None), INV), (dict(s=None), INV), (dict(dx=None), INV), (dict(rstd=None), INV), (dict(rstd=513), INV),
    (dict(gdt=2), INV), (dict(dt=-1), INV), (dict(rows=-1), INV), (dict(ldg=63), INV), (dict(lds=63), INV),
    (dict(ldx=63), INV), (dict(ldu=63), INV), (dict(dw=705), INV), (dict(w=258), INV), (dict(wdt=5), INV),
    (dict(dx=641), INV), (dict(dx=64, ldx=72), INV), (dict(dx=128, ldx=72), INV), (dict(dx=576, ldx=72), INV),
    (dict(dx=64, gdt=0), INV), (dict(ws=None), WSP), (dict(ws=40), WSP), (dict(wsb=256), WSP),
    (dict(rows=1 << 31), UNS), (dict(rows=0, dw=None, dout=None), OK), (dict(cols=0), OK)])
def test_rms_norm_backward_refusals(kw, rc):
    assert _norm_bwd(**kw) == rc


def test_norm_workspace_bytes():
    f = M.moe_rms_norm_workspace_bytes
    assert f(-1, 8) == f(8, -1) == f(1 << 31, 8) == f(8, 1 << 25) == 0
    sizes = [f(r, 7168) for r in (0, 1, 2, 100, 1000, 10 ** 6)]
    assert sizes[0] > 0 and all(a <= b for a, b in zip(sizes, sizes[1:]))


def _tensor(**kw):
    d = dict(param=64, copy=128, grad=192, m=256, v=320, m_scales=384, v_scales=448, n=100, param_dtype=0, grad_dtype=1,
             state_dtype=0, weight_decay=0.1)
    d.update(kw)
    return M.AdamWTensor(**d)


def _step(count=1, params=True, tensor=None, **kw):
    d = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=1, seed=0)
    d.update(kw)
    t = (M.AdamWTensor * 1)(_tensor(**(tensor or {})))
    return M.lib().moe_adamw(t if tensor is not False else None, count,
                             ctypes.byref(M.AdamWParams(**d)) if params else None, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(count=-1), INV), (dict(tensor=False), INV), (dict(params=False), INV), (dict(beta1=1.0), INV),
    (dict(beta1=-0.1), INV), (dict(beta2=1.0), INV), (dict(beta2=NAN), INV), (dict(eps=0.0), INV),
    (dict(eps=1e-17), INV), (dict(eps=NAN), INV),
    (dict(lr=INF), INV), (dict(lr=NAN), INV), (dict(step=0), INV), (dict(device_lr=66), INV), (dict(device_step=68), INV),
    (dict(grad_scale=65), INV), (dict(count=0), OK), (dict(count=0, tensor=False), OK),
    (dict(tensor=dict(n=0, param=None, grad=None, m=None, v=None)), OK)])
def test_adamw_refusals(kw, rc):
    assert _step(**kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(param=None), INV), (dict(grad=None), INV), (dict(m=None), INV), (dict(v=None), INV), (dict(n=-1), INV),
    (dict(param=66), INV), (dict(copy=129), INV), (dict(grad=193), INV), (dict(m=258), INV), (dict(v=322), INV),
    (dict(param_dtype=2), INV), (dict(grad_dtype=2), INV), (dict(state_dtype=1), INV), (dict(weight_decay=-0.1), INV),
    (dict(weight_decay=NAN), INV), (dict(weight_decay=INF), INV), (dict(state_dtype=2, m_scales=None), INV),
    (dict(state_dtype=2, v_scales=None), INV), (dict(n=(1 << 40) + 1), UNS)])
def test_adamw_refuses_a_bad_tensor(kw, rc):
    assert _step(tensor=kw) == rc


def _gnorm(count=1, tensor=None, max_norm=1.0, norm=64, factor=128, ws=32, wsb=1 << 20):
    t = (M.AdamWTensor * 1)(_tensor(**(tensor or {})))
    return M.lib().moe_grad_norm(t if tensor is not False else None, count, max_norm, norm, factor, ws, wsb, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(count=-1), INV), (dict(tensor=False), INV), (dict(norm=None, factor=None), INV), (dict(norm=65), INV),
    (dict(factor=130), INV), (dict(max_norm=0.0), INV), (dict(max_norm=NAN), INV), (dict(max_norm=-1.0), INV),
    (dict(tensor=dict(grad=None)), INV), (dict(tensor=dict(grad=193)), INV), (dict(tensor=dict(n=-1)), INV),
    (dict(tensor=dict(grad_dtype=3)), INV), (dict(tensor=dict(n=1 << 41)), UNS), (dict(ws=None), WSP),
    (dict(ws=48), WSP), (dict(wsb=256), WSP)])
def test_grad_norm_refusals(kw, rc):
    assert _gnorm(**kw) == rc


def test_structs_have_the_headers_layout():
    assert ctypes.sizeof(M.AdamWTensor) == 80 and M.AdamWTensor.n.offset == 56
    assert M.AdamWTensor.weight_decay.offset == 76
    assert ctypes.sizeof(M.AdamWParams) == 72 and M.AdamWParams.device_lr.offset == 48


def test_python_entry_points_refuse_what_they_cannot_pass_on():
    x, w = torch.zeros(4, 32), torch.ones(32)
    with pytest.raises(ValueError):
        M.moe_rms_norm(x, w, x)                            # not on a CUDA device
    with pytest.raises(TypeError):
        M.moe_rms_norm(x.half(), w, x)
    with pytest.raises(ValueError):
        M.moe_rms_norm_backward(x, x, w, torch.zeros(4), x)
    with pytest.raises(ValueError):
        M.AdamWTensors([x], [x], [x], [x])
    with pytest.raises(ValueError):
        M.AdamWTensors([x, x], [x], [x], [x])
    with pytest.raises(TypeError):
        M.AdamWTensors.of_grads([x.half()])


def test_gradients_in_written_memory_are_found():
    written = [(100, 200, "params[0]"), (200, 300, "m[0]"), (1000, 1004, "v[0]")]
    for grads, want in (([], None), ([(0, 100), (300, 700), (1004, 8)], None), ([(150, 0)], None),
                        ([(0, 101)], "grads[0] and params[0]"), ([(199, 1)], "grads[0] and params[0]"),
                        ([(200, 4)], "grads[0] and m[0]"), ([(0, 50), (120, 4)], "grads[1] and params[0]"),
                        ([(0, 2000)], "grads[0] and v[0]"), ([(299, 2)], "grads[0] and m[0]"),
                        ([(900, 100), (1003, 1)], "grads[1] and v[0]")):
        assert M._first_overlap(written, grads) == want
    assert M._first_overlap([], [(0, 10)]) is None
