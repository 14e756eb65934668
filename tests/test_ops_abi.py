"""Refusals of the operators around the layer, decided on the host before any launch, and
of their Python entry points."""
import pytest
import torch

from token_dispatch_expert_top_gb300 import moe as M

INV, UNS, WSP, OK = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED, M.MOE_ERR_WORKSPACE, M.MOE_OK
NAN, INF = float("nan"), float("inf")


def _embed(ids=16, id_bytes=4, N=4, table=16, tdt=1, V=8, H=16, ld=16, scale=1.0, out=16, odt=1, ldo=16, ws=None,
           wsb=0):
    return M.lib().moe_embedding(ids, id_bytes, N, table, tdt, V, H, ld, scale, out, odt, ldo, ws, wsb, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(ids=None), INV), (dict(table=None), INV), (dict(out=None), INV), (dict(id_bytes=2), INV),
    (dict(ids=18), INV), (dict(ids=20, id_bytes=8), INV), (dict(N=-1), INV), (dict(V=0), INV), (dict(H=0), INV),
    (dict(ld=15), INV), (dict(ldo=15), INV), (dict(tdt=2), INV), (dict(odt=7), INV), (dict(table=17), INV),
    (dict(out=18, odt=0), INV), (dict(scale=NAN), INV), (dict(scale=INF), INV), (dict(ld=1 << 61), INV),
    (dict(N=(1 << 30) + 1), UNS), (dict(V=1 << 31), UNS), (dict(H=(1 << 24) + 1, ld=1 << 25, ldo=1 << 25), UNS),
    (dict(ws=16, wsb=256), WSP), (dict(ws=32, wsb=255), WSP), (dict(N=0, ids=None, out=None), OK)])
def test_embedding_refusals(kw, rc):
    assert _embed(**kw) == rc


def _embed_bwd(ids=16, id_bytes=4, N=4, V=8, H=16, dout=16, gdt=1, ldg=16, scale=1.0, dtable=16, tdt=0, ldt=16,
               acc=0, ws=32, wsb=1 << 20):
    return M.lib().moe_embedding_backward(ids, id_bytes, N, V, H, dout, gdt, ldg, scale, dtable, tdt, ldt, acc, ws,
                                          wsb, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(ids=None), INV), (dict(dout=None), INV), (dict(dtable=None), INV), (dict(id_bytes=1), INV),
    (dict(N=-1), INV), (dict(V=0), INV), (dict(ldg=15), INV), (dict(ldt=15), INV), (dict(gdt=2), INV),
    (dict(tdt=-1), INV), (dict(dtable=18), INV), (dict(scale=NAN), INV), (dict(N=(1 << 30) + 1), UNS),
    (dict(ws=None), WSP), (dict(ws=48), WSP), (dict(wsb=256), WSP), (dict(N=0, ids=None, dout=None, acc=1), OK)])
def test_embedding_backward_refusals(kw, rc):
    assert _embed_bwd(**kw) == rc


def test_embedding_workspace_bytes():
    f = M.moe_embedding_workspace_bytes
    assert f(-1, 8, 8) == f(8, 0, 8) == f(8, 8, 0) == f((1 << 30) + 1, 8, 8) == 0
    assert 0 < f(0, 8, 8) <= f(1, 8, 8) < f(1000, 8, 8) < f(1000, 8, 800)
    # two FP32 partial rows per range of at most 32 tokens, and the sorted list
    assert f(1 << 16, 1000, 7168) >= (1 << 16) * 8


@pytest.mark.parametrize("H", [1, 64, 256, 257, 1409, 2048, 7168, 100_000])
def test_a_longer_batchs_embedding_workspace_serves_a_shorter_one(H):
    f = M.moe_embedding_workspace_bytes
    sizes = [f(n, 32000, H) for n in range(0, 20_000)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    wide = [f(n, 32000, H) for n in range(20_000, 1 << 30, 7_654_321)]
    assert sizes[-1] <= wide[0] and all(a <= b for a, b in zip(wide, wide[1:]))


def _logp(logits=16, dt=1, T=4, V=64, ld=64, scale=1.0, targets=16, id_bytes=4, logp=16, entropy=16, stats=16,
          n_top=2, ti=16, tl=16, ws=None, wsb=0):
    return M.lib().moe_token_logprobs(logits, dt, T, V, ld, scale, targets, id_bytes, logp, entropy, stats, n_top,
                                      ti, tl, ws, wsb, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(logits=None), INV), (dict(logits=17), INV), (dict(dt=2), INV), (dict(T=-1), INV), (dict(V=0), INV),
    (dict(ld=63), INV), (dict(scale=0.0), INV), (dict(scale=-1.0), INV), (dict(scale=NAN), INV),
    (dict(scale=INF), INV), (dict(targets=None), INV), (dict(logp=None), INV), (dict(id_bytes=3), INV),
    (dict(targets=18), INV), (dict(n_top=-1), INV), (dict(n_top=65), INV), (dict(n_top=33), UNS),
    (dict(ti=None), INV), (dict(tl=None), INV), (dict(entropy=18), INV), (dict(stats=17), INV),
    (dict(V=(1 << 22) + 1, ld=1 << 23), UNS), (dict(T=1 << 31), UNS), (dict(ws=32, wsb=128), WSP),
    (dict(ws=40, wsb=512), WSP), (dict(T=0, logits=None), OK)])
def test_token_logprobs_refusals(kw, rc):
    assert _logp(**kw) == rc


def _logp_bwd(logits=16, dt=1, T=4, V=64, ld=64, scale=1.0, targets=16, id_bytes=4, stats=16, entropy=16, gl=16,
              gh=16, d=32, ldd=64, ws=None, wsb=0):
    return M.lib().moe_token_logprobs_backward(logits, dt, T, V, ld, scale, targets, id_bytes, stats, entropy, gl, gh,
                                               d, ldd, ws, wsb, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(logits=None), INV), (dict(d=None), INV), (dict(d=33), INV), (dict(stats=None), INV),
    (dict(gl=None, gh=None), INV), (dict(targets=None), INV), (dict(entropy=None), INV), (dict(scale=0.0), INV),
    (dict(ldd=63), INV), (dict(dt=3), INV), (dict(id_bytes=16), INV), (dict(d=16, ldd=72), INV), (dict(gl=17), INV),
    (dict(V=(1 << 22) + 1, ld=1 << 23, ldd=1 << 23), UNS), (dict(ws=32, wsb=0), WSP), (dict(T=0, d=None), OK)])
def test_token_logprobs_backward_refusals(kw, rc):
    assert _logp_bwd(**kw) == rc


def _drop(x=16, dt=1, rows=4, cols=8, ldx=8, res=None, ldr=0, p=0.5, seed=1, off=0, out=32, ldo=8):
    return M.lib().moe_dropout(x, dt, rows, cols, ldx, res, ldr, p, seed, off, out, ldo, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(x=None), INV), (dict(out=None), INV), (dict(dt=2), INV), (dict(rows=-1), INV), (dict(cols=-1), INV),
    (dict(ldx=7), INV), (dict(ldo=7), INV), (dict(res=16, ldr=7), INV), (dict(p=-0.01), INV), (dict(p=1.01), INV),
    (dict(p=NAN), INV), (dict(x=17), INV), (dict(out=16, ldo=9), INV), (dict(res=32, ldr=9), INV),
    (dict(rows=0, x=None), OK), (dict(cols=0), OK)])
def test_dropout_refusals(kw, rc):
    assert _drop(**kw) == rc


def test_python_entry_points_refuse_what_they_cannot_pass_on():
    x, i = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        M.moe_embedding(i, x, x)                           # not on a CUDA device
    with pytest.raises(TypeError):
        M.moe_embedding(i, x.double(), x)
    with pytest.raises(TypeError):
        M.moe_dropout(x.half(), x.half(), 0.5, 1)
    with pytest.raises(ValueError):
        M.moe_dropout(torch.tensor(1.0), x, 0.5, 1)
    with pytest.raises(ValueError):
        M.moe_token_logprobs(x, i)
