"""The operators around the layer straight behind the kernels that write their inputs.  Their
launches overlap the end of the kernel before them in the stream, so each has to wait for it
before it reads anything: many repeats without a host sync, on inputs that change every time,
and every result is compared bit for bit with one computed from the same inputs at leisure.
Gradients sum small whole numbers, which FP32 adds exactly in any order."""
import pytest
import torch

from gpu_common import need_cuda

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def M():
    need_cuda()
    from token_dispatch_expert_top_gb300 import moe
    return moe


def _sums(ids, dout, V):
    live = ids >= 0
    out = torch.zeros((V, dout.shape[1]), device="cuda")
    return out.index_add_(0, ids.clamp(min=0).long(), dout.float() * live.unsqueeze(1))


@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
@pytest.mark.parametrize("N,H,dtype", [(1, 2048, BF16), (700, 72, BF16), (700, 73, F32), (3000, 1409, BF16)])
def test_lookup_behind_the_kernels_that_write_ids_and_table(M, N, H, dtype, idt):
    V, repeats = 999, 60
    gen = torch.Generator(device="cuda").manual_seed(N + H)
    all_ids = torch.randint(-1, V, (repeats, N), generator=gen, device="cuda").to(idt)
    tables = torch.randn((3, V, H), generator=gen, device="cuda").to(dtype)
    ids, table = torch.zeros(N, dtype=idt, device="cuda"), torch.empty((V, H), dtype=dtype, device="cuda")
    outs = torch.full((repeats, N, H), 7.0, dtype=dtype, device="cuda")
    torch.cuda.synchronize()
    for i in range(repeats):
        if i % 2:                                          # the ids are the last thing written ...
            M.moe_dropout(tables[i % 3], table, 0.0, 1, 0)
            torch.add(all_ids[i], 0, out=ids)
        else:                                              # ... or the table, by a kernel that overlaps too
            torch.add(all_ids[i], 0, out=ids)
            M.moe_dropout(tables[i % 3], table, 0.0, 1, 0)
        M.moe_embedding(ids, table, outs[i])
    for i in range(repeats):
        want = tables[i % 3][all_ids[i].clamp(min=0).long()] * (all_ids[i] >= 0).unsqueeze(1)
        assert torch.equal(outs[i], want)


@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
@pytest.mark.parametrize("N,V,H", [(600, 800, 40), (1500, 800, 40), (5000, 3000, 136)])
def test_table_gradient_behind_the_kernels_that_write_its_inputs(M, N, V, H, idt):
    repeats = 40
    gen = torch.Generator(device="cuda").manual_seed(N)
    all_ids = torch.randint(-1, V, (repeats, N), generator=gen, device="cuda").to(idt)
    rows = torch.randint(-8, 9, (3, N, H), generator=gen, device="cuda").float()
    ids, dout = torch.zeros(N, dtype=idt, device="cuda"), torch.empty((N, H), device="cuda")
    outs = torch.full((repeats, V, H), 7.0, device="cuda")
    ws = torch.empty(M.moe_embedding_workspace_bytes(N, V, H), dtype=torch.uint8, device="cuda")
    M.moe_workspace_init(ws)
    torch.cuda.synchronize()
    for i in range(repeats):
        if i % 2:
            M.moe_dropout(rows[i % 3], dout, 0.0, 1, 0)
            torch.add(all_ids[i], 0, out=ids)
        else:
            torch.add(all_ids[i], 0, out=ids)
            M.moe_dropout(rows[i % 3], dout, 0.0, 1, 0)
        M.moe_embedding_backward(ids, dout, outs[i], 1.0, False, ws)
    for i in range(repeats):
        assert torch.equal(outs[i], _sums(all_ids[i], rows[i % 3], V))
    assert M.moe_last_device_status(ws) == M.MOE_OK


@pytest.mark.parametrize("V,H,dtype", [(70_001, 1024, F32), (20_000, 7168, BF16)])
def test_large_table_gradient_zeroes_the_rows_of_its_own_ids(M, V, H, dtype):
    """A table of more than 256 MB: its zero rows are found from marks that the ordering of the
    same call has just written, over another call's.  Rows of 4 KB (several to a CTA, the last
    CTA not full) and of 14 KB."""
    N, repeats = 2000, 12
    gen = torch.Generator(device="cuda").manual_seed(V)
    all_ids = torch.randint(-1, V, (repeats, N), generator=gen, device="cuda").int()
    dout = torch.randint(-8, 9, (N, H), generator=gen, device="cuda").to(dtype)
    ids = torch.zeros(N, dtype=torch.int32, device="cuda")
    a, b = (torch.full((V, H), 5.0, dtype=dtype, device="cuda") for _ in range(2))
    ws = torch.empty(M.moe_embedding_workspace_bytes(N, V, H), dtype=torch.uint8, device="cuda")
    M.moe_workspace_init(ws)
    for i in range(0, repeats, 2):
        for j, out in ((i, a), (i + 1, b)):                # two in a row: the second one's marks over the first's
            torch.add(all_ids[j], 0, out=ids)
            M.moe_embedding_backward(ids, dout, out, 1.0, False, ws)
        assert torch.equal(a, _sums(all_ids[i], dout, V).to(dtype))
        assert torch.equal(b, _sums(all_ids[i + 1], dout, V).to(dtype))
    assert M.moe_last_device_status(ws) == M.MOE_OK


@pytest.mark.parametrize("T,V", [(1, 50_001), (40, 3001), (700, 2500)])
def test_log_probabilities_and_gradient_behind_the_kernels_that_write_the_logits(M, T, V):
    repeats = 30
    gen = torch.Generator(device="cuda").manual_seed(T)
    source = torch.randn((3, T, V), generator=gen, device="cuda").to(BF16)
    all_t = torch.randint(-1, V, (repeats, T), generator=gen, device="cuda").int()
    f = dict(dtype=F32, device="cuda")
    g = torch.ones(T, **f)

    def call(x, t, ws=None):
        o = [torch.empty(T, **f), torch.empty(T, **f), torch.empty((T, 2), **f),
             torch.empty((T, 4), dtype=torch.int32, device="cuda"), torch.empty((T, 4), **f), torch.empty_like(x)]
        M.moe_token_logprobs(x, t, *o[:5], 1.25, ws)
        M.moe_token_logprobs_backward(x, t, o[2], o[1], g, g, o[5], 1.25, ws)
        return o

    want = []
    for i in range(repeats):
        want.append(call(source[i % 3], all_t[i]))
        torch.cuda.synchronize()
    x, t = torch.zeros((T, V), dtype=BF16, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    got = []
    for i in range(repeats):
        if i % 2:
            M.moe_dropout(source[i % 3], x, 0.0, 1, 0)
            torch.add(all_t[i], 0, out=t)
        else:
            torch.add(all_t[i], 0, out=t)
            M.moe_dropout(source[i % 3], x, 0.0, 1, 0)
        got.append(call(x, t))
    for w, o in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(w, o))
