"""The operators around the layer inside a CUDA graph: one capture, replayed on new inputs in
the same buffers, gives the bits that direct calls give."""
import pytest
import torch

from gpu_common import need_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,V,H,n", [(1, 5003, 264, 20), (64, 1001, 40, 5), (1500, 777, 128, 3)])
def test_graph_replays_equal_direct_calls(N, V, H, n):
    need_cuda()
    from token_dispatch_expert_top_gb300 import moe as M
    dev = dict(device="cuda")
    ids, targets = (torch.zeros(N, dtype=torch.int32, **dev) for _ in range(2))
    table, dtable = torch.zeros(V, H, dtype=torch.bfloat16, **dev), torch.empty(V, H, **dev)
    x, h = (torch.empty(N, H, dtype=torch.bfloat16, **dev) for _ in range(2))
    logits, dlogits = torch.zeros(N, V, dtype=torch.bfloat16, **dev), torch.empty(N, V, dtype=torch.bfloat16, **dev)
    logp, entropy, g = torch.empty(N, **dev), torch.empty(N, **dev), torch.ones(N, **dev)
    stats = torch.empty(N, 2, **dev)
    top_idx, top_logp = torch.empty(N, n, dtype=torch.int32, **dev), torch.empty(N, n, **dev)
    ws = torch.empty(M.moe_embedding_workspace_bytes(N, V, H), dtype=torch.uint8, **dev)
    M.moe_workspace_init(ws)
    results = (x, h, logp, entropy, stats, top_idx, top_logp, dlogits, dtable)

    def step():
        M.moe_embedding(ids, table, x, 2.0, ws)
        M.moe_dropout(x, h, 0.25, 9, 4, residual=x)
        M.moe_token_logprobs(logits, targets, logp, entropy, stats, top_idx, top_logp, 1.5, ws)
        M.moe_token_logprobs_backward(logits, targets, stats, entropy, g, g, dlogits, 1.5, ws)
        M.moe_embedding_backward(ids, h, dtable, 0.5, False, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        ids.copy_(torch.randint(-1, V, (N,), generator=gen, **dev))
        targets.copy_(torch.randint(-1, V, (N,), generator=gen, **dev))
        table.copy_(torch.randn(V, H, generator=gen, **dev))
        logits.copy_(torch.randn(N, V, generator=gen, **dev))
        step()
        want = [r.clone() for r in results]
        for r in results:
            r.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(r, w) for r, w in zip(results, want))
    assert M.moe_last_device_status(ws) == M.MOE_OK
