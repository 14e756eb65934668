"""A small language model around one MoE layer, from token ids to log probabilities and back:

    x0 = scale * table[ids]                    moe_embedding
    y  = layer(x0)                             moe_forward_train / moe_forward
    h  = x0 + dropout(y)                       moe_dropout, the residual stream
    logits = h . table^T                       a plain matrix product (tied head)
    logp, entropy, alternatives                moe_token_logprobs

and the gradients in the other direction: moe_token_logprobs_backward over the logits' own
buffer, the two products of the head, moe_dropout again with the same counters,
moe_backward, and moe_embedding_backward accumulated onto the head's part of the table's
gradient.  PyTorch allocates memory and multiplies the head's matrices; everything else
runs in libmoe's kernels.

    python -m token_dispatch_expert_top_gb300.lm        # a few steps on synthetic tokens
"""
from __future__ import annotations

import torch

from . import moe as M
from .layer import MoeLayer


class MoeLM:
    """Token embedding, a MoeLayer with residual dropout, and a tied head.

    table: [V][H] BF16, the embedding and the head; layer: a BF16 or MXFP8 MoeLayer (made
    with train=True for `forward_train`) whose N is the number of tokens of a call."""

    def __init__(self, layer: MoeLayer, table: torch.Tensor, embed_scale: float = 1.0, dropout: float = 0.1,
                 seed: int = 0):
        self.layer, self.table = layer, table.contiguous()
        self.embed_scale, self.dropout, self.seed, self.step = embed_scale, dropout, seed, 0
        self.kept = False                                     # what `backward` needs is in place
        V, H = table.shape
        N, dev = layer.w.N, table.device
        f32 = dict(dtype=torch.float32, device=dev)
        self.x0 = torch.empty((N, H), dtype=torch.bfloat16, device=dev)
        self.h = torch.empty_like(self.x0)
        self.logits = torch.empty((N, V), dtype=torch.bfloat16, device=dev)
        self.logp, self.entropy, self.stats = torch.empty(N, **f32), torch.empty(N, **f32), torch.empty((N, 2), **f32)
        self.ws = torch.empty(M.moe_embedding_workspace_bytes(N, V, H), dtype=torch.uint8, device=dev)
        M.moe_workspace_init(self.ws)
        if layer.train:
            self.dh, self.dy, self.dx0 = (torch.empty_like(self.x0) for _ in range(3))
            self.dtable = torch.empty((V, H), **f32)

    def score(self, ids: torch.Tensor, targets: torch.Tensor, n_top: int = 0, temperature: float = 1.0):
        """(logp, entropy, top_idx, top_logp) of the targets' and the n_top likeliest tokens,
        without dropout; every tensor is the model's own and is overwritten by the next call
        (the top lists are new).  What an earlier forward_train kept for `backward` is lost."""
        self.kept = False
        M.moe_embedding(ids, self.table, self.x0, self.embed_scale, self.ws)
        y = self.layer.forward(self.x0)
        M.moe_dropout(y, self.h, 0.0, self.seed, 0, residual=self.x0)
        torch.mm(self.h, self.table.t(), out=self.logits)
        N = self.h.shape[0]
        top_idx = torch.empty((N, n_top), dtype=torch.int32, device=self.h.device)
        top_logp = torch.empty((N, n_top), dtype=torch.float32, device=self.h.device)
        M.moe_token_logprobs(self.logits, targets, self.logp, self.entropy, None, top_idx, top_logp, 1.0 / temperature,
                             self.ws)
        return self.logp, self.entropy, top_idx, top_logp

    def forward_train(self, ids: torch.Tensor, targets: torch.Tensor):
        """(logp, entropy) of the targets, keeping what `backward` needs.  Negative ids and
        targets are padding."""
        self.kept = False
        self.ids, self.targets = ids, targets
        self.step += 1
        M.moe_embedding(ids, self.table, self.x0, self.embed_scale, self.ws)
        y = self.layer.forward_train(self.x0)
        M.moe_dropout(y, self.h, self.dropout, self.seed, self.step, residual=self.x0)
        torch.mm(self.h, self.table.t(), out=self.logits)
        M.moe_token_logprobs(self.logits, targets, self.logp, self.entropy, self.stats, scale=1.0, ws=self.ws)
        self.kept = True
        return self.logp, self.entropy

    def backward(self, g_logp: torch.Tensor, g_entropy: torch.Tensor | None = None, weights: bool = True):
        """Gradients of the last forward_train for the gradients of its two results:
        (dtable, the layer's (dW_router, dbias, dW_gate_up, dW_down)).  Overwrites the logits: once
        per forward_train, and before any `score`."""
        if not self.kept:
            raise RuntimeError("backward: no forward_train's tensors are kept (one backward each, no score between)")
        self.kept = False
        M.moe_token_logprobs_backward(self.logits, self.targets, self.stats,
                                      None if g_entropy is None else self.entropy, g_logp, g_entropy, self.logits,
                                      1.0, self.ws)
        dlogits = self.logits
        torch.mm(dlogits, self.table, out=self.dh)
        torch.mm(dlogits.t(), self.h, out_dtype=torch.float32, out=self.dtable)   # not rounded to BF16 on the way
        M.moe_dropout(self.dh, self.dy, self.dropout, self.seed, self.step)
        dx, *rest = self.layer.backward(self.dy, self.x0, weights=weights)
        torch.add(dx, self.dh, out=self.dx0)                  # through the layer and past it
        M.moe_embedding_backward(self.ids, self.dx0, self.dtable, self.embed_scale, True, self.ws)
        return self.dtable, rest

    def device_status(self) -> int:
        """The first device error of the model's own calls or of its layer's, then reset."""
        s = M.moe_last_device_status(self.ws)
        s = s or self.layer.device_status()
        return s or (self.layer.backward_status() if self.layer.train else 0)


def main(steps: int = 20, V: int = 1000, lr: float = 300.0) -> list[float]:
    """Fits the table to one batch of synthetic tokens; returns the mean losses."""
    from . import synth
    w = synth.Workload("lm_small", N=256, H=512, I=256, E=16, k=4, S=4, dtype="bf16")
    layer = MoeLayer(w, synth.make_inputs(w), train=True)
    gen = torch.Generator(device="cuda").manual_seed(1)
    table = (torch.randn((V, w.H), generator=gen, device="cuda") / w.H ** 0.5).to(torch.bfloat16)
    lm = MoeLM(layer, table, embed_scale=w.H ** 0.5)
    ids = torch.randint(0, V, (w.N + 1,), generator=gen, device="cuda")
    ids, targets = ids[:-1].int(), ids[1:].int()
    targets[::16] = -1                                        # positions without a target
    live = (targets >= 0).float()
    g_logp = -live / live.sum()                               # the mean negative log probability
    losses = []
    for step in range(steps):
        logp, _ = lm.forward_train(ids, targets)
        losses.append(float(-(logp * live).sum() / live.sum()))
        dtable, _ = lm.backward(g_logp, weights=False)
        lm.table.add_(dtable.to(torch.bfloat16), alpha=-lr / w.N)
        if step % 5 == 0 or step == steps - 1:
            print(f"step {step:3d}  loss {losses[-1]:.4f}")
    assert lm.device_status() == M.MOE_OK
    logp, entropy, top_idx, top_logp = lm.score(ids, targets, n_top=3)
    print(f"token 0 -> {int(targets[1])}: log p {float(logp[1]):.3f}, entropy {float(entropy[1]):.3f}, "
          f"top {[(int(i), round(float(p), 3)) for i, p in zip(top_idx[1], top_logp[1])]}")
    return losses


if __name__ == "__main__":
    main()
