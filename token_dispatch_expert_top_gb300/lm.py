"""A small language model around one MoE layer, from token ids to log probabilities and back:

    x0 = scale * table[ids]                    moe_embedding
    y  = layer(x0)                             moe_forward_train / moe_forward
    h  = x0 + dropout(y)                       moe_dropout, the residual stream
    logits = h . table^T                       a plain matrix product (tied head)
    logp, entropy, alternatives                moe_token_logprobs

and the gradients in the other direction: moe_token_logprobs_backward over the logits' own
buffer, the two products of the head, moe_dropout again with the same counters,
moe_backward, and moe_embedding_backward accumulated onto the head's part of the table's
gradient.  With `norm_eps`, the layer and the head read normalised rows, as transformer
blocks have them:

    y  = layer(norm(x0) * w_in)                moe_rms_norm, moe_rms_norm_backward
    logits = (norm(x0 + dropout(y)) * w_out) . table^T

and LmOptimizer turns the gradients into new weights: moe_grad_norm over all of them, then one
moe_adamw.  PyTorch allocates memory and multiplies the head's matrices; everything else runs in
libmoe's kernels.

    python -m token_dispatch_expert_top_gb300.lm            # a few steps on synthetic tokens
    python -m token_dispatch_expert_top_gb300.lm --adamw    # the same with norms, clipping and AdamW
"""
from __future__ import annotations

import torch

from . import moe as M
from .layer import MoeLayer


class MoeLM:
    """Token embedding, a MoeLayer with residual dropout, and a tied head.

    table: [V][H] BF16, the embedding and the head; layer: a BF16 or MXFP8 MoeLayer (made
    with train=True for `forward_train`) whose N is the number of tokens of a call.
    norm_eps: root-mean-square norms, each with FP32 weights, in front of the layer and of the
    head (None: none)."""

    def __init__(self, layer: MoeLayer, table: torch.Tensor, embed_scale: float = 1.0, dropout: float = 0.1,
                 seed: int = 0, norm_eps: float | None = None):
        self.layer, self.table, self.norm_eps = layer, table.contiguous(), norm_eps
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
        if norm_eps is not None:
            self.w_in, self.w_out = torch.ones(H, **f32), torch.ones(H, **f32)
            self.n_in, self.n_out = torch.empty_like(self.x0), torch.empty_like(self.x0)
            self.r_in, self.r_out = torch.empty(N, **f32), torch.empty(N, **f32)
            if layer.train:
                self.dw_in, self.dw_out = torch.empty(H, **f32), torch.empty(H, **f32)
                self.norm_ws = torch.empty(M.moe_rms_norm_workspace_bytes(N, H), dtype=torch.uint8, device=dev)
                M.moe_workspace_init(self.norm_ws)

    def _read(self, x: torch.Tensor, which: str) -> torch.Tensor:
        """What the layer ("in") or the head ("out") reads of rows x: their norm, or x itself."""
        if self.norm_eps is None:
            return x
        w, n, r = (getattr(self, f"{k}_{which}") for k in ("w", "n", "r"))
        M.moe_rms_norm(x, w, n, self.norm_eps, rstd=r)
        return n

    def _read_backward(self, dn: torch.Tensor, x: torch.Tensor, which: str, dx: torch.Tensor,
                       dsum: torch.Tensor | None = None) -> torch.Tensor:
        """The gradient of x for that of _read's result, and dsum where rows pass it, too."""
        w, r, dw = (getattr(self, f"{k}_{which}") for k in ("w", "r", "dw"))
        M.moe_rms_norm_backward(dn, x, w, r, dx, dw, dsum=dsum, ws=self.norm_ws)
        return dx

    def score(self, ids: torch.Tensor, targets: torch.Tensor, n_top: int = 0, temperature: float = 1.0):
        """(logp, entropy, top_idx, top_logp) of the targets' and the n_top likeliest tokens,
        without dropout; every tensor is the model's own and is overwritten by the next call
        (the top lists are new).  What an earlier forward_train kept for `backward` is lost."""
        self.kept = False
        M.moe_embedding(ids, self.table, self.x0, self.embed_scale, self.ws)
        y = self.layer.forward(self._read(self.x0, "in"))
        M.moe_dropout(y, self.h, 0.0, self.seed, 0, residual=self.x0)
        torch.mm(self._read(self.h, "out"), self.table.t(), out=self.logits)
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
        y = self.layer.forward_train(self._read(self.x0, "in"))
        M.moe_dropout(y, self.h, self.dropout, self.seed, self.step, residual=self.x0)
        torch.mm(self._read(self.h, "out"), self.table.t(), out=self.logits)
        M.moe_token_logprobs(self.logits, targets, self.logp, self.entropy, self.stats, scale=1.0, ws=self.ws)
        self.kept = True
        return self.logp, self.entropy

    def backward(self, g_logp: torch.Tensor, g_entropy: torch.Tensor | None = None, weights: bool = True):
        """Gradients of the last forward_train for the gradients of its two results:
        (dtable, the layer's (dW_router, dbias, dW_gate_up, dW_down)); the norms' are dw_in and
        dw_out.  Overwrites the logits: once per forward_train, and before any `score`."""
        if not self.kept:
            raise RuntimeError("backward: no forward_train's tensors are kept (one backward each, no score between)")
        self.kept = False
        M.moe_token_logprobs_backward(self.logits, self.targets, self.stats,
                                      None if g_entropy is None else self.entropy, g_logp, g_entropy, self.logits,
                                      1.0, self.ws)
        dlogits, norms = self.logits, self.norm_eps is not None
        torch.mm(dlogits, self.table, out=self.dh)
        torch.mm(dlogits.t(), self.n_out if norms else self.h, out_dtype=torch.float32,
                 out=self.dtable)                             # not rounded to BF16 on the way
        if norms:
            self._read_backward(self.dh, self.h, "out", self.dh)
        M.moe_dropout(self.dh, self.dy, self.dropout, self.seed, self.step)
        dx, *rest = self.layer.backward(self.dy, self.n_in if norms else self.x0, weights=weights)
        if norms:                                             # through the layer and past it
            self._read_backward(dx, self.x0, "in", self.dx0, dsum=self.dh)
        else:
            torch.add(dx, self.dh, out=self.dx0)
        M.moe_embedding_backward(self.ids, self.dx0, self.dtable, self.embed_scale, True, self.ws)
        return self.dtable, rest

    def device_status(self) -> int:
        """The first device error of the model's own calls or of its layer's, then reset."""
        s = M.moe_last_device_status(self.ws)
        s = s or self.layer.device_status()
        return s or (self.layer.backward_status() if self.layer.train else 0)


class LmOptimizer:
    """AdamW over a MoeLM's table, norm weights and router, with the gradients' global norm clipped.

    The table and the router have FP32 master weights, whose BF16 copies are the model's (a step below half a
    last place of BF16 would be lost otherwise).  They are taken from the model when this is made: weights loaded
    into it later want a new optimiser.  The norms' weights are stepped in place.  (The layer holds its expert
    weights packed for its GEMMs; their gradients are the caller's.)  eight_bits: moments of the matrices in MXFP8
    codes, a quarter of their memory; seed: of their rounding, whose bits are others than those of a dropout of the
    same seed.  The step number is on the device, so that a step can be captured."""

    DOMAIN = int.from_bytes(b"moe_adam", "big")               # both draw from the same counters: another key

    def __init__(self, lm: MoeLM, lr: float = 1e-3, betas=(0.9, 0.95), eps: float = 1e-8, weight_decay: float = 0.1,
                 max_norm: float = 1.0, eight_bits: bool = False, seed: int = 0):
        self.lm, self.betas, self.eps, self.max_norm, self.seed = lm, betas, eps, max_norm, seed ^ self.DOMAIN
        dev = lm.table.device
        self.master, self.router_master = lm.table.float(), lm.layer.w_router.float()
        params, copies = [self.master, self.router_master], [lm.table, lm.layer.w_router]
        grads, decay = [lm.dtable, lm.layer.dw_router], [weight_decay, 0.0]
        if lm.norm_eps is not None:
            params += [lm.w_in, lm.w_out]
            grads += [lm.dw_in, lm.dw_out]
            copies, decay = copies + [None, None], decay + [0.0, 0.0]
        m, v, ms, vs = [], [], [], []
        for p in params:
            eight = eight_bits and p.dim() == 2
            m.append(torch.zeros(p.shape, dtype=torch.uint8 if eight else torch.float32, device=dev))
            v.append(torch.zeros_like(m[-1]))
            blocks = (p.numel() + 31) // 32
            ms.append(torch.zeros(blocks, dtype=torch.uint8, device=dev) if eight else None)
            vs.append(torch.zeros(blocks, dtype=torch.uint8, device=dev) if eight else None)
        self.tensors = M.AdamWTensors(params, grads, m, v, copies=copies, m_scales=ms, v_scales=vs, weight_decay=decay)
        self.lr = torch.full((1,), lr, dtype=torch.float32, device=dev)
        self.number = torch.zeros(1, dtype=torch.int64, device=dev)
        self.norm, self.factor = torch.empty(1, device=dev), torch.empty(1, device=dev)
        self.ws = torch.empty(M.moe_grad_norm_workspace_bytes(), dtype=torch.uint8, device=dev)
        M.moe_workspace_init(self.ws)

    def step(self) -> torch.Tensor:
        """One update from the gradients of the last MoeLM.backward; returns their norm (on the
        device).  If it is not finite the weights stay as they are, and the step does not count."""
        M.moe_grad_norm(self.tensors, self.norm, self.factor, self.max_norm, self.ws)
        self.number.add_(self.norm.isfinite())
        M.moe_adamw(self.tensors, self.lr, self.number, *self.betas, self.eps, grad_scale=self.factor, seed=self.seed)
        return self.norm


def main(steps: int = 20, V: int = 1000, lr: float = 300.0, adamw: bool = False) -> list[float]:
    """Fits the table to one batch of synthetic tokens; returns the mean losses.  adamw: a model with
    norms, stepped by LmOptimizer (lr is its own then)."""
    from . import synth
    w = synth.Workload("lm_small", N=256, H=512, I=256, E=16, k=4, S=4, dtype="bf16")
    layer = MoeLayer(w, synth.make_inputs(w), train=True)
    gen = torch.Generator(device="cuda").manual_seed(1)
    table = (torch.randn((V, w.H), generator=gen, device="cuda") / w.H ** 0.5).to(torch.bfloat16)
    lm = MoeLM(layer, table, embed_scale=w.H ** 0.5, norm_eps=1e-6 if adamw else None)
    optimizer = LmOptimizer(lm, lr=3e-3, eight_bits=True) if adamw else None
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
        if adamw:
            optimizer.step()
        else:
            lm.table.add_(dtable.to(torch.bfloat16), alpha=-lr / w.N)
        if step % 5 == 0 or step == steps - 1:
            print(f"step {step:3d}  loss {losses[-1]:.4f}")
    assert lm.device_status() == M.MOE_OK
    logp, entropy, top_idx, top_logp = lm.score(ids, targets, n_top=3)
    print(f"token 0 -> {int(targets[1])}: log p {float(logp[1]):.3f}, entropy {float(entropy[1]):.3f}, "
          f"top {[(int(i), round(float(p), 3)) for i, p in zip(top_idx[1], top_logp[1])]}")
    return losses


if __name__ == "__main__":
    import sys
    main(adamw="--adamw" in sys.argv[1:])
