"""The operators around the MoE layer, as they are measured: token embedding and its
gradient, log probabilities of given tokens with entropy and top alternatives and their
gradient, and dropout from a counter-based generator with the residual add.

``run`` takes one pass through one of them: through the framework's entry points where
``own`` is true, otherwise in elementary torch operations in 32 bits, rounded once."""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one sequence's next token on its way into the model
        dict(name="embed_token", op="embed", N=1, V=32000, H=2048, dtype="bf16", scale=1.0, neg=0.0),
        # the 8192-token batch of the DeepSeek-V3-shaped layer, left padding among it
        dict(name="embed_batch", op="embed", N=8192, V=128000, H=7168, dtype="bf16", scale=1.0, neg=0.02),
        # a short ragged fine-tuning batch with FP32 gradients and an odd row length
        dict(name="embed_grad_ragged", op="embed_grad", N=777, V=5003, H=1409, dtype="f32", grad="f32",
             scale=37.5, neg=0.05),
        # the 16384-token training step's table gradient, kept in FP32; Zipf-like tokens
        dict(name="embed_grad_batch", op="embed_grad", N=16384, V=128000, H=7168, dtype="bf16", grad="f32",
             scale=1.0, neg=0.0),
        # one decoded token: its log probability and 20 alternatives, at a temperature
        dict(name="logp_token", op="logp", T=1, V=128000, pad=0, dtype="f32", scale=1.25, mask=0.0, top=20),
        # a decode batch over an odd vocabulary under a grammar mask
        dict(name="logp_decode", op="logp", T=64, V=50001, pad=0, dtype="bf16", scale=1.0, mask=0.3, top=5),
        # scoring the 8192 tokens of a prompt batch, logits in rows padded past the vocabulary
        dict(name="logp_prompt", op="logp", T=8192, V=127901, pad=99, dtype="bf16", scale=1.0, mask=0.0, top=8),
        # a small policy update, FP32 logits, prompt tokens without a target
        dict(name="logp_train_ragged", op="logp_train", T=333, V=5003, pad=5, dtype="f32", scale=1.0,
             mask=0.1, ignore=0.3),
        # a policy update's log probabilities, entropies and logit gradients
        dict(name="logp_train_batch", op="logp_train", T=4096, V=128000, pad=0, dtype="bf16", scale=1.0,
             mask=0.0, ignore=0.1),
        # the residual stream of a few tokens
        dict(name="dropout_small", op="dropout", R=7, C=2048, pad=0, dtype="bf16", p=0.1, residual=True),
        # the layer's output on its way into the residual stream of 16384 tokens
        dict(name="dropout_residual", op="dropout", R=16384, C=7168, pad=0, dtype="bf16", p=0.1, residual=True),
        # the gradient on its way back, FP32, odd rows inside a wider buffer
        dict(name="dropout_grad", op="dropout", R=4001, C=1409, pad=7, dtype="f32", p=0.25, residual=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _even(rng, n, unit):
    """n, or in half the draws the multiple of unit below it."""
    n = n // unit * unit if n >= unit and rng.random() < 0.5 else n
    return n + unit if n == 3072 else n


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "logp", "logp_train", "dropout"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("embed", "embed_grad"):
        c = dict(op=op, N=_log(rng, 1, 16384), V=_log(rng, 1000, 128000), H=_log(rng, 64, 7168), dtype=dtype,
                 scale=rng.choice([1.0, 1.0, 45.25]), neg=rng.choice([0.0, 0.05]))
        c["H"] = _even(rng, c["H"], 128)
        if op == "embed_grad":
            c["grad"] = rng.choice(["f32", dtype])
        return c
    if op in ("logp", "logp_train"):
        V = _log(rng, 1000, 160000)
        T = min(_log(rng, 1, 8192), 1900000000 // (V * (2 if dtype == "bf16" else 4) * (1 if op == "logp" else 2)))
        V = _even(rng, V, 40)
        c = dict(op=op, T=T, V=V, pad=rng.choice([0, 0, 1, 64]), dtype=dtype, scale=rng.choice([1.0, 1.25, 0.7]),
                 mask=rng.choice([0.0, 0.2]))
        if op == "logp":
            c["top"] = rng.choice([0, 1, 5, 20, 32])
        else:
            c["ignore"] = rng.choice([0.0, 0.3])
        return c
    C = _even(rng, _log(rng, 64, 8192), 80)
    return dict(op=op, R=_log(rng, 1, 14000), C=C, pad=rng.choice([0, 0, 3, 64]), dtype=dtype,
                p=rng.choice([0.05, 0.1, 0.3, 0.5]), residual=rng.choice([True, False]))


# ------------------------------------------------------------------ inputs
def _tokens(n, V, neg, gen):
    """Zipf-like token ids (log-uniform ranks, the ranks scattered over the vocabulary), a
    share of them -1: no token."""
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(V + 1.0)).floor().long() - 1).clamp(0, V - 1)
    ids = torch.randperm(V, generator=gen, device="cuda")[rank]
    if neg:
        drop = torch.rand(n, generator=gen, device="cuda") < neg
        ids = torch.where(drop, torch.full_like(ids, -1), ids)
    return ids.int()


def _normal(rows, cols, pad, dtype, gen, std=1.0):
    """N(0, std^2) in a [rows][cols + pad] buffer, as the [rows][cols] view of it."""
    out = torch.empty((rows, cols + pad), dtype=DT[dtype], device="cuda")
    return out.normal_(0.0, std, generator=gen)[:, :cols]


def prepare(case, seed):
    c, op = case, case["op"]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=c)
    if op == "embed":
        s["ids"] = _tokens(c["N"], c["V"], c["neg"], gen)
        s["table"] = _normal(c["V"], c["H"], 0, c["dtype"], gen, 0.02)
        s["out"] = torch.empty((c["N"], c["H"]), dtype=DT[c["dtype"]], device="cuda")
    elif op == "embed_grad":
        s["ids"] = _tokens(c["N"], c["V"], c["neg"], gen)
        s["dout"] = _normal(c["N"], c["H"], 0, c["dtype"], gen, 1e-3)
        s["dtable"] = torch.empty((c["V"], c["H"]), dtype=DT[c["grad"]], device="cuda")
    elif op in ("logp", "logp_train"):
        T, V = c["T"], c["V"]
        s["logits"] = _normal(T, V, c["pad"], c["dtype"], gen, 2.5)
        t = torch.randint(0, V, (T,), generator=gen, device="cuda")
        rows = torch.arange(T, device="cuda")
        # the token that was taken is often one of the likely ones
        s["logits"][rows, t] += (torch.rand(T, generator=gen, device="cuda") * 14).to(DT[c["dtype"]])
        if c["mask"]:
            # a band of the vocabulary is ruled out for every row, and the last row keeps
            # only its token; a mask never rules out the token that was taken
            off = torch.rand(V, generator=gen, device="cuda") < c["mask"]
            kept = s["logits"][rows, t]
            s["logits"].masked_fill_(off, float("-inf"))
            s["logits"][T - 1] = float("-inf")
            s["logits"][rows, t] = kept
        if op == "logp_train" and c["ignore"]:
            t = torch.where(torch.rand(T, generator=gen, device="cuda") < c["ignore"], torch.full_like(t, -1), t)
        s["targets"] = t.int()
        f32 = dict(dtype=torch.float32, device="cuda")
        s["logp"], s["entropy"], s["stats"] = (torch.empty(T, **f32), torch.empty(T, **f32),
                                               torch.empty((T, 2), **f32))
        if op == "logp":
            s["top_idx"] = torch.empty((T, c["top"]), dtype=torch.int32, device="cuda")
            s["top_logp"] = torch.empty((T, c["top"]), **f32)
        else:
            # advantages and an entropy bonus, as means over the tokens
            s["g_logp"] = -torch.randn(T, generator=gen, **f32) / T
            s["g_entropy"] = torch.full((T,), -0.01 / T, **f32)
            s["dlogits"] = torch.empty((T, V), dtype=DT[c["dtype"]], device="cuda")
    else:
        s["x"] = _normal(c["R"], c["C"], c["pad"], c["dtype"], gen)
        s["residual"] = _normal(c["R"], c["C"], c["pad"], c["dtype"], gen) if c["residual"] else None
        s["out"] = torch.empty((c["R"], c["C"]), dtype=DT[c["dtype"]], device="cuda")
        s["seed"], s["offset"] = 0x9E3779B97F4A7C15 ^ (seed * 2654435761), 3 * seed + 1
        s["seed"] &= (1 << 64) - 1
    if own:
        from token_dispatch_expert_top_gb300 import moe as M
        s["M"] = M
        # the workspace that a program keeps beside its tensors
        n = M.moe_embedding_workspace_bytes(c["N"], c["V"], c["H"]) if op == "embed_grad" else 256
        s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        M.moe_workspace_init(s["ws"])
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    c, M, op = s["case"], s["M"], s["case"]["op"]
    if op == "embed":
        M.moe_embedding(s["ids"], s["table"], s["out"], c["scale"], s["ws"])
        return s["out"]
    if op == "embed_grad":
        M.moe_embedding_backward(s["ids"], s["dout"], s["dtable"], c["scale"], False, s["ws"])
        return s["dtable"]
    if op == "logp":
        M.moe_token_logprobs(s["logits"], s["targets"], s["logp"], s["entropy"], None, s["top_idx"],
                             s["top_logp"], c["scale"], s["ws"])
        return dict(logp=s["logp"], entropy=s["entropy"], top_idx=s["top_idx"], top_logp=s["top_logp"])
    if op == "logp_train":
        M.moe_token_logprobs(s["logits"], s["targets"], s["logp"], s["entropy"], s["stats"], None, None,
                             c["scale"], s["ws"])
        M.moe_token_logprobs_backward(s["logits"], s["targets"], s["stats"], s["entropy"], s["g_logp"],
                                      s["g_entropy"], s["dlogits"], c["scale"], s["ws"])
        return dict(logp=s["logp"], entropy=s["entropy"], dlogits=s["dlogits"])
    M.moe_dropout(s["x"], s["out"], c["p"], s["seed"], s["offset"], s["residual"])
    return s["out"]


def _run_plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "embed":
        ids = s["ids"].long()
        rows = s["table"][ids.clamp(min=0)].float() * c["scale"]
        return (rows * (ids >= 0).unsqueeze(1)).to(DT[c["dtype"]])
    if op == "embed_grad":
        ids = s["ids"].long()
        grad = torch.zeros((c["V"], c["H"]), dtype=torch.float32, device="cuda")
        grad.index_add_(0, ids.clamp(min=0), s["dout"].float() * (ids >= 0).unsqueeze(1))
        return grad.mul_(c["scale"]).to(DT[c["grad"]])
    if op == "dropout":
        kept, keep_scale = _keep_plain(c["R"], c["C"], c["p"], s["seed"], s["offset"])
        y = s["x"].float() * kept * keep_scale
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(DT[c["dtype"]])
    t = s["targets"].long()
    x = s["logits"].float()
    z = (x - x.amax(1, keepdim=True)) * c["scale"]
    e = torch.exp(z)
    total = e.sum(1, keepdim=True)
    z = z - torch.log(total)                                # log p; -inf where masked
    p = e.div_(total)
    entropy = -(p * z.clamp(min=-1e4)).sum(1)
    logp = torch.where(t >= 0, z.gather(1, t.clamp(min=0).unsqueeze(1)).squeeze(1), 0.0)
    if op == "logp":
        # an order without ties: the logit's bits as an integer, then the lower index
        b = (x + 0.0).view(torch.int32).long()
        key = torch.where(b < 0, -1 - (b & 0x7FFFFFFF), b) * (1 << 32) + (c["V"] - 1 - torch.arange(c["V"], device="cuda"))
        idx = torch.topk(key, c["top"], dim=1, sorted=True).indices
        return dict(logp=logp, entropy=entropy, top_idx=idx.int(), top_logp=z.gather(1, idx))
    g = torch.where(t >= 0, s["g_logp"], 0.0)
    dx = -p * (g.unsqueeze(1) + s["g_entropy"].unsqueeze(1) * (z.clamp(min=-1e4) + entropy.unsqueeze(1)))
    dx.scatter_add_(1, t.clamp(min=0).unsqueeze(1), g.unsqueeze(1))
    return dict(logp=logp, entropy=entropy, dlogits=(dx * c["scale"]).to(DT[c["dtype"]]))


def _keep_plain(R, C, p, seed, offset):
    """The kept elements of an [R][C] matrix (Philox4x32-10, eight elements a counter, 16
    bits each) and the factor that keeps the mean."""
    low = 0xFFFFFFFF
    blocks = -(-C // 8)
    i = torch.arange(R * blocks, device="cuda")
    x0, x1 = i & low, i >> 32
    x2, x3 = torch.full_like(i, offset & low), torch.full_like(i, offset >> 32 & low)
    k0, k1 = seed & low, seed >> 32 & low
    for _ in range(10):                                     # the generator's rounds
        a, b = x0 * 0xD2511F53, x2 * 0xCD9E8D57             # only their low 64 bits are used
        x0, x1, x2, x3 = (b >> 32 & low) ^ x1 ^ k0, b & low, (a >> 32 & low) ^ x3 ^ k1, a & low
        k0, k1 = k0 + 0x9E3779B9 & low, k1 + 0xBB67AE85 & low
    w = torch.stack((x0, x1, x2, x3), 1)
    bits = torch.stack((w & 0xFFFF, w >> 16), 2).view(R, blocks * 8)[:, :C]
    thr = round(p * 65536)
    return bits >= thr, 65536.0 / (65536 - thr)


# ------------------------------------------------------------------ the least a pass can move and compute
def work(case):
    c, op = case, case["op"]
    size = {"bf16": 2, "f32": 4}
    e = size[c["dtype"]]
    if op in ("embed", "embed_grad"):
        live = c["N"] * (1 - c["neg"])
        if op == "embed":
            return dict(bytes=c["N"] * (4 + c["H"] * e) + live * c["H"] * e, flops=c["N"] * c["H"])
        return dict(bytes=c["N"] * 4 + live * c["H"] * e + c["V"] * c["H"] * size[c["grad"]],
                    flops=live * c["H"])
    if op == "dropout":
        n = c["R"] * c["C"]
        return dict(bytes=n * e * (3 if c["residual"] else 2), flops=3 * n)
    n = c["T"] * c["V"]
    if op == "logp":
        return dict(bytes=n * e + c["T"] * (12 + 8 * c["top"]), flops=6 * n)
    # without both passes' results in hand the gradient cannot begin, so the logits that
    # do not stay on the chip are read again; one read is the least
    return dict(bytes=2 * n * e + c["T"] * 20, flops=12 * n)


# ------------------------------------------------------------------ the same in 64 bits
def exact(case, seed):
    c, op = case, case["op"]
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if op == "embed":
        out = torch.zeros((c["N"], c["H"]), dtype=torch.float64, device="cuda")
        live = torch.nonzero(s["ids"] >= 0).squeeze(1)
        out[live] = s["table"].index_select(0, s["ids"][live]).double() * c["scale"]
        return out
    if op == "embed_grad":
        # each live token's row, in the order of the ids; every id's run of rows is summed
        live = torch.nonzero(s["ids"] >= 0).squeeze(1)
        ids, order = torch.sort(s["ids"][live].long(), stable=True)
        rows = s["dout"][live[order]].double()
        out = torch.zeros((c["V"], c["H"]), dtype=torch.float64, device="cuda")
        v, n = torch.unique_consecutive(ids, return_counts=True)
        if len(v):
            out[v] = torch.segment_reduce(rows, "sum", lengths=n, axis=0)
        return out * c["scale"]
    if op == "dropout":
        import numpy as np
        R, C, mask = c["R"], c["C"], (1 << 32) - 1
        B = (C + 7) // 8
        half = np.empty((R * B, 8), dtype=np.uint16)
        m32, sh, off = np.uint64(mask), np.uint64(32), s["offset"]
        for at in range(0, R * B, 1 << 16):                 # pieces that stay in the cache
            n = np.arange(at, min(R * B, at + (1 << 16)), dtype=np.uint64)
            ctr = [n & m32, n >> sh, np.full_like(n, off & mask), np.full_like(n, (off >> 32) & mask)]
            key = [s["seed"] & mask, s["seed"] >> 32]
            for _ in range(10):
                a, b = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
                ctr = [(b >> sh) ^ ctr[1] ^ np.uint64(key[0]), b & m32, (a >> sh) ^ ctr[3] ^ np.uint64(key[1]), a & m32]
                key = [(key[0] + 0x9E3779B9) & mask, (key[1] + 0xBB67AE85) & mask]
            for i, w in enumerate(ctr):
                half[at:at + len(n), 2 * i] = w & np.uint64(0xFFFF)
                half[at:at + len(n), 2 * i + 1] = w >> np.uint64(16)
        thr = round(c["p"] * 65536)
        keep = torch.from_numpy(half.reshape(R, B * 8)[:, :C].astype(np.int32) >= thr).cuda()
        y = torch.where(keep, s["x"].double() * (65536.0 / (65536 - thr)), 0.0)
        return y if s["residual"] is None else y + s["residual"].double()
    T, V, top = c["T"], c["V"], c.get("top", 0)
    logp, entropy = (torch.zeros(T, dtype=torch.float64, device="cuda") for _ in range(2))
    top_logp = torch.empty((T, top), dtype=torch.float64, device="cuda")
    dlogits = torch.empty((T, V), dtype=torch.float64, device="cuda") if op == "logp_train" else None
    step = max(1, (1 << 27) // V)
    for r in range(0, T, step):
        x = s["logits"][r:r + step].double() * c["scale"]
        t = s["targets"][r:r + step].long()
        lp = x - torch.logsumexp(x, 1, keepdim=True)
        p = torch.exp(lp)
        plp = torch.where(p > 0, p * lp, 0.0)
        h = -plp.sum(1)
        entropy[r:r + step] = h
        has = torch.nonzero(t >= 0).squeeze(1)
        logp[r:r + step][has] = lp[has, t[has]]
        if op == "logp":
            top_logp[r:r + step] = torch.topk(lp, top, dim=1).values
        else:
            gl, gh = s["g_logp"][r:r + step].double(), s["g_entropy"][r:r + step].double()
            d = -gh[:, None] * (plp + p * h[:, None])
            d[has] -= gl[has, None] * p[has]
            d[has, t[has]] += gl[has]
            dlogits[r:r + step] = d * c["scale"]
    if op == "logp":
        return dict(logp=logp, entropy=entropy, top_idx=None, top_logp=top_logp)
    return dict(logp=logp, entropy=entropy, dlogits=dlogits)
