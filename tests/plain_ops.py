"""Plain 64-bit forms of the operators around the layer (token embedding, token log
probabilities, dropout and their gradients), written from the formulas in include/moe.h.
Test infrastructure only."""
import numpy as np


def embedding(ids, table, scale):
    out = np.zeros((len(ids), table.shape[1]))
    for n, v in enumerate(ids):
        if 0 <= v < table.shape[0]:
            out[n] = scale * table[v]
    return out


def embedding_grad(ids, dout, V, scale):
    """(gradient, sum of the absolute terms, tokens per id)."""
    g, a, cnt = np.zeros((V, dout.shape[1])), np.zeros((V, dout.shape[1])), np.zeros(V, dtype=np.int64)
    for n, v in enumerate(ids):
        if 0 <= v < V:
            g[v] += scale * dout[n]
            a[v] += abs(scale) * np.abs(dout[n])
            cnt[v] += 1
    return g, a, cnt


def logp_rows(x, scale):
    """[T][V] log probabilities; -inf where masked."""
    with np.errstate(all="ignore"):
        m = x.max(1, keepdims=True)
        z = np.where(np.isneginf(x), -np.inf, (x - m) * scale)
        lp = z - np.log(np.exp(z).sum(1, keepdims=True))
    lp[np.isneginf(m[:, 0])] = -np.inf
    return lp


def entropy_rows(lp):
    p = np.exp(lp)
    return -np.where(p > 0, p * np.where(np.isneginf(lp), 0.0, lp), 0.0).sum(1)


def token_logprobs(x, targets, scale):
    """(logp of the targets, entropy, all log probabilities)."""
    lp = logp_rows(x, scale)
    logp = np.array([lp[r, t] if 0 <= t < x.shape[1] else 0.0 for r, t in enumerate(targets)])
    return logp, entropy_rows(lp), lp


def top_rows(x, n):
    """Indices of the n largest logits, descending, ties to the lower index (-0 equals +0)."""
    return np.argsort(-(x + 0.0), axis=1, kind="stable")[:, :n].astype(np.int32)


def token_logprobs_grad(x, targets, scale, g_logp, g_entropy):
    T, V = x.shape
    lp = logp_rows(x, scale)
    h = entropy_rows(lp)
    p = np.exp(lp)
    d = -g_entropy[:, None] * p * (np.where(p > 0, lp, 0.0) + h[:, None])
    for r, t in enumerate(targets):
        if 0 <= t < V:
            d[r] -= g_logp[r] * p[r]
            d[r, t] += g_logp[r]
    d *= scale
    d[np.isneginf(x)] = 0.0
    return d


def philox(ctr, key):
    """Philox4x32-10 of one counter (four words) under a key (two words)."""
    m = 0xFFFFFFFF
    x, k = list(ctr), list(key)
    for _ in range(10):
        a, b = x[0] * 0xD2511F53, x[2] * 0xCD9E8D57
        x = [(b >> 32) ^ x[1] ^ k[0], b & m, (a >> 32) ^ x[3] ^ k[1], a & m]
        k = [(k[0] + 0x9E3779B9) & m, (k[1] + 0xBB67AE85) & m]
    return x


def dropout_bits(rows, cols, seed, offset):
    """[rows][cols] of the 16 bits that decide each element."""
    B, m = (cols + 7) // 8, 0xFFFFFFFF
    bits = np.empty((rows * B, 8), dtype=np.int64)
    for b in range(rows * B):
        w = philox([b & m, b >> 32, offset & m, offset >> 32], [seed & m, seed >> 32])
        for i in range(8):
            bits[b, i] = w[i // 2] >> (16 * (i % 2)) & 0xFFFF
    return bits.reshape(rows, B * 8)[:, :cols]


def dropout(x, p, seed, offset, residual=None):
    thr = round(p * 65536)
    keep = dropout_bits(*x.shape, seed, offset) >= thr
    y = np.where(keep, x * (65536.0 / (65536 - thr) if thr < 65536 else 0.0), 0.0)
    return y if residual is None else y + residual
