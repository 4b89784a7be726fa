"""Float64 restatement of the operators on the paged cache in the context's
type: norms with rotation, append and edits, the attention weight that entries
gather, and eviction by it.  Plain loops over requests, heads and blocks."""
from __future__ import annotations

import numpy as np

from . import verifier as V

BLOCK = 16


def norm(x, weight, eps):
    """x [T, heads, d] / sqrt(mean x^2 + eps) * weight [d] (None: x itself)."""
    x = np.asarray(x, dtype=np.float64)
    if weight is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)


class Cache:
    """Entries [blocks, n_kv, 16, d], a table of blocks, lengths."""

    def __init__(self, num_blocks, n_kv, d, table):
        self.pools = [np.zeros((num_blocks, n_kv, BLOCK, d)) for _ in range(2)]
        self.weights = np.zeros((num_blocks, n_kv, BLOCK))
        self.table = np.array(table)
        self.seq_len = np.zeros(len(self.table), np.int64)
        self.pending = np.zeros(len(self.table), np.int64)

    def length(self, b):
        return int(self.seq_len[b] + self.pending[b])

    def append(self, b, k, v):
        for i in range(len(k)):
            slot = self.length(b)
            blk = self.table[b, slot // BLOCK]
            self.pools[0][blk, :, slot % BLOCK] = k[i]
            self.pools[1][blk, :, slot % BLOCK] = v[i]
            self.pending[b] += 1

    def _of(self, array, b, lo, hi):
        rows = [array[self.table[b, s // BLOCK], :, s % BLOCK] for s in range(lo, hi)]
        return np.stack(rows) if rows else np.zeros((0,) + array.shape[1:2] + array.shape[3:])

    def values(self, b, lo=0, hi=None):
        """(K, V) of slots lo .. hi - 1: [n, n_kv, d]."""
        hi = self.length(b) if hi is None else hi
        return [self._of(p, b, lo, hi) for p in self.pools]

    def weight(self, b, hi=None):
        """[n, n_kv]"""
        return self._of(self.weights, b, 0, self.length(b) if hi is None else hi)

    def commit(self, b, n_keep):
        L, P = int(self.seq_len[b]), int(self.pending[b])
        for s in range(L + n_keep, L + P):
            for p in self.pools:
                p[self.table[b, s // BLOCK], :, s % BLOCK] = 0
        self.seq_len[b], self.pending[b] = L + n_keep, 0


def seen_of(n, L, mask=None):
    """Which of L slots each of the last n rows sees."""
    return V.causal(n, L) if mask is None else V.unpack_mask(mask, n, L)


def gathered(q, k, lse, seen, scale):
    """Weights [L, n_kv] that rows q [n, n_q, d] give the entries k [L, n_kv,
    d], and a bound on the sum of |scale q k| weighted by them."""
    n_kv, G = k.shape[1], q.shape[1] // k.shape[1]
    out, size = np.zeros(k.shape[:2]), np.zeros(k.shape[:2])
    for g in range(n_kv):
        for h in range(g * G, (g + 1) * G):
            z = scale * (q[:, h] @ k[:, g].T)
            at = np.isfinite(lse[:, h])
            with np.errstate(invalid="ignore"):
                p = np.where(seen[at], np.exp(z[at] - lse[at, h][:, None]), 0.0)
            out[:, g] += p.sum(0)
            size[:, g] += (p * scale * (np.abs(q[at, h]) @ np.abs(k[:, g]).T)).sum(0)
    return out, size


def kept(weight, budget, sink, recent):
    """The slots of one head that stay, ascending: weight [L]."""
    L = len(weight)
    if L <= budget:
        return np.arange(L)
    always = [t for t in range(L) if t < sink or t >= L - recent]
    order = sorted((t for t in range(sink, L - recent)),
                   key=lambda t: (-(weight[t] if weight[t] == weight[t] else -np.inf), weight[t] != weight[t], t))
    return np.array(sorted(always + order[:budget - len(always)]), dtype=np.int64)
