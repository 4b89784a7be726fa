"""Float64 restatement of the verifier's side of a draft-and-verify step:
rotary positions, the 8-bit paged cache, attention over it, and penalties,
biases and masks on logits.  Plain loops over requests and blocks; codes of the
8-bit format are enumerated, not computed with casts."""
from __future__ import annotations

import numpy as np

BLOCK = 16
NAN_CODE = 0x7F


def e4m3_table() -> np.ndarray:
    """Values of the 256 codes: 1 sign, 4 exponent (bias 7), 3 mantissa bits;
    0x7f and 0xff are NaN, there are no infinities."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = np.nan if (c & 0x7F) == NAN_CODE else (-v if c & 0x80 else v)
    return out


VALUES = e4m3_table()
_POS = VALUES[:NAN_CODE]        # 0 .. 448, ascending


def e4m3_encode(x) -> np.ndarray:
    """Nearest code (ties to the even mantissa), clamped to +-448; NaN for
    what is not finite."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.nan_to_num(np.abs(x), nan=0.0, posinf=0.0), 448.0)
    hi = np.clip(np.searchsorted(_POS, a), 0, len(_POS) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(_POS[hi] == a, hi, code)
    code = code | np.where(np.signbit(x), 0x80, 0)
    return np.where(np.isfinite(x), code, NAN_CODE).astype(np.uint8)


def block_scale(x) -> float:
    """Smallest power of two (at least 2^-126) with max|x| <= 448 s over the
    finite values; 0 if they are all zero or there are none."""
    a = np.abs(np.asarray(x, dtype=np.float64))
    a = a[np.isfinite(a)]
    top = float(a.max()) if a.size else 0.0
    if top == 0.0:
        return 0.0
    s = 2.0 ** -126
    while top > 448.0 * s:
        s *= 2.0
    return s


def rope_frequencies(rotary_dim, theta=1e6, scaling="none", factor=1.0, original_max_pos=0, low_freq_factor=1.0,
                     high_freq_factor=4.0, beta_fast=32.0, beta_slow=1.0, magnitude=0.0):
    """(angle per position of each pair, factor on the rotated elements)."""
    f = np.array([theta ** (-2.0 * i / rotary_dim) for i in range(rotary_dim // 2)])
    mag = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        r = original_max_pos * f / (2 * np.pi)
        w = np.clip((r - low_freq_factor) / (high_freq_factor - low_freq_factor), 0, 1)
        f = w * f + (1 - w) * f / factor
    elif scaling == "yarn":
        c = [rotary_dim * np.log(original_max_pos / (2 * np.pi * b)) / (2 * np.log(theta))
             for b in (beta_fast, beta_slow)]
        lo, hi = max(np.floor(c[0]), 0), min(np.ceil(c[1]), rotary_dim - 1)
        w = np.clip((np.arange(rotary_dim // 2) - lo) / max(hi - lo, 0.001), 0, 1)
        f = (1 - w) * f + w * f / factor
        mag = 0.1 * np.log(factor) + 1.0 if factor > 1 else 1.0
    return f, (magnitude or mag)


def rope(x, positions, layout="half", rotary_dim=None, **kw):
    """x [T, heads, d] rotated to positions [T]."""
    x = np.array(x, dtype=np.float64)
    rd = x.shape[-1] if rotary_dim is None else rotary_dim
    f, mag = rope_frequencies(rd, **kw)
    ang = np.asarray(positions, dtype=np.float64)[:, None] * f[None]
    c, s = np.cos(ang)[:, None] * mag, np.sin(ang)[:, None] * mag
    ia = np.arange(rd // 2) if layout == "half" else 2 * np.arange(rd // 2)
    ib = ia + (rd // 2 if layout == "half" else 1)
    a, b = x[..., ia].copy(), x[..., ib].copy()
    x[..., ia], x[..., ib] = a * c - b * s, b * c + a * s
    return x


class Cache8:
    """Codes [blocks, n_kv, 16, d], scales [blocks, n_kv], table, lengths."""

    def __init__(self, num_blocks, n_kv, d, table):
        self.codes = [np.zeros((num_blocks, n_kv, BLOCK, d), np.uint8) for _ in range(2)]
        self.scale = [np.zeros((num_blocks, n_kv)) for _ in range(2)]
        self.table = np.array(table)
        self.seq_len = np.zeros(len(self.table), np.int64)
        self.pending = np.zeros(len(self.table), np.int64)

    def _put(self, w, b, slot, rows):
        """Store rows [n, n_kv, d] from `slot` on; slots below hold entries
        within the first block."""
        i = 0
        while i < len(rows):
            blk, s0 = self.table[b, slot // BLOCK], slot % BLOCK
            n = min(BLOCK - s0, len(rows) - i)
            for g in range(rows.shape[1]):
                x = rows[i:i + n, g]
                was = self.scale[w][blk, g] if s0 else 0.0
                now = max(was, block_scale(x))
                tile = self.codes[w][blk, g]
                if was > 0 and now > was:
                    tile[:s0] = e4m3_encode(VALUES[tile[:s0]] * (was / now))
                tile[s0:s0 + n] = e4m3_encode(x / now) if now else np.where(np.isfinite(x), 0, NAN_CODE)
                if now == 0:
                    tile[s0:s0 + n] |= np.where(np.isfinite(x) & np.signbit(x), 0x80, 0).astype(np.uint8)
                self.scale[w][blk, g] = now
            i, slot = i + n, slot + n

    def append(self, b, k, v):
        start = int(self.seq_len[b] + self.pending[b])
        self._put(0, b, start, np.asarray(k, dtype=np.float64))
        self._put(1, b, start, np.asarray(v, dtype=np.float64))
        self.pending[b] += len(k)

    def values(self, b, lo, hi):
        """(K, V) of slots lo .. hi - 1: [n, n_kv, d]."""
        out = []
        for w in range(2):
            rows = [VALUES[self.codes[w][self.table[b, s // BLOCK], :, s % BLOCK]]
                    * self.scale[w][self.table[b, s // BLOCK]][:, None] for s in range(lo, hi)]
            out.append(np.stack(rows) if rows else np.zeros((0,) + self.codes[w].shape[1:2] + self.codes[w].shape[3:]))
        return out

    def _drop(self, b, lo, hi):
        for s in range(lo, hi):
            blk = self.table[b, s // BLOCK]
            for w in range(2):
                self.codes[w][blk, :, s % BLOCK] = 0
                if s % BLOCK == 0:
                    self.scale[w][blk] = 0.0

    def commit(self, b, n_keep, keep=None):
        L, P = int(self.seq_len[b]), int(self.pending[b])
        if keep is not None:
            kept = self.values(b, L, L + P)
            for w in range(2):
                self._put(w, b, L, kept[w][np.asarray(keep[:n_keep], dtype=int)])
        self._drop(b, L + n_keep, L + P)
        self.seq_len[b], self.pending[b] = L + n_keep, 0

    def truncate(self, b, new_len):
        self._drop(b, new_len, int(self.seq_len[b] + self.pending[b]))
        self.seq_len[b], self.pending[b] = new_len, 0


def attention(q, k, v, seen, scale):
    """q [n, n_q, d], k and v [L, n_kv, d], seen [n, L] truth values.
    Returns (out, lse, sum_t p_t |v_t|, largest scale * sum |q_d k_d|)."""
    n, n_q, d = q.shape
    G = n_q // k.shape[1]
    out, lse, mass = np.zeros((n, n_q, d)), np.full((n, n_q), -np.inf), np.zeros((n, n_q, d))
    size = np.zeros((n, n_q))
    for i in range(n):
        at = np.nonzero(seen[i])[0]
        if not len(at):
            continue
        for h in range(n_q):
            kk, vv = k[at, h // G], v[at, h // G]
            z = scale * (kk @ q[i, h])
            m = z.max()
            p = np.exp(z - m)
            t = p.sum()
            out[i, h], mass[i, h] = p @ vv / t, p @ np.abs(vv) / t
            lse[i, h] = m + np.log(t)
            size[i, h] = scale * (np.abs(kk) @ np.abs(q[i, h])).max()
    return out, lse, mass, size


def causal(n, L):
    return np.arange(L)[None] <= (L - n + np.arange(n))[:, None]


def unpack_mask(words, n, L):
    """seen [n, L] of the mask words [n, W]: everything before the last n
    slots, and those whose bit is set."""
    seen = np.ones((n, L), bool)
    w = np.asarray(words).astype(np.int64) & 0xFFFFFFFF
    for i in range(n):
        for j in range(n):
            seen[i, L - n + j] = bool(w[i, j // 32] >> (j % 32) & 1)
    return seen


def process_logits(z, counts, before=(), repetition=1.0, frequency=0.0, presence=0.0, bias=(), allowed=None):
    """One row z [V]; counts [V] (bit 31: in the prompt); before: the drafts
    in front of the row; bias: (token, value) pairs; allowed: truth values.
    Returns (out, bound on the size of what was added up)."""
    z = np.array(z, dtype=np.float64)
    V = len(z)
    c = (np.asarray(counts).astype(np.int64) & 0x7FFFFFFF).astype(np.float64)
    met = np.asarray(counts) < 0
    for t in before:
        if 0 <= t < V:
            c[t] += 1
    met = met | (c > 0)
    with np.errstate(invalid="ignore"):
        z1 = np.where(met, np.where(z > 0, z / repetition, z * repetition), z)
        size = np.abs(z1) + np.abs(frequency * c) + np.abs(presence) * (c > 0)
        out = z1 - frequency * c - presence * (c > 0)
        for t, x in bias:
            if 0 <= t < V:
                out[t] += x
                size[t] += abs(x)
    if allowed is not None:
        out = np.where(allowed, out, -np.inf)
    return out, size
