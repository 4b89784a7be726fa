"""Each entry's own softmax weight, read through values that are one in a column
of their own, where the running maximum moves within a step of 128 slots and
scores are large.

Scores are sums of products that float32 holds exactly, so a weight is off by its
exponential (2^-22, and 2^-24 of an exponent of at most 2^8: 2^-16), by one rounding
where it becomes an operand of the product (bf16: half a step, 2^-8), by the factors
that move earlier results (2^-22 each) and, below 2^13, by a reference that is itself
rounded when it passes a power of two (2^-12); the result by one more rounding to bf16:
relative to the weight itself  2 * 2^-8 + 2^-16 (their product) + 2^-15 + 2^-12.
float32 heads: 2^-15 and the rounding of the scaled score, 2^-24 of it, twice.
"""
import numpy as np
import pytest
import torch

from test_gpu_verifier import M_, clean, context, i32

pytestmark = pytest.mark.gpu

SPLIT = {"zero": 0, "near 2^12": 2832, "near 2^16": 45420, "near 2^20": 726800, "beyond 2^20": 1441792, "near 2^21": 1453608,
         "below -2^20": -1441792, "near -2^16": -45420}


def parts(base):
    """A whole number as two products of bf16 numbers of up to eight bits and a rest below 256."""
    s, n = (-1 if base < 0 else 1), abs(base)
    hi, lo = n // 65536, n % 65536
    assert hi < 256
    return [(256.0, s * 256.0 * hi), (256.0, float(s * (lo // 256))), (1.0, float(s * (lo % 256)))]


def make(base, dtype, L, probe, levels, rows, B, n_q, hd):
    """B requests over the same blocks; deltas from the base in half units: levels by quarter of the probed step."""
    M = M_()
    ctx = context(n_q, 1, hd, dtype, max_batch=B)
    nb = (L + 15) // 16
    delta = np.zeros(nb * 16)
    t = np.arange(128)
    delta[probe:probe + 128] = np.asarray(levels)[t // 32] + 0.5 * ((5 * t) % 9)
    k = np.zeros((nb * 16, hd))
    q = np.zeros((n_q, hd))
    for d, (a, b) in enumerate(parts(base)):
        q[:, d], k[:, d] = a, b
    q[:, 3], k[:, 3] = 1.0 + np.arange(n_q) % 4, delta
    v = np.zeros((nb * 16, hd))
    v[probe + t[:hd], t[:hd]] = 1.0
    kv = M.KVCache.empty(ctx, nb, i32(np.tile(np.arange(nb), (B, 1))))
    for pool, x in ((kv.k_pool, k), (kv.v_pool, v)):
        pool.copy_(torch.from_numpy(x.reshape(nb, 16, 1, hd).transpose(0, 2, 1, 3).copy()))
        np.testing.assert_array_equal(pool.double().cpu().numpy()[:, 0].reshape(-1, hd), x)
    kv.seq_len.fill_(L)
    qd = torch.from_numpy(q).to(ctx.dtype).cuda()[None].repeat(B * rows, 1, 1)
    z = base + q[:, 3:4] * delta[None, :L]                      # [n_q, L], exact
    return ctx, kv, qd, z


@pytest.mark.parametrize("base", list(SPLIT))
@pytest.mark.parametrize("dtype,L,probe,rows,B", [
    ("bf16", 128, 0, 1, 1), ("bf16", 127, 0, 1, 3), ("bf16", 384, 256, 1, 160), ("bf16", 900, 512, 200, 4),
    ("f32", 384, 256, 1, 3), ("f32", 300, 128, 40, 2)])
@pytest.mark.parametrize("levels", [(0, 8, 16, 10), (0, 0, 0, 12), (2, 0, 7, 20)])
def test_each_entry_has_its_weight(base, dtype, L, probe, rows, B, levels):
    M = M_()
    hd, n_q = 128, 4
    ctx, kv, q, z = make(SPLIT[base], dtype, L, probe, levels, rows, B, n_q, hd)
    out = torch.zeros_like(q)
    off = np.arange(B + 1) * rows
    M.mtp_kv_attention(ctx, kv, q, i32(off), out, M.AttentionWorkspace(ctx), rows, scale=1.0)
    clean(ctx)
    got = out.double().cpu().numpy().reshape(B, rows, n_q, hd)
    per = 2.0 ** -7 + 2.0 ** -16 + 2.0 ** -15 + 2.0 ** -12 if dtype == "bf16" else 2.0 ** -15 + 2.0 ** -22 * 1.5 * np.abs(z).max()
    worst = 0.0
    for r in range(rows):
        n = L - rows + 1 + r                                    # row r sees so many
        p = np.exp(z[:, :n] - z[:, :n].max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        want = np.zeros((n_q, hd))
        m = max(0, min(n - probe, hd))
        want[:, :m] = p[:, probe:probe + m]
        off_by = np.abs(got[:, r] - want)
        assert (off_by <= per * want + 2.0 ** -100).all(), "row %d: %.3g times what is allowed" % (r, (off_by / (per * want + 2.0 ** -100)).max())
        worst = max(worst, (off_by / (want + 2.0 ** -100)).max())
    if dtype == "bf16":
        assert worst > 2.0 ** -9                                # (the values do go through roundings)
