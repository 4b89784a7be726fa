"""Attention read entry by entry: values are zero but for single slots, one in a
column of its own, so that each result is one entry's weight and is compared
relative to it.  Slots lie at the ends of blocks, steps, tiles and contexts and,
moved along, wherever a segment is cut into pieces; contexts are long enough for
a lost or doubled entry to be far below a tolerance of the whole row.

Tolerance, relative to a weight: scores are sums of head_dim products in float32,
any order, off by 2^-18 S with S = scale * max_t sum_d |q_d k_d|; a weight is off by
twice that, and 2^-20 for the exponential; its normalising sum by as much again:
2^-16 S + 2^-19.  bf16 heads: half a step (2^-8) where the weight becomes an operand and
half a step where the result is stored, and their product; float32: 2^-24 there.
"""
import numpy as np
import pytest
import torch

from test_gpu_verifier import M_, TORCH, clean, context, i32

pytestmark = pytest.mark.gpu


def probes(L, hd, shift):
    """hd different slots of L (all of them if there are fewer): ends, boundaries, the rest spread."""
    at = [0, L - 1, L - 2, 1]
    for step in (16, 64, 128, 256, 512):
        for i in range(1, 1 + L // step):
            if i <= 4 or i >= L // step - 3:
                at += [i * step - 1, i * step]
    at = [t for t in dict.fromkeys(at) if 0 <= t < L][:hd // 2]
    spread = [(int(x) + shift) % L for x in np.linspace(0, L - 1, 3 * hd)]
    return list(dict.fromkeys(at + spread))[:hd]


def check(dtype, n_q, n_kv, hd, lens, rows, shift=0, tree=False):
    M = M_()
    torch.manual_seed(shift)
    rng = np.random.default_rng(shift)
    B, G = len(lens), n_q // n_kv
    ctx = context(n_q, n_kv, hd, dtype, max_batch=B)
    need = [(L + 15) // 16 for L in lens]
    table, order, at = np.zeros((B, max(need)), np.int64), rng.permutation(sum(need)), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    kv = M.KVCache.empty(ctx, sum(need), i32(table))
    kv.k_pool.normal_()
    kv.seq_len.copy_(i32(lens)), kv.pending.zero_()
    where = [probes(L, hd, shift) for L in lens]
    for b, ts in enumerate(where):
        t = torch.as_tensor(ts)
        kv.v_pool[torch.as_tensor(table[b])[t // 16].cuda(), :, (t % 16).cuda(), torch.arange(len(ts)).cuda()] = 1.0
    T, off = sum(rows), np.concatenate([[0], np.cumsum(rows)])
    q = torch.randn(T, n_q, hd, device="cuda").to(TORCH[dtype])
    words = (max(rows) + 31) // 32
    bits = rng.random((T, words * 32)) < 0.5
    mask = (bits.reshape(T, words, 32) << np.arange(32)).sum(-1).astype(np.int64)
    mask = i32(np.where(mask >= 2 ** 31, mask - 2 ** 32, mask)) if tree else None
    out = torch.full((T, n_q, hd), 5.0, device="cuda").to(TORCH[dtype])
    M.mtp_kv_attention(ctx, kv, q, i32(off), out, M.AttentionWorkspace(ctx), max(rows), mask=mask)
    clean(ctx)
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    for b, (L, n) in enumerate(zip(lens, rows)):
        k = kv.k_pool[torch.as_tensor(table[b, :need[b]]).cuda()].transpose(1, 2).flatten(0, 1)[:L].double()   # [L, n_kv, hd]
        i, t = torch.arange(n, device="cuda")[:, None], torch.arange(L, device="cuda")[None]
        sees = t <= L - n + i
        if tree:
            mine = torch.as_tensor(bits[off[b]:off[b + 1], :n]).cuda()
            sees = torch.cat([torch.ones(n, L - n, dtype=torch.bool, device="cuda"), mine], 1)
        at = torch.as_tensor(where[b]).cuda()
        for h in range(n_q):
            z = q[off[b]:off[b + 1], h].double() @ k[:, h // G].T * hd ** -0.5
            size = (q[off[b]:off[b + 1], h].double().abs() @ k[:, h // G].T.abs() * hd ** -0.5).max(1, keepdim=True).values
            p = torch.softmax(z.masked_fill(~sees, -float("inf")), 1).nan_to_num(0.0)
            want = torch.zeros(n, hd, dtype=torch.float64, device="cuda")
            want[:, :len(at)] = p[:, at]
            tol = (2 * half + half * half + 2.0 ** -16 * size + 2.0 ** -19) * want
            bad = ~((out[off[b]:off[b + 1], h].double() - want).abs() <= tol)
            assert not bad.any(), "request %d, head %d: rows %s, slots %s" % (
                b, h, bad.nonzero()[:4, 0].tolist(), [where[b][c] if c < len(at) else -1 for c in bad.nonzero()[:4, 1].tolist()])


SHAPES = [("bf16", 8, 2, 128), ("bf16", 4, 1, 64), ("f32", 8, 2, 128), ("f32", 2, 2, 64)]


@pytest.mark.parametrize("dtype,n_q,n_kv,hd", SHAPES)
@pytest.mark.parametrize("shift", [0, 37])
def test_decoding(dtype, n_q, n_kv, hd, shift):
    check(dtype, n_q, n_kv, hd, [1, 15, 127, 129, 1000, 5003, 40001], [1] * 7, shift)


@pytest.mark.parametrize("dtype,n_q,n_kv,hd", SHAPES)
def test_one_request_alone(dtype, n_q, n_kv, hd):
    for L in (20000, 33333):
        check(dtype, n_q, n_kv, hd, [L], [1], L)


@pytest.mark.parametrize("dtype,n_q,n_kv,hd", SHAPES)
@pytest.mark.parametrize("tree", [False, True])
def test_a_few_rows(dtype, n_q, n_kv, hd, tree):
    check(dtype, n_q, n_kv, hd, [6, 131, 2050, 9001], [6, 5, 6, 2], 11, tree)
    check(dtype, n_q, n_kv, hd, [33, 300, 12000], [33, 20, 33], 5, tree)


@pytest.mark.parametrize("dtype,n_q,n_kv,hd", SHAPES)
def test_chunks(dtype, n_q, n_kv, hd):
    check(dtype, n_q, n_kv, hd, [301, 3000, 64, 6001], [301, 257, 1, 100], 3)


@pytest.mark.parametrize("hd", [64, 128])
def test_whole_segments_in_the_order_of_their_size(hd):
    """Enough rows that segments are handed out whole."""
    check("bf16", 16, 4, hd, [5000, 900], [5000, 300], 1)
