"""Eviction where a table is much wider than some of its contexts: a cluster
shares a head's slots, and short requests leave some of its thread blocks few
slots, none, or slots that always stay."""
import numpy as np
import pytest
import torch

from oracle import paged as P
from test_gpu_verifier import M_, clean, context, i32

pytestmark = pytest.mark.gpu


def evict_wide(ctx, max_blocks, lens, budgets, rng, sink=0, recent=0, top=6):
    """Weights below `top`, many of them equal; against the oracle's choice, entries by their bits."""
    M, c = M_(), ctx.cfg
    B, n_kv, hd = len(lens), int(c.n_kv_heads), int(c.head_dim)
    need = [(L + 15) // 16 for L in lens]
    nb, room = sum(need) + 1, max(1, max(min(L, b) for L, b in zip(lens, budgets)))
    order, at = rng.permutation(nb), 0
    table = np.full((B, max_blocks), -1, np.int64)            # blocks behind a context are nobody's
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    kv = M.KVCache.empty(ctx, nb, i32(table))
    kv.k_pool.copy_(torch.from_numpy(rng.normal(size=kv.k_pool.shape)))
    kv.v_pool.copy_(torch.from_numpy(rng.normal(size=kv.v_pool.shape)))
    kv.seq_len.copy_(i32(lens))
    w = torch.from_numpy(rng.integers(0, top, (nb, n_kv, 16)).astype(np.float32)).cuda()
    per = (room + 15) // 16
    to = M.KVCache.empty(ctx, B * per, i32(rng.permutation(B * per).reshape(B, per)))
    to_w = torch.full((B * per, n_kv, 16), -3.0, device="cuda")
    kept = torch.full((B, n_kv, room), -9, dtype=torch.int32, device="cuda")
    M.mtp_kv_evict(ctx, kv, w, i32(budgets), to, to_w, kept, sink=sink, recent=recent)
    clean(ctx)
    assert to.seq_len.tolist() == [min(L, b) for L, b in zip(lens, budgets)] and not to.pending.any()
    for b, L in enumerate(lens):
        n = min(L, budgets[b])
        blocks, dst = (torch.as_tensor(t[b, :m].astype(np.int64)).cuda() for t, m in ((table, need[b]), (to.block_table.cpu().numpy(), (n + 15) // 16)))
        k, v, x = (y[blocks].transpose(1, 2).flatten(0, 1) for y in (kv.k_pool, kv.v_pool, w))   # [slots, n_kv, ..]
        tk, tv, tx = (y[dst].transpose(1, 2).flatten(0, 1) for y in (to.k_pool, to.v_pool, to_w))
        for g in range(n_kv):
            want = P.kept(x[:L, g].cpu().numpy(), budgets[b], sink, recent)
            np.testing.assert_array_equal(kept[b, g, :n].cpu().numpy(), want, err_msg="request %d, head %d" % (b, g))
            assert bool((kept[b, g, n:] == -1).all())
            at = torch.as_tensor(want).cuda()
            assert torch.equal(tk[:n, g], k[at, g]) and torch.equal(tv[:n, g], v[at, g]) and torch.equal(tx[:n, g], x[at, g])


@pytest.mark.parametrize("recent", [0, 1, 2, 3])
@pytest.mark.parametrize("max_blocks,lens", [
    (129, [1, 101, 127, 130, 383, 2001]), (257, [301, 601, 2, 1027, 1101, 4112]), (600, [130, 9599, 385, 1151, 2049, 3]),
    (1024, [301, 9000, 2, 1101, 16384, 513])])
def test_short_requests_in_a_wide_table(max_blocks, lens, recent):
    """Two and four thread blocks a head; budgets of nothing, one, below the length by one and at it."""
    rng = np.random.default_rng(max_blocks + recent)
    ctx = context(2, 2, 64, "bf16", max_batch=6)
    for budgets in ([max(L // 3, recent) for L in lens], [max(L - 1, recent) for L in lens], [recent] * 6, [recent + 1] * 6,
                    [max(L if i % 2 else L - 2, recent) for i, L in enumerate(lens)]):
        evict_wide(ctx, max_blocks, lens, budgets, rng, recent=recent)


@pytest.mark.parametrize("dtype,n_kv,hd", [("f32", 1, 128), ("bf16", 8, 128)])
def test_regions_that_cross_shares(dtype, n_kv, hd):
    """The first and last entries fill a share, or several; weights of many and of one value."""
    rng = np.random.default_rng(n_kv)
    ctx = context(n_kv, n_kv, hd, dtype, max_batch=4)
    for sink, recent, top in ((0, 0, 1000), (130, 0, 6), (0, 130, 6), (129, 200, 1), (300, 1, 50), (3, 700, 6)):
        lens = [301, 1101, 2050, 6001]
        evict_wide(ctx, 600, lens, [sink + recent + x for x in (0, 7, 100, 1)], rng, sink, recent, top)


def test_every_length_up_to_a_cluster_of_full_shares():
    """One request a length, ten at a time, four thread blocks a head."""
    rng = np.random.default_rng(4)
    ctx = context(1, 1, 64, "bf16", max_batch=10)
    for first in range(1, 1160, 110):
        lens = [first + 11 * i for i in range(10)]
        evict_wide(ctx, 300, lens, [L // 2 for L in lens], rng)


@pytest.mark.parametrize("max_blocks", [40, 257])
@pytest.mark.parametrize("bad", [-1, 38])
def test_entries_of_a_block_outside_the_pool_count_as_zeros(max_blocks, bad):
    """Their weight too: above negative ones and NaN, equal to zeros, below the rest."""
    M = M_()
    ctx = context(1, 1, 64, "bf16", max_batch=1)
    nb, L = 38, 600
    rng = np.random.default_rng(max_blocks)
    table = np.concatenate([np.arange(nb), np.full(max_blocks - nb, -1)])[None]
    table[0, [1, 20]] = bad
    kv, to = M.KVCache.empty(ctx, nb, i32(table)), M.KVCache.empty(ctx, nb, i32(np.arange(nb)[None]))
    kv.k_pool.fill_(1.0), kv.v_pool.fill_(2.0)
    kv.seq_len.fill_(L)
    w = torch.from_numpy(rng.choice(np.array([-1.0, 0.0, np.nan, 1.0], np.float32), (nb, 1, 16))).cuda()
    flat = w.flatten().cpu().numpy()[:L].copy()
    for x in (1, 20):
        flat[16 * x:16 * x + 16] = 0.0
    for budget in (50, 180, 300, 599):
        kept = torch.zeros((1, 1, 600), dtype=torch.int32, device="cuda")
        to_w = torch.full((nb, 1, 16), 5.0, device="cuda")
        M.mtp_kv_evict(ctx, kv, w, i32([budget]), to, to_w, kept, sink=1, recent=3)
        assert M.mtp_get_device_error(ctx) == M.MTP_ERR_CAPACITY
        want = P.kept(flat, budget, 1, 3)
        np.testing.assert_array_equal(kept[0, 0, :budget].cpu().numpy(), want)
        lost = torch.as_tensor(np.isin(want // 16, (1, 20))).cuda()
        assert bool(lost.any()) or budget == 50
        got = to.k_pool[:, 0].flatten(0, 1)[:budget]
        assert bool((got[lost] == 0).all()) and bool((got[~lost] == 1).all())
        np.testing.assert_array_equal(to_w.flatten()[:budget].cpu().numpy(), flat[want])
