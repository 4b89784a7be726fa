"""The operators on the paged cache in the context's type as a program uses
them: a prompt in chunks, the weights that its entries gather, eviction,
drafting and verification on what stays; captured, on two streams, on one
workspace after another, and calls of many segments."""
import numpy as np
import pytest
import torch

import oracle as O
import synth
from gpu_util import F32_LOGIT_TOL, LOGIT_TOL, check_logits, dev, download_kv, host as bits, make_context, oracle_weights, upload_weights
from oracle import paged as P
from oracle import verifier as V
from test_gpu_kv_rows import attend, close, exact_on_gpu, host, i32, M_, norm_tol, out_tol, same_bits, turned
from test_gpu_verifier import TORCH, clean, context, normal

pytestmark = pytest.mark.gpu


class Prompt:
    """Prompts of `lens` rows that enter a cache in chunks, each attended over and weighed; then thinned out."""

    def __init__(self, ctx, lens, chunk, budget, rng, sink=2, recent=8):
        M, c = M_(), ctx.cfg
        self.ctx, self.lens, self.chunk, self.sink, self.recent = ctx, lens, chunk, sink, recent
        self.dtype = "bf16" if c.dtype else "f32"
        B, n_q, n_kv, hd = len(lens), int(c.n_q_heads), int(c.n_kv_heads), int(c.head_dim)
        width, small = (max(lens) + 31) // 16, (budget + 47) // 16
        perm = rng.permutation(B * (width + small))
        self.kv = M.KVCache.empty(ctx, B * (width + small), i32(perm[:B * width].reshape(B, width)))
        self.to = M.KVCache(self.kv.k_pool, self.kv.v_pool, i32(perm[B * width:].reshape(B, small)), i32(np.zeros(B)),
                            i32(np.zeros(B)), i32(np.zeros(B)))
        self.weights = torch.full((B * (width + small), n_kv, 16), float("nan"), device="cuda")
        self.kept = torch.zeros((B, n_kv, budget), dtype=torch.int32, device="cuda")
        self.budget = i32(np.full(B, budget))
        self.rope, self.ws = M.RopeTable(hd), M.AttentionWorkspace(ctx)
        self.qw, self.kw = (normal(rng, (hd,), self.dtype)[0] for _ in range(2))
        self.steps = []
        for lo in range(0, max(lens), chunk):
            n = np.array([max(0, min(chunk, L - lo)) for L in lens])
            off = np.concatenate([[0], np.cumsum(n)])
            T = int(off[-1])
            pos = np.concatenate([np.arange(lo, lo + x) for x in n])
            self.steps.append(dict(n=n, off=i32(off), pos=i32(pos), T=T, packed=torch.zeros((T, (n_q + 2 * n_kv) * hd), dtype=ctx.dtype, device="cuda"),
                                   q=torch.zeros((T, n_q, hd), dtype=ctx.dtype, device="cuda"), out=torch.zeros((T, n_q, hd), dtype=ctx.dtype, device="cuda"),
                                   lse=torch.zeros((T, n_q), device="cuda"), first=i32(np.minimum(lo, lens)), keep=i32(n)))
        self.shape = n_q, n_kv, hd

    def feed(self, rng):
        for s in self.steps:
            s["packed"].copy_(torch.from_numpy(rng.normal(size=s["packed"].shape)).to(self.ctx.dtype))

    def clear(self):
        for t in (self.kv.k_pool, self.kv.v_pool, self.kv.seq_len, self.kv.pending, self.to.seq_len, self.to.pending):
            t.zero_()

    def run(self):
        M, (n_q, n_kv, hd) = M_(), self.shape
        for s in self.steps:
            q, k, v = (s["packed"][:, a * hd:b * hd].unflatten(1, (b - a, hd)) for a, b in ((0, n_q), (n_q, n_q + n_kv), (n_q + n_kv, n_q + 2 * n_kv)))
            M.mtp_kv_append(self.ctx, self.kv, k, v, s["off"], q=q, q_out=s["q"], positions=s["pos"], rope=self.rope,
                            q_weight=self.qw, k_weight=self.kw)
            M.mtp_kv_attention(self.ctx, self.kv, s["q"], s["off"], s["out"], self.ws, self.chunk, lse=s["lse"])
            M.mtp_kv_attention_weights(self.ctx, self.kv, s["q"], s["off"], s["lse"], self.weights, self.chunk, first=s["first"])
            M.mtp_kv_commit(self.ctx, self.kv, s["keep"])
        M.mtp_kv_evict(self.ctx, self.kv, self.weights, self.budget, self.to, None, self.kept, sink=self.sink, recent=self.recent)
        M.mtp_kv_truncate(self.ctx, self.kv, torch.zeros_like(self.kv.seq_len))

    def results(self):
        return [t.clone() for s in self.steps for t in (s["q"], s["out"], s["lse"])] + [
            t.clone() for t in (self.kept, self.kv.k_pool, self.kv.v_pool, self.to.seq_len, self.kv.seq_len)]


@pytest.mark.parametrize("dtype,n_q,n_kv,hd", [("bf16", 8, 2, 128), ("f32", 4, 2, 64), ("bf16", 4, 4, 64)])
def test_prompts_in_chunks_thinned_out(dtype, n_q, n_kv, hd):
    """Every chunk's queries, keys and results, the gathered weights' choice, and what lies in the cache afterwards."""
    rng = np.random.default_rng(hd)
    ctx = context(n_q, n_kv, hd, dtype, max_batch=3)
    lens, budget = [150, 37, 90], 40
    s = Prompt(ctx, lens, 48, budget, rng)
    s.feed(rng)
    s.run()
    clean(ctx)
    qw, kw = host(s.qw), host(s.kw)
    K, Vv = ([np.zeros((0, n_kv, hd)) for _ in lens] for _ in range(2))
    gathered, slack = ([np.zeros((0, n_kv)) for _ in lens] for _ in range(2))
    for st in s.steps:
        p64, off, pos = host(st["packed"]), host(st["off"]).astype(int), host(st["pos"]).astype(int)
        q64, k64, v64 = (p64[:, a * hd:b * hd].reshape(-1, b - a, hd) for a, b in ((0, n_q), (n_q, n_q + n_kv), (n_q + n_kv, n_q + 2 * n_kv)))
        want_q = turned(q64, qw, 1e-6, pos, hd, "half")
        close(host(st["q"]), want_q, norm_tol(want_q, P.norm(q64, qw, 1e-6), dtype), "q")
        # keys as they are stored: rounded once
        k_st = torch.from_numpy(turned(k64, kw, 1e-6, pos, hd, "half")).to(TORCH[dtype]).double().numpy()
        for b in range(len(lens)):
            lo, hi = off[b], off[b + 1]
            if lo == hi:
                continue
            K[b], Vv[b] = np.concatenate([K[b], k_st[lo:hi]]), np.concatenate([Vv[b], v64[lo:hi]])
            L, n = len(K[b]), hi - lo
            o, ls, mass, size = V.attention(host(st["q"])[lo:hi], K[b], Vv[b], P.seen_of(n, L), hd ** -0.5)
            # a stored key next to a rounding border may be the other one: half a step of it, times the query
            more = (2.0 ** -8 if dtype == "bf16" else 2.0 ** -20) * size
            close(host(st["out"])[lo:hi], o, out_tol(o, mass, size, dtype) + 4 * more[..., None] * mass, "out")
            close(host(st["lse"])[lo:hi], ls, 2.0 ** -20 + 2.0 ** -17 * size + 2 * more + 2.0 ** -22 * np.abs(ls), "lse")
            add, asize = P.gathered(host(st["q"])[lo:hi], K[b], host(st["lse"])[lo:hi], P.seen_of(n, L), hd ** -0.5)
            pad = np.zeros((n, n_kv))
            gathered[b] = np.concatenate([gathered[b], pad]) + add
            slack[b] = np.concatenate([slack[b], pad]) + 2.0 ** -14 * add + ((2.0 ** -8 if dtype == "bf16" else 2.0 ** -17) * asize)
    kept = s.kept.cpu().numpy()
    for b, L in enumerate(lens):
        n = min(L, budget)
        blocks = s.to.block_table[b].cpu().numpy()
        for g in range(n_kv):
            mine = kept[b, g, :n]
            assert (np.diff(mine) > 0).all() and (kept[b, g, n:] == -1).all()
            if L > budget:
                assert set(range(2)) <= set(mine) and set(range(L - 8, L)) <= set(mine)
                # no entry that went outweighs one that stayed by more than the sums' errors
                free = np.arange(2, L - 8)
                stay, went = np.intersect1d(free, mine), np.setdiff1d(free, mine)
                w, e = gathered[b][:, g], slack[b][:, g]
                assert (w[went] - e[went]).max() <= (w[stay] + e[stay]).min()
            for j, t in enumerate(mine):
                at = int(blocks[j // 16]), g, j % 16
                assert np.array_equal(host(s.kv.v_pool[at]), Vv[b][t, g])
                close(host(s.kv.k_pool[at]), K[b][t, g], 2 * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -17) * np.abs(K[b][t, g]).max(), "kept key")
    assert s.to.seq_len.tolist() == [min(L, budget) for L in lens] and not s.kv.seq_len.any()
    for blk in s.kv.block_table.flatten().tolist():          # the old blocks are given back empty
        assert not s.kv.k_pool[blk].any() and not s.kv.v_pool[blk].any()


def test_prompts_captured_and_replayed():
    """All of it in a graph, replayed on new inputs, gives the bits that it gives when called; another context's
    graph of its own, replayed in between, changes nothing."""
    got = []
    for graph in (False, True):
        rng = np.random.default_rng(5)
        runs = [Prompt(context(8, 2, 128, "bf16", max_batch=2), [700, 130], 256, 64, rng) for _ in range(2)]
        graphs = []
        if graph:
            for s in runs:
                side = torch.cuda.Stream()
                with torch.cuda.stream(side):
                    g = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(g, stream=side):
                        s.run()
                graphs.append(g)
        for _ in range(3):
            for s in runs:
                s.feed(rng)
                s.clear()
            torch.cuda.synchronize()
            for i, s in enumerate(runs):
                graphs[i].replay() if graph else s.run()
            torch.cuda.synchronize()
            got.append([s.results() for s in runs])
        for s in runs:
            clean(s.ctx)
    for a, b in zip(got[:3], got[3:]):
        for x, y in zip(a, b):
            for u, v in zip(x, y):
                assert same_bits(u, v)


def test_two_streams_at_once():
    """Two prompts of one context on two streams, a cache and a workspace each, against one after the other."""
    rng = np.random.default_rng(6)
    ctx = context(8, 2, 128, "bf16", max_batch=2)
    runs = [Prompt(ctx, [600 + 100 * i, 33], 300, 50, rng) for i in range(2)]
    want = []
    for s in runs:
        s.feed(rng)
        s.run()
        torch.cuda.synchronize()
        want.append(s.results())
    for _ in range(5):
        for s in runs:
            s.clear()
        torch.cuda.synchronize()
        for s in runs:
            with torch.cuda.stream(torch.cuda.Stream()):
                s.run()
        torch.cuda.synchronize()
        for s, w in zip(runs, want):
            for a, b in zip(s.results(), w):
                assert same_bits(a, b)
    clean(ctx)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_drafts_on_a_thinned_cache(dtype):
    """The head's own cache: filled by mtp_kv_append, thinned out by weights, drafted on, against the oracle's draft
    over the entries that stayed; then the drafts are committed and attended over."""
    M = M_()
    rng = np.random.default_rng(7)
    cfg = synth.TINY_F32 if dtype == "f32" else synth.MTPShape("thin_bf16", H=512, n_q=8, n_kv=2, head_dim=128, ffn=1536, vocab=5003,
                                                               batch=1, K=3, dtype="bf16", ctx_lo=40, ctx_hi=40, seed_index=61)
    w = synth.make_weights(cfg, norm="random")
    ctx = make_context(cfg, upload_weights(w), max_pos=1024)
    L, budget, K = 200, 60, cfg.K
    kv = M.KVCache.empty(ctx, 40, i32(rng.permutation(40)[:16].reshape(1, 16)))
    rest = np.setdiff1d(np.arange(40), kv.block_table.cpu().numpy().ravel())
    to = M.KVCache(kv.k_pool, kv.v_pool, i32(rest[:6].reshape(1, 6)), i32([0]), i32([0]), i32([0]))
    k, v = (normal(rng, (L, cfg.n_kv, cfg.head_dim), dtype)[0] for _ in range(2))
    M.mtp_kv_append(ctx, kv, k, v, i32([0, L]), positions=i32(np.arange(L)), rope=M.RopeTable(cfg.head_dim, theta=cfg.rope_theta))
    M.mtp_kv_commit(ctx, kv, i32([L]))
    weights = torch.rand((40, cfg.n_kv, 16), device="cuda")
    kept = torch.empty((1, cfg.n_kv, budget), dtype=torch.int32, device="cuda")
    M.mtp_kv_evict(ctx, kv, weights, i32([budget]), to, None, kept, sink=4, recent=16)
    M.mtp_kv_truncate(ctx, kv, i32([0]))
    clean(ctx)
    twin = download_kv(to)
    di = synth.make_draft_inputs(cfg, w, np.array([L]))
    ids = torch.empty((1, K), dtype=torch.int32, device="cuda")
    logits = torch.empty((1, K, cfg.vocab), dtype=torch.float32, device="cuda")
    M.mtp_draft(ctx, dev(di.hidden), dev(di.embeds), dev(di.positions), to, K, ids, logits)
    clean(ctx)
    res = O.draft(oracle_weights(cfg, w), O.widen(di.hidden, dtype), O.widen(di.embeds, dtype), di.positions, twin, K,
                  chain_ids=bits(ids)[:, :K - 1])
    check_logits(bits(logits), res.logits, F32_LOGIT_TOL if dtype == "f32" else LOGIT_TOL)
    M.mtp_kv_commit(ctx, to, i32([2]))
    assert to.seq_len.tolist() == [budget + 2]
    q, q64 = normal(rng, (2, cfg.n_q, cfg.head_dim), dtype)
    out, lse = attend(ctx, to, q, [0, 2], 2)
    row = to.block_table[0].long()
    kk, vv = (host(p[row].transpose(1, 2).flatten(0, 1)[:budget + 2]) for p in (to.k_pool, to.v_pool))
    want, wl, mass, size = V.attention(q64, kk, vv, V.causal(2, budget + 2), cfg.head_dim ** -0.5)
    close(host(out), want, out_tol(want, mass, size, dtype), "out")
    clean(ctx)


def pooled(ctx, lens, new, rng):
    """A cache of that many entries, random numbers in every slot of its pools."""
    M = M_()
    need = [(a + n + 15) // 16 for a, n in zip(lens, new)]
    table, perm, at = np.zeros((len(lens), max(need)), np.int64), rng.permutation(sum(need)), 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    kv = M.KVCache.empty(ctx, sum(need), i32(table))
    g = torch.Generator(device="cuda").manual_seed(len(lens))
    for pool in (kv.k_pool, kv.v_pool):
        pool.copy_(torch.randn(pool.shape, generator=g, device="cuda"))
    kv.seq_len.copy_(i32(lens)), kv.pending.copy_(i32(new))
    return kv


@pytest.mark.parametrize("lens,new,n_q,n_kv,hd", [
    ([0], [2600], 32, 8, 128), ([100], [5200], 32, 8, 64), ([0, 3000, 17, 900, 0], [1000, 1, 700, 950, 0], 32, 8, 128),
    ([5] * 40, [130] * 40, 16, 4, 64), ([0, 60000], [4000, 3], 32, 8, 128)])
def test_calls_of_many_segments(lens, new, n_q, n_kv, hd):
    """Enough rows for the segments to be handed out whole, by size, and batches where one context is too long for that."""
    rng = np.random.default_rng(len(lens))
    ctx = context(n_q, n_kv, hd, "bf16", max_batch=len(lens))
    kv = pooled(ctx, lens, new, rng)
    off = np.concatenate([[0], np.cumsum(new)])
    q = torch.randn((int(off[-1]) + 3, n_q, hd), device="cuda").bfloat16()
    out, lse = attend(ctx, kv, q, off, max(new))
    clean(ctx)
    for b in range(len(lens)) if len(lens) < 10 else (0, 17, 39):
        if new[b] == 0:
            continue
        for h0 in (0, n_q - n_q // n_kv):      # a kv head's queries at a time, the first and the last
            G = n_q // n_kv
            one = M_().KVCache(kv.k_pool[:, h0 // G:h0 // G + 1].contiguous(), kv.v_pool[:, h0 // G:h0 // G + 1].contiguous(), kv.block_table, kv.seq_len, kv.pending)
            want, wl, mass, size = exact_on_gpu(q[:, h0:h0 + G], one, b, off[b], off[b + 1], hd ** -0.5, G)
            close(host(out[off[b]:off[b + 1], h0:h0 + G]), want, out_tol(want, mass, size, "bf16"), "out of request %d" % b)
            close(host(lse[off[b]:off[b + 1], h0:h0 + G]), wl, 2.0 ** -20 + 2.0 ** -17 * size + 2.0 ** -22 * np.abs(wl), "lse")
    assert bool((out[off[-1]:] == 5).all())
    again = attend(ctx, kv, q, off, max(new))
    assert same_bits(again[0], out) and same_bits(again[1], lse)


def test_many_segments_with_a_request_left_out():
    """One request's length does not fit its table: it alone is left, and reported."""
    M = M_()
    rng = np.random.default_rng(3)
    ctx = context(32, 8, 64, "bf16", max_batch=3)
    kv = pooled(ctx, [0, 10, 0], [1500, 400, 1500], rng)
    off = np.array([0, 1500, 1900, 3400])
    q = torch.randn((3400, 32, 64), device="cuda").bfloat16()
    want, want_lse = attend(ctx, kv, q, off, 1500)
    clean(ctx)
    kv.seq_len[1] = 10 ** 6
    out, lse = attend(ctx, kv, q, off, 1500)
    assert M.mtp_get_device_error(ctx) == M.MTP_ERR_CAPACITY
    assert bool((out[1500:1900] == 5).all()) and same_bits(out[:1500], want[:1500]) and same_bits(out[1900:], want[1900:])
    kv.seq_len[1] = 10
    out, lse = attend(ctx, kv, q, np.array([0, 1500, 1400, 3400]), 2000)     # offsets that go back: nothing happens
    assert M.mtp_get_device_error(ctx) == M.MTP_ERR_DEVICE_ARGS and bool((out == 5).all())


def test_masks_over_many_segments():
    """Trees of many requests, more segments than thread blocks."""
    rng = np.random.default_rng(4)
    B, rows = 96, 200
    ctx = context(4, 4, 64, "bf16", max_batch=B)
    lens = rng.integers(0, 200, B).tolist()
    kv = pooled(ctx, lens, [rows] * B, rng)
    off = np.arange(B + 1) * rows
    q = torch.randn((B * rows, 4, 64), device="cuda").bfloat16()
    tri = torch.ones((rows, rows), dtype=torch.bool).tril()
    bits_ = torch.zeros((rows, 224), dtype=torch.int64)
    bits_[:, :rows] = tri
    words = (bits_.view(rows, 7, 32) << torch.arange(32)).sum(-1)
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).int().repeat(B, 1).cuda()
    out, lse = attend(ctx, kv, q, off, rows, mask=words)          # causal, said by a mask
    want, _ = attend(ctx, kv, q, off, rows)
    clean(ctx)
    # the same numbers in steps cut elsewhere: each within its own tolerance of the exact result
    for b in (0, 50, 95):
        e, wl, mass, size = exact_on_gpu(q, kv, b, off[b], off[b + 1], 0.125, 1)
        for got in (out, want):
            close(host(got[off[b]:off[b + 1]]), e, out_tol(e, mass, size, "bf16"), "out")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_results_off_32_bytes_and_reused_workspaces(dtype):
    """An out tensor on 16 bytes alone; one workspace for a split call, then for calls that leave requests out."""
    M = M_()
    rng = np.random.default_rng(9)
    ctx = context(8, 2, 64, dtype, max_batch=2)
    kv = pooled(ctx, [9000, 40], [3, 200], rng)
    off = [0, 3, 203]
    q = torch.randn((203, 8, 64), device="cuda").to(TORCH[dtype])
    ws = M.AttentionWorkspace(ctx)
    ws.ws.fill_(0xFF)
    want, want_lse = attend(ctx, kv, q, off, 200, ws=ws)
    step = 16 // q.element_size()
    wide = torch.full((203 * 512 + step,), 5.0, dtype=TORCH[dtype], device="cuda")
    out = wide[step:].view(203, 8, 64)
    M.mtp_kv_attention(ctx, kv, q, i32(off), out, ws, 200)
    assert same_bits(out, want) and bool((wide[:step] == 5).all())
    for some in ([0, 0, 200], [0, 3, 3]):
        a = attend(ctx, kv, q, some, 200, ws=ws)
        b = attend(ctx, kv, q, some, 200)
        assert same_bits(a[0], b[0]) and same_bits(a[1], b[1])
    bad = torch.full((203 * 512 + 1,), 5.0, dtype=TORCH[dtype], device="cuda")[1:].view(203, 8, 64)
    with pytest.raises(M.MTPError):
        M.mtp_kv_attention(ctx, kv, q, i32(off), bad, ws, 200)
    clean(ctx)


@pytest.mark.parametrize("lens,new", [([30000], [1000]), ([900] * 8, [64] * 8), ([200] * 64, [1] * 64)])
def test_many_calls_without_a_wait_between(lens, new):
    """Calls queued one behind another, long and short segments: every wait in them ends, the results stay."""
    M = M_()
    rng = np.random.default_rng(12)
    ctx = context(32, 8, 128, "bf16", max_batch=len(lens))
    kv = pooled(ctx, lens, new, rng)
    off = np.concatenate([[0], np.cumsum(new)])
    q = torch.randn((int(off[-1]), 32, 128), device="cuda").bfloat16()
    ws = M.AttentionWorkspace(ctx)
    want, want_lse = attend(ctx, kv, q, off, max(new), ws=ws)
    for _ in range(40):
        M.mtp_kv_attention(ctx, kv, q, i32(off), want, ws, max(new), lse=want_lse)
    out, lse = attend(ctx, kv, q, off, max(new), ws=ws)
    clean(ctx)
    assert same_bits(out, want) and same_bits(lse, want_lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("slope", [0.5, 4.0, 30.0, -0.5, -30.0])
@pytest.mark.parametrize("rows", [1, 40, 300])
def test_scores_that_rise_or_fall_along_the_context(dtype, slope, rows):
    """Each 32 entries' largest score lies powers of two above (below) the ones before: the softmax's reference moves
    within steps and between them, from the first step to the ones that rows see only part of."""
    rng = np.random.default_rng(rows)
    ctx = context(8, 2, 128, dtype, max_batch=2)
    lens, new = [500, 0], [rows, rows]
    kv = pooled(ctx, lens, new, rng)
    for b in range(2):
        for i in range((lens[b] + new[b] + 15) // 16):
            t = torch.arange(16 * i, 16 * i + 16, device="cuda")
            kv.k_pool[int(kv.block_table[b, i]), :, :, 0] = (t * slope / 16).to(ctx.dtype)
    q = torch.randn((2 * rows, 8, 128), device="cuda").to(ctx.dtype)
    q[..., 0] = 11.0
    off = [0, rows, 2 * rows]
    out, lse = attend(ctx, kv, q, off, rows)
    clean(ctx)
    for b in range(2):
        want, wl, mass, size = exact_on_gpu(q, kv, b, off[b], off[b + 1], 128 ** -0.5, 4)
        close(host(out[off[b]:off[b + 1]]), want, out_tol(want, mass, size, dtype), "out")
        close(host(lse[off[b]:off[b + 1]]), wl, 2.0 ** -20 + 2.0 ** -17 * size + 2.0 ** -22 * np.abs(wl), "lse")
