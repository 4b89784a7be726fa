"""mtp_draft_kv8: the draft steps on an 8-bit cache, against the float64 oracle
with its cache replaced by the 8-bit twin (oracle/verifier.py).

Tolerances are those of mtp_draft (tests/gpu_util.py).  The twin quantizes the
oracle's own keys and values; where the GPU's, good to 2^-8, fall on the other
side of a rounding border, an element of one new entry moves by a step (2^-3 of
its value at most).  At that rate (2^-8 / 2^-3, one element in 32) such an
entry's score moves by about 2^-3 / sqrt(32) of an element's share of it, which
is far below the 2e-2 that logits are held to."""
import numpy as np
import pytest
import torch

import oracle as O
import oracle.mtp_oracle as core
import synth
from gpu_util import F32_LOGIT_TOL, LOGIT_TOL, Guarded, check_ids_are_argmax_of_own_logits, check_logits, dev, host
from oracle import verifier as V
from test_gpu_draft import Case

pytestmark = pytest.mark.gpu


def M_():
    import mtp_self_speculative_gb300 as M
    return M


def small(name, batch, K=3, lo=1, hi=70, **kw):
    base = dict(H=512, n_q=8, n_kv=2, head_dim=128, ffn=1536, vocab=5003, dtype="bf16")
    base.update(kw)
    return synth.MTPShape(name, batch=batch, K=K, ctx_lo=lo, ctx_hi=hi, seed_index=71, **base)


class Case8(Case):
    """A draft case whose initial cache is quantized, on the GPU and in the twin."""

    def __init__(self, cfg, **kw):
        super().__init__(cfg, norm="random", **kw)
        M, kv0 = M_(), self.kv0
        nb = kv0.k_pool.shape[0]
        self.kv = M.KVCache8.empty(self.ctx, nb, dev(kv0.block_table))
        self.twin = V.Cache8(nb, cfg.n_kv, cfg.head_dim, kv0.block_table)
        off = np.concatenate([[0], np.cumsum(self.lens)]).astype(np.int32)
        rows = [np.zeros((0, cfg.n_kv, cfg.head_dim), kv0.k_pool.dtype)] * 2
        for b, L in enumerate(self.lens):
            k, v = (np.stack([p[kv0.block_table[b, s // 16], :, s % 16] for s in range(int(L))]) if L else rows[0][:0]
                    for p in (kv0.k_pool, kv0.v_pool))
            rows = [np.concatenate([rows[0], k]), np.concatenate([rows[1], v])]
            self.twin.append(b, O.widen(k, cfg.dtype), O.widen(v, cfg.dtype))
            self.twin.commit(b, int(L))
        M.mtp_kv8_append(self.ctx, self.kv, dev(rows[0]), dev(rows[1]), dev(off))
        M.mtp_kv8_commit(self.ctx, self.kv, self.kv.pending)
        self.ws = M.Draft8Workspace(self.ctx)
        self.check_prefix()

    def check_prefix(self, drafted=0, requests=None):
        """Lengths, and the codes and scales of all whole blocks below them."""
        np.testing.assert_array_equal(self.kv.seq_len.cpu().numpy(), self.twin.seq_len)
        np.testing.assert_array_equal(self.kv.pending.cpu().numpy(), self.twin.pending)
        for b in range(self.B):
            for j in range(int(self.twin.seq_len[b]) // 16):
                blk = self.twin.table[b, j]
                for w, (pool, scale) in enumerate(((self.kv.k_pool, self.kv.k_scale), (self.kv.v_pool, self.kv.v_scale))):
                    np.testing.assert_array_equal(pool[blk].cpu().numpy(), self.twin.codes[w][blk])
                    np.testing.assert_array_equal(scale[blk].cpu().numpy(), self.twin.scale[w][blk])

    def draft(self, forced=True, stream=None):
        M, cfg, B, K = M_(), self.cfg, self.B, self.K
        ids, logits = Guarded((B, K), torch.int32, fill=-7), Guarded((B, K, cfg.vocab), torch.float32)
        hout = Guarded((B, cfg.H), torch.float32)
        chain = dev(self.chain[:, :K - 1].copy()) if forced and K > 1 else None
        M.mtp_draft_kv8(self.ctx, *self.inputs, self.kv, K, ids.t, self.ws, logits=logits.t, hidden_out=hout.t,
                        chain_ids=chain, stream=stream)
        torch.cuda.synchronize()
        for g, name in ((ids, "draft_ids"), (logits, "logits"), (hout, "hidden_out")):
            g.check(name)
        return host(ids.t), host(logits.t), host(hout.t)

    def expect(self, monkeypatch):
        """The oracle's forced draft, its cache accesses sent to the twin."""
        cfg, twin = self.cfg, self.twin

        def write(kv, b, slot, k, v, dtype):
            assert slot == twin.seq_len[b] + twin.pending[b]
            twin.append(b, *(O.widen(core.store_kv_values(x, dtype), dtype)[None] for x in (k, v)))

        with monkeypatch.context() as m:
            m.setattr(core, "_kv_write_slot", write)
            m.setattr(core, "kv_read_slots", lambda kv, b, n, dtype: tuple(twin.values(b, 0, n)))
            return self.oracle(np.arange(self.B), forced=True)[0]


CASES = [(synth.TINY_F32, {}, F32_LOGIT_TOL), (small("kv8_b1", 1), {}, LOGIT_TOL), (small("kv8_b3", 3), {}, LOGIT_TOL),
         (small("kv8_b7", 7), {}, LOGIT_TOL),                                       # tensor-core projections
         (small("kv8_d64", 2, head_dim=64), {}, LOGIT_TOL), (small("kv8_k18", 2, K=18, lo=5, hi=30), {}, LOGIT_TOL),
         (small("kv8_f32", 3, n_q=4, n_kv=4, dtype="f32", lo=15, hi=33), {}, F32_LOGIT_TOL),
         (small("kv8_q4", 2, H=1024, ffn=2048, vocab=4099), dict(weight_format="int4_g64"), LOGIT_TOL)]


@pytest.mark.parametrize("cfg,kw,tol", CASES, ids=[c[0].name for c in CASES])
def test_draft_on_the_8_bit_cache(cfg, kw, tol, monkeypatch):
    """Forced-chain logits and hidden state against the oracle; the new entries; roll-back; the same draft again."""
    M = M_()
    case = Case8(cfg, **kw)
    before = int(M.mtp_launch_count(case.ctx))
    ids, logits, hout = case.draft()
    assert M.mtp_get_device_error(case.ctx) == 0 and M.mtp_launch_count(case.ctx) > before
    check_ids_are_argmax_of_own_logits(ids, logits)
    res = case.expect(monkeypatch)
    check_logits(logits, res.logits, tol)
    err = np.max(np.abs(hout - res.hidden_out), -1) / np.max(np.abs(res.hidden_out), -1)
    assert np.max(err) <= tol
    case.check_prefix()
    # the drafted entries: at most a step of the format, and what the head itself may be off, from the twin's
    for b in range(case.B):
        L = int(case.lens[b])
        off = np.zeros(case.B + 1, np.int32)
        off[b + 1:] = case.K
        out = [torch.empty(case.K, cfg.n_kv, cfg.head_dim, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        start = np.zeros(case.B, np.int32)
        start[b] = L
        M.mtp_kv8_read(case.ctx, case.kv, dev(start), dev(off), *out)
        for got, want in zip(out, case.twin.values(b, L, L + case.K)):
            g = got.double().cpu().numpy()
            assert np.all(np.abs(g - want) <= 2.0 ** -3 * np.abs(want) + (2.0 ** -9 + tol) * np.max(np.abs(want)))
    M.mtp_kv8_rollback(case.ctx, case.kv)
    for b in range(case.B):
        case.twin.commit(b, 0)
    case.check_prefix()
    again = case.draft()
    np.testing.assert_array_equal(again[0], ids)     # (tail blocks keep their grown scales: the values are the same)
    assert M.mtp_get_device_error(case.ctx) == 0


def test_draft_verify_commit_over_several_steps():
    """Free-running drafts, synthetic verification, commit: lengths as on a bf16 cache, and a second run repeats the ids."""
    M = M_()
    cfg = small("kv8_loop", 2, K=4, lo=10, hi=40)
    runs = []
    for _ in range(2):
        case = Case8(cfg)
        B, K = case.B, case.K
        hist = []
        lens = case.lens.astype(np.int64).copy()
        rng = np.random.default_rng(3)
        for step in range(2):
            ids, logits, _ = case.draft(forced=False)
            hist.append(ids)
            check_ids_are_argmax_of_own_logits(ids, logits)
            acc = rng.integers(0, K + 1, B).astype(np.int32)
            if step == 0:
                acc[:] = 0       # the cache was made with room for K + 3 more entries
            M.mtp_kv8_commit_accepted(case.ctx, case.kv, dev(acc), extra=1)
            lens += np.minimum(acc + 1, K)
            np.testing.assert_array_equal(case.kv.seq_len.cpu().numpy(), lens)
            assert not case.kv.pending.any()
            pos = case.di.positions + 1
            case.inputs = case.inputs[:2] + (dev(pos.astype(np.int32)),)
        assert M.mtp_get_device_error(case.ctx) == 0
        runs.append(hist)
    for a, b in zip(*runs):
        np.testing.assert_array_equal(a, b)


@pytest.mark.parametrize("batch", [2, 7])
def test_requests_with_pending_entries_are_refused(batch):
    """Its cache and counts stay; the others draft as they would."""
    M = M_()
    cfg = small("kv8_pend", batch)
    good = Case8(cfg).draft()
    case = Case8(cfg)
    case.kv.pending[1] = 1
    pools = [t.clone() for t in (case.kv.k_pool, case.kv.v_pool, case.kv.k_scale, case.kv.v_scale)]
    ids, logits, _ = case.draft()
    assert M.mtp_get_device_error(case.ctx) == M.MTP_ERR_DEVICE_ARGS
    assert case.kv.pending.tolist() == [1 if b == 1 else cfg.K for b in range(batch)]
    for t, was in zip((case.kv.k_pool, case.kv.v_pool, case.kv.k_scale, case.kv.v_scale), pools):
        for blk in case.twin.table[1]:
            if blk >= 0:
                assert torch.equal(t[int(blk)], was[int(blk)])
    others = [b for b in range(batch) if b != 1]
    np.testing.assert_array_equal(logits[others], good[1][others])


def test_a_cache_that_is_full_and_bad_calls():
    M = M_()
    case = Case8(small("kv8_full", 2, lo=14, hi=14))
    case.kv.block_table = case.kv.block_table[:, :1].contiguous()      # 16 slots, 14 + 3 wanted
    case.draft()
    assert M.mtp_get_device_error(case.ctx) == M.MTP_ERR_CAPACITY
    assert case.kv.pending.tolist() == [2, 2]
    ids = torch.empty(2, 3, dtype=torch.int32, device="cuda")
    with pytest.raises(M.MTPError):
        M.mtp_draft_kv8(case.ctx, *case.inputs, case.kv, 0, torch.empty(2, 0, dtype=torch.int32, device="cuda"), case.ws)
    case.ws.bytes -= 1
    with pytest.raises(M.MTPError):
        M.mtp_draft_kv8(case.ctx, *case.inputs, case.kv, 3, ids, case.ws)
    with pytest.raises(ValueError):
        M.mtp_draft_kv8(case.ctx, *case.inputs, case.kv, 3, ids[:, :2], case.ws)
    bare = M.mtp_init(M.make_config(hidden=512, n_q_heads=8, n_kv_heads=2, head_dim=128, ffn=1536, vocab=5003, max_batch=2))
    with pytest.raises(M.MTPError):
        M.Draft8Workspace(bare)


def test_drafts_captured_and_replayed():
    """A captured draft, replayed after a roll-back, gives the ids and logits of the called one."""
    M = M_()
    for batch in (1, 7):
        case = Case8(small("kv8_graph", batch))
        B, K = case.B, case.K
        want = case.draft(forced=False)
        M.mtp_kv8_rollback(case.ctx, case.kv)
        ids, logits = torch.empty(B, K, dtype=torch.int32, device="cuda"), torch.empty(B, K, case.cfg.vocab, device="cuda")
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                M.mtp_draft_kv8(case.ctx, *case.inputs, case.kv, K, ids, case.ws, logits=logits)
                M.mtp_kv8_rollback(case.ctx, case.kv)
        for _ in range(3):
            ids.fill_(-1)
            g.replay()
            torch.cuda.synchronize()
            np.testing.assert_array_equal(host(ids), want[0])
            np.testing.assert_array_equal(host(logits), want[1])
        assert M.mtp_get_device_error(case.ctx) == 0


@pytest.mark.parametrize("cfg,tol,persistent", [(synth.TINY_F32, F32_LOGIT_TOL, 0), (small("rope_b1", 1), LOGIT_TOL, 0),
                                                (small("rope_p", 2), LOGIT_TOL, 4), (small("rope_b7", 7), LOGIT_TOL, 0)],
                         ids=["f32", "b1", "persistent", "b7"])
@pytest.mark.parametrize("kw", [dict(scaling="linear", factor=4.0), dict(scaling="yarn", factor=8.0, original_max_pos=64),
                                dict(theta=5000.0, magnitude=0.5)], ids=["linear", "yarn", "theta"])
def test_drafts_with_a_rotary_table_of_their_own(cfg, tol, persistent, kw, monkeypatch):
    """mtp_set_rope: the head's drafts follow the table's frequencies and magnitude; the default table gives the default."""
    M = M_()
    case = Case(cfg, norm="random", persistent_max_batch=persistent)
    plain = case.gpu_draft()[1]
    kw = {"theta": cfg.rope_theta, **kw}
    M.mtp_set_rope(case.ctx, M.RopeTable(cfg.head_dim, **kw))
    ids, logits, hout, _ = case.gpu_draft()
    with monkeypatch.context() as m:
        m.setattr(core, "rope", lambda x, pos, theta: V.rope(x[None], [pos], **kw)[0])
        res, _ = case.oracle(np.arange(case.B))
    check_logits(logits, res.logits, tol)
    assert not np.array_equal(logits, plain)
    M.mtp_set_rope(case.ctx, M.RopeTable(cfg.head_dim, theta=cfg.rope_theta))
    check_logits(case.gpu_draft()[1], plain.astype(np.float64), 1e-3 if cfg.dtype == "f32" else 1e-2)


def test_rotary_tables_that_do_not_fit_the_head_are_refused():
    M = M_()
    case = Case(synth.TINY_F32)
    for kw in (dict(rotary_dim=32), dict(rotary_dim=64, layout="interleaved"), dict(rotary_dim=128)):
        with pytest.raises(M.MTPError):
            M.mtp_set_rope(case.ctx, M.RopeTable(**kw))
    bare = M.mtp_init(M.make_config(hidden=256, n_q_heads=4, n_kv_heads=2, head_dim=64, ffn=256, vocab=100))
    with pytest.raises(M.MTPError):
        M.mtp_set_rope(bare, M.RopeTable(64))


RANGE_CASES = [(small("kv8_range_b2", 2), {}), (small("kv8_range_b7", 7), {}),          # the streamed and the tcgen05 projections
               (small("kv8_range_f32", 3, n_q=4, n_kv=4, head_dim=64, dtype="f32"), {}),
               (small("kv8_range_q4", 2, H=1024, ffn=2048, vocab=4099), dict(weight_format="int4_g64"))]


@pytest.mark.parametrize("cfg,kw", RANGE_CASES, ids=[c[0].name for c in RANGE_CASES])
def test_positions_out_of_range_leave_the_entries_and_scales(cfg, kw):
    """A step whose position lies outside 0 .. max_pos - 1 writes no entry, whatever the workspace held: its slot stays
    zero, the scales and the committed entries of the tail block stay as they were; `pending` grows as on a 16-bit
    cache.  Request 0 leaves the range at step 2, request 1 before step 1, and is below it in a second run."""
    M = M_()
    lens = [21, 37, 5, 16, 1, 60, 33][:cfg.batch]
    limit = max(lens) + cfg.K + 8
    fields = ("k_pool", "v_pool", "k_scale", "v_scale")

    def bytes_of(case, b):
        return [getattr(case.kv, f)[case.kv.block_table[b][case.kv.block_table[b] >= 0].long()].clone() for f in fields]

    for pos1 in (limit, -cfg.K):
        got = []
        for K in (cfg.K, 1):
            case = Case8(cfg, lens=lens, **kw)
            assert case.ctx.cfg.max_pos == limit
            case.inputs[2][:2] = torch.tensor([limit - 1, pos1])
            case.ws.ws.fill_(0x7E)                # 8e37 in both types
            before = bytes_of(case, 1)
            case.K = K
            _, logits, _ = case.draft()
            assert M.mtp_get_device_error(case.ctx) == M.MTP_ERR_CAPACITY
            assert case.kv.pending.tolist() == [K] * case.B
            for a, b in zip(bytes_of(case, 1), before):
                assert torch.equal(a, b)
            # the slots that were skipped: no bits
            for b, first in ((0, lens[0] + 1), (1, lens[1])):
                for s in range(first, lens[b] + K):
                    for pool in (case.kv.k_pool, case.kv.v_pool):
                        assert not pool[case.kv.block_table[b, s // 16].long(), :, s % 16].any()
            got.append((bytes_of(case, 0), logits))
            M.mtp_kv8_rollback(case.ctx, case.kv)
            for a, b in zip(bytes_of(case, 1), before):
                assert torch.equal(a, b)
        # after three steps request 0 holds what it holds after its only one within the range
        for a, b in zip(got[0][0], got[1][0]):
            assert torch.equal(a, b)
        if cfg.batch > 2:                         # the others draft as they would
            good = Case8(cfg, lens=lens, **kw).draft()[1]
            np.testing.assert_array_equal(got[0][1][2:], good[2:])


@pytest.mark.parametrize("cfg", [small("kv8_tail", 3), small("kv8_tail_b7", 7), small("kv8_tail_f32", 2, dtype="f32", head_dim=64)],
                         ids=lambda c: c.name)
def test_a_drafted_entry_that_raises_its_blocks_scale(cfg):
    """Committed entries of a tail block, far smaller than the drafted one: their codes are the old ones, rounded once
    to the scale that the block has afterwards."""
    M = M_()
    lens = [21, 37, 5, 15, 1, 60, 33][:cfg.batch]
    case = Case8(cfg, lens=lens)
    rng = np.random.default_rng(7)
    zero = np.zeros(case.B, np.int32)
    M.mtp_kv8_truncate(case.ctx, case.kv, dev(zero))
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    rows = torch.from_numpy(rng.normal(size=(off[-1], cfg.n_kv, cfg.head_dim)) * 2.0 ** -5)
    rows = rows.to(torch.bfloat16 if cfg.dtype == "bf16" else torch.float32)
    for b in range(case.B):
        case.twin.truncate(b, 0)
        case.twin.append(b, rows[off[b]:off[b + 1]].double().numpy(), rows[off[b]:off[b + 1]].double().numpy())
        case.twin.commit(b, lens[b])
    M.mtp_kv8_append(case.ctx, case.kv, rows.cuda(), rows.cuda(), dev(off))
    M.mtp_kv8_commit(case.ctx, case.kv, case.kv.pending)
    case.K = 1
    case.draft()
    assert M.mtp_get_device_error(case.ctx) == 0
    grown = 0
    for b in range(case.B):
        blk, held = case.twin.table[b, lens[b] // 16], lens[b] % 16
        for w, (pool, scale) in enumerate(((case.kv.k_pool, case.kv.k_scale), (case.kv.v_pool, case.kv.v_scale))):
            codes, now = pool[blk].cpu().numpy(), scale[blk].double().cpu().numpy()
            was = case.twin.scale[w][blk]
            assert np.all(now >= was)
            grown += int(np.sum((now > was) & (was > 0)))
            for g in range(cfg.n_kv):
                if held:
                    want = V.e4m3_encode(V.VALUES[case.twin.codes[w][blk, g, :held]] * (was[g] / now[g]))
                    np.testing.assert_array_equal(codes[g, :held], want)
            assert not codes[:, held + 1:].any()
    assert grown > 0


def test_a_rotary_table_is_in_place_when_mtp_set_rope_returns():
    """A draft on another stream, right behind the call, reads the new table to its end."""
    M = M_()
    case = Case(synth.TINY_F32, norm="random")
    cfg, limit = case.cfg, 1 << 18
    ctx = M.mtp_init(M.make_config(cfg.H, cfg.n_q, cfg.n_kv, cfg.head_dim, cfg.ffn, cfg.vocab, cfg.eps, cfg.rope_theta,
                                   cfg.dtype, case.B, case.K, 16, limit), case.wdev)
    case.ctx = ctx
    case.inputs[2].fill_(limit - case.K)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for theta in (5000.0, 1e6, 20000.0):
        got = []
        for fresh in (True, False):
            kvd = M.KVCache(*(dev(x) for x in (case.kv0.k_pool, case.kv0.v_pool, case.kv0.block_table, case.kv0.seq_len,
                                               case.kv0.pending)))
            ids = torch.empty(case.B, case.K, dtype=torch.int32, device="cuda")
            logits = torch.empty(case.B, case.K, cfg.vocab, device="cuda")
            torch.cuda.synchronize()
            if fresh:
                M.mtp_set_rope(ctx, M.RopeTable(cfg.head_dim, theta=theta))
            M.mtp_draft(ctx, *case.inputs, kvd, case.K, ids, logits, stream=side)
            torch.cuda.synchronize()
            got.append(host(logits))
        np.testing.assert_array_equal(*got)
    assert M.mtp_get_device_error(ctx) == 0


def test_a_new_context_is_ready_for_any_stream():
    """A draft on another stream right behind mtp_init reads the whole rotary table; an error word that was read and
    cleared takes nothing with it that a later call on that stream reports."""
    M = M_()
    case = Case(synth.TINY_F32, norm="random")
    cfg, limit = case.cfg, 1 << 18
    case.inputs[2].fill_(limit - case.K)
    side = torch.cuda.Stream()
    got = []
    for _ in range(2):
        kvd = M.KVCache(*(dev(x) for x in (case.kv0.k_pool, case.kv0.v_pool, case.kv0.block_table, case.kv0.seq_len,
                                           case.kv0.pending)))
        ids = torch.empty(case.B, case.K, dtype=torch.int32, device="cuda")
        logits = torch.empty(case.B, case.K, cfg.vocab, device="cuda")
        torch.cuda.synchronize()
        if not got:
            ctx = M.mtp_init(M.make_config(cfg.H, cfg.n_q, cfg.n_kv, cfg.head_dim, cfg.ffn, cfg.vocab, cfg.eps,
                                           cfg.rope_theta, cfg.dtype, case.B, case.K, 16, limit), case.wdev)
        M.mtp_draft(ctx, *case.inputs, kvd, case.K, ids, logits, stream=side)
        torch.cuda.synchronize()
        got.append(host(logits))
    np.testing.assert_array_equal(*got)
    for _ in range(50):       # pending entries left by the drafts above: refused each time
        M.mtp_draft(ctx, *case.inputs, kvd, case.K, ids, logits, stream=side)
        assert M.mtp_get_device_error(ctx) == M.MTP_ERR_DEVICE_ARGS
