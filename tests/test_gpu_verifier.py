"""GPU parity of the verifier's side: rotary positions, the 8-bit cache
(append, read, edits), attention over it and logit processing, against the
float64 oracle (oracle/verifier.py).

Tolerances.  A result stored in a type t is off by at most eps(t) / 2 of its
value from what was computed (bf16 2^-8, float32 2^-24, e4m3 2^-4 or half its
smallest step).  What was computed is off from the exact value by float32
rounding:
  rotation  two products and a sum of factors that are good to 2^-22 (a
            cosine off by 1.2e-7 at most): 2^-20 (|a| + |b|);
  scores    a sum of head_dim products in float32, any order, from operands
            kept to 22 bits: 2^-18 S, S = scale * max_t sum_d |q_d k_d|;
            a weight is then off by twice that, plus 2^-20 for the exponential,
            plus, where weights are held in 11 bits (bf16 heads), 2^-11;
  outputs   so a sum of weighted values is off by that times sum_t p_t |v_t|
            (`mass`), of which the normalising sum takes as much again;
  logits    at most eight operations: 8 * 2^-24 of the sizes added up.
"""
import numpy as np
import pytest
import torch

from oracle import verifier as V

pytestmark = pytest.mark.gpu

HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def M_():
    import mtp_self_speculative_gb300 as M
    return M


def context(n_q=8, n_kv=2, hd=64, dtype="bf16", max_batch=8, vocab=1000, max_k=5):
    M = M_()
    return M.mtp_init(M.make_config(hidden=256, n_q_heads=n_q, n_kv_heads=n_kv, head_dim=hd, ffn=256, vocab=vocab,
                                    dtype=dtype, max_batch=max_batch, max_k=max_k))


def clean(ctx):
    assert M_().mtp_get_device_error(ctx) == 0


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def normal(rng, shape, dtype, scale=1.0):
    """(device tensor, the same values as float64)"""
    t = torch.from_numpy(rng.normal(size=shape) * scale).to(TORCH[dtype])
    return t.cuda(), t.double().numpy()


def host(t):
    return t.detach().double().cpu().numpy()


def same_bits(a, b):
    """Equal, NaN by NaN."""
    view = torch.int16 if a.element_size() == 2 else torch.int32
    return torch.equal(a.contiguous().view(view), b.contiguous().view(view))


def close(got, want, tol, what):
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - want) <= tol)
    bad &= ~(np.isnan(got) & np.isnan(want)) & ~((got == want) & np.isinf(want))
    assert not bad.any(), "%s: %d of %d off, worst %.3g times what is allowed" % (
        what, bad.sum(), bad.size, np.nanmax(np.abs(got - want) / np.maximum(tol, 1e-300)))


# ---------------------------------------------------------------- rotation

def rope_tol(x, want, dtype, mag=1.0):
    """Both members of a pair are at most the row's largest element."""
    return HALF_STEP[dtype] * np.abs(want) + 2.0 ** -19 * mag * np.abs(x).max(-1, keepdims=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,heads,hd,rd,layout,kw", [
    (1, 1, 64, 64, "half", dict()), (1, 32, 128, 128, "half", dict()),
    (37, 5, 128, 128, "interleaved", dict(scaling="linear", factor=4.0)),
    (300, 3, 64, 2, "half", dict(theta=10000.0)), (19, 4, 64, 62, "half", dict()),
    (33, 2, 128, 96, "half", dict(scaling="parts", factor=8.0, original_max_pos=8192)),
    (33, 7, 128, 34, "interleaved", dict(scaling="yarn", factor=16.0, original_max_pos=4096)),
    (1025, 8, 64, 48, "interleaved", dict()), (65, 40, 128, 64, "half", dict(magnitude=0.75))])
def test_rope(dtype, T, heads, hd, rd, layout, kw):
    M = M_()
    rng = np.random.default_rng(T + heads)
    ctx = context(hd=hd, dtype=dtype)
    x, x64 = normal(rng, (T, heads, hd), dtype)
    # near, far and negative positions, and the type's limits
    pos = rng.integers(-2 ** 20, 2 ** 20, T)
    pos[:4] = [0, 131071, 2 ** 31 - 1, -2 ** 31][:min(4, T)]
    tab = M.RopeTable(rd, layout=layout, **kw)
    before = x.clone()
    out = torch.full_like(x, 7.0)
    assert M.mtp_rope(ctx, x, i32(pos), tab, out) is out
    assert torch.equal(x, before)
    want = V.rope(x64, pos, layout, rd, **kw)
    # the table rounds a phase to 2^-53 of a turn per position relative to its size: at 2^31 positions 2^-24 turns
    far = 2 * np.pi * np.abs(pos)[:, None, None] * 2.0 ** -52
    close(host(out), want, rope_tol(x64, want, dtype, tab.magnitude) + far * np.abs(x64).max(-1, keepdims=True), "rope")
    assert torch.equal(out[..., rd:], x[..., rd:])
    M.mtp_rope(ctx, x, i32(pos), tab)          # in place
    assert torch.equal(x, out)
    clean(ctx)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("off", [0, 1, 8])
def test_rope_of_a_packed_projections_slice(dtype, layout, off):
    """Rows of a wider tensor, at an element offset that leaves them unaligned; what lies around them stays."""
    M = M_()
    rng = np.random.default_rng(off)
    ctx = context(hd=64, dtype=dtype)
    wide, w64 = normal(rng, (21, off + 3 * 64 + 5), dtype)
    x = wide[:, off:off + 192].unflatten(1, (3, 64))
    before = wide.clone()
    M.mtp_rope(ctx, x, i32(np.arange(21)), M.RopeTable(64, layout=layout))
    want = V.rope(w64[:, off:off + 192].reshape(21, 3, 64), np.arange(21), layout)
    close(host(wide)[:, off:off + 192].reshape(21, 3, 64), want, rope_tol(w64[:, off:off + 192].reshape(21, 3, 64), want, dtype), "rope")
    assert torch.equal(wide[:, :off], before[:, :off]) and torch.equal(wide[:, off + 192:], before[:, off + 192:])
    clean(ctx)


# ------------------------------------------------------------------- cache

def make_cache(ctx, B, max_blocks, rng, spare=3):
    """An empty device cache with a shuffled table, guard blocks around the pools, and the oracle's twin."""
    M = M_()
    c = ctx.cfg
    nb = B * max_blocks + spare
    table = rng.permutation(nb)[:B * max_blocks].reshape(B, max_blocks)
    kv = M.KVCache8.empty(ctx, nb, i32(table))
    kv.guards = []
    for name in ("k_pool", "v_pool"):
        wide = torch.full((nb + 2, c.n_kv_heads, 16, c.head_dim), 0xA5, dtype=torch.uint8, device="cuda")
        wide[1:-1] = 0
        setattr(kv, name, wide[1:-1])
        kv.guards.append(wide)
    return kv, V.Cache8(nb, c.n_kv_heads, c.head_dim, table)


def check_cache(ctx, kv, twin, codes=True):
    for w in kv.guards:
        assert bool((w[0] == 0xA5).all()) and bool((w[-1] == 0xA5).all()), "bytes around a pool overwritten"
    np.testing.assert_array_equal(kv.seq_len.cpu().numpy(), twin.seq_len)
    np.testing.assert_array_equal(kv.pending.cpu().numpy(), twin.pending)
    assert not kv.arrive.any()
    if codes:
        for w, (pool, scale) in enumerate(((kv.k_pool, kv.k_scale), (kv.v_pool, kv.v_scale))):
            np.testing.assert_array_equal(scale.cpu().numpy(), twin.scale[w])
            np.testing.assert_array_equal(pool.cpu().numpy(), twin.codes[w])


def append_both(ctx, kv, twin, counts, rng, scale=1.0, first=0, extra=0, **kw):
    """Append counts[b] rows to each request on both sides (no rotation: bit-exact)."""
    M, c = M_(), ctx.cfg
    dt = "bf16" if c.dtype else "f32"
    T = first + int(np.sum(counts)) + extra
    off = first + np.concatenate([[0], np.cumsum(counts)])
    k, k64 = normal(rng, (T, c.n_kv_heads, c.head_dim), dt, scale)
    v, v64 = normal(rng, (T, c.n_kv_heads, c.head_dim), dt, scale * 3)
    M.mtp_kv8_append(ctx, kv, k, v, i32(off), **kw)
    for b in range(len(counts)):
        twin.append(b, k64[off[b]:off[b + 1]], v64[off[b]:off[b + 1]])
    return off


@pytest.mark.parametrize("dtype,n_q,n_kv,hd", [("bf16", 8, 2, 64), ("f32", 4, 4, 128), ("bf16", 8, 1, 128),
                                               ("f32", 2, 2, 64), ("bf16", 32, 8, 128)])
def test_append_and_edits_are_bit_exact(dtype, n_q, n_kv, hd):
    """Sequences of appends (blocks that fill, cross and grow their scale), commits, roll-backs and truncations."""
    M = M_()
    rng = np.random.default_rng(hd + n_q)
    ctx = context(n_q, n_kv, hd, dtype, max_batch=4)
    kv, twin = make_cache(ctx, 4, 6, rng)
    # lengths of one, of a whole block, across blocks, and none; rows in front of the first and behind the last
    for counts, scale in (([1, 16, 37, 0], 1.0), ([1, 0, 3, 17], 30.0), ([14, 1, 1, 1], 1e-3)):
        append_both(ctx, kv, twin, counts, rng, scale, first=2, extra=3)
        check_cache(ctx, kv, twin)
    keep = [16, 3, 0, 18]
    M.mtp_kv8_commit(ctx, kv, i32(keep))
    for b, n in enumerate(keep):
        twin.commit(b, n)
    check_cache(ctx, kv, twin)
    append_both(ctx, kv, twin, [5, 6, 7, 8], rng, 100.0)
    M.mtp_kv8_commit_accepted(ctx, kv, i32([0, 9, 2, 7]), extra=1)
    for b, n in enumerate([1, 6, 3, 8]):
        twin.commit(b, n)
    check_cache(ctx, kv, twin)
    append_both(ctx, kv, twin, [40, 1, 16, 2], rng)
    M.mtp_kv8_rollback(ctx, kv)
    for b in range(4):
        twin.commit(b, 0)
    check_cache(ctx, kv, twin)
    append_both(ctx, kv, twin, [2, 2, 2, 2], rng)
    new = [17, 0, 3, 16]
    M.mtp_kv8_truncate(ctx, kv, i32(new))
    for b, n in enumerate(new):
        twin.truncate(b, n)
    check_cache(ctx, kv, twin)
    clean(ctx)


def test_append_in_more_waves_than_fit_the_gpu():
    """Thousands of thread blocks, half of them for a second cache block that a request's rows do not reach: one that
    starts after the others of its request have ended still counts from the old length.  Starts 0, 6, 12, 18, 24: from
    6 on, rows counted from the new length would reach the second block."""
    ctx = context(8, 8, 64, "bf16", max_batch=500)
    rng = np.random.default_rng(11)
    kv, twin = make_cache(ctx, 500, 2, rng)
    for _ in range(5):
        append_both(ctx, kv, twin, [6] * 500, rng)
        check_cache(ctx, kv, twin)
    clean(ctx)


@pytest.mark.parametrize("dtype,hd", [("bf16", 128), ("f32", 64)])
def test_append_of_extreme_values(dtype, hd):
    """Zeros of both signs, the type's largest and smallest numbers, infinities and NaN; appended in two steps."""
    ctx = context(4, 2, hd, dtype, max_batch=2)
    rng = np.random.default_rng(5)
    M = M_()
    kv, twin = make_cache(ctx, 2, 3, rng)
    big = float(torch.finfo(TORCH[dtype]).max)
    rows = np.zeros((12, 2, hd))
    rows[1] = -0.0
    rows[2, 0, ::3], rows[3, 1, 5] = np.inf, np.nan
    rows[4], rows[5, 0] = 1e-38, big
    rows[6] = rng.normal(size=(2, hd)) * 1e-39
    rows[7, :, 3] = -np.inf
    rows[8:] = rng.normal(size=(4, 2, hd))
    for part in (rows[:4], rows[4:5], rows[6:7], rows[8:], rows[5:6]):
        t = torch.from_numpy(part).to(TORCH[dtype]).cuda()
        n = len(part)
        M.mtp_kv8_append(ctx, kv, torch.cat([t, t]), torch.cat([t, t]), i32([0, n, 2 * n]))
        for b in range(2):
            twin.append(b, host(t), host(t))
        check_cache(ctx, kv, twin)
    clean(ctx)


@pytest.mark.parametrize("dtype,n_q,n_kv,hd,rd,layout", [("bf16", 8, 2, 64, 64, "half"), ("f32", 4, 4, 128, 128, "half"),
                                                         ("bf16", 32, 8, 128, 128, "interleaved"), ("bf16", 4, 4, 128, 62, "half"),
                                                         ("f32", 8, 1, 64, 6, "interleaved"), ("bf16", 16, 4, 128, 96, "half")])
def test_append_rotates_keys_and_queries(dtype, n_q, n_kv, hd, rd, layout):
    """Strided k, v and q of one packed projection; entries read back within half a step of the rotated values."""
    M = M_()
    rng = np.random.default_rng(rd)
    ctx = context(n_q, n_kv, hd, dtype, max_batch=3)
    kv, twin = make_cache(ctx, 3, 5, rng)
    append_both(ctx, kv, twin, [3, 0, 20], rng)
    M.mtp_kv8_commit(ctx, kv, i32([3, 0, 20]))
    counts = np.array([30, 1, 5])
    off = np.concatenate([[0], np.cumsum(counts)])
    T = int(off[-1])
    packed, p64 = normal(rng, (T, (n_q + 2 * n_kv) * hd), dtype)
    q, k, v = (packed[:, a * hd:e * hd].unflatten(1, (e - a, hd))
               for a, e in ((0, n_q), (n_q, n_q + n_kv), (n_q + n_kv, n_q + 2 * n_kv)))
    pos = rng.integers(0, 200000, T)
    tab = M.RopeTable(rd, layout=layout)
    q_out = torch.empty(T, n_q, hd, dtype=TORCH[dtype], device="cuda")
    before = packed.clone()
    M.mtp_kv8_append(ctx, kv, k, v, i32(off), q=q, q_out=q_out, positions=i32(pos), rope=tab)
    assert torch.equal(packed, before)
    q64, k64 = p64[:, :n_q * hd].reshape(T, n_q, hd), p64[:, n_q * hd:(n_q + n_kv) * hd].reshape(T, n_kv, hd)
    v64 = p64[:, (n_q + n_kv) * hd:].reshape(T, n_kv, hd)
    want_q, want_k = V.rope(q64, pos, layout, rd), V.rope(k64, pos, layout, rd)
    close(host(q_out), want_q, rope_tol(q64, want_q, dtype), "q")
    k_out = torch.empty(T + 2, n_kv, hd, dtype=torch.bfloat16, device="cuda").fill_(9.0)
    v_out = k_out.clone()
    M.mtp_kv8_read(ctx, kv, i32([3, 0, 20]), i32(off), k_out, v_out)
    clean(ctx)
    assert bool((k_out[T:] == 9).all()) and bool((v_out[T:] == 9).all())
    for b in range(3):
        for i in range(counts[b]):
            r, slot = off[b] + i, [3, 0, 20][b] + i
            s = kv.k_scale[twin.table[b, slot // 16]].double().cpu().numpy()[:, None]
            tol = np.maximum(2.0 ** -4 * np.abs(want_k[r]), s * 2.0 ** -10) + 2.0 ** -18 * np.abs(k64[r]).max()
            close(host(k_out)[r], want_k[r], tol, "k")
    # values are not rotated: exact
    for b in range(3):
        twin.commit(b, [3, 0, 20][b])
        twin.append(b, want_k[off[b]:off[b + 1]], v64[off[b]:off[b + 1]])
        np.testing.assert_array_equal(host(v_out)[off[b]:off[b + 1]], twin.values(b, [3, 0, 20][b], [3, 0, 20][b] + counts[b])[1])
    M.mtp_kv8_append(ctx, kv, k[:0], v[:0], i32([0, 0, 0, 0]))   # nothing to append
    M.mtp_kv8_rollback(ctx, kv)
    M.mtp_kv8_append(ctx, kv, k, v, i32(off), q=q, positions=i32(pos), rope=tab)   # queries in place
    assert torch.equal(q.contiguous(), q_out) and torch.equal(packed[:, n_q * hd:], before[:, n_q * hd:])
    check_cache(ctx, kv, twin, codes=False)
    clean(ctx)


def test_path_commit_moves_and_requantizes():
    """Paths over blocks of different scales, the empty path, the whole tree; and lists that are refused."""
    M = M_()
    rng = np.random.default_rng(11)
    ctx = context(4, 2, 64, "bf16", max_batch=4)
    kv, twin = make_cache(ctx, 4, 20, rng)
    append_both(ctx, kv, twin, [13, 0, 16, 7], rng, 0.1)
    M.mtp_kv8_commit(ctx, kv, i32([13, 0, 16, 7]))
    for b, n in enumerate([13, 0, 16, 7]):
        twin.commit(b, n)
    append_both(ctx, kv, twin, [10, 40, 20, 5], rng, 1.0)
    append_both(ctx, kv, twin, [10, 5, 200, 0], rng, 50.0)
    keep = np.zeros((4, 30), np.int64)
    paths = [[0, 3, 11, 19], [1, 2, 30, 44], [], [0, 1, 2, 3, 4]]
    for b, p in enumerate(paths):
        keep[b, :len(p)] = p
    M.mtp_kv8_commit_path(ctx, kv, i32(keep), i32([len(p) for p in paths]))
    for b, p in enumerate(paths):
        twin.commit(b, len(p), p)
    check_cache(ctx, kv, twin)
    clean(ctx)
    # not ascending, named twice, out of range, more than there are: unchanged, and the others go through
    append_both(ctx, kv, twin, [4, 4, 4, 4], rng)
    bad = i32([[1, 0], [2, 2], [0, 4], [1, 3]])
    M.mtp_kv8_commit_path(ctx, kv, bad, i32([2, 2, 2, 2]))
    twin.commit(3, 2, [1, 3])
    assert M.mtp_get_device_error(ctx) == M.MTP_ERR_DEVICE_ARGS
    check_cache(ctx, kv, twin)


def test_edits_refuse_bad_counts_and_leave_the_request():
    M = M_()
    rng = np.random.default_rng(12)
    ctx = context(4, 2, 64, "bf16", max_batch=4)
    kv, twin = make_cache(ctx, 4, 4, rng)
    append_both(ctx, kv, twin, [5, 5, 5, 5], rng)
    M.mtp_kv8_commit(ctx, kv, i32([6, -1, 2, 5]))
    twin.commit(2, 2)
    twin.commit(3, 5)
    assert M.mtp_get_device_error(ctx) == M.MTP_ERR_DEVICE_ARGS
    check_cache(ctx, kv, twin)
    M.mtp_kv8_truncate(ctx, kv, i32([5, 6, -1, 4]))
    twin.truncate(0, 5)
    twin.truncate(3, 4)
    assert M.mtp_get_device_error(ctx) == M.MTP_ERR_DEVICE_ARGS
    check_cache(ctx, kv, twin)
    M.mtp_kv8_commit_accepted(ctx, kv, i32([-1, -1, -1, 2 ** 31 - 1]))
    twin.commit(3, 0)
    assert M.mtp_get_device_error(ctx) == M.MTP_ERR_DEVICE_ARGS
    check_cache(ctx, kv, twin)
    with pytest.raises(M.MTPError):
        M.mtp_kv8_commit_accepted(ctx, kv, i32([0] * 4), extra=2)


def test_append_refusals():
    """Bad offsets: nothing happens.  A request that does not fit: it alone is left.  A block id outside the pool."""
    M = M_()
    rng = np.random.default_rng(13)
    ctx = context(4, 2, 64, "bf16", max_batch=3)
    kv, twin = make_cache(ctx, 3, 2, rng)
    k = torch.randn(40, 2, 64, device="cuda").bfloat16()
    for off in ([0, 5, 4, 10], [-1, 2, 3, 4], [0, 1, 2, 41]):
        M.mtp_kv8_append(ctx, kv, k, k, i32(off))
        assert M.mtp_get_device_error(ctx) == M.MTP_ERR_DEVICE_ARGS
        check_cache(ctx, kv, twin)
    M.mtp_kv8_append(ctx, kv, k, k, i32([0, 1, 34, 36]))    # 33 rows into 2 blocks
    assert M.mtp_get_device_error(ctx) == M.MTP_ERR_CAPACITY
    k64 = host(k)
    twin.append(0, k64[:1], k64[:1])
    twin.append(2, k64[34:36], k64[34:36])
    check_cache(ctx, kv, twin)
    kv.block_table[1, 0] = kv.k_pool.shape[0]
    M.mtp_kv8_append(ctx, kv, k, k, i32([0, 0, 20, 20]))
    assert M.mtp_get_device_error(ctx) == M.MTP_ERR_CAPACITY
    assert kv.pending.tolist() == [1, 20, 2] and not kv.arrive.any()
    kv.seq_len[0] = -1
    M.mtp_kv8_append(ctx, kv, k, k, i32([0, 3, 3, 3]))
    assert M.mtp_get_device_error(ctx) == M.MTP_ERR_DEVICE_ARGS
    out = torch.full((8, 2, 64), 3.0, device="cuda").bfloat16()
    M.mtp_kv8_read(ctx, kv, i32([0, 0, 0]), i32([0, 0, 0, 3]), out, out.clone())    # only 2 held
    assert M.mtp_get_device_error(ctx) == M.MTP_ERR_DEVICE_ARGS and bool((out == 3).all())
    with pytest.raises(ValueError):
        M.mtp_kv8_append(ctx, kv, k, k[:39], i32([0, 0, 0, 0]))
    with pytest.raises(ValueError):
        M.mtp_kv8_append(ctx, kv, k.transpose(0, 1).contiguous().transpose(0, 1), k, i32([0, 0, 0, 0]))
    with pytest.raises(M.MTPError):
        M.mtp_kv8_append(ctx, kv, k, k, i32([0, 0, 0, 0]), rope=M.RopeTable(64))      # no positions
    with pytest.raises(M.MTPError):
        M.mtp_kv8_append(ctx, kv, k, k, i32([0, 0, 0, 0]), positions=i32(np.zeros(40)), rope=M.RopeTable(128))


# --------------------------------------------------------------- attention

def filled(ctx, lens, new, rng, max_blocks=None, spare=3, loud=True):
    """A cache of lens[b] committed and new[b] pending entries with random codes (device and host values)."""
    M, c = M_(), ctx.cfg
    B = len(lens)
    total = np.asarray(lens) + np.asarray(new)
    width = max_blocks or max(1, int((total.max() + 15) // 16))
    kv, twin = make_cache(ctx, B, width, rng, spare)
    for w, (pool, scale) in enumerate(((kv.k_pool, kv.k_scale), (kv.v_pool, kv.v_scale))):
        x = V.e4m3_encode(rng.normal(size=twin.codes[w].shape) * 60)
        s = 2.0 ** (rng.integers(-9, -3, twin.scale[w].shape) if loud else rng.integers(-7, -5, twin.scale[w].shape))
        for b in range(B):       # entries that are held, and nothing behind them
            for j in range(width):
                n = int(np.clip(total[b] - 16 * j, 0, 16))
                blk = twin.table[b, j]
                twin.codes[w][blk, :, :n] = x[blk, :, :n]
                twin.scale[w][blk] = s[blk] if n else 0
        pool.copy_(torch.from_numpy(twin.codes[w]))
        scale.copy_(torch.from_numpy(twin.scale[w]))
    twin.seq_len[:], twin.pending[:] = lens, new
    kv.seq_len.copy_(i32(lens))
    kv.pending.copy_(i32(new))
    return kv, twin


def attend(ctx, kv, q, off, max_rows, mask=None, scale=None, ws=None, q_view=None):
    """The call with guarded outputs; rows outside the offsets must stay."""
    from gpu_util import Guarded
    M, c = M_(), ctx.cfg
    T = q.shape[0]
    out = Guarded((T, c.n_q_heads, c.head_dim), q.dtype, fill=77.0)
    lse = Guarded((T, c.n_q_heads), torch.float32, fill=77.0)
    M.mtp_kv8_attention(ctx, kv, q if q_view is None else q_view, i32(off), out.t, ws or M.Attention8Workspace(ctx),
                        max_rows, mask=mask, lse=lse.t, scale=scale)
    torch.cuda.synchronize()
    out.check("out")
    lse.check("lse")
    for r in list(range(0, off[0])) + list(range(off[-1], T)):
        assert bool((out.t[r] == 77).all()) and bool((lse.t[r] == 77).all()), "row %d outside the offsets written" % r
    return host(out.t), host(lse.t)


def compare_attention(ctx, twin, q64, off, got, lse, dtype, words=None, scale=None, requests=None):
    c = ctx.cfg
    scale = c.head_dim ** -0.5 if scale is None else scale
    for b in range(len(off) - 1) if requests is None else requests:
        n = off[b + 1] - off[b]
        if n == 0:
            continue
        L = int(twin.seq_len[b] + twin.pending[b])
        k, v = twin.values(b, 0, L)
        seen = V.causal(n, L) if words is None else V.unpack_mask(words[off[b]:off[b + 1]], n, L)
        o, ls, mass, size = V.attention(q64[off[b]:off[b + 1]], k, v, seen, scale)
        w = 2.0 ** -18 * size + (2.0 ** -10 if dtype == "bf16" else 2.0 ** -18)
        close(got[off[b]:off[b + 1]], o, HALF_STEP[dtype] * np.abs(o) + w[..., None] * mass, "out of request %d" % b)
        close(lse[off[b]:off[b + 1]], ls, 2.0 ** -18 * size + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(ls), ls, 0))), "lse")


def check_attention(ctx, kv, twin, new, rng, dtype, words=None, scale=None, max_rows=None, qsize=1.0):
    c = ctx.cfg
    off = 1 + np.concatenate([[0], np.cumsum(new)])
    q, q64 = normal(rng, (int(off[-1]) + 2, c.n_q_heads, c.head_dim), dtype, qsize)
    got, lse = attend(ctx, kv, q, off, max_rows or max(1, int(max(new))), None if words is None else i32(words), scale)
    clean(ctx)
    compare_attention(ctx, twin, q64, off, got, lse, dtype, words, scale)


LAYOUTS = [("bf16", 32, 8, 128), ("bf16", 8, 2, 64), ("f32", 4, 4, 128), ("f32", 8, 1, 64), ("bf16", 8, 1, 128),
           ("bf16", 2, 2, 64), ("f32", 4, 2, 128)]


@pytest.mark.parametrize("dtype,n_q,n_kv,hd", LAYOUTS)
def test_decode_over_ragged_lengths(dtype, n_q, n_kv, hd):
    rng = np.random.default_rng(n_q * hd)
    ctx = context(n_q, n_kv, hd, dtype, max_batch=9)
    lens = [0, 1, 14, 15, 16, 31, 32, 300, 1025]
    kv, twin = filled(ctx, lens, [1] * 9, rng)
    check_attention(ctx, kv, twin, [1] * 9, rng, dtype)


@pytest.mark.parametrize("dtype,n_q,n_kv,hd", LAYOUTS)
@pytest.mark.parametrize("rows", [2, 6, 9, 33])
def test_verify_rows_are_causal(dtype, n_q, n_kv, hd, rows):
    """Requests of fewer rows than max_rows and of none among them."""
    rng = np.random.default_rng(rows + hd)
    ctx = context(n_q, n_kv, hd, dtype, max_batch=5)
    new = [rows, 1, 0, rows - 1, rows]
    kv, twin = filled(ctx, [0, 15, 40, 130, 513], new, rng)
    check_attention(ctx, kv, twin, new, rng, dtype)


@pytest.mark.parametrize("dtype,n_q,n_kv,hd", [("bf16", 8, 1, 128), ("f32", 4, 2, 64), ("bf16", 4, 4, 64)])
@pytest.mark.parametrize("rows", [101, 256])
def test_many_rows(dtype, n_q, n_kv, hd, rows):
    rng = np.random.default_rng(rows)
    ctx = context(n_q, n_kv, hd, dtype, max_batch=2)
    kv, twin = filled(ctx, [3, 200], [rows, rows - 7], rng)
    check_attention(ctx, kv, twin, [rows, rows - 7], rng, dtype, max_rows=256)


def tree_words(rng, counts, words, blank=()):
    """Ancestor masks of random trees; bits beyond a request's rows set at random (ignored); `blank` rows see nothing."""
    out, at = np.zeros((int(np.sum(counts)), words), np.int64), 0
    for n in counts:
        bits = np.zeros((n, 32 * words), bool)
        for i in range(n):
            up = int(rng.integers(-1, i)) if i else -1
            if up >= 0:
                bits[i, :n] = bits[up, :n]
            bits[i, i] = True
        bits[:, n:] = rng.random((n, 32 * words - n)) < 0.5
        out[at:at + n] = (bits.reshape(n, words, 32) << np.arange(32)).sum(-1)
        at += n
    for r in blank:
        out[r] = 0
    return np.where(out >= 2 ** 31, out - 2 ** 32, out).astype(np.int32)


@pytest.mark.parametrize("dtype,n_q,n_kv,hd", LAYOUTS)
@pytest.mark.parametrize("rows", [3, 32, 61])
def test_tree_masks_and_rows_that_see_nothing(dtype, n_q, n_kv, hd, rows):
    rng = np.random.default_rng(rows)
    ctx = context(n_q, n_kv, hd, dtype, max_batch=4)
    new = [rows, 1, rows - 1, 2]
    kv, twin = filled(ctx, [0, 0, 77, 256], new, rng)
    W = (rows + 31) // 32 + 1
    words = tree_words(rng, new, W, blank=(1, rows))    # a row of request 0 and the only one of request 1
    off = np.concatenate([[0], np.cumsum(new)])
    q, q64 = normal(rng, (int(off[-1]), n_q, hd), dtype)
    got, lse = attend(ctx, kv, q, off, rows, i32(words))
    clean(ctx)
    compare_attention(ctx, twin, q64, off, got, lse, dtype, words)
    for r in (1, rows):
        assert (got[r] == 0).all() and np.isneginf(lse[r]).all()


@pytest.mark.parametrize("dtype,hd", [("bf16", 128), ("f32", 64), ("bf16", 64), ("f32", 128)])
def test_nan_entries_reach_only_rows_that_see_them(dtype, hd):
    """NaN in later rows' keys and values, and in slots behind the last entry (another request's left-overs)."""
    rng = np.random.default_rng(21)
    ctx = context(8, 2, hd, dtype, max_batch=2)
    new = [6, 4]
    kv, twin = filled(ctx, [19, 30], new, rng)
    slots = [(0, 22, 0), (0, 23, 1), (1, 33, 1)]   # (request, slot, K or V): rows 3, 4 of request 0, row 3 of request 1
    for b, s, w in slots:
        (kv.k_pool, kv.v_pool)[w][twin.table[b, s // 16], :, s % 16, 7] = 0x7F
    for w, pool in enumerate((kv.k_pool, kv.v_pool)):
        pool[twin.table[0, 1], :, 25 - 16:] = 0x7F
        pool[twin.table[1, 2], :, 34 - 32:] = 0xFF
    off = np.array([0, 6, 10])
    q, q64 = normal(rng, (10, 8, hd), dtype)
    got, lse = attend(ctx, kv, q, off, 6)
    clean(ctx)
    seen_k = [3, 4, 5]
    for r in range(10):
        if r in seen_k:
            assert np.isnan(got[r]).all() and np.isnan(lse[r]).all()
        elif r == 9:     # a NaN value: its dimension only
            assert np.isnan(got[r, :, 7]).all() and np.isfinite(np.delete(got[r], 7, -1)).all()
    for b, rows in ((0, [0, 1, 2]), (1, [0, 1, 2])):
        L = int(twin.seq_len[b] + twin.pending[b])
        k, v = twin.values(b, 0, L)
        o, ls, mass, size = V.attention(q64[off[b]:off[b + 1]], k, v, V.causal(new[b], L), hd ** -0.5)
        w = 2.0 ** -18 * size + 2.0 ** -10
        g = got[off[b]:off[b + 1]]
        close(g[rows], o[rows], (HALF_STEP[dtype] * np.abs(o) + w[..., None] * mass)[rows], "rows before the NaN")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_of_any_size(dtype):
    """Tiny and huge queries (one key takes all the weight), block scales far apart, a scale of its own."""
    rng = np.random.default_rng(22)
    ctx = context(4, 2, 128, dtype, max_batch=2)
    for qsize in (1e-30, 1e-3, 40.0, 3e4):
        kv, twin = filled(ctx, [200, 77], [2, 1], rng)
        check_attention(ctx, kv, twin, [2, 1], rng, dtype, qsize=qsize)
    for shift in (-40, 40):
        kv, twin = filled(ctx, [200, 77], [2, 1], rng)
        for w, s in ((0, kv.k_scale), (1, kv.v_scale)):
            f = 2.0 ** (rng.integers(-3, 1, twin.scale[w].shape) if w == 0 else rng.integers(min(0, shift), max(1, shift), twin.scale[w].shape))
            twin.scale[w] *= f
            s.copy_(torch.from_numpy(twin.scale[w]))
        check_attention(ctx, kv, twin, [2, 1], rng, dtype, scale=0.03)


def test_attention_refusals():
    M = M_()
    rng = np.random.default_rng(23)
    ctx = context(4, 2, 64, "bf16", max_batch=3)
    kv, twin = filled(ctx, [20, 5, 60], [2, 2, 2], rng)
    q, q64 = normal(rng, (6, 4, 64), "bf16")
    off = np.array([0, 2, 4, 6])
    good, good_lse = attend(ctx, kv, q, off, 2)
    for bad in ([0, 3, 2, 6], [0, 2, 4, 7], [-1, 2, 4, 6]):
        out = torch.full((6, 4, 64), 5.0, device="cuda").bfloat16()
        M.mtp_kv8_attention(ctx, kv, q, i32(bad), out, M.Attention8Workspace(ctx), 3)
        assert M.mtp_get_device_error(ctx) == M.MTP_ERR_DEVICE_ARGS and bool((out == 5).all())
    ws = M.Attention8Workspace(ctx)
    # request 0 has more rows than max_rows; request 1 fewer entries than rows; request 2 longer than its table
    kv.pending[1] = -4
    kv.seq_len[2] = 63
    out = torch.full((6, 4, 64), 5.0, device="cuda").bfloat16()
    M.mtp_kv8_attention(ctx, kv, q, i32([0, 2, 4, 6]), out, ws, 1)
    assert M.mtp_get_device_error(ctx) == M.MTP_ERR_DEVICE_ARGS and bool((out == 5).all())
    M.mtp_kv8_attention(ctx, kv, q, i32([0, 2, 4, 6]), out, ws, 2)
    assert M.mtp_get_device_error(ctx) in (M.MTP_ERR_DEVICE_ARGS, M.MTP_ERR_CAPACITY)
    assert bool((out[2:] == 5).all())
    np.testing.assert_array_equal(host(out[:2]), good[:2])        # the others are served
    # the workspace still serves a good call
    kv.pending[1], kv.seq_len[2] = 2, 60
    got, lse = attend(ctx, kv, q, off, 2, ws=ws)
    np.testing.assert_array_equal(got, good)
    np.testing.assert_array_equal(lse, good_lse)
    clean(ctx)
    # a block id outside the pool counts as zeros: like a block of zero codes
    blk = int(twin.table[2, 1])
    kv.block_table[2, 1] = kv.k_pool.shape[0] + 5
    got, lse = attend(ctx, kv, q, off, 2)
    assert M.mtp_get_device_error(ctx) == M.MTP_ERR_CAPACITY
    for w in range(2):
        twin.codes[w][blk] = 0
    compare_attention(ctx, twin, q64, off, got, lse, "bf16")
    for kw in (dict(max_rows=0), dict(max_rows=257), dict(scale=0.0), dict(scale=float("nan"))):
        with pytest.raises(M.MTPError):
            M.mtp_kv8_attention(ctx, kv, q, i32(off), out, ws, **{"max_rows": 2, **kw})
    with pytest.raises(M.MTPError):      # one word cannot hold 33 rows
        M.mtp_kv8_attention(ctx, kv, q, i32(off), out, ws, 33, mask=i32(np.zeros((6, 1))))


def test_attention_rows_of_a_packed_projection_and_repeated_calls():
    M = M_()
    rng = np.random.default_rng(24)
    for dtype, off0 in (("bf16", 0), ("bf16", 3), ("f32", 1)):
        ctx = context(8, 2, 128, dtype, max_batch=2)
        kv, twin = filled(ctx, [500, 33], [3, 2], rng)
        packed, p64 = normal(rng, (5, off0 + 8 * 128 + 9), dtype)
        view = packed[:, off0:off0 + 1024].unflatten(1, (8, 128))
        off = np.array([0, 3, 5])
        ws = M.Attention8Workspace(ctx)
        first = attend(ctx, kv, view.contiguous(), off, 3, ws=ws)
        for _ in range(3):
            again = attend(ctx, kv, view.contiguous(), off, 3, ws=ws, q_view=view)
            np.testing.assert_array_equal(again[0], first[0])
            np.testing.assert_array_equal(again[1], first[1])
        compare_attention(ctx, twin, p64[:, off0:off0 + 1024].reshape(5, 8, 128), off, *first, dtype)
        clean(ctx)


def test_long_context_and_large_batches():
    """Splits over a long context, and more requests than thread blocks; against float64 on the GPU."""
    M = M_()
    for B, ctxlen, rows, n_q, n_kv, hd, dtype in ((1, 70000, 1, 8, 2, 128, "bf16"), (1, 20000, 5, 8, 2, 64, "f32"),
                                                  (300, 90, 2, 4, 4, 64, "bf16"), (40, 3000, 1, 8, 1, 128, "f32")):
        g = torch.Generator(device="cuda").manual_seed(B + rows)
        ctx = context(n_q, n_kv, hd, dtype, max_batch=B)
        lens = torch.randint(max(1, ctxlen // 2), ctxlen + 1, (B,), generator=g, device="cuda")
        lens[0] = ctxlen
        width = int((ctxlen + rows + 15) // 16)
        table = torch.randperm(B * width, generator=g, device="cuda").view(B, width).int()
        kv = M.KVCache8.empty(ctx, B * width, table)
        for pool, scale in ((kv.k_pool, kv.k_scale), (kv.v_pool, kv.v_scale)):
            pool.copy_((torch.randn(pool.shape, generator=g, device="cuda") * 50).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
            scale.copy_(torch.exp2(torch.randint(-7, -4, scale.shape, generator=g, device="cuda").float()))
        kv.seq_len.copy_(lens)
        kv.pending.fill_(rows)
        q = torch.randn(B * rows, n_q, hd, generator=g, device="cuda").to(TORCH[dtype])
        out, lse = torch.empty_like(q), torch.empty(B * rows, n_q, device="cuda")
        M.mtp_kv8_attention(ctx, kv, q, i32(np.arange(B + 1) * rows), out, M.Attention8Workspace(ctx), rows, lse=lse)
        clean(ctx)
        for b in sorted({0, 1 % B, B // 2, B - 1}):
            L = int(lens[b]) + rows
            at = table[b].long()
            k, v = ((p[at].view(torch.float8_e4m3fn).double() * s[at].double()[..., None, None]).transpose(1, 2).flatten(0, 1)[:L]
                    .repeat_interleave(n_q // n_kv, 1) for p, s in ((kv.k_pool, kv.k_scale), (kv.v_pool, kv.v_scale)))
            qq = q[b * rows:(b + 1) * rows].double()
            z = torch.einsum("rhd,thd->rht", qq, k) * hd ** -0.5
            size = (torch.einsum("rhd,thd->rht", qq.abs(), k.abs()) * hd ** -0.5).amax(-1)
            seen = torch.from_numpy(V.causal(rows, L)).cuda()[:, None]
            z = z.masked_fill(~seen, -float("inf"))
            p = torch.softmax(z, -1)
            want, mass = torch.einsum("rht,thd->rhd", p, v), torch.einsum("rht,thd->rhd", p, v.abs())
            w = 2.0 ** -18 * size + (2.0 ** -10 if dtype == "bf16" else 2.0 ** -18)
            close(host(out[b * rows:(b + 1) * rows]), host(want), host(HALF_STEP[dtype] * want.abs() + w[..., None] * mass), "out")
            close(host(lse[b * rows:(b + 1) * rows]), host(torch.logsumexp(z, -1)), host(2.0 ** -18 * size + 2.0 ** -16), "lse")


def test_pools_beyond_two_gigabytes():
    """Block ids whose byte offsets pass 2^31: append, attention, read, roll-back in the last blocks of a 2.2 GB pool."""
    M = M_()
    rng = np.random.default_rng(31)
    ctx = context(8, 8, 128, "bf16", max_batch=1)
    nb = 140000
    table = np.array([[nb - 1, nb - 2, nb - 3]])
    kv = M.KVCache8.empty(ctx, nb, i32(table))
    twin = V.Cache8(4, 8, 128, [[3, 2, 1]])
    kv.guards = []
    off = append_both(ctx, kv, twin, [40], rng)
    q, q64 = normal(rng, (40, 8, 128), "bf16")
    got, lse = attend(ctx, kv, q, off, 40)
    compare_attention(ctx, twin, q64, off, got, lse, "bf16")
    for w, pool in enumerate((kv.k_pool, kv.v_pool)):
        np.testing.assert_array_equal(pool[nb - 3:].cpu().numpy(), twin.codes[w][1:])
        assert not pool[:nb - 3].any()
    M.mtp_kv8_rollback(ctx, kv)
    assert not kv.k_pool.any() and not kv.v_pool.any() and not kv.k_scale.any()
    clean(ctx)


def test_a_reused_workspace_carries_nothing_over():
    """A call that split its segments, then calls that leave requests (or everything) out, on one workspace."""
    M = M_()
    rng = np.random.default_rng(61)
    ctx = context(8, 2, 128, "bf16", max_batch=3)
    kv, twin = filled(ctx, [2500, 40, 1800], [2, 2, 2], rng)
    ws = M.Attention8Workspace(ctx)
    q, q64 = normal(rng, (6, 8, 128), "bf16")
    off = np.array([0, 2, 4, 6])
    got, lse = attend(ctx, kv, q, off, 2, ws=ws)
    compare_attention(ctx, twin, q64, off, got, lse, "bf16")
    for bad in ([0, 5, 4, 6], [0, 2, 4, 7]):
        out = torch.full((6, 8, 128), 5.0, device="cuda").bfloat16()
        M.mtp_kv8_attention(ctx, kv, q, i32(bad), out, ws, 2)
        assert M.mtp_get_device_error(ctx) == M.MTP_ERR_DEVICE_ARGS and bool((out == 5).all())
    # requests 0 and 2 have no rows this time; request 1's are its last two entries as before
    some = np.array([3, 3, 5, 5])
    got, lse = attend(ctx, kv, q, some, 2, ws=ws)
    compare_attention(ctx, twin, q64, some, got, lse, "bf16")
    kv.pending[2] = -1                      # request 2 is left out, the others are served
    out = torch.full((6, 8, 128), 5.0, device="cuda").bfloat16()
    M.mtp_kv8_attention(ctx, kv, q, i32(off), out, ws, 2)
    assert M.mtp_get_device_error(ctx) == M.MTP_ERR_DEVICE_ARGS
    assert bool((out[4:] == 5).all()) and bool((out[:4] != 5).any(-1).all())


def test_batches_above_the_limit_are_refused():
    M = M_()
    ctx = context(1, 1, 64, "bf16", max_batch=1025)
    kv = M.KVCache8.empty(ctx, 1, i32(np.zeros((1025, 1))))
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(M.MTPError):
        M.mtp_kv8_attention(ctx, kv, q, i32(np.zeros(1026)), torch.empty_like(q), M.Attention8Workspace(ctx), 1)
    clean(ctx)


def test_commit_of_the_pending_counts_themselves():
    """n_keep may be the cache's own pending array (keep everything)."""
    M = M_()
    rng = np.random.default_rng(62)
    ctx = context(8, 8, 64, "bf16", max_batch=3)
    kv, twin = make_cache(ctx, 3, 4, rng)
    for _ in range(3):
        append_both(ctx, kv, twin, [5, 17, 0], rng)
        M.mtp_kv8_commit(ctx, kv, kv.pending)
        for b, n in enumerate([5, 17, 0]):
            twin.commit(b, n)
        check_cache(ctx, kv, twin)
    clean(ctx)


@pytest.mark.parametrize("dtype,hd,layout", [("bf16", 128, "half"), ("f32", 64, "interleaved"), ("bf16", 64, "half")])
@pytest.mark.parametrize("shift", [1, 4])
def test_append_of_unaligned_rows(dtype, hd, layout, shift):
    """k, v and q as slices that start off a 16-byte boundary, against the same values in aligned tensors."""
    M = M_()
    rng = np.random.default_rng(shift + hd)
    ctx = context(4, 2, hd, dtype, max_batch=2)
    off, pos, tab = i32([0, 19, 22]), i32(rng.integers(0, 5000, 22)), M.RopeTable(hd, layout=layout)
    wide, _ = normal(rng, (22, shift + 8 * hd + 3), dtype)
    q, k, v = (wide[:, shift + a * hd:shift + e * hd].unflatten(1, (e - a, hd)) for a, e in ((0, 4), (4, 6), (6, 8)))
    got = []
    for parts in ((q, k, v), tuple(t.contiguous() for t in (q, k, v))):
        kv, _ = make_cache(ctx, 2, 3, np.random.default_rng(1))
        out = torch.empty(22, 4, hd, dtype=TORCH[dtype], device="cuda")
        M.mtp_kv8_append(ctx, kv, parts[1], parts[2], off, q=parts[0], q_out=out, positions=pos, rope=tab)
        got.append((out, kv.k_pool.clone(), kv.v_pool.clone(), kv.k_scale.clone(), kv.v_scale.clone(), kv.pending.clone()))
    clean(ctx)
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_rows_beyond_two_giga_elements():
    """Rotation and logits in the last rows of tensors of more than 2^31 elements."""
    M = M_()
    rng = np.random.default_rng(63)
    ctx = context(2, 2, 128, "bf16")
    wide = torch.zeros(70000, 32768, dtype=torch.bfloat16, device="cuda")
    x = wide[:, -256:].unflatten(1, (2, 128))
    part, p64 = normal(rng, (5, 2, 128), "bf16")
    x[-5:] = part
    pos = np.arange(70000) % 9001
    M.mtp_rope(ctx, x, i32(pos), M.RopeTable(128))
    want = V.rope(p64, pos[-5:])
    close(host(x[-5:]), want, rope_tol(p64, want, "bf16"), "rope")
    assert not wide[:, :-256].any() and not wide[:-5].any()
    del wide, x
    V_ = 151936
    ctx = context(vocab=V_, dtype="bf16", max_batch=1)
    z = torch.zeros(14500, V_, dtype=torch.bfloat16, device="cuda")
    z[-2:, -3:] = 1.0
    M.mtp_logits_process(ctx, z, i32([14498, 14500]), bias_offsets=i32([0, 1]), bias_tokens=i32([V_ - 1]),
                         bias_values=torch.tensor([2.0], device="cuda"))
    assert z[-2:, -3:].tolist() == [[1.0, 1.0, 3.0]] * 2 and not z[:-2].any() and not z[-2:, :-3].any()
    clean(ctx)


# ------------------------------------------------------------------ logits

def logits_case(rng, B, V_, dtype, rows, penalties=True, drafts=True, bias=0, masks=0):
    ctx = context(vocab=V_, dtype=dtype, max_batch=B)
    off = 1 + np.concatenate([[0], np.cumsum(rows)])
    n = int(off[-1]) + 2
    z, z64 = normal(rng, (n, V_), dtype, 4.0)
    kw, ref = {}, dict(off=off)
    if penalties:
        counts = np.where(rng.random((B, V_)) < 0.1, rng.integers(1, 9, (B, V_)), 0)
        counts = counts | np.where(rng.random((B, V_)) < 0.1, -2 ** 31, 0)
        ref["counts"] = counts.astype(np.int32)
        ref["p"] = [(rng.random(B) * 1.5 + 0.4).astype(np.float32), (rng.random(B) - 0.4).astype(np.float32),
                    (rng.random(B) - 0.4).astype(np.float32)]
        kw.update(counts=i32(counts), **{k: torch.from_numpy(x).cuda() for k, x in zip(("repetition", "frequency", "presence"), ref["p"])})
    if drafts:
        w = max(1, max(rows) - 1)
        d = rng.integers(0, V_, (B, w))
        d[:, w // 2] = d[:, 0]          # the same token twice
        if w > 2:
            d[0, 1] = -1                # none
        ref["drafts"] = d
        kw["drafts"] = i32(d)
    if bias:
        per = rng.integers(0, bias + 1, B)
        per[0] = bias
        bo = np.concatenate([[0], np.cumsum(per)])
        bt, bv = rng.integers(0, V_, bo[-1]), rng.normal(size=bo[-1]).astype(np.float32) * 5
        bt[1:bias:3] = bt[0]            # one token named many times
        ref["bias"] = (bo, bt, bv)
        kw.update(bias_offsets=i32(bo), bias_tokens=i32(bt), bias_values=torch.from_numpy(bv).cuda())
    if masks:
        words = rng.integers(-2 ** 31, 2 ** 31, (masks, (V_ + 31) // 32)) & rng.integers(-2 ** 31, 2 ** 31, (masks, (V_ + 31) // 32))
        words[-1] = 0                   # nothing allowed
        mi = rng.integers(-1, masks, n)
        mi[off[0]] = masks - 1
        ref["mask"] = (words, mi)
        kw.update(mask=i32(words), mask_index=i32(mi))
    return ctx, z, z64, kw, ref


def expect_logits(z64, ref, b, j):
    off, V_ = ref["off"], z64.shape[1]
    row = off[b] + j
    p = [float(x[b]) for x in ref["p"]] if "p" in ref else [1.0, 0.0, 0.0]
    counts = ref["counts"][b] if "counts" in ref else np.zeros(V_, np.int32)
    before = ref["drafts"][b, :j] if "drafts" in ref else ()
    bias = ()
    if "bias" in ref:
        bo, bt, bv = ref["bias"]
        bias = [(int(t), float(x)) for t, x in zip(bt[bo[b]:bo[b + 1]], bv[bo[b]:bo[b + 1]])]
    allowed = None
    if "mask" in ref and ref["mask"][1][row] >= 0:
        w = ref["mask"][0][ref["mask"][1][row]].astype(np.int64) & 0xFFFFFFFF
        v = np.arange(V_)
        allowed = (w[v // 32] >> (v % 32) & 1).astype(bool)
    return V.process_logits(z64[row], counts, before, *p, bias, allowed)


def check_logits(ctx, z, z64, kw, ref, dtype):
    from gpu_util import Guarded
    M = M_()
    off = ref["off"]
    out = Guarded(tuple(z.shape), z.dtype, fill=55.0)
    before = z.clone()
    M.mtp_logits_process(ctx, z, i32(off), out.t, **kw)
    clean(ctx)
    out.check("out")
    assert same_bits(z, before)
    assert bool((out.t[:off[0]] == 55).all()) and bool((out.t[off[-1]:] == 55).all())
    got = host(out.t)
    for b in range(len(off) - 1):
        for j in range(off[b + 1] - off[b]):
            want, size = expect_logits(z64, ref, b, j)
            n_bias = len(ref["bias"][1]) if "bias" in ref else 0
            fin = np.isfinite(want)
            tol = np.where(fin, HALF_STEP[dtype] * np.abs(np.where(fin, want, 0)) + (8 + n_bias) * 2.0 ** -24 * size, 0)
            close(got[off[b] + j], want, tol, "logits of request %d, row %d" % (b, j))
    M.mtp_logits_process(ctx, z, i32(off), **kw)         # in place
    assert same_bits(z[off[0]:off[-1]], out.t[off[0]:off[-1]]) and same_bits(z[off[-1]:], before[off[-1]:])
    clean(ctx)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V_,rows,kw", [
    (1, [1], dict()), (7, [2, 1], dict(bias=3, masks=2)), (1000, [6, 1, 0, 3], dict(bias=40, masks=4)),
    (1000, [1, 1], dict(drafts=False)), (1023, [3, 2], dict(masks=3)), (4097, [4, 6], dict(bias=300)),
    (33, [5], dict(bias=100, masks=1)), (5000, [2], dict(penalties=False, drafts=False, bias=10, masks=2)),
    (8192, [9, 9, 9], dict(bias=33, masks=5)), (64, [3], dict(penalties=False, drafts=False))])
def test_logits(dtype, V_, rows, kw):
    rng = np.random.default_rng(V_)
    check_logits(*logits_case(rng, len(rows), V_, dtype, rows, **kw), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logits_that_are_not_finite(dtype):
    """NaN and infinities stay what they are, and masked ones become -inf; a bias of -inf bans a token."""
    M = M_()
    rng = np.random.default_rng(41)
    ctx, z, z64, kw, ref = logits_case(rng, 1, 300, dtype, [2], masks=2)
    for i, x in enumerate((np.nan, np.inf, -np.inf)):
        z[:, i::7] = x
        z64[:, i::7] = x
    check_logits(ctx, z, z64, kw, ref, dtype)
    z = torch.zeros(1, 300, dtype=TORCH[dtype], device="cuda")
    M.mtp_logits_process(ctx, z, i32([0, 1]), bias_offsets=i32([0, 2]), bias_tokens=i32([5, 299]),
                         bias_values=torch.tensor([-float("inf"), 2.0], device="cuda"))
    assert torch.isneginf(z[0, 5]) and z[0, 299] == 2 and int((z != 0).sum()) == 2
    clean(ctx)


def test_logits_refusals():
    M = M_()
    rng = np.random.default_rng(42)
    ctx, z, z64, kw, ref = logits_case(rng, 3, 500, "f32", [2, 2, 2], bias=4, masks=2)
    off = ref["off"]

    def fails(change, bad_requests=(), bad_rows=(), code=None):
        out = torch.full_like(z, 3.0)
        args = {k: (v.clone() if v is not None else None) for k, v in kw.items()}
        change(args)
        o = args.pop("row_offsets", i32(off))
        M.mtp_logits_process(ctx, z, o, out, **args)
        assert M.mtp_get_device_error(ctx) == M.MTP_ERR_DEVICE_ARGS
        for b in bad_requests:
            assert bool((out[off[b]:off[b + 1]] == 3).all()), b
        for r in bad_rows:
            assert bool((out[r] == 3).all()), r
        rest = [b for b in range(3) if b not in bad_requests]
        for b in rest:
            for j in range(2):
                if off[b] + j not in bad_rows:
                    want, size = expect_logits(z64, ref, b, j)
                    fin = np.isfinite(want)
                    close(host(out[off[b] + j]), want, np.where(fin, 2.0 ** -20 * (1 + size), 0), "the others")

    for name, value in (("repetition", 0.0), ("repetition", float("nan")), ("repetition", -1.0), ("frequency", float("inf")),
                        ("presence", float("nan"))):
        fails(lambda a: a[name].__setitem__(1, value), [1])
    fails(lambda a: a["mask_index"].__setitem__(int(off[1]), 2), (), [int(off[1])])
    fails(lambda a: a["mask_index"].__setitem__(int(off[1]), -2), (), [int(off[1])])
    fails(lambda a: a["bias_offsets"].__setitem__(3, 10 ** 6), [2])
    fails(lambda a: a.update(row_offsets=i32([off[0], off[1], off[2], 10 ** 6])), [2])
    # a bias token outside the vocabulary is skipped
    at = int(kw["bias_offsets"][0])
    saved = ref["bias"][1].copy()
    ref["bias"][1][at] = 500
    fails(lambda a: a["bias_tokens"].__setitem__(at, 500))
    ref["bias"][1][:] = saved
    with pytest.raises(M.MTPError):
        M.mtp_logits_process(ctx, z, i32(off), repetition=kw["repetition"])    # no counts
    with pytest.raises(ValueError):
        M.mtp_logits_process(ctx, z[:, :499], i32(off))
    with pytest.raises(ValueError):
        M.mtp_logits_process(ctx, z, i32(off), mask=kw["mask"][:, :-1].contiguous(), mask_index=kw["mask_index"])


def test_token_counts():
    M = M_()
    rng = np.random.default_rng(43)
    V_, B = 700, 3
    ctx = context(vocab=V_, max_batch=B)
    counts = torch.zeros(B, V_, dtype=torch.int32, device="cuda")
    want = np.zeros((B, V_), np.int64)
    for width, n in ((1, [1, 0, 1]), (5000, [5000, 17, 0]), (130, [0, 130, 129])):
        tok = rng.integers(0, V_, (B, width))
        tok[:, 0] = 3                    # a token named by all
        M.mtp_token_counts_add(ctx, counts, i32(tok), i32(n))
        for b in range(B):
            np.add.at(want[b], tok[b, :n[b]], 1)
    M.mtp_token_counts_add(ctx, counts, i32([[5, 5], [6, 0], [0, 0]]), i32([2, 1, 0]), in_prompt=True)
    want[0, 5] -= 2 ** 31
    want[1, 6] -= 2 ** 31
    np.testing.assert_array_equal(counts.cpu().numpy(), want)
    clean(ctx)
    M.mtp_token_counts_add(ctx, counts, i32([[V_, 1], [-1, 2], [3, 4]]), i32([2, 2, 3]))
    assert M.mtp_get_device_error(ctx) == M.MTP_ERR_DEVICE_ARGS
    want[0, 1] += 1
    want[1, 2] += 1
    np.testing.assert_array_equal(counts.cpu().numpy(), want)


# --------------------------------------------------------------- together

class Step:
    """A verifier's step of B requests with K drafts: append, attend, process, verify, commit, count."""

    def __init__(self, B, K, dtype, rng, graph=False):
        M = M_()
        self.B, self.K, self.dtype = B, K, dtype
        self.ctx = context(8, 2, 64, dtype, max_batch=B, vocab=900, max_k=K)
        self.kv, self.twin = make_cache(self.ctx, B, 12, rng)
        T, dt = B * (K + 1), TORCH[dtype]
        self.off = np.arange(B + 1) * (K + 1)
        z = lambda *s, d=dt: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
        self.packed, self.pos = z(T, 12 * 64), z(T, d=torch.int32)
        self.q = self.packed[:, :512].unflatten(1, (8, 64))
        self.k, self.v = (self.packed[:, a:a + 128].unflatten(1, (2, 64)) for a in (512, 640))
        self.q_out, self.out, self.lse = z(T, 8, 64), z(T, 8, 64), z(T, 8, d=torch.float32)
        self.logits, self.done = z(T, 900), z(T, 900)
        self.drafts, self.accepted, self.bonus = (z(B, K, d=torch.int32), z(B, d=torch.int32), z(B, d=torch.int32))
        self.num, self.counts = i32([K] * B), z(B, 900, d=torch.int32)
        self.rep = torch.full((B,), 1.3, device="cuda")
        self.freq = torch.full((B,), 0.5, device="cuda")
        self.offsets, self.ones = i32(self.off), i32([1] * B)
        self.rope, self.ws = M.RopeTable(64), M.Attention8Workspace(self.ctx)

    def run(self):
        M, c = M_(), self.ctx
        M.mtp_kv8_append(c, self.kv, self.k, self.v, self.offsets, q=self.q, q_out=self.q_out, positions=self.pos, rope=self.rope)
        M.mtp_kv8_attention(c, self.kv, self.q_out, self.offsets, self.out, self.ws, self.K + 1, lse=self.lse)
        M.mtp_logits_process(c, self.logits, self.offsets, self.done, counts=self.counts, drafts=self.drafts,
                             repetition=self.rep, frequency=self.freq)
        M.mtp_verify(c, self.done, self.offsets, self.drafts, self.num, self.accepted, self.bonus)
        M.mtp_kv8_commit_accepted(c, self.kv, self.accepted, extra=1)
        M.mtp_token_counts_add(c, self.counts, self.drafts, self.accepted)
        M.mtp_token_counts_add(c, self.counts, self.bonus.view(-1, 1), self.ones)

    def feed(self, rng):
        """New rows: float64 copies, positions, logits and drafts (often what the processed target would say)."""
        self.packed.copy_(torch.from_numpy(rng.normal(size=self.packed.shape)))
        self.logits.copy_(torch.from_numpy(rng.normal(size=self.logits.shape) * 2))
        self.drafts.copy_(i32(rng.integers(0, 900, self.drafts.shape)))
        counts = self.counts.cpu().numpy()
        z = host(self.logits)
        for b in range(self.B):
            for j in range(int(rng.integers(0, self.K + 1))):
                want, _ = V.process_logits(z[self.off[b] + j], counts[b], self.drafts[b, :j].tolist(), 1.3, 0.5)
                self.drafts[b, j] = int(np.argmax(want))
        start = self.twin.seq_len
        self.pos.copy_(i32(np.concatenate([start[b] + np.arange(self.K + 1) for b in range(self.B)])))

    def check(self, rng, counts):
        """One step's results against the oracle; the cache twin takes the same step."""
        p = host(self.packed)
        T = len(p)
        pos = self.pos.cpu().numpy()
        q64, k64 = p[:, :512].reshape(T, 8, 64), V.rope(p[:, 512:640].reshape(T, 2, 64), pos)
        v64 = p[:, 640:].reshape(T, 2, 64)
        want_q = V.rope(q64, pos)
        close(host(self.q_out), want_q, rope_tol(q64, want_q, self.dtype), "q")
        k_codes, v_codes = self.before
        z, drafts = host(self.logits), self.drafts.cpu().numpy()
        acc, bon = self.accepted.cpu().numpy(), self.bonus.cpu().numpy()
        for b in range(self.B):
            self.twin.append(b, k64[self.off[b]:self.off[b + 1]], v64[self.off[b]:self.off[b + 1]])
            rows = [V.process_logits(z[self.off[b] + j], counts[b], drafts[b, :j].tolist(), 1.3, 0.5)[0]
                    for j in range(self.K + 1)]
            # the processed rows are rounded to the type before they are compared: ties there go to the lowest id
            r = [int(np.argmax(torch.from_numpy(x).float().to(TORCH[self.dtype]).float().numpy())) for x in rows]
            a = 0
            while a < self.K and drafts[b, a] == r[a]:
                a += 1
            assert (acc[b], bon[b]) == (a, r[a]), b
            L = int(self.twin.seq_len[b] + self.twin.pending[b])
            k, v = self.twin.values(b, 0, L)
            o, ls, mass, size = V.attention(host(self.q_out)[self.off[b]:self.off[b + 1]], k, v, V.causal(self.K + 1, L), 0.125)
            # keys next to a rounding border may take the other code (a step of 2^-3 of their value): they are few
            err = np.abs(host(self.out)[self.off[b]:self.off[b + 1]] - o)
            w = 2.0 ** -18 * size + 2.0 ** -10
            assert np.mean(err > HALF_STEP[self.dtype] * np.abs(o) + w[..., None] * mass) < 0.05
            self.twin.commit(b, min(a + 1, self.K + 1))
        check_cache(self.ctx, self.kv, self.twin, codes=False)
        clean(self.ctx)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_steps_together(dtype):
    """Five steps as a program would run them, the cache and counts carried along."""
    rng = np.random.default_rng(51)
    s = Step(3, 4, dtype, rng)
    for _ in range(5):
        s.feed(rng)
        counts = s.counts.cpu().numpy()
        s.before = (s.kv.k_pool.clone(), s.kv.v_pool.clone())
        s.run()
        s.check(rng, counts)
    assert int(s.counts.sum()) == int(s.twin.seq_len.sum())     # a token counted for each one emitted


def test_steps_captured_and_replayed():
    """The step in a graph, replayed on new inputs, gives what it gives when called; two graphs, a workspace each."""
    steps = []
    for graph in (False, True):
        rng = np.random.default_rng(52)
        s = Step(2, 3, "bf16", rng)
        if graph:
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=side):
                    s.run()
        got = []
        for _ in range(4):
            s.feed(rng)
            torch.cuda.synchronize()
            g.replay() if graph else s.run()
            torch.cuda.synchronize()
            s.twin.seq_len[:] = s.kv.seq_len.cpu().numpy()
            got.append([t.clone() for t in (s.q_out, s.out, s.lse, s.done, s.accepted, s.bonus, s.kv.k_pool, s.kv.k_scale, s.counts)])
        clean(s.ctx)
        steps.append(got)
    for a, b in zip(*steps):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_two_streams_at_once():
    """Two caches with a workspace each on two streams of one context, against the same calls one after the other."""
    M = M_()
    rng = np.random.default_rng(53)
    ctx = context(8, 2, 128, "bf16", max_batch=4)
    sets = []
    for i in range(2):
        kv, _ = filled(ctx, [3000 + i, 17, 900, 0], [2] * 4, rng)
        q, _ = normal(rng, (8, 8, 128), "bf16")
        sets.append((kv, q, torch.zeros_like(q), M.Attention8Workspace(ctx), i32(np.arange(5) * 2)))
    want = []
    for kv, q, out, ws, off in sets:
        M.mtp_kv8_attention(ctx, kv, q, off, out, ws, 2)
        want.append(out.clone())
        out.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for (kv, q, out, ws, off), st in zip(sets, streams):
            M.mtp_kv8_attention(ctx, kv, q, off, out, ws, 2, stream=st)
    torch.cuda.synchronize()
    for (kv, q, out, ws, off), w in zip(sets, want):
        assert torch.equal(out, w)
    clean(ctx)


# ----------------------------------------------------- limits and bad inputs

def test_path_commit_of_entries_in_blocks_outside_the_pool():
    """A kept entry's own block, or the one it would move to, has no place in the pool: reported, the request left as it
    was.  Where only dropped entries lie in such a block, the path is committed and the block reported."""
    M = M_()
    rng = np.random.default_rng(71)
    ctx = context(4, 2, 64, "bf16", max_batch=5)
    kv, twin = make_cache(ctx, 5, 4, rng)
    append_both(ctx, kv, twin, [12] * 5, rng)
    M.mtp_kv8_commit(ctx, kv, i32([12] * 5))
    for b in range(5):
        twin.commit(b, 12)
    append_both(ctx, kv, twin, [24] * 5, rng)             # slots 12 .. 35: blocks 0, 1, 2
    table = kv.block_table.clone()
    nb = kv.k_pool.shape[0]
    kv.block_table[0, 1] = nb                             # every entry kept
    kv.block_table[1, 2] = -1                             # kept entries come from block 2 only
    kv.block_table[2, 0] = 2 ** 31 - 1                    # entries of block 2 would move into block 0
    kv.block_table[3, 2] = nb + 7                         # block 2 holds dropped entries only
    paths = [list(range(24)), [0, 1, 20, 23], [21, 22], [0, 2, 9], [1, 5, 23]]
    keep = np.zeros((5, 24), np.int64)
    for b, p in enumerate(paths):
        keep[b, :len(p)] = p
    M.mtp_kv8_commit_path(ctx, kv, i32(keep), i32([len(p) for p in paths]))
    assert M.mtp_get_device_error(ctx) == M.MTP_ERR_CAPACITY
    assert kv.seq_len.tolist() == [12, 12, 12, 15, 15] and kv.pending.tolist() == [24, 24, 24, 0, 0]
    assert not kv.arrive.any()
    lost = twin.table[3, 2]
    left = [(w[lost].copy(), s[lost].copy()) for w, s in zip(twin.codes, twin.scale)]
    for b in (3, 4):
        twin.commit(b, len(paths[b]), paths[b])
    for w in range(2):                                    # the block that could not be reached keeps its bytes
        twin.codes[w][lost], twin.scale[w][lost] = left[w]
    check_cache(ctx, kv, twin)
    kv.block_table.copy_(table)
    M.mtp_kv8_commit_path(ctx, kv, i32(keep), i32([24, 4, 2, 0, 0]))
    for b in range(3):
        twin.commit(b, len(paths[b]), paths[b])
    check_cache(ctx, kv, twin)
    clean(ctx)


def test_a_path_commit_that_keeps_everything_reports_a_bad_block():
    M = M_()
    rng = np.random.default_rng(72)
    ctx = context(2, 2, 128, "f32", max_batch=1)
    kv, twin = make_cache(ctx, 1, 2, rng)
    append_both(ctx, kv, twin, [20], rng)
    kv.block_table[0, 1] = -1
    M.mtp_kv8_commit_path(ctx, kv, i32(np.arange(20)[None]), i32([20]))
    assert M.mtp_get_device_error(ctx) == M.MTP_ERR_CAPACITY
    check_cache(ctx, kv, twin)


def test_a_cache_is_checked_again_for_another_context_and_after_a_change():
    """Its device, shapes and layout belong to what was checked; a copy is a cache of its own."""
    import copy
    M = M_()
    rng = np.random.default_rng(73)
    ctx = context(4, 2, 64, "bf16", max_batch=2)
    kv, twin = make_cache(ctx, 2, 6, rng)
    append_both(ctx, kv, twin, [20, 3], rng)
    other = M.Context(0, ctx.cfg, None, device=1)
    other.cfg = ctx.cfg
    with pytest.raises(ValueError):
        kv.struct(other)
    two = copy.deepcopy(kv)
    assert two.k_pool.data_ptr() != kv.k_pool.data_ptr() and two.struct(ctx).k_pool == two.k_pool.data_ptr()
    M.mtp_kv8_rollback(ctx, two)
    assert two.pending.tolist() == [0, 0] and kv.pending.tolist() == [20, 3]
    kept = kv.block_table.clone()
    kv.block_table.resize_(2, 3)
    kv.block_table.copy_(kept[:, :3])
    assert kv.struct(ctx).max_blocks == 3
    append_both(ctx, kv, twin, [5, 5], rng)
    check_cache(ctx, kv, twin)
    kv.block_table.t_()
    with pytest.raises(ValueError):
        kv.struct(ctx)
    kv.block_table.t_()
    kv.arrive.resize_(1)
    with pytest.raises(ValueError):
        kv.struct(ctx)
    kv.arrive.resize_(2)
    kv.struct(ctx)
    clean(ctx)


def test_a_context_keeps_the_configuration_it_was_made_with():
    """Changing the struct for the next context changes nothing about the first."""
    M = M_()
    rng = np.random.default_rng(74)
    cfg = M.make_config(hidden=256, n_q_heads=4, n_kv_heads=2, head_dim=64, ffn=256, vocab=100, dtype="bf16", max_batch=2, max_k=5)
    ctx = M.mtp_init(cfg)
    cfg.head_dim, cfg.n_kv_heads, cfg.vocab = 128, 4, 50
    M.mtp_init(cfg)
    kv, twin = make_cache(ctx, 2, 3, rng)
    assert tuple(kv.k_pool.shape[1:]) == (2, 16, 64)
    append_both(ctx, kv, twin, [20, 3], rng)
    check_cache(ctx, kv, twin)
    counts = torch.zeros(2, 100, dtype=torch.int32, device="cuda")
    M.mtp_token_counts_add(ctx, counts, i32([[99], [0]]), i32([1, 1]))
    assert counts[0, 99] == 1 and int(counts.sum()) == 2
    clean(ctx)


@pytest.mark.parametrize("dtype,n_q,n_kv,hd", [("bf16", 4, 2, 128), ("f32", 4, 2, 128), ("bf16", 8, 1, 64), ("f32", 2, 2, 64)])
@pytest.mark.parametrize("rows", [1, 5])
def test_scores_beyond_the_24_bits_of_a_float(dtype, n_q, n_kv, hd, rows):
    """Scores so large that float32 holds them in steps of many whole units: the result is still a weighted mean of the
    values seen, the entry itself where one leads by more than the scores' own rounding, and lse follows the scores.

    A score is off by 2^-18 S at most (S as above), so an entry that leads the next by 2^-16 S and by 64 units leads
    it by more than 30 units when computed: the others weigh less than e^-30 each, 200 of them below 2^-34.  Its own
    weight is off by 2^-11 where weights are held in 11 bits."""
    rng = np.random.default_rng(rows + hd)
    ctx = context(n_q, n_kv, hd, dtype, max_batch=3)
    new = [rows, 1, rows]
    for qsize in (1e6, 3e6, 1e7, 3e7, 1e8, 3e8, 1e9, 1e12, 1e20, 1e30):
        kv, twin = filled(ctx, [200, 77, 0], new, rng)
        off = np.concatenate([[0], np.cumsum(new)])
        q, q64 = normal(rng, (int(off[-1]), n_q, hd), dtype, qsize)
        got, lse = attend(ctx, kv, q, off, rows)
        clean(ctx)
        sure = 0
        for b in range(3):
            n, L = new[b], int(twin.seq_len[b] + twin.pending[b])
            k, v = twin.values(b, 0, L)
            _, ls, _, size = V.attention(q64[off[b]:off[b + 1]], k, v, V.causal(n, L), hd ** -0.5)
            close(lse[off[b]:off[b + 1]], ls, 2.0 ** -18 * size + 2.0 ** -20 * np.abs(ls), "lse")
            for i in range(n):
                seen = L - n + i + 1
                for h in range(n_q):
                    g, o = h // (n_q // n_kv), got[off[b] + i, h]
                    lo, hi = v[:seen, g].min(0), v[:seen, g].max(0)
                    # a mean in float32, and the type's half step
                    room = (2.0 ** -9 + HALF_STEP[dtype]) * np.abs(v[:seen, g]).max()
                    assert np.all(o >= lo - room) and np.all(o <= hi + room), (qsize, b, i, h)
                    z = np.sort(hd ** -0.5 * (k[:seen, g] @ q64[off[b] + i, h]))[::-1]
                    if seen == 1 or z[0] - z[1] > 2.0 ** -16 * size[i, h] + 64:
                        top = int(np.argmax(k[:seen, g] @ q64[off[b] + i, h]))
                        w = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -20
                        room = (HALF_STEP[dtype] + w) * np.abs(v[top, g]) + 2.0 ** -20 * np.abs(v[:seen, g]).max()
                        assert np.all(np.abs(o - v[top, g]) <= room), (qsize, b, i, h)
                        sure += 1
        assert sure >= sum(new) * n_q * 3 // 4


@pytest.mark.parametrize("dtype,hd,rows", [("bf16", 128, 1), ("f32", 128, 1), ("bf16", 64, 6), ("f32", 64, 3)])
def test_close_scores_far_from_zero(dtype, hd, rows):
    """Every key has the same large product with the query and one of its own within 28 units: what float32 keeps of the
    difference decides, the result is a weighted mean of the values seen and lse follows the scores."""
    rng = np.random.default_rng(rows)
    ctx = context(8, 2, hd, dtype, max_batch=2)
    new, off = [rows, rows], np.array([0, rows, 2 * rows])
    for e in range(18, 36):
        kv, twin = filled(ctx, [150, 40], new, rng)
        held = twin.scale[0] > 0
        twin.codes[0][:] = 0
        twin.codes[0][held, :, 0] = V.e4m3_encode(1.0)
        twin.codes[0][held, :, 1] = V.e4m3_encode(rng.uniform(-28, 28, (int(held.sum()), 16)))
        twin.scale[0][held] = 1.0
        for b, L in ((0, 150 + rows), (1, 40 + rows)):      # nothing behind the last entry
            if L % 16:
                twin.codes[0][twin.table[b, L // 16], :, L % 16:] = 0
        kv.k_pool.copy_(torch.from_numpy(twin.codes[0]))
        kv.k_scale.copy_(torch.from_numpy(twin.scale[0]))
        q64 = np.zeros((2 * rows, 8, hd))
        q64[..., 0] = 2.0 ** e * rng.integers(128, 256, (2 * rows, 8)) / 128 * rng.choice([-1, 1], (2 * rows, 8))
        q64[..., 1] = 1.0
        got, lse = attend(ctx, kv, torch.from_numpy(q64).to(TORCH[dtype]).cuda(), off, rows, scale=1.0)
        clean(ctx)
        for b in range(2):
            L = int(twin.seq_len[b] + twin.pending[b])
            k, v = twin.values(b, 0, L)
            _, ls, _, size = V.attention(q64[off[b]:off[b + 1]], k, v, V.causal(rows, L), 1.0)
            close(lse[off[b]:off[b + 1]], ls, 2.0 ** -18 * size + 2.0 ** -20 * np.abs(ls), "lse")
            for i in range(rows):
                seen = v[:L - rows + i + 1].repeat(4, 1)
                room = (2.0 ** -9 + HALF_STEP[dtype]) * np.abs(seen).max((0, 2))[:, None]
                o = got[off[b] + i]
                assert np.all(o >= seen.min(0) - room) and np.all(o <= seen.max(0) + room), (e, b, i)


def test_logits_with_drafts_of_no_width():
    """No drafts (K = 0): one row a request; a second row has no draft to follow and is refused."""
    M = M_()
    rng = np.random.default_rng(75)
    ctx, z, z64, kw, ref = logits_case(rng, 2, 300, "f32", [1, 1], drafts=False)
    none = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    want = M.mtp_logits_process(ctx, z, i32(ref["off"]), torch.full_like(z, 3.0), **kw)
    got = M.mtp_logits_process(ctx, z, i32(ref["off"]), torch.full_like(z, 3.0), drafts=none, **kw)
    clean(ctx)
    assert torch.equal(got, want)
    out = torch.full_like(z, 3.0)
    M.mtp_logits_process(ctx, z, i32([0, 2, 3]), out, drafts=none, **kw)
    assert M.mtp_get_device_error(ctx) == M.MTP_ERR_DEVICE_ARGS
    assert bool((out[:2] == 3).all()) and bool((out[2] != 3).any())
    M.mtp_logits_process(ctx, z, i32([0, 2, 3]), out, drafts=none)         # nothing is counted: no penalties
    clean(ctx)
    assert torch.equal(out[:3], z[:3])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_appended_keys_and_the_attention_over_them(dtype):
    """Append and attend step by step: every code is the oracle's or the next one, and the attention over the codes that
    the cache holds is within its own tolerance, with no exceptions; then the draft rows are committed as accepted."""
    M = M_()
    rng = np.random.default_rng(76)
    ctx = context(8, 2, 64, dtype, max_batch=3)
    kv, twin = make_cache(ctx, 3, 8, rng)
    tab, ws = M.RopeTable(64), M.Attention8Workspace(ctx)
    for step in range(5):
        new = [5, 5, int(rng.integers(1, 6))]
        off = np.concatenate([[0], np.cumsum(new)])
        T = int(off[-1])
        (q, q64), (k, k64), (v, v64) = (normal(rng, (T, n, 64), dtype) for n in (8, 2, 2))
        pos = np.concatenate([twin.seq_len[b] + np.arange(new[b]) for b in range(3)])
        q_out = torch.empty_like(q)
        M.mtp_kv8_append(ctx, kv, k, v, i32(off), q=q, q_out=q_out, positions=i32(pos), rope=tab)
        got, lse = attend(ctx, kv, q_out, off, 5, ws=ws)
        clean(ctx)
        want_k = V.rope(k64, pos)
        for b in range(3):
            start = int(twin.seq_len[b])
            twin.append(b, want_k[off[b]:off[b + 1]], v64[off[b]:off[b + 1]])
            for slot in range(start, start + new[b]):
                blk, s = twin.table[b, slot // 16], slot % 16
                for w, (pool, scale) in enumerate(((kv.k_pool, kv.k_scale), (kv.v_pool, kv.v_scale))):
                    ds, os_ = scale[blk].double().cpu().numpy()[:, None], twin.scale[w][blk][:, None]
                    dv, ov = V.VALUES[pool[blk, :, s].cpu().numpy()] * ds, V.VALUES[twin.codes[w][blk, :, s]] * os_
                    if w:
                        np.testing.assert_array_equal(dv, ov)
                    else:
                        assert np.all(np.abs(dv - ov) <= np.maximum(2.0 ** -3 * np.maximum(np.abs(dv), np.abs(ov)),
                                                                    2.0 ** -9 * np.maximum(ds, os_)))
            for blk in twin.table[b, start // 16:(start + new[b] + 15) // 16]:
                for w, (pool, scale) in enumerate(((kv.k_pool, kv.k_scale), (kv.v_pool, kv.v_scale))):
                    twin.codes[w][blk], twin.scale[w][blk] = pool[blk].cpu().numpy(), scale[blk].double().cpu().numpy()
        compare_attention(ctx, twin, host(q_out), off, got, lse, dtype)
        acc = rng.integers(0, 5, 3)
        M.mtp_kv8_commit_accepted(ctx, kv, i32(acc), extra=1)
        for b in range(3):
            twin.commit(b, min(int(acc[b]) + 1, new[b]))
        check_cache(ctx, kv, twin)
    clean(ctx)


def test_entries_below_bf16_are_read_back_rounded():
    """Scales of 2^-124 and more: every entry exactly.  2^-126 and 2^-125: the smallest codes lie below bf16's smallest
    number and are rounded to it."""
    M = M_()
    rng = np.random.default_rng(77)
    ctx = context(2, 2, 64, "f32", max_batch=4)
    kv, twin = make_cache(ctx, 4, 1, rng)
    top = np.array([448.0 * 2.0 ** -126, 448.0 * 2.0 ** -125, 448.0 * 2.0 ** -124, 1.0])
    rows = np.repeat(top, 16)[:, None, None] * 2.0 ** rng.uniform(-22, 0, (64, 2, 64)) * rng.choice([-1, 1], (64, 2, 64))
    rows[::16, :, 0] = top[:, None]
    t = torch.from_numpy(rows).float()
    M.mtp_kv8_append(ctx, kv, t.cuda(), t.cuda(), i32(np.arange(5) * 16))
    for b in range(4):
        twin.append(b, t[16 * b:16 * b + 16].double().numpy(), t[16 * b:16 * b + 16].double().numpy())
    check_cache(ctx, kv, twin)
    out = [torch.empty(64, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    M.mtp_kv8_read(ctx, kv, i32([0] * 4), i32(np.arange(5) * 16), *out)
    clean(ctx)
    for b in range(4):
        assert (twin.scale[0][twin.table[b, 0]] == (top[b] / 448 if b < 3 else 2.0 ** -8)).all()
        for got, want in zip(out, twin.values(b, 0, 16)):
            assert torch.equal(got[16 * b:16 * b + 16].cpu(), torch.from_numpy(want).float().bfloat16())
            if b >= 2:
                np.testing.assert_array_equal(host(got[16 * b:16 * b + 16]), want)


@pytest.mark.parametrize("dtype,hd", [("bf16", 128), ("f32", 64)])
def test_path_commit_of_the_most_entries(dtype, hd):
    """256 pending entries, all kept or every second one; 257 are refused."""
    M = M_()
    rng = np.random.default_rng(78)
    ctx = context(2, 2, hd, dtype, max_batch=3)
    kv, twin = make_cache(ctx, 3, 18, rng)
    append_both(ctx, kv, twin, [7, 16, 0], rng, 8.0)
    M.mtp_kv8_commit(ctx, kv, kv.pending)
    for b, n in enumerate([7, 16, 0]):
        twin.commit(b, n)
    for n in (100, 156):
        append_both(ctx, kv, twin, [n, n, n + n // 156], rng, 1.0 + n)
    keep = np.zeros((3, 256), np.int64)
    keep[0], keep[1, :128] = np.arange(256), np.arange(1, 256, 2)
    M.mtp_kv8_commit_path(ctx, kv, i32(keep), i32([256, 128, 1]))
    twin.commit(0, 256, keep[0])
    twin.commit(1, 128, keep[1, :128])
    assert M.mtp_get_device_error(ctx) == M.MTP_ERR_DEVICE_ARGS
    check_cache(ctx, kv, twin)


def test_attention_of_the_most_requests():
    """1024 requests of 0 to 2 rows, each with a length of its own."""
    rng = np.random.default_rng(79)
    ctx = context(4, 2, 64, "bf16", max_batch=1024)
    new = rng.integers(0, 3, 1024)
    kv, twin = filled(ctx, rng.integers(0, 70, 1024), new, rng)
    check_attention(ctx, kv, twin, new, rng, "bf16")
