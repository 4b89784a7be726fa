"""GPU parity of the operators on the paged cache in the context's type:
norms with rotation, append, attention of new rows, the attention weight that
entries gather, and eviction by it, against the float64 oracle
(oracle/paged.py, oracle/verifier.py).

Tolerances.  A result stored in a type t is off by at most eps(t) / 2 of its
value from what was computed (bf16 2^-8, float32 2^-24).  What was computed is
off from the exact value by float32 rounding:
  norm      a sum of head_dim squares in float32 (relative 2^-18 for 128 terms,
            any order), halved by the root, the root itself and two products:
            2^-18 of the normed value, which is at most the row's largest;
  rotation  2^-19 of the row's largest (two products and a sum of factors that
            are good to 2^-22);
  scores    a sum of head_dim products in float32, any order, of operands taken
            as they are: 2^-18 S, S = scale * max_t sum_d |q_d k_d|; a weight is
            then off by twice that (with the rounding of its exponent), plus
            2^-20 for the exponential, plus 2^-8 where weights are rounded to
            bf16 for the product with the values;
  outputs   so a sum of weighted values is off by that times sum_t p_t |v_t|
            (`mass`), of which the normalising sum takes as much again.
"""
import numpy as np
import pytest
import torch

from oracle import paged as P
from oracle import verifier as V
from test_gpu_verifier import HALF_STEP, M_, TORCH, clean, close, context, host, i32, normal, same_bits

pytestmark = pytest.mark.gpu


def view_bits(x):
    return x.contiguous().view(torch.int16 if x.element_size() == 2 else torch.int32)


def make_cache(ctx, B, max_blocks, rng, spare=3):
    """An empty device cache with a shuffled table and guard blocks around the pools, and the oracle's twin."""
    M, c = M_(), ctx.cfg
    nb = B * max_blocks + spare
    table = rng.permutation(nb)[:B * max_blocks].reshape(B, max_blocks)
    kv = M.KVCache.empty(ctx, nb, i32(table))
    kv.guards = []
    for name in ("k_pool", "v_pool"):
        wide = torch.full((nb + 2, c.n_kv_heads, 16, c.head_dim), 7.0, dtype=ctx.dtype, device="cuda")
        wide[1:-1] = 0
        setattr(kv, name, wide[1:-1])
        kv.guards.append(wide)
    return kv, P.Cache(nb, c.n_kv_heads, c.head_dim, table)


def check_cache(kv, twin, tol=None):
    """Lengths, guards and every slot of the pools; tol: of the keys (None: exact)."""
    for w in kv.guards:
        assert bool((w[0] == 7).all()) and bool((w[-1] == 7).all()), "a block around a pool overwritten"
    np.testing.assert_array_equal(kv.seq_len.cpu().numpy(), twin.seq_len)
    np.testing.assert_array_equal(kv.pending.cpu().numpy(), twin.pending)
    assert not kv.arrive.any()
    if tol is None:
        np.testing.assert_array_equal(host(kv.k_pool), twin.pools[0])
    np.testing.assert_array_equal(host(kv.v_pool), twin.pools[1])


def dtype_of(ctx):
    return "bf16" if ctx.cfg.dtype else "f32"


def append_both(ctx, kv, twin, counts, rng, scale=1.0, first=0, extra=0):
    """Append counts[b] rows to each request on both sides, as they are: exact."""
    M, c = M_(), ctx.cfg
    T = first + int(np.sum(counts)) + extra
    off = first + np.concatenate([[0], np.cumsum(counts)])
    k, k64 = normal(rng, (T, c.n_kv_heads, c.head_dim), dtype_of(ctx), scale)
    v, v64 = normal(rng, (T, c.n_kv_heads, c.head_dim), dtype_of(ctx))
    M.mtp_kv_append(ctx, kv, k, v, i32(off))
    for b in range(len(counts)):
        twin.append(b, k64[off[b]:off[b + 1]], v64[off[b]:off[b + 1]])
    return off


def filled(ctx, lens, new, rng, scale=1.0):
    """A cache with lens[b] committed entries and new[b] pending ones."""
    width = max(1, (max(a + n for a, n in zip(lens, new)) + 15) // 16)
    kv, twin = make_cache(ctx, len(lens), width, rng)
    append_both(ctx, kv, twin, lens, rng, scale)
    M_().mtp_kv_commit(ctx, kv, i32(lens))
    for b, n in enumerate(lens):
        twin.commit(b, n)
    if sum(new):
        append_both(ctx, kv, twin, new, rng, scale)
    return kv, twin


# ------------------------------------------------------- norms and rotation

def turned(x64, w64, eps, pos, rd, layout):
    y = P.norm(x64, w64, eps)
    return y if rd is None else V.rope(y, pos, layout, rd)


def norm_tol(want, y64, dtype):
    return HALF_STEP[dtype] * np.abs(want) + 2.0 ** -17 * np.abs(y64).max(-1, keepdims=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,n_q,n_kv,hd,rd,layout,weights", [
    (1, 8, 2, 64, 64, "half", "qk"), (1, 32, 8, 128, 128, "half", "qk"), (37, 4, 4, 128, 128, "interleaved", "qk"),
    (300, 8, 1, 64, 2, "half", "k"), (19, 2, 2, 64, 62, "half", "q"), (33, 8, 2, 128, 96, "half", "qk"),
    (65, 1, 1, 128, 34, "interleaved", "qk"), (1025, 16, 4, 64, 48, "interleaved", ""), (130, 8, 8, 128, None, "half", "qk"),
    (2000, 32, 8, 128, 64, "half", "qk")])
def test_norm_and_rotation(dtype, T, n_q, n_kv, hd, rd, layout, weights):
    M = M_()
    rng = np.random.default_rng(T + hd)
    ctx = context(n_q, n_kv, hd, dtype)
    q, q64 = normal(rng, (T, n_q, hd), dtype, 3.0)
    k, k64 = normal(rng, (T, n_kv, hd), dtype, 0.1)
    if T > 4:
        q[1], q64[1] = 0.0, 0.0                              # the norm of nothing
        k[2, 0], k64[2, 0] = 1e-4, k[2, 0].new_tensor(1e-4).double().item()   # eps counts
    qw, qw64 = normal(rng, (hd,), dtype)
    kw, kw64 = normal(rng, (hd,), dtype)
    pos = rng.integers(-2 ** 20, 2 ** 20, T)
    tab = None if rd is None else M.RopeTable(rd, layout=layout)
    before = q.clone(), k.clone()
    out = [torch.full_like(x, 9.0) for x in (q, k)]
    kw_args = dict(q_weight=qw if "q" in weights else None, k_weight=kw if "k" in weights else None, eps=1e-6,
                   positions=i32(pos), rope=tab)
    assert M.mtp_qk_norm_rope(ctx, q, k, q_out=out[0], k_out=out[1], **kw_args) == (out[0], out[1])
    assert torch.equal(q, before[0]) and torch.equal(k, before[1])
    for got, x64, w64, name in ((out[0], q64, qw64, "q"), (out[1], k64, kw64, "k")):
        w64 = w64 if name in weights else None
        close(host(got), turned(x64, w64, 1e-6, pos, rd, layout),
              norm_tol(turned(x64, w64, 1e-6, pos, rd, layout), P.norm(x64, w64, 1e-6), dtype), name)
    # one side alone, then both in place: the same bits
    alone = torch.full_like(k, 9.0)
    if rd is not None or "k" in weights:
        M.mtp_qk_norm_rope(ctx, None, k, k_weight=kw_args["k_weight"], positions=i32(pos), rope=tab, k_out=alone)
        assert same_bits(alone, out[1])
    M.mtp_qk_norm_rope(ctx, q, k, **kw_args)
    assert same_bits(q, out[0]) and same_bits(k, out[1])
    clean(ctx)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout,rd", [("half", 64), ("interleaved", 40)])
@pytest.mark.parametrize("off", [0, 1, 8])
def test_norm_of_a_packed_projections_slices(dtype, layout, rd, off):
    """q and k of one wide tensor, at an offset that leaves rows unaligned: the bits of aligned copies; what lies around stays."""
    M = M_()
    rng = np.random.default_rng(off)
    ctx = context(4, 2, 64, dtype)
    wide, _ = normal(rng, (21, off + 8 * 64 + 5), dtype)
    before = wide.clone()
    q, k = (wide[:, off + a * 64:off + b * 64].unflatten(1, (b - a, 64)) for a, b in ((0, 4), (4, 6)))
    w, _ = normal(rng, (64,), dtype)
    tab = M.RopeTable(rd, layout=layout)
    pos = i32(rng.integers(0, 100000, 21))
    want = M.mtp_qk_norm_rope(ctx, q.contiguous(), k.contiguous(), w, w, positions=pos, rope=tab)
    M.mtp_qk_norm_rope(ctx, q, k, w, w, positions=pos, rope=tab)
    # (the sum of squares adds the same elements in another order where pairs are loaded one by one)
    tol = 2.0 ** -17 * 8 + HALF_STEP[dtype] * 2 * host(want[0]).__abs__()
    close(host(q), host(want[0]), tol, "q")
    close(host(k), host(want[1]), 2.0 ** -17 * 8 + HALF_STEP[dtype] * 2 * host(want[1]).__abs__(), "k")
    assert torch.equal(wide[:, :off], before[:, :off]) and torch.equal(wide[:, off + 6 * 64:], before[:, off + 6 * 64:])
    clean(ctx)


def test_norm_refusals():
    M = M_()
    ctx = context(4, 2, 64, "bf16")
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    w, pos, tab = torch.ones(64, dtype=torch.bfloat16, device="cuda"), i32([0, 1, 2]), M.RopeTable(64)
    for kw, err in ((dict(q=None, k=None), ValueError), (dict(q_weight=None, k_weight=None, rope=None), M.MTPError),
                    (dict(positions=None), M.MTPError), (dict(positions=i32([0, 1])), ValueError),
                    (dict(rope=M.RopeTable(128)), M.MTPError), (dict(eps=0.0), M.MTPError), (dict(eps=float("nan")), M.MTPError),
                    (dict(q_weight=w.float()), ValueError), (dict(q_weight=w[:32]), ValueError), (dict(q=q.float()), ValueError),
                    (dict(k=k[:2]), ValueError), (dict(q=q.cpu()), ValueError), (dict(q=q.transpose(0, 1)), ValueError),
                    (dict(q=None), ValueError), (dict(q_out=k), ValueError)):
        args = dict(q=q, k=k, q_weight=w, k_weight=w, positions=pos, rope=tab)
        args.update(kw)
        with pytest.raises(err):
            M.mtp_qk_norm_rope(ctx, args.pop("q"), args.pop("k"), **args)
    M.mtp_qk_norm_rope(ctx, q[:0], k[:0], w, w, positions=pos[:0], rope=tab)
    clean(ctx)


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("dtype,n_q,n_kv,hd", [("bf16", 8, 2, 64), ("f32", 4, 4, 128), ("bf16", 8, 1, 128),
                                               ("f32", 2, 2, 64), ("bf16", 32, 8, 128)])
def test_append_and_edits_are_exact(dtype, n_q, n_kv, hd):
    """Lengths of one, of a whole block, across blocks, and none; rows in front of the first and behind the last."""
    M = M_()
    rng = np.random.default_rng(hd + n_q)
    ctx = context(n_q, n_kv, hd, dtype, max_batch=4)
    kv, twin = make_cache(ctx, 4, 6, rng)
    for counts in ([1, 16, 37, 0], [1, 0, 3, 17], [14, 1, 1, 1]):
        append_both(ctx, kv, twin, counts, rng, first=2, extra=3)
        check_cache(kv, twin)
    M.mtp_kv_commit(ctx, kv, i32([16, 3, 0, 18]))
    for b, n in enumerate([16, 3, 0, 18]):
        twin.commit(b, n)
    check_cache(kv, twin)
    append_both(ctx, kv, twin, [40, 6, 7, 8], rng)
    M.mtp_kv_rollback(ctx, kv)
    for b in range(4):
        twin.commit(b, 0)
    append_both(ctx, kv, twin, [5, 5, 5, 5], rng)
    check_cache(kv, twin)
    clean(ctx)


def test_append_to_more_requests_than_fit_the_gpu():
    ctx = context(8, 8, 64, "bf16", max_batch=900)
    rng = np.random.default_rng(11)
    kv, twin = make_cache(ctx, 900, 2, rng)
    for _ in range(4):
        append_both(ctx, kv, twin, [7] * 900, rng)
        check_cache(kv, twin)
    clean(ctx)


@pytest.mark.parametrize("dtype,n_q,n_kv,hd,rd,layout", [
    ("bf16", 8, 2, 64, 64, "half"), ("f32", 4, 4, 128, 128, "half"), ("bf16", 32, 8, 128, 128, "interleaved"),
    ("bf16", 4, 4, 128, 62, "half"), ("f32", 8, 1, 64, 6, "interleaved"), ("bf16", 16, 4, 128, None, "half")])
@pytest.mark.parametrize("shift", [0, 3])
def test_append_norms_and_rotates(dtype, n_q, n_kv, hd, rd, layout, shift):
    """k, v and q of one packed projection: what mtp_qk_norm_rope gives for the same rows, bit for bit."""
    M = M_()
    rng = np.random.default_rng(hd + shift)
    ctx = context(n_q, n_kv, hd, dtype, max_batch=3)
    kv, twin = make_cache(ctx, 3, 5, rng)
    append_both(ctx, kv, twin, [3, 0, 20], rng)
    M.mtp_kv_commit(ctx, kv, i32([3, 0, 20]))
    for b, n in enumerate([3, 0, 20]):
        twin.commit(b, n)
    counts = np.array([30, 1, 5])
    off = np.concatenate([[0], np.cumsum(counts)])
    T = int(off[-1])
    packed, _ = normal(rng, (T, shift + (n_q + 2 * n_kv) * hd), dtype)
    q, k, v = (packed[:, shift + a * hd:shift + e * hd].unflatten(1, (e - a, hd))
               for a, e in ((0, n_q), (n_q, n_q + n_kv), (n_q + n_kv, n_q + 2 * n_kv)))
    qw, kw = (normal(rng, (hd,), dtype)[0] for _ in range(2))
    pos, tab = i32(rng.integers(0, 200000, T)), None if rd is None else M.RopeTable(rd, layout=layout)
    want = M.mtp_qk_norm_rope(ctx, q, k, qw, kw, positions=pos, rope=tab, q_out=q.contiguous(), k_out=k.contiguous())
    # (the reference rows are strided as the appended ones are, so both take the same path)
    got = torch.full((T, n_q, hd), 9.0, dtype=TORCH[dtype], device="cuda")
    M.mtp_kv_append(ctx, kv, k, v, i32(off), q=q, q_out=got, positions=pos, rope=tab, q_weight=qw, k_weight=kw)
    clean(ctx)
    assert same_bits(got, want[0])
    for b in range(3):
        twin.append(b, host(want[1])[off[b]:off[b + 1]], host(v)[off[b]:off[b + 1]])
    check_cache(kv, twin)
    # a decoding step of the same context: q in place, no norms
    if rd is not None:
        M.mtp_kv_commit(ctx, kv, kv.pending.clone())
        one = i32([0, 1, 2, 3])
        kk = k[:3].contiguous()
        want_k = M.mtp_qk_norm_rope(ctx, None, kk, positions=pos[:3], rope=tab, k_out=torch.empty_like(kk))[1]
        qq = q[:3].contiguous()
        want_q = M.mtp_qk_norm_rope(ctx, qq, None, positions=pos[:3], rope=tab, q_out=torch.empty_like(qq))[0]
        M.mtp_kv_append(ctx, kv, kk, v[:3].contiguous(), one, q=qq, positions=pos[:3], rope=tab)
        assert same_bits(qq, want_q)
        for b in range(3):
            twin.commit(b, int(counts[b]))
            twin.append(b, host(want_k)[b:b + 1], host(v)[b:b + 1])
        check_cache(kv, twin)
    M.mtp_kv_append(ctx, kv, k[:0], v[:0], i32([0, 0, 0, 0]))   # nothing to append
    check_cache(kv, twin)
    clean(ctx)


def test_append_refusals():
    """Bad offsets: nothing happens.  A request that does not fit: it alone is left.  A block id outside the pool."""
    M = M_()
    rng = np.random.default_rng(13)
    ctx = context(4, 2, 64, "bf16", max_batch=4)
    kv, twin = make_cache(ctx, 4, 2, rng)
    append_both(ctx, kv, twin, [3, 4, 5, 30], rng)
    k, _ = normal(rng, (12, 2, 64), "bf16")
    for off in ([0, 3, 2, 6, 9], [-1, 3, 5, 6, 9], [0, 3, 5, 6, 13]):
        M.mtp_kv_append(ctx, kv, k, k, i32(off))
        assert M.mtp_get_device_error(ctx) == M.MTP_ERR_DEVICE_ARGS
        check_cache(kv, twin)
    off = [0, 3, 6, 9, 12]                                    # the last one has room for two
    M.mtp_kv_append(ctx, kv, k, k, i32(off))
    assert M.mtp_get_device_error(ctx) == M.MTP_ERR_CAPACITY
    for b in range(3):
        twin.append(b, host(k)[off[b]:off[b + 1]], host(k)[off[b]:off[b + 1]])
    check_cache(kv, twin)
    kv.seq_len[1] = -1
    M.mtp_kv_append(ctx, kv, k[:1], k[:1], i32([0, 0, 1, 1, 1]))
    assert M.mtp_get_device_error(ctx) == M.MTP_ERR_DEVICE_ARGS
    kv.seq_len[1] = 0
    check_cache(kv, twin)
    for bad in (-1, kv.k_pool.shape[0]):
        kv.block_table[0, 0] = bad                            # its next row lies in that block
        before = kv.k_pool.clone()
        M.mtp_kv_append(ctx, kv, k[:1], k[:1], i32([0, 1, 1, 1, 1]))
        assert M.mtp_get_device_error(ctx) == M.MTP_ERR_CAPACITY
        assert torch.equal(kv.k_pool, before)
    bare = M.KVCache(kv.k_pool, kv.v_pool, kv.block_table, kv.seq_len, kv.pending)
    for args, kw, err in (((ctx, bare, k, k, i32(off)), {}, ValueError), ((ctx, kv, k, k[:3], i32(off)), {}, ValueError),
                          ((ctx, kv, k, k, i32(off[:4])), {}, ValueError), ((ctx, kv, k.float(), k, i32(off)), {}, ValueError),
                          ((ctx, kv, k, k, i32(off)), dict(q_weight=k[0, 0]), ValueError),
                          ((ctx, kv, k, k, i32(off)), dict(rope=M.RopeTable(64)), M.MTPError),
                          ((ctx, kv, k, k, i32(off)), dict(q=torch.zeros(12, 4, 64, dtype=torch.bfloat16, device="cuda")), M.MTPError),
                          ((ctx, kv, k, k, i32(off)), dict(k_weight=k[0, 0].contiguous(), eps=-1.0), M.MTPError)):
        with pytest.raises(err):
            M.mtp_kv_append(*args, **kw)
    clean(ctx)


# --------------------------------------------------------------- attention

def attend(ctx, kv, q, off, max_rows, **kw):
    M = M_()
    out, lse = torch.full_like(q, 5.0).contiguous(), torch.full(q.shape[:2], 5.0, device="cuda")
    ws = kw.pop("ws", None) or M.AttentionWorkspace(ctx)
    M.mtp_kv_attention(ctx, kv, q, i32(off), out, ws, max_rows, lse=lse, **kw)
    return out, lse


def out_tol(want, mass, size, dtype):
    per = 2.0 ** -18 + 2.0 ** -17 * size[..., None] + (2.0 ** -8 if dtype == "bf16" else 0.0)
    return HALF_STEP[dtype] * np.abs(want) + 2 * per * mass


def check_attention(ctx, kv, twin, new, rng, mask=None, max_rows=None, qscale=1.0, scale=None, extra=0):
    c = ctx.cfg
    dtype = dtype_of(ctx)
    T = int(np.sum(new)) + extra
    off = np.concatenate([[0], np.cumsum(new)])
    q, q64 = normal(rng, (T, c.n_q_heads, c.head_dim), dtype, qscale)
    out, lse = attend(ctx, kv, q, off, max_rows or max(new), mask=None if mask is None else i32(mask), scale=scale)
    clean(ctx)
    sc = c.head_dim ** -0.5 if scale is None else scale
    for b, n in enumerate(new):
        if n == 0:
            continue
        L = twin.length(b)
        k, v = twin.values(b)
        seen = P.seen_of(n, L, None if mask is None else mask[off[b]:off[b + 1]])
        want, wl, mass, size = V.attention(q64[off[b]:off[b + 1]], k, v, seen, sc)
        close(host(out)[off[b]:off[b + 1]], want, out_tol(want, mass, size, dtype), "out of request %d" % b)
        close(host(lse)[off[b]:off[b + 1]], wl, 2.0 ** -20 + 2.0 ** -17 * size + 2.0 ** -22 * np.abs(np.nan_to_num(wl, neginf=0)), "lse")
    if extra:
        assert bool((out[off[-1]:] == 5).all()) and bool((lse[off[-1]:] == 5).all()), "rows behind the last one written"
    return q, out, lse


SHAPES = [("bf16", 8, 2, 64), ("bf16", 4, 4, 128), ("bf16", 8, 1, 128), ("bf16", 4, 2, 64), ("f32", 4, 2, 64),
          ("f32", 2, 2, 128), ("f32", 8, 1, 128)]


@pytest.mark.parametrize("dtype,n_q,n_kv,hd", SHAPES)
def test_decode_over_ragged_lengths(dtype, n_q, n_kv, hd):
    rng = np.random.default_rng(n_q * hd)
    ctx = context(n_q, n_kv, hd, dtype, max_batch=11)
    lens = [0, 1, 14, 15, 16, 31, 32, 127, 128, 300, 1025]
    kv, twin = filled(ctx, lens, [1] * len(lens), rng)
    check_attention(ctx, kv, twin, [1] * len(lens), rng, extra=2)


@pytest.mark.parametrize("dtype,n_q,n_kv,hd", SHAPES)
@pytest.mark.parametrize("rows", [2, 17, 64])
def test_new_rows_are_causal(dtype, n_q, n_kv, hd, rows):
    """Requests of fewer rows than max_rows, of one and of none among them."""
    rng = np.random.default_rng(rows + hd)
    ctx = context(n_q, n_kv, hd, dtype, max_batch=5)
    new = [rows, 1, 0, max(1, rows - 3), rows // 2 + 1]
    kv, twin = filled(ctx, [0, 33, 5, 130, 16], new, rng)
    check_attention(ctx, kv, twin, new, rng, extra=1)


@pytest.mark.parametrize("dtype,n_q,n_kv,hd", [("bf16", 8, 2, 128), ("bf16", 2, 2, 64), ("f32", 4, 2, 64)])
def test_a_chunk_of_a_prompt(dtype, n_q, n_kv, hd):
    """More rows than a tile holds, an odd number of them, behind and without earlier entries; decoding rows beside."""
    rng = np.random.default_rng(hd)
    ctx = context(n_q, n_kv, hd, dtype, max_batch=3)
    new = [333, 1, 290]
    kv, twin = filled(ctx, [0, 200, 75], new, rng)
    check_attention(ctx, kv, twin, new, rng, max_rows=1000)


def tree_words(rng, new, rows):
    """Random ancestors; some rows see nothing of the new entries, bits behind a request's rows are set."""
    words = (rows + 31) // 32
    out = np.zeros((int(np.sum(new)), words), np.int64)
    at = 0
    for n in new:
        for i in range(n):
            bits = rng.random(words * 32) < 0.3
            bits[i] = True
            if i % 5 == 3:
                bits[:n] = False
            out[at + i] = [int(sum(1 << j for j in range(32) if bits[32 * w + j])) for w in range(words)]
        at += n
    return np.where(out >= 2 ** 31, out - 2 ** 32, out)


@pytest.mark.parametrize("dtype,n_q,n_kv,hd", SHAPES)
@pytest.mark.parametrize("rows", [6, 33, 61])
def test_tree_masks_and_rows_that_see_nothing(dtype, n_q, n_kv, hd, rows):
    rng = np.random.default_rng(rows)
    ctx = context(n_q, n_kv, hd, dtype, max_batch=4)
    new = [rows, 1, rows - 1, 4]
    kv, twin = filled(ctx, [0, 130, 21, 0], new, rng)
    mask = tree_words(rng, new, rows)
    _, out, lse = check_attention(ctx, kv, twin, new, rng, mask=mask)
    assert bool((out[3] == 0).all()) and bool(torch.isneginf(lse[3]).all())   # nothing before it, nothing of its own


@pytest.mark.parametrize("dtype,n_q,n_kv,hd,rows", [("bf16", 8, 2, 128, 9), ("bf16", 4, 2, 64, 70), ("f32", 8, 2, 64, 9),
                                                    ("bf16", 8, 2, 128, 200)])
def test_entries_that_are_not_finite_reach_only_rows_that_see_them(dtype, n_q, n_kv, hd, rows):
    """NaN and infinities in the later rows' keys and values, and in slots behind the last entry of a block."""
    M = M_()
    rng = np.random.default_rng(21)
    ctx = context(n_q, n_kv, hd, dtype, max_batch=2)
    kv, twin = filled(ctx, [20, 3], [rows, 5], rng)
    q, q64 = normal(rng, (rows + 5, n_q, hd), dtype)
    off = [0, rows, rows + 5]
    ws = M.AttentionWorkspace(ctx)
    want, want_lse = attend(ctx, kv, q, off, rows, ws=ws)
    # behind the last entries: whatever lies there
    for b in range(2):
        L = twin.length(b)
        if L % 16:
            blk = int(twin.table[b, L // 16])
            kv.k_pool[blk, :, L % 16:] = float("nan")
            kv.v_pool[blk, :, L % 16:] = float("inf")
    got, lse = attend(ctx, kv, q, off, rows, ws=ws)
    assert same_bits(got, want) and same_bits(lse, want_lse)
    # row 5 of the first request and later ones see the entry; row 4 does not
    slot = 20 + 5
    blk = int(twin.table[0, slot // 16])
    kv.v_pool[blk, 0, slot % 16, 3] = float("nan")
    kv.v_pool[blk, 0, slot % 16, 7] = float("inf")
    got, lse = attend(ctx, kv, q, off, rows, ws=ws)
    assert same_bits(lse, want_lse)
    G = n_q // n_kv
    assert same_bits(got[:5], want[:5]) and same_bits(got[rows:], want[rows:]) and same_bits(got[:, G:], want[:, G:])
    assert bool(torch.isnan(got[5:rows, :G, 3]).all()) and not bool(torch.isfinite(got[5:rows, :G, 7]).any())
    rest = [d for d in range(hd) if d not in (3, 7)]
    assert same_bits(got[5:rows, :G][..., rest], want[5:rows, :G][..., rest])
    kv.v_pool[blk, 0, slot % 16] = 0
    kv.k_pool[blk, 0, slot % 16, 0] = float("nan")
    got, lse = attend(ctx, kv, q, off, rows, ws=ws)
    assert same_bits(got[:5], want[:5]) and same_bits(lse[:5], want_lse[:5]) and same_bits(got[:, G:], want[:, G:])
    assert bool(torch.isnan(got[5:rows, :G]).all()) and bool(torch.isnan(lse[5:rows, :G]).all())
    clean(ctx)


@pytest.mark.parametrize("dtype,rows", [("bf16", 4), ("f32", 4), ("bf16", 100)])
def test_scores_of_any_size(dtype, rows):
    """Tiny and huge queries (one key takes all the weight), and a scale of its own."""
    rng = np.random.default_rng(22)
    ctx = context(4, 2, 128, dtype, max_batch=2)
    kv, twin = filled(ctx, [90, 10], [rows, rows], rng)
    for qscale, scale in ((1e-20, None), (30.0, None), (1.0, 3.5), (1.0, 1e-6)):
        check_attention(ctx, kv, twin, [rows, rows], rng, qscale=qscale, scale=scale)


@pytest.mark.parametrize("dtype,rows", [("bf16", 4), ("f32", 4), ("bf16", 100)])
def test_scores_far_beyond_the_24_bits_of_a_float(dtype, rows):
    """Scores of 2^20 to 2^100: the result is a weighted mean of values seen, and lse follows the largest score."""
    M = M_()
    rng = np.random.default_rng(23)
    ctx = context(4, 2, 64, dtype, max_batch=1)
    kv, twin = filled(ctx, [150], [rows], rng)
    k, v = twin.values(0)
    for e in (20, 29, 31, 33, 60, 100):
        q, q64 = normal(rng, (rows, 4, 64), dtype, 2.0 ** (e / 2))
        out, lse = attend(ctx, kv, q, [0, rows], rows, scale=2.0 ** (e / 2 - 3))
        assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
        seen = P.seen_of(rows, 150 + rows)
        for i in range(rows):
            for h in range(4):
                z = 2.0 ** (e / 2 - 3) * (k[:, h // 2] @ q64[i, h])
                z[~seen[i]] = -np.inf
                order = np.argsort(z)
                size = 2.0 ** (e / 2 - 3) * (np.abs(k[:, h // 2]) @ np.abs(q64[i, h])).max()
                assert abs(float(lse[i, h]) - z[order[-1]]) <= 2.0 ** -17 * size + 10
                if z[order[-1]] - z[order[-2]] > 2.0 ** -16 * size + 40:      # one key takes all the weight
                    want = v[order[-1], h // 2]
                    close(host(out)[i, h], want, 2 * HALF_STEP[dtype] * np.abs(want) + 2.0 ** -20, "out")
    clean(ctx)


def exact_on_gpu(q, kv, b, lo, hi, scale, G):
    """float64 attention of one request on the GPU, (out, lse, mass, size)."""
    n, L = hi - lo, int(kv.seq_len[b] + kv.pending[b])
    row = kv.block_table[b, :(L + 15) // 16].long()
    k, v = (p[row].transpose(1, 2).flatten(0, 1)[:L].double() for p in (kv.k_pool, kv.v_pool))
    see = torch.ones((n, L), dtype=torch.bool, device="cuda").tril(L - n)
    got = [[], [], [], []]
    for h in range(q.shape[1]):
        x = q[lo:hi, h].double()
        z = (x @ k[:, h // G].T * scale).masked_fill(~see, -float("inf"))
        p = torch.softmax(z, -1)
        got[0].append(p @ v[:, h // G])
        got[1].append(torch.logsumexp(z, -1))
        got[2].append(p @ v[:, h // G].abs())
        got[3].append((x.abs() @ k[:, h // G].abs().T * scale).amax(-1))
    return [torch.stack(x, 1).cpu().numpy() for x in got]


@pytest.mark.parametrize("lens,new,n_q,n_kv,hd,dtype", [
    ([70000], [1], 8, 2, 128, "bf16"), ([20000], [5], 8, 2, 64, "f32"), ([0], [4096], 8, 2, 128, "bf16"),
    ([5000], [1500], 8, 1, 128, "bf16"), ([3, 9000, 50, 700], [700, 1, 33, 1024], 8, 2, 64, "bf16"),
    ([777] * 300, [1] * 300, 4, 4, 128, "bf16"), ([100, 4000], [900, 300], 2, 2, 128, "bf16"),
    ([100, 1300], [400, 300], 4, 2, 128, "f32"), ([40] * 200, [3] * 200, 4, 4, 64, "bf16"),
    ([1] * 1024, [2] * 1024, 2, 1, 64, "bf16")])
def test_long_contexts_and_large_batches(lens, new, n_q, n_kv, hd, dtype):
    """Splits over a long context, tiles over many rows, more segments than thread blocks; against float64 on the GPU."""
    M = M_()
    rng = np.random.default_rng(len(lens))
    B = len(lens)
    ctx = context(n_q, n_kv, hd, dtype, max_batch=B)
    need = [(a + n + 15) // 16 for a, n in zip(lens, new)]
    nb, width = sum(need), max(need)
    table, perm, at = np.zeros((B, width), np.int64), rng.permutation(nb), 0
    for b in range(B):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
    kv = M.KVCache.empty(ctx, nb, i32(table))
    g = torch.Generator(device="cuda").manual_seed(B)
    for pool in (kv.k_pool, kv.v_pool):     # (slots behind the last entries hold numbers too: nothing reads them)
        pool.copy_(torch.randn(pool.shape, generator=g, device="cuda"))
    kv.seq_len.copy_(i32(lens)), kv.pending.copy_(i32(new))
    off = np.concatenate([[0], np.cumsum(new)])
    q = torch.randn((int(off[-1]), n_q, hd), generator=g, device="cuda").to(TORCH[dtype])
    out, lse = attend(ctx, kv, q, off, max(new))
    clean(ctx)
    for b in (range(B) if B < 10 else list(range(0, B, B // 7)) + [B - 1]):
        want, wl, mass, size = exact_on_gpu(q, kv, b, off[b], off[b + 1], hd ** -0.5, n_q // n_kv)
        close(host(out[off[b]:off[b + 1]]), want, out_tol(want, mass, size, dtype), "out of request %d" % b)
        close(host(lse[off[b]:off[b + 1]]), wl, 2.0 ** -20 + 2.0 ** -17 * size + 2.0 ** -22 * np.abs(wl), "lse")
    # the same call again: the same bits
    again, lse2 = attend(ctx, kv, q, off, max(new))
    assert same_bits(again, out) and same_bits(lse2, lse)


def test_attention_of_a_packed_projection_and_repeated_calls():
    M = M_()
    rng = np.random.default_rng(24)
    for dtype, off0, rows in (("bf16", 0, 40), ("bf16", 3, 40), ("f32", 1, 9), ("bf16", 3, 2)):
        ctx = context(8, 2, 128, dtype, max_batch=2)
        kv, twin = filled(ctx, [100, 7], [rows, rows], rng)
        packed, _ = normal(rng, (2 * rows, off0 + 12 * 128), dtype)
        q = packed[:, off0:off0 + 8 * 128].unflatten(1, (8, 128))
        ws = M.AttentionWorkspace(ctx)
        ws.ws.fill_(0xA5)
        want = attend(ctx, kv, q.contiguous(), [0, rows, 2 * rows], rows)
        for _ in range(3):
            got = attend(ctx, kv, q, [0, rows, 2 * rows], rows, ws=ws)
            assert same_bits(got[0], want[0]) and same_bits(got[1], want[1])
        clean(ctx)


def test_attention_refusals():
    M = M_()
    rng = np.random.default_rng(23)
    ctx = context(4, 2, 64, "bf16", max_batch=3)
    kv, twin = filled(ctx, [5, 40, 3], [2, 2, 2], rng)
    q, _ = normal(rng, (6, 4, 64), "bf16")
    ws = M.AttentionWorkspace(ctx)
    off = [0, 2, 4, 6]
    want, want_lse = attend(ctx, kv, q, off, 2, ws=ws)
    for bad in ([0, 2, 1, 6], [0, 2, 4, 7], [-1, 2, 4, 6]):
        out, lse = attend(ctx, kv, q, bad, 6, ws=ws)
        assert M.mtp_get_device_error(ctx) == M.MTP_ERR_DEVICE_ARGS
        assert bool((out == 5).all()) and bool((lse == 5).all())
    for change, error in ((lambda: kv.pending.__setitem__(1, 100), M.MTP_ERR_CAPACITY),
                          (lambda: kv.seq_len.__setitem__(1, -1), M.MTP_ERR_DEVICE_ARGS),
                          (lambda: kv.seq_len.__setitem__(1, 2 ** 31 - 1), M.MTP_ERR_CAPACITY)):
        keep = kv.seq_len.clone(), kv.pending.clone()
        change()
        out, lse = attend(ctx, kv, q, off, 2, ws=ws)
        assert M.mtp_get_device_error(ctx) == error
        assert bool((out[2:4] == 5).all()) and bool((lse[2:4] == 5).all())
        assert same_bits(out[:2], want[:2]) and same_bits(out[4:], want[4:])
        kv.seq_len.copy_(keep[0]), kv.pending.copy_(keep[1])
    out, _ = attend(ctx, kv, q, [0, 3, 4, 6], 2, ws=ws)          # more rows than max_rows
    assert M.mtp_get_device_error(ctx) == M.MTP_ERR_DEVICE_ARGS
    assert bool((out[:3] == 5).all()) and bool((out[3:] != 5).any())
    # a block id outside the pool: reported, its entries count as zeros
    for bad in (-1, kv.k_pool.shape[0]):
        blk = int(kv.block_table[1, 1])
        kept = kv.k_pool[blk].clone(), kv.v_pool[blk].clone()
        kv.k_pool[blk], kv.v_pool[blk] = 0, 0
        zeros = attend(ctx, kv, q, off, 2, ws=ws)
        kv.k_pool[blk], kv.v_pool[blk] = kept
        kv.block_table[1, 1] = bad
        got = attend(ctx, kv, q, off, 2, ws=ws)
        assert M.mtp_get_device_error(ctx) == M.MTP_ERR_CAPACITY
        assert same_bits(got[0], zeros[0]) and same_bits(got[1], zeros[1])
        kv.block_table[1, 1] = blk
    out = torch.empty_like(q)
    mask = i32(np.zeros((6, 1)))
    for kw, err in ((dict(max_rows=0), M.MTPError), (dict(mask=mask, max_rows=257), M.MTPError), (dict(mask=mask, max_rows=33), M.MTPError),
                    (dict(scale=0.0), M.MTPError), (dict(scale=float("nan")), M.MTPError), (dict(mask=mask[:3]), ValueError),
                    (dict(lse=torch.empty(6, 4, device="cuda", dtype=torch.bfloat16)), ValueError)):
        with pytest.raises(err):
            M.mtp_kv_attention(ctx, kv, q, i32(off), out, ws, **{**dict(max_rows=2), **kw})
    with pytest.raises(ValueError):
        M.mtp_kv_attention(ctx, kv, q, i32(off), out[:3], ws, 2)
    with pytest.raises(ValueError):
        M.mtp_kv_attention(context(4, 2, 128, "bf16"), kv, q, i32(off), out, ws, 2)
    big = context(1, 1, 64, "bf16", max_batch=1025)
    with pytest.raises(M.MTPError):
        M.mtp_kv_attention(big, M.KVCache.empty(big, 1, i32(np.zeros((1025, 1)))), q[:, :1], i32(np.zeros(1026)), out[:, :1].contiguous(),
                           M.AttentionWorkspace(big), 1)
    M.mtp_kv_attention(ctx, kv, q[:0], i32([0, 0, 0, 0]), out[:0], ws, 1)
    clean(ctx)


def test_pools_beyond_two_gigabytes():
    """Block ids whose byte offsets pass 2^31: append, attention, weights, eviction in the last blocks of a pool."""
    M = M_()
    rng = np.random.default_rng(31)
    ctx = context(8, 8, 128, "bf16", max_batch=1)
    nb = 2 ** 31 // (8 * 16 * 128 * 2) + 600
    table = np.array([[nb - 1, 3, nb - 300, nb - 2]])
    kv = M.KVCache.empty(ctx, nb, i32(table))
    kv.guards = []
    twin = P.Cache(8, 8, 128, np.array([[0, 1, 2, 3]]))
    append_both(ctx, kv, twin, [50], rng)
    check_attention(ctx, kv, twin, [50], rng)
    for w in range(2):
        pool = (kv.k_pool, kv.v_pool)[w]
        np.testing.assert_array_equal(host(pool[torch.as_tensor(table[0]).cuda()]), twin.pools[w][:4])
    weights = torch.zeros((nb, 8, 16), device="cuda")
    q, _ = normal(rng, (1, 8, 128), "bf16")
    lse = attend(ctx, kv, q, [0, 1], 1)[1]
    M.mtp_kv_attention_weights(ctx, kv, q, i32([0, 1]), lse, weights, 1, first=i32([0]))
    close(host(weights.sum((0, 2))), np.ones(8), 1e-5, "sum of weights")
    M.mtp_kv_commit(ctx, kv, kv.pending.clone())
    to = M.KVCache(kv.k_pool, kv.v_pool, i32([[nb - 400, nb - 401]]), i32([0]), i32([0]))
    kept = torch.empty((1, 8, 20), dtype=torch.int32, device="cuda")
    M.mtp_kv_evict(ctx, kv, weights, i32([20]), to, None, kept)
    clean(ctx)
    k = twin.values(0)[0]
    for g in range(8):
        at = kept[0, g].cpu().numpy()
        np.testing.assert_array_equal(host(kv.k_pool[nb - 400, g]), k[at[:16], g])
        np.testing.assert_array_equal(host(kv.k_pool[nb - 401, g, :4]), k[at[16:], g])


# ----------------------------------------------------------------- weights

def check_weights(ctx, kv, twin, new, rng, mask=None, first=None, max_rows=None, rows=None, qscale=1.0):
    """Weights from random earlier ones; rows (None: new): how many of each request's last rows weigh."""
    M, c = M_(), ctx.cfg
    dtype = dtype_of(ctx)
    rows = new if rows is None else rows
    off = np.concatenate([[0], np.cumsum(rows)])
    q, q64 = normal(rng, (int(off[-1]), c.n_q_heads, c.head_dim), dtype, qscale)
    mk = None if mask is None else i32(mask)
    lse = attend(ctx, kv, q, off, max_rows or max(rows), mask=mk)[1]
    before = torch.rand((kv.k_pool.shape[0], c.n_kv_heads, 16), device="cuda")
    got = before.clone()
    M.mtp_kv_attention_weights(ctx, kv, q, i32(off), lse, got, max_rows or max(rows), mask=mk,
                               first=None if first is None else i32(first))
    clean(ctx)
    want, tol = host(before), np.zeros(before.shape)
    for b, n in enumerate(rows):
        L = twin.length(b)
        if n == 0:
            continue
        k = twin.values(b)[0]
        add, size = P.gathered(q64[off[b]:off[b + 1]], k, host(lse)[off[b]:off[b + 1]],
                               P.seen_of(n, L, None if mask is None else mask[off[b]:off[b + 1]]), c.head_dim ** -0.5)
        for t in range(L):
            at = twin.table[b, t // 16], slice(None), t % 16
            if t >= (L - n if first is None else first[b]):
                want[at] = 0
            want[at] += add[t]
            # the exponent's rounding is relative to lse too (at most 100 here); sums of at most 4096 terms
            tol[at] = 2.0 ** -17 * size[t] + 2.0 ** -16 * add[t] + 2.0 ** -23 * want[at] + 1e-30
    close(host(got), want, tol, "weights")
    again = before.clone()
    M.mtp_kv_attention_weights(ctx, kv, q, i32(off), lse, again, max_rows or max(rows), mask=mk,
                               first=None if first is None else i32(first))
    assert same_bits(again, got)
    return got


@pytest.mark.parametrize("dtype,n_q,n_kv,hd", SHAPES)
def test_weights_of_decoding_rows(dtype, n_q, n_kv, hd):
    rng = np.random.default_rng(hd)
    ctx = context(n_q, n_kv, hd, dtype, max_batch=8)
    lens = [0, 1, 15, 16, 127, 128, 300, 700]
    kv, twin = filled(ctx, lens, [1] * 8, rng)
    check_weights(ctx, kv, twin, [1] * 8, rng)


@pytest.mark.parametrize("dtype,n_q,n_kv,hd", SHAPES)
@pytest.mark.parametrize("rows", [3, 40, 150])
def test_weights_of_chunks(dtype, n_q, n_kv, hd, rows):
    """All rows of a chunk, entries that start anew from a slot of their own, and the last rows alone."""
    rng = np.random.default_rng(rows)
    ctx = context(n_q, n_kv, hd, dtype, max_batch=4)
    new = [rows, 1, 0, rows - 1]
    lens = [0, 60, 9, 131]
    kv, twin = filled(ctx, lens, new, rng)
    check_weights(ctx, kv, twin, new, rng, max_rows=rows + 5)
    check_weights(ctx, kv, twin, new, rng, first=[0, 70, 0, 100])
    check_weights(ctx, kv, twin, new, rng, rows=[2, 1, 0, 1], first=lens)


@pytest.mark.parametrize("dtype,n_q,n_kv,hd", [("bf16", 8, 2, 128), ("bf16", 4, 4, 64), ("f32", 4, 2, 64)])
def test_weights_under_tree_masks(dtype, n_q, n_kv, hd):
    rng = np.random.default_rng(6)
    ctx = context(n_q, n_kv, hd, dtype, max_batch=4)
    new = [33, 1, 32, 4]
    kv, twin = filled(ctx, [0, 130, 21, 0], new, rng)
    check_weights(ctx, kv, twin, new, rng, mask=tree_words(rng, new, 33))


def test_weights_sum_to_the_rows_heads():
    """Over all entries of a kv head, n rows' weights sum to n times its group."""
    M = M_()
    rng = np.random.default_rng(7)
    for dtype in ("bf16", "f32"):
        ctx = context(8, 2, 128, dtype, max_batch=1)
        kv, twin = filled(ctx, [500], [300], rng)
        q, _ = normal(rng, (300, 8, 128), dtype)
        lse = attend(ctx, kv, q, [0, 300], 300)[1]
        w = torch.full((kv.k_pool.shape[0], 2, 16), float("nan"), device="cuda")
        M.mtp_kv_attention_weights(ctx, kv, q, i32([0, 300]), lse, w, 300, first=i32([0]))
        total = w[kv.block_table[0].long()].transpose(1, 2).flatten(0, 1)[:800].double().sum(0).cpu().numpy()
        close(total, np.full(2, 1200.0), np.full(2, 1200 * 2.0 ** -15), "sum")
        assert bool(torch.isnan(w[kv.block_table[0].long()].transpose(1, 2).flatten(0, 1)[800:]).all())
        clean(ctx)


def test_weights_ignore_what_rows_do_not_see():
    """Keys that are not finite behind the rows, rows of no weight, and entries without one."""
    M = M_()
    rng = np.random.default_rng(8)
    for dtype, rows in (("bf16", 30), ("f32", 30), ("bf16", 3)):
        ctx = context(4, 2, 64, dtype, max_batch=1)
        kv, twin = filled(ctx, [21], [rows], rng)
        q, _ = normal(rng, (rows, 4, 64), dtype)
        lse = attend(ctx, kv, q, [0, rows], rows)[1]
        lse[1] = -float("inf")
        w = torch.zeros((kv.k_pool.shape[0], 2, 16), device="cuda")
        M.mtp_kv_attention_weights(ctx, kv, q, i32([0, rows]), lse, w, rows)
        L = 21 + rows
        blk, at = int(twin.table[0, (L - 1) // 16]), (L - 1) % 16
        if at < 15:
            kv.k_pool[int(twin.table[0, L // 16]), :, at + 1:] = float("nan")
        kv.k_pool[blk, 0, at] = float("nan")       # the last row alone sees it
        got = torch.zeros_like(w)
        M.mtp_kv_attention_weights(ctx, kv, q, i32([0, rows]), lse, got, rows)
        assert bool(torch.isnan(got[blk, 0, at]))
        got[blk, 0, at] = w[blk, 0, at]
        assert same_bits(got, w)
        clean(ctx)


def test_weights_refusals():
    M = M_()
    rng = np.random.default_rng(9)
    ctx = context(4, 2, 64, "bf16", max_batch=2)
    kv, twin = filled(ctx, [5, 40], [2, 2], rng)
    q, _ = normal(rng, (4, 4, 64), "bf16")
    lse = attend(ctx, kv, q, [0, 2, 4], 2)[1]
    w = torch.full((kv.k_pool.shape[0], 2, 16), 2.0, device="cuda")
    for bad in ([0, 2, 1], [0, 2, 5], [-1, 2, 4]):
        M.mtp_kv_attention_weights(ctx, kv, q, i32(bad), lse, w, 4)
        assert M.mtp_get_device_error(ctx) == M.MTP_ERR_DEVICE_ARGS and bool((w == 2).all())
    M.mtp_kv_attention_weights(ctx, kv, q, i32([0, 2, 4]), lse, w, 1)
    assert M.mtp_get_device_error(ctx) == M.MTP_ERR_DEVICE_ARGS and bool((w == 2).all())
    M.mtp_kv_attention_weights(ctx, kv, q, i32([0, 2, 4]), lse, w, 2, first=i32([-1, 0]))
    assert M.mtp_get_device_error(ctx) == M.MTP_ERR_DEVICE_ARGS
    assert bool((w[kv.block_table[0].long()] == 2).all()) and bool((w[kv.block_table[1].long()] != 2).any())
    for args, kw, err in (((ctx, kv, q, i32([0, 2, 4]), lse[:2], w, 2), {}, ValueError),
                          ((ctx, kv, q, i32([0, 2, 4]), lse, w[:1], 2), {}, ValueError),
                          ((ctx, kv, q, i32([0, 2, 4]), lse, w.double(), 2), {}, ValueError),
                          ((ctx, kv, q, i32([0, 2, 4]), lse, w, 0), {}, M.MTPError),
                          ((ctx, kv, q, i32([0, 2, 4]), lse, w, 2), dict(first=i32([0])), ValueError),
                          ((ctx, kv, q, i32([0, 2, 4]), lse, w, 2), dict(scale=-1.0), M.MTPError)):
        with pytest.raises(err):
            M.mtp_kv_attention_weights(*args, **kw)
    clean(ctx)


# ---------------------------------------------------------------- eviction

def check_evict(ctx, lens, budgets, rng, sink=0, recent=0, weights=None, width=None, share_pool=False):
    """Entries that name themselves (request, slot, head), weights given or with many equal ones."""
    M, c = M_(), ctx.cfg
    B, n_kv, hd = len(lens), int(c.n_kv_heads), int(c.head_dim)
    src_w, dst_w = max(1, (max(lens) + 15) // 16), max(1, (max(budgets) + 15) // 16)
    nb = B * (src_w + dst_w) + 2
    perm = rng.permutation(nb)
    table, to_table = perm[:B * src_w].reshape(B, src_w), perm[B * src_w:B * (src_w + dst_w)].reshape(B, dst_w)
    kv = M.KVCache.empty(ctx, nb, i32(table))
    if share_pool:
        to = M.KVCache(kv.k_pool, kv.v_pool, i32(to_table), i32(np.full(B, 77)), i32(np.full(B, 3)))
    else:
        to = M.KVCache.empty(ctx, nb, i32(to_table))
    w = np.zeros((nb, n_kv, 16), np.float32)
    W = []
    for b, L in enumerate(lens):
        x = rng.integers(0, 6, (L, n_kv)).astype(np.float32) if weights is None else weights(b, L, n_kv)
        W.append(x)
        for t in range(L):
            w[table[b, t // 16], :, t % 16] = x[t]
            kv.k_pool[int(table[b, t // 16]), :, t % 16] = torch.arange(n_kv, device="cuda")[:, None].to(ctx.dtype)
    kv.v_pool.copy_(torch.randn(kv.v_pool.shape, device="cuda"))
    kv.k_pool.copy_(torch.randn(kv.k_pool.shape, device="cuda"))
    if share_pool:
        for blk in to_table.ravel():
            kv.k_pool[int(blk)], kv.v_pool[int(blk)] = 0, 0
    kv.seq_len.copy_(i32(lens))
    k0, v0 = kv.k_pool.clone(), kv.v_pool.clone()
    room = width or dst_w * 16
    kept = torch.full((B, n_kv, room), -9, dtype=torch.int32, device="cuda")
    to_w = torch.zeros((nb, n_kv, 16), device="cuda")
    wd = torch.from_numpy(w).cuda()
    M.mtp_kv_evict(ctx, kv, wd, i32(budgets), to, to_w, kept, sink=sink, recent=recent)
    clean(ctx)
    got = kept.cpu().numpy()
    want_k, want_v, want_w = (torch.zeros_like(k0), torch.zeros_like(v0), torch.zeros_like(to_w))
    if share_pool:
        want_k, want_v = k0.clone(), v0.clone()
    for b, L in enumerate(lens):
        n = min(L, budgets[b])
        for g in range(n_kv):
            mine = P.kept(W[b][:, g], budgets[b], sink, recent)
            np.testing.assert_array_equal(got[b, g, :n], mine)
            assert (got[b, g, n:] == -1).all()
            for j, t in enumerate(mine):
                s, d = (int(table[b, t // 16]), g, int(t % 16)), (int(to_table[b, j // 16]), g, j % 16)
                want_k[d], want_v[d], want_w[d] = k0[s], v0[s], wd[s]
    assert torch.equal(to.k_pool, want_k) and torch.equal(to.v_pool, want_v) and same_bits(to_w, want_w)
    if not share_pool:
        assert torch.equal(kv.k_pool, k0) and torch.equal(kv.v_pool, v0)
    np.testing.assert_array_equal(to.seq_len.cpu().numpy(), [min(a, b) for a, b in zip(lens, budgets)])
    assert not to.pending.any()
    np.testing.assert_array_equal(kv.seq_len.cpu().numpy(), lens)


@pytest.mark.parametrize("dtype,n_kv,hd", [("bf16", 2, 64), ("f32", 1, 128), ("bf16", 1, 128), ("f32", 2, 64)])
def test_evict(dtype, n_kv, hd):
    """Ties everywhere; budgets above, at and below the lengths, of nothing, and with no room beside what always stays."""
    rng = np.random.default_rng(hd)
    ctx = context(n_kv, n_kv, hd, dtype, max_batch=6)
    check_evict(ctx, [0, 1, 20, 33, 65, 100], [8, 8, 20, 32, 9, 17], rng, sink=2, recent=5)
    check_evict(ctx, [50, 1, 17, 40, 64, 90], [0, 0, 16, 1, 33, 89], rng)
    check_evict(ctx, [50, 9, 17, 40, 64, 90], [8, 8, 8, 8, 8, 8], rng, sink=3, recent=5, share_pool=True)
    check_evict(ctx, [50, 9, 17, 40, 64, 90], [8, 8, 8, 8, 8, 8], rng, recent=8, width=11)


def test_evict_by_weights_of_every_size():
    """Weights over all magnitudes, all equal ones, zeros of both signs, infinities and NaN."""
    rng = np.random.default_rng(2)
    ctx = context(2, 2, 64, "bf16", max_batch=3)
    def spread(b, L, n):
        return np.exp(rng.normal(size=(L, n)) * 20).astype(np.float32)
    def equal(b, L, n):
        return np.full((L, n), [0.0, 1.5, 1e-40][b], np.float32)
    def odd(b, L, n):
        x = rng.normal(size=(L, n)).astype(np.float32)
        x[::5], x[1::5, 0], x[2::7], x[3::7, 1], x[4::9] = 0.0, -0.0, np.nan, np.inf, -np.inf
        return x
    for f in (spread, equal, odd):
        check_evict(ctx, [300, 129, 47], [100, 60, 46], rng, sink=1, recent=7, weights=f)


def test_evict_of_long_contexts():
    """More entries than the selection holds in shared memory; against a sort on the GPU."""
    M = M_()
    ctx = context(2, 2, 64, "bf16", max_batch=2)
    lens, budget, sink, recent = [70001, 52000], 1000, 4, 100
    need = [(n + 15) // 16 for n in lens]
    table = np.zeros((2, max(need)), np.int64)
    table[0, :need[0]], table[1, :need[1]] = np.arange(need[0]), need[0] + np.arange(need[1])
    kv = M.KVCache.empty(ctx, sum(need), i32(table))
    kv.k_pool.copy_(torch.randn(kv.k_pool.shape, device="cuda")), kv.v_pool.copy_(torch.randn(kv.v_pool.shape, device="cuda"))
    kv.seq_len.copy_(i32(lens))
    w = torch.rand((sum(need), 2, 16), device="cuda").mul(1e4).round()     # ties
    to = M.KVCache.empty(ctx, 126, i32(np.arange(126).reshape(2, 63)))
    kept = torch.empty((2, 2, 1000), dtype=torch.int32, device="cuda")
    M.mtp_kv_evict(ctx, kv, w, i32([budget] * 2), to, None, kept, sink=sink, recent=recent)
    clean(ctx)
    for b in range(2):
        flat, kf = (x[torch.as_tensor(table[b, :need[b]]).cuda()].transpose(1, 2).flatten(0, 1)[:lens[b]] for x in (w, kv.k_pool))
        flat[:sink], flat[lens[b] - recent:] = float("inf"), float("inf")
        for g in range(2):
            want = torch.sort(flat[:, g], descending=True, stable=True).indices[:budget].sort().values
            assert torch.equal(kept[b, g].long(), want)
            got = to.k_pool[63 * b:63 * b + 63, g].flatten(0, 1)[:budget]
            assert torch.equal(got, kf[want, g])


def test_evict_refusals():
    M = M_()
    ctx = context(4, 2, 64, "bf16", max_batch=2)
    def fresh():
        kv, to = M.KVCache.empty(ctx, 9, i32([[0, 1, 2], [3, 4, 5]])), M.KVCache.empty(ctx, 4, i32([[0, 1], [2, 3]]))
        kv.k_pool.fill_(1.0)
        kv.seq_len.copy_(i32([40, 33])), to.seq_len.fill_(7)
        return kv, to
    w, kept = torch.rand((9, 2, 16), device="cuda"), torch.full((2, 2, 32), -9, dtype=torch.int32, device="cuda")
    budget = i32([20, 20])
    for change, err, kw in ((lambda kv, to: kv.pending.__setitem__(0, 1), M.MTP_ERR_DEVICE_ARGS, {}),
                            (lambda kv, to: kv.seq_len.__setitem__(0, -1), M.MTP_ERR_DEVICE_ARGS, {}),
                            (lambda kv, to: kv.seq_len.__setitem__(0, 49), M.MTP_ERR_CAPACITY, {}),
                            (lambda kv, to: None, M.MTP_ERR_DEVICE_ARGS, dict(budget=i32([-1, 20]))),
                            (lambda kv, to: None, M.MTP_ERR_DEVICE_ARGS, dict(budget=i32([9, 20]), sink=5, recent=5)),
                            (lambda kv, to: None, M.MTP_ERR_CAPACITY, dict(budget=i32([33, 20])))):
        kv, to = fresh()
        change(kv, to)
        kept.fill_(-9)
        kw = dict(kw)
        M.mtp_kv_evict(ctx, kv, w, kw.pop("budget", budget), to, None, kept, **kw)
        assert M.mtp_get_device_error(ctx) == err
        assert bool((kept[0] == -9).all()) and bool((kept[1] != -9).any())
        assert to.seq_len.tolist() == [7, 20] and not to.k_pool[:2].any() and bool(to.k_pool[2].any())
    # blocks outside the pools
    kv, to = fresh()
    kv.block_table[0, 1] = 9
    to.block_table[1, 0] = -1
    M.mtp_kv_evict(ctx, kv, w, i32([40, 20]).clamp(max=32), to, None, kept)
    assert M.mtp_get_device_error(ctx) == M.MTP_ERR_CAPACITY
    kv, to = fresh()
    for args, kw, e in (((ctx, kv, w, budget, kv, None, kept), {}, M.MTPError), ((ctx, kv, w, budget[:1], to, None, kept), {}, ValueError),
                        ((ctx, kv, w[:3], budget, to, None, kept), {}, ValueError), ((ctx, kv, w, budget, to, w, kept), {}, ValueError),
                        ((ctx, kv, w, budget, to, None, kept[0]), {}, ValueError), ((ctx, kv, w, budget, to, None, kept), dict(sink=-1), M.MTPError),
                        ((ctx, kv, w, budget, M.KVCache.empty(ctx, 4, i32([[0, 1]])), None, kept), {}, ValueError)):
        with pytest.raises(e):
            M.mtp_kv_evict(*args, **kw)
    clean(ctx)
