"""The operators on the paged cache in the context's type, without a device:
calls without a context, shapes that the wrappers refuse, when a cache is looked
at again, and hand-made pins of the restatement."""
import copy
import ctypes

import numpy as np
import pytest
import torch

from oracle import paged as P
from oracle import verifier as V
from test_verifier_pins import cpu_context

I32, F32, BF = dict(dtype=torch.int32), dict(dtype=torch.float32), dict(dtype=torch.bfloat16)


def test_calls_without_context_are_rejected():
    from mtp_self_speculative_gb300 import _lib as L
    lib = L.load()
    kv, t = ctypes.byref(L.MTPKV(16, 16, 16, 16, 16, 1, 1)), ctypes.byref(L.MTPRopeTable())
    assert lib.mtp_qk_norm_rope(None, None, 1, 16, 64, 16, 16, 64, None, 0, None, None, 0, 1e-6, 16, t) == L.MTP_ERR_INVALID
    assert lib.mtp_kv_append(None, None, 1, 1, 16, 16, 64, None, 16, 64, None, 0, None, None, 0, 1e-6, None, None, kv,
                             16) == L.MTP_ERR_INVALID
    assert lib.mtp_kv_attention_workspace_bytes(None) == 0
    assert lib.mtp_kv_attention(None, None, 1, 1, 16, 1, 16, 64, kv, None, 0, 1.0, 16, None, 16, 1 << 40) == L.MTP_ERR_INVALID
    assert lib.mtp_kv_attention_weights(None, None, 1, 1, 16, 1, 16, 64, kv, None, 0, 1.0, 16, None, 16) == L.MTP_ERR_INVALID
    assert lib.mtp_kv_evict(None, None, 1, kv, 16, 16, 0, 0, kv, None, 16, 1) == L.MTP_ERR_INVALID
    with pytest.raises(Exception):
        import mtp_self_speculative_gb300 as M
        M.AttentionWorkspace(cpu_context())


class NoWorkspace:
    device, ptr, bytes = 0, 256, 1 << 40


def test_wrappers_check_shapes_before_any_call():
    """CPU tensors throughout: a wrong shape or type is reported first, and the well-formed rest stops at the
    device-pointer check."""
    import mtp_self_speculative_gb300 as M
    ctx = cpu_context()
    q, k = torch.zeros(4, 8, 64, **BF), torch.zeros(4, 2, 64, **BF)
    off, rope, at = torch.zeros(3, **I32), M.RopeTable(64), torch.zeros(4, **I32)
    with pytest.raises(ValueError, match="neither"):
        M.mtp_qk_norm_rope(ctx, None, None)
    with pytest.raises(ValueError, match="need q"):
        M.mtp_qk_norm_rope(ctx, None, k, q_weight=torch.zeros(64, **BF))
    for bad in (q.float(), q[:, :7], q[:, :, :32], q.flatten(1)):
        with pytest.raises(ValueError):
            M.mtp_qk_norm_rope(ctx, bad, None, positions=at, rope=rope)
    with pytest.raises(ValueError, match="CUDA"):
        M.mtp_qk_norm_rope(ctx, q, k, positions=at, rope=rope)
    kv = M.KVCache.empty(ctx, 3, torch.zeros(2, 3, **I32))
    for call in (lambda: M.mtp_kv_append(ctx, kv, k, k, off),
                 lambda: M.mtp_kv_attention(ctx, kv, q, off, torch.zeros_like(q), NoWorkspace, 1),
                 lambda: M.mtp_kv_attention_weights(ctx, kv, q, off, torch.zeros(4, 8), torch.zeros(3, 2, 16), 1),
                 lambda: M.mtp_kv_evict(ctx, kv, torch.zeros(3, 2, 16), torch.zeros(2, **I32), kv, None, torch.zeros(2, 2, 5, **I32))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for field, value in (("k_pool", kv.k_pool.float()), ("v_pool", kv.v_pool[:2]), ("seq_len", kv.seq_len.long()),
                         ("pending", kv.pending[:1]), ("block_table", kv.block_table[0]), ("k_pool", kv.k_pool[0]),
                         ("arrive", torch.zeros(1, **I32))):
        other = copy.copy(kv)
        setattr(other, field, value)
        with pytest.raises(ValueError):
            M.mtp_kv_commit(ctx, other, torch.zeros(2, **I32))


def pointers(monkeypatch):
    import mtp_self_speculative_gb300 as M
    checked = []

    def pointer(ctx, t, dtype, name, shape=None):
        if t is None:
            return None
        checked.append((ctx.device, name))
        if (dtype is not None and t.dtype is not dtype) or not t.is_contiguous() or (shape is not None and tuple(t.shape) != tuple(shape)):
            raise ValueError(name)
        return t.data_ptr()

    monkeypatch.setattr(M, "_dev_ptr", pointer)
    monkeypatch.setattr(M, "_row_ptr", lambda ctx, t, name, rows, heads: (pointer(ctx, t, ctx.dtype, name, (rows, heads, ctx.head_dim)), heads * ctx.head_dim))
    monkeypatch.setattr(M, "_ctx_stream", lambda ctx, stream: 0)
    return M, checked


def test_a_cache_is_checked_for_each_context_and_after_a_change(monkeypatch):
    M, checked = pointers(monkeypatch)
    ctx, other = cpu_context(), cpu_context()
    other.cfg, ctx.device, other.device = ctx.cfg, 0, 1
    kv = M.KVCache.empty(ctx, 3, torch.zeros(2, 6, **I32))

    def struct(c=ctx, cache=kv):
        return cache._checked_struct(c)[0]
    assert struct().max_blocks == 6
    checked.clear()
    assert struct().num_blocks == 3 and not checked
    struct(other)
    assert {d for d, _ in checked} == {1} and len(checked) == 6
    two = copy.deepcopy(kv)
    assert struct(cache=two).k_pool == two.k_pool.data_ptr() != kv.k_pool.data_ptr()
    kv.block_table.resize_(2, 3)
    assert struct().max_blocks == 3
    for change, back in ((lambda: kv.block_table.t_(), lambda: kv.block_table.t_()),
                         (lambda: kv.pending.resize_(1), lambda: kv.pending.resize_(2)),
                         (lambda: kv.arrive.resize_(1), lambda: kv.arrive.resize_(2)),
                         (lambda: kv.v_pool.resize_(2, 2, 16, 64), lambda: kv.v_pool.resize_(3, 2, 16, 64)),
                         (lambda: setattr(kv, "k_pool", kv.k_pool.view(torch.int16)),
                          lambda: setattr(kv, "k_pool", kv.k_pool.view(torch.bfloat16)))):
        struct()
        change()
        with pytest.raises(ValueError):
            struct()
        back()
        struct()
    kv.block_table = torch.zeros(2, 2, **I32)
    assert struct().max_blocks == 2
    kv.arrive = None
    struct()
    with pytest.raises(ValueError, match="arrive"):
        M.mtp_kv_append(ctx, kv, torch.zeros(1, 2, 64, **BF), torch.zeros(1, 2, 64, **BF), torch.zeros(3, **I32))
    small = cpu_context(n_kv_heads=1)
    small.device = 0
    with pytest.raises(ValueError):
        struct(small)


def test_other_arguments_are_checked(monkeypatch):
    M, _ = pointers(monkeypatch)
    ctx = cpu_context()
    ctx.device = 0
    kv, to = M.KVCache.empty(ctx, 3, torch.zeros(2, 3, **I32)), M.KVCache.empty(ctx, 3, torch.zeros(1, 3, **I32))
    q, k, off = torch.zeros(4, 8, 64, **BF), torch.zeros(4, 2, 64, **BF), torch.zeros(3, **I32)
    w, kept, budget = torch.zeros(3, 2, 16), torch.zeros(2, 2, 5, **I32), torch.zeros(2, **I32)
    out, lse = torch.zeros_like(q), torch.zeros(4, 8)
    bad = [lambda: M.mtp_qk_norm_rope(ctx, q, None, q_weight=q[0, 0], k_out=k), lambda: M.mtp_qk_norm_rope(ctx, None, k, k_weight=k[0, 0], q_out=q),
           lambda: M.mtp_kv_append(ctx, kv, k, k[:3], off), lambda: M.mtp_kv_append(ctx, kv, k, k, off[:2]),
           lambda: M.mtp_kv_append(ctx, kv, k, k, off, q_out=q), lambda: M.mtp_kv_append(ctx, kv, k, k, off, q=q[:3]),
           lambda: M.mtp_kv_append(ctx, kv, k, k, off, k_weight=torch.zeros(32, **BF)),
           lambda: M.mtp_kv_append(ctx, kv, k, k, off, positions=torch.zeros(3, **I32), rope=M.RopeTable(64)),
           lambda: M.mtp_kv_attention(ctx, kv, q, off, out[:3], NoWorkspace, 1),
           lambda: M.mtp_kv_attention(ctx, kv, q, off, out, NoWorkspace, 1, lse=lse[:, :7]),
           lambda: M.mtp_kv_attention(ctx, kv, q, off, out, NoWorkspace, 1, mask=torch.zeros(3, 1, **I32)),
           lambda: M.mtp_kv_attention(ctx, kv, q, off[:2], out, NoWorkspace, 1),
           lambda: M.mtp_kv_attention_weights(ctx, kv, q, off, lse[:3], w, 1),
           lambda: M.mtp_kv_attention_weights(ctx, kv, q, off, lse, w[:2], 1),
           lambda: M.mtp_kv_attention_weights(ctx, kv, q, off, lse, w, 1, first=off),
           lambda: M.mtp_kv_evict(ctx, kv, w, budget, to, None, kept),
           lambda: M.mtp_kv_evict(ctx, kv, w, budget[:1], copy.deepcopy(kv), None, kept),
           lambda: M.mtp_kv_evict(ctx, kv, w, budget, copy.deepcopy(kv), w[:2], kept),
           lambda: M.mtp_kv_evict(ctx, kv, w, budget, copy.deepcopy(kv), None, kept[0]),
           lambda: M.mtp_kv_evict(ctx, kv, w, budget, copy.deepcopy(kv), None, kept[:, :1])]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail("call %d was taken" % i)

    class Elsewhere(NoWorkspace):
        device = 1
    with pytest.raises(ValueError, match="cuda:1"):
        M.mtp_kv_attention(ctx, kv, q, off, out, Elsewhere, 1)


def test_norm_of_a_hand_made_head():
    x = np.array([[[3.0, -4.0, 0.0, 0.0]]])
    np.testing.assert_allclose(P.norm(x, [1.0, 2.0, 1.0, 1.0], 0.0), [[[1.2, -3.2, 0.0, 0.0]]])
    assert P.norm(x, None, 1e-6) is not None and (P.norm(x, None, 1e-6) == x).all()


def test_weights_of_rows_are_their_softmax():
    rng = np.random.default_rng(2)
    q, k, v = rng.normal(size=(3, 4, 8)), rng.normal(size=(9, 2, 8)), rng.normal(size=(9, 2, 8))
    seen = V.causal(3, 9)
    _, lse, _, _ = V.attention(q, k, v, seen, 0.4)
    w, _ = P.gathered(q, k, lse, seen, 0.4)
    np.testing.assert_allclose(w.sum(0), [6.0, 6.0])            # three rows, two heads a group
    z = np.exp(0.4 * k[:, 1] @ q[2, 3])
    alone, _ = P.gathered(q[2:], k, lse[2:], seen[2:], 0.4)
    one = np.exp(0.4 * k[:, 1] @ q[2, 2])
    np.testing.assert_allclose(alone[:, 1], z / z.sum() + one / one.sum())
    assert (P.gathered(q[:1], k, lse[:1], seen[:1], 0.4)[0][7:] == 0).all()


@pytest.mark.parametrize("weight,budget,sink,recent,want", [
    ([5, 1, 2, 2, 9, 0], 3, 0, 0, [0, 2, 4]),                   # equal ones from the lowest slot on
    ([5, 1, 2, 2, 9, 0], 3, 1, 1, [0, 4, 5]),
    ([0, 0, 0, 0, 0, 0], 3, 1, 2, [0, 4, 5]),
    ([1, np.nan, -0.0, 0.0, -1, 2], 4, 0, 0, [0, 2, 3, 5]),
    ([1, np.nan, -np.inf, np.inf, -1, 2], 5, 0, 0, [0, 2, 3, 4, 5]),
    ([3, 2, 1], 0, 0, 0, []), ([3, 2, 1], 7, 2, 2, [0, 1, 2])])
def test_what_stays_of_hand_made_weights(weight, budget, sink, recent, want):
    assert P.kept(np.array(weight, float), budget, sink, recent).tolist() == want


def test_a_hand_made_cache():
    c = P.Cache(4, 1, 2, [[2, 0]])
    k = np.arange(34.0).reshape(17, 1, 2)
    c.append(0, k, -k)
    assert (c.pools[0][2, 0, 0] == [0, 1]).all() and (c.pools[1][0, 0, 0] == [-32, -33]).all()
    c.commit(0, 3)
    assert c.length(0) == 3 and (c.pools[0][2, 0, 3:] == 0).all() and (c.pools[0][0] == 0).all()
    assert (c.values(0)[0] == k[:3]).all()
