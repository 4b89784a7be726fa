"""Lengths at which a slot or a step past it would not be an int are refused,
and leave everything as it was.  The tables are that wide; their blocks are one."""
import pytest
import torch

from test_gpu_verifier import M_, clean, context, i32

pytestmark = pytest.mark.gpu

MOST = 1 << 30


@pytest.fixture(scope="module")
def wide():
    M = M_()
    ctx = context(1, 1, 64, "bf16", max_batch=1)
    kv = M.KVCache.empty(ctx, 1, torch.zeros((1, MOST // 16 + 4), dtype=torch.int32, device="cuda"))
    return ctx, kv


def test_append_up_to_the_last_slot(wide):
    M, (ctx, kv) = M_(), wide
    k = torch.full((2, 1, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    kv.k_pool.zero_(), kv.v_pool.zero_()
    for sl, pe in ((MOST - 1, 0), (5, MOST - 6), (MOST - 2, 5)):
        kv.seq_len.fill_(sl), kv.pending.fill_(pe)
        M.mtp_kv_append(ctx, kv, k, k, i32([0, 2]))
        assert M.mtp_get_device_error(ctx) == M.MTP_ERR_CAPACITY
        assert kv.seq_len.item() == sl and kv.pending.item() == pe and not kv.k_pool.any() and not kv.arrive.any()
    kv.seq_len.fill_(MOST - 2), kv.pending.fill_(0)
    M.mtp_kv_append(ctx, kv, k, k, i32([0, 2]))
    clean(ctx)
    assert kv.pending.item() == 2 and bool((kv.k_pool[0, 0, 14:] == 3).all()) and not kv.k_pool[0, 0, :14].any()


def test_eviction_of_more_entries_than_slots_can_name(wide):
    M, (ctx, kv) = M_(), wide
    kv.seq_len.fill_(MOST + 1), kv.pending.fill_(0)
    to = M.KVCache.empty(ctx, 2, i32([[0, 1]]))
    to.seq_len.fill_(7)
    kept = torch.full((1, 1, 20), -9, dtype=torch.int32, device="cuda")
    w = torch.zeros((1, 1, 16), device="cuda")
    M.mtp_kv_evict(ctx, kv, w, i32([20]), to, None, kept)
    assert M.mtp_get_device_error(ctx) == M.MTP_ERR_CAPACITY
    assert bool((kept == -9).all()) and to.seq_len.item() == 7 and not to.k_pool.any()


def test_a_list_wider_than_any_length_is_refused_on_the_host(wide):
    from mtp_self_speculative_gb300 import _lib as L
    M, (ctx, kv) = M_(), wide
    to = M.KVCache.empty(ctx, 2, i32([[0, 1]]))
    w, b, kept = torch.zeros((1, 1, 16), device="cuda"), i32([20]), torch.zeros(20, dtype=torch.int32, device="cuda")
    st = [x._checked_struct(ctx)[0] for x in (kv, to)]
    got = L.load().mtp_kv_evict(ctx.handle, None, 1, st[0], w.data_ptr(), b.data_ptr(), 0, 0, st[1], None, kept.data_ptr(),
                                MOST + 1)
    assert got == L.MTP_ERR_INVALID
