"""The oracle of the verifier's side (8-bit format, rotary, attention, logits)
against independent facts, and the refusals of the new entry points.  CPU only:
no call here launches work."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import verifier as V


def test_code_values_and_rounding_equal_the_formats_own_cast():
    codes = torch.arange(256, dtype=torch.int64).to(torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(V.VALUES, want)
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.normal(size=20000) * np.exp2(rng.integers(-12, 8, 20000)), V._POS, -V._POS,
                        (V._POS[1:] + V._POS[:-1]) / 2])          # ties included
    x = x[np.abs(x) <= 448].astype(np.float32)
    got = V.e4m3_encode(x)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(got, want)
    assert V.e4m3_encode([np.nan, np.inf, -np.inf]).tolist() == [0x7F] * 3


@pytest.mark.parametrize("top,s", [(448.0, 1.0), (449.0, 2.0), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8), (1.7501, 2.0 ** -7),
                                   (0.0, 0.0), (3e38, 2.0 ** 120), (1e-44, 2.0 ** -126)])
def test_block_scale(top, s):
    assert V.block_scale([0.0, -top, top / 2, np.inf, np.nan]) == s


def test_rotation_keeps_norms_and_inner_products_of_equal_distance():
    rng = np.random.default_rng(2)
    for layout in ("half", "interleaved"):
        q, k = rng.normal(size=(1, 1, 32)), rng.normal(size=(1, 1, 32))
        dots = [(V.rope(q, [p + 7], layout) * V.rope(k, [p], layout)).sum() for p in (0, 5, 100000)]
        assert np.ptp(dots) < 1e-9
        np.testing.assert_allclose((V.rope(q, [12345], layout) ** 2).sum(), (q ** 2).sum())
    x = rng.normal(size=(1, 2, 16))
    np.testing.assert_array_equal(V.rope(x, [9], rotary_dim=6)[..., 6:], x[..., 6:])


def table(**kw):
    import mtp_self_speculative_gb300 as M
    return M.RopeTable(**kw)


@pytest.mark.parametrize("kw", [dict(rotary_dim=128, theta=1e6), dict(rotary_dim=64, theta=10000.0, scaling="linear", factor=4.0),
                                dict(rotary_dim=128, scaling="parts", factor=8.0, original_max_pos=8192),
                                dict(rotary_dim=48, scaling="yarn", factor=16.0, original_max_pos=4096, layout="interleaved"),
                                dict(rotary_dim=2, theta=10000.0), dict(rotary_dim=64, scaling="linear", factor=0.05)])
def test_rope_table_holds_the_formulas_phases(kw):
    t = table(**kw)
    f, mag = V.rope_frequencies(**{k: v for k, v in kw.items() if k != "layout"})
    for i, x in enumerate(f):
        turn = x / (2 * math.pi) % 1.0
        diff = abs(t.turns[i] / 2.0 ** 64 - turn)
        # theta and factor pass through float32 fields (exact here but for 0.05); pow and the division round in 64 bits
        tol = 1e-14 if kw.get("factor") != 0.05 else 1e-6
        assert min(diff, 1 - diff) < tol, i
    assert abs(t.magnitude - mag) <= 2.0 ** -24 * mag
    assert table(rotary_dim=8, magnitude=1.5).magnitude == 1.5


@pytest.mark.parametrize("bad", [dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=130), dict(rotary_dim=64, theta=1.0),
                                 dict(rotary_dim=64, theta=float("nan")), dict(rotary_dim=64, scaling="linear", factor=0.0),
                                 dict(rotary_dim=64, scaling="parts", factor=2.0), dict(rotary_dim=64, magnitude=-1.0),
                                 dict(rotary_dim=64, scaling="parts", factor=2.0, original_max_pos=10, low_freq_factor=4.0),
                                 dict(rotary_dim=64, scaling="yarn", factor=2.0, original_max_pos=10, beta_slow=0.0),
                                 dict(rotary_dim=64, scaling="yarn", factor=2.0, original_max_pos=10, beta_fast=0.5),
                                 dict(rotary_dim=64, scaling="yarn", factor=float("inf"), original_max_pos=10)])
def test_rope_table_refuses_bad_parameters(bad):
    import mtp_self_speculative_gb300 as M
    with pytest.raises(M.MTPError):
        M.RopeTable(**bad)
    with pytest.raises(ValueError):
        M.RopeTable(64, layout="rows")


def test_calls_without_context_are_rejected():
    from mtp_self_speculative_gb300 import _lib as L
    lib = L.load()
    kv, tab, la = L.MTPKV8(16, 16, 16, 16, 16, 16, 16, 16, 1, 1), L.MTPRopeTable(), L.MTPLogitsArgs()
    k, t = ctypes.byref(kv), ctypes.byref(tab)
    assert lib.mtp_rope(None, None, 1, 1, 16, 64, 16, t, 16, 64) == L.MTP_ERR_INVALID
    assert lib.mtp_kv8_append(None, None, 1, 1, 16, 16, 64, 16, 64, 16, t, None, 0, None, 0, k) == L.MTP_ERR_INVALID
    assert lib.mtp_kv8_read(None, None, 1, k, 16, 1, 16, 16, 16) == L.MTP_ERR_INVALID
    for fn in (lib.mtp_kv8_commit, lib.mtp_kv8_truncate):
        assert fn(None, None, 1, k, 16) == L.MTP_ERR_INVALID
    assert lib.mtp_kv8_commit_accepted(None, None, 1, k, 16, 1) == L.MTP_ERR_INVALID
    assert lib.mtp_kv8_rollback(None, None, 1, k) == L.MTP_ERR_INVALID
    assert lib.mtp_kv8_commit_path(None, None, 1, k, 16, 1, 16) == L.MTP_ERR_INVALID
    assert lib.mtp_kv8_attention_workspace_bytes(None) == 0
    assert lib.mtp_kv8_attention(None, None, 1, 1, 16, 1, 16, 64, k, None, 0, 1.0, 16, None, 16, 1 << 30) == L.MTP_ERR_INVALID
    assert lib.mtp_token_counts_add(None, None, 1, 16, 1, 16, 0, 16) == L.MTP_ERR_INVALID
    assert lib.mtp_logits_process(None, None, ctypes.byref(la)) == L.MTP_ERR_INVALID
    assert lib.mtp_rope_table_make(None, t) == L.MTP_ERR_INVALID
    assert lib.mtp_set_rope(None, t) == L.MTP_ERR_INVALID
    assert lib.mtp_draft_kv8_workspace_bytes(None) == 0
    assert lib.mtp_draft_kv8(None, None, 1, 16, 16, 16, k, 1, None, 16, None, None, 256, 1 << 30) == L.MTP_ERR_INVALID


def cpu_context(**kw):
    import mtp_self_speculative_gb300 as M
    base = dict(hidden=256, n_q_heads=8, n_kv_heads=2, head_dim=64, ffn=256, vocab=100, dtype="bf16", max_batch=4)
    base.update(kw)
    return M.Context(0, M.make_config(**base), None)


def test_wrappers_check_shapes_before_any_call():
    """CPU tensors throughout: a wrong shape or type is reported first, and the
    well-formed rest stops at the device-pointer check."""
    import mtp_self_speculative_gb300 as M
    ctx = cpu_context()
    bf, i32 = torch.bfloat16, dict(dtype=torch.int32)
    rope = M.RopeTable(64)
    with pytest.raises(ValueError, match="head_dim"):
        M.mtp_rope(ctx, torch.zeros(4, 64, dtype=bf), torch.zeros(4, **i32), rope)
    with pytest.raises(ValueError, match="x must be"):
        M.mtp_rope(ctx, torch.zeros(4, 8, 32, dtype=bf), torch.zeros(4, **i32), rope)
    with pytest.raises(ValueError, match="bfloat16"):
        M.mtp_rope(ctx, torch.zeros(4, 8, 64), torch.zeros(4, **i32), rope)
    with pytest.raises(ValueError, match="CUDA"):
        M.mtp_rope(ctx, torch.zeros(4, 8, 64, dtype=bf), torch.zeros(4, **i32), rope)
    kv = M.KVCache8.empty(ctx, 3, torch.zeros(2, 3, **i32))
    with pytest.raises(ValueError, match="CUDA"):
        M.mtp_kv8_rollback(ctx, kv)
    kv.k_pool = kv.k_pool.float()
    with pytest.raises(ValueError, match="uint8 or float8"):
        M.mtp_kv8_rollback(ctx, kv)
    x = torch.zeros(3, 100, dtype=bf)
    with pytest.raises(ValueError, match="row_offsets"):
        M.mtp_logits_process(ctx, x, torch.zeros(1, **i32))
    with pytest.raises(ValueError, match="go together"):
        M.mtp_logits_process(ctx, x, torch.zeros(2, **i32), bias_offsets=torch.zeros(2, **i32))
    with pytest.raises(ValueError, match="go together"):
        M.mtp_logits_process(ctx, x, torch.zeros(2, **i32), mask=torch.zeros(1, 4, **i32))


def test_a_cache_is_checked_for_each_context_and_after_a_change(monkeypatch):
    """What was checked belongs to a context's device and configuration and to the fields' shapes and layout (pointers
    are not looked at here: the tensors are the CPU's)."""
    import copy
    import mtp_self_speculative_gb300 as M
    checked = []

    def pointer(ctx, t, dtype, name, shape=None):
        checked.append((ctx.device, name))
        if (dtype is not None and t.dtype is not dtype) or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
            raise ValueError(name)
        return t.data_ptr()

    monkeypatch.setattr(M, "_dev_ptr", pointer)
    ctx, other = cpu_context(), cpu_context()
    other.cfg, ctx.device, other.device = ctx.cfg, 0, 1
    kv = M.KVCache8.empty(ctx, 3, torch.zeros(2, 6, dtype=torch.int32))
    assert kv.struct(ctx).max_blocks == 6
    checked.clear()
    kv.struct(other)
    assert {d for d, _ in checked} == {1} and len(checked) == 8
    two = copy.deepcopy(kv)
    assert two.struct(ctx).k_pool == two.k_pool.data_ptr() != kv.k_pool.data_ptr()
    kv.block_table.resize_(2, 3)
    assert kv.struct(ctx).max_blocks == 3
    for change, back in ((lambda: kv.block_table.t_(), lambda: kv.block_table.t_()),
                         (lambda: kv.pending.resize_(1), lambda: kv.pending.resize_(2)),
                         (lambda: kv.v_scale.resize_(3, 1), lambda: kv.v_scale.resize_(3, 2)),
                         (lambda: setattr(kv, "v_scale", kv.v_scale.view(torch.int32)),
                          lambda: setattr(kv, "v_scale", kv.v_scale.view(torch.float32)))):
        change()
        with pytest.raises(ValueError):
            kv.struct(ctx)
        back()
        kv.struct(ctx)
    kv.block_table = torch.zeros(2, 2, dtype=torch.int32)
    assert kv.struct(ctx).max_blocks == 2
    kv.block_table.t_()                       # the same shape
    with pytest.raises(ValueError):
        kv.struct(ctx)
    kv.block_table.t_()
    small = cpu_context(n_kv_heads=1)
    small.device = 0
    with pytest.raises(ValueError):
        kv.struct(small)


def test_a_context_keeps_the_configuration_it_was_made_with():
    import mtp_self_speculative_gb300 as M
    cfg = M.make_config(hidden=256, n_q_heads=8, n_kv_heads=2, head_dim=64, ffn=256, vocab=100, dtype="bf16", max_batch=4)
    ctx = M.Context(0, cfg, None)
    cfg.head_dim, cfg.vocab = 128, 7
    assert (ctx.cfg.head_dim, ctx.cfg.vocab, ctx.head_dim, ctx.vocab) == (64, 100, 64, 100)


def test_processed_logits_of_a_hand_made_row():
    z = np.array([2.0, -2.0, 1.0, 0.5, 3.0])
    counts = np.array([1, 2, 0, -2 ** 31, 0], dtype=np.int64).astype(np.int32)
    got, _ = V.process_logits(z, counts, before=[2], repetition=2.0, frequency=0.25, presence=0.5,
                              bias=[(4, 1.0), (4, 2.0)], allowed=np.array([1, 1, 1, 1, 1], bool))
    np.testing.assert_allclose(got, [1.0 - 0.25 - 0.5, -4.0 - 0.5 - 0.5, 0.5 - 0.25 - 0.5, 0.25, 6.0])
    got, _ = V.process_logits(z, counts, allowed=np.array([0, 1, 0, 1, 0], bool))
    assert np.isneginf(got[[0, 2, 4]]).all() and np.isfinite(got[[1, 3]]).all()


def test_attention_of_one_visible_entry_is_that_entry():
    rng = np.random.default_rng(3)
    q, k, v = rng.normal(size=(2, 4, 8)), rng.normal(size=(5, 2, 8)), rng.normal(size=(5, 2, 8))
    seen = np.zeros((2, 5), bool)
    seen[0, 3] = True
    out, lse, mass, _ = V.attention(q, k, v, seen, 0.5)
    np.testing.assert_allclose(out[0, 1], v[3, 0])
    np.testing.assert_allclose(lse[0, 3], 0.5 * k[3, 1] @ q[0, 3])
    assert (out[1] == 0).all() and np.isneginf(lse[1]).all() and (mass[1] == 0).all()
