"""MTP self-speculative draft-and-verify step on one GB300 (sm_103a).

A thin binding over the C ABI of ``libmtp.so`` (declared in include/mtp.h):
the functions below carry the C names and only marshal arguments -- torch
tensors become device pointers, torch streams become cudaStream_t handles.
Every step of the method runs in the library's CUDA kernels; PyTorch is used
for device memory and streams only.  There is no CPU path: if the library is
missing, importing the binding raises.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Dict, Optional

import torch

from . import _lib as L
from ._lib import (  # noqa: F401
    KERNEL_NAMES, MTP_DTYPE_BF16, MTP_DTYPE_F32, MTP_ERR_BOUNDS, MTP_ERR_CAPACITY, MTP_ERR_CUDA, MTP_ERR_DEVICE_ARGS,
    MTP_ERR_INVALID, MTP_ERR_OOM, MTP_ERR_TIMEOUT, MTP_KERNEL_ATTENTION, MTP_KERNEL_DOWN, MTP_KERNEL_EH_PROJ,
    MTP_KERNEL_GATE_UP, MTP_KERNEL_KV_EDIT, MTP_KERNEL_LM_HEAD, MTP_KERNEL_O_PROJ, MTP_KERNEL_QKV_ROPE,
    MTP_KERNEL_VERIFY, MTP_KERNEL_DRAFT_PERSISTENT, MTP_OK, MTP_WEIGHTS_DENSE, MTP_WEIGHTS_INT4_G64, MTPConfig, MTPKV,
    MTPKV8, MTPLogitsArgs, MTPLoop, MTPRopeParams, MTPRopeTable, MTPTree, MTPWeights, MTP_ROPE_HALF,
    MTP_ROPE_INTERLEAVED, MTP_ROPE_SCALE_LINEAR, MTP_ROPE_SCALE_NONE, MTP_ROPE_SCALE_PARTS, MTP_ROPE_SCALE_YARN,
    WEIGHT_FIELDS,
)

_clib = L.load()


class MTPError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s (%d)" % (where, _clib.mtp_status_str(status).decode(), status))


def _check(status: int, where: str) -> None:
    if status != MTP_OK:
        raise MTPError(status, where)


def _ptr(t: Optional[torch.Tensor], dtype=None, name="tensor") -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def torch_dtype(dtype_code: int) -> torch.dtype:
    return torch.bfloat16 if dtype_code == MTP_DTYPE_BF16 else torch.float32


@dataclass
class KVCache:
    """Caller-owned paged MTP KV cache (device tensors)."""
    k_pool: torch.Tensor        # [num_blocks, n_kv, block_size, head_dim]
    v_pool: torch.Tensor
    block_table: torch.Tensor   # [B, max_blocks] int32
    seq_len: torch.Tensor       # [B] int32
    pending: torch.Tensor       # [B] int32

    def struct(self) -> MTPKV:
        return MTPKV(_ptr(self.k_pool, name="k_pool"), _ptr(self.v_pool, name="v_pool"),
                     _ptr(self.block_table, torch.int32, "block_table"), _ptr(self.seq_len, torch.int32, "seq_len"),
                     _ptr(self.pending, torch.int32, "pending"), int(self.k_pool.shape[0]),
                     int(self.block_table.shape[1]))


class Context:
    """Owns an mtp_ctx handle and keeps the borrowed weight tensors alive."""

    def __init__(self, handle: int, cfg: MTPConfig, weights: Optional[Dict[str, torch.Tensor]],
                 device: Optional[int] = None):
        self.handle = handle
        self.cfg = MTPConfig.from_buffer_copy(cfg)   # the library's copy does not change either
        self.weights = weights
        self.device = device
        self.dtype, self.head_dim, self.vocab = torch_dtype(cfg.dtype), int(cfg.head_dim), int(cfg.vocab)

    def close(self):
        if self.handle:
            _clib.mtp_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def make_config(hidden, n_q_heads, n_kv_heads, head_dim, ffn, vocab, eps=1e-6, rope_theta=1e6, dtype="bf16",
                max_batch=1, max_k=5, block_size=16, max_pos=32768, tc_min_batch=0,
                persistent_max_batch=0, weight_format="dense") -> MTPConfig:
    code = MTP_DTYPE_BF16 if dtype in ("bf16", MTP_DTYPE_BF16, torch.bfloat16) else MTP_DTYPE_F32
    wf = MTP_WEIGHTS_INT4_G64 if weight_format in ("int4_g64", MTP_WEIGHTS_INT4_G64) else MTP_WEIGHTS_DENSE
    return MTPConfig(hidden, n_q_heads, n_kv_heads, head_dim, ffn, vocab, eps, rope_theta, code, max_batch, max_k,
                     block_size, max_pos, tc_min_batch, persistent_max_batch, wf)


def mtp_init(cfg: MTPConfig, weights: Optional[Dict[str, torch.Tensor]] = None, device: Optional[int] = None
             ) -> Context:
    """Create a context.  ``weights`` maps the mtp_weights field names to
    device tensors (``lm_head`` optional: tied to ``embed``); None for a
    verify/KV-only context."""
    if device is None:
        device = torch.cuda.current_device()
    wst = None
    if weights is not None:
        dt = torch_dtype(cfg.dtype)
        wst = MTPWeights(*[_ptr(weights.get(n), dt, n) if weights.get(n) is not None else None
                           for n in WEIGHT_FIELDS])
    out = ctypes.c_void_p()
    _check(_clib.mtp_init(ctypes.byref(cfg), ctypes.byref(wst) if wst is not None else None, int(device),
                         ctypes.byref(out)), "mtp_init")
    return Context(out.value, cfg, weights, int(device))


def mtp_draft(ctx: Context, hidden: torch.Tensor, embeds: torch.Tensor, positions: torch.Tensor, kv: KVCache, K: int,
              draft_ids: torch.Tensor, logits: Optional[torch.Tensor] = None, hidden_out: Optional[torch.Tensor] = None,
              chain_ids: Optional[torch.Tensor] = None, stream=None) -> None:
    dt = torch_dtype(ctx.cfg.dtype)
    B = int(hidden.shape[0])
    kvs = kv.struct()
    _check(_clib.mtp_draft(ctx.handle, _stream(stream), B, _ptr(hidden, dt, "hidden"), _ptr(embeds, dt, "embeds"),
                          _ptr(positions, torch.int32, "positions"), ctypes.byref(kvs), int(K),
                          _ptr(chain_ids, torch.int32, "chain_ids"), _ptr(draft_ids, torch.int32, "draft_ids"),
                          _ptr(logits, torch.float32, "logits"), _ptr(hidden_out, torch.float32, "hidden_out")),
           "mtp_draft")


def _check_verify_shapes(target_logits: torch.Tensor, row_offsets: torch.Tensor, drafts: torch.Tensor,
                         num_drafts: torch.Tensor, accepted: torch.Tensor, bonus: torch.Tensor, vocab: int,
                         where: str) -> int:
    """Shape checks the C entry points cannot make (they receive plain
    pointers): the kernel reads num_rows x vocab logits and B + 1 offsets and
    writes B results, so a mismatch here would read or write past a buffer.
    Returns B."""
    if target_logits.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("%s: target_logits must be float32 or bfloat16, got %s" % (where, target_logits.dtype))
    if target_logits.dim() != 2 or int(target_logits.shape[1]) != int(vocab) or int(target_logits.shape[0]) < 1:
        raise ValueError("%s: target_logits must be [num_rows >= 1, vocab=%d], got %s"
                         % (where, vocab, tuple(target_logits.shape)))
    if num_drafts.dim() != 1:
        raise ValueError("%s: num_drafts must be 1-D [B]" % where)
    B = int(num_drafts.shape[0])
    if row_offsets.dim() != 1 or int(row_offsets.shape[0]) != B + 1:
        raise ValueError("%s: row_offsets must be [B + 1] = [%d], got %s" % (where, B + 1, tuple(row_offsets.shape)))
    if drafts.dim() != 2 or int(drafts.shape[0]) != B:
        raise ValueError("%s: drafts must be [B=%d, stride], got %s" % (where, B, tuple(drafts.shape)))
    for t, name in ((accepted, "accepted"), (bonus, "bonus")):
        if t.numel() != B:
            raise ValueError("%s: %s must hold B=%d entries, got %d" % (where, name, B, t.numel()))
    return B


def mtp_verify(ctx: Context, target_logits: torch.Tensor, row_offsets: torch.Tensor, drafts: torch.Tensor,
               num_drafts: torch.Tensor, accepted: torch.Tensor, bonus: torch.Tensor, stream=None) -> None:
    dt = torch_dtype(ctx.cfg.dtype)
    B = _check_verify_shapes(target_logits, row_offsets, drafts, num_drafts, accepted, bonus, ctx.cfg.vocab,
                             "mtp_verify")
    _check(_clib.mtp_verify(ctx.handle, _stream(stream), B, _ptr(target_logits, dt, "target_logits"),
                           int(target_logits.shape[0]), _ptr(row_offsets, torch.int32, "row_offsets"), _ptr(drafts, torch.int32, "drafts"),
                           int(drafts.shape[1]), _ptr(num_drafts, torch.int32, "num_drafts"),
                           _ptr(accepted, torch.int32, "accepted"), _ptr(bonus, torch.int32, "bonus")), "mtp_verify")


def mtp_verify_noalloc(target_logits: torch.Tensor, row_offsets: torch.Tensor, drafts: torch.Tensor,
                       num_drafts: torch.Tensor, accepted: torch.Tensor, bonus: torch.Tensor, vocab: int,
                       max_k: int, stream=None) -> None:
    """mtp_verify without a context and without any device allocation (for
    callers whose device memory is owned by a fixed plan or another pool, or
    who cannot take cudaMalloc's device-wide synchronisation); the shape is
    passed directly and the scratch is the library's fixed device array.
    target_logits must be float32 or bfloat16 [num_rows, vocab]; the shape
    checks run before anything reaches the library."""
    B = _check_verify_shapes(target_logits, row_offsets, drafts, num_drafts, accepted, bonus, vocab,
                             "mtp_verify_noalloc")
    code = MTP_DTYPE_BF16 if target_logits.dtype == torch.bfloat16 else MTP_DTYPE_F32
    _check(_clib.mtp_verify_noalloc(_stream(stream), B, int(vocab), code, int(max_k),
                                    _ptr(target_logits, name="target_logits"), int(target_logits.shape[0]),
                                    _ptr(row_offsets, torch.int32, "row_offsets"), _ptr(drafts, torch.int32, "drafts"),
                                    int(drafts.shape[1]), _ptr(num_drafts, torch.int32, "num_drafts"),
                                    _ptr(accepted, torch.int32, "accepted"), _ptr(bonus, torch.int32, "bonus")),
           "mtp_verify_noalloc")


# ------------------------------------------------ speculative loop harness

def mtp_synth_target(ctx: Context, seq_hash: torch.Tensor, last_tok: torch.Tensor, drafts: Optional[torch.Tensor],
                     K: int, sticky_thr: int, logits: torch.Tensor, row_offsets: Optional[torch.Tensor] = None,
                     num_drafts: Optional[torch.Tensor] = None, stream=None) -> None:
    """Synthetic verifier rows (include/mtp.h): seq_hash is an int64 tensor
    holding the 64-bit prefix hashes."""
    B = int(last_tok.shape[0])
    dt = torch_dtype(ctx.cfg.dtype)
    _check(_clib.mtp_synth_target(ctx.handle, _stream(stream), B, int(K), _ptr(num_drafts, torch.int32, "num_drafts"),
                                  _ptr(seq_hash, torch.int64, "seq_hash"),
                                  _ptr(last_tok, torch.int32, "last_tok"), _ptr(drafts, torch.int32, "drafts"),
                                  ctypes.c_uint64(int(sticky_thr)), _ptr(logits, dt, "logits"),
                                  _ptr(row_offsets, torch.int32, "row_offsets")), "mtp_synth_target")


def mtp_loop_advance(ctx: Context, K: int, drafts: Optional[torch.Tensor], accepted: torch.Tensor,
                     bonus: torch.Tensor, seq_hash: torch.Tensor, last_tok: torch.Tensor, positions: torch.Tensor,
                     hidden: torch.Tensor, embeds: torch.Tensor, out_tokens: torch.Tensor, out_len: torch.Tensor,
                     stream=None) -> None:
    B = int(accepted.shape[0])
    dt = torch_dtype(ctx.cfg.dtype)
    _check(_clib.mtp_loop_advance(ctx.handle, _stream(stream), B, int(K), _ptr(drafts, torch.int32, "drafts"),
                                  _ptr(accepted, torch.int32, "accepted"), _ptr(bonus, torch.int32, "bonus"),
                                  _ptr(seq_hash, torch.int64, "seq_hash"), _ptr(last_tok, torch.int32, "last_tok"),
                                  _ptr(positions, torch.int32, "positions"), _ptr(hidden, dt, "hidden"),
                                  _ptr(embeds, dt, "embeds"), _ptr(out_tokens, torch.int32, "out_tokens"),
                                  _ptr(out_len, torch.int32, "out_len"), int(out_tokens.shape[1])),
           "mtp_loop_advance")


def mtp_draft_confidence(ctx: Context, logits: torch.Tensor, tau: float, conf: torch.Tensor,
                         num_drafts: Optional[torch.Tensor] = None, stream=None) -> None:
    """conf [B, K] = probability of each draft step's argmax under logits
    [B, K, V] (fp32); num_drafts [B] = leading run with conf > tau."""
    B, K = int(logits.shape[0]), int(logits.shape[1])
    _check(_clib.mtp_draft_confidence(ctx.handle, _stream(stream), B, K, _ptr(logits, torch.float32, "logits"),
                                      float(tau), _ptr(conf, torch.float32, "conf"),
                                      _ptr(num_drafts, torch.int32, "num_drafts")), "mtp_draft_confidence")


def mtp_adapt_k(K: int, accepted: int, drafted: int, k_min: int, k_max: int) -> int:
    return int(_clib.mtp_adapt_k(int(K), int(accepted), int(drafted), int(k_min), int(k_max)))


class SpecLoop:
    """Device state and scratch of mtp_spec_loop for B requests, K drafts per
    step (K = 0: plain greedy decoding with the verifier), out_cap tokens;
    conf_threshold > 0 proposes only the leading confident drafts."""

    def __init__(self, ctx: Context, B: int, K: int, sticky_thr: int, out_cap: int, device="cuda",
                 conf_threshold: float = 0.0):
        dt = torch_dtype(ctx.cfg.dtype)
        H, V = ctx.cfg.hidden, ctx.cfg.vocab
        i32 = dict(dtype=torch.int32, device=device)
        self.B, self.K, self.sticky_thr = B, K, int(sticky_thr)
        self.seq_hash = torch.zeros(B, dtype=torch.int64, device=device)
        self.last_tok = torch.zeros(B, **i32)
        self.positions = torch.zeros(B, **i32)
        self.hidden = torch.zeros((B, H), dtype=dt, device=device)
        self.embeds = torch.zeros((B, H), dtype=dt, device=device)
        self.drafts = torch.zeros((B, max(K, 1)), **i32)
        self.accepted = torch.zeros(B, **i32)
        self.bonus = torch.zeros(B, **i32)
        self.num_drafts = torch.zeros(B, **i32)
        self.row_offsets = torch.zeros(B + 1, **i32)
        self.target_logits = torch.zeros((B * (K + 1), V), dtype=dt, device=device)
        self.out_tokens = torch.zeros((B, out_cap), **i32)
        self.out_len = torch.zeros(B, **i32)
        self.conf_threshold = float(conf_threshold)
        on = conf_threshold > 0 and K > 0
        self.draft_logits = torch.zeros((B, K, V) if on else (1,), dtype=torch.float32, device=device)
        self.conf = torch.zeros((B, K) if on else (1,), dtype=torch.float32, device=device)

    def struct(self) -> MTPLoop:
        return MTPLoop(self.B, self.K, self.sticky_thr, self.seq_hash.data_ptr(), self.last_tok.data_ptr(),
                       self.positions.data_ptr(), self.hidden.data_ptr(), self.embeds.data_ptr(),
                       self.drafts.data_ptr(), self.accepted.data_ptr(), self.bonus.data_ptr(),
                       self.num_drafts.data_ptr(), self.row_offsets.data_ptr(), self.target_logits.data_ptr(),
                       self.out_tokens.data_ptr(), self.out_len.data_ptr(), int(self.out_tokens.shape[1]),
                       self.conf_threshold, self.draft_logits.data_ptr(), self.conf.data_ptr())


def mtp_spec_loop(ctx: Context, kv: Optional[KVCache], loop: SpecLoop, iters: int, stream=None) -> None:
    st = loop.struct()
    kvs = kv.struct() if kv is not None else None
    _check(_clib.mtp_spec_loop(ctx.handle, _stream(stream), ctypes.byref(kvs) if kvs is not None else None,
                               ctypes.byref(st), int(iters)), "mtp_spec_loop")


class TreeDraft:
    """Buffers of tree drafting for B requests (branching, depth, n_assist);
    ``scratch_blocks`` is an int32 device tensor of free block ids of the cache
    pool ((depth-1) * B * branching * 2 of them)."""

    def __init__(self, ctx: Context, B: int, branching: int, depth: int, n_assist: int, max_blocks: int,
                 scratch_blocks: Optional[torch.Tensor], device="cuda"):
        n = int(_clib.mtp_tree_workspace_bytes(ctx.handle, B, branching, depth, n_assist, max_blocks))
        if n == 0:
            raise MTPError(MTP_ERR_INVALID, "mtp_tree_workspace_bytes")
        self.B, self.branching, self.depth, self.n_assist = B, branching, depth, n_assist
        self.ws = torch.empty(n, dtype=torch.uint8, device=device)
        self.scratch_blocks = scratch_blocks
        i32 = dict(dtype=torch.int32, device=device)
        self.tokens = torch.zeros((B, n_assist), **i32)
        self.parents = torch.zeros((B, n_assist), **i32)
        self.depths = torch.zeros((B, n_assist), **i32)

    def struct(self) -> MTPTree:
        sb = self.scratch_blocks.data_ptr() if self.scratch_blocks is not None else None
        return MTPTree(self.B, self.branching, self.depth, self.n_assist, sb, self.ws.data_ptr(),
                       int(self.ws.numel()), self.tokens.data_ptr(), self.parents.data_ptr(), self.depths.data_ptr())


def mtp_draft_tree(ctx: Context, hidden: torch.Tensor, embeds: torch.Tensor, positions: torch.Tensor, kv: KVCache,
                   tree: TreeDraft, stream=None) -> None:
    dt = torch_dtype(ctx.cfg.dtype)
    kvs, ts = kv.struct(), tree.struct()
    _check(_clib.mtp_draft_tree(ctx.handle, _stream(stream), _ptr(hidden, dt, "hidden"), _ptr(embeds, dt, "embeds"),
                                _ptr(positions, torch.int32, "positions"), ctypes.byref(kvs), ctypes.byref(ts)),
           "mtp_draft_tree")


def mtp_synth_target_tree(ctx: Context, tree: TreeDraft, seq_hash: torch.Tensor, last_tok: torch.Tensor,
                          sticky_thr: int, logits: torch.Tensor, row_offsets: Optional[torch.Tensor] = None,
                          stream=None) -> None:
    ts = tree.struct()
    _check(_clib.mtp_synth_target_tree(ctx.handle, _stream(stream), ctypes.byref(ts),
                                       _ptr(seq_hash, torch.int64, "seq_hash"), _ptr(last_tok, torch.int32, "last_tok"),
                                       ctypes.c_uint64(int(sticky_thr)), _ptr(logits, torch_dtype(ctx.cfg.dtype), "logits"),
                                       _ptr(row_offsets, torch.int32, "row_offsets")), "mtp_synth_target_tree")


def mtp_verify_tree(ctx: Context, tree: TreeDraft, target_logits: torch.Tensor, accepted: torch.Tensor,
                    bonus: torch.Tensor, path_tokens: torch.Tensor, stream=None) -> None:
    ts = tree.struct()
    _check(_clib.mtp_verify_tree(ctx.handle, _stream(stream), ctypes.byref(ts),
                                 _ptr(target_logits, torch_dtype(ctx.cfg.dtype), "target_logits"),
                                 _ptr(accepted, torch.int32, "accepted"), _ptr(bonus, torch.int32, "bonus"),
                                 _ptr(path_tokens, torch.int32, "path_tokens")), "mtp_verify_tree")


def mtp_tree_commit(ctx: Context, kv: KVCache, tree: TreeDraft, accepted: torch.Tensor, stream=None) -> None:
    kvs, ts = kv.struct(), tree.struct()
    _check(_clib.mtp_tree_commit(ctx.handle, _stream(stream), ctypes.byref(kvs), ctypes.byref(ts),
                                 _ptr(accepted, torch.int32, "accepted")), "mtp_tree_commit")


def mtp_tree_loop(ctx: Context, kv: KVCache, loop: SpecLoop, tree: TreeDraft, iters: int, stream=None) -> None:
    kvs, ls, ts = kv.struct(), loop.struct(), tree.struct()
    _check(_clib.mtp_tree_loop(ctx.handle, _stream(stream), ctypes.byref(kvs), ctypes.byref(ls), ctypes.byref(ts),
                               int(iters)), "mtp_tree_loop")


def mtp_quantize_int4_g64(w: torch.Tensor, q: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                          stream=None) -> None:
    """INT4 asymmetric group-64 quantization of a bf16 matrix [rows, cols]:
    q [rows, cols/2] uint8, scales [rows, cols/64] fp16 (or int16 bits),
    zeros [rows, cols/64] uint8."""
    rows, cols = int(w.shape[0]), int(w.shape[1])
    _check(_clib.mtp_quantize_int4_g64(_stream(stream), _ptr(w, name="w"), rows, cols, _ptr(q, name="q"),
                                       _ptr(scales, name="scales"), _ptr(zeros, name="zeros")),
           "mtp_quantize_int4_g64")


def mtp_quantize_int8_rows(w: torch.Tensor, q: torch.Tensor, scales: torch.Tensor, stream=None) -> None:
    """INT8 symmetric per-row quantization of a bf16 matrix [rows, cols]:
    q [rows, cols] int8, scales [rows] fp16 (or int16 bits)."""
    rows, cols = int(w.shape[0]), int(w.shape[1])
    _check(_clib.mtp_quantize_int8_rows(_stream(stream), _ptr(w, name="w"), rows, cols, _ptr(q, name="q"),
                                        _ptr(scales, name="scales")), "mtp_quantize_int8_rows")


def mtp_kv_commit(ctx: Context, kv: KVCache, n_keep: torch.Tensor, stream=None) -> None:
    kvs = kv.struct()
    _check(_clib.mtp_kv_commit(ctx.handle, _stream(stream), int(kv.seq_len.shape[0]), ctypes.byref(kvs),
                              _ptr(n_keep, torch.int32, "n_keep")), "mtp_kv_commit")


def mtp_kv_commit_accepted(ctx: Context, kv: KVCache, accepted: torch.Tensor, extra: int = 1, stream=None) -> None:
    kvs = kv.struct()
    _check(_clib.mtp_kv_commit_accepted(ctx.handle, _stream(stream), int(kv.seq_len.shape[0]), ctypes.byref(kvs),
                                       _ptr(accepted, torch.int32, "accepted"), int(extra)), "mtp_kv_commit_accepted")


def mtp_kv_rollback(ctx: Context, kv: KVCache, stream=None) -> None:
    kvs = kv.struct()
    _check(_clib.mtp_kv_rollback(ctx.handle, _stream(stream), int(kv.seq_len.shape[0]), ctypes.byref(kvs)),
           "mtp_kv_rollback")


def mtp_kv_truncate(ctx: Context, kv: KVCache, new_len: torch.Tensor, stream=None) -> None:
    kvs = kv.struct()
    _check(_clib.mtp_kv_truncate(ctx.handle, _stream(stream), int(kv.seq_len.shape[0]), ctypes.byref(kvs),
                                _ptr(new_len, torch.int32, "new_len")), "mtp_kv_truncate")


# -------------------- rotary positions, the 8-bit KV cache, logit processing

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _dev_ptr(ctx: Context, t: Optional[torch.Tensor], dtype, name: str, shape=None) -> Optional[int]:
    """_ptr with the context's device and a shape (None entries: any size)."""
    if t is None:
        return None
    if (t.get_device() == ctx.device and (dtype is None or t.dtype is dtype) and t.is_contiguous()
            and (shape is None or t.shape == shape)):
        return t.data_ptr()
    p = _ptr(t, dtype, name)
    if ctx.device is not None and t.device.index != ctx.device:
        raise ValueError("%s must be on the context's device cuda:%d, got %s" % (name, ctx.device, t.device))
    if shape is not None and (t.dim() != len(shape) or any(w is not None and int(s) != w
                                                           for s, w in zip(t.shape, shape))):
        raise ValueError("%s must be %s, got %s"
                         % (name, ["any" if w is None else w for w in shape], tuple(t.shape)))
    return p


def _row_ptr(ctx: Context, t: torch.Tensor, name: str, rows: int, heads: int):
    """Pointer and row stride of a [rows, heads, head_dim] tensor in the
    context's dtype whose rows are contiguous (a slice of a packed [rows,
    width] projection, say)."""
    hd, dt = ctx.head_dim, ctx.dtype
    if t.get_device() == ctx.device and t.dtype is dt and t.is_contiguous() and t.shape == (rows, heads, hd):
        return t.data_ptr(), heads * hd
    if t.shape != (rows, heads, hd):
        raise ValueError("%s must be [%d, %d, %d], got %s" % (name, rows, heads, hd, tuple(t.shape)))
    if t.dtype is not dt:
        raise ValueError("%s must be %s, got %s" % (name, dt, t.dtype))
    if t.get_device() != ctx.device:
        if not t.is_cuda:
            raise ValueError("%s must be a CUDA tensor" % name)
        raise ValueError("%s must be on the context's device cuda:%s, got %s" % (name, ctx.device, t.device))
    s0, s1, s2 = t.stride()
    if rows and (s2 != 1 or (heads > 1 and s1 != hd) or (rows > 1 and s0 < heads * hd)):
        raise ValueError("%s must have contiguous, non-overlapping rows, got strides %s" % (name, (s0, s1, s2)))
    return t.data_ptr(), (s0 if rows > 1 else heads * hd)


def _ctx_stream(ctx: Context, stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(ctx.device)
    return torch.cuda.current_stream(ctx.device).cuda_stream


class RopeTable(MTPRopeTable):
    """Rotary table (host memory) for mtp_rope and mtp_kv8_append: ``layout``
    "half" or "interleaved", ``scaling`` "none", "linear", "parts" or "yarn"
    (include/mtp.h gives each formula)."""

    LAYOUTS = {"half": MTP_ROPE_HALF, "interleaved": MTP_ROPE_INTERLEAVED}
    SCALINGS = {"none": MTP_ROPE_SCALE_NONE, "linear": MTP_ROPE_SCALE_LINEAR, "parts": MTP_ROPE_SCALE_PARTS,
                "yarn": MTP_ROPE_SCALE_YARN}

    def __init__(self, rotary_dim: int, theta: float = 1e6, layout: str = "half", scaling: str = "none",
                 factor: float = 1.0, original_max_pos: int = 0, low_freq_factor: float = 1.0,
                 high_freq_factor: float = 4.0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                 magnitude: float = 0.0):
        super().__init__()
        if layout not in self.LAYOUTS or scaling not in self.SCALINGS:
            raise ValueError("RopeTable: layout %r, scaling %r" % (layout, scaling))
        p = MTPRopeParams(self.LAYOUTS[layout], int(rotary_dim), self.SCALINGS[scaling], theta, factor,
                          low_freq_factor, high_freq_factor, beta_fast, beta_slow, int(original_max_pos), magnitude)
        _check(_clib.mtp_rope_table_make(ctypes.byref(p), ctypes.byref(self)), "mtp_rope_table_make")


def mtp_set_rope(ctx: Context, rope: RopeTable) -> None:
    """Use the table (half layout, the whole head) for the head's own rotary
    embedding in every later draft; waits for the device's work."""
    _check(_clib.mtp_set_rope(ctx.handle, rope), "mtp_set_rope")


def mtp_rope(ctx: Context, x: torch.Tensor, positions: torch.Tensor, rope: RopeTable,
             out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rotate x [T, heads, head_dim] to ``positions`` [T] into ``out`` (None:
    in place); rows may be strided.  Returns out."""
    out = x if out is None else out
    if x.dim() != 3:
        raise ValueError("x must be [T, heads, head_dim], got %s" % (tuple(x.shape),))
    T, heads = int(x.shape[0]), int(x.shape[1])
    xp, xs = _row_ptr(ctx, x, "x", T, heads)
    op, os_ = (xp, xs) if out is x else _row_ptr(ctx, out, "out", T, heads)
    if T == 0:
        return out
    _check(_clib.mtp_rope(ctx.handle, _ctx_stream(ctx, stream), T, heads, xp, xs,
                          _dev_ptr(ctx, positions, torch.int32, "positions", (T,)), rope, op, os_),
           "mtp_rope")
    return out


@dataclass
class KVCache8:
    """Caller-owned paged 8-bit KV cache (device tensors; mtp_kv8)."""
    k_pool: torch.Tensor        # [num_blocks, n_kv, 16, head_dim] e4m3 codes (uint8 or float8_e4m3fn)
    v_pool: torch.Tensor
    k_scale: torch.Tensor       # [num_blocks, n_kv] float32
    v_scale: torch.Tensor
    block_table: torch.Tensor   # [B, max_blocks] int32
    seq_len: torch.Tensor       # [B] int32
    pending: torch.Tensor       # [B] int32
    arrive: torch.Tensor        # [B] int32, zeroed once

    @classmethod
    def empty(cls, ctx: Context, num_blocks: int, block_table: torch.Tensor) -> "KVCache8":
        """An empty cache of num_blocks blocks for the requests of block_table."""
        c, dev, B = ctx.cfg, block_table.device, int(block_table.shape[0])
        pools = [torch.zeros((num_blocks, c.n_kv_heads, 16, c.head_dim), dtype=torch.uint8, device=dev)
                 for _ in range(2)]
        scales = [torch.zeros((num_blocks, c.n_kv_heads), dtype=torch.float32, device=dev) for _ in range(2)]
        ints = [torch.zeros(B, dtype=torch.int32, device=dev) for _ in range(3)]
        return cls(pools[0], pools[1], scales[0], scales[1], block_table, ints[0], ints[1], ints[2])

    def struct(self, ctx: Context) -> MTPKV8:
        return self._checked_struct(ctx)[0]

    def _checked_struct(self, ctx: Context):
        """(struct, B, n_q, n_kv, head_dim).  The checks run again when a field
        was assigned, has other storage or another size than when they last
        ran (the block table: another shape or layout), and for another
        context."""
        done = self.__dict__.get("_checked")
        if done is not None and done[3] is ctx.cfg and done[4] == ctx.device:
            kp, vp, ks, vs, bt, sl, pe, ar = done[1]
            if done[0] == (kp.data_ptr(), vp.data_ptr(), ks.data_ptr(), vs.data_ptr(), bt.data_ptr(), sl.data_ptr(),
                           pe.data_ptr(), ar.data_ptr(), kp.nbytes, vp.nbytes, ks.nbytes, vs.nbytes, sl.nbytes,
                           pe.nbytes, ar.nbytes, bt.shape) and bt.is_contiguous():
                return done[2]
        c = ctx.cfg
        nb, B = int(self.k_pool.shape[0]), int(self.seq_len.shape[0])
        if self.block_table.dim() != 2:
            raise ValueError("block_table must be [B, max_blocks]")
        pool, per = (nb, c.n_kv_heads, 16, c.head_dim), (nb, c.n_kv_heads)
        for t, name in ((self.k_pool, "k_pool"), (self.v_pool, "v_pool")):
            if t.dtype not in (torch.uint8, torch.float8_e4m3fn):
                raise ValueError("%s must be uint8 or float8_e4m3fn, got %s" % (name, t.dtype))
        i32, f32 = torch.int32, torch.float32
        st = MTPKV8(_dev_ptr(ctx, self.k_pool, None, "k_pool", pool), _dev_ptr(ctx, self.v_pool, None, "v_pool", pool),
                    _dev_ptr(ctx, self.k_scale, f32, "k_scale", per), _dev_ptr(ctx, self.v_scale, f32, "v_scale", per),
                    _dev_ptr(ctx, self.block_table, i32, "block_table", (B, int(self.block_table.shape[1]))),
                    _dev_ptr(ctx, self.seq_len, i32, "seq_len", (B,)),
                    _dev_ptr(ctx, self.pending, i32, "pending", (B,)),
                    _dev_ptr(ctx, self.arrive, i32, "arrive", (B,)), nb, int(self.block_table.shape[1]))
        got = (st, B, int(c.n_q_heads), int(c.n_kv_heads), int(c.head_dim))
        fields = kp, vp, ks, vs, bt, sl, pe, ar = (self.k_pool, self.v_pool, self.k_scale, self.v_scale,
                                                   self.block_table, self.seq_len, self.pending, self.arrive)
        seen = tuple(t.data_ptr() for t in fields) + tuple(t.nbytes for t in (kp, vp, ks, vs, sl, pe, ar)) + (bt.shape,)
        self.__dict__["_checked"] = (seen, fields, got, c, ctx.device)
        return got

    def __setattr__(self, name, value):
        self.__dict__.pop("_checked", None)
        object.__setattr__(self, name, value)

    def __getstate__(self):
        """A copy (copy.deepcopy, pickle) is checked for itself."""
        return {k: v for k, v in self.__dict__.items() if k != "_checked"}


def mtp_kv8_append(ctx: Context, kv: KVCache8, k: torch.Tensor, v: torch.Tensor, row_offsets: torch.Tensor,
                   q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                   positions: Optional[torch.Tensor] = None, rope: Optional[RopeTable] = None, stream=None) -> None:
    """Append the rows of k and v [T, n_kv, head_dim] to the requests' caches
    as pending entries, k rotated by ``rope`` at ``positions`` if given; q
    [T, n_q, head_dim] is rotated by the same table into q_out (None: in
    place).  Rows may be strided."""
    st, B, n_q, n_kv, _ = kv._checked_struct(ctx)
    T = k.shape[0]
    kp, ks = _row_ptr(ctx, k, "k", T, n_kv)
    vp, vs = _row_ptr(ctx, v, "v", T, n_kv)
    qp, qs, qop, qos = None, 0, None, 0
    if q is not None:
        qp, qs = _row_ptr(ctx, q, "q", T, n_q)
        qop, qos = (qp, qs) if q_out is None or q_out is q else _row_ptr(ctx, q_out, "q_out", T, n_q)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if T == 0:
        return
    _check(_clib.mtp_kv8_append(ctx.handle, _ctx_stream(ctx, stream), B, T,
                                _dev_ptr(ctx, row_offsets, torch.int32, "row_offsets", (B + 1,)), kp, ks, vp, vs,
                                _dev_ptr(ctx, positions, torch.int32, "positions", (T,)), rope, qp, qs, qop, qos,
                                st), "mtp_kv8_append")


def mtp_kv8_read(ctx: Context, kv: KVCache8, start: torch.Tensor, row_offsets: torch.Tensor, k_out: torch.Tensor,
                 v_out: torch.Tensor, stream=None) -> None:
    """Entries start[b] .. of each request, as many as it has rows in
    row_offsets, into k_out and v_out [T, n_kv, head_dim] bf16."""
    st, B, _, n_kv, hd = kv._checked_struct(ctx)
    T = k_out.shape[0]
    kp = _dev_ptr(ctx, k_out, torch.bfloat16, "k_out", (T, n_kv, hd))
    vp = _dev_ptr(ctx, v_out, torch.bfloat16, "v_out", (T, n_kv, hd))
    if T == 0:
        return
    _check(_clib.mtp_kv8_read(ctx.handle, _ctx_stream(ctx, stream), B, st,
                              _dev_ptr(ctx, start, torch.int32, "start", (B,)), T,
                              _dev_ptr(ctx, row_offsets, torch.int32, "row_offsets", (B + 1,)), kp, vp),
           "mtp_kv8_read")


def mtp_kv8_commit(ctx: Context, kv: KVCache8, n_keep: torch.Tensor, stream=None) -> None:
    st, B = kv._checked_struct(ctx)[:2]
    _check(_clib.mtp_kv8_commit(ctx.handle, _ctx_stream(ctx, stream), B, st,
                                _dev_ptr(ctx, n_keep, torch.int32, "n_keep", (B,))), "mtp_kv8_commit")


def mtp_kv8_commit_accepted(ctx: Context, kv: KVCache8, accepted: torch.Tensor, extra: int = 1, stream=None) -> None:
    st, B = kv._checked_struct(ctx)[:2]
    _check(_clib.mtp_kv8_commit_accepted(ctx.handle, _ctx_stream(ctx, stream), B, st,
                                         _dev_ptr(ctx, accepted, torch.int32, "accepted", (B,)), int(extra)),
           "mtp_kv8_commit_accepted")


def mtp_kv8_rollback(ctx: Context, kv: KVCache8, stream=None) -> None:
    st, B = kv._checked_struct(ctx)[:2]
    _check(_clib.mtp_kv8_rollback(ctx.handle, _ctx_stream(ctx, stream), B, st), "mtp_kv8_rollback")


def mtp_kv8_truncate(ctx: Context, kv: KVCache8, new_len: torch.Tensor, stream=None) -> None:
    st, B = kv._checked_struct(ctx)[:2]
    _check(_clib.mtp_kv8_truncate(ctx.handle, _ctx_stream(ctx, stream), B, st,
                                  _dev_ptr(ctx, new_len, torch.int32, "new_len", (B,))), "mtp_kv8_truncate")


def mtp_kv8_commit_path(ctx: Context, kv: KVCache8, keep: torch.Tensor, n_keep: torch.Tensor, stream=None) -> None:
    """Keep the pending entries keep[b, :n_keep[b]] (ascending), drop the rest."""
    st, B = kv._checked_struct(ctx)[:2]
    kp = _dev_ptr(ctx, keep, torch.int32, "keep", (B, None))
    _check(_clib.mtp_kv8_commit_path(ctx.handle, _ctx_stream(ctx, stream), B, st, kp,
                                     int(keep.shape[1]), _dev_ptr(ctx, n_keep, torch.int32, "n_keep", (B,))),
           "mtp_kv8_commit_path")


class Attention8Workspace:
    """Scratch of mtp_kv8_attention; calls that may run at the same time need
    one each (graphs that contain such calls included)."""

    def __init__(self, ctx: Context):
        n = int(_clib.mtp_kv8_attention_workspace_bytes(ctx.handle))
        if n == 0:
            raise MTPError(MTP_ERR_INVALID, "mtp_kv8_attention_workspace_bytes")
        self.device, self.bytes = ctx.device, n
        self.ws = torch.empty(n, dtype=torch.uint8, device="cuda:%d" % ctx.device)
        self.ptr = self.ws.data_ptr()


def mtp_kv8_attention(ctx: Context, kv: KVCache8, q: torch.Tensor, row_offsets: torch.Tensor, out: torch.Tensor,
                      ws: Attention8Workspace, max_rows: int, mask: Optional[torch.Tensor] = None,
                      lse: Optional[torch.Tensor] = None, scale: Optional[float] = None, stream=None) -> None:
    """out [T, n_q, head_dim] = attention of the rows q (may be strided) over
    the requests' caches: the rows of request b are its last entries; causal
    among them, or as the bits of mask [T, words] say.  ``max_rows``: at least
    the rows of any request; lse [T, n_q] float32; scale: 1 / sqrt(head_dim)."""
    st, B, n_q, _, hd = kv._checked_struct(ctx)
    T = q.shape[0]
    qp, qs = _row_ptr(ctx, q, "q", T, n_q)
    op = _dev_ptr(ctx, out, ctx.dtype, "out", (T, n_q, hd))
    lp = _dev_ptr(ctx, lse, torch.float32, "lse", (T, n_q))
    words = mask.shape[-1] if mask is not None else 0
    mp = _dev_ptr(ctx, mask, torch.int32, "mask", (T, words))
    if ws.device != ctx.device:
        raise ValueError("the workspace belongs to cuda:%s" % ws.device)
    if T == 0:
        return
    _check(_clib.mtp_kv8_attention(ctx.handle, _ctx_stream(ctx, stream), B, T,
                                   _dev_ptr(ctx, row_offsets, torch.int32, "row_offsets", (B + 1,)), max_rows,
                                   qp, qs, st, mp, words, hd ** -0.5 if scale is None else scale, op, lp, ws.ptr,
                                   ws.bytes), "mtp_kv8_attention")


class Draft8Workspace:
    """Scratch of mtp_draft_kv8.  Drafts of one context share its activations
    too, so they are ordered by the caller, on one workspace or several."""

    def __init__(self, ctx: Context):
        n = int(_clib.mtp_draft_kv8_workspace_bytes(ctx.handle))
        if n == 0:
            raise MTPError(MTP_ERR_INVALID, "mtp_draft_kv8_workspace_bytes")
        self.device, self.bytes = ctx.device, n
        self.ws = torch.empty(n, dtype=torch.uint8, device="cuda:%d" % ctx.device)
        self.ptr = self.ws.data_ptr()


def mtp_draft_kv8(ctx: Context, hidden: torch.Tensor, embeds: torch.Tensor, positions: torch.Tensor, kv: KVCache8,
                  K: int, draft_ids: torch.Tensor, ws: Draft8Workspace, logits: Optional[torch.Tensor] = None,
                  hidden_out: Optional[torch.Tensor] = None, chain_ids: Optional[torch.Tensor] = None,
                  stream=None) -> None:
    """mtp_draft with the head's cache in 8 bits."""
    st, B = kv._checked_struct(ctx)[:2]
    H, V, dt, i32, f32 = int(ctx.cfg.hidden), ctx.vocab, ctx.dtype, torch.int32, torch.float32
    if ws.device != ctx.device:
        raise ValueError("the workspace belongs to cuda:%s" % ws.device)
    _check(_clib.mtp_draft_kv8(ctx.handle, _ctx_stream(ctx, stream), B, _dev_ptr(ctx, hidden, dt, "hidden", (B, H)),
                               _dev_ptr(ctx, embeds, dt, "embeds", (B, H)),
                               _dev_ptr(ctx, positions, i32, "positions", (B,)), st, int(K),
                               _dev_ptr(ctx, chain_ids, i32, "chain_ids", (B, K - 1)),
                               _dev_ptr(ctx, draft_ids, i32, "draft_ids", (B, K)),
                               _dev_ptr(ctx, logits, f32, "logits", (B, K, V)),
                               _dev_ptr(ctx, hidden_out, f32, "hidden_out", (B, H)), ws.ptr, ws.bytes),
           "mtp_draft_kv8")


def mtp_token_counts_add(ctx: Context, counts: torch.Tensor, tokens: torch.Tensor, n_tokens: torch.Tensor,
                         in_prompt: bool = False, stream=None) -> None:
    """Count tokens[b, :n_tokens[b]] in counts [B, vocab] int32 (in_prompt:
    mark them as occurring in the prompt instead)."""
    B = int(n_tokens.shape[0])
    tp = _dev_ptr(ctx, tokens, torch.int32, "tokens", (B, tokens.shape[-1]))
    if int(tokens.shape[1]) == 0:
        return
    _check(_clib.mtp_token_counts_add(ctx.handle, _ctx_stream(ctx, stream), B, tp, int(tokens.shape[1]),
                                      _dev_ptr(ctx, n_tokens, torch.int32, "n_tokens", (B,)), int(bool(in_prompt)),
                                      _dev_ptr(ctx, counts, torch.int32, "counts", (B, ctx.cfg.vocab))),
           "mtp_token_counts_add")


def mtp_logits_process(ctx: Context, logits: torch.Tensor, row_offsets: torch.Tensor,
                       out: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None,
                       drafts: Optional[torch.Tensor] = None, repetition: Optional[torch.Tensor] = None,
                       frequency: Optional[torch.Tensor] = None, presence: Optional[torch.Tensor] = None,
                       bias_offsets: Optional[torch.Tensor] = None, bias_tokens: Optional[torch.Tensor] = None,
                       bias_values: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
                       mask_index: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Penalties (counts [B, vocab], repetition / frequency / presence [B],
    drafts [B, stride]), biases (bias_offsets [B + 1] into bias_tokens and
    bias_values) and bit masks (mask [masks, ceil(vocab / 32)], mask_index
    [rows]) on logits [rows, vocab] into out (None: in place).  Returns out."""
    V, dt, i32, f32 = ctx.vocab, ctx.dtype, torch.int32, torch.float32
    if row_offsets.dim() != 1 or row_offsets.shape[0] < 2:
        raise ValueError("row_offsets must be [B + 1]")
    if (bias_offsets is None) != (bias_tokens is None) or (bias_offsets is None) != (bias_values is None):
        raise ValueError("bias_offsets, bias_tokens and bias_values go together")
    if (mask is None) != (mask_index is None):
        raise ValueError("mask and mask_index go together")
    B, rows = row_offsets.shape[0] - 1, logits.shape[0]
    lp = _dev_ptr(ctx, logits, dt, "logits", (rows, V))
    if out is None:
        out = logits
    op = lp if out is logits else _dev_ptr(ctx, out, dt, "out", (rows, V))
    a = MTPLogitsArgs(B, rows, _dev_ptr(ctx, row_offsets, i32, "row_offsets"), lp, op)
    if counts is not None:
        a.counts = _dev_ptr(ctx, counts, i32, "counts", (B, V))
    if drafts is not None:
        a.drafts_stride = drafts.shape[-1]
        # (drafts of no width have no memory: with counts, any address says that
        # they are given, so that a request's second row is refused)
        a.drafts = _dev_ptr(ctx, drafts, i32, "drafts", (B, a.drafts_stride)) or (a.counts and a.row_offsets)
    one = (B,)
    if repetition is not None:
        a.repetition = _dev_ptr(ctx, repetition, f32, "repetition", one)
    if frequency is not None:
        a.frequency = _dev_ptr(ctx, frequency, f32, "frequency", one)
    if presence is not None:
        a.presence = _dev_ptr(ctx, presence, f32, "presence", one)
    if bias_offsets is not None:
        a.num_bias = n = bias_tokens.numel()
        a.bias_offsets = _dev_ptr(ctx, bias_offsets, i32, "bias_offsets", (B + 1,))
        a.bias_tokens = _dev_ptr(ctx, bias_tokens, i32, "bias_tokens", (n,))
        a.bias_values = _dev_ptr(ctx, bias_values, f32, "bias_values", (n,))
    if mask is not None:
        a.num_masks = n = mask.shape[0]
        a.mask = _dev_ptr(ctx, mask, i32, "mask", (n, (V + 31) // 32))
        a.mask_index = _dev_ptr(ctx, mask_index, i32, "mask_index", (rows,))
    if rows == 0:
        return out
    _check(_clib.mtp_logits_process(ctx.handle, _ctx_stream(ctx, stream), a), "mtp_logits_process")
    return out


def mtp_selftest_wait_timeout(ctx: Context, which: int, stream=None) -> None:
    _check(_clib.mtp_selftest_wait_timeout(ctx.handle, _stream(stream), int(which)), "mtp_selftest_wait_timeout")


def mtp_selftest_bounds(ctx: Context, stream=None) -> None:
    _check(_clib.mtp_selftest_bounds(ctx.handle, _stream(stream)), "mtp_selftest_bounds")


def mtp_get_device_error(ctx: Context) -> int:
    return int(_clib.mtp_get_device_error(ctx.handle))


def mtp_destroy(ctx: Context) -> None:
    ctx.close()


def mtp_status_str(status: int) -> str:
    return _clib.mtp_status_str(int(status)).decode()


def mtp_stream_copy(dst: torch.Tensor, src: torch.Tensor, nbytes: Optional[int] = None, stream=None) -> None:
    n = src.numel() * src.element_size() if nbytes is None else nbytes
    _check(_clib.mtp_stream_copy(_stream(stream), _ptr(dst, name="dst"), _ptr(src, name="src"), n),
           "mtp_stream_copy")


def mtp_stream_read(src: torch.Tensor, nbytes: Optional[int] = None, err_word: Optional[torch.Tensor] = None,
                    stream=None) -> None:
    n = src.numel() * src.element_size() if nbytes is None else nbytes
    _check(_clib.mtp_stream_read(_stream(stream), _ptr(src, name="src"), n, _ptr(err_word, torch.int32, "err_word")),
           "mtp_stream_read")


def mtp_profile_begin(ctx: Context, kernel: int, capacity: int) -> None:
    _check(_clib.mtp_profile_begin(ctx.handle, int(kernel), int(capacity)), "mtp_profile_begin")


def mtp_profile_end(ctx: Context, max_out: int = 1 << 16):
    buf = (ctypes.c_float * max_out)()
    n = ctypes.c_int(0)
    _check(_clib.mtp_profile_end(ctx.handle, buf, max_out, ctypes.byref(n)), "mtp_profile_end")
    return [float(buf[i]) for i in range(n.value)]


def mtp_launch_count(ctx: Context) -> int:
    return int(_clib.mtp_launch_count(ctx.handle))


MTP_PATH_LM_DEFERRED = 0
MTP_PATH_ATTN_CLUSTER = 1


def mtp_path_count(ctx: Context, path: int) -> int:
    """How often the context took launch-time path `path` (include/mtp.h)."""
    return int(_clib.mtp_path_count(ctx.handle, int(path)))
