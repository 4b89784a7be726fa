"""Measured cases of the paged cache in the context's own type: norms and
rotation of query and key heads, appending to the cache, attention of a chunk
of new rows over it, the attention weight that its entries gather, and
eviction by that weight.

``run`` computes an operator's plain form from elementary torch operations
where ``own`` is false and calls the package's entry points where it is true;
``exact`` gives the same outputs from the definitions in 64 bits.  Head shapes
(32 query and 8 key/value heads of 128, and the smaller 64-wide ones) are those
of this repository's configurations.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

BLOCK = 16          # tokens per cache block
EPS = 1e-6          # of the heads' norms


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of 32 requests: norms and rotation of their query and key heads
        dict(name="norm rope decode 32", op="norm", dtype="bf16", tokens=32, n_q=32, n_kv=8, dim=128, rotary=128,
             layout="half", far=131072),
        # a prompt's query and key heads
        dict(name="norm rope prompt 8192", op="norm", dtype="bf16", tokens=8192, n_q=32, n_kv=8, dim=128, rotary=128,
             layout="half", far=131072),
        # one verify step of 32 requests with 5 drafts each: 6 new rows a request into ragged caches
        dict(name="append verify 32x6", op="append", dtype="bf16", batch=32, rows=6, ragged=False, ctx=4096, n_q=32,
             n_kv=8, dim=128, rotary=128, layout="half"),
        # four prompts of unequal length entering empty caches
        dict(name="append prompts 4x4096", op="append", dtype="bf16", batch=4, rows=4096, ragged=True, ctx=0, n_q=32,
             n_kv=8, dim=128, rotary=128, layout="half"),
        # a long prompt in one piece, causal from its first token
        dict(name="attention prompt 8192", op="attention", dtype="bf16", batch=1, rows=8192, ragged=False, ctx=0,
             n_q=32, n_kv=8, dim=128, tree=False),
        # a serving step that mixes chunks of prompts with requests that are nearly done: 1 to 512 new rows each
        dict(name="attention mixed 16x512", op="attention", dtype="bf16", batch=16, rows=512, ragged=True, ctx=4096,
             n_q=32, n_kv=8, dim=128, tree=False),
        # a serving batch decoding one token each, contexts from almost nothing to 8192
        dict(name="attention decode 64 ragged", op="attention", dtype="bf16", batch=64, rows=1, ragged=False, ctx=8192,
             n_q=32, n_kv=8, dim=128, tree=False),
        # verification of packed draft trees in float32, an odd number of rows, some without an ancestor in the tree
        dict(name="attention tree f32", op="attention", dtype="f32", batch=4, rows=33, ragged=True, ctx=1500, n_q=4,
             n_kv=2, dim=64, tree=True),
        # the last 32 rows of four long prompts weigh the prompts' entries before they are thinned out
        dict(name="weights window 4x32", op="weights", dtype="bf16", batch=4, rows=32, ragged=False, ctx=16384, n_q=32,
             n_kv=8, dim=128, tree=False),
        # a decoding batch adds each step's weights to what its entries gathered before
        dict(name="weights decode 32 ragged", op="weights", dtype="bf16", batch=32, rows=1, ragged=False, ctx=4096,
             n_q=32, n_kv=8, dim=128, tree=False),
        # four long prompts thinned out to 2048 entries a head
        dict(name="evict 4x16384 to 2048", op="evict", dtype="bf16", batch=4, ragged=False, ctx=16384, budget=2048,
             sink=4, recent=256, n_q=32, n_kv=8, dim=128),
        # a batch of shorter contexts, some of them below what they may keep, in float32
        dict(name="evict f32 ragged", op="evict", dtype="f32", batch=24, ragged=True, ctx=1100, budget=500, sink=1,
             recent=33, n_q=4, n_kv=2, dim=64),
    ]


def _between(rng, lo, hi):
    """A whole number, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "append", "attention", "attention", "weights", "evict"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dim = rng.choice([64, 128])
    n_kv = rng.choice([1, 2, 4, 8])
    n_q = n_kv * rng.choice([1, 2, 4, 8] if n_kv < 8 else [1, 2, 4])
    heads = dict(n_q=n_q, n_kv=n_kv, dim=dim)
    turn = dict(layout=rng.choice(["half", "interleaved"]),
                rotary=rng.choice([dim, dim, dim // 2, dim - 16, 2 * rng.randint(1, dim // 2)]))
    if op == "norm":
        return dict(op=op, dtype=dtype, tokens=_between(rng, 1, 8192), far=_between(rng, 1000, 1000000), **heads, **turn)
    batch = _between(rng, 1, 64)
    if op == "append":
        return dict(op=op, dtype=dtype, batch=batch, rows=_between(rng, 1, max(1, 8192 // batch)),
                    ragged=rng.random() < 0.5, ctx=rng.choice([0, _between(rng, 1, 3000)]), **heads, **turn)
    if op == "evict":
        ctx = _between(rng, 2, max(40, 65536 // batch))
        budget = _between(rng, 1, ctx)
        sink = rng.randint(0, min(4, budget))
        return dict(op=op, dtype=dtype, batch=batch, ragged=rng.random() < 0.7, ctx=ctx, budget=budget, sink=sink,
                    recent=rng.randint(0, (budget - sink) // 2), **heads)
    most = 256 if dtype == "f32" else 2048 if op == "attention" else 512
    rows = rng.choice([1, 1, 6, _between(rng, 2, max(2, min(most, 8192 // batch)))])
    ctx = _between(rng, 1, max(2, min(65536, 200000 // batch, (1 << 24) // (batch * rows))))
    return dict(op=op, dtype=dtype, batch=batch, rows=rows, ragged=rows > 1 and rng.random() < 0.5, ctx=ctx,
                tree=1 < rows <= 256 and rng.random() < 0.3, **heads)


# ------------------------------------------------------------------ inputs

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) * 7919 + 29)
    return g


def _normal(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _offsets(counts):
    return torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(counts, 0)]).to(torch.int32)


def _lengths(case):
    """New rows and earlier entries of each request: part of a case's sizes, so the same for every seed."""
    h = _gen(sum(v for v in case.values() if isinstance(v, int)), "cpu")
    B, rows = case["batch"], case.get("rows", 0)
    new = torch.randint(1, rows + 1, (B,), generator=h) if case["ragged"] and rows else torch.full((B,), rows)
    if case["op"] == "append" or (B > 1 and (case["op"] != "evict" or case["ragged"])):
        # an evicted cache holds an entry at least
        return new, torch.randint(1 if case["op"] == "evict" else 0, case["ctx"] + 1, (B,), generator=h)
    return new, torch.full((B,), case["ctx"])


def _table(g, need, spare=3):
    """A block table in a shuffled order, and how many blocks a pool has for it."""
    width, total = max(1, int(need.max())), max(1, int(need.sum()))
    order = torch.randperm(total + spare, generator=g, device="cuda")[:total].to(torch.int32)
    table = torch.zeros((len(need), width), dtype=torch.int32, device="cuda")
    held = torch.arange(width, device="cuda")[None] < need.cuda()[:, None]
    table[held] = order[:int(need.sum())]
    return table, total + spare, held


def _cache(case, g, lens, new):
    """A paged cache holding lens[b] entries a request and room for new[b] more; slots that nothing holds are zero."""
    n_kv, dim, dt = case["n_kv"], case["dim"], _dtype(case)
    table, blocks, held = _table(g, (lens + new + BLOCK - 1) // BLOCK)
    filled = torch.zeros(blocks, dtype=torch.int64, device="cuda")
    fill = (lens.cuda()[:, None] - BLOCK * torch.arange(table.shape[1], device="cuda")[None]).clamp(0, BLOCK)
    filled[table[held].long()] = fill[held]
    live = (torch.arange(BLOCK, device="cuda")[None] < filled[:, None])[:, None, :, None]
    pools = [(torch.randn((blocks, n_kv, BLOCK, dim), generator=g, device="cuda") * live).to(dt) for _ in range(2)]
    zero = torch.zeros(len(lens), dtype=torch.int32, device="cuda")
    return dict(k_pool=pools[0], v_pool=pools[1], table=table, seq_len=lens.to(torch.int32).cuda(),
                pending=zero, arrive=zero.clone(), live=live[:, :, :, 0])


def _norm_weights(case, g):
    return [(1 + 0.2 * _normal(g, (case["dim"],))).to(_dtype(case)) for _ in range(2)]


def _inputs(case, seed):
    g, h = _gen(seed), _gen(seed, "cpu")
    dt, op, n_q, n_kv, dim = _dtype(case), case["op"], case["n_q"], case["n_kv"], case["dim"]
    s = {}
    if op == "norm":
        T = case["tokens"]
        s.update(q=_normal(g, (T, n_q, dim), dt) * 3, k=_normal(g, (T, n_kv, dim), dt) * 3,
                 positions=torch.randint(0, case["far"], (T,), generator=g, device="cuda", dtype=torch.int32))
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        s["q_weight"], s["k_weight"] = _norm_weights(case, g)
        return s
    new, lens = _lengths(case)
    T = int(new.sum())
    if op == "evict":
        s["cache"] = c = _cache(case, g, lens, new)
        # gathered weights are spread over magnitudes, and many entries have none at all
        w = torch.exp(3 * _normal(g, (c["k_pool"].shape[0], n_kv, BLOCK)) - 4)
        w = w * (torch.rand(w.shape, generator=g, device="cuda") > 0.15)
        s["weights"] = w * c["live"]
        s["budget"] = torch.full((case["batch"],), case["budget"], dtype=torch.int32, device="cuda")
        table, blocks, _ = _table(g, torch.full((case["batch"],), -(-case["budget"] // BLOCK)))
        zero = torch.zeros(case["batch"], dtype=torch.int32, device="cuda")
        s["into"] = dict(k_pool=torch.zeros((blocks, n_kv, BLOCK, dim), dtype=dt, device="cuda"), table=table,
                         v_pool=torch.zeros((blocks, n_kv, BLOCK, dim), dtype=dt, device="cuda"), seq_len=zero,
                         pending=zero.clone())
        s["into_weights"] = torch.zeros((blocks, n_kv, BLOCK), device="cuda")
        s["kept"] = torch.zeros((case["batch"], n_kv, table.shape[1] * BLOCK), dtype=torch.int32, device="cuda")
        return s
    s.update(row_offsets=_offsets(new).cuda(), q=_normal(g, (T, n_q, dim), dt))
    if op == "append":
        s["cache"] = _cache(case, g, lens, new)
        s["k"], s["v"] = _normal(g, (T, n_kv, dim), dt), _normal(g, (T, n_kv, dim), dt)
        s["q_out"] = torch.empty_like(s["q"])
        s["q_weight"], s["k_weight"] = _norm_weights(case, g)
        s["positions"] = torch.cat([torch.arange(a, a + n) for a, n in zip(lens.tolist(), new.tolist())]).int().cuda()
        return s
    # the rows' own entries are in the cache already, behind lens[b] committed ones
    s["cache"] = _cache(case, g, lens + new, torch.zeros_like(new))
    s["cache"]["seq_len"], s["cache"]["pending"] = lens.int().cuda(), new.int().cuda()
    if case["tree"]:
        # each node's parent is an earlier node or none; a node sees itself and its ancestors
        words = (case["rows"] + 31) // 32
        bits = torch.zeros((T, words * 32), dtype=torch.bool)
        at = 0
        for n in new.tolist():
            up = [-1] + [int(torch.randint(-1, i, (1,), generator=h)) for i in range(1, n)]
            for i in range(n):
                if up[i] >= 0:
                    bits[at + i] = bits[at + up[i]]
                bits[at + i, i] = True
            at += n
        packed = (bits.view(T, words, 32).long() << torch.arange(32, dtype=torch.int64)).sum(-1)
        s["mask"] = torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).int().cuda()
    if op == "attention":
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((T, n_q), dtype=torch.float32, device="cuda")
    else:
        s["lse"] = _softmax_parts(case, s)[2]
        blocks = s["cache"]["k_pool"].shape[0]
        s["weights"] = torch.rand((blocks, n_kv, BLOCK), generator=g, device="cuda") * s["cache"]["live"]
    return s


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = dict(case)
    if own:
        state.update(_handles(case, state))
    return state


def _handles(case, state):
    """What a program that uses the package keeps: the context, the caches' handles, the rotary table, a workspace."""
    import mtp_self_speculative_gb300 as M
    cfg = M.make_config(hidden=256, n_q_heads=case["n_q"], n_kv_heads=case["n_kv"], head_dim=case["dim"], ffn=256,
                        vocab=1, dtype=case["dtype"], max_batch=case.get("batch", 1))
    got = dict(M=M, ctx=M.mtp_init(cfg))
    if "rotary" in case:
        got["rope"] = M.RopeTable(case["rotary"], theta=1e6, layout=case["layout"])
    for name, c in (("kv", state.get("cache")), ("kv_into", state.get("into"))):
        if c is not None:
            got[name] = M.KVCache(c["k_pool"], c["v_pool"], c["table"], c["seq_len"], c["pending"], c.get("arrive"))
    if case["op"] == "attention":
        got["ws"] = M.AttentionWorkspace(got["ctx"])
    return got


# ----------------------------------------------------------------- passes

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        M, ctx = s["M"], s["ctx"]
        if op == "norm":
            M.mtp_qk_norm_rope(ctx, s["q"], s["k"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                               positions=s["positions"], rope=s["rope"], q_out=s["q_out"], k_out=s["k_out"])
            return dict(q=s["q_out"], k=s["k_out"])
        c = s["cache"]
        if op == "append":
            c["pending"].zero_()
            M.mtp_kv_append(ctx, s["kv"], s["k"], s["v"], s["row_offsets"], q=s["q"], q_out=s["q_out"],
                            positions=s["positions"], rope=s["rope"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                            eps=EPS)
            return dict(q=s["q_out"], k_pool=c["k_pool"], v_pool=c["v_pool"], pending=c["pending"])
        if op == "attention":
            M.mtp_kv_attention(ctx, s["kv"], s["q"], s["row_offsets"], s["out"], s["ws"], max_rows=case["rows"],
                               mask=s.get("mask"), lse=s["lse"])
            return dict(out=s["out"], lse=s["lse"])
        if op == "weights":
            M.mtp_kv_attention_weights(ctx, s["kv"], s["q"], s["row_offsets"], s["lse"], s["weights"],
                                       max_rows=case["rows"], mask=s.get("mask"))
            return s["weights"]
        M.mtp_kv_evict(ctx, s["kv"], s["weights"], s["budget"], s["kv_into"], s["into_weights"], s["kept"],
                       sink=case["sink"], recent=case["recent"])
    elif op == "norm":
        return dict(q=_plain_turn(case, s["q"], s["q_weight"], s["positions"]),
                    k=_plain_turn(case, s["k"], s["k_weight"], s["positions"]))
    elif op == "append":
        return _plain_append(case, s)
    elif op == "attention":
        return _plain_attention(case, s)
    elif op == "weights":
        return _plain_weights(case, s)
    else:
        _plain_evict(case, s)
    n = s["into"]
    return dict(k_pool=n["k_pool"], v_pool=n["v_pool"], weights=s["into_weights"], kept=s["kept"], length=n["seq_len"])


def _plain_turn(case, x, weight, positions):
    """Norm over each head and rotation, in float32; the angles in 64 bits, as far positions need."""
    r = case["rotary"]
    f = torch.exp(torch.arange(r // 2, device="cuda", dtype=torch.float64) * (-2.0 * math.log(1e6) / r))
    angle = positions.double()[:, None] * f[None]
    c, s = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    y = x.float()
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * weight.float()
    if case["layout"] == "half":
        a, b = y[..., :r // 2], y[..., r // 2:r]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([turned, y[..., r:]], -1).to(x.dtype)


def _rows(s):
    """The request, and the place within its rows, of each row."""
    off = s["row_offsets"].long()
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(off, t, right=True) - 1
    return b, t - off[b]


def _plain_append(case, s):
    c = s["cache"]
    c["pending"].zero_()
    b, i = _rows(s)
    slot = (c["seq_len"] + c["pending"]).long()[b] + i
    block, at = c["table"].long()[b, slot // BLOCK], slot % BLOCK
    c["k_pool"][block, :, at] = _plain_turn(case, s["k"], s["k_weight"], s["positions"])
    c["v_pool"][block, :, at] = s["v"]
    c["pending"] += s["row_offsets"][1:] - s["row_offsets"][:-1]
    return dict(q=_plain_turn(case, s["q"], s["q_weight"], s["positions"]), k_pool=c["k_pool"], v_pool=c["v_pool"],
                pending=c["pending"])


def _gathered(c, pool):
    """A pool's entries as [B, n_kv, slots, dim] in float32."""
    return c[pool][c["table"].long()].float().transpose(1, 2).flatten(2, 3)


def _softmax_parts(case, s):
    """Scores [B, n_kv, rows x G, slots] (-inf where a row does not see a slot), their maxima, and each row's
    logarithm of the softmax sum."""
    c, G = s["cache"], case["n_q"] // case["n_kv"]
    B, rows, n_kv, dim = case["batch"], case["rows"], case["n_kv"], case["dim"]
    b, i = _rows(s)
    q = torch.zeros((B, rows, n_kv, G, dim), dtype=torch.float32, device="cuda")
    q[b, i] = s["q"].float().view(-1, n_kv, G, dim)
    k = _gathered(c, "k_pool")
    score = (q.permute(0, 2, 1, 3, 4).reshape(B, n_kv, rows * G, dim) @ k.transpose(2, 3)).mul_(1 / math.sqrt(dim))
    unseen = ~_seen(case, s, k.shape[2])
    score.view(B, n_kv, rows, G, -1).masked_fill_(unseen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    lse = (top + torch.log(torch.exp(score - top).sum(-1, keepdim=True))).view(B, n_kv, rows, G)
    return score, top, lse.permute(0, 2, 1, 3)[b, i].flatten(1, 2).contiguous()


def _seen(case, s, slots):
    """Which slots each of the B x rows query rows may look at: [B, rows, slots]."""
    c, rows = s["cache"], case["rows"]
    count = (s["row_offsets"][1:] - s["row_offsets"][:-1]).long()
    base = ((c["seq_len"] + c["pending"]).long() - count)[:, None, None]
    at = torch.arange(slots, device="cuda")[None, None]
    if "mask" not in s:
        return at <= base + torch.arange(rows, device="cuda")[None, :, None]
    bits = ((s["mask"][:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1).flatten(1).bool()
    row = (s["row_offsets"][:-1].long()[:, None] + torch.arange(rows, device="cuda")[None]).clamp(max=bits.shape[0] - 1)
    j = (at - base).clamp(0, bits.shape[1] - 1).expand(-1, rows, -1)
    return (at < base) | (bits[row].gather(2, j) & (at >= base) & (at < base + count[:, None, None]))


def _plain_attention(case, s):
    G, n_kv = case["n_q"] // case["n_kv"], case["n_kv"]
    b, i = _rows(s)
    score, top, lse = _softmax_parts(case, s)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = (p @ _gathered(s["cache"], "v_pool")) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.view(case["batch"], n_kv, case["rows"], G, -1).permute(0, 2, 1, 3, 4)[b, i].flatten(1, 2)
    return dict(out=o.to(_dtype(case)), lse=lse)


def _plain_weights(case, s):
    c, G, n_kv = s["cache"], case["n_q"] // case["n_kv"], case["n_kv"]
    B, rows = case["batch"], case["rows"]
    b, i = _rows(s)
    score = _softmax_parts(case, s)[0]
    lse = torch.full((B, rows, n_kv, G), math.inf, device="cuda")     # rows that a request does not have weigh nothing
    lse[b, i] = s["lse"].view(-1, n_kv, G)
    p = torch.exp(score - lse.permute(0, 2, 1, 3).reshape(B, n_kv, rows * G, 1)).sum(2)      # [B, n_kv, slots]
    length = (c["seq_len"] + c["pending"]).long()
    base = length - (s["row_offsets"][1:] - s["row_offsets"][:-1]).long()
    slot = torch.arange(p.shape[2], device="cuda")
    bb, t = torch.nonzero(slot[None] < length[:, None], as_tuple=True)
    block = c["table"].long()[bb, t // BLOCK]
    old = s["weights"][block, :, t % BLOCK] * (t < base[bb])[:, None]
    s["weights"][block, :, t % BLOCK] = old + p[bb, :, t]
    return s["weights"]


def _plain_evict(case, s):
    c, n = s["cache"], s["into"]
    L = c["seq_len"].long()[:, None, None]
    w = s["weights"][c["table"].long()].transpose(1, 2).flatten(2)                          # [B, n_kv, slots]
    slot = torch.arange(w.shape[2], device="cuda")
    forced = (slot < case["sink"]) | (slot >= L - case["recent"])
    w = torch.where(slot < L, torch.where(forced, torch.full_like(w, math.inf), w), torch.full_like(w, -math.inf))
    first = torch.sort(w, dim=-1, descending=True, stable=True).indices
    keep = torch.minimum(s["budget"].long(), c["seq_len"].long())[:, None, None]
    room = s["kept"].shape[2]
    first = torch.nn.functional.pad(first, (0, max(0, room - first.shape[2])))[..., :room]
    j = torch.arange(room, device="cuda")
    order = torch.where(j < keep, first, torch.full_like(first, 1 << 40)).sort(-1).values
    s["kept"].copy_(torch.where(j < keep, order, torch.full_like(order, -1)))
    bb, g, jj = torch.nonzero((j < keep).expand(s["kept"].shape), as_tuple=True)
    src = order[bb, g, jj]
    frm, to = c["table"].long()[bb, src // BLOCK], n["table"].long()[bb, jj // BLOCK]
    n["k_pool"][to, g, jj % BLOCK] = c["k_pool"][frm, g, src % BLOCK]
    n["v_pool"][to, g, jj % BLOCK] = c["v_pool"][frm, g, src % BLOCK]
    s["into_weights"][to, g, jj % BLOCK] = s["weights"][frm, g, src % BLOCK]
    n["seq_len"].copy_(keep[:, 0, 0])
    n["pending"].zero_()


# ------------------------------------------------------- 64-bit definitions

def _turn(case, x, weight, positions):
    """The norm, and rotary positions as products of complex numbers, in 64 bits."""
    r = case["rotary"]
    f = 1e6 ** (-torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r)
    w = torch.polar(torch.ones((len(positions), 1, r // 2), dtype=torch.float64, device="cuda"),
                    (positions.double()[:, None] * f[None])[:, None])
    x = x.double()
    x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / case["dim"] + EPS) * weight.double()
    if case["layout"] == "half":
        z = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * w
        x[..., :r // 2], x[..., r // 2:r] = z.real, z.imag
    else:
        z = torch.complex(x[..., 0:r:2].contiguous(), x[..., 1:r:2].contiguous()) * w
        x[..., 0:r:2], x[..., 1:r:2] = z.real, z.imag
    return x


def _entries(c, pool, b, length):
    """Request b's first `length` entries of a pool, [length, n_kv, ...]."""
    row = c["table"][b, :(length + BLOCK - 1) // BLOCK].long()
    return pool[row].transpose(1, 2).flatten(0, 1)[:length]


def _scores64(case, s, b, g):
    """Request b's scores of kv head g, [rows, G, entries], -inf where a row does not see an entry."""
    c, G = s["cache"], case["n_q"] // case["n_kv"]
    lo, hi = int(s["row_offsets"][b]), int(s["row_offsets"][b + 1])
    n, L = hi - lo, int(c["seq_len"][b]) + int(c["pending"][b])
    k = _entries(c, c["k_pool"], b, L)[:, g].double()
    z = torch.einsum("rhd,td->rht", s["q"][lo:hi, g * G:(g + 1) * G].double(), k) / math.sqrt(case["dim"])
    see = torch.ones((n, L), dtype=torch.bool, device="cuda").tril(L - n)
    if "mask" in s:
        j = torch.arange(n, device="cuda")
        see[:, L - n:] = ((s["mask"][lo:hi].long()[:, j // 32] >> (j % 32)) & 1).bool()
    return z.masked_fill_(~see[:, None], -math.inf), lo, hi, L


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "norm":
        return dict(q=_turn(case, s["q"], s["q_weight"], s["positions"]),
                    k=_turn(case, s["k"], s["k_weight"], s["positions"]))
    c, G, B, n_kv = s["cache"], case["n_q"] // case["n_kv"], case["batch"], case["n_kv"]
    if op == "append":
        k = _turn(case, s["k"], s["k_weight"], s["positions"])
        pools = [c["k_pool"].double(), c["v_pool"].double()]
        off = s["row_offsets"].tolist()
        for b, start in enumerate(c["seq_len"].tolist()):
            t = torch.arange(start, start + off[b + 1] - off[b], device="cuda")
            block = c["table"][b].long()[t // BLOCK]
            pools[0][block, :, t % BLOCK] = k[off[b]:off[b + 1]]
            pools[1][block, :, t % BLOCK] = s["v"][off[b]:off[b + 1]].double()
        return dict(q=_turn(case, s["q"], s["q_weight"], s["positions"]), k_pool=pools[0], v_pool=pools[1],
                    pending=s["row_offsets"][1:] - s["row_offsets"][:-1])
    if op == "attention":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
        for b in range(B):
            for g in range(n_kv):
                z, lo, hi, L = _scores64(case, s, b, g)
                v = _entries(c, c["v_pool"], b, L)[:, g].double()
                lse[lo:hi, g * G:(g + 1) * G] = torch.logsumexp(z, -1)
                out[lo:hi, g * G:(g + 1) * G] = torch.einsum("rht,td->rhd", torch.softmax(z, -1), v)
        return dict(out=out, lse=lse)
    if op == "weights":
        got = s["weights"].double()
        for b in range(B):
            for g in range(n_kv):
                z, lo, hi, L = _scores64(case, s, b, g)
                add = torch.exp(z - s["lse"][lo:hi, g * G:(g + 1) * G].double()[..., None]).sum((0, 1))
                t = torch.arange(L, device="cuda")
                block = c["table"][b].long()[t // BLOCK]
                got[block, g, t % BLOCK] = torch.where(t < L - (hi - lo), got[block, g, t % BLOCK], 0.0) + add
        return got
    n = s["into"]
    pools = [torch.zeros(n["k_pool"].shape, dtype=torch.float64, device="cuda") for _ in range(2)]
    weights, kept = s["into_weights"].double(), torch.full_like(s["kept"], -1)
    length = torch.minimum(s["budget"], c["seq_len"])
    for b in range(B):
        L, m = int(c["seq_len"][b]), int(length[b])
        w = _entries(c, s["weights"][..., None], b, L)[..., 0]
        for g in range(n_kv):
            order = w[:, g].double().cpu().numpy()
            if m < L:
                # those that stay in any case first, then by weight, then by place
                t = np.arange(L)
                free = (t >= case["sink"]) & (t < L - case["recent"])
                mine = np.sort(np.lexsort((t, -order, free))[:m])
            else:
                mine = np.arange(L)
            j, src = torch.arange(m, device="cuda"), torch.from_numpy(mine).cuda()
            to = n["table"][b].long()[j // BLOCK]
            kept[b, g, :m] = src.int()
            weights[to, g, j % BLOCK] = w[src, g].double()
            for pool, name in zip(pools, ("k_pool", "v_pool")):
                pool[to, g, j % BLOCK] = _entries(c, c[name], b, L)[src, g].double()
    return dict(k_pool=pools[0], v_pool=pools[1], weights=weights, kept=kept, length=length)


# -------------------------------------------------------------------- work

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op, n_q, n_kv, dim = case["op"], case["n_q"], case["n_kv"], case["dim"]
    if op == "norm":
        T = case["tokens"]
        return dict(bytes=2 * T * (n_q + n_kv) * dim * e + 4 * T,
                    flops=T * (n_q + n_kv) * (4 * dim + 3 * case["rotary"]))
    new, lens = _lengths(case)
    T, tokens = int(new.sum()), int((lens + new).sum())
    if op == "append":
        # read q, k and v; write q and the entries
        return dict(bytes=T * (2 * n_q + 4 * n_kv) * dim * e + 4 * T,
                    flops=T * (n_q + n_kv) * (4 * dim + 3 * case["rotary"]))
    if op == "evict":
        # read all weights; read and write what stays: keys, values, weights; write its list
        kept = int(lens.clamp(max=case["budget"]).sum())
        return dict(bytes=n_kv * (4 * tokens + kept * (4 * dim * e + 8)), flops=0)
    pairs = int((new * lens + new * (new + 1) // 2).sum())
    if op == "weights":
        return dict(bytes=tokens * n_kv * (dim * e + 8) + T * n_q * (dim * e + 4), flops=2 * pairs * n_q * dim)
    return dict(bytes=tokens * n_kv * 2 * dim * e + T * n_q * (2 * dim * e + 4), flops=4 * pairs * n_q * dim)
