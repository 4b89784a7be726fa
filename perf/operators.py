"""Measured cases of the serving operators: rotary positions, appending to and
attending over a paged 8-bit key/value cache, and penalties, biases and
grammar masks on logits.

``run`` computes an operator's plain form from elementary torch operations
where ``own`` is false and calls the package's entry points where it is true;
``exact`` gives the same outputs from the definitions in 64 bits.  Head shapes
(32 query and 8 key/value heads of 128, and the smaller 64-wide ones) and the
vocabulary of 151936 are those of this repository's configurations.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 16          # tokens per cache block
LARGEST = 448.0     # largest finite magnitude of the 8-bit format (e4m3)


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of 32 requests: the queries of 32 heads, positions spread over a long context
        dict(name="rope decode 32", op="rope", dtype="bf16", tokens=32, heads=32, dim=128, rotary=128,
             layout="half", scaling="linear", factor=4.0, far=131072),
        # a prompt's queries, frequencies scaled by parts for a longer context than trained
        dict(name="rope prompt 8192", op="rope", dtype="bf16", tokens=8192, heads=32, dim=128, rotary=128,
             layout="half", scaling="parts", factor=8.0, far=131072),
        # a float32 head of odd length that rotates three quarters of each head in adjacent pairs
        dict(name="rope partial f32", op="rope", dtype="f32", tokens=1733, heads=8, dim=64, rotary=48,
             layout="interleaved", scaling="yarn", factor=16.0, far=60000),
        # one verify step of 32 requests with 5 drafts each: 6 new tokens a request into ragged caches
        dict(name="append verify 32x6", op="append", dtype="bf16", batch=32, rows=6, ragged=False, ctx=4096,
             n_q=32, n_kv=8, dim=128, rotary=128, layout="half"),
        # four prompts of unequal length entering empty caches
        dict(name="append prompts 4x2048", op="append", dtype="bf16", batch=4, rows=2048, ragged=True, ctx=0,
             n_q=32, n_kv=8, dim=128, rotary=128, layout="half"),
        # one request decoding one token on a long context
        dict(name="attention 1x32768", op="attention", dtype="bf16", batch=1, rows=1, ctx=32768, n_q=32, n_kv=8,
             dim=128, tree=False),
        # a serving batch decoding, contexts from almost nothing to 8192
        dict(name="attention 64 ragged 8192", op="attention", dtype="bf16", batch=64, rows=1, ctx=8192, n_q=32,
             n_kv=8, dim=128, tree=False),
        # verification of 5 drafts per request, causal among the new rows
        dict(name="attention verify 16x6", op="attention", dtype="bf16", batch=16, rows=6, ctx=4096, n_q=32, n_kv=8,
             dim=128, tree=False),
        # verification of packed draft trees, some rows without an ancestor in them, in float32
        dict(name="attention tree f32", op="attention", dtype="f32", batch=4, rows=33, ctx=1500, n_q=4, n_kv=2,
             dim=64, tree=True),
        # one request's 6 target rows: penalties only
        dict(name="logits 1x6", op="logits", dtype="bf16", batch=1, rows=6, vocab=151936, history=2000, bias=0,
             masks=0),
        # a serving batch's target rows: penalties, biases and a grammar for most rows
        dict(name="logits 64x6 all", op="logits", dtype="bf16", batch=64, rows=6, vocab=151936, history=4000,
             bias=64, masks=96),
        # a small odd vocabulary in float32
        dict(name="logits f32 odd", op="logits", dtype="f32", batch=7, rows=4, vocab=50257, history=300, bias=17,
             masks=5),
    ]


def _between(rng, lo, hi):
    """A whole number, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attention", "attention", "logits"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    dim = rng.choice([64, 128])
    n_kv = rng.choice([1, 2, 4, 8])
    n_q = n_kv * rng.choice([1, 2, 4, 8] if n_kv < 8 else [1, 2, 4])
    layout = rng.choice(["half", "interleaved"])
    rotary = rng.choice([dim, dim, dim // 2, dim - 16, 2 * rng.randint(1, dim // 2)])
    if op == "rope":
        return dict(op=op, dtype=dtype, tokens=_between(rng, 1, 4096), heads=n_q, dim=dim, rotary=rotary,
                    layout=layout, scaling=rng.choice(["none", "linear", "parts", "yarn"]),
                    factor=rng.choice([2.0, 4.0, 8.0, 16.0]), far=_between(rng, 1000, 1000000))
    if op == "append":
        batch = _between(rng, 1, 64)
        return dict(op=op, dtype=dtype, batch=batch, rows=_between(rng, 1, max(1, 4096 // batch)),
                    ragged=rng.random() < 0.5, ctx=rng.choice([0, _between(rng, 1, 3000)]), n_q=n_q, n_kv=n_kv,
                    dim=dim, rotary=rotary, layout=layout)
    if op == "attention":
        batch = _between(rng, 1, 64)
        rows = rng.choice([1, 1, 2, 6, _between(rng, 2, 64)])
        ctx = _between(rng, 1, max(2, 200000 // (batch * max(1, rows // 4))))
        return dict(op=op, dtype=dtype, batch=batch, rows=rows, ctx=ctx, n_q=n_q, n_kv=n_kv, dim=dim,
                    tree=rows > 1 and rng.random() < 0.5)
    batch = _between(rng, 1, 48)
    return dict(op=op, dtype=dtype, batch=batch, rows=rng.choice([1, 2, 6, 9]), vocab=_between(rng, 1000, 151936),
                history=_between(rng, 1, 4000), bias=rng.choice([0, 1, 64, 300]), masks=rng.choice([0, 1, 24]))


# ------------------------------------------------------------------ inputs

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _normal(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(g, lo, hi, shape, dtype=torch.int32):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=dtype)


def _offsets(counts):
    return torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(counts, 0)]).to(torch.int32)


def _rope_arguments(case):
    return dict(layout=case["layout"], rotary_dim=case["rotary"], theta=1e6, scaling=case.get("scaling", "none"),
                factor=case.get("factor", 1.0), original_max_pos=8192, low_freq_factor=1.0, high_freq_factor=4.0,
                beta_fast=32.0, beta_slow=1.0)


def _pow2_at_least(x):
    """The smallest power of two that is not below x (x > 0), 0 for 0; exact for float32."""
    m, e = torch.frexp(x)
    e = torch.where(m == 0.5, e - 1, e)
    return torch.where(x > 0, torch.ldexp(torch.ones_like(x), e.clamp(min=-126)), torch.zeros_like(x))


def _cache(case, g, lens, new):
    """A paged cache holding lens[b] entries a request and room for new[b] more, its blocks in a shuffled order."""
    n_kv, dim = case["n_kv"], case["dim"]
    need = (lens + new + BLOCK - 1) // BLOCK
    width, total = max(1, int(need.max())), max(1, int(need.sum()))
    blocks = total + 3
    order = torch.randperm(blocks, generator=g, device="cuda")[:total].to(torch.int32)
    table = torch.zeros((len(lens), width), dtype=torch.int32, device="cuda")
    held = torch.arange(width, device="cuda")[None] < need.cuda()[:, None]
    table[held] = order
    pools, scales = [], []
    # how many leading tokens of each pool block hold an entry
    filled = torch.zeros(blocks, dtype=torch.int64, device="cuda")
    fill = (lens.cuda()[:, None] - BLOCK * torch.arange(width, device="cuda")[None]).clamp(0, BLOCK)
    filled[table[held].long()] = fill[held]
    live = (torch.arange(BLOCK, device="cuda")[None] < filled[:, None])[:, None, :, None]
    for _ in range(2):
        # entries of unit size, some blocks and heads a few times larger or smaller
        size = torch.exp2(torch.randn((blocks, n_kv, 1, 1), generator=g, device="cuda") * 0.7)
        x = torch.randn((blocks, n_kv, BLOCK, dim), generator=g, device="cuda", dtype=torch.float32)
        x = x * size * live
        s = _pow2_at_least(x.abs().amax((2, 3)) / LARGEST)
        q = torch.where(s[:, :, None, None] > 0, x / s[:, :, None, None], torch.zeros_like(x))
        pools.append(q.to(torch.float8_e4m3fn).view(torch.uint8))
        scales.append(s)
        del x, q
    batch = len(lens)
    return dict(k_pool=pools[0], v_pool=pools[1], k_scale=scales[0], v_scale=scales[1], table=table,
                seq_len=lens.to(torch.int32).cuda(), pending=torch.zeros(batch, dtype=torch.int32, device="cuda"),
                arrive=torch.zeros(batch, dtype=torch.int32, device="cuda"))


def _lengths(case):
    """New rows and earlier entries of each request: part of a case's sizes, so the same for every seed."""
    h = _gen(sum(v for v in case.values() if isinstance(v, int)), "cpu")
    B, rows = case["batch"], case["rows"]
    ragged = case["ragged"] if case["op"] == "append" else case["tree"]
    new = torch.randint(1, rows + 1, (B,), generator=h) if ragged else torch.full((B,), rows)
    if case["op"] == "append":
        return new, torch.randint(0, case["ctx"] + 1, (B,), generator=h)
    lens = torch.randint(0, case["ctx"] + 1, (B,), generator=h) if B > 1 else torch.full((B,), case["ctx"])
    return new, lens


def _inputs(case, seed):
    g, h = _gen(seed), _gen(seed, "cpu")
    dt, op = _dtype(case), case["op"]
    if op == "rope":
        return dict(x=_normal(g, (case["tokens"], case["heads"], case["dim"]), dt),
                    positions=_ints(g, 0, case["far"], (case["tokens"],)))
    if op == "logits":
        B, V, rows = case["batch"], case["vocab"], case["rows"]
        n = B * rows
        # tokens repeat: half of a history comes from 200 common ids
        def some(shape):
            a, b = _ints(g, 0, V, shape), _ints(g, 0, min(200, V), shape)
            return torch.where(torch.rand(shape, generator=g, device="cuda") < 0.5, a, b)
        counts = torch.zeros((B, V), dtype=torch.int32, device="cuda")
        one = torch.ones((B, case["history"]), dtype=torch.int32, device="cuda")
        counts.scatter_add_(1, some((B, case["history"])).long(), one)
        prompt = torch.zeros((B, V), dtype=torch.bool, device="cuda")
        prompt.scatter_(1, some((B, case["history"])).long(), True)
        counts = counts | torch.where(prompt, torch.full_like(counts, -2 ** 31), torch.zeros_like(counts))
        s = dict(x=_normal(g, (n, V), dt) * 3, counts=counts,
                 row_offsets=torch.arange(0, n + 1, rows, dtype=torch.int32, device="cuda"),
                 drafts=some((B, max(1, rows - 1))), out=torch.empty((n, V), dtype=dt, device="cuda"),
                 repetition=1 + torch.rand(B, generator=g, device="cuda"),
                 frequency=torch.rand(B, generator=g, device="cuda") - 0.3,
                 presence=torch.rand(B, generator=g, device="cuda") - 0.3)
        if case["bias"]:
            per = torch.full((B,), case["bias"], dtype=torch.int64)
            s["bias_offsets"] = _offsets(per).cuda()
            s["bias_tokens"] = _ints(g, 0, V, (B * case["bias"],))
            s["bias_values"] = _normal(g, (B * case["bias"],)) * 5
        if case["masks"]:
            words = (V + 31) // 32
            bits = [_ints(g, -2 ** 31, 2 ** 31, (case["masks"], words), torch.int64).to(torch.int32) for _ in range(3)]
            s["mask"] = bits[0] & bits[1] & bits[2]  # an eighth of the vocabulary allowed
            s["mask"][-1] = 0                        # a grammar that allows nothing
            s["mask_index"] = _ints(g, -1, case["masks"], (n,))
        return s
    new, lens = _lengths(case)
    T = int(new.sum())
    s = dict(row_offsets=_offsets(new).cuda(), q=_normal(g, (T, case["n_q"], case["dim"]), dt))
    if op == "append":
        s["cache"] = _cache(case, g, lens, new)
        s["k"] = _normal(g, (T, case["n_kv"], case["dim"]), dt)
        s["v"] = _normal(g, (T, case["n_kv"], case["dim"]), dt)
        s["q_out"] = torch.empty_like(s["q"])
        s["positions"] = torch.cat([torch.arange(a, a + n) for a, n in zip(lens.tolist(), new.tolist())]).int().cuda()
        # the entries to be read back: from the start of the block that the first new one enters
        s["read_start"] = (lens // BLOCK * BLOCK).int().cuda()
        s["read_offsets"] = _offsets(lens % BLOCK + new).cuda()
        n = int((lens % BLOCK + new).sum())
        # bfloat16 holds every value of the cache (4 significant bits times a power of two) exactly
        s["k_out"] = torch.empty((n, case["n_kv"], case["dim"]), dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.empty_like(s["k_out"])
        return s
    # the rows' own entries are in the cache already, behind lens[b] committed ones
    s["cache"] = _cache(case, g, lens + new, torch.zeros_like(new))
    s["cache"]["seq_len"] = lens.int().cuda()
    s["cache"]["pending"] = new.int().cuda()
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((T, case["n_q"]), dtype=torch.float32, device="cuda")
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
        shift = torch.arange(32, dtype=torch.int64)
        packed = (bits.view(T, words, 32).long() << shift).sum(-1)
        s["mask"] = torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).int().cuda()
    return s


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = dict(case)
    if own:
        state.update(_handles(case, state))
    return state


def _handles(case, state):
    """What a program that uses the package keeps: the context, the cache's handle, the rotary table, a workspace."""
    import mtp_self_speculative_gb300 as M
    cfg = M.make_config(hidden=256, n_q_heads=case.get("n_q", case.get("heads", 1)),
                        n_kv_heads=case.get("n_kv", case.get("heads", 1)), head_dim=case.get("dim", 128), ffn=256,
                        vocab=case.get("vocab", 1), dtype=case["dtype"], max_batch=case.get("batch", 1), max_k=100)
    got = dict(M=M, ctx=M.mtp_init(cfg))
    if case["op"] in ("rope", "append"):
        got["rope"] = M.RopeTable(**_rope_arguments(case))
    if "cache" in state:
        c = state["cache"]
        got["kv"] = M.KVCache8(c["k_pool"], c["v_pool"], c["k_scale"], c["v_scale"], c["table"], c["seq_len"],
                               c["pending"], c["arrive"])
    if case["op"] == "attention":
        got["ws"] = M.Attention8Workspace(got["ctx"])
    if case["op"] == "rope":
        got["out"] = torch.empty_like(state["x"])
    return got


# ----------------------------------------------------------------- passes

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        M, ctx = s["M"], s["ctx"]
        if op == "rope":
            M.mtp_rope(ctx, s["x"], s["positions"], s["rope"], s["out"])
            return s["out"]
        if op == "append":
            s["cache"]["pending"].zero_()
            M.mtp_kv8_append(ctx, s["kv"], s["k"], s["v"], s["row_offsets"], q=s["q"], q_out=s["q_out"],
                             positions=s["positions"], rope=s["rope"])
            M.mtp_kv8_read(ctx, s["kv"], s["read_start"], s["read_offsets"], s["k_out"], s["v_out"])
            return dict(q=s["q_out"], k=s["k_out"], v=s["v_out"], pending=s["cache"]["pending"])
        if op == "attention":
            M.mtp_kv8_attention(ctx, s["kv"], s["q"], s["row_offsets"], s["out"], s["ws"], max_rows=case["rows"],
                                mask=s.get("mask"), lse=s["lse"])
            return dict(out=s["out"], lse=s["lse"])
        M.mtp_logits_process(ctx, s["x"], s["row_offsets"], s["out"], counts=s["counts"], drafts=s["drafts"],
                             repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
                             bias_offsets=s.get("bias_offsets"), bias_tokens=s.get("bias_tokens"),
                             bias_values=s.get("bias_values"), mask=s.get("mask"), mask_index=s.get("mask_index"))
        return s["out"]
    if op == "rope":
        return _plain_rope(case, s["x"].float(), s["positions"]).to(s["x"].dtype)
    if op == "append":
        return _plain_append(case, s)
    if op == "attention":
        return _plain_attention(case, s)
    return _plain_logits(case, s)


def _frequencies(case):
    """Angle per position of each rotated pair, in 64 bits, and the factor on the rotated values."""
    a = _rope_arguments(case)
    d, theta, factor = a["rotary_dim"], a["theta"], a["factor"]
    i = torch.arange(d // 2, device="cuda", dtype=torch.float64)
    f = torch.exp(i * (-2.0 * math.log(theta) / d))
    if a["scaling"] == "none":
        return f, 1.0
    if a["scaling"] == "linear":
        return f / factor, 1.0
    if a["scaling"] == "parts":
        turns = a["original_max_pos"] * f / (2 * math.pi)
        keep = ((turns - a["low_freq_factor"]) / (a["high_freq_factor"] - a["low_freq_factor"])).clamp(0, 1)
        return f * keep + f / factor * (1 - keep), 1.0
    at = [d * math.log(a["original_max_pos"] / (b * 2 * math.pi)) / (2 * math.log(theta))
          for b in (a["beta_fast"], a["beta_slow"])]
    lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), d - 1)
    ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
    return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0


def _plain_rope(case, x, positions):
    """x [T, heads, dim] in float32; the angles in 64 bits, as far positions need."""
    r = case["rotary"]
    f, factor = _frequencies(case)
    angle = positions.double()[:, None] * f[None]
    c, s = (torch.cos(angle) * factor).float()[:, None], (torch.sin(angle) * factor).float()[:, None]
    if case["layout"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([turned, x[..., r:]], -1)


def _rows(case, s):
    """The request, and the place within its rows, of each row."""
    off = s["row_offsets"].long()
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(off, t, right=True) - 1
    return b, t - off[b]


def _plain_append(case, s):
    c, dt = s["cache"], _dtype(case)
    n_kv, dim = case["n_kv"], case["dim"]
    c["pending"].zero_()
    b, i = _rows(case, s)
    start = (c["seq_len"] + c["pending"]).long()
    slot = start[b] + i
    # the blocks that take part, as rows of a dense [requests, blocks a request, 16 tokens] window
    first = start // BLOCK
    count = (s["row_offsets"][1:] - s["row_offsets"][:-1]).long()
    width = (case["rows"] + 2 * BLOCK - 2) // BLOCK
    w = torch.arange(width, device="cuda")[None]
    used = w < ((start + count + BLOCK - 1) // BLOCK - first)[:, None]
    held = c["table"].shape[1]
    block = c["table"].long().gather(1, (first[:, None] + w).clamp(max=held - 1))
    token = torch.arange(BLOCK, device="cuda")
    old = ((first[:, None] + w)[:, :, None] * BLOCK + token) < start[:, None, None]       # [B, width, 16]
    out = {}
    for name, x in (("k", _plain_rope(case, s["k"].float(), s["positions"])), ("v", s["v"].float())):
        pool, scale = c[name + "_pool"], c[name + "_scale"]
        win = torch.zeros((len(first), width * BLOCK, n_kv, dim), dtype=torch.float32, device="cuda")
        win[b, slot - first[b] * BLOCK] = x
        win = win.view(len(first), width, BLOCK, n_kv, dim).permute(0, 1, 3, 2, 4)
        was = scale[block]                                                              # [B, width, n_kv]
        before = pool[block].view(torch.float8_e4m3fn).float() * was[..., None, None]
        keeps = old.any(-1)[..., None]
        now = torch.maximum(_pow2_at_least(win.abs().amax((3, 4)) / LARGEST),
                            torch.where(keeps, was, torch.zeros_like(was)))
        win = torch.where(old[:, :, None, :, None], before, win)
        q = torch.where(now[..., None, None] > 0, win / now[..., None, None], torch.zeros_like(win))
        q = q.to(torch.float8_e4m3fn)
        pool[block[used]] = q.view(torch.uint8)[used]
        scale[block[used]] = now[used]
        # the entries read back
        rb, ri = _read_rows(s)
        value = (q.float() * now[..., None, None]).bfloat16().permute(0, 1, 3, 2, 4).reshape(len(first), -1, n_kv, dim)
        out[name] = value[rb, ri]
    c["pending"] += count.int()
    return dict(q=_plain_rope(case, s["q"].float(), s["positions"]).to(dt), k=out["k"], v=out["v"],
                pending=c["pending"])


def _read_rows(s):
    off = s["read_offsets"].long()
    t = torch.arange(s["k_out"].shape[0], device="cuda")
    b = torch.searchsorted(off, t, right=True) - 1
    return b, t - off[b]


def _gathered(c, name, dtype=torch.float32):
    """A cache's values as [B, slots, n_kv, dim]."""
    block = c["table"].long()
    x = c[name + "_pool"].view(torch.float8_e4m3fn)[block].to(dtype) * c[name + "_scale"][block].to(dtype)[..., None, None]
    return x.transpose(2, 3).flatten(1, 2)


def _seen(case, s, slots):
    """Which slots each of the B x rows query rows may look at: [B, rows, slots]."""
    c, rows = s["cache"], case["rows"]
    length = (c["seq_len"] + c["pending"]).long()
    count = (s["row_offsets"][1:] - s["row_offsets"][:-1]).long()
    base = (length - count)[:, None, None]
    at = torch.arange(slots, device="cuda")[None, None]
    if "mask" not in s:
        return at <= base + torch.arange(rows, device="cuda")[None, :, None]
    bits = (s["mask"][:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
    bits = bits.flatten(1).bool()                                                       # [T, words * 32]
    row = (s["row_offsets"][:-1].long()[:, None] + torch.arange(rows, device="cuda")[None]).clamp(max=bits.shape[0] - 1)
    j = (at - base).clamp(0, bits.shape[1] - 1).expand(-1, rows, -1)
    own_rows = bits[row].gather(2, j)
    return (at < base) | (own_rows & (at >= base) & (at < base + count[:, None, None]))


def _plain_attention(case, s):
    dt, G = _dtype(case), case["n_q"] // case["n_kv"]
    B, rows, n_kv, dim = case["batch"], case["rows"], case["n_kv"], case["dim"]
    b, i = _rows(case, s)
    q = torch.zeros((B, rows, n_kv, G, dim), dtype=torch.float32, device="cuda")
    q[b, i] = s["q"].float().view(-1, n_kv, G, dim)
    k, v = _gathered(s["cache"], "k"), _gathered(s["cache"], "v")                       # [B, slots, n_kv, dim]
    slots = k.shape[1]
    q = q.permute(0, 2, 1, 3, 4).reshape(B, n_kv, rows * G, dim)
    score = (q @ k.permute(0, 2, 3, 1)) / math.sqrt(dim)
    seen = _seen(case, s, slots)[:, None, :, None].expand(B, n_kv, rows, G, slots).reshape(score.shape)
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = (p @ v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + torch.log(total)).view(B, n_kv, rows, G)
    o = o.view(B, n_kv, rows, G, dim).permute(0, 2, 1, 3, 4)[b, i].flatten(1, 2)
    return dict(out=o.to(dt), lse=lse.permute(0, 2, 1, 3)[b, i].flatten(1, 2))


def _plain_logits(case, s):
    x = s["x"].float()
    n, V = x.shape
    B, rows = case["batch"], case["rows"]
    x = x.view(B, rows, V)
    count = (s["counts"] & 0x7FFFFFFF)[:, None].expand(B, rows, V).float()
    # row j has the drafts before it behind it
    if rows > 1:
        d = s["drafts"].long()[:, None].expand(B, rows, rows - 1)
        before = torch.arange(rows - 1, device="cuda")[None, None] < torch.arange(rows, device="cuda")[None, :, None]
        count = count.clone().scatter_add_(2, d, before.float().expand(B, rows, rows - 1))
    met = (count > 0) | (s["counts"] < 0)[:, None]
    r, f, p = (s[k][:, None, None] for k in ("repetition", "frequency", "presence"))
    x = torch.where(met, torch.where(x > 0, x / r, x * r), x)
    x = x - f * count - p * (count > 0).float()
    if "bias_offsets" in s:
        b = torch.arange(B, device="cuda").repeat_interleave(case["bias"])
        add = torch.zeros((B, V), dtype=torch.float32, device="cuda")
        add.index_put_((b, s["bias_tokens"].long()), s["bias_values"], accumulate=True)
        x = x + add[:, None]
    x = x.reshape(n, V)
    if "mask" in s:
        bits = ((s["mask"][:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1).bool().flatten(1)[:, :V]
        ok = bits[s["mask_index"].long().clamp(min=0)] | (s["mask_index"] < 0)[:, None]
        x = x.masked_fill(~ok, -math.inf)
    return x.to(_dtype(case))


# ------------------------------------------------------- 64-bit definitions

def _turn(case, x, positions):
    """Rotary positions as products of complex numbers, in 64 bits."""
    r = case["rotary"]
    f, factor = _frequencies(case)
    w = torch.polar(torch.full((len(positions), 1, r // 2), factor, dtype=torch.float64, device="cuda"),
                    (positions.double()[:, None] * f[None])[:, None])
    x = x.double().clone()
    if case["layout"] == "half":
        z = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * w
        x[..., :r // 2], x[..., r // 2:r] = z.real, z.imag
    else:
        z = torch.complex(x[..., 0:r:2].contiguous(), x[..., 1:r:2].contiguous()) * w
        x[..., 0:r:2], x[..., 1:r:2] = z.real, z.imag
    return x


def _nearest8(x):
    """The nearest number of the 8-bit format (4 exponent bits, least exponent -6, 3 mantissa bits), ties to even."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "rope":
        return _turn(case, s["x"], s["positions"])
    if op == "append":
        c = s["cache"]
        off, roff = s["row_offsets"].tolist(), s["read_offsets"].tolist()
        out = dict(q=_turn(case, s["q"], s["positions"]), pending=s["row_offsets"][1:] - s["row_offsets"][:-1])
        for name in ("k", "v"):
            x = _turn(case, s["k"], s["positions"]) if name == "k" else s["v"].double()
            got = torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda")
            for b, start in enumerate(c["seq_len"].tolist()):
                new, lo = x[off[b]:off[b + 1]], start // BLOCK * BLOCK
                row = c["table"][b].long()
                for at in range(lo, start + len(new), BLOCK):
                    j = row[at // BLOCK]
                    had = max(0, start - at)
                    vals = new[max(0, at - start):at + BLOCK - start]
                    was = c[name + "_scale"][j].double() if had else torch.zeros(case["n_kv"], dtype=torch.float64, device="cuda")
                    top = vals.abs().amax((0, 2))
                    scale = torch.maximum(was, torch.exp2(torch.ceil(torch.log2(top / LARGEST))))
                    kept = c[name + "_pool"][j].view(torch.float8_e4m3fn).double() * c[name + "_scale"][j].double()[:, None, None]
                    both = torch.cat([kept.transpose(0, 1)[:had], vals]) / scale[:, None]
                    at_out = roff[b] + at - lo
                    got[at_out:at_out + len(both)] = _nearest8(both) * scale[:, None]
            out[name] = got
        return out
    if op == "attention":
        c, G = s["cache"], case["n_q"] // case["n_kv"]
        off, length = s["row_offsets"].tolist(), (c["seq_len"] + c["pending"]).tolist()
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
        for b in range(case["batch"]):
            n, L = off[b + 1] - off[b], length[b]
            one = {k: c[k] for k in ("k_pool", "v_pool", "k_scale", "v_scale")}
            one["table"] = c["table"][b:b + 1, :(L + BLOCK - 1) // BLOCK]
            k, v = (_gathered(one, x, torch.float64)[0, :L].repeat_interleave(G, 1) for x in ("k", "v"))
            see = torch.ones((n, L), dtype=torch.bool, device="cuda").tril(L - n)
            if "mask" in s:
                words = s["mask"][off[b]:off[b + 1]].long()
                j = torch.arange(n, device="cuda")
                see[:, L - n:] = ((words[:, j // 32] >> (j % 32)) & 1).bool()
            z = torch.einsum("rhd,thd->rht", s["q"][off[b]:off[b + 1]].double(), k) / math.sqrt(case["dim"])
            z = z.masked_fill(~see[:, None], -math.inf)
            lse[off[b]:off[b + 1]] = torch.logsumexp(z, -1)
            out[off[b]:off[b + 1]] = torch.einsum("rht,thd->rhd", torch.softmax(z, -1), v)
        return dict(out=out, lse=lse)
    n, V = s["x"].shape
    off = s["row_offsets"].tolist()
    got = torch.empty((n, V), dtype=torch.float64, device="cuda")
    for b in range(case["batch"]):
        c = (s["counts"][b].long() & 0x7FFFFFFF).double()
        prompt = s["counts"][b] < 0
        bias = torch.zeros(V, dtype=torch.float64, device="cuda")
        if case["bias"]:
            m = slice(b * case["bias"], (b + 1) * case["bias"])
            bias.index_add_(0, s["bias_tokens"][m].long(), s["bias_values"][m].double())
        r, f, p = (s[k][b].double() for k in ("repetition", "frequency", "presence"))
        for j, row in enumerate(range(off[b], off[b + 1])):
            if j:
                c[s["drafts"][b, j - 1].long()] += 1
            z = s["x"][row].double()
            z = torch.where((c > 0) | prompt, torch.maximum(z, z * 0) / r + torch.minimum(z, z * 0) * r, z)
            z = z - f * c - p * torch.sign(c) + bias
            if case["masks"] and int(s["mask_index"][row]) >= 0:
                word = s["mask"][int(s["mask_index"][row])].long()
                v = torch.arange(V, device="cuda")
                z[((word[v // 32] >> (v % 32)) & 1) == 0] = -math.inf
            got[row] = z
    return got


# -------------------------------------------------------------------- work

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * case["heads"]
        return dict(bytes=2 * n * case["dim"] * e + 4 * case["tokens"], flops=3 * n * case["rotary"])
    if op == "append":
        new, lens = _lengths(case)
        T, R = int(new.sum()), int((lens % BLOCK + new).sum())
        q, kv = case["n_q"] * case["dim"], case["n_kv"] * case["dim"]
        # read q, k, v; write q and the codes; read the codes back and write their values
        return dict(bytes=T * (2 * q * e + 2 * kv * (e + 1) + 4) + R * 2 * kv * 3, flops=T * (3 * q + 8 * kv))
    if op == "attention":
        new, lens = _lengths(case)
        T, tokens = int(new.sum()), int((lens + new).sum())
        bytes_ = tokens * case["n_kv"] * (case["dim"] * 2 + 8 / BLOCK) + T * case["n_q"] * (2 * case["dim"] * e + 4)
        pairs = int((new * lens + new * (new + 1) // 2).sum())
        return dict(bytes=bytes_, flops=4 * pairs * case["n_q"] * case["dim"])
    rows, V = case["batch"] * case["rows"], case["vocab"]
    mask = min(case["masks"], rows) * ((V + 31) // 32) * 4
    return dict(bytes=2 * rows * V * e + 4 * case["batch"] * V + mask + 8 * case["batch"] * case["bias"],
                flops=5 * rows * V)
