"""Elements behind the rotated part of a head, without a norm weight: they come
out as they went in, infinities, NaN and zeros of either sign next to one
another among them, whatever the rotary width leaves of a lane's pairs."""
import numpy as np
import pytest
import torch

from oracle import verifier as V
from test_gpu_kv_rows import close, norm_tol, same_bits
from test_gpu_verifier import M_, clean, context, host, i32, normal

pytestmark = pytest.mark.gpu

ODD = [float("inf"), 0.0, float("nan"), -0.0, 2.0, float("-inf"), -0.0, 0.0, float("nan"), -3.0, float("inf")]


def heads(rng, T, n, hd, rd, dtype):
    x, x64 = normal(rng, (T, n, hd), dtype)
    for t in range(T):
        for h in range(n):
            for e in range(rd, hd):
                if (e + t + h) % 3:
                    x[t, h, e] = ODD[(3 * e + t + h) % len(ODD)]
    return x, x64


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("hd,rd", [(64, 2), (64, 34), (64, 50), (64, 62), (128, 6), (128, 16), (128, 34), (128, 96), (128, 98), (128, 126)])
def test_elements_behind_the_rotated_part_pass(dtype, layout, hd, rd):
    M = M_()
    rng = np.random.default_rng(rd)
    ctx = context(4, 2, hd, dtype, max_batch=2)
    T = 21
    q, q64 = heads(rng, T, 4, hd, rd, dtype)
    k, k64 = heads(rng, T, 2, hd, rd, dtype)
    v = torch.zeros_like(k)
    pos = rng.integers(0, 5000, T)
    rope = M.RopeTable(rd, layout=layout)
    qo, ko = M.mtp_qk_norm_rope(ctx, q, k, positions=i32(pos), rope=rope, q_out=torch.zeros_like(q), k_out=torch.zeros_like(k))
    kv = M.KVCache.empty(ctx, 2, i32([[1], [0]]))
    qa = torch.zeros_like(q)
    M.mtp_kv_append(ctx, kv, k, v, i32([0, 5, 21]), q=q, q_out=qa, positions=i32(pos), rope=rope)
    clean(ctx)
    stored = torch.cat([kv.k_pool[1][:, :5], kv.k_pool[0][:, :16]], 1).transpose(0, 1)
    for got, x, x64 in ((qo, q, q64), (ko, k, k64), (qa, q, q64), (stored, k, k64)):
        a, b = got[..., rd:], x[..., rd:]
        nan = torch.isnan(b)
        assert torch.equal(torch.isnan(a), nan)
        assert same_bits(torch.where(nan, torch.zeros_like(a), a), torch.where(nan, torch.zeros_like(b), b))
        x64 = x64.copy()
        x64[..., rd:] = 0.0
        want = V.rope(x64, pos, layout, rd)
        close(host(got)[..., :rd], want[..., :rd], norm_tol(want, x64, dtype)[..., :rd], "rotated part")
