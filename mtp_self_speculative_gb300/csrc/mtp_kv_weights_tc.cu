// The attention weight that the entries of a paged cache gather, on the tensor
// cores (tcgen05), bf16 heads:
//
//   w[t, g] = (t < first ? w[t, g] : 0) + sum_{r, h} 2^(c s_t - log2 e * lse[r, h]),
//   s_t = q[r, h] . K[t, g] over the rows r that see t and the heads h of g's group.
//
// The entries are the rows of the products (S^T = K Q^T, 128 x 128), so that a
// thread owns an entry and its sum never leaves a register: no reduction across
// threads, no atomics, one order.  A unit is 256 entries of a kv head (two
// tiles of keys, a softmax group each) with all (row, query head) pairs that may
// see them, 128 at a time.  Fourteen warps, one thread block per SM:
//   warps 0-3, 4-7   a group's 128 entries: scores from tensor memory (two
//            buffers each, so that products run under the exponentials), the pairs'
//            lse from shared memory
//   warp 8   finds the units of the block's share and loads their keys, two units
//            in flight
//   warp 9   issues the products
//   warps 10-13  load the pairs' queries and lse, three tiles in flight; a unit with
//            the queries of the one before (decoding, a window) takes them
//            over
// Many rows (128 x 128 exponentials a tile and group at 16 results a cycle, as many
// cycles as the products) are bound by both (a chunk of 2048 rows behind 2048 earlier
// entries 125 us, 410 TFLOP/s); few rows by reading the keys: 32
// decoding rows on 4096 entries at most, 32 query and 8 kv heads of 128, 28 us, 4.8
// TB/s (352 us on the float32 pipe); the last 32 rows of four prompts of 8192 21 us
// (582 us).
#include <math.h>

#include "mtp_kv_tc.cuh"

namespace mtp {

constexpr int kWtThreads = 448;
constexpr int kWtEntries = 256;     // entries of a unit
constexpr int kWtPairs = 128;       // pairs of a tile of queries
constexpr int kWtQ = 3;             // tiles of queries in flight
constexpr int kWtLead = 2;          // tiles that a unit's keys count for in the split

template <int HD>
struct WtShape {
  static constexpr int kHalves = HD / 64;
  static constexpr int kTile = 128 * HD * 2;
  static constexpr int kBytes = (2 * 2 + kWtQ) * kTile;
};

struct WtUnit {
  int b;                 // request, or -1: no more work
  int g, o0, n, L, base;
  int t0;                // the first entry
  int row0, tiles;       // the first row that may see it, tiles of pairs from there on
  int same;              // its only tile of queries is the last unit's
};

struct WtShared {
  uint64_t k_full[2], k_empty[2], q_full[kWtQ], q_empty[kWtQ], s_full[2][2], s_empty[2][2], unit_full[2], unit_empty[2];
  WtUnit unit[2];
  float lse[kWtQ][kWtPairs];
  uint32_t tmem;
  volatile int abort_flag;
};

// Units before entry tile x of a kv head: its tiles of pairs, and kWtLead.
// Rows of a tile of pairs divide 256, so that the causal part is a sum of
// consecutive numbers.
struct WtCost {
  int per;          // rows of a tile of pairs
  bool masked;
  __device__ __forceinline__ long long before(int x, int base, int n) const {
    const int whole = masked ? x : min(x, (base + kWtEntries - 1) / kWtEntries), rest = x - whole;
    long long c = (long long)whole * ((n + per - 1) / per) + (long long)x * kWtLead;
    if (rest > 0) {
      const long long sum = (long long)(whole + x - 1) * rest / 2;    // whole + .. + (x - 1)
      c += (long long)rest * ((base + n + per - 1) / per) - kWtEntries / per * sum;
    }
    return c;
  }
};
struct WtUnits {
  const RowsArgs& a;
  WtCost c;
  __device__ __forceinline__ long long operator()(int L, int n, int b) const {
    if (a.first && a.first[b] < 0) return -1;
    return a.n_kv * c.before((L + kWtEntries - 1) / kWtEntries, L - n, n);
  }
};

template <int HD>
__global__ void __launch_bounds__(kWtThreads, 1) kv_weights_tc_kernel(const __grid_constant__ CUtensorMap kmap,
                                                                      const RowsArgs a) {
  using S = WtShape<HD>;
  extern __shared__ __align__(1024) unsigned char smem[];   // keys [2][2], then queries [kWtQ]
  __shared__ WtShared sm;
  __shared__ long long wsum[kWtThreads / 32];
  unsigned char* qs = smem + 4 * S::kTile;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = 1 << a.g_shift, per = kWtPairs >> a.g_shift;
  int* pre = reinterpret_cast<int*>(qs);   // until the queries come
  const WtCost cost{per, a.mask != nullptr};

  if (smem_addr(smem) & 1023) {   // (the declaration above asks for it)
    if (tid == 0) set_error(a.err, MTP_ERR_BOUNDS);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.k_full[i], 1);
      mbar_init(&sm.k_empty[i], 1);
      mbar_init(&sm.unit_full[i], 1);
      mbar_init(&sm.unit_empty[i], 13);
      for (int j = 0; j < 2; ++j) {
        mbar_init(&sm.s_full[i][j], 1);
        mbar_init(&sm.s_empty[i][j], 4);
      }
    }
    for (int i = 0; i < kWtQ; ++i) {
      mbar_init(&sm.q_full[i], 4);
      mbar_init(&sm.q_empty[i], 9);
    }
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sm.tmem)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tmem_before();
  __syncthreads();
  tmem_after();
  const uint32_t tmem = sm.tmem;
  pdl_wait();
  pdl_trigger();
  Split sp;
  const bool work = rows_split<kWtThreads>(a, WtUnits{a, cost}, 1, pre, wsum, sp);
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    ok = ok && __all_sync(0xffffffffu, at_wait(bar, parity, &sm.abort_flag));
    return ok;
  };

  // The producer looks up where its share begins before the others start.
  int b = 0, g = 0, t = 0, o0 = 0, n = 0, L = 0, tiles = 0;
  long long at = 0;        // the units before (request b, kv head g, entry tile t)
  auto enter = [&]() {     // request b, if it has units
    const int e = rows_request(a, b, o0, n, L);
    tiles = (L + kWtEntries - 1) / kWtEntries;
    return e == MTP_OK && n > 0 && !(a.first && a.first[b] < 0);
  };
  if (work && warp == 8) {
    int hi = a.B;
    while (hi - b > 1) {
      const int m = (b + hi) >> 1;
      if ((uint32_t)pre[m] <= sp.u0) b = m;
      else hi = m;
    }
    enter();
    const long long head = cost.before(tiles, L - n, n), rel = sp.u0 - (uint32_t)pre[b];
    g = (int)(rel / head);
    const long long in = rel - g * head;
    int t1 = tiles;
    while (t1 - t > 1) {
      const int m = (t + t1) >> 1;
      if (cost.before(m, L - n, n) <= in) t = m;
      else t1 = m;
    }
    if (cost.before(t, L - n, n) < in) ++t;     // begun in the share before
    at = pre[b] + g * head + cost.before(t, L - n, n);
  }
  __syncthreads();

  if (work && warp == 8) {
    // ------------------------------------------------------- units and keys
    const int groups = a.kv.num_blocks * a.n_kv * 2;   // of the pool: a box from there on is zeros
    int last_b = -1, last_g = -1, last_row0 = -1;      // the last unit's queries, if it had one tile
    uint32_t issued = 0;
    for (int nu = 0;; ++nu) {
      if (t >= tiles) {
        t = 0;
        ++g;
      }
      while (g >= a.n_kv && ++b < a.B)   // the next request with units
        if (enter()) g = 0;
      const bool any = b < a.B && at < sp.u1;
      if (!wait(&sm.unit_empty[nu & 1], ((nu >> 1) & 1) ^ 1)) break;
      const int base = L - n, t0 = t * kWtEntries, row0 = a.mask ? 0 : max(0, t0 - base);
      const int qt = any ? (n - row0 + per - 1) / per : 0;
      const bool same = qt == 1 && last_b == b && last_g == g && last_row0 == row0;
      if (lane == 0) {
        WtUnit& u = sm.unit[nu & 1];
        u.b = any ? b : -1;
        u.g = g;
        u.o0 = o0;
        u.n = n;
        u.L = L;
        u.base = base;
        u.t0 = t0;
        u.row0 = row0;
        u.tiles = qt;
        u.same = same;
        mbar_arrive(&sm.unit_full[nu & 1]);
      }
      if (!any) break;
      last_b = qt == 1 ? b : -1;
      last_g = g;
      last_row0 = row0;
      // keys: two tiles of eight blocks; lane l < 16 looks up block l
      const int32_t* table = a.kv.block_table + (long long)b * a.kv.max_blocks;
      int row = groups;
      if (lane < 16 && t0 + lane * kBlk < L) {
        const int blk = table[(t0 >> 4) + lane];
        if (blk < 0 || blk >= a.kv.num_blocks) set_error(a.err, MTP_ERR_CAPACITY);
        else row = (blk * a.n_kv + g) * 2;
      }
      const int st = nu & 1;
      if (!wait(&sm.k_empty[st], ((nu >> 1) & 1) ^ 1)) break;
      if (lane == 0) mbar_expect_tx(&sm.k_full[st], 2 * S::kTile);
      __syncwarp();
      const uint32_t dst = smem_addr(smem) + st * 2 * S::kTile, bar = smem_addr(&sm.k_full[st]);
#pragma unroll
      for (int pg = 0; pg < kWtEntries / kBlk; ++pg)
        at_tma(dst + pg * (kBlk * HD * 2), &kmap, __shfl_sync(0xffffffffu, row, pg), bar);
      issued = nu + 1;
      at += qt + kWtLead;
      ++t;
    }
    if (!ok) {   // copies in flight land before the block ends
      for (uint32_t x = issued > 2 ? issued - 2 : 0; x < issued; ++x)
        mbar_wait_bounded(&sm.k_full[x & 1], (x >> 1) & 1, 1u << 20);
    }
  } else if (work && warp == 9) {
    // ------------------------------------------------------------- products
    constexpr uint32_t kBase = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(128 >> 4) << 24);
    constexpr uint32_t kGroup = S::kHalves * 1024;
    const uint64_t k_desc = at_desc(smem_addr(smem), kGroup, 16), q_desc = at_desc(smem_addr(qs), kGroup, 16);
    uint32_t qi = 0, x = 0;   // tiles of queries taken; products' turns
    for (int nu = 0; wait(&sm.unit_full[nu & 1], (nu >> 1) & 1); ++nu) {
      const WtUnit& u = sm.unit[nu & 1];
      const int b = u.b, tiles = u.tiles, same = u.same, pairs = (u.n - u.row0) << a.g_shift;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.unit_empty[nu & 1]);
      if (b < 0) break;
      if (!wait(&sm.k_full[nu & 1], (nu >> 1) & 1)) break;
      for (int k = 0; k < tiles; ++k) {
        if (!same) {
          if (qi > 0) mma_commit(&sm.q_empty[(qi - 1) % kWtQ]);   // done with the tile before
          if (!wait(&sm.q_full[qi % kWtQ], (qi / kWtQ) & 1)) break;
          ++qi;
        }
        const uint32_t cols = min(kWtPairs, (pairs - k * kWtPairs + 15) & ~15);
        const uint32_t idesc = kBase | ((cols >> 3) << 17);
        const uint64_t qd = q_desc + ((qi - 1) % kWtQ) * (S::kTile >> 4);
        for (int w = 0; w < 2; ++w) {
          if (!wait(&sm.s_empty[w][x & 1], ((x >> 1) & 1) ^ 1)) break;
          tmem_after();
          const uint64_t kd = k_desc + ((nu & 1) * 2 + w) * (S::kTile >> 4);
          unrolled<HD / 16>([&](auto y) {
            constexpr int kk = decltype(y)::value;
            constexpr uint32_t off = (kk >> 2) * (1024 >> 4) + (kk & 3) * 2;
            mma_ss<off, off>(tmem + w * 256 + (x & 1) * 128, kd, qd, idesc, kk > 0);
          });
          mma_commit(&sm.s_full[w][x & 1]);
        }
        if (!ok) break;
        ++x;
      }
      if (!ok) break;
      mma_commit(&sm.k_empty[nu & 1]);
    }
  } else if (work && warp >= 10) {
    // -------------------------------------------------------------- queries
    const int r = tid - 320;               // 0 .. 127
    constexpr int CH = HD / 8;             // 16-byte chunks of a pair; copies of a thread
    uint32_t qi = 0, out = 0;              // tiles asked for, and published
    // A tile is there: turn its lse into exponents' offsets, publish it
    auto publish = [&](uint32_t q) {
      float* l = &sm.lse[q % kWtQ][r];
      const float y = *l;
      *l = y == -INFINITY ? INFINITY : y * kLog2e;   // a row that sees nothing weighs nothing
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_full[q % kWtQ]);
    };
    for (int nu = 0; wait(&sm.unit_full[nu & 1], (nu >> 1) & 1); ++nu) {
      const WtUnit& u = sm.unit[nu & 1];
      const int b = u.b, g = u.g, o0 = u.o0, n = u.n, row0 = u.row0, tiles = u.tiles, same = u.same;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.unit_empty[nu & 1]);
      if (b < 0) break;
      for (int k = 0; k < tiles && !same; ++k) {
        if (!wait(&sm.q_empty[qi % kWtQ], ((qi / kWtQ) & 1) ^ 1)) break;
        const int i0 = row0 + k * per, c = r % CH;
        unsigned char* dst = qs + (qi % kWtQ) * S::kTile;
#pragma unroll
        for (int y = 0; y < CH; ++y) {
          const int pr = r / CH + y * (128 / CH), i = min(i0 + (pr >> a.g_shift), n - 1);
          const bool none = i0 + (pr >> a.g_shift) >= n;
          const uint16_t* src = (const uint16_t*)a.q + (long long)(o0 + i) * a.q_stride +
                                (long long)(g * G + (pr & (G - 1))) * HD + c * 8;
          unsigned char* to = dst + ((pr >> 3) * S::kHalves + (c >> 3)) * 1024 + (pr & 7) * 128 + (((c & 7) ^ (pr & 7)) << 4);
          if (a.q_vec) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(to)), "l"(src), "r"(none ? 0 : 16) : "memory");
          } else {
            const uint4 v = make_uint4((uint32_t)src[0] | (uint32_t)src[1] << 16, (uint32_t)src[2] | (uint32_t)src[3] << 16,
                                       (uint32_t)src[4] | (uint32_t)src[5] << 16, (uint32_t)src[6] | (uint32_t)src[7] << 16);
            *reinterpret_cast<uint4*>(to) = none ? make_uint4(0, 0, 0, 0) : v;
          }
        }
        const int i = min(i0 + (r >> a.g_shift), n - 1);
        const float* lp = a.lse + (long long)(o0 + i) * (a.n_kv << a.g_shift) + g * G + (r & (G - 1));
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(&sm.lse[qi % kWtQ][r])), "l"(lp) : "memory");
        asm volatile("cp.async.commit_group;" ::: "memory");
        ++qi;
        if (out + 1 < qi) {
          asm volatile("cp.async.wait_group 1;" ::: "memory");
          publish(out++);
        }
      }
      if (!ok) break;
      // The last tile may wait for the next unit's first one, but only if that is
      // there already: units behind this one may come when this one is done.
      const WtUnit& v = sm.unit[(nu + 1) & 1];
      if (out < qi && (!__all_sync(0xffffffffu, mbar_test_wait(&sm.unit_full[(nu + 1) & 1], ((nu + 1) >> 1) & 1)) ||
                       v.b < 0 || v.same)) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        publish(out++);
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  } else if (work) {
    // -------------------------------------------------------------- weights
    const int w = warp >> 2, r = tid & 127;
    const uint32_t at0 = tmem + ((uint32_t)((warp & 3) * 32) << 16) + w * 256;
    uint32_t qi = 0, x = 0;
    for (int nu = 0; wait(&sm.unit_full[nu & 1], (nu >> 1) & 1); ++nu) {
      const WtUnit& u = sm.unit[nu & 1];
      const int b = u.b, g = u.g, o0 = u.o0, n = u.n, L = u.L, base = u.base, row0 = u.row0, tiles = u.tiles, same = u.same;
      const int t0 = u.t0 + w * 128, t = t0 + r;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.unit_empty[nu & 1]);
      if (b < 0) break;
      // what the sum is added to, under the first products
      float* dst = nullptr;
      float old = 0.0f;
      if (t < L) {
        const int blk = a.kv.block_table[(long long)b * a.kv.max_blocks + (t >> 4)];
        const long long e = ((long long)blk * a.n_kv + g) * kBlk + (t & 15);
        if (blk >= 0 && blk < a.kv.num_blocks && MTP_IN_BOUNDS(a.err, e, (long long)a.kv.num_blocks * a.n_kv * kBlk)) {
          dst = a.weights + e;
          if (t < (a.first ? a.first[b] : base)) old = *dst;
        }
      }
      const int see0 = a.mask ? 0 : max(0, t - base);      // the first row that sees the entry (without a mask)
      uint64_t sum[2] = {0ull, 0ull};
      for (int k = 0; k < tiles; ++k) {
        if (!same) {
          if (qi > 0 && lane == 0) mbar_arrive(&sm.q_empty[(qi - 1) % kWtQ]);
          if (!wait(&sm.q_full[qi % kWtQ], (qi / kWtQ) & 1)) break;
          ++qi;
        }
        if (!wait(&sm.s_full[w][x & 1], (x >> 1) & 1)) break;
        tmem_after();
        const float* lse = sm.lse[(qi - 1) % kWtQ];
        const int i0 = row0 + k * per, pairs = min(kWtPairs, (n - i0) << a.g_shift);
        // whether every entry of the group is seen by all pairs of the tile
        const bool part = pairs < kWtPairs || a.mask || t0 + 127 > base + i0;
        const int from = (see0 - i0) << a.g_shift;          // the first pair that sees the entry
        const uint32_t s_at = at0 + (x & 1) * 128;
        auto add = [&](uint32_t (&v)[32], int c, bool all) {
          const uint64_t cc = two(a.c, a.c);
          uint32_t bits = ~0u;
          if (!all) {
            if (a.mask) {
              bits = 0;
              const int j = t - base;
              for (int e = 0; e < 32; e += G) {
                const int i = i0 + ((32 * c + e) >> a.g_shift);
                if (i < n && t < L &&
                    (j < 0 || (a.mask[(long long)(o0 + i) * a.mask_words + (j >> 5)] >> (j & 31) & 1)))
                  bits |= low_bits(G) << e;
              }
            } else {
              bits = low_bits(pairs - 32 * c) & ~low_bits(from - 32 * c);
            }
          }
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 l = *reinterpret_cast<const float4*>(lse + 32 * c + e);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float x0, x1;
              untwo(fma2(two(__uint_as_float(v[e + 2 * h]), __uint_as_float(v[e + 2 * h + 1])), cc,
                         h ? two(-l.z, -l.w) : two(-l.x, -l.y)), x0, x1);
              x0 = exp2_fast(x0);
              x1 = exp2_fast(x1);
              if (!all) {
                x0 = bits & (1u << (e + 2 * h)) ? x0 : 0.0f;
                x1 = bits & (2u << (e + 2 * h)) ? x1 : 0.0f;
              }
              sum[h] = add2(sum[h], two(x0, x1));
            }
          }
        };
        uint32_t va[32], vb[32];
        if (!part) {
          tmem_ld(s_at, va);
#pragma unroll 1
          for (int c = 0; c < 4; c += 2) {
            tmem_wait_ld();
            tmem_ready(va);
            tmem_ld(s_at + 32 * c + 32, vb);
            add(va, c, true);
            tmem_wait_ld();
            tmem_ready(vb);
            if (c == 0) tmem_ld(s_at + 64, va);
            add(vb, c + 1, true);
          }
        } else {
#pragma unroll 1
          for (int c = 0; 32 * c < pairs; ++c) {
            tmem_ld(s_at + 32 * c, va);
            tmem_wait_ld();
            tmem_ready(va);
            add(va, c, false);
          }
        }
        tmem_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.s_empty[w][x & 1]);
        ++x;
      }
      if (!ok) break;
      if (dst) {
        float l0, l1;
        untwo(add2(sum[0], sum[1]), l0, l1);
        *dst = old + (l0 + l1);
      }
    }
  }
  if (!ok) {
    sm.abort_flag = 1;
    if (lane == 0) set_error(a.err, MTP_ERR_TIMEOUT);
  }
  tmem_before();
  __syncthreads();
  if (warp == 9) {
    tmem_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

template <int HD>
static cudaError_t weights_tc_launch(mtp_ctx* ctx, cudaStream_t s, const RowsArgs& a) {
  using S = WtShape<HD>;
  CUtensorMap km;
  const uint64_t rows = (uint64_t)a.kv.num_blocks * a.n_kv * kBlk;
  if (rows > INT32_MAX || !make_block_map(&km, a.kv.k_pool, rows, HD)) return cudaErrorInvalidValue;
  const cudaError_t e = ensure_smem((const void*)kv_weights_tc_kernel<HD>, S::kBytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv_weights_tc_kernel<HD>, dim3(ctx->num_sms), dim3(kWtThreads), S::kBytes, s, km, a);
}
cudaError_t launch_weights_tc(mtp_ctx* ctx, cudaStream_t s, const RowsArgs& a) {
  return ctx->cfg.head_dim == 128 ? weights_tc_launch<128>(ctx, s, a) : weights_tc_launch<64>(ctx, s, a);
}

}  // namespace mtp
