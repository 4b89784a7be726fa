// Attention of new rows over the paged cache on the tensor cores (tcgen05),
// bf16 heads: prompts, chunks of them, draft rows and decoding rows alike.
//
//   out[r, h] = sum_t p_t V[t, g] / sum_t p_t,  p_t = 2^(c s_t - m),
//   s_t = q[r, h] . K[t, g], c = scale * log2 e, m a reference near the running
// maximum.
//
// A segment is 256 (row, query head) pairs of one kv head; a step takes 128
// slots (eight cache blocks).  One thread block per SM, twelve warps:
//   warps 0-3, 4-7  two softmax groups; group w owns the 128 x 128 scores S_w
//            and the result O_w in tensor memory, a thread a row: it reads its
//            128 scores, takes the reference off, writes the weights as bf16
//            over the scores (the A operand of the second product) and keeps the
//            sum.  O_w is scaled only when a row's maximum passes its reference
//            by 8 (powers of two), so most steps touch it with products alone.
//   warp 8   finds the segments of the block's share, and loads cache blocks
//            (a box each, 128-byte swizzle) into a ring of K and V tiles, into
//            the next segment's as soon as the ring has room
//   warp 9   issues the products: S_w = Q_w K^T, O_w += P_w V, the two groups'
//            in turn, so that one group's softmax runs under the other's products
//   warps 10, 11  look through the V tiles that some row sees only part of for
//            entries that are not finite (0 * inf) and put zeros there; the rows
//            that see such an entry get it at the end.
// With more than 128 pairs the groups take 128 pairs each of every step; with up
// to 128 (decoding rows, the end of a chunk) both take all of them, of
// every other step, and the two results are joined from tensor memory.
//
// Work is split over the flattened (request, kv head, tile, step) sequence in
// equal shares, found on the device from the lengths; a segment that spans
// thread blocks leaves its pieces in the workspace for rows_join_kernel.
//
// The weights' rounding to bf16 (once, half a step of 2^-8; the normalising sum takes
// them unrounded) is the second product's: its operands have one type, and V is bf16.  A
// second operand for the rounding's rest would make three products of two.  Results are
// off by 0.0021 to 0.0023 of themselves against 64 bits, where weights held in float32
// and results rounded once give 0.0016 to 0.0017.
//
// What bounds it: for few rows the cache's bytes (64 requests of 4096 entries: 167
// us, 6.4 TB/s).  For many the chain of a group's step: its products (two of 512
// cycles at the pipe's peak) and its softmax (1000 cycles for 128 scores a
// thread) follow one another, and the other group fills no more than its own two
// products of the pipe meanwhile; a step of both takes 3100 cycles against 2048
// of products.  8192 rows, 32 query heads of 128: 335 to 342 us, 1610 to 1640 TFLOP/s, and
// 366 us, 1500 TFLOP/s, once thousands of calls have brought the GPU to its power cap
// (1905 MHz); 1024 rows on 32768 entries 340 to 365 us, 1530 to 1650 TFLOP/s.  A segment costs some 6500 cycles besides
// its steps (the last products, 128 x 128 results a group to be scaled and
// written, the first step and the one that is partly seen), so short contexts pay
// more: 16 chunks of 512 rows on up to 1500 entries take 130 to 140 us.  Tried and
// not kept: results staged in a fifth tile's place and stored by the copy engine
// (the same times, long contexts 361 -> 370 us), first and partly seen steps in
// the pass of the others (its code then runs slower, 350 -> 357 us at the time),
// every sixth, fourth or third pair of exponentials as a polynomial on the
// multiply-add pipe (358, 377 and 376 us: the softmax is bound by issuing, not by
// the exponentials).  With the softmax left out the products and copies alone
// take 302 us of the prompt's 335.
#include <cuda.h>
#include <math.h>

#include "mtp_kv_tc.cuh"

namespace mtp {

constexpr int kAtThreads = 384;
constexpr float kAtSlack = 8.0f;    // how far (powers of two) a maximum may pass its reference
constexpr float kAtCoarse = 67108864.0f;   // from 2^26 on the reference's rounding is some units
constexpr float kAtWhole = 4096.0f;        // from 2^12 on references are whole numbers

template <int HD>
struct AtShape {
  static constexpr int kHalves = HD / 64;
  static constexpr int kTile = kAtStep * HD * 2;              // bytes of a K or V tile, and of 128 pairs' queries
  // Five tiles of 32 KB are what fits.  (Four: 1024 rows on 32768 entries 370 instead
  // of 361 us at the time, a prompt of 8192 338 instead of 335.)
  static constexpr int kStages = HD == 128 ? 5 : 8;
  static constexpr int kBytes = 2 * kTile + kStages * kTile;
};

struct AtPiece {
  int b;            // request, or -1: no more work
  int g, o0, n, base, end, i0;
  int s_lo, tiles;  // first step, number of steps
  int edge;         // the first step that some row sees only part of
  int valid;        // pairs
  int slot;         // where a piece of a spanning segment goes; -1: the whole segment
  int dirty;        // an entry that is not finite was taken out of V
};

// Bit e: whether a row sees slot t + e.  Without mask words it sees the slots
// up to `last`; with them those below base, and of the n new ones those named.
__device__ __forceinline__ uint32_t at_seen(const int32_t* words, int last, int t, int base, int n) {
  if (!words) return low_bits(last - t + 1);
  const int j = t - base;
  if (j <= -32) return ~0u;
  const int have = (n + 31) >> 5;       // words that hold the row's bits
  if (j < 0) return low_bits(-j) | ((uint32_t)words[0] & low_bits(n)) << -j;
  const int x = j >> 5;
  const uint32_t lo = x < have ? (uint32_t)words[x] : 0u, hi = x + 1 < have ? (uint32_t)words[x + 1] : 0u;
  return __funnelshift_r(lo, hi, j & 31) & low_bits(n - j);
}

// Halves of a word that hold bf16 numbers that are not finite: bit 15, bit 31.
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) {
  return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}

// Ring positions of a piece of n steps: K0 K1 V0 K2 V1 .. K(n-1) V(n-2) V(n-1).
__device__ __forceinline__ uint32_t ring_k(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ uint32_t ring_v(int j, int n) { return j == n - 1 ? 2 * n - 1 : 2 * j + 2; }

template <int HD>
struct AtShared {
  uint64_t full[AtShape<HD>::kStages], empty[AtShape<HD>::kStages];
  // (o_full: results of a segment.  Not a phase of s_full, as the next segment's scores are not waited for by anyone
  // and could complete the next phase before a slow warp has seen that one.)
  uint64_t s_full[2], o_full[2], p_ready[2], q_full[2], q_empty[2], q_ready[2], scan, clean, merged, piece_full[2], piece_empty[2];
  AtPiece piece[2];
  float ml[2][128][2];
  uint32_t tmem;
  volatile int abort_flag;
};

template <int HD>
__global__ void __launch_bounds__(kAtThreads, 1) kv_attn_tc_kernel(const __grid_constant__ CUtensorMap qmap,
                                                                   const __grid_constant__ CUtensorMap kmap,
                                                                   const __grid_constant__ CUtensorMap vmap,
                                                                   const RowsArgs a, const SegShape sh) {
  using S = AtShape<HD>;
  constexpr int NS = S::kStages;
  extern __shared__ __align__(1024) unsigned char smem[];   // tiles: the swizzle wants 1024-byte boundaries
  __shared__ AtShared<HD> sm;
  __shared__ long long wsum[kAtThreads / 32];
  int* pre = a.pre + (long long)blockIdx.x * (kKvMaxB + 1);
  unsigned char* ring = smem + 2 * S::kTile;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = 1 << a.g_shift;

  if (smem_addr(smem) & 1023) {   // (the declaration above asks for it)
    if (tid == 0) set_error(a.err, MTP_ERR_BOUNDS);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&sm.s_full[w], 1);
      mbar_init(&sm.o_full[w], 1);
      mbar_init(&sm.p_ready[w], 4);
      mbar_init(&sm.q_ready[w], 4);
      mbar_init(&sm.q_full[w], 1);
      mbar_init(&sm.q_empty[w], 1);
      mbar_init(&sm.piece_full[w], 1);
      mbar_init(&sm.piece_empty[w], 11);
    }
    mbar_init(&sm.scan, 1);
    mbar_init(&sm.clean, 2);
    mbar_init(&sm.merged, 8);
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
  if (tid == 0) a.meta[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
  Split sp;
  const bool sorted = a.plan && __ldcg(a.plan) == 1;
  const bool work = sorted || rows_split<kAtThreads>(a, SegUnits{a, sh}, sh.lead + 1, pre, wsum, sp);

  if (work && warp == 8) {
    // ------------------------------------------------------------- producer
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    uint32_t rb = 0, issued = 0, asked[2] = {0, 0};
    int np = 0;
    bool ok = true;
    const int page = lane & 7;
    const int oob = a.kv.num_blocks * a.n_kv * 2;   // groups of the pool: a box from there on is zeros
    uint32_t u = sp.u0;
    const int items = sorted ? __ldcg(a.plan + 1) : 0;
    while (ok) {
      Piece p{};
      bool any = false;
      if (sorted) {
        int item = lane == 0 ? atomicAdd(a.plan + 2, 1) : 0;
        item = __shfl_sync(0xffffffffu, item, 0);
        if (item < items) {
          any = true;
          const int2 t = __ldcg(reinterpret_cast<const int2*>(a.plan + 4) + item / a.n_kv);
          p.b = t.x;
          p.tile = t.y;
          p.g = item % a.n_kv;
          rows_request(a, p.b, p.o0, p.n, p.L);
          p.base = p.L - p.n;
          p.end = seg_end(sh, p.tile, p.base, p.n, a.mask != nullptr);
          p.s_hi = (p.end + kAtStep - 1) / kAtStep;
        }
      }
      while (!sorted && u < sp.u1) {
        find_piece(a, sh, pre, sp, u, p);
        u = p.next;
        if (p.s_lo < p.s_hi) {
          any = true;
          break;
        }
      }
      ok = __all_sync(0xffffffffu, at_wait(&sm.piece_empty[np & 1], ((np >> 1) & 1) ^ 1, &sm.abort_flag));
      if (!ok) break;
      const bool whole = p.c_first == p.c_last;
      const int i0 = p.tile << sh.rows, valid = min(kAtPairs, (p.n - i0) << a.g_shift);
      if (lane == 0) {
        AtPiece& q = sm.piece[np & 1];
        q.b = any ? p.b : -1;
        q.g = p.g;
        q.o0 = p.o0;
        q.n = p.n;
        q.base = p.base;
        q.end = p.end;
        q.i0 = i0;
        q.s_lo = p.s_lo;
        q.tiles = p.s_hi - p.s_lo;
        // the first step with a slot that the segment's first row (or, under a mask, some row) may not see
        q.edge = (p.base + (a.mask ? 0 : i0 + 1)) / kAtStep;
        q.valid = valid;
        q.slot = whole ? -1 : ((int)blockIdx.x == p.c_first ? 1 : 0);
        q.dirty = 0;
        mbar_arrive(&sm.piece_full[np & 1]);
        if (any && !whole && (int)blockIdx.x == p.c_first) {
          a.meta[2 * blockIdx.x] = make_int4(p.c_last - p.c_first + 1, p.c_first, valid, p.g);
          a.meta[2 * blockIdx.x + 1] = make_int4(p.o0 + i0, 0, 0, 0);
        }
      }
      ++np;
      if (!any) break;
      const int n = p.s_hi - p.s_lo;
      const int32_t* table = a.kv.block_table + (long long)p.b * a.kv.max_blocks;
      auto row_of = [&](int j) -> int {   // the pool's group of eight rows where this lane's block of step j begins
        const int t = (p.s_lo + j) * kAtStep + page * kBlk;
        if (j >= n || t >= p.end) return oob;
        const int blk = table[t >> 4];
        if (blk < 0 || blk >= a.kv.num_blocks) {
          set_error(a.err, MTP_ERR_CAPACITY);
          return oob;
        }
        return (blk * a.n_kv + p.g) * 2;
      };
      auto issue = [&](const CUtensorMap* map, uint32_t it, int row) -> bool {
        const int st = it % NS;
        if (!__all_sync(0xffffffffu, at_wait(&sm.empty[st], ((it / NS) & 1) ^ 1, &sm.abort_flag))) return false;
        if (lane == 0) mbar_expect_tx(&sm.full[st], S::kTile);
        __syncwarp();
        const uint32_t dst = smem_addr(ring) + st * S::kTile, bar = smem_addr(&sm.full[st]);
#pragma unroll
        for (int pg = 0; pg < kAtStep / kBlk; ++pg)
          at_tma(dst + pg * (kBlk * HD * 2), map, __shfl_sync(0xffffffffu, row, pg), bar);
        issued = it + 1;
        return true;
      };
      // queries: 128 pairs a group, or all of up to 128 in the first tile (those
      // past the request's rows are another's, or zeros: nobody writes their results)
      auto queries = [&](int w) -> bool {
        if (!__all_sync(0xffffffffu, at_wait(&sm.q_empty[w], (asked[w] & 1) ^ 1, &sm.abort_flag))) return false;
        if (lane == 0) mbar_expect_tx(&sm.q_full[w], S::kTile);
        __syncwarp();
#pragma unroll
        for (int half = 0; half < S::kHalves; ++half)
          at_tma_q(smem_addr(smem) + w * S::kTile + half * (128 * 128), &qmap, p.o0 + i0 + ((w * 128) >> a.g_shift), half, p.g,
                   smem_addr(&sm.q_full[w]));
        ++asked[w];
        return true;
      };
      int r0 = row_of(0), r1 = row_of(1);
      if (a.q_vec) ok = queries(0);
      if (ok) ok = issue(&kmap, rb, r0);
      if (ok && a.q_vec && valid > 128) ok = queries(1);
      for (int j = 0; j < n && ok; ++j) {
        const int r2 = row_of(j + 2);   // looked up two steps ahead
        if (j + 1 < n) ok = issue(&kmap, rb + ring_k(j + 1), r1);
        if (ok) ok = issue(&vmap, rb + ring_v(j, n), r0);
        r0 = r1;
        r1 = r2;
      }
      rb += 2 * n;
    }
    if (!ok) {
      if (lane == 0) set_error(a.err, MTP_ERR_TIMEOUT);
      sm.abort_flag = 1;
      // copies in flight land before the block ends
      for (uint32_t it = issued > NS ? issued - NS : 0; it < issued; ++it)
        mbar_wait_bounded(&sm.full[it % NS], (it / NS) & 1, 1u << 20);
      for (int w = 0; w < 2; ++w)
        if (asked[w]) mbar_wait_bounded(&sm.q_full[w], (asked[w] - 1) & 1, 1u << 20);
    }
  } else if (work && warp == 9) {
    // ------------------------------------------------------------- products
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    constexpr uint32_t kBase = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(128 >> 4) << 24);
    constexpr uint32_t kIdS = kBase | ((uint32_t)(kAtStep >> 3) << 17);
    constexpr uint32_t kIdO = kBase | (1u << 16) | ((uint32_t)(HD >> 3) << 17);   // B (V) is MN-major
    // (descriptors differ in the address field alone, which counts 16 bytes)
    constexpr uint32_t kGroup = S::kHalves * 1024;       // bytes of eight rows
    const uint64_t q_desc = at_desc(smem_addr(smem), 1024, 16), k_desc = at_desc(smem_addr(ring), kGroup, 16),
                   v_desc = at_desc(smem_addr(ring), kGroup, 1024);
    uint32_t rb = 0, cleans = 0, p_count[2] = {0, 0}, q_count[2] = {0, 0};
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && __all_sync(0xffffffffu, at_wait(bar, parity, &sm.abort_flag));
      return ok;
    };
    for (int np = 0; wait(&sm.piece_full[np & 1], (np >> 1) & 1); ++np) {
      const AtPiece& p = sm.piece[np & 1];
      if (p.b < 0) break;
      const int n = p.tiles, first_edge = max(0, p.edge - p.s_lo);
      const bool split = p.valid <= 128;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.piece_empty[np & 1]);
      auto at_ring = [&](uint32_t pos) { return (rb + pos) % NS; };
      auto wait_ring = [&](uint32_t pos) { return wait(&sm.full[at_ring(pos)], ((rb + pos) / NS) & 1); };
      auto free_ring = [&](uint32_t pos) { mma_commit(&sm.empty[at_ring(pos)]); };
      auto scores = [&](int w, int j) {                // S_w = Q K_j^T
        const uint64_t qd = q_desc + (split ? 0 : w * (S::kTile >> 4)), kd = k_desc + at_ring(ring_k(j)) * (S::kTile >> 4);
        tmem_after();
        unrolled<HD / 16>([&](auto x) {
          constexpr int kk = decltype(x)::value;
          mma_ss<(kk >> 2) * (128 * 128 >> 4) + (kk & 3) * 2, (kk >> 2) * (1024 >> 4) + (kk & 3) * 2>(tmem + w * 128, qd, kd,
                                                                                                 kIdS, kk > 0);
        });
        // the last product that reads these queries
        if (j + 1 >= n && a.q_vec) mma_commit(&sm.q_empty[split ? 0 : w]);
      };
      auto values = [&](int w, int j, bool start) {    // O_w += P_w V_j
        const uint64_t vd = v_desc + at_ring(ring_v(j, n)) * (S::kTile >> 4);
        tmem_after();
        unrolled<kAtStep / 16>([&](auto x) {
          constexpr int kk = decltype(x)::value;
          mma_ts<kk * 8, kk * (kBlk * HD * 2 >> 4)>(tmem + 256 + w * HD, tmem + w * 128, vd, kIdO, !(start && kk == 0));
        });
      };
      // V_j is there; where some row sees only part of it, it is looked through
      // meanwhile (the scanning warps come when they are called: ahead of the
      // ring they could not tell its phases apart)
      auto wait_v = [&](int j) {
        if (!wait_ring(ring_v(j, n))) return false;
        if (j >= first_edge && lane == 0) mbar_arrive(&sm.scan);
        __syncwarp();
        return true;
      };
      auto wait_clean = [&](int j) { return j < first_edge || wait(&sm.clean, cleans++ & 1); };
      auto wait_p = [&](int w) { return wait(&sm.p_ready[w], p_count[w]++ & 1); };
      auto wait_q = [&](int w) {
        return a.q_vec ? wait(&sm.q_full[w], q_count[w]++ & 1) : wait(&sm.q_ready[w], np & 1);
      };
      if (!wait_q(0) || !wait_ring(ring_k(0))) break;
      scores(0, 0);
      mma_commit(&sm.s_full[0]);
      if (split) free_ring(ring_k(0));
      if ((!split || !a.q_vec) && !wait_q(1)) break;
      // A wait takes some 150 cycles even when there is nothing to wait for, and
      // the products in the pipe cover about 200: one wait at most stands
      // between two runs of eight products.
      if (!split) {
        scores(1, 0);
        mma_commit(&sm.s_full[1]);
        free_ring(ring_k(0));
        if (!wait_v(0)) break;
        for (int j = 0; j < n; ++j) {
          const bool more = j + 1 < n;
          if (!wait_p(0) || !wait_clean(j)) break;
          values(0, j, j == 0);
          if (more) {
            if (!wait_ring(ring_k(j + 1))) break;
            scores(0, j + 1);
          }
          mma_commit(more ? &sm.s_full[0] : &sm.o_full[0]);
          if (!wait_p(1)) break;
          values(1, j, j == 0);
          free_ring(ring_v(j, n));
          if (more) scores(1, j + 1);
          mma_commit(more ? &sm.s_full[1] : &sm.o_full[1]);
          if (more) {
            free_ring(ring_k(j + 1));
            if (!wait_v(j + 1)) break;
          }
        }
      } else {
        if (n > 1) {
          if (!wait_ring(ring_k(1))) break;
          scores(1, 1);
          mma_commit(&sm.s_full[1]);
          free_ring(ring_k(1));
        }
        for (int j = 0; j < n; ++j) {
          const int w = j & 1;
          if (!wait_v(j) || !wait_p(w) || !wait_clean(j)) break;
          values(w, j, j < 2);
          free_ring(ring_v(j, n));
          if (j + 2 < n) {
            if (!wait_ring(ring_k(j + 2))) break;
            scores(w, j + 2);
            free_ring(ring_k(j + 2));
          }
          mma_commit(j + 2 < n ? &sm.s_full[w] : &sm.o_full[w]);
        }
      }
      if (!ok) break;
      rb += 2 * n;
    }
    if (!ok) {
      sm.abort_flag = 1;
      if (lane == 0) set_error(a.err, MTP_ERR_TIMEOUT);
    }
  } else if (work && warp >= 10) {
    // ------------------------------------- entries of V that are not finite
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    uint32_t rb = 0, scans = 0;
    bool ok = true;
    for (int np = 0; ok; ++np) {
      ok = __all_sync(0xffffffffu, at_wait(&sm.piece_full[np & 1], (np >> 1) & 1, &sm.abort_flag));
      if (!ok) break;
      AtPiece& p = sm.piece[np & 1];
      if (p.b < 0) break;
      const int n = p.tiles;
      for (int j = max(0, p.edge - p.s_lo); j < n; ++j) {
        const uint32_t it = rb + ring_v(j, n);
        ok = __all_sync(0xffffffffu, at_wait(&sm.scan, scans++ & 1, &sm.abort_flag) &&
                                         at_wait(&sm.full[it % NS], (it / NS) & 1, &sm.abort_flag));
        if (!ok) break;
        uint4* tile = reinterpret_cast<uint4*>(ring + (size_t)(it % NS) * S::kTile);
        bool found = false;
#pragma unroll 8
        for (int i = (warp - 10) * 32 + lane; i < S::kTile / 16; i += 64) {
          const uint4 x = tile[i];
          found |= (not_finite2(x.x) | not_finite2(x.y) | not_finite2(x.z) | not_finite2(x.w)) != 0;
        }
        if (found) {
          for (int i = (warp - 10) * 32 + lane; i < S::kTile / 16; i += 64) {
            uint4 x = tile[i];
            x.x &= ~((not_finite2(x.x) >> 15) * 0xFFFFu);
            x.y &= ~((not_finite2(x.y) >> 15) * 0xFFFFu);
            x.z &= ~((not_finite2(x.z) >> 15) * 0xFFFFu);
            x.w &= ~((not_finite2(x.w) >> 15) * 0xFFFFu);
            tile[i] = x;
          }
          *(volatile int*)&p.dirty = 1;   // (before the products that the results wait for)
          fence_async();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.clean);
      }
      rb += 2 * n;
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&sm.piece_empty[np & 1]);
    }
    if (!ok) sm.abort_flag = 1;
  } else if (work) {
    // -------------------------------------------------------------- softmax
    // registers of the block's launch, 384 x 168: 256 x 216 and 128 x 72
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int w = warp >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + w * 128, o_at = tmem + lanes + 256;
    uint32_t s_count = 0, o_count = 0, merges = 0;   // phases of s_full[w], o_full[w] and merged
    bool ok = true;
    // Queries whose rows do not lie on 16 bytes: fetched by the groups themselves,
    // between two segments.
    auto store_q = [&](const AtPiece& p) {
      if (p.b < 0) return;
      if (p.valid > 128 || w == 0) {
#pragma unroll 1
        for (int x = r; x < 128 * HD / 8; x += 128) {
          const int pair = x / (HD / 8), c = x % (HD / 8), i = p.i0 + ((w * 128 + pair) >> a.g_shift);
          uint4 v = make_uint4(0, 0, 0, 0);
          if (i < p.n) {
            const uint16_t* s = (const uint16_t*)a.q + (long long)(p.o0 + i) * a.q_stride + (long long)(p.g * G + (pair & (G - 1))) * HD + c * 8;
            v = make_uint4((uint32_t)s[0] | (uint32_t)s[1] << 16, (uint32_t)s[2] | (uint32_t)s[3] << 16,
                           (uint32_t)s[4] | (uint32_t)s[5] << 16, (uint32_t)s[6] | (uint32_t)s[7] << 16);
          }
          *reinterpret_cast<uint4*>(smem + w * S::kTile + (c >> 3) * (128 * 128) + pair * 128 + (((c & 7) ^ (pair & 7)) << 4)) = v;
        }
        fence_async();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_ready[w]);
    };
    auto wait_piece = [&](int np) {
      return (bool)__all_sync(0xffffffffu, at_wait(&sm.piece_full[np & 1], (np >> 1) & 1, &sm.abort_flag));
    };
    for (int np = 0; ok; ++np) {
      ok = wait_piece(np);
      if (!ok) break;
      const AtPiece& p = sm.piece[np & 1];
      if (p.b < 0) break;
      if (!a.q_vec) store_q(p);
      const int n = p.tiles, s_lo = p.s_lo, i0 = p.i0, rows = p.n, base = p.base, g = p.g, o0 = p.o0;
      const bool split = p.valid <= 128;
      const int mine = split ? (n + 1 - w) / 2 : n;       // steps of this group
      // ---- this thread's row
      const int pr = split ? r : w * 128 + r;
      const int i = i0 + (pr >> a.g_shift);
      const bool live = i < rows;
      const int last = min(base + i, p.end - 1);           // the last slot that the row sees (without a mask)
      const int32_t* words = a.mask && live ? a.mask + (long long)(o0 + i) * a.mask_words : nullptr;
      // the first step that some row of this group sees only part of
      const int edge = a.mask || split ? p.edge : (base + i0 + ((w * 128) >> a.g_shift) + 1) / kAtStep;
      float m = kKvLeast, l = 0.0f;
      bool coarse = false;
      for (int x = 0; x < mine; ++x) {
        const int j = split ? 2 * x + w : x;
        ok = __all_sync(0xffffffffu, at_wait(&sm.s_full[w], s_count & 1, &sm.abort_flag));
        if (!ok) break;
        ++s_count;
        tmem_after();
        const bool part = s_lo + j >= edge;                // some row sees only part of the step
        const int t0 = (s_lo + j) * kAtStep;
        uint64_t sum[2] = {0ull, 0ull};
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        auto most = [&](const uint32_t (&v)[32]) {
#pragma unroll
          for (int e = 0; e < 32; e += 2) mx[(e >> 1) & 3] = max3(mx[(e >> 1) & 3], __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
        };
        auto top = [&]() { return fmaxf(__fmul_rn(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), a.c), kKvLeast); };
        auto weights = [&](uint32_t (&v)[32], uint32_t* pw, uint64_t cc, uint64_t mm) {
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float x0, x1;
            untwo(fma2(two(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), cc, mm), x0, x1);
            x0 = exp2_fast(x0);
            x1 = exp2_fast(x1);
            sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], two(x0, x1));
            pw[e / 2] = pack2_bf16(x0, x1);
          }
        };
        bool done = false;
        if (x > 0 && !part && !coarse) {
          // One pass, 32 columns at a time: weights by the reference as it is, and
          // the maximum next to them.  Where that passes the reference by more
          // than the slack (rarely) the pass counts for nothing; the scores
          // are still there, as the weights go over them at the end.  (No
          // question is asked within it: with two per 32 columns the loads'
          // latency showed, 1910 instead of 1240 cycles a step.)
          uint32_t pw[64], va[32], vb[32];
          const uint64_t cc = two(a.c, a.c), mm = two(-m, -m);
          tmem_ld(s_at, va);
          tmem_wait_ld();
          tmem_ready(va);
          tmem_ld(s_at + 32, vb);
          most(va);
          weights(va, pw, cc, mm);
          tmem_wait_ld();
          tmem_ready(vb);
          tmem_ld(s_at + 64, va);
          most(vb);
          weights(vb, pw + 16, cc, mm);
          tmem_wait_ld();
          tmem_ready(va);
          tmem_ld(s_at + 96, vb);
          most(va);
          weights(va, pw + 32, cc, mm);
          tmem_wait_ld();
          tmem_ready(vb);
          most(vb);
          weights(vb, pw + 48, cc, mm);
          done = !__any_sync(0xffffffffu, top() > m + kAtSlack);
          if (done) {
            tmem_st(s_at, pw);
            tmem_st(s_at + 32, pw + 32);
          }
        }
        if (!done) {
          sum[0] = sum[1] = 0ull;
          // The first step, steps that some row sees only part of, and those that
          // move the reference: 32 columns at a time in little code (fetching
          // instructions that a segment runs once or twice costs more than running
          // them), the maximum before the weights, which go, two a word, over columns
          // 16 c .. that are done with.  Where a later quarter moves the reference, the
          // weights written before move with it: by whole powers of two, so
          // that they are not rounded again.  A reference plus a whole number is a
          // float to 2^-12 while it is small; larger references are whole numbers
          // themselves, so that their sums are exact.
          mx[0] = mx[1] = mx[2] = mx[3] = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            tmem_ld(s_at + 32 * c, v);
            tmem_wait_ld();
            tmem_ready(v);
            if (part) {
              const uint32_t bits = at_seen(words, last, t0 + 32 * c, base, rows);
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = bits & (1u << e) ? v[e] : 0xFF800000u;
            }
            most(v);
            const float t = top();
            const float whole = fabsf(t) < kAtWhole ? t : ceilf(t);
            if (x == 0 && c == 0) {
              m = whole;
            } else if (__any_sync(0xffffffffu, t > m + kAtSlack)) {
              // (2^-256 is zero: then, and where nothing is written yet, any distance does)
              const float up = t - m < 256.0f && (c > 0 || fabsf(t) < kAtWhole) ? m + ceilf(t - m) : whole;
              const float mn = t > m + kAtSlack ? up : m;
              const float alpha = exp2_fast(m - mn);
              const uint32_t f = pack2_bf16(alpha, alpha);
              m = mn;
              l *= alpha;
              sum[0] = mul2(sum[0], two(alpha, alpha));
              sum[1] = mul2(sum[1], two(alpha, alpha));
              tmem_wait_st();
#pragma unroll 1
              for (int d = 0; d < c; ++d) {
                uint32_t o[16];
                tmem_ld16(s_at + 16 * d, o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = mul_bf16x2(o[e], f);
                tmem_st16(s_at + 16 * d, o);
              }
              // (S_w full: the products into O_w before it have ended)
#pragma unroll 1
              for (int c0 = 0; c0 < HD && x > 0; c0 += 16) {
                uint32_t o[16];
                tmem_ld16(o_at + w * HD + c0, o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st16(o_at + w * HD + c0, o);
              }
            }
            // from kAtCoarse on the reference is rounded to whole units: scores are
            // then rounded like it before it is taken off
            coarse = __any_sync(0xffffffffu, fabsf(m) > kAtCoarse && m != kKvLeast);
            const float f = coarse ? 1.0f : a.c;
            if (coarse) {
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__fmul_rn(__uint_as_float(v[e]), a.c));
            }
            const uint64_t cc = two(f, f), mm = two(-m, -m);
            uint32_t pw[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float x0, x1;
              untwo(fma2(two(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), cc, mm), x0, x1);
              x0 = exp2_fast(x0);
              x1 = exp2_fast(x1);
              sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], two(x0, x1));
              pw[e / 2] = pack2_bf16(x0, x1);
            }
            tmem_st16(s_at + 16 * c, pw);
          }
        }
        float l0, l1;
        untwo(add2(sum[0], sum[1]), l0, l1);
        l += l0 + l1;
        tmem_wait_st();
        tmem_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_ready[w]);
      }
      if (!ok) break;
      // ---- results: O_w of 128 pairs, or both groups' parts of the same pairs, half of the columns each
      if (mine > 0) {
        ok = __all_sync(0xffffffffu, at_wait(&sm.o_full[w], o_count & 1, &sm.abort_flag));
        if (!ok) break;
        ++o_count;
      }
      float f0 = 1.0f, f1 = 0.0f;
      const bool both = split && n > 1;
      if (split) {
        if (w == 0 || mine > 0) {
          sm.ml[w][r][0] = m;
          sm.ml[w][r][1] = l;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.merged);
        ok = __all_sync(0xffffffffu, at_wait(&sm.merged, merges++ & 1, &sm.abort_flag));
        if (!ok) break;
        if (!both) {
          m = sm.ml[0][r][0];
          l = sm.ml[0][r][1];
        } else {
          const float m0 = sm.ml[0][r][0], m1 = sm.ml[1][r][0];
          m = fmaxf(m0, m1);
          f0 = exp2_fast(m0 - m);
          f1 = exp2_fast(m1 - m);
          l = sm.ml[0][r][1] * f0 + sm.ml[1][r][1] * f1;
        }
      }
      tmem_after();
      const int c_lo = split ? w * (HD / 2) : 0, c_hi = split ? c_lo + HD / 2 : HD;
      const uint32_t o_mine = split ? o_at : o_at + w * HD;
      const bool dirty = *(volatile const int*)&p.dirty;
      const long long row = (long long)(o0 + i) * (a.n_kv << a.g_shift) + g * G + (pr & (G - 1));
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      // A thread writes its row, 32 bytes at a time: whole sectors.
      uint16_t* out = (uint16_t*)a.out + row * HD;
      const bool out32 = !((uintptr_t)a.out & 31);
      float* piece = p.slot < 0 ? nullptr : a.part + ((2ll * blockIdx.x + p.slot) * kAtPairs + pr) * (HD + 4);
      uint32_t v[32];
      tmem_ld(o_mine + c_lo, v);
#pragma unroll 1
      for (int c0 = c_lo; c0 < c_hi; c0 += 32) {
        float y[32];
        tmem_wait_ld();
        tmem_ready(v);
#pragma unroll
        for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(v[e]);
        if (both) {
          tmem_ld(o_at + HD + c0, v);
          tmem_wait_ld();
          tmem_ready(v);
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = y[e] * f0 + __uint_as_float(v[e]) * f1;
        }
        if (c0 + 32 < c_hi) tmem_ld(o_mine + c0 + 32, v);
        if (dirty && live) {
          // what the row sees of the entries that were taken out
          for (int t = max(s_lo, p.edge) * kAtStep; t < min(p.end, (s_lo + n) * kAtStep); ++t) {
            if (!row_sees(words, i, t, base, rows)) continue;
            const int blk = a.kv.block_table[(long long)p.b * a.kv.max_blocks + (t >> 4)];
            if (blk < 0 || blk >= a.kv.num_blocks) continue;
            const uint16_t* vr = (const uint16_t*)a.kv.v_pool + (((long long)blk * a.n_kv + g) * kBlk + (t & 15)) * HD + c0;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if ((vr[e] & 0x7F80u) == 0x7F80u) y[e] += elem<uint16_t>(vr + e);
          }
        }
        if (piece) {   // (rows of HD + 4 floats: on 16 bytes)
          if (live) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) *reinterpret_cast<float4*>(piece + c0 + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
          }
          continue;
        }
        uint32_t z[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) z[e] = pack2_bf16(y[2 * e] * inv, y[2 * e + 1] * inv);
        if (live && MTP_IN_BOUNDS(a.err, row * HD + c0 + 31, (long long)a.T * (a.n_kv << a.g_shift) * HD)) {
          if (out32) {
            st_global32(out + c0, z);
            st_global32(out + c0 + 16, z + 8);
          } else {
#pragma unroll
            for (int e = 0; e < 16; e += 4) *reinterpret_cast<uint4*>(out + c0 + 2 * e) = make_uint4(z[e], z[e + 1], z[e + 2], z[e + 3]);
          }
        }
      }
      if (live && c_lo == 0 && piece) *reinterpret_cast<float2*>(piece + HD) = make_float2(m, l);
      if (live && c_lo == 0 && p.slot < 0 && a.lse) a.lse[row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
      if (split) {
        // the other group's part is read: it may go on to its next products
        tmem_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.merged);
        ok = __all_sync(0xffffffffu, at_wait(&sm.merged, merges++ & 1, &sm.abort_flag));
        if (!ok) break;
        tmem_after();
      }
      tmem_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.piece_empty[np & 1]);
    }
    if (!ok) {
      sm.abort_flag = 1;
      if (lane == 0) set_error(a.err, MTP_ERR_TIMEOUT);
    }
  }
  tmem_before();
  __syncthreads();
  if (warp == 9) {
    tmem_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

// Sorts a call's tiles by their steps (counting sort, the largest first), or
// leaves the call to the split in equal shares where that is the better one:
// where a segment is larger than a share, or too few of them would leave SMs
// idle at the end.  Causal prompts: the split's pieces cost a segment's write
// and read in float32, all thread blocks at the same time, and a start and
// an end each (8192 rows 512 -> 406 us, 4096 rows 185 -> 138).
constexpr int kPlanThreads = 1024;
constexpr int kPlanBins = 1024;
__global__ void __launch_bounds__(kPlanThreads) rows_plan_kernel(const RowsArgs a, const SegShape sh, int blocks) {
  __shared__ int before[kKvMaxB + 1];    // tiles before each request
  __shared__ int bins[kPlanBins];
  __shared__ long long warps[32];
  __shared__ int most_s;
  pdl_wait();
  pdl_trigger();
  const int b = threadIdx.x, lane = b & 31, warp = b >> 5;
  const bool masked = a.mask != nullptr;
  static_assert(kKvMaxB <= kPlanThreads, "a thread a request");
  int bad = 0, tiles = 0, most = 0;
  long long units = 0;
  if (b == 0) most_s = 0;
  if (b < kPlanBins) bins[b] = 0;
  if (b < a.B) {
    const int r0 = a.row_offsets[b], r1 = a.row_offsets[b + 1];
    if (r0 < 0 || r1 < r0 || r1 > a.T) {
      bad = 1;
    } else if (r1 > r0) {
      int o0, n, L;
      const int e = rows_request(a, b, o0, n, L);
      if (e != MTP_OK) {
        set_error(a.err, e);   // (that request is left out)
      } else {
        tiles = seg_tiles(sh, n);
        units = a.n_kv * seg_units_before(sh, tiles, L - n, n, masked);
        most = ceil_shift(L, sh.step);
      }
    }
  }
  // sums over the requests: tiles in the low 31 bits, units above (tiles of a call fit: T < 2^30)
  bad = __syncthreads_or(bad);
  auto scan = [&](long long v, long long& all) {
    long long x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 31) warps[warp] = x;
    __syncthreads();
    long long add = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < 32; ++w) {
      if (w < warp) add += warps[w];
      all += warps[w];
    }
    return add + x - v;
  };
  long long all_tiles, all_units;
  const long long tile0 = scan(tiles, all_tiles);
  scan(units, all_units);
  if (b < a.B) before[b] = (int)min(tile0, (long long)INT32_MAX);
  if (b == 0) before[a.B] = (int)min(all_tiles, (long long)INT32_MAX);
  if (tiles) atomicMax(&most_s, most);
  __syncthreads();
  const long long share = (all_units + blocks - 1) / blocks;
  const bool sort = !bad && all_tiles <= kPlanTiles && all_tiles * a.n_kv >= 2 * blocks && most_s + sh.lead <= share;
  if (b == 0) {
    a.plan[0] = sort;
    a.plan[1] = sort ? (int)(all_tiles * a.n_kv) : 0;
    a.plan[2] = 0;
  }
  if (!sort) return;
  const int nt = (int)all_tiles;
  auto find = [&](int e, int& req, int& tile) {   // entry e, and its bin (0: the most steps)
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int m = (lo + hi) >> 1;
      if (before[m] <= e) lo = m;
      else hi = m;
    }
    req = lo;
    tile = e - before[lo];
    int o0, n, L;
    rows_request(a, lo, o0, n, L);
    const int steps = ceil_shift(seg_end(sh, tile, L - n, n, masked), sh.step);
    return kPlanBins - 1 - (int)((long long)steps * (kPlanBins - 1) / most_s);
  };
  int req, tile;
  for (int e = b; e < nt; e += kPlanThreads) atomicAdd(&bins[find(e, req, tile)], 1);
  __syncthreads();
  long long none;
  const int at = (int)scan(bins[b], none);
  __syncthreads();
  bins[b] = at;
  __syncthreads();
  int2* list = reinterpret_cast<int2*>(a.plan + 4);
  for (int e = b; e < nt; e += kPlanThreads) {
    const int bin = find(e, req, tile);
    list[atomicAdd(&bins[bin], 1)] = make_int2(req, tile);
  }
}

template <int HD>
static cudaError_t attn_tc_launch(mtp_ctx* ctx, cudaStream_t s, RowsArgs a) {
  using S = AtShape<HD>;
  CUtensorMap qm, km, vm;
  const uint64_t rows = (uint64_t)a.kv.num_blocks * a.n_kv * kBlk;
  if (rows > INT32_MAX || !make_block_map(&km, a.kv.k_pool, rows, HD) || !make_block_map(&vm, a.kv.v_pool, rows, HD))
    return cudaErrorInvalidValue;
  qm = km;   // (not read where the queries cannot be mapped)
  if (a.q_vec && !make_query_map(&qm, a.q, a.q_stride, a.T, a.n_kv << a.g_shift, 1 << a.g_shift, HD)) return cudaErrorInvalidValue;
  const cudaError_t e = ensure_smem((const void*)kv_attn_tc_kernel<HD>, S::kBytes);
  if (e != cudaSuccess) return e;
  const SegShape sh{8 - a.g_shift, 7, 2};   // 256 pairs, 128 slots
  static_assert(kAtPairs == 1 << 8 && kAtStep == 1 << 7, "shifts");
  // enough rows for two segments a thread block: the plan may sort them
  if (((long long)a.T << a.g_shift) * a.n_kv < 2ll * kAtPairs * ctx->num_sms) {
    a.plan = nullptr;
  } else {
    const cudaError_t pe = launch_pdl(rows_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, a, sh, ctx->num_sms);
    if (pe != cudaSuccess) return pe;
    ctx->launches++;
  }
  return launch_pdl(kv_attn_tc_kernel<HD>, dim3(ctx->num_sms), dim3(kAtThreads), S::kBytes, s, qm, km, vm, a, sh);
}
cudaError_t launch_attn_tc(mtp_ctx* ctx, cudaStream_t s, const RowsArgs& a) {
  return ctx->cfg.head_dim == 128 ? attn_tc_launch<128>(ctx, s, a) : attn_tc_launch<64>(ctx, s, a);
}

}  // namespace mtp
