// Attention of new rows over the paged cache, and the attention weight that
// its entries gather, on the float32 pipe: the form for float32 heads.
//
//   out[r, h] = sum_t p_t V[t, g] / sum_t p_t,  p_t = 2^(c s_t - m),
//   s_t = q[r, h] . K[t, g], c = scale * log2 e, m the running maximum;
//   w[t, g] += sum_{r, h} 2^(c s_t - log2 e * lse[r, h]).
//
// The (row, query head) pairs that share a kv head are the rows of a tile;
// segments are cut over the thread blocks and joined as on the tensor cores.
//
// Few pairs (up to 32): a call is bound by the cache's bytes, and what has to be
// short is the chain from an entry's arrival to the next.  Each warp keeps a
// softmax of its own over eight slots of a step, copies those itself and waits
// for nobody: a ring of halves (a step's keys, a step's values) holds 192 KB.
// Four lanes share a key and hold its parts in registers; three exchanges sum
// four pairs' products over them, so that each lane ends with one pair's score.
// The warps' results are joined once a segment.  32 requests of 0 to 4096
// entries, 32 query and 8 kv heads of 128: 102 us, 5.2 TB/s of entries (386 us
// when a tile's threads shared one softmax and met twice a step).  Tiles of 8
// pairs run 16 warps at 128 registers, tiles of 32 run 8 at 255: for 4 pairs
// that is 102 us against 131; 24 pairs take 86 us against 136 in tiles of 64.
//
// Many pairs: the float32 pipe is the bound.  16 x 16 threads hold 4 x 4 scores
// each, entries come in two stages; 256 rows on 16000 entries: 2.22 ms, 30
// TFLOP/s (tiles of 32 as above: 3.42 ms).
//
// Weights: keys stay in registers, sixteen slots a warp, and the rows pass;
// 32 decoding requests as above 77 us (385 us with the keys in shared memory),
// 256 rows on 16000 entries 1.15 ms (1.86 ms).
#include <math.h>

#include "mtp_kv16.cuh"

namespace mtp {

constexpr int kRowsThreads = 256;
constexpr int kRowsStep = 64;       // slots of a step
constexpr int kRowsPairs = 64;      // pairs of a tile
constexpr int kRowsShare = 2;       // units of a thread block at least: trees of 33 rows 21.7 us (three: 26.2, one: 22.2)
constexpr int kWeightSlots = 128;   // slots of a thread block of the weights' kernel, sixteen a warp
constexpr int kWeightPairs = 64;

template <bool V> struct Flag { static constexpr bool value = V; };

// Few pairs: a ring of halves, each the keys or the values of a step.
template <int HD, int PAIRS>
struct FewShape {
  static constexpr int kWarps = PAIRS == 8 ? 16 : 8, kThreads = 32 * kWarps, kStep = 8 * kWarps;
  static constexpr int kHalf = kStep * HD, kRing = 49152 / kHalf;   // floats; halves
  static constexpr int kQ = PAIRS * HD, kP = kWarps * PAIRS * 8;
  static constexpr int kBytes = (kQ + kP + kRing * kHalf) * 4;
  static_assert(kRing * kHalf >= kWarps * PAIRS * (HD + 2), "the warps' results are joined in the ring's place");
};
// Many pairs: two stages of keys and values.
template <int HD>
struct ManyShape {
  static constexpr int kQ = HD * kRowsPairs, kP = kRowsPairs * (kRowsStep + 4);   // floats
  static constexpr int kBytes = (kQ + kP + 2 * 2 * kRowsStep * HD) * 4;
};

// 16 bytes global -> shared; none of them (zeros) unless `there`.
__device__ __forceinline__ void rows_cp(float* dst, const float* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// Staged rows of HD floats: 16-byte chunk c of row r lies at chunk c ^ (r & 7).
template <int HD>
__device__ __forceinline__ int rows_at(int r, int c) {
  return r * HD + ((c ^ (r & 7)) << 2);
}

// Queries of a tile, a pair's row at a time; pairs past the request's rows are zero.
// (SPREAD: four rows by four, 16-byte chunk c lies at chunk c ^ (r / 4 & 7).)
template <int HD, int PAIRS, int THREADS, bool SPREAD>
__device__ __forceinline__ void load_queries(const RowsArgs& a, float* qs, int o0, int i0, int n, int g) {
  constexpr int CH = HD / 4;
  const int G = 1 << a.g_shift;
  for (int x = threadIdx.x; x < PAIRS * CH; x += THREADS) {
    const int r = x / CH, c = x % CH, i = i0 + (r >> a.g_shift);
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (i < n) {
      const float* src = (const float*)a.q + (long long)(o0 + i) * a.q_stride + (long long)(g * G + (r & (G - 1))) * HD + c * 4;
      if (a.q_vec) v = *reinterpret_cast<const float4*>(src);
      else v = make_float4(src[0], src[1], src[2], src[3]);
    }
    *reinterpret_cast<float4*>(qs + r * HD + ((SPREAD ? c ^ (r / 4 & 7) : c) << 2)) = v;
  }
}

// The slot of eight that a lane takes, together with three lanes beside it (chunks lane % 4, + 4, ...): lanes 8 j ..
// 8 j + 7 read rows j and j + 4 of a stage, whose chunks lie in different banks.
__device__ __forceinline__ int lane_slot(int lane) { return (lane >> 2 & 1) * 4 + (lane >> 3); }

// Scores of four pairs (rows of qs from `q` on) and the NS keys of which this lane and the three beside it hold the
// parts: lane % 4 = j gets pair j's.  Three exchanges sum four pairs over four lanes.
template <int HD, int NS>
__device__ __forceinline__ void four_scores(const float* q, const float4 (&k)[NS][HD / 16], int lane, float (&s)[NS]) {
  uint64_t acc[NS][4];
#pragma unroll
  for (int n = 0; n < NS; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[n][j] = 0;   // two zeros
#pragma unroll
  for (int i = 0; i < HD / 16; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 x = *reinterpret_cast<const float4*>(q + j * HD + ((lane & 3) + 4 * i) * 4);
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        acc[n][j] = fma2(two(x.x, x.y), two(k[n][i].x, k[n][i].y), acc[n][j]);
        acc[n][j] = fma2(two(x.z, x.w), two(k[n][i].z, k[n][i].w), acc[n][j]);
      }
    }
#pragma unroll
  for (int n = 0; n < NS; ++n) {
    float y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float lo, hi;
      untwo(acc[n][j], lo, hi);
      y[j] = lo + hi;
    }
    const bool b0 = lane & 1, b1 = lane & 2;
    const float e = (b0 ? y[1] : y[0]) + __shfl_xor_sync(0xffffffffu, b0 ? y[0] : y[1], 1);
    const float f = (b0 ? y[3] : y[2]) + __shfl_xor_sync(0xffffffffu, b0 ? y[2] : y[3], 1);
    s[n] = (b1 ? f : e) + __shfl_xor_sync(0xffffffffu, b1 ? e : f, 2);
  }
}

template <int HD, int PAIRS>
__global__ void __launch_bounds__(FewShape<HD, PAIRS>::kThreads, 1) rows_few_kernel(const RowsArgs a, const SegShape sh) {
  using S = FewShape<HD, PAIRS>;
  constexpr int CH = HD / 4, NG = PAIRS / 4, RING = S::kRing, PASS = 32 / CH, STEP = S::kStep;
  extern __shared__ __align__(16) float smem[];
  __shared__ int pre[kKvMaxB + 1];
  __shared__ long long wsum[S::kWarps];
  float* qs = smem;                       // [pairs][HD]
  float* kv = qs + S::kQ + S::kP;         // [RING][STEP][HD]
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, G = 1 << a.g_shift;
  float* ps = qs + S::kQ + w * (PAIRS * 8);   // this warp's, [pair][8 slots]
  if (tid == 0) a.meta[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
  Split sp;
  if (!rows_split<S::kThreads>(a, SegUnits{a, sh}, kRowsShare, pre, wsum, sp)) return;
  for (uint32_t u = sp.u0; u < sp.u1;) {
    Piece p;
    find_piece(a, sh, pre, sp, u, p);
    u = p.next;
    if (p.s_lo >= p.s_hi) continue;
    const int i0 = p.tile << sh.rows, valid = min(PAIRS, (p.n - i0) << a.g_shift);
    const int32_t* table = a.kv.block_table + (long long)p.b * a.kv.max_blocks;
    // a warp copies its own eight slots, which lie in one block; its id is looked up a step ahead
    int id = 0, id_v = 0;
    auto look = [&](int step) {
      const int t = step * STEP + w * 8;
      id = step < p.s_hi && t < p.end ? table[t >> 4] : 0;
    };
    // unit h: the keys (h even) or values of step s_lo + h / 2
    auto copy = [&](int h, int at) {
      const int step = p.s_lo + (h >> 1);
      if (step < p.s_hi) {
        if (!(h & 1)) id_v = id;
        const int t0 = step * STEP + w * 8;
        const bool good = id_v >= 0 && id_v < a.kv.num_blocks;
        const int live = good ? p.end - t0 : 0;
        const int r0 = lane / CH, c = lane % CH;
        float* dst = kv + at * S::kHalf + w * 8 * HD;
        const float* src = (const float*)(h & 1 ? a.kv.v_pool : a.kv.k_pool) +
                           (((long long)(good ? id_v : 0) * a.n_kv + p.g) * kBlk + (t0 & 15) + r0) * HD + c * 4;
#pragma unroll
        for (int x = 0; x < 8 / PASS; ++x) {
          const int t = r0 + x * PASS;
          rows_cp(dst + rows_at<HD>(t, c), src + x * PASS * HD, t < live);
        }
        if (!good && t0 < p.end && lane == 0) set_error(a.err, MTP_ERR_CAPACITY);
        if (!(h & 1)) look(step + 1);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    look(p.s_lo);
    __syncthreads();              // the last piece's results are read
#pragma unroll
    for (int x = 0; x < RING - 1; ++x) copy(x, x);
    load_queries<HD, PAIRS, S::kThreads, false>(a, qs, p.o0, i0, p.n, p.g);
    __syncthreads();
    // o: four columns of every pair; m and l: lane % 4 = j has the maximum of pair 4 x + j, and its slot's share of the sum
    float o[PAIRS][4], m[NG], l[NG];
#pragma unroll
    for (int x = 0; x < NG; ++x) {
      m[x] = kKvLeast;
      l[x] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < PAIRS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;
    int at = 0;     // where unit h lies
    // the next unit's place, which the last one leaves, is filled; then unit h is there
    auto next = [&](int h) -> const float* {
      __syncwarp();
      copy(h + RING - 1, at == 0 ? RING - 1 : at - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(RING - 1) : "memory");
      __syncwarp();
      const float* here = kv + at * S::kHalf + w * 8 * HD;
      at = at == RING - 1 ? 0 : at + 1;
      return here;
    };
    for (int step = p.s_lo; step < p.s_hi; ++step) {
      const int t0 = step * STEP, h = 2 * (step - p.s_lo);
      // slots that some row of the tile does not see: from the first new one that its first row may not see
      const bool edge = t0 + STEP > p.base + (a.mask ? 0 : i0 + 1);
      const float* ks = next(h);
      const int sl = lane_slot(lane), t = t0 + w * 8 + sl;
      float4 k[1][HD / 16];
#pragma unroll
      for (int i = 0; i < HD / 16; ++i) k[0][i] = *reinterpret_cast<const float4*>(ks + rows_at<HD>(sl, (lane & 3) + 4 * i));
#pragma unroll
      for (int x = 0; x < NG; ++x) {
        if (4 * x >= valid) break;
        float s[1];
        four_scores<HD, 1>(qs + 4 * x * HD, k, lane, s);
        s[0] *= a.c;
        bool seen = true;
        if (edge) {
          const int row = i0 + ((4 * x + (lane & 3)) >> a.g_shift);
          const int32_t* words = a.mask && row < p.n ? a.mask + (long long)(p.o0 + row) * a.mask_words : nullptr;
          seen = row < p.n && t < p.end && row_sees(words, row, t, p.base, p.n);
        }
        if (__any_sync(0xffffffffu, seen && s[0] > m[x])) {
          float mx = seen ? s[0] : kKvLeast;
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
          mx = fmaxf(m[x], mx);
          const float alpha = exp2f(m[x] - mx);
          m[x] = mx;
          l[x] *= alpha;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float f = __shfl_sync(0xffffffffu, alpha, j);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[4 * x + j][e] *= f;
          }
        }
        const float e = seen ? exp2f(s[0] - m[x]) : 0.0f;
        l[x] += e;
        // (-1: unseen, so that 0 times an entry that is not finite is left out)
        ps[(4 * x + (lane & 3)) * 8 + sl] = seen ? e : -1.0f;
      }
      const float* vs = next(h + 1);
      auto values = [&](auto checked) {
        // heads of 64 take four slots a half warp
#pragma unroll
        for (int h = 0; h < CH / 16; ++h) {
          const int first = HD == 128 ? 4 * h : lane / CH * 4;
          float4 v[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) v[y] = *reinterpret_cast<const float4*>(vs + rows_at<HD>(first + y, lane % CH));
#pragma unroll
          for (int x = 0; x < NG; ++x) {
            if (4 * x >= valid) break;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float e[4];
              *reinterpret_cast<float4*>(e) = *reinterpret_cast<const float4*>(ps + (4 * x + j) * 8 + first);
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                if (decltype(checked)::value && e[y] == -1.0f) continue;
                o[4 * x + j][0] = fmaf(e[y], v[y].x, o[4 * x + j][0]);
                o[4 * x + j][1] = fmaf(e[y], v[y].y, o[4 * x + j][1]);
                o[4 * x + j][2] = fmaf(e[y], v[y].z, o[4 * x + j][2]);
                o[4 * x + j][3] = fmaf(e[y], v[y].w, o[4 * x + j][3]);
              }
            }
          }
        }
      };
      if (edge) values(Flag<true>{});
      else values(Flag<false>{});
    }
    // ---- the warps' results joined, in the ring's place
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    float* os = kv;                                        // [warp][pair][HD]
    float* ml = kv + S::kWarps * PAIRS * HD;         // [warp][pair][2]
#pragma unroll
    for (int x = 0; x < NG; ++x) {
      if (4 * x >= valid) break;
      float sum = l[x];
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (lane < 4) *reinterpret_cast<float2*>(ml + (w * PAIRS + 4 * x + lane) * 2) = make_float2(m[x], sum);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float4 y = make_float4(o[4 * x + j][0], o[4 * x + j][1], o[4 * x + j][2], o[4 * x + j][3]);
        if (HD == 64) {
          y.x += __shfl_xor_sync(0xffffffffu, y.x, 16);
          y.y += __shfl_xor_sync(0xffffffffu, y.y, 16);
          y.z += __shfl_xor_sync(0xffffffffu, y.z, 16);
          y.w += __shfl_xor_sync(0xffffffffu, y.w, 16);
        }
        if (lane < CH) *reinterpret_cast<float4*>(os + (w * PAIRS + 4 * x + j) * HD + lane * 4) = y;
      }
    }
    __syncthreads();
    const bool whole = p.c_first == p.c_last;
    const int slot = (int)blockIdx.x == p.c_first ? 1 : 0;
    for (int x = tid; x < valid * CH; x += S::kThreads) {
      const int r = x / CH, c = x % CH;
      float M = kKvLeast, L = 0.0f;
#pragma unroll
      for (int y = 0; y < S::kWarps; ++y) M = fmaxf(M, ml[(y * PAIRS + r) * 2]);
      float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int y = 0; y < S::kWarps; ++y) {
        const float2 z = *reinterpret_cast<const float2*>(ml + (y * PAIRS + r) * 2);
        const float4 v = *reinterpret_cast<const float4*>(os + (y * PAIRS + r) * HD + c * 4);
        const float f = exp2f(z.x - M);
        L = fmaf(z.y, f, L);
        sum.x = fmaf(v.x, f, sum.x);
        sum.y = fmaf(v.y, f, sum.y);
        sum.z = fmaf(v.z, f, sum.z);
        sum.w = fmaf(v.w, f, sum.w);
      }
      if (whole) {
        const long long row = (long long)(p.o0 + i0 + (r >> a.g_shift)) * (a.n_kv << a.g_shift) + p.g * G + (r & (G - 1));
        rows_finish<float, HD>(a, row, c, sum, M, L);
      } else {
        float* pr = a.part + ((2ll * blockIdx.x + slot) * PAIRS + r) * (HD + 4);
        *reinterpret_cast<float4*>(pr + 4 * c) = sum;
        if (c == 0) *reinterpret_cast<float2*>(pr + HD) = make_float2(M, L);
      }
    }
    if (tid == 0 && slot == 1 && !whole) {
      a.meta[2 * blockIdx.x] = make_int4(p.c_last - p.c_first + 1, p.c_first, valid, p.g);
      a.meta[2 * blockIdx.x + 1] = make_int4(p.o0 + i0, 0, 0, 0);
    }
  }
}

template <int HD>
__global__ void __launch_bounds__(kRowsThreads) rows_many_kernel(const RowsArgs a, const SegShape sh) {
  using S = ManyShape<HD>;
  constexpr int RT = 4, ROWS = kRowsPairs, CH = HD / 4, PASS = kRowsThreads / CH;   // rows that the block copies at a time
  constexpr int OC = HD / 64;     // float4 columns of the result per thread and pair
  constexpr int PP = kRowsStep + 4;
  extern __shared__ __align__(16) float smem[];
  __shared__ int pre[kKvMaxB + 1];
  __shared__ long long wsum[kRowsThreads / 32];
  float* qs = smem;                       // [ROWS][HD]
  float* ps = qs + S::kQ;                 // [ROWS][PP]
  float* kv = ps + S::kP;                 // [2][keys, values][kRowsStep][HD]
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, G = 1 << a.g_shift;
  if (tid == 0) a.meta[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
  Split sp;
  if (!rows_split<kRowsThreads>(a, SegUnits{a, sh}, kRowsShare, pre, wsum, sp)) return;
  for (uint32_t u = sp.u0; u < sp.u1;) {
    Piece p;
    find_piece(a, sh, pre, sp, u, p);
    u = p.next;
    if (p.s_lo >= p.s_hi) continue;
    const int i0 = p.tile << sh.rows;
    const int32_t* table = a.kv.block_table + (long long)p.b * a.kv.max_blocks;
    // a step's block ids, the same for all threads; looked up a step ahead of the copy
    int ids[kRowsStep / kBlk];
    auto look = [&](int step) {
#pragma unroll
      for (int i = 0; i < kRowsStep / kBlk; ++i) {
        const int t = step * kRowsStep + i * kBlk;
        ids[i] = step < p.s_hi && t < p.end ? table[t >> 4] : 0;
      }
    };
    auto copy = [&](int step, int stage) {
      if (step < p.s_hi) {
        const int c = tid % CH, t0 = step * kRowsStep;
        float* dst = kv + stage * (2 * kRowsStep * HD);
#pragma unroll
        for (int x = 0; x < kRowsStep / PASS; ++x) {
          const int t = tid / CH + x * PASS, blk = ids[x * PASS / kBlk];
          const bool good = blk >= 0 && blk < a.kv.num_blocks, there = good && t0 + t < p.end;
          const long long at = (((long long)(there ? blk : 0) * a.n_kv + p.g) * kBlk + (t & 15)) * HD + c * 4;
          rows_cp(dst + rows_at<HD>(t, c), (const float*)a.kv.k_pool + at, there);
          rows_cp(dst + kRowsStep * HD + rows_at<HD>(t, c), (const float*)a.kv.v_pool + at, there);
          if (!good && t0 + t < p.end && c == 0) set_error(a.err, MTP_ERR_CAPACITY);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    look(p.s_lo);
    __syncthreads();              // the last piece's tiles are done with
    copy(p.s_lo, 0);
    look(p.s_lo + 1);
    load_queries<HD, ROWS, kRowsThreads, true>(a, qs, p.o0, i0, p.n, p.g);
    float o[RT][OC][4], m[RT], l[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      m[i] = kKvLeast;
      l[i] = 0.0f;
#pragma unroll
      for (int c = 0; c < OC; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][c][e] = 0.0f;
    }
    for (int step = p.s_lo; step < p.s_hi; ++step) {
      const int t0 = step * kRowsStep, stage = (step - p.s_lo) & 1;
      // slots that some row of the tile does not see: from the first new one that its first row may not see
      const bool edge = t0 + kRowsStep > p.base + (a.mask ? 0 : i0 + 1);
      copy(step + 1, stage ^ 1);
      look(step + 2);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncthreads();
      const float* ks = kv + stage * (2 * kRowsStep * HD);
      const float* vs = ks + kRowsStep * HD;
      // scores of pairs RT ty .. and slots tx + 16 j
      float s[RT][4];
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.0f;
#pragma unroll 4
      for (int c = 0; c < CH; ++c) {
        float4 k[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) k[j] = *reinterpret_cast<const float4*>(ks + rows_at<HD>(tx + 16 * j, c));
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const float4 q = *reinterpret_cast<const float4*>(qs + (ty * RT + i) * HD + ((c ^ (ty & 7)) << 2));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[i][j] = fmaf(q.x, k[j].x, s[i][j]);
            s[i][j] = fmaf(q.y, k[j].y, s[i][j]);
            s[i][j] = fmaf(q.z, k[j].z, s[i][j]);
            s[i][j] = fmaf(q.w, k[j].w, s[i][j]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int row = i0 + ((ty * RT + i) >> a.g_shift);
        const int32_t* words = a.mask && row < p.n ? a.mask + (long long)(p.o0 + row) * a.mask_words : nullptr;
        bool seen[4];
        float mx = kKvLeast;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = t0 + tx + 16 * j;
          seen[j] = !edge || (row < p.n && t < p.end && row_sees(words, row, t, p.base, p.n));
          s[i][j] *= a.c;
          if (seen[j]) mx = fmaxf(mx, s[i][j]);
        }
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float mn = fmaxf(m[i], mx), alpha = exp2f(m[i] - mn);
        m[i] = mn;
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = seen[j] ? exp2f(s[i][j] - mn) : 0.0f;
          sum += e;
          // (-1: unseen, so that 0 times an entry that is not finite is left out)
          ps[(ty * RT + i) * PP + tx + 16 * j] = seen[j] ? e : -1.0f;
        }
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        l[i] = l[i] * alpha + sum;
#pragma unroll
        for (int c = 0; c < OC; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][c][e] *= alpha;
      }
      __syncwarp();   // a warp reads back only its own pairs
      auto values = [&](auto checked) {
#pragma unroll 2
        for (int t = 0; t < kRowsStep; t += 4) {
          float w[RT][4];
#pragma unroll
          for (int i = 0; i < RT; ++i)
            *reinterpret_cast<float4*>(w[i]) = *reinterpret_cast<const float4*>(ps + (ty * RT + i) * PP + t);
#pragma unroll
          for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int c = 0; c < OC; ++c) {
              const float4 v = *reinterpret_cast<const float4*>(vs + rows_at<HD>(t + y, 16 * c + tx));
#pragma unroll
              for (int i = 0; i < RT; ++i) {
                if (decltype(checked)::value && w[i][y] == -1.0f) continue;
                o[i][c][0] = fmaf(w[i][y], v.x, o[i][c][0]);
                o[i][c][1] = fmaf(w[i][y], v.y, o[i][c][1]);
                o[i][c][2] = fmaf(w[i][y], v.z, o[i][c][2]);
                o[i][c][3] = fmaf(w[i][y], v.w, o[i][c][3]);
              }
            }
        }
      };
      if (edge) values(Flag<true>{});
      else values(Flag<false>{});
      __syncthreads();   // the stage is free for the step after the next
    }
    // ---- results, or a piece of them
    const bool whole = p.c_first == p.c_last;
    const int slot = (int)blockIdx.x == p.c_first ? 1 : 0;
    const int valid = min(ROWS, (p.n - i0) << a.g_shift);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int r = ty * RT + i;
      if (r >= valid) continue;
      const long long row = (long long)(p.o0 + i0 + (r >> a.g_shift)) * (a.n_kv << a.g_shift) + p.g * G + (r & (G - 1));
#pragma unroll
      for (int c = 0; c < OC; ++c) {
        const float4 x = make_float4(o[i][c][0], o[i][c][1], o[i][c][2], o[i][c][3]);
        if (whole) {
          rows_finish<float, HD>(a, row, 16 * c + tx, x, m[i], l[i]);
        } else {
          float* pr = a.part + ((2ll * blockIdx.x + slot) * ROWS + r) * (HD + 4);
          *reinterpret_cast<float4*>(pr + 64 * c + 4 * tx) = x;
          if (c == 0 && tx == 0) *reinterpret_cast<float2*>(pr + HD) = make_float2(m[i], l[i]);
        }
      }
    }
    if (tid == 0 && slot == 1 && !whole) {
      a.meta[2 * blockIdx.x] = make_int4(p.c_last - p.c_first + 1, p.c_first, valid, p.g);
      a.meta[2 * blockIdx.x + 1] = make_int4(p.o0 + i0, 0, 0, 0);
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Joins the pieces of the segments that span thread blocks: thread block (x,
// y) takes the segment that begins in the first kernel's block x, and of its
// pairs the y-th group; a thread owns four elements of a pair.
constexpr int kRowsJoinThreads = 256;
template <typename T, int HD>
__global__ void __launch_bounds__(kRowsJoinThreads) rows_join_kernel(const RowsArgs a, int rows) {
  constexpr int LANES = HD / 4, PER = kRowsJoinThreads / LANES, AHEAD = 4;
  pdl_wait();
  pdl_trigger();
  const int4 seg = a.meta[2 * blockIdx.x];
  if (seg.x == 0) return;
  const int first_row = a.meta[2 * blockIdx.x + 1].x, d4 = threadIdx.x % LANES, G = 1 << a.g_shift;
  for (int r = blockIdx.y * PER + threadIdx.x / LANES; r < seg.z; r += PER * gridDim.y) {
    float M = kKvLeast, Ls = 0.0f;
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int k0 = 0; k0 < seg.x; k0 += AHEAD) {
      float2 ml[AHEAD];
      float4 y[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {   // no branches: all loads go out together
        const int kk = min(k0 + k, seg.x - 1);
        const float* pr = a.part + ((2ll * (seg.y + kk) + (kk == 0 ? 1 : 0)) * rows + r) * (HD + 4);
        ml[k] = __ldcg(reinterpret_cast<const float2*>(pr + HD));
        y[k] = __ldcg(reinterpret_cast<const float4*>(pr) + d4);
      }
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        if (k0 + k >= seg.x) break;
        const float mn = fmaxf(M, ml[k].x), f0 = exp2f(M - mn), f1 = exp2f(ml[k].x - mn);
        Ls = Ls * f0 + ml[k].y * f1;
        x.x = x.x * f0 + y[k].x * f1;
        x.y = x.y * f0 + y[k].y * f1;
        x.z = x.z * f0 + y[k].z * f1;
        x.w = x.w * f0 + y[k].w * f1;
        M = mn;
      }
    }
    const long long row = (long long)(first_row + (r >> a.g_shift)) * (a.n_kv << a.g_shift) + seg.w * G + (r & (G - 1));
    rows_finish<T, HD>(a, row, d4, x, M, Ls);
  }
}

// Thread block (128 slots, kv head, request): the weights of its entries, whose
// keys stay in registers; all rows that may see them pass in tiles of 64 pairs.
template <int HD>
__global__ void __launch_bounds__(kRowsThreads, 2) rows_weights_kernel(const RowsArgs a) {
  extern __shared__ __align__(16) float qs[];   // [pairs][HD]
  __shared__ float lse_s[kWeightPairs];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int t0 = blockIdx.x * kWeightSlots, g = blockIdx.y, b = blockIdx.z, G = 1 << a.g_shift;
  int bad = 0;
  for (int x = tid; x < a.B; x += kRowsThreads) {
    const int r0 = a.row_offsets[x], r1 = a.row_offsets[x + 1];
    bad |= r0 < 0 || r1 < r0 || r1 > a.T;
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) set_error(a.err, MTP_ERR_DEVICE_ARGS);
    return;
  }
  int o0, n, L;
  const int err = rows_request(a, b, o0, n, L);
  if (n == 0) return;
  const int base = L - n, first = a.first ? a.first[b] : base;
  if (err != MTP_OK || first < 0) {
    if (tid == 0 && t0 == 0 && g == 0) set_error(a.err, err != MTP_OK ? err : MTP_ERR_DEVICE_ARGS);
    return;
  }
  if (t0 >= L) return;
  // a warp's sixteen slots are a block; a lane has parts of two of them
  const int tw = t0 + w * kBlk, sl = lane_slot(lane);
  int blk = -1;
  if (tw < L) {
    blk = a.kv.block_table[(long long)b * a.kv.max_blocks + tw / kBlk];
    if (blk < 0 || blk >= a.kv.num_blocks) {
      if (lane == 0) set_error(a.err, MTP_ERR_CAPACITY);
      blk = -1;
    }
  }
  float4 k[2][HD / 16];
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int i = 0; i < HD / 16; ++i) {
      k[x][i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (blk >= 0)   // (slots from L on are read and not used)
        k[x][i] = reinterpret_cast<const float4*>((const float*)a.kv.k_pool + (((long long)blk * a.n_kv + g) * kBlk + sl + 8 * x) * HD)[(lane & 3) + 4 * i];
    }
  float acc[2] = {0.0f, 0.0f};
  const int row0 = a.mask ? 0 : max(0, t0 - base);   // rows before it see none of these slots
  const int tile_rows = kWeightPairs >> a.g_shift;
  for (int i0 = row0; i0 < n; i0 += tile_rows) {
    const int valid = min(kWeightPairs, (n - i0) << a.g_shift);
    __syncthreads();
    load_queries<HD, kWeightPairs, kRowsThreads, false>(a, qs, o0, i0, n, g);
    if (tid < kWeightPairs) {
      const int i = i0 + (tid >> a.g_shift);
      const float l = i < n ? a.lse[(long long)(o0 + i) * (a.n_kv << a.g_shift) + g * G + (tid & (G - 1))] : -INFINITY;
      lse_s[tid] = l == -INFINITY ? INFINITY : l * kLog2e;   // a row that sees nothing weighs nothing
    }
    __syncthreads();
    const bool edge = t0 + kWeightSlots > base + (a.mask ? 0 : i0 + 1) || valid % 4;
    for (int x = 0; x < valid; x += 4) {
      float s[2];
      four_scores<HD, 2>(qs + x * HD, k, lane, s);
      const int r = x + (lane & 3), row = i0 + (r >> a.g_shift);
      const float l = lse_s[r];
      const int32_t* words = a.mask && row < n ? a.mask + (long long)(o0 + row) * a.mask_words : nullptr;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int t = tw + sl + 8 * y;
        if (!edge || (row < n && t < L && row_sees(words, row, t, base, n))) acc[y] += exp2f(fmaf(s[y], a.c, -l));
      }
    }
  }
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    acc[y] += __shfl_xor_sync(0xffffffffu, acc[y], 1);
    acc[y] += __shfl_xor_sync(0xffffffffu, acc[y], 2);
  }
  const int t = tw + sl + 8 * (lane & 1);
  if ((lane & 2) == 0 && t < L && blk >= 0) {
    const long long at = ((long long)blk * a.n_kv + g) * kBlk + (t & 15);
    if (MTP_IN_BOUNDS(a.err, at, (long long)a.kv.num_blocks * a.n_kv * kBlk))
      a.weights[at] = (t < first ? a.weights[at] : 0.0f) + (lane & 1 ? acc[1] : acc[0]);
  }
}

template <typename T, int HD>
static cudaError_t rows_join_launch(cudaStream_t s, const RowsArgs& a, int grid, int pairs) {
  const int per = kRowsJoinThreads / (HD / 4);
  const long long most = (long long)a.max_rows << a.g_shift;   // pairs of a segment
  const int groups = ((int)(most < pairs ? most : pairs) + per - 1) / per;
  return launch_pdl(rows_join_kernel<T, HD>, dim3(grid, groups), dim3(kRowsJoinThreads), 0, s, a, pairs);
}

template <int HD>
static cudaError_t rows_attn_launch(mtp_ctx* ctx, cudaStream_t s, const RowsArgs& a) {
  const int pairs = (int)((long long)a.max_rows << a.g_shift < kRowsPairs ? a.max_rows << a.g_shift : kRowsPairs);
  const int tile = pairs <= 8 ? 8 : pairs <= 32 ? 32 : kRowsPairs;
  const int grid = (tile == kRowsPairs && HD == 64 ? 2 : 1) * ctx->num_sms;   // what shared memory holds
  const auto go = [&](auto kernel, int threads, int bytes, int step) {
    const cudaError_t e = ensure_smem((const void*)kernel, bytes);
    const SegShape sh{(tile == 8 ? 3 : tile == 32 ? 5 : 6) - a.g_shift, step, 2};
    return e != cudaSuccess ? e : launch_pdl(kernel, dim3(grid), dim3(threads), bytes, s, a, sh);
  };
  static_assert(FewShape<HD, 8>::kStep == 128 && FewShape<HD, 32>::kStep == 64 && kRowsStep == 64 && kRowsPairs == 64, "shifts");
  cudaError_t e;
  if (tile == 8) e = go(rows_few_kernel<HD, 8>, FewShape<HD, 8>::kThreads, FewShape<HD, 8>::kBytes, 7);
  else if (tile == 32) e = go(rows_few_kernel<HD, 32>, FewShape<HD, 32>::kThreads, FewShape<HD, 32>::kBytes, 6);
  else e = go(rows_many_kernel<HD>, kRowsThreads, ManyShape<HD>::kBytes, 6);
  return e != cudaSuccess ? e : rows_join_launch<float, HD>(s, a, grid, tile);
}
static cudaError_t launch_rows_attn(mtp_ctx* ctx, cudaStream_t s, const RowsArgs& a) {
  ctx->launches += 2;
  if (ctx->cfg.dtype == MTP_DTYPE_BF16) {
    const cudaError_t e = launch_attn_tc(ctx, s, a);
    if (e != cudaSuccess) return e;
    return ctx->cfg.head_dim == 128 ? rows_join_launch<uint16_t, 128>(s, a, ctx->num_sms, kAtPairs)
                                    : rows_join_launch<uint16_t, 64>(s, a, ctx->num_sms, kAtPairs);
  }
  return ctx->cfg.head_dim == 128 ? rows_attn_launch<128>(ctx, s, a) : rows_attn_launch<64>(ctx, s, a);
}

template <int HD>
static cudaError_t rows_weights_launch(mtp_ctx* ctx, cudaStream_t s, const RowsArgs& a) {
  const int smem = kWeightPairs * HD * 4;
  const cudaError_t e = ensure_smem((const void*)rows_weights_kernel<HD>, smem);
  if (e != cudaSuccess) return e;
  const int tiles = (int)(((long long)a.kv.max_blocks * kBlk + kWeightSlots - 1) / kWeightSlots);
  return launch_pdl(rows_weights_kernel<HD>, dim3(tiles, a.n_kv, a.B), dim3(kRowsThreads), smem, s, a);
}
static cudaError_t launch_rows_weights(mtp_ctx* ctx, cudaStream_t s, const RowsArgs& a) {
  ctx->launches++;
  if (ctx->cfg.dtype == MTP_DTYPE_BF16) return launch_weights_tc(ctx, s, a);
  return ctx->cfg.head_dim == 128 ? rows_weights_launch<128>(ctx, s, a) : rows_weights_launch<64>(ctx, s, a);
}

// Workspace: what the join kernel joins, then two pieces a thread block.
constexpr int kRowsMaxBlocks = 2;    // thread blocks per SM at most
static size_t rows_meta_bytes(const mtp_ctx* ctx) { return (size_t)kRowsMaxBlocks * ctx->num_sms * 2 * sizeof(int4); }
constexpr size_t kPlanBytes = (4 + 2 * (size_t)kPlanTiles) * sizeof(int);
static size_t rows_pre_bytes(const mtp_ctx* ctx) {
  return ((size_t)ctx->num_sms * (kKvMaxB + 1) * sizeof(int) + 255) & ~(size_t)255;
}

// The checks that both calls share; fills in the common arguments.
static mtp_status rows_args(mtp_ctx* ctx, int B, int T, const int32_t* row_offsets, int max_rows, const void* q,
                            int64_t q_stride, const mtp_kv* kv, const int32_t* mask, int mask_words, float scale,
                            RowsArgs& a) {
  if (!ctx || B < 1 || B > ctx->cfg.max_batch || B > kKvMaxB || T < 0 || T > (1 << 30) || !row_offsets || !q ||
      !kv16_ok(kv))
    return MTP_ERR_INVALID;
  const mtp_config& c = ctx->cfg;
  if (max_rows < 1 || q_stride < (int64_t)c.n_q_heads * c.head_dim) return MTP_ERR_INVALID;
  if (mask && (max_rows > 256 || mask_words < (max_rows + 31) / 32)) return MTP_ERR_INVALID;
  if (!(scale > 0.0f) || !isfinite(scale)) return MTP_ERR_INVALID;
  a.q = q;
  a.row_offsets = row_offsets;
  a.mask = mask;
  a.kv = *kv;
  a.err = ctx->err;
  a.q_stride = q_stride;
  a.B = B;
  a.T = T;
  a.max_rows = max_rows;
  a.mask_words = mask_words;
  a.n_kv = c.n_kv_heads;
  a.g_shift = group_shift(c);
  const int per16 = c.dtype == MTP_DTYPE_BF16 ? 8 : 4;
  a.q_vec = !((uintptr_t)q & 15) && q_stride % per16 == 0;
  a.c = scale * kLog2e;
  return MTP_OK;
}

}  // namespace mtp

using namespace mtp;

extern "C" {

size_t mtp_kv_attention_workspace_bytes(const mtp_ctx* ctx) {
  if (!ctx) return 0;
  const int pairs = ctx->cfg.dtype == MTP_DTYPE_BF16 ? kAtPairs : kRowsMaxBlocks * kRowsPairs;   // of an SM's thread blocks
  return rows_meta_bytes(ctx) + rows_pre_bytes(ctx) + kPlanBytes + (size_t)2 * ctx->num_sms * pairs * (ctx->cfg.head_dim + 4) * sizeof(float);
}

mtp_status mtp_kv_attention(mtp_ctx* ctx, void* stream, int B, int T, const int32_t* row_offsets, int max_rows,
                            const void* q, int64_t q_stride, const mtp_kv* kv, const int32_t* mask, int mask_words,
                            float scale, void* out, float* lse, void* ws, size_t ws_bytes) {
  RowsArgs a{};
  const mtp_status st = rows_args(ctx, B, T, row_offsets, max_rows, q, q_stride, kv, mask, mask_words, scale, a);
  if (st != MTP_OK) return st;
  if (!out || ((uintptr_t)out & 15) || !ws || ((uintptr_t)ws & 15) || ws_bytes < mtp_kv_attention_workspace_bytes(ctx))
    return MTP_ERR_INVALID;
  if (T == 0) return MTP_OK;
  DeviceGuard dev(ctx->device);
  if (!dev.ok) return MTP_ERR_CUDA;
  a.out = out;
  a.lse = lse;
  a.meta = (int4*)ws;
  a.pre = (int*)((char*)ws + rows_meta_bytes(ctx));
  a.plan = (int*)((char*)ws + rows_meta_bytes(ctx) + rows_pre_bytes(ctx));
  a.part = (float*)((char*)a.plan + kPlanBytes);
  return launch_status(launch_rows_attn(ctx, (cudaStream_t)stream, a));
}

mtp_status mtp_kv_attention_weights(mtp_ctx* ctx, void* stream, int B, int T, const int32_t* row_offsets, int max_rows,
                                    const void* q, int64_t q_stride, const mtp_kv* kv, const int32_t* mask,
                                    int mask_words, float scale, const float* lse, const int32_t* first,
                                    float* weights) {
  RowsArgs a{};
  const mtp_status st = rows_args(ctx, B, T, row_offsets, max_rows, q, q_stride, kv, mask, mask_words, scale, a);
  if (st != MTP_OK) return st;
  if (!lse || !weights || a.n_kv > 65535) return MTP_ERR_INVALID;
  if (T == 0) return MTP_OK;
  DeviceGuard dev(ctx->device);
  if (!dev.ok) return MTP_ERR_CUDA;
  a.lse = const_cast<float*>(lse);
  a.first = first;
  a.weights = weights;
  return launch_status(launch_rows_weights(ctx, (cudaStream_t)stream, a));
}

}  // extern "C"
