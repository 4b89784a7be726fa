// Attention of new rows over the paged cache, and the attention weight that
// its entries gather, on the float32 pipe: the form for float32 heads.
//
//   out[r, h] = sum_t p_t V[t, g] / sum_t p_t,  p_t = 2^(c s_t - m),
//   s_t = q[r, h] . K[t, g], c = scale * log2 e, m the running maximum;
//   w[t, g] += sum_{r, h} 2^(c s_t - log2 e * lse[r, h]).
//
// The (row, query head) pairs that share a kv head are the rows of a tile; a
// step takes 64 slots.  16 x 16 threads hold RT x 4 scores each and read both
// operands from shared memory as float4 (queries and keys transposed), so that
// for RT = 4 two shared loads feed sixteen multiply-adds and the float32 pipe is
// the bound; RT = 1 serves decoding rows, which are bound by the cache's bytes.
#include <math.h>

#include "mtp_kv16.cuh"

namespace mtp {

constexpr int kRowsThreads = 256;
constexpr int kRowsStep = 64;       // slots of a step
constexpr int kRowsPitch = kRowsStep + 4;

template <bool V> struct Flag { static constexpr bool value = V; };

template <int HD, int RT>
struct RowsShape {
  static constexpr int kRows = 16 * RT;                    // pairs of a tile
  static constexpr int kQ = HD * kRows, kK = HD * kRowsPitch;   // floats
  static constexpr int kWeightBytes = (kQ + kK) * 4;
};
template <int HD, int RT>
struct AttnShape {
  static constexpr int kRows = 16 * RT;
  static constexpr int kQ = HD * kRows, kP = kRows * (kRowsStep + 4);   // floats
  static constexpr int kBytes = (kQ + kP + 2 * 2 * kRowsStep * HD) * 4;
};

// Queries of a tile, transposed: qs[d][pair]; pairs past the request's rows are zero.
template <typename T, int HD, int ROWS>
__device__ __forceinline__ void load_queries(const RowsArgs& a, float* qs, int o0, int i0, int n, int g) {
  const int G = 1 << a.g_shift;
  for (int x = threadIdx.x; x < ROWS * (HD / 4); x += kRowsThreads) {
    const int r = x % ROWS, d = x / ROWS * 4, i = i0 + (r >> a.g_shift);
    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (i < n) {
      const T* p = (const T*)a.q + (long long)(o0 + i) * a.q_stride + (long long)(g * G + (r & (G - 1))) * HD + d;
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = elem<T>(p + e);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) qs[(d + e) * ROWS + r] = y[e];
  }
}

// Entries of a step: keys transposed (ks[d][slot]) or values as they lie
// (vs[slot][d]).  Slots from `end` on, and blocks outside the pool, are zero.
template <typename T, int HD, bool TRANSPOSE>
__device__ __forceinline__ void load_entries(const RowsArgs& a, const void* pool, float* dst, const int* blocks, int t0,
                                             int end, int g) {
  for (int x = threadIdx.x; x < kRowsStep * (HD / 4); x += kRowsThreads) {
    int t, d;
    if (TRANSPOSE) {   // a warp takes 8 slots x 4 quads: whole sectors, two lanes a bank
      const int w = x >> 5, l = x & 31;
      t = (w % (kRowsStep / 8)) * 8 + (l & 7);
      d = ((w / (kRowsStep / 8)) * 4 + (l >> 3)) * 4;
    } else {
      t = x / (HD / 4);
      d = x % (HD / 4) * 4;
    }
    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const int blk = blocks[t >> 4];
    if (t0 + t < end && blk >= 0) {
      const T* p = (const T*)pool + (((long long)blk * a.n_kv + g) * kBlk + (t & 15)) * HD + d;
      if constexpr (sizeof(T) == 4) {
        const float4 u = *reinterpret_cast<const float4*>(p);
        y[0] = u.x; y[1] = u.y; y[2] = u.z; y[3] = u.w;
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        y[0] = bf16_lo(u.x); y[1] = bf16_hi(u.x); y[2] = bf16_lo(u.y); y[3] = bf16_hi(u.y);
      }
    }
    if (TRANSPOSE) {
#pragma unroll
      for (int e = 0; e < 4; ++e) dst[(d + e) * kRowsPitch + t] = y[e];
    } else {
      *reinterpret_cast<float4*>(dst + t * HD + d) = make_float4(y[0], y[1], y[2], y[3]);
    }
  }
}

// The step's block ids (-1: outside the pool).
__device__ __forceinline__ void load_blocks(const RowsArgs& a, int* blocks, int b, int t0, int end) {
  if (threadIdx.x < kRowsStep / kBlk) {
    const int t = t0 + threadIdx.x * kBlk;
    int blk = -1;
    if (t < end) {
      blk = a.kv.block_table[(long long)b * a.kv.max_blocks + (t >> 4)];
      if (blk < 0 || blk >= a.kv.num_blocks) {
        set_error(a.err, MTP_ERR_CAPACITY);
        blk = -1;
      }
    }
    blocks[threadIdx.x] = blk;
  }
}

// Scores of pairs RT ty .. and slots 4 tx ..
template <int HD, int RT>
__device__ __forceinline__ void tile_scores(const float* qs, const float* ks, int ty, int tx, float (&s)[RT][4]) {
  constexpr int ROWS = 16 * RT;
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = 0.0f;
#pragma unroll 8
  for (int d = 0; d < HD; ++d) {
    float q[RT];
    if constexpr (RT == 4) {
      const float4 u = *reinterpret_cast<const float4*>(qs + d * ROWS + 4 * ty);
      q[0] = u.x; q[1] = u.y; q[2] = u.z; q[3] = u.w;
    } else {
      q[0] = qs[d * ROWS + ty];
    }
    const float4 k = *reinterpret_cast<const float4*>(ks + d * kRowsPitch + 4 * tx);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      s[i][0] = fmaf(q[i], k.x, s[i][0]);
      s[i][1] = fmaf(q[i], k.y, s[i][1]);
      s[i][2] = fmaf(q[i], k.z, s[i][2]);
      s[i][3] = fmaf(q[i], k.w, s[i][3]);
    }
  }
}

// 16 bytes global -> shared; none of them (zeros) for bytes = 0.
__device__ __forceinline__ void rows_cp(float* dst, const float* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// Staged rows of HD floats: 16-byte chunk c of row r lies at chunk c ^ (r & 7),
// so that eight lanes that read one chunk of eight rows meet no bank twice.
template <int HD>
__device__ __forceinline__ int rows_at(int r, int c) {
  return r * HD + ((c ^ (r & 7)) << 2);
}

template <int HD, int RT>
__global__ void __launch_bounds__(kRowsThreads) rows_attn_kernel(const RowsArgs a, const SegShape sh) {
  using S = AttnShape<HD, RT>;
  constexpr int ROWS = S::kRows, CH = HD / 4, PASS = kRowsThreads / CH;   // rows that the block copies at a time
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
  if (!rows_split<kRowsThreads>(a, SegUnits{a, sh}, sh.lead + 1, pre, wsum, sp)) return;
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
    // queries, a pair's row at a time; pairs past the request's rows are zero
    for (int x = tid; x < ROWS * CH; x += kRowsThreads) {
      const int r = x / CH, c = x % CH, i = i0 + (r >> a.g_shift);
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (i < p.n) {
        const float* src = (const float*)a.q + (long long)(p.o0 + i) * a.q_stride + (long long)(p.g * G + (r & (G - 1))) * HD + c * 4;
        if (a.q_vec) v = *reinterpret_cast<const float4*>(src);
        else v = make_float4(src[0], src[1], src[2], src[3]);
      }
      *reinterpret_cast<float4*>(qs + r * HD + ((c ^ (r / RT & 7)) << 2)) = v;
    }
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

// Thread block (step of slots, kv head, request): the weights of 64 entries, its
// keys kept in shared memory, all rows that may see them in tiles of 64 pairs.
template <typename T, int HD>
__global__ void __launch_bounds__(kRowsThreads) rows_weights_kernel(const RowsArgs a) {
  constexpr int RT = 4, ROWS = 64;
  using S = RowsShape<HD, RT>;
  extern __shared__ __align__(16) float smem[];
  __shared__ int blocks[kRowsStep / kBlk];
  __shared__ float lse_s[ROWS];
  __shared__ float sums[16][kRowsStep + 1];
  float* qs = smem;
  float* ks = qs + S::kQ;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int t0 = blockIdx.x * kRowsStep, g = blockIdx.y, b = blockIdx.z, G = 1 << a.g_shift;
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
  load_blocks(a, blocks, b, t0, L);
  __syncthreads();
  load_entries<T, HD, true>(a, a.kv.k_pool, ks, blocks, t0, L, g);
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const int row0 = a.mask ? 0 : max(0, t0 - base);   // rows before it see none of these slots
  const int tile_rows = ROWS >> a.g_shift;
  for (int i0 = row0; i0 < n; i0 += tile_rows) {
    __syncthreads();
    load_queries<T, HD, ROWS>(a, qs, o0, i0, n, g);
    if (tid < ROWS) {
      const int i = i0 + (tid >> a.g_shift);
      const float l = i < n ? a.lse[(long long)(o0 + i) * (a.n_kv << a.g_shift) + g * G + (tid & (G - 1))] : -INFINITY;
      lse_s[tid] = l == -INFINITY ? INFINITY : l * kLog2e;   // a row that sees nothing weighs nothing
    }
    __syncthreads();
    float s[RT][4];
    tile_scores<HD, RT>(qs, ks, ty, tx, s);
    const bool edge = t0 + kRowsStep > base + (a.mask ? 0 : i0 + 1) || i0 + tile_rows > n;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int r = ty * RT + i, row = i0 + (r >> a.g_shift);
      const int32_t* words = a.mask && row < n ? a.mask + (long long)(o0 + row) * a.mask_words : nullptr;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = t0 + 4 * tx + j;
        if (!edge || (row < n && t < L && row_sees(words, row, t, base, n)))
          acc[j] += exp2f(fmaf(s[i][j], a.c, -lse_s[r]));
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) sums[ty][4 * tx + j] = acc[j];
  __syncthreads();
  const int t = t0 + tid;
  if (tid < kRowsStep && t < L && blocks[tid >> 4] >= 0) {
    float x = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) x += sums[i][tid];
    const long long at = ((long long)blocks[tid >> 4] * a.n_kv + g) * kBlk + (t & 15);
    if (MTP_IN_BOUNDS(a.err, at, (long long)a.kv.num_blocks * a.n_kv * kBlk))
      a.weights[at] = (t < first ? a.weights[at] : 0.0f) + x;
  }
}

template <typename T, int HD>
static cudaError_t rows_join_launch(cudaStream_t s, const RowsArgs& a, int grid, int pairs) {
  const int per = kRowsJoinThreads / (HD / 4);
  const long long most = (long long)a.max_rows << a.g_shift;   // pairs of a segment
  const int groups = ((int)(most < pairs ? most : pairs) + per - 1) / per;
  return launch_pdl(rows_join_kernel<T, HD>, dim3(grid, groups), dim3(kRowsJoinThreads), 0, s, a, pairs);
}

template <int HD, int RT>
static cudaError_t rows_attn_launch(mtp_ctx* ctx, cudaStream_t s, const RowsArgs& a) {
  using S = AttnShape<HD, RT>;
  cudaError_t e = ensure_smem((const void*)rows_attn_kernel<HD, RT>, S::kBytes);
  if (e != cudaSuccess) return e;
  const SegShape sh{(RT == 1 ? 4 : 6) - a.g_shift, 6, 2};   // 16 or 64 pairs, 64 slots
  static_assert(S::kRows == (RT == 1 ? 16 : 64) && kRowsStep == 64, "shifts");
  const int grid = (HD == 64 ? 2 : 1) * ctx->num_sms;   // what shared memory holds
  e = launch_pdl(rows_attn_kernel<HD, RT>, dim3(grid), dim3(kRowsThreads), S::kBytes, s, a, sh);
  return e != cudaSuccess ? e : rows_join_launch<float, HD>(s, a, grid, S::kRows);
}
static cudaError_t launch_rows_attn(mtp_ctx* ctx, cudaStream_t s, const RowsArgs& a) {
  ctx->launches += 2;
  if (ctx->cfg.dtype == MTP_DTYPE_BF16) {
    const cudaError_t e = launch_attn_tc(ctx, s, a);
    if (e != cudaSuccess) return e;
    return ctx->cfg.head_dim == 128 ? rows_join_launch<uint16_t, 128>(s, a, ctx->num_sms, kAtPairs)
                                    : rows_join_launch<uint16_t, 64>(s, a, ctx->num_sms, kAtPairs);
  }
  const bool few = (a.max_rows << a.g_shift) <= 16;
  if (ctx->cfg.head_dim == 128) return few ? rows_attn_launch<128, 1>(ctx, s, a) : rows_attn_launch<128, 4>(ctx, s, a);
  return few ? rows_attn_launch<64, 1>(ctx, s, a) : rows_attn_launch<64, 4>(ctx, s, a);
}

template <int HD>
static cudaError_t rows_weights_launch(mtp_ctx* ctx, cudaStream_t s, const RowsArgs& a) {
  const int smem = RowsShape<HD, 4>::kWeightBytes;
  const cudaError_t e = ensure_smem((const void*)rows_weights_kernel<float, HD>, smem);
  if (e != cudaSuccess) return e;
  const int tiles = (int)(((long long)a.kv.max_blocks * kBlk + kRowsStep - 1) / kRowsStep);
  return launch_pdl(rows_weights_kernel<float, HD>, dim3(tiles, a.n_kv, a.B), dim3(kRowsThreads), smem, s, a);
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
  const int pairs = ctx->cfg.dtype == MTP_DTYPE_BF16 ? kAtPairs : kRowsMaxBlocks * 64;   // of an SM's thread blocks
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
