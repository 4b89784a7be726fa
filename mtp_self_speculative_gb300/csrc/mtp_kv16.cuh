// What the operators on the paged cache in the context's type share: element
// access, the checks of a cache, a request's place in a call, and how a
// call's work is split over thread blocks.
#pragma once

#include "mtp_kv8.cuh"

namespace mtp {

constexpr int kKvMaxB = 1024;                 // requests of a call (prefix sums in shared memory)
constexpr int kKvMaxSlots = 1 << 30;          // entries of a request: slots and the ends of tiles are ints
constexpr float kKvLeast = -3.4028235e38f;    // the softmax reference of a row that has seen nothing
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

inline bool kv16_ok(const mtp_kv* kv) {
  return kv && kv->k_pool && kv->v_pool && kv->block_table && kv->seq_len && kv->pending && kv->num_blocks > 0 &&
         kv->max_blocks > 0 && !((uintptr_t)kv->k_pool & 15) && !((uintptr_t)kv->v_pool & 15);
}

inline int group_shift(const mtp_config& c) {
  int s = 0;
  while ((1 << s) < c.n_q_heads / c.n_kv_heads) ++s;
  return s;
}

template <typename T> __device__ __forceinline__ float elem(const T* p);
template <> __device__ __forceinline__ float elem<float>(const float* p) { return *p; }
template <> __device__ __forceinline__ float elem<uint16_t>(const uint16_t* p) {
  return __uint_as_float((uint32_t)*p << 16);
}

// 16 bytes as floats.
template <typename T>
__device__ __forceinline__ void widen16(uint4 u, float* x) {
  if constexpr (sizeof(T) == 2) {
    x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x); x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
    x[4] = bf16_lo(u.z); x[5] = bf16_hi(u.z); x[6] = bf16_lo(u.w); x[7] = bf16_hi(u.w);
  } else {
    x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y); x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
  }
}
__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <typename T>
__device__ __forceinline__ uint4 narrow16(const float* x) {
  if constexpr (sizeof(T) == 2)
    return make_uint4(pack2_bf16(x[0], x[1]), pack2_bf16(x[2], x[3]), pack2_bf16(x[4], x[5]), pack2_bf16(x[6], x[7]));
  else
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}

// 2^x to 2^-22 of its value; results below 2^-126 are zero.
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two floats at a time.
__device__ __forceinline__ uint64_t two(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void untwo(uint64_t x, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// --------------------------------------- attention of new rows over a cache
struct RowsArgs {
  const void* q;
  void* out;
  float* lse;                    // attention: written (may be null); weights: read
  const int32_t* row_offsets;
  const int32_t* mask;
  mtp_kv kv;
  int* err;
  long long q_stride;
  int B, T, max_rows, mask_words, n_kv, g_shift;
  int q_vec;                     // query rows allow 16-byte loads
  float c;                       // scale * log2(e)
  // attention: pieces of segments that span thread blocks
  float* part;                   // [2 * grid][rows of a segment][HD + 4]: o, then reference and sum
  int4* meta;                    // [2 * grid]: per thread block, the spanning segment that begins in it
  int* pre;                      // tensor-core form: [grid][kKvMaxB + 1] units before each request
  int* plan;                     // tensor-core form, or null: RowsPlan
  // weights
  float* weights;                // [num_blocks, n_kv, 16]
  const int32_t* first;          // [B] or null
};

constexpr int kAtPairs = 256;      // pairs of a tile of the tensor-core kernel

// The tensor-core form of the attention (bf16 heads); its pieces are joined as
// the other form's.
cudaError_t launch_attn_tc(mtp_ctx* ctx, cudaStream_t s, const RowsArgs& a);
// The same of the entries' weights.
cudaError_t launch_weights_tc(mtp_ctx* ctx, cudaStream_t s, const RowsArgs& a);

// A call's segments in the order of their size, for calls of many segments:
// whole ones are then handed out, the largest first, and none leaves pieces.
// plan[0]: 1, or 0 for the split in equal shares; plan[1]: items (a tile and a
// kv head each); plan[2]: the next item; from plan[4] on (request, tile).
constexpr int kPlanTiles = 32768;

// Request b's first row, rows and entries; 0, or the error that leaves it out.
__device__ __forceinline__ int rows_request(const RowsArgs& a, int b, int& o0, int& n, int& L) {
  o0 = a.row_offsets[b];
  const int o1 = a.row_offsets[b + 1], sl = a.kv.seq_len[b], pe = a.kv.pending[b];
  n = o1 - o0;
  const long long len = (long long)sl + pe;
  L = (int)len;
  if (n > a.max_rows || sl < 0 || pe < 0 || len < n) return MTP_ERR_DEVICE_ARGS;
  if (len > (long long)a.kv.max_blocks * kBlk || len > kKvMaxSlots) return MTP_ERR_CAPACITY;
  return MTP_OK;
}

// Whether row i of a request's n new rows sees slot t (row_words: its mask
// words, or null; t below base is seen by every row).
__device__ __forceinline__ bool row_sees(const int32_t* row_words, int i, int t, int base, int n) {
  const int j = t - base;
  if (j < 0) return true;
  if (!row_words) return j <= i;
  return j < n && (row_words[j >> 5] >> (j & 31) & 1);
}

// A segment is (request, kv head, tile of new rows); its steps are tiles of
// STEP slots, from slot 0 to the last one that a row of the tile sees.  Row
// tiles of `rows` rows and steps are powers of two, so the number of steps
// before a tile has a closed form:
//   sum_{y=1..t} ceil((base + y rows) / STEP).
struct SegShape {
  int rows, step;   // shifts: new rows of a tile; slots of a step
  int lead;         // steps that a segment's start and end count for
};
__host__ __device__ __forceinline__ int ceil_shift(int x, int s) { return (x + (1 << s) - 1) >> s; }
__host__ __device__ __forceinline__ long long ceil_sum(long long x, int s) {   // sum_{y=1..x} ceil(y / 2^s)
  const long long a = x >> s, r = x - (a << s);
  return (a * (a + 1) << s >> 1) + r * (a + 1);
}
__host__ __device__ __forceinline__ int seg_tiles(const SegShape& s, int n) { return ceil_shift(n, s.rows); }
// One past the last slot that a row of tile t sees.
__host__ __device__ __forceinline__ int seg_end(const SegShape& s, int t, int base, int n, bool masked) {
  const long long e = (long long)(t + 1) << s.rows;
  return masked || e > n ? base + n : base + (int)e;
}
// Units (steps, and `lead` more for each tile) before tile t of a head.
__host__ __device__ __forceinline__ long long seg_units_before(const SegShape& s, int t, int base, int n, bool masked) {
  const int all = seg_tiles(s, n);
  const long long last = ceil_shift(base + n, s.step);
  if (masked) return t * (last + s.lead);
  const int full = t < all ? t : all - 1;       // tiles that end at a multiple of their rows
  long long u;
  if (s.rows >= s.step) {
    u = full * (long long)ceil_shift(base, s.step) + ((long long)full * (full + 1) / 2 << (s.rows - s.step));
  } else {
    const int c = ceil_shift(base, s.rows), q = s.step - s.rows;
    u = ceil_sum((long long)c + full, q) - ceil_sum(c, q);
  }
  if (t == all) u += last;
  return u + (long long)t * s.lead;
}

// The split of a call: units before each request, and the share of a thread
// block.  Every thread of the block calls rows_split; false: nothing to do.
// units(L, n, b): those of a request with n rows among L entries; less than 0:
// the request is left out as its arguments are wrong.
struct Split {
  int share;        // units of a thread block
  uint32_t u0, u1;  // this block's
};
template <int THREADS, typename F>
__device__ __forceinline__ bool rows_split(const RowsArgs& a, F&& request_units, int min_share, int* pre, long long* wsum,
                                           Split& sp) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  long long carry = 0;
  int bad = 0;
  for (int b0 = 0; b0 < a.B; b0 += THREADS) {
    const int b = b0 + tid;
    long long units = 0;
    if (b < a.B) {
      const int r0 = a.row_offsets[b], r1 = a.row_offsets[b + 1];
      if (r0 < 0 || r1 < r0 || r1 > a.T) {
        bad = 1;
      } else if (r1 > r0) {
        int o0, n, L;
        int e = rows_request(a, b, o0, n, L);
        if (e == MTP_OK) {
          units = request_units(L, n, b);
          if (units < 0) {
            units = 0;
            e = MTP_ERR_DEVICE_ARGS;
          }
        }
        if (e != MTP_OK && blockIdx.x == 0) set_error(a.err, e);
      }
    }
    long long x = units;  // inclusive scan over the block
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    long long add = carry, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) add += wsum[w];
      all += wsum[w];
    }
    if (b < a.B) pre[b + 1] = (int)min(add + x, (long long)INT32_MAX);
    carry += all;
    __syncthreads();
  }
  if (tid == 0) pre[0] = 0;
  const bool refused = __syncthreads_or(bad);
  if (refused || carry > INT32_MAX - (1 << 20)) {   // (or more steps than a call can count)
    if (tid == 0 && blockIdx.x == 0) set_error(a.err, refused ? MTP_ERR_DEVICE_ARGS : MTP_ERR_CAPACITY);
    return false;
  }
  const uint32_t total = (uint32_t)carry;
  sp.share = max((int)((total + gridDim.x - 1) / gridDim.x), min_share);
  const unsigned long long u = (unsigned long long)blockIdx.x * sp.share;
  if (u >= total) return false;
  sp.u0 = (uint32_t)u;
  sp.u1 = (uint32_t)min(u + sp.share, (unsigned long long)total);
  return true;
}

// Units of a request of the attention.
struct SegUnits {
  const RowsArgs& a;
  const SegShape& s;
  __device__ __forceinline__ long long operator()(int L, int n, int) const {
    return a.n_kv * seg_units_before(s, seg_tiles(s, n), L - n, n, a.mask != nullptr);
  }
};

// The part of a segment that falls into a thread block's share.
struct Piece {
  int b, g, tile, o0, n, L, base;
  int end;              // one past the last slot that the tile sees
  int s_lo, s_hi;       // this block's steps
  int c_first, c_last;  // the thread blocks that have steps of the segment
  uint32_t next;        // the first unit after the segment, or the share's end
};
__device__ __forceinline__ void find_piece(const RowsArgs& a, const SegShape& s, const int* pre, const Split& sp,
                                           uint32_t u, Piece& p) {
  int lo = 0, hi = a.B;   // the last request whose units begin at or before u, and that has some
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if ((uint32_t)pre[m] <= u) lo = m;
    else hi = m;
  }
  p.b = lo;
  rows_request(a, lo, p.o0, p.n, p.L);
  p.base = p.L - p.n;
  const bool masked = a.mask != nullptr;
  const int tiles = seg_tiles(s, p.n);
  const uint32_t per_head = (uint32_t)seg_units_before(s, tiles, p.base, p.n, masked);
  const uint32_t rel = u - (uint32_t)pre[lo];
  p.g = (int)(rel / per_head);
  const uint32_t in_head = rel - (uint32_t)p.g * per_head;
  int t0 = 0, t1 = tiles;
  while (t1 - t0 > 1) {
    const int m = (t0 + t1) >> 1;
    if ((uint32_t)seg_units_before(s, m, p.base, p.n, masked) <= in_head) t0 = m;
    else t1 = m;
  }
  p.tile = t0;
  p.end = seg_end(s, t0, p.base, p.n, masked);
  const int steps = ceil_shift(p.end, s.step);
  const uint32_t seg0 = (uint32_t)pre[lo] + (uint32_t)p.g * per_head + (uint32_t)seg_units_before(s, t0, p.base, p.n, masked);
  const uint32_t work0 = seg0 + s.lead, seg1 = work0 + steps;
  p.s_lo = u > work0 ? (int)(u - work0) : 0;
  p.s_hi = sp.u1 > work0 ? (int)(min(sp.u1, seg1) - work0) : 0;
  p.c_first = (int)(work0 / sp.share);
  p.c_last = (int)((seg1 - 1) / sp.share);
  p.next = min(seg1, sp.u1);
}

// The result of column d4 .. d4 + 3 of a (row, query head) and its lse.
template <typename T, int HD>
__device__ __forceinline__ void rows_finish(const RowsArgs& a, long long row, int d4, float4 x, float ref, float sum) {
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  if (!MTP_IN_BOUNDS(a.err, row * HD + d4 * 4 + 3, (long long)a.T * (a.n_kv << a.g_shift) * HD)) return;
  T* op = (T*)a.out + row * HD + d4 * 4;
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint2*>(op) = make_uint2(pack2_bf16(x.x * inv, x.y * inv), pack2_bf16(x.z * inv, x.w * inv));
  else
    *reinterpret_cast<float4*>(op) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
  if (a.lse && d4 == 0) a.lse[row] = sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * kLn2;
}

}  // namespace mtp
