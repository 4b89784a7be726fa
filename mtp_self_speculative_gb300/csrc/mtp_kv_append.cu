// Norms of query and key heads with their rotation, and appending to the paged
// cache in the context's type.
//
//   y = x / sqrt(mean x^2 + eps) * w   over each head,
//   out = magnitude * (a cos - b sin, b cos + a sin) for its pairs (a, b).
//
// The work is a copy with some thirty operations per element, so memory bounds
// it.  HD / 16 lanes share a head, eight pairs each: both members of a pair and
// their cosine stay in one thread, the mean is three (two) shuffles, and a
// thread computes its eight cosines once for all heads that it walks over, the
// next head's elements on their way.  8192 tokens of 32 query and 8 key heads of
// 128, bf16: 33 us, 5.0 TB/s; with values appended to a cache (four prompts,
// 8192 rows) 42 us, 4.3 TB/s.  A batch of 32 tokens is bound by the chain of loads:
// 3.1 us, appended 6.8 us (offsets, lengths and blocks first).  float32, 8192 tokens: 59
// us, 5.7 TB/s, appended 82 us, 4.9 TB/s.
#include <math.h>

#include "mtp_kv16.cuh"

namespace mtp {

constexpr int kNormThreads = 128;

struct NormSide {
  const void* x;         // [T, heads, HD], rows `stride` apart, or null
  const void* w;         // [HD] or null: no norm
  void* out;
  long long stride, out_stride, extent;   // elements; the extent for bounds-checked builds
  int heads, per;        // heads of a thread block
};

struct NormArgs {
  NormSide q, k;
  const void* v;         // append: [T, n_kv, HD]
  long long v_stride;
  const int32_t* positions;
  const int32_t* row_offsets;
  mtp_kv kv;
  int32_t* arrive;
  int* err;
  float eps;
  int B, T, rd;          // rd: rotated elements of a head (0: none)
  int k_groups, v_groups; // grid.y: groups of key heads, of value heads (append), then of query heads
  int v_per;
};

// The eight pairs of a unit: pair-slot j = 8 u + e is the rotating pair j of
// the head, or behind those the two elements rd + 2 (j - rd / 2).
__device__ __forceinline__ void pair_at(int j, int rd, int layout, int& ia, int& ib) {
  if (j >= rd / 2) {
    ia = 2 * j;
    ib = ia + 1;
  } else if (layout == MTP_ROPE_HALF) {
    ia = j;
    ib = j + rd / 2;
  } else {
    ia = 2 * j;
    ib = ia + 1;
  }
}

// Sixteen elements of a head, x[e] and x[8 + e] the members of pair e.  VEC:
// rows on 16 bytes and rd a multiple of 16; then a unit is two runs of eight
// (half layout, rotating) or one of sixteen, and is fetched first and widened
// later, so that a thread has the next head's on its way.
template <typename T, bool VEC> struct Unit {
  static constexpr int N = 16 / sizeof(T);
  uint4 v[VEC ? 16 / N : 1];
  float f[VEC ? 1 : 16];
  __device__ __forceinline__ void load(const T* head, int u, int rd, int layout) {
    if constexpr (VEC) {
      const bool split = layout == MTP_ROPE_HALF && 8 * u < rd / 2;
      const T* pa = head + (split ? 8 * u : 16 * u);
      const T* pb = split ? pa + rd / 2 : pa + 8;
#pragma unroll
      for (int i = 0; i < 8; i += N) {
        v[i / N] = *reinterpret_cast<const uint4*>(pa + i);
        v[(8 + i) / N] = *reinterpret_cast<const uint4*>(pb + i);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        int ia, ib;
        pair_at(8 * u + e, rd, layout, ia, ib);
        f[e] = elem<T>(head + ia);
        f[8 + e] = elem<T>(head + ib);
      }
    }
  }
  __device__ __forceinline__ void get(int u, int rd, int layout, float (&x)[16]) const {
    if constexpr (VEC) {
      const bool split = layout == MTP_ROPE_HALF && 8 * u < rd / 2;
      float y[16];
#pragma unroll
      for (int i = 0; i < 16; i += N) widen16<T>(v[i / N], y + i);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = split ? y[e] : y[2 * e];
        x[8 + e] = split ? y[8 + e] : y[2 * e + 1];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = f[e];
    }
  }
};
template <typename T, bool VEC>
__device__ __forceinline__ void unit_store(T* head, int u, int rd, int layout, const float (&x)[16]) {
  if constexpr (VEC) {
    constexpr int N = 16 / sizeof(T);
    const bool split = layout == MTP_ROPE_HALF && 8 * u < rd / 2;
    T* pa = head + (split ? 8 * u : 16 * u);
    T* pb = split ? pa + rd / 2 : pa + 8;
    float y[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = split ? x[i] : x[(i & 1) * 8 + i / 2];
      y[8 + i] = split ? x[8 + i] : x[(i & 1) * 8 + 4 + i / 2];
    }
#pragma unroll
    for (int i = 0; i < 8; i += N) {
      *reinterpret_cast<uint4*>(pa + i) = narrow16<T>(y + i);
      *reinterpret_cast<uint4*>(pb + i) = narrow16<T>(y + 8 + i);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      int ia, ib;
      pair_at(8 * u + e, rd, layout, ia, ib);
      Elem<T>::store1(head + ia, x[e]);
      Elem<T>::store1(head + ib, x[8 + e]);
    }
  }
}

// Thread block (tokens, group of heads): LPH lanes a token and head.  With
// CACHE groups of value heads are copied into the cache, and keys go there too.
template <typename T, int HD, bool VEC, bool CACHE>
__global__ void __launch_bounds__(kNormThreads) qk_norm_rope_kernel(const NormArgs a,
                                                                    const __grid_constant__ mtp_rope_table tab) {
  constexpr int LPH = HD / 16;
  constexpr int TOK = kNormThreads / LPH;     // tokens of a thread block
  __shared__ long long at_s[TOK];             // append: element offset of a token's slot at kv head 0, or -1
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, u = tid % LPH, t0 = blockIdx.x * TOK, t = t0 + tid / LPH;
  const int y = blockIdx.y;
  const bool keys = y < a.k_groups, vals = CACHE && !keys && y < a.k_groups + a.v_groups, cached = keys || vals;
  const NormSide& s = keys ? a.k : a.q;
  const int group = keys ? y : y - a.k_groups - (vals ? 0 : a.v_groups);
  if constexpr (CACHE) {
    // every thread block looks at all offsets; lengths come along, so that the
    // common batch waits for one round of loads
    int bad = 0, sl0 = 0, pe0 = 0;
    if (tid < TOK) at_s[tid] = -2;            // a row of no request
    if (cached && tid < a.B) {
      sl0 = a.kv.seq_len[tid];
      pe0 = a.kv.pending[tid];
    }
    for (int b = tid; b < a.B; b += kNormThreads) {
      const int o0 = a.row_offsets[b], o1 = a.row_offsets[b + 1];
      bad |= o0 < 0 || o1 < o0 || o1 > a.T;
    }
    if (__syncthreads_or(bad)) {
      if (tid == 0) set_error(a.err, MTP_ERR_DEVICE_ARGS);
      return;
    }
    for (int b = tid; b < a.B; b += kNormThreads) {
      const int o0 = a.row_offsets[b], o1 = a.row_offsets[b + 1];
      const int lo = max(o0, t0), hi = min(o1, t0 + TOK);
      if (lo >= hi) continue;
      if (!cached) {
        for (int x = lo; x < hi; ++x) at_s[x - t0] = 0;
        continue;
      }
      const int sl = b == tid ? sl0 : a.kv.seq_len[b], pe = b == tid ? pe0 : a.kv.pending[b];
      int e = MTP_OK;
      if (sl < 0 || pe < 0 || sl > INT32_MAX - pe) e = MTP_ERR_DEVICE_ARGS;
      else if ((long long)sl + pe + (o1 - o0) > min((long long)a.kv.max_blocks * kBlk, (long long)kKvMaxSlots)) e = MTP_ERR_CAPACITY;
      if (e != MTP_OK) {
        set_error(a.err, e);
        continue;
      }
      int held = -1, blk = 0;
      for (int x = lo; x < hi; ++x) {
        const int slot = sl + pe + (x - o0);
        if (slot >> 4 != held) {
          held = slot >> 4;
          blk = a.kv.block_table[(long long)b * a.kv.max_blocks + held];
          if (blk < 0 || blk >= a.kv.num_blocks) {
            set_error(a.err, MTP_ERR_CAPACITY);
            blk = -1;
          }
        }
        at_s[x - t0] = blk < 0 ? -1 : ((long long)blk * a.k.heads * kBlk + (slot & 15)) * HD;
      }
      // all of the request's thread blocks have read its old length before the
      // last one of them publishes the new one
      const int blocks = (o1 - 1) / TOK - o0 / TOK + 1;
      if (arrive_last(a.arrive + b, blocks * (a.k_groups + a.v_groups))) a.kv.pending[b] = pe + (o1 - o0);
    }
    __syncthreads();
  }
  const bool live = t < a.T && (!CACHE || at_s[tid / LPH] >= 0);
  if (!__any_sync(0xffffffffu, live)) return;
  const long long kv_extent = (long long)a.kv.num_blocks * a.k.heads * kBlk * HD;
  (void)kv_extent;   // bounds-checked builds only
  if constexpr (CACHE) {
    if (vals) {        // a copy
      if (!live) return;
      const T* src = (const T*)a.v + (long long)t * a.v_stride;
#pragma unroll 4
      for (int h = group * a.v_per; h < min(a.k.heads, (group + 1) * a.v_per); ++h) {
        const long long at = at_s[tid / LPH] + (long long)h * kBlk * HD;
        if (!MTP_IN_BOUNDS(a.err, at + HD - 1, kv_extent)) continue;
        T* dst = (T*)a.kv.v_pool + at;
        if constexpr (VEC) {
          constexpr int N = 16 / sizeof(T);
#pragma unroll
          for (int i = 0; i < 16 / N; ++i)
            *reinterpret_cast<uint4*>(dst + (i * LPH + u) * N) = *reinterpret_cast<const uint4*>(src + h * HD + (i * LPH + u) * N);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) dst[i * LPH + u] = src[h * HD + i * LPH + u];
        }
      }
      return;
    }
  }
  const int h0 = group * s.per, h1 = min(s.heads, h0 + s.per);
  const int rd = a.rd;
  // two pairs at a time: (a, b) become (a c - b s, b c + a s), as rope_first and
  // rope_second round them
  uint64_t cc[4], ss[4], wa[4], wb[4];
  const int pos = live && rd ? a.positions[t] : 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 c[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int j = 8 * u + 2 * i + e;
      c[e] = j < rd / 2 ? rope_cos_sin(pos, tab.turns[j], tab.magnitude) : make_float2(1.0f, 0.0f);
    }
    cc[i] = two(c[0].x, c[1].x);
    ss[i] = two(c[0].y, c[1].y);
  }
  {
    float w[16];
    if (s.w) {
      Unit<T, false> v;
      v.load((const T*)s.w, u, rd, tab.layout);
      v.get(u, rd, tab.layout, w);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      wa[i] = s.w ? two(w[2 * i], w[2 * i + 1]) : 0ull;
      wb[i] = s.w ? two(w[8 + 2 * i], w[9 + 2 * i]) : 0ull;
    }
  }
  const int turns = rd / 2 - 8 * u;       // pairs of the unit that turn: all from 8 on (VEC: 8 or none)
  // Each thread has its next head on its way.  (out may be x, so the compiler may
  // not fetch it ahead of the store by itself; two or three heads ahead cost
  // more in registers than they gain.)
  const T* row = (const T*)s.x + (long long)(live ? t : 0) * s.stride;
  Unit<T, VEC> ahead;
  ahead.load(row + (long long)h0 * HD, u, rd, tab.layout);
  for (int h = h0; h < h1; ++h) {
    float x[16];
    ahead.get(u, rd, tab.layout, x);
    if (h + 1 < h1) ahead.load(row + (long long)(h + 1) * HD, u, rd, tab.layout);
    uint64_t A[4], B[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      A[i] = two(x[2 * i], x[2 * i + 1]);
      B[i] = two(x[8 + 2 * i], x[9 + 2 * i]);
    }
    if (s.w) {
      uint64_t q0 = mul2(A[0], A[0]), q1 = mul2(B[0], B[0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) {
        q0 = fma2(A[i], A[i], q0);
        q1 = fma2(B[i], B[i], q1);
      }
      float lo, hi;
      untwo(add2(q0, q1), lo, hi);
      float sq = lo + hi;
#pragma unroll
      for (int o = 1; o < LPH; o <<= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
      const float r = rsqrtf(sq * (1.0f / HD) + a.eps);
      const uint64_t rr = two(r, r);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        A[i] = mul2(mul2(A[i], rr), wa[i]);
        B[i] = mul2(mul2(B[i], rr), wb[i]);
      }
    }
    if (!live) continue;
    if (turns > 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t p = fma2(A[i], cc[i], mul2(B[i], ss[i]) ^ 0x8000000080000000ull);   // minus
        const uint64_t q = fma2(B[i], cc[i], mul2(A[i], ss[i]));
        // pairs behind the rotated part stay as they are (0 times an infinite partner
        // is not 0); the lower half of A[i] and B[i] is the first of their two pairs
        const uint64_t stay = VEC || turns >= 2 * i + 2 ? 0ull : turns == 2 * i + 1 ? 0xFFFFFFFF00000000ull : ~0ull;
        A[i] = (A[i] & stay) | (p & ~stay);
        B[i] = (B[i] & stay) | (q & ~stay);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      untwo(A[i], x[2 * i], x[2 * i + 1]);
      untwo(B[i], x[8 + 2 * i], x[9 + 2 * i]);
    }
    if (CACHE && keys) {
      const long long at = at_s[tid / LPH] + (long long)h * kBlk * HD;
      if (MTP_IN_BOUNDS(a.err, at + HD - 1, kv_extent))
        unit_store<T, VEC>((T*)a.kv.k_pool + at, u, rd, tab.layout, x);
    } else {
      const long long at = (long long)t * s.out_stride + (long long)h * HD;
      if (MTP_IN_BOUNDS(a.err, at + HD - 1, s.extent)) unit_store<T, VEC>((T*)s.out + at, u, rd, tab.layout, x);
    }
  }
}

template <typename T, bool CACHE>
static cudaError_t norm_launch(mtp_ctx* ctx, cudaStream_t s, NormArgs a, const mtp_rope_table& tab) {
  const int hd = ctx->cfg.head_dim, tok = kNormThreads / (hd / 16);
  constexpr int N = 16 / sizeof(T);
  uintptr_t bits = (uintptr_t)a.q.x | (uintptr_t)a.q.out | (uintptr_t)a.k.x | (uintptr_t)a.k.out | (uintptr_t)a.v;
  long long strides = a.q.stride | a.q.out_stride | a.k.stride | a.k.out_stride | a.v_stride;
  const bool vec = !(bits & 15) && strides % N == 0 && a.rd % 16 == 0;
  const int gx = (a.T + tok - 1) / tok;
  // a thread computes its cosines once for its heads; few tokens split the
  // heads over more thread blocks until there are about 8 per SM
  const int heads = (a.q.x ? a.q.heads : 0) + (a.k.x ? a.k.heads * (CACHE ? 2 : 1) : 0);
  int groups = (8 * ctx->num_sms + gx - 1) / gx;
  int per = (heads + groups - 1) / groups;
  per = per < 1 ? 1 : per;
  a.q.per = per;
  a.k.per = per;
  a.v_per = per;
  a.k_groups = a.k.x ? (a.k.heads + per - 1) / per : 0;
  a.v_groups = CACHE ? a.k_groups : 0;
  const int q_groups = a.q.x ? (a.q.heads + a.q.per - 1) / a.q.per : 0;
  const dim3 grid(gx, a.k_groups + a.v_groups + q_groups), block(kNormThreads);
  ctx->launches++;
  if (hd == 128)
    return vec ? launch_pdl(qk_norm_rope_kernel<T, 128, true, CACHE>, grid, block, 0, s, a, tab)
               : launch_pdl(qk_norm_rope_kernel<T, 128, false, CACHE>, grid, block, 0, s, a, tab);
  return vec ? launch_pdl(qk_norm_rope_kernel<T, 64, true, CACHE>, grid, block, 0, s, a, tab)
             : launch_pdl(qk_norm_rope_kernel<T, 64, false, CACHE>, grid, block, 0, s, a, tab);
}

// A side's checks: rows of `heads` heads, in place only with one stride.
static bool side_ok(const NormSide& s, int hd) {
  const int64_t row = (int64_t)s.heads * hd;
  return s.out && s.stride >= row && s.out_stride >= row && (s.x != s.out || s.stride == s.out_stride);
}

}  // namespace mtp

using namespace mtp;

extern "C" {

mtp_status mtp_qk_norm_rope(mtp_ctx* ctx, void* stream, int T, const void* q, int64_t q_stride, const void* q_weight,
                            void* q_out, int64_t q_out_stride, const void* k, int64_t k_stride, const void* k_weight,
                            void* k_out, int64_t k_out_stride, float eps, const int32_t* positions,
                            const mtp_rope_table* rope) {
  if (!ctx || T < 0 || T > (1 << 30) || (!q && !k)) return MTP_ERR_INVALID;
  const mtp_config& c = ctx->cfg;
  if (rope && (!rope_table_ok(rope, c.head_dim) || !positions)) return MTP_ERR_INVALID;
  if (!rope && (!q || !q_weight) && (!k || !k_weight)) return MTP_ERR_INVALID;   // nothing to do
  if ((q_weight || k_weight) && (!(eps > 0.0f) || !isfinite(eps))) return MTP_ERR_INVALID;
  NormArgs a{};
  a.q.heads = c.n_q_heads;
  a.k.heads = c.n_kv_heads;
  if (q) {
    a.q = {q, q_weight, q_out, q_stride, q_out_stride, (int64_t)(T - 1) * q_out_stride + c.n_q_heads * c.head_dim, c.n_q_heads, 0};
    if (!side_ok(a.q, c.head_dim)) return MTP_ERR_INVALID;
  }
  if (k) {
    a.k = {k, k_weight, k_out, k_stride, k_out_stride, (int64_t)(T - 1) * k_out_stride + c.n_kv_heads * c.head_dim, c.n_kv_heads, 0};
    if (!side_ok(a.k, c.head_dim)) return MTP_ERR_INVALID;
  }
  if (T == 0) return MTP_OK;
  DeviceGuard dev(ctx->device);
  if (!dev.ok) return MTP_ERR_CUDA;
  a.positions = positions;
  a.err = ctx->err;
  a.eps = eps;
  a.T = T;
  mtp_rope_table tab = {};
  if (rope) tab = *rope;
  a.rd = tab.rotary_dim;
  return launch_status(c.dtype == MTP_DTYPE_BF16 ? norm_launch<uint16_t, false>(ctx, (cudaStream_t)stream, a, tab)
                                                 : norm_launch<float, false>(ctx, (cudaStream_t)stream, a, tab));
}

mtp_status mtp_kv_append(mtp_ctx* ctx, void* stream, int B, int T, const int32_t* row_offsets, const void* k,
                         int64_t k_stride, const void* k_weight, const void* v, int64_t v_stride, const void* q,
                         int64_t q_stride, const void* q_weight, void* q_out, int64_t q_out_stride, float eps,
                         const int32_t* positions, const mtp_rope_table* rope, const mtp_kv* kv, int32_t* arrive) {
  if (!ctx || B < 1 || B > ctx->cfg.max_batch || T < 0 || T > (1 << 30) || !row_offsets || !k || !v || !arrive ||
      !kv16_ok(kv))
    return MTP_ERR_INVALID;
  const mtp_config& c = ctx->cfg;
  const int64_t kw = (int64_t)c.n_kv_heads * c.head_dim;
  if (k_stride < kw || v_stride < kw) return MTP_ERR_INVALID;
  if (rope && (!rope_table_ok(rope, c.head_dim) || !positions)) return MTP_ERR_INVALID;
  if ((q_weight || k_weight) && (!(eps > 0.0f) || !isfinite(eps))) return MTP_ERR_INVALID;
  NormArgs a{};
  a.q.heads = c.n_q_heads;
  if (q) {
    if (!rope && !q_weight) return MTP_ERR_INVALID;
    a.q = {q, q_weight, q_out, q_stride, q_out_stride, (int64_t)(T - 1) * q_out_stride + c.n_q_heads * c.head_dim, c.n_q_heads, 0};
    if (!side_ok(a.q, c.head_dim)) return MTP_ERR_INVALID;
  }
  if (T == 0) return MTP_OK;
  DeviceGuard dev(ctx->device);
  if (!dev.ok) return MTP_ERR_CUDA;
  a.k = {k, k_weight, nullptr, k_stride, 0, 0, c.n_kv_heads, 0};
  a.v = v;
  a.v_stride = v_stride;
  a.positions = positions;
  a.row_offsets = row_offsets;
  a.kv = *kv;
  a.arrive = arrive;
  a.err = ctx->err;
  a.eps = eps;
  a.B = B;
  a.T = T;
  mtp_rope_table tab = {};
  if (rope) tab = *rope;
  a.rd = tab.rotary_dim;
  return launch_status(c.dtype == MTP_DTYPE_BF16 ? norm_launch<uint16_t, true>(ctx, (cudaStream_t)stream, a, tab)
                                                 : norm_launch<float, true>(ctx, (cudaStream_t)stream, a, tab));
}

}  // extern "C"
