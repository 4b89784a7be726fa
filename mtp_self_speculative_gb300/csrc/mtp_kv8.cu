// The paged 8-bit KV cache: append with rotary and quantization, read-back,
// commit / rollback / truncate and the commit of a packed tree's path.
//
// A block of 16 tokens and one kv head share a scale s, a power of two with
// max|x| <= 448 s; an entry's value is code * s.  With a power of two the
// rescaling that a growing block needs is exact (only values that fall under
// the format's smallest normal number are rounded again), and every value is
// a bf16 number (the smallest codes of scales 2^-126 and 2^-125 lie below
// bf16's smallest).
#include "mtp_kv8.cuh"

namespace mtp {

constexpr int kAppendThreads = 128;

// ------------------------------------------------------------------ append
struct Append8Args {
  const void* k;
  const void* v;
  const void* q;
  void* q_out;
  long long k_stride, v_stride, q_stride, q_out_stride, q_extent;
  const int32_t* row_offsets;
  const int32_t* positions;
  mtp_kv8 kv;
  int* err;
  int B, T, n_kv, g_shift;
  int rope;    // rotate k (and q)
  int vec;     // k and v: rows on 16 bytes, rotary_dim a multiple of 8
  int q_vec;   // q and q_out: rows on 16 bytes, rotary_dim a multiple of 16
};

// A unit is one cache block that takes new rows.  Request b's units start at
// floor(off_b / 16) + 2 b, which leaves it floor(n_b / 16) + 2 at least: as
// many as n_b rows can touch.
__device__ __forceinline__ int append_unit(int o, int b) { return (o >> 4) + 2 * b; }

template <typename T> __device__ __forceinline__ float get1(const T* p);
template <> __device__ __forceinline__ float get1<float>(const float* p) { return *p; }
template <> __device__ __forceinline__ float get1<uint16_t>(const uint16_t* p) {
  return __uint_as_float((uint32_t)*p << 16);
}

// N elements (4, or 8 on 16 bytes) as floats, and back.
template <typename T, int N>
__device__ __forceinline__ void load_n(const T* p, float* x) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 y = *reinterpret_cast<const float4*>(p + i);
      x[i] = y.x; x[i + 1] = y.y; x[i + 2] = y.z; x[i + 3] = y.w;
    }
  } else if constexpr (N == 4) {
    const uint2 y = *reinterpret_cast<const uint2*>(p);
    x[0] = bf16_lo(y.x); x[1] = bf16_hi(y.x); x[2] = bf16_lo(y.y); x[3] = bf16_hi(y.y);
  } else {
    const uint4 y = *reinterpret_cast<const uint4*>(p);
    x[0] = bf16_lo(y.x); x[1] = bf16_hi(y.x); x[2] = bf16_lo(y.y); x[3] = bf16_hi(y.y);
    x[4] = bf16_lo(y.z); x[5] = bf16_hi(y.z); x[6] = bf16_lo(y.w); x[7] = bf16_hi(y.w);
  }
}
template <typename T>
__device__ __forceinline__ void store_8(T* p, const float* x) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

__device__ __forceinline__ uint32_t e4m3_pack4(const float* x, float inv) {
  return e4m3_pack2(e4m3_in(x[0], inv), e4m3_in(x[1], inv)) |
         (e4m3_pack2(e4m3_in(x[2], inv), e4m3_in(x[3], inv)) << 16);
}

// The queries of 16 rows and one kv head's group: they need the rows' offsets
// (which rows there are) and positions, but nothing of the cache.
template <typename T, int HD>
__device__ __forceinline__ void append_queries(const Append8Args& a, const mtp_rope_table& tab, int u, int g) {
  const int G = 1 << a.g_shift, tid = threadIdx.x;
  int bad = 0;
  for (int b = tid; b < a.B; b += kAppendThreads) {
    const int o0 = a.row_offsets[b], o1 = a.row_offsets[b + 1];
    bad |= o0 < 0 || o1 < o0 || o1 > a.T;
  }
  const int r0 = max(16 * u, a.row_offsets[0]), rows = min(16 * u + 16, a.row_offsets[a.B]) - r0;
  if (__syncthreads_or(bad) || rows <= 0) return;   // (the cache's thread blocks report it)
  const int rd = tab.rotary_dim;
  const T* q0 = (const T*)a.q + (long long)r0 * a.q_stride + (long long)g * G * HD;
  T* w0 = (T*)a.q_out + (long long)r0 * a.q_out_stride + (long long)g * G * HD;
  auto q_at = [&](int r, int h) -> long long { return (long long)(r0 + r) * a.q_out_stride + ((long long)g * G + h) * HD; };
  (void)q_at;   // bounds-checked builds only
  if (a.q_vec) {
    // a thread owns 8 pairs (or 8 elements past the rotated part) of a
    // row and walks over heads; few rows share the heads among threads
    const int turning = rd / 16, units = turning + (a.q == a.q_out ? 0 : (HD - rd) / 8);
    int hs = 1;
    while (hs < G && 2 * hs * rows * units <= kAppendThreads) hs *= 2;
    for (int i = tid; i < rows * units * hs; i += kAppendThreads) {
      const int h0 = i % hs, x = i / hs, r = x / units, un = x - r * units;
      const T* qr = q0 + (long long)r * a.q_stride;
      T* wr = w0 + (long long)r * a.q_out_stride;
      if (un >= turning) {
        const int e = rd + 8 * (un - turning);
        for (int h = h0; h < G; h += hs) {
          if (!MTP_IN_BOUNDS(a.err, q_at(r, h) + e + 7, a.q_extent)) continue;
          float y[8];
          load_n<T, 8>(qr + h * HD + e, y);
          store_8(wr + h * HD + e, y);
        }
        continue;
      }
      const bool hf = tab.layout == MTP_ROPE_HALF;
      const int xa = hf ? 8 * un : 16 * un, xb = hf ? 8 * un + rd / 2 : 16 * un + 8;
      const int pos = a.positions[r0 + r];
      float2 cs[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) cs[e] = rope_cos_sin(pos, tab.turns[8 * un + e], tab.magnitude);
      for (int h = h0; h < G; h += hs) {
        float p[16], y[16];
        load_n<T, 8>(qr + h * HD + xa, p);
        load_n<T, 8>(qr + h * HD + xb, p + 8);
        if (hf) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            y[e] = rope_first(p[e], p[8 + e], cs[e]);
            y[8 + e] = rope_second(p[e], p[8 + e], cs[e]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            y[2 * e] = rope_first(p[2 * e], p[2 * e + 1], cs[e]);
            y[2 * e + 1] = rope_second(p[2 * e], p[2 * e + 1], cs[e]);
          }
        }
        if (!MTP_IN_BOUNDS(a.err, q_at(r, h) + xb + 7, a.q_extent)) continue;
        store_8(wr + h * HD + xa, y);
        store_8(wr + h * HD + xb, y + 8);
      }
    }
  } else {
    for (int i = tid; i < rows * (HD / 2); i += kAppendThreads) {
      const int r = i / (HD / 2), pe = i - r * (HD / 2);
      const T* qr = q0 + (long long)r * a.q_stride;
      T* wr = w0 + (long long)r * a.q_out_stride;
      const bool turn = pe < rd / 2, hf = turn && tab.layout == MTP_ROPE_HALF;
      const int ia = hf ? pe : 2 * pe, ib = hf ? pe + rd / 2 : 2 * pe + 1;
      float2 c = make_float2(0.0f, 0.0f);
      if (turn) c = rope_cos_sin(a.positions[r0 + r], tab.turns[pe], tab.magnitude);
      for (int h = 0; h < G; ++h) {
        if (!MTP_IN_BOUNDS(a.err, q_at(r, h) + ib, a.q_extent)) continue;
        if (turn) {
          const float x = get1<T>(qr + h * HD + ia), y = get1<T>(qr + h * HD + ib);
          Elem<T>::store1(wr + h * HD + ia, rope_first(x, y, c));
          Elem<T>::store1(wr + h * HD + ib, rope_second(x, y, c));
        } else if (a.q != a.q_out) {
          wr[h * HD + ia] = qr[h * HD + ia];
          wr[h * HD + ib] = qr[h * HD + ib];
        }
      }
    }
  }
}

// Thread block (unit, kv head, 0): the unit's new rows of k and v; (16 rows, kv
// head, 1): the head's queries, in blocks of their own so that neither waits
// for the other (one after the other: 11.6 and 29.9 us for 32 x 6 rows and four
// prompts).  16 (HD = 128) or 8 threads share a row, each with 8
// elements: two fours half the rotated part apart (half layout, aligned) or
// eight next to one another, so that a thread has both members of its pairs,
// computes their cosine once, and nothing goes through shared memory but the
// two maxima.  What bounds a decoding step is the chain of dependent loads:
// lengths, then rows, positions and block id together, then the old scale.
// 32 requests x 6 rows with 32 query heads, and reading 461 entries back: 10.2 us
// for both; four prompts of 2425 rows together, 26.4 us, 0.39 of the copy rate:
// nothing is saturated (ALU pipe 32 %, DRAM 17 %), and each thread block works
// out its rows' cosines anew, 16 times for a token with eight kv heads and
// queries, where the rotary kernel alone does it once for many heads.
template <typename T, int HD>
__global__ void __launch_bounds__(kAppendThreads) kv8_append_kernel(const Append8Args a,
                                                                    const __grid_constant__ mtp_rope_table tab) {
  constexpr int W = kAppendThreads / 32;
  constexpr int LPR = HD / 8;                          // threads of a row
  constexpr int PASS = kBlk * LPR / kAppendThreads;    // rows per thread
  constexpr int STEP = kAppendThreads / LPR;
  __shared__ float red[2][W];
  __shared__ int sh[5];
  pdl_wait();
  pdl_trigger();
  const int u = blockIdx.x, g = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (blockIdx.z == 1) {
    append_queries<T, HD>(a, tab, u, g);
    return;
  }
  // ---- the unit's request; every thread checks some of the offsets
  if (tid == 0) sh[0] = -1;
  __syncthreads();
  int bad = 0;
  for (int b = tid; b < a.B; b += kAppendThreads) {
    const int o0 = a.row_offsets[b], o1 = a.row_offsets[b + 1], sl = a.kv.seq_len[b], pe = a.kv.pending[b];
    if (o0 < 0 || o1 < o0 || o1 > a.T) {
      bad = 1;
    } else if (o1 > o0 && append_unit(o0, b) <= u && u < append_unit(o1, b + 1)) {
      sh[0] = b; sh[1] = o0; sh[2] = o1; sh[3] = sl; sh[4] = pe;
    }
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) set_error(a.err, MTP_ERR_DEVICE_ARGS);
    return;
  }
  const int b = sh[0];
  if (b < 0) return;
  const int o0 = sh[1], n_new = sh[2] - o0, P = sh[4];
  const int all = (append_unit(sh[2], b + 1) - append_unit(o0, b)) * a.n_kv;   // the request's thread blocks
  if (sh[3] < 0 || P < 0 || sh[3] > INT32_MAX - P) {
    if (tid == 0) set_error(a.err, MTP_ERR_DEVICE_ARGS);
    return;
  }
  const int start = sh[3] + P;
  if ((long long)start + n_new > (long long)a.kv.max_blocks * kBlk) {
    if (tid == 0) set_error(a.err, MTP_ERR_CAPACITY);
    return;
  }
  const int first = start >> 4, last = (start + n_new - 1) >> 4, bi = first + (u - append_unit(o0, b));
  if (bi > last) {   // no rows left for it; it has read the old length, so it counts
    if (tid == 0 && arrive_last(a.kv.arrive + b, all)) a.kv.pending[b] = P + n_new;
    return;
  }
  const int s0 = max(start - bi * kBlk, 0);                  // first new slot within the block
  const int s1 = min(start + n_new - bi * kBlk, kBlk);       // one past the last
  const int r0 = o0 + bi * kBlk + s0 - start;                // input row of slot s0
  const int blk = a.kv.block_table[(long long)b * a.kv.max_blocks + bi];
  const int rd = a.rope ? tab.rotary_dim : 0;
  // ---- rows: slot s0 + tid / LPR, + STEP, ...
  const int e8 = tid % LPR;
  const bool split = a.vec && tab.layout == MTP_ROPE_HALF && e8 < rd / 8;   // elements 4 e8 .., rd / 2 + 4 e8 ..
  const int ea = split ? 4 * e8 : 8 * e8, eb = split ? rd / 2 + 4 * e8 : 8 * e8 + 4;
  float kx[PASS][8], vx[PASS][8];
  float amax[2] = {0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < PASS; ++j) {
    const int i = tid / LPR + j * STEP;
    if (i >= s1 - s0) continue;
    const T* kr = (const T*)a.k + (long long)(r0 + i) * a.k_stride + g * HD;
    const T* vr = (const T*)a.v + (long long)(r0 + i) * a.v_stride + g * HD;
    if (a.vec) {
      load_n<T, 4>(kr + ea, kx[j]);
      load_n<T, 4>(kr + eb, kx[j] + 4);
      load_n<T, 8>(vr + 8 * e8, vx[j]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        kx[j][e] = get1<T>(kr + 8 * e8 + e);
        vx[j][e] = get1<T>(vr + 8 * e8 + e);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < PASS; ++j) {
    const int i = tid / LPR + j * STEP;
    if (i >= s1 - s0) continue;
    if (rd) {
      const int pos = a.positions[r0 + i];
      if (split) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 c = rope_cos_sin(pos, tab.turns[ea + e], tab.magnitude);
          const float x = kx[j][e], y = kx[j][4 + e];
          kx[j][e] = rope_first(x, y, c);
          kx[j][4 + e] = rope_second(x, y, c);
        }
      } else if (tab.layout == MTP_ROPE_INTERLEAVED) {   // a pair lies within a thread's eight
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          if (8 * e8 + e >= rd) continue;
          const float2 c = rope_cos_sin(pos, tab.turns[4 * e8 + e / 2], tab.magnitude);
          const float x = kx[j][e], y = kx[j][e + 1];
          kx[j][e] = rope_first(x, y, c);
          kx[j][e + 1] = rope_second(x, y, c);
        }
      } else if (!a.vec) {                               // halves that do not fall on fours: partners one by one
        const T* kr = (const T*)a.k + (long long)(r0 + i) * a.k_stride + g * HD;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int d = 8 * e8 + e;
          if (d >= rd) continue;
          const bool low = d < rd / 2;
          const float2 c = rope_cos_sin(pos, tab.turns[low ? d : d - rd / 2], tab.magnitude);
          const float y = get1<T>(kr + (low ? d + rd / 2 : d - rd / 2));
          kx[j][e] = low ? rope_first(kx[j][e], y, c) : rope_second(y, kx[j][e], c);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (finite_f(kx[j][e])) amax[0] = fmaxf(amax[0], fabsf(kx[j][e]));
      if (finite_f(vx[j][e])) amax[1] = fmaxf(amax[1], fabsf(vx[j][e]));
    }
  }
  const bool good = blk >= 0 && blk < a.kv.num_blocks;
  const long long t = (long long)(good ? blk : 0) * a.n_kv + g;
  float was[2] = {0.0f, 0.0f};
  if (s0 > 0 && good) {
    was[0] = a.kv.k_scale[t];
    was[1] = a.kv.v_scale[t];
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const float m = warp_max(amax[w]);
    if (lane == 0) red[w][warp] = m;
  }
  __syncthreads();   // (also: all have read the old scales)
  if (!good) {
    if (tid == 0) set_error(a.err, MTP_ERR_CAPACITY);
  } else {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      float m = red[w][0];
#pragma unroll
      for (int i = 1; i < W; ++i) m = fmaxf(m, red[w][i]);
      uint8_t* tile = (uint8_t*)(w ? a.kv.v_pool : a.kv.k_pool) + t * (kBlk * HD);
      const float now = fmaxf(was[w], e4m3_scale(m));
      const float inv = now > 0.0f ? 1.0f / now : 0.0f;
      // entries of a block whose scale grows
      if (was[w] > 0.0f && now > was[w]) {
        const float f = was[w] * inv;
        for (int i = tid; i < s0 * (HD / 4); i += kAppendThreads) {
          uint32_t* p = (uint32_t*)tile + i;
          const uint32_t c = *p;
          const float2 x = e4m3_to_float2(c & 0xFFFFu), y = e4m3_to_float2(c >> 16);
          *p = e4m3_pack2(x.x * f, x.y * f) | (e4m3_pack2(y.x * f, y.y * f) << 16);
        }
      }
#pragma unroll
      for (int j = 0; j < PASS; ++j) {
        const int i = tid / LPR + j * STEP;
        if (i >= s1 - s0) continue;
        const float* x = w ? vx[j] : kx[j];
        uint8_t* row = tile + (s0 + i) * HD;
        if (!MTP_IN_BOUNDS(a.err, t * (kBlk * HD) + (s0 + i) * HD + HD - 1, (long long)a.kv.num_blocks * a.n_kv * kBlk * HD)) continue;
        *(uint32_t*)(row + (w ? 8 * e8 : ea)) = e4m3_pack4(x, inv);
        *(uint32_t*)(row + (w ? 8 * e8 + 4 : eb)) = e4m3_pack4(x + 4, inv);
      }
      if (tid == 0) (w ? a.kv.v_scale : a.kv.k_scale)[t] = now;
    }
  }
  // the last of the request's thread blocks publishes the new length: all
  // have read the old one by then, those that had no rows to write too (one
  // that starts late would take the new length for the old)
  if (tid == 0 && arrive_last(a.kv.arrive + b, all)) a.kv.pending[b] = P + n_new;
}

// -------------------------------------------------------------------- read
struct Read8Args {
  mtp_kv8 kv;
  const int32_t* start;
  const int32_t* row_offsets;
  uint16_t* k_out;
  uint16_t* v_out;
  int* err;
  int B, T, n_kv;
};

// Thread block: one row, all kv heads; a thread turns 8 codes into 16 bytes.
// Bound by its three dependent loads (offsets, block id, codes), which every
// row's thread block makes for itself: 2425 rows of 8 heads 8 us, of which the
// bytes (15 MB) need 2.2.
template <int HD>
__global__ void __launch_bounds__(128) kv8_read_kernel(const Read8Args a) {
  const int r = blockIdx.x;
  __shared__ int sh[5];
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) sh[0] = -1;
  __syncthreads();
  int bad = 0;
  for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
    const int o0 = a.row_offsets[b], o1 = a.row_offsets[b + 1], s = a.start[b];
    const long long L = (long long)a.kv.seq_len[b] + a.kv.pending[b];
    if (o0 < 0 || o1 < o0 || o1 > a.T) {
      bad = 1;
    } else if (o0 <= r && r < o1) {
      sh[0] = b;
      sh[1] = s < 0 || (long long)s + (o1 - o0) > L ? -1 : s + (r - o0);
    }
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) set_error(a.err, MTP_ERR_DEVICE_ARGS);
    return;
  }
  const int b = sh[0], slot = sh[1];
  if (b < 0) return;
  if (slot < 0) {
    if (threadIdx.x == 0) set_error(a.err, MTP_ERR_DEVICE_ARGS);
    return;
  }
  const int bi = slot >> 4, off = slot & 15;
  const int blk = bi < a.kv.max_blocks ? a.kv.block_table[(long long)b * a.kv.max_blocks + bi] : -1;
  if (blk < 0 || blk >= a.kv.num_blocks) {
    if (threadIdx.x == 0) set_error(a.err, MTP_ERR_CAPACITY);
    return;
  }
  constexpr int VEC = HD / 8;
  const int per = a.n_kv * VEC;
  for (int i = threadIdx.x; i < 2 * per; i += blockDim.x) {
    const int w = i >= per;
    const int j = i - w * per, g = j / VEC, e = j - g * VEC;
    const long long tile = (long long)blk * a.n_kv + g;
    const uint2 c = *((const uint2*)(w ? a.kv.v_pool : a.kv.k_pool) + (tile * kBlk + off) * VEC + e);
    const float s = (w ? a.kv.v_scale : a.kv.k_scale)[tile];
    uint32_t o[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float2 y = e4m3_to_float2((x < 2 ? c.x : c.y) >> (16 * (x & 1)) & 0xFFFFu);
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[x]) : "f"(y.y * s), "f"(y.x * s));
    }
    const long long at = ((long long)r * a.n_kv + g) * HD + 8 * e;
    if (!MTP_IN_BOUNDS(a.err, at + 7, (long long)a.T * a.n_kv * HD)) continue;
    *reinterpret_cast<uint4*>((w ? a.v_out : a.k_out) + at) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// ------------------------------------------------------------------- edits
struct Edit8Args {
  mtp_kv8 kv;
  const int32_t* arg;    // n_keep, accepted or new_len
  const int32_t* keep;   // a path's places among the pending entries, or null
  int* err;
  int keep_stride, mode, extra, n_kv, hd;
};

constexpr int kPathMax = 256;  // pending entries of a path commit
constexpr int kEditThreads = 128;

// Thread block (kv head, request).  Zeroes the dropped slots of its head; a
// path commit first takes the kept entries into shared memory as codes with
// their blocks' scales.  For the drafts of a step, a few KB per request, launch
// and two dependent loads bound it.  A prompt or a long context that is dropped
// is cleared by the same one thread block a head, a table lookup per 16 bytes:
// the layout is not made for that, and no time is given for it.
__global__ void __launch_bounds__(kEditThreads) kv8_edit_kernel(const Edit8Args a) {
  extern __shared__ __align__(16) uint8_t kept[];   // path: [n][hd] codes
  __shared__ float kept_scale[kPathMax];
  __shared__ float red[kEditThreads / 32];
  __shared__ int sh[4];
  pdl_wait();
  pdl_trigger();
  const int g = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int32_t* keep = a.keep ? a.keep + (long long)b * a.keep_stride : nullptr;
  if (tid == 0) {
    const int L = a.kv.seq_len[b], P = a.kv.pending[b];
    bool good = L >= 0 && P >= 0 && L <= INT32_MAX - P;
    int nl = L;
    if (good) {
      if (a.mode == KV_TRUNCATE) {
        const int n = a.arg[b];
        good = n >= 0 && n <= L + P;
        nl = n;
      } else {
        int n = 0;
        if (a.mode == KV_COMMIT) n = a.arg[b];
        if (a.mode == KV_COMMIT_ACCEPTED) {
          const int acc = a.arg[b];
          good = acc >= 0;
          n = acc >= P ? P : min(acc + a.extra, P);
        }
        good = good && n >= 0 && n <= P;
        if (keep && good) {
          good = P <= kPathMax && n <= a.keep_stride;
          for (int j = 0; good && j < n; ++j)
            good = keep[j] >= 0 && keep[j] < P && (j == 0 || keep[j] > keep[j - 1]);
        }
        nl = good ? L + n : L;
      }
    }
    if (good && (long long)L + P > (long long)a.kv.max_blocks * kBlk) {
      set_error(a.err, MTP_ERR_CAPACITY);
      good = false;
    } else if (!good) {
      set_error(a.err, MTP_ERR_DEVICE_ARGS);
    }
    sh[0] = good;
    sh[1] = nl;
    sh[2] = L;
    sh[3] = L + P;
  }
  __syncthreads();
  if (!sh[0]) return;
  const int nl = sh[1], L = sh[2], end = sh[3];
  const int32_t* row = a.kv.block_table + (long long)b * a.kv.max_blocks;
  if (keep) {
    // a kept entry that lies in a block outside the pool, or would move to one,
    // would be lost: the request stays as it is
    int lost = 0;
    for (int j = tid; j < nl - L; j += kEditThreads) {
      const int from = row[(L + keep[j]) >> 4], to = row[(L + j) >> 4];
      lost |= from < 0 || from >= a.kv.num_blocks || to < 0 || to >= a.kv.num_blocks;
    }
    if (__syncthreads_or(lost)) {
      if (tid == 0) set_error(a.err, MTP_ERR_CAPACITY);
      return;
    }
  }
  // the last head's block publishes the lengths; all have read them
  if (tid == 0 && arrive_last(a.kv.arrive + b, a.n_kv)) {
    a.kv.seq_len[b] = nl;
    a.kv.pending[b] = 0;
  }
  const int vec = a.hd / 16;
  for (int w = 0; w < 2; ++w) {
    uint4* pool = (uint4*)(w ? a.kv.v_pool : a.kv.k_pool);
    float* scale = w ? a.kv.v_scale : a.kv.k_scale;
    auto tile_of = [&](int slot) -> long long {
      const int blk = row[slot >> 4];
      return blk >= 0 && blk < a.kv.num_blocks ? (long long)blk * a.n_kv + g : -1;
    };
    if (keep) {
      const int n = nl - L;
      for (int i = tid; i < n * vec; i += kEditThreads) {
        const int j = i / vec, e = i - j * vec, slot = L + keep[j];
        const long long t = tile_of(slot);
        ((uint4*)kept)[i] = pool[(t * kBlk + (slot & 15)) * vec + e];
        if (e == 0) kept_scale[j] = scale[t];
      }
      __syncthreads();
      for (int bi = L >> 4; bi * kBlk < nl; ++bi) {
        const int s0 = max(L - bi * kBlk, 0), s1 = min(nl - bi * kBlk, kBlk);
        const int j0 = bi * kBlk + s0 - L;
        float m = 0.0f;
        for (int i = tid; i < (s1 - s0) * (a.hd / 2); i += kEditThreads) {
          const int j = j0 + i / (a.hd / 2);
          const float2 x = e4m3_to_float2(((const uint16_t*)kept)[(long long)j0 * (a.hd / 2) + i]);
          if (finite_f(x.x)) m = fmaxf(m, fabsf(x.x * kept_scale[j]));
          if (finite_f(x.y)) m = fmaxf(m, fabsf(x.y * kept_scale[j]));
        }
        m = warp_max(m);
        if ((tid & 31) == 0) red[tid >> 5] = m;
        __syncthreads();
        for (int i = 0; i < kEditThreads / 32; ++i) m = fmaxf(m, red[i]);
        const long long t = tile_of(bi * kBlk);
        uint16_t* tile = (uint16_t*)(pool + t * kBlk * vec);
        const float was = s0 > 0 ? scale[t] : 0.0f;
        const float now = fmaxf(was, e4m3_scale(m));
        const float inv = now > 0.0f ? 1.0f / now : 0.0f;
        if (was > 0.0f && now > was) {
          for (int i = tid; i < s0 * (a.hd / 2); i += kEditThreads) {
            const float2 x = e4m3_to_float2(tile[i]);
            tile[i] = (uint16_t)e4m3_pack2(x.x * (was * inv), x.y * (was * inv));
          }
        }
        for (int i = tid; i < (s1 - s0) * (a.hd / 2); i += kEditThreads) {
          const int j = j0 + i / (a.hd / 2);
          const float2 x = e4m3_to_float2(((const uint16_t*)kept)[(long long)j0 * (a.hd / 2) + i]);
          tile[s0 * (a.hd / 2) + i] =
              (uint16_t)e4m3_pack2(x.x * kept_scale[j] * inv, x.y * kept_scale[j] * inv);
        }
        __syncthreads();
        if (tid == 0) scale[t] = now;
        __syncthreads();
      }
    }
    // dropped slots, and the scales of blocks left without an entry
    const int cnt = end - nl;
    for (long long i = tid; i < (long long)cnt * vec; i += kEditThreads) {
      const int slot = nl + (int)(i / vec), e = (int)(i % vec);
      const long long t = tile_of(slot);
      if (t < 0) {
        set_error(a.err, MTP_ERR_CAPACITY);
        continue;
      }
      if (!MTP_IN_BOUNDS(a.err, (t * kBlk + (slot & 15)) * vec + e, (long long)a.kv.num_blocks * a.n_kv * kBlk * vec)) continue;
      pool[(t * kBlk + (slot & 15)) * vec + e] = make_uint4(0, 0, 0, 0);
      if (e == 0 && (slot & 15) == 0) scale[t] = 0.0f;
    }
    __syncthreads();
  }
}

}  // namespace mtp

using namespace mtp;

extern "C" {

mtp_status mtp_kv8_append(mtp_ctx* ctx, void* stream, int B, int T, const int32_t* row_offsets, const void* k,
                          int64_t k_stride, const void* v, int64_t v_stride, const int32_t* positions,
                          const mtp_rope_table* rope, const void* q, int64_t q_stride, void* q_out,
                          int64_t q_out_stride, const mtp_kv8* kv) {
  if (!ctx || B < 1 || B > ctx->cfg.max_batch || T < 0 || !row_offsets || !k || !v || !kv8_ok(kv))
    return MTP_ERR_INVALID;
  const mtp_config& c = ctx->cfg;
  const int64_t kw = (int64_t)c.n_kv_heads * c.head_dim, qw = (int64_t)c.n_q_heads * c.head_dim;
  if (k_stride < kw || v_stride < kw) return MTP_ERR_INVALID;
  if (rope && (!rope_table_ok(rope, c.head_dim) || !positions)) return MTP_ERR_INVALID;
  if (q && (!rope || !q_out || q_stride < qw || q_out_stride < qw || (q == q_out && q_stride != q_out_stride)))
    return MTP_ERR_INVALID;
  if (c.n_kv_heads > 65535 || T > (1 << 30) || B > (1 << 28)) return MTP_ERR_INVALID;
  if (T == 0) return MTP_OK;
  DeviceGuard dev(ctx->device);
  if (!dev.ok) return MTP_ERR_CUDA;
  Append8Args a{};
  a.k = k;
  a.v = v;
  a.q = q;
  a.q_out = q_out;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_stride = q_stride;
  a.q_out_stride = q_out_stride;
  a.q_extent = (int64_t)(T - 1) * q_out_stride + qw;
  a.row_offsets = row_offsets;
  a.positions = positions;
  a.kv = *kv;
  a.err = ctx->err;
  a.B = B;
  a.T = T;
  a.n_kv = c.n_kv_heads;
  for (a.g_shift = 0; (1 << a.g_shift) < c.n_q_heads / c.n_kv_heads; ++a.g_shift) {
  }
  a.rope = rope != nullptr;
  mtp_rope_table tab = {};
  if (rope) tab = *rope;
  const bool bf = c.dtype == MTP_DTYPE_BF16;
  const int per16 = bf ? 8 : 4;   // elements of 16 bytes
  a.vec = !(((uintptr_t)k | (uintptr_t)v) & 15) && k_stride % per16 == 0 && v_stride % per16 == 0 &&
          tab.rotary_dim % 8 == 0;
  a.q_vec = !(((uintptr_t)q | (uintptr_t)q_out) & 15) && q_stride % per16 == 0 && q_out_stride % per16 == 0 &&
            tab.rotary_dim % 16 == 0;
  const dim3 grid(T / 16 + 2 * B, c.n_kv_heads, q ? 2 : 1), block(kAppendThreads);
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e =
      c.head_dim == 128 ? (bf ? launch_pdl(kv8_append_kernel<uint16_t, 128>, grid, block, 0, s, a, tab)
                              : launch_pdl(kv8_append_kernel<float, 128>, grid, block, 0, s, a, tab))
                        : (bf ? launch_pdl(kv8_append_kernel<uint16_t, 64>, grid, block, 0, s, a, tab)
                              : launch_pdl(kv8_append_kernel<float, 64>, grid, block, 0, s, a, tab));
  ctx->launches++;
  return launch_status(e);
}

mtp_status mtp_kv8_read(mtp_ctx* ctx, void* stream, int B, const mtp_kv8* kv, const int32_t* start, int T,
                        const int32_t* row_offsets, void* k_out, void* v_out) {
  if (!ctx || B < 1 || B > ctx->cfg.max_batch || T < 0 || !start || !row_offsets || !k_out || !v_out || !kv8_ok(kv) ||
      (((uintptr_t)k_out | (uintptr_t)v_out) & 15))
    return MTP_ERR_INVALID;
  if (T == 0) return MTP_OK;
  DeviceGuard dev(ctx->device);
  if (!dev.ok) return MTP_ERR_CUDA;
  Read8Args a{*kv, start, row_offsets, (uint16_t*)k_out, (uint16_t*)v_out, ctx->err, B, T, ctx->cfg.n_kv_heads};
  const cudaError_t e = ctx->cfg.head_dim == 128
                            ? launch_pdl(kv8_read_kernel<128>, dim3(T), dim3(128), 0, (cudaStream_t)stream, a)
                            : launch_pdl(kv8_read_kernel<64>, dim3(T), dim3(128), 0, (cudaStream_t)stream, a);
  ctx->launches++;
  return launch_status(e);
}

static mtp_status kv8_edit(mtp_ctx* ctx, void* stream, int B, const mtp_kv8* kv, int mode, const int32_t* arg,
                           int extra, const int32_t* keep, int keep_stride) {
  if (!ctx || B < 1 || B > ctx->cfg.max_batch || B > 65535 || !kv8_ok(kv)) return MTP_ERR_INVALID;
  if (mode != KV_ROLLBACK && !arg) return MTP_ERR_INVALID;
  DeviceGuard dev(ctx->device);
  if (!dev.ok) return MTP_ERR_CUDA;
  Edit8Args a{*kv, arg, keep, ctx->err, keep_stride, mode, extra, ctx->cfg.n_kv_heads, ctx->cfg.head_dim};
  const size_t smem = keep ? (size_t)kPathMax * ctx->cfg.head_dim : 0;  // at most 32 KB
  const cudaError_t e = launch_pdl(kv8_edit_kernel, dim3(ctx->cfg.n_kv_heads, B), dim3(kEditThreads), smem,
                                   (cudaStream_t)stream, a);
  ctx->launches++;
  return launch_status(e);
}

mtp_status mtp_kv8_commit(mtp_ctx* ctx, void* stream, int B, const mtp_kv8* kv, const int32_t* n_keep) {
  return kv8_edit(ctx, stream, B, kv, KV_COMMIT, n_keep, 0, nullptr, 0);
}

mtp_status mtp_kv8_commit_accepted(mtp_ctx* ctx, void* stream, int B, const mtp_kv8* kv, const int32_t* accepted,
                                   int extra) {
  if (extra < 0 || extra > 1) return MTP_ERR_INVALID;
  return kv8_edit(ctx, stream, B, kv, KV_COMMIT_ACCEPTED, accepted, extra, nullptr, 0);
}

mtp_status mtp_kv8_rollback(mtp_ctx* ctx, void* stream, int B, const mtp_kv8* kv) {
  return kv8_edit(ctx, stream, B, kv, KV_ROLLBACK, nullptr, 0, nullptr, 0);
}

mtp_status mtp_kv8_truncate(mtp_ctx* ctx, void* stream, int B, const mtp_kv8* kv, const int32_t* new_len) {
  return kv8_edit(ctx, stream, B, kv, KV_TRUNCATE, new_len, 0, nullptr, 0);
}

mtp_status mtp_kv8_commit_path(mtp_ctx* ctx, void* stream, int B, const mtp_kv8* kv, const int32_t* keep,
                               int keep_stride, const int32_t* n_keep) {
  if (!keep || keep_stride < 1) return MTP_ERR_INVALID;
  return kv8_edit(ctx, stream, B, kv, KV_COMMIT, n_keep, 0, keep, keep_stride);
}

}  // extern "C"
