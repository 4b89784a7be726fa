// Rotary positions as an operator of its own: half and interleaved pairs,
// part of the head, frequencies scaled for long contexts.
//
//   out = magnitude * (a cos - b sin, b cos + a sin) for each pair (a, b) of
//   a head, angle = position * f_i.
//
// The work is a copy with a few multiplications per element, so memory bounds
// it: each element is read and written once, 16 bytes at a time where rows
// and pairs allow.  A thread owns one unit of a token's head, computes that
// unit's cosines and sines once, and walks over the heads.  8192 tokens x 32
// heads of 128 in bf16: 25.2 us, 5.3 TB/s (one element a thread: 42.1 us).
#include <math.h>
#include <stdlib.h>

#include "mtp_kv8.cuh"

namespace mtp {

struct RopeArgs {
  const void* x;
  void* out;
  const int32_t* positions;
  int* err;
  long long x_stride, out_stride, out_extent;   // elements; the extent for bounds-checked builds
  int T, heads, hd;
  int rot_units, units;   // rotating units of a head, and those with the copied ones
  int heads_per_block;
};

template <typename T> __device__ __forceinline__ float rope_get(const T* p);
template <> __device__ __forceinline__ float rope_get<float>(const float* p) { return *p; }
template <> __device__ __forceinline__ float rope_get<uint16_t>(const uint16_t* p) {
  return __uint_as_float((uint32_t)*p << 16);
}

// A thread's unit of 2 N elements of a head: N = 8 (bf16) or 4 (float32)
// elements at two places (half layout) or the 2 N next to one another, in
// 16-byte vectors, when the rows, the rotated part and the halves start on
// 16 bytes.
template <typename T>
__device__ __forceinline__ void rope_load(const T* p, float* x) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  if constexpr (sizeof(T) == 2) {
    x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x); x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
    x[4] = bf16_lo(u.z); x[5] = bf16_hi(u.z); x[6] = bf16_lo(u.w); x[7] = bf16_hi(u.w);
  } else {
    x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y); x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
  }
}
template <typename T>
__device__ __forceinline__ void rope_store(T* p, const float* x) {
  uint4 u;
  if constexpr (sizeof(T) == 2) {
    u.x = (uint32_t)f32_to_bf16_rne(x[0]) | ((uint32_t)f32_to_bf16_rne(x[1]) << 16);
    u.y = (uint32_t)f32_to_bf16_rne(x[2]) | ((uint32_t)f32_to_bf16_rne(x[3]) << 16);
    u.z = (uint32_t)f32_to_bf16_rne(x[4]) | ((uint32_t)f32_to_bf16_rne(x[5]) << 16);
    u.w = (uint32_t)f32_to_bf16_rne(x[6]) | ((uint32_t)f32_to_bf16_rne(x[7]) << 16);
  } else {
    u = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
  *reinterpret_cast<uint4*>(p) = u;
}

template <typename T, int LAYOUT>
__global__ void __launch_bounds__(128) rope_vec_kernel(const RopeArgs a, const __grid_constant__ mtp_rope_table tab) {
  constexpr int N = 16 / sizeof(T);
  pdl_wait();
  pdl_trigger();
  const long long item = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (item >= (long long)a.T * a.units) return;
  const int t = (int)(item / a.units), u = (int)(item - (long long)t * a.units);
  const int h0 = blockIdx.y * a.heads_per_block, h1 = min(a.heads, h0 + a.heads_per_block);
  const T* x = (const T*)a.x + (long long)t * a.x_stride;
  T* o = (T*)a.out + (long long)t * a.out_stride;
  if (u >= a.rot_units) {  // N elements past the rotated part
    const int e = tab.rotary_dim + (u - a.rot_units) * N;
#pragma unroll 4
    for (int h = h0; h < h1; ++h)
      if (MTP_IN_BOUNDS(a.err, (long long)t * a.out_stride + h * a.hd + e + N - 1, a.out_extent))
        *reinterpret_cast<uint4*>(o + h * a.hd + e) = *reinterpret_cast<const uint4*>(x + h * a.hd + e);
    return;
  }
  const int pos = a.positions[t];
  const int ea = LAYOUT == MTP_ROPE_HALF ? u * N : u * 2 * N;
  const int eb = LAYOUT == MTP_ROPE_HALF ? ea + tab.rotary_dim / 2 : ea + N;
  float2 cs[N];
#pragma unroll
  for (int i = 0; i < N; ++i) cs[i] = rope_cos_sin(pos, tab.turns[u * N + i], tab.magnitude);
#pragma unroll 2
  for (int h = h0; h < h1; ++h) {
    float p[2 * N], r[2 * N];
    rope_load(x + h * a.hd + ea, p);
    rope_load(x + h * a.hd + eb, p + N);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int ia = LAYOUT == MTP_ROPE_HALF ? i : 2 * i, ib = LAYOUT == MTP_ROPE_HALF ? i + N : 2 * i + 1;
      r[ia] = rope_first(p[ia], p[ib], cs[i]);
      r[ib] = rope_second(p[ia], p[ib], cs[i]);
    }
    if (!MTP_IN_BOUNDS(a.err, (long long)t * a.out_stride + h * a.hd + eb + N - 1, a.out_extent)) continue;
    rope_store(o + h * a.hd + ea, r);
    rope_store(o + h * a.hd + eb, r + N);
  }
}

// Any alignment and rotated part: a thread owns one pair, or one element past
// the rotated part, of a token's heads.
template <typename T>
__global__ void __launch_bounds__(128) rope_kernel(const RopeArgs a, const __grid_constant__ mtp_rope_table tab) {
  pdl_wait();
  pdl_trigger();
  const long long item = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (item >= (long long)a.T * a.units) return;
  const int t = (int)(item / a.units), u = (int)(item - (long long)t * a.units);
  const int h0 = blockIdx.y * a.heads_per_block, h1 = min(a.heads, h0 + a.heads_per_block);
  const T* x = (const T*)a.x + (long long)t * a.x_stride;
  T* o = (T*)a.out + (long long)t * a.out_stride;
  if (u >= a.rot_units) {  // an element past the rotated part
    const int e = tab.rotary_dim + (u - a.rot_units);
    for (int h = h0; h < h1; ++h)
      if (MTP_IN_BOUNDS(a.err, (long long)t * a.out_stride + h * a.hd + e, a.out_extent)) o[h * a.hd + e] = x[h * a.hd + e];
    return;
  }
  const float2 cs = rope_cos_sin(a.positions[t], tab.turns[u], tab.magnitude);
  const int ia = tab.layout == MTP_ROPE_HALF ? u : 2 * u;
  const int ib = tab.layout == MTP_ROPE_HALF ? u + tab.rotary_dim / 2 : 2 * u + 1;
  for (int h = h0; h < h1; ++h) {
    const float p = rope_get<T>(x + h * a.hd + ia), q = rope_get<T>(x + h * a.hd + ib);
    if (!MTP_IN_BOUNDS(a.err, (long long)t * a.out_stride + h * a.hd + ib, a.out_extent)) continue;
    Elem<T>::store1(o + h * a.hd + ia, rope_first(p, q, cs));
    Elem<T>::store1(o + h * a.hd + ib, rope_second(p, q, cs));
  }
}

template <typename T>
static cudaError_t rope_launch(mtp_ctx* ctx, cudaStream_t s, RopeArgs a, const mtp_rope_table& tab) {
  constexpr int N = 16 / sizeof(T);
  const bool half = tab.layout == MTP_ROPE_HALF;
  // the half layout wants its second half on 16 bytes too
  const bool vec = !(((uintptr_t)a.x | (uintptr_t)a.out) & 15) && a.x_stride % N == 0 && a.out_stride % N == 0 &&
                   tab.rotary_dim % (2 * N) == 0;
  const int per = vec ? N : 1;
  a.rot_units = tab.rotary_dim / 2 / per;
  a.units = a.rot_units + (a.x == a.out ? 0 : (a.hd - tab.rotary_dim) / per);
  const long long items = (long long)a.T * a.units, gx = (items + 127) / 128;
  if (gx > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  // a thread computes its unit's cosines once for all its heads; few tokens
  // split the heads over more threads until there are about 16 blocks per SM
  const long long want = 16ll * ctx->num_sms;
  int gy = gx >= want ? 1 : (int)((want + gx - 1) / gx);
  gy = gy < a.heads ? gy : a.heads;
  gy = gy < 65535 ? gy : 65535;
  a.heads_per_block = (a.heads + gy - 1) / gy;
  gy = (a.heads + a.heads_per_block - 1) / a.heads_per_block;
  const dim3 grid((unsigned)gx, gy);
  if (!vec) return launch_pdl(rope_kernel<T>, grid, dim3(128), 0, s, a, tab);
  return half ? launch_pdl(rope_vec_kernel<T, MTP_ROPE_HALF>, grid, dim3(128), 0, s, a, tab)
              : launch_pdl(rope_vec_kernel<T, MTP_ROPE_INTERLEAVED>, grid, dim3(128), 0, s, a, tab);
}

}  // namespace mtp

using namespace mtp;

extern "C" {

mtp_status mtp_rope_table_make(const mtp_rope_params* p, mtp_rope_table* out) {
  if (!p || !out) return MTP_ERR_INVALID;
  if (p->layout != MTP_ROPE_HALF && p->layout != MTP_ROPE_INTERLEAVED) return MTP_ERR_INVALID;
  if (p->rotary_dim < 2 || p->rotary_dim > 128 || p->rotary_dim % 2) return MTP_ERR_INVALID;
  if (p->scaling < MTP_ROPE_SCALE_NONE || p->scaling > MTP_ROPE_SCALE_YARN) return MTP_ERR_INVALID;
  if (!(p->theta > 1.0f) || !isfinite(p->theta) || !isfinite(p->magnitude) || p->magnitude < 0.0f)
    return MTP_ERR_INVALID;
  const bool scaled = p->scaling != MTP_ROPE_SCALE_NONE;
  if (scaled && (!(p->factor > 0.0f) || !isfinite(p->factor))) return MTP_ERR_INVALID;
  if (p->scaling >= MTP_ROPE_SCALE_PARTS && p->original_max_pos <= 0) return MTP_ERR_INVALID;
  if (p->scaling == MTP_ROPE_SCALE_PARTS && (!(p->high_freq_factor > p->low_freq_factor) ||
                                             !isfinite(p->high_freq_factor) || !isfinite(p->low_freq_factor)))
    return MTP_ERR_INVALID;
  if (p->scaling == MTP_ROPE_SCALE_YARN && (!(p->beta_fast > p->beta_slow) || !(p->beta_slow > 0.0f) ||
                                            !isfinite(p->beta_fast)))
    return MTP_ERR_INVALID;
  const double pi2 = 6.283185307179586476925;
  const int d = p->rotary_dim;
  const double s = scaled ? (double)p->factor : 1.0;
  double lo = 0.0, hi = 0.0;
  if (p->scaling == MTP_ROPE_SCALE_YARN) {
    const double den = 2.0 * log((double)p->theta);
    lo = floor(d * log(p->original_max_pos / (pi2 * p->beta_fast)) / den);
    hi = ceil(d * log(p->original_max_pos / (pi2 * p->beta_slow)) / den);
    if (lo < 0.0) lo = 0.0;
    if (hi > d - 1) hi = d - 1;
  }
  mtp_rope_table t = {};
  t.layout = p->layout;
  t.rotary_dim = d;
  t.magnitude = p->magnitude > 0.0f ? p->magnitude
                : (p->scaling == MTP_ROPE_SCALE_YARN && s > 1.0) ? (float)(0.1 * log(s) + 1.0)
                                                                  : 1.0f;
  for (int i = 0; i < d / 2; ++i) {
    double f = pow((double)p->theta, -2.0 * i / d);
    if (p->scaling == MTP_ROPE_SCALE_LINEAR) {
      f /= s;
    } else if (p->scaling == MTP_ROPE_SCALE_PARTS) {
      const double r = p->original_max_pos * f / pi2;
      double w = (r - p->low_freq_factor) / ((double)p->high_freq_factor - p->low_freq_factor);
      w = w < 0.0 ? 0.0 : w > 1.0 ? 1.0 : w;
      f = w * f + (1.0 - w) * f / s;
    } else if (p->scaling == MTP_ROPE_SCALE_YARN) {
      double w = (i - lo) / (hi - lo > 0.001 ? hi - lo : 0.001);
      w = w < 0.0 ? 0.0 : w > 1.0 ? 1.0 : w;
      f = (1.0 - w) * f + w * f / s;
    }
    // the fraction of a turn per position, modulo whole turns (a factor below
    // 1 can push it past one)
    double turn = f / pi2;
    turn -= floor(turn);
    t.turns[i] = turn >= 1.0 ? 0ull : (uint64_t)(turn * 18446744073709551616.0);
  }
  *out = t;
  return MTP_OK;
}

mtp_status mtp_set_rope(mtp_ctx* ctx, const mtp_rope_table* rope) {
  if (!ctx || !ctx->has_weights || !rope_table_ok(rope, ctx->cfg.head_dim)) return MTP_ERR_INVALID;
  const int half = ctx->cfg.head_dim / 2;
  if (rope->layout != MTP_ROPE_HALF || rope->rotary_dim != ctx->cfg.head_dim) return MTP_ERR_INVALID;
  DeviceGuard dev(ctx->device);
  if (!dev.ok) return MTP_ERR_CUDA;
  const size_t n = (size_t)ctx->cfg.max_pos * half;
  float2* tab = (float2*)malloc(n * sizeof(float2));
  if (!tab) return MTP_ERR_OOM;
  for (int p = 0; p < ctx->cfg.max_pos; ++p)
    for (int i = 0; i < half; ++i) {
      // the exact phase, as a signed fraction of a turn, to an angle
      const double turn = (double)(int64_t)((uint64_t)p * rope->turns[i]) / 18446744073709551616.0;
      const double ang = turn * 6.283185307179586476925;
      tab[(size_t)p * half + i] = make_float2((float)(cos(ang) * rope->magnitude), (float)(sin(ang) * rope->magnitude));
    }
  // work that reads the old table finishes first; a copy from pageable memory
  // may return before its last bytes have arrived, and a draft on a stream that
  // does not wait for the default one may come next
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(ctx->rope, tab, n * sizeof(float2), cudaMemcpyHostToDevice);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  free(tab);
  return launch_status(e);
}

mtp_status mtp_rope(mtp_ctx* ctx, void* stream, int T, int heads, const void* x, int64_t x_stride,
                    const int32_t* positions, const mtp_rope_table* rope, void* out, int64_t out_stride) {
  if (!ctx || T < 0 || heads < 1 || !x || !out || !positions || !rope_table_ok(rope, ctx->cfg.head_dim))
    return MTP_ERR_INVALID;
  const int hd = ctx->cfg.head_dim;
  const int64_t row = (int64_t)heads * hd;
  if (heads > (1 << 20) || x_stride < row || out_stride < row || (x == out && x_stride != out_stride))
    return MTP_ERR_INVALID;
  if (T == 0) return MTP_OK;
  DeviceGuard dev(ctx->device);
  if (!dev.ok) return MTP_ERR_CUDA;
  RopeArgs a{};
  a.x = x;
  a.out = out;
  a.positions = positions;
  a.err = ctx->err;
  a.out_extent = (int64_t)(T - 1) * out_stride + row;
  a.x_stride = x_stride;
  a.out_stride = out_stride;
  a.T = T;
  a.heads = heads;
  a.hd = hd;
  const cudaError_t e = ctx->cfg.dtype == MTP_DTYPE_BF16 ? rope_launch<uint16_t>(ctx, (cudaStream_t)stream, a, *rope)
                                                         : rope_launch<float>(ctx, (cudaStream_t)stream, a, *rope);
  if (e == cudaErrorInvalidValue) return MTP_ERR_INVALID;
  ctx->launches++;
  return launch_status(e);
}

}  // extern "C"
