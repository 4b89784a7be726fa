// Rotary positions as an operator of its own: half and interleaved pairs,
// part of the head, frequencies scaled for long contexts.
//
//   out = magnitude * (a cos - b sin, b cos + a sin) for each pair (a, b) of
//   a head, angle = position * f_i.
//
// The work is a copy with a few multiplications per element, so memory bounds
// it: each element is read and written once, 16 bytes at a time where rows
// and pairs allow.  A thread owns one unit of a token's head -- the two
// vectors (half layout) or the one vector (interleaved) that hold its pairs --
// computes that unit's cosines and sines once, and walks over the heads.
#include <math.h>

#include "mtp_kv8.cuh"

namespace mtp {

struct RopeArgs {
  const void* x;
  void* out;
  const int32_t* positions;
  long long x_stride, out_stride;
  int T, heads, hd;
  int rot_units, units;   // rotating units of a head, and those plus the copied ones
  int heads_per_block;
};

template <typename T> __device__ __forceinline__ float rope_get(const T* p);
template <> __device__ __forceinline__ float rope_get<float>(const float* p) { return *p; }
template <> __device__ __forceinline__ float rope_get<uint16_t>(const uint16_t* p) {
  return __uint_as_float((uint32_t)*p << 16);
}

template <typename T>
__global__ void __launch_bounds__(256) rope_kernel(const RopeArgs a, const __grid_constant__ mtp_rope_table tab) {
  const long long item = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (item >= (long long)a.T * a.units) return;
  const int t = (int)(item / a.units), u = (int)(item - (long long)t * a.units);
  const int h0 = blockIdx.y * a.heads_per_block, h1 = min(a.heads, h0 + a.heads_per_block);
  const T* x = (const T*)a.x + (long long)t * a.x_stride;
  T* o = (T*)a.out + (long long)t * a.out_stride;
  if (u >= a.rot_units) {  // an element past the rotated part
    const int e = tab.rotary_dim + (u - a.rot_units);
    for (int h = h0; h < h1; ++h) o[h * a.hd + e] = x[h * a.hd + e];
    return;
  }
  const float2 cs = rope_cos_sin(a.positions[t], tab.turns[u], tab.magnitude);
  const int ia = tab.layout == MTP_ROPE_HALF ? u : 2 * u;
  const int ib = tab.layout == MTP_ROPE_HALF ? u + tab.rotary_dim / 2 : 2 * u + 1;
  for (int h = h0; h < h1; ++h) {
    const float p = rope_get<T>(x + h * a.hd + ia), q = rope_get<T>(x + h * a.hd + ib);
    Elem<T>::store1(o + h * a.hd + ia, p * cs.x - q * cs.y);
    Elem<T>::store1(o + h * a.hd + ib, q * cs.x + p * cs.y);
  }
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
  a.x_stride = x_stride;
  a.out_stride = out_stride;
  a.T = T;
  a.heads = heads;
  a.hd = hd;
  a.rot_units = rope->rotary_dim / 2;
  a.units = a.rot_units + (x == out ? 0 : hd - rope->rotary_dim);
  a.heads_per_block = heads;
  const long long items = (long long)T * a.units;
  const long long gx = (items + 255) / 256;
  if (gx > 0x7FFFFFFFll) return MTP_ERR_INVALID;
  if (ctx->cfg.dtype == MTP_DTYPE_BF16)
    rope_kernel<uint16_t><<<dim3((unsigned)gx, 1), 256, 0, (cudaStream_t)stream>>>(a, *rope);
  else
    rope_kernel<float><<<dim3((unsigned)gx, 1), 256, 0, (cudaStream_t)stream>>>(a, *rope);
  ctx->launches++;
  return launch_status(cudaGetLastError());
}

}  // extern "C"
