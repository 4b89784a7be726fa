// The 8-bit KV cache's number format, the rotary phases and the small host
// helpers shared by the kernels of the verifier's side (rotary, append,
// attention over the 8-bit cache, logits).
#pragma once

#include "mtp_common.cuh"

namespace mtp {

constexpr int kBlk = 16;          // tokens per cache block
constexpr float kE4m3Max = 448.0f;

// Makes the context's device current for the length of a call and puts the
// caller's device back.
struct DeviceGuard {
  int prev = -1, want = -1;
  bool ok = false;
  explicit DeviceGuard(int device) : want(device) {
    ok = cudaGetDevice(&prev) == cudaSuccess && (prev == want || cudaSetDevice(want) == cudaSuccess);
  }
  ~DeviceGuard() {
    if (ok && prev != want) cudaSetDevice(prev);
  }
};

inline mtp_status launch_status(cudaError_t e) {
  if (e != cudaSuccess) {
    cudaGetLastError();
    return MTP_ERR_CUDA;
  }
  return MTP_OK;
}

// Two floats to two e4m3 codes (lo in the low byte), round to nearest even,
// clamped to +-448; NaN becomes 0x7f.
__device__ __forceinline__ uint32_t e4m3_pack2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two e4m3 codes to two halves (exact: fp16 has more exponent and mantissa
// bits; NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3_unpack2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}

// Four codes to two pairs of halves.
__device__ __forceinline__ void e4m3_unpack4(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}

__device__ __forceinline__ float2 e4m3_to_float2(uint32_t two) {
  const uint32_t h = e4m3_unpack2(two);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The smallest power of two s (at least 2^-126) with amax <= 448 s; 0 for 0.
// 448 = 1.75 * 2^8: with amax = m * 2^x, 1 <= m < 2, s = 2^(x - 8) or, for
// m > 1.75, 2^(x - 7).  amax is finite and not negative.
__device__ __forceinline__ float e4m3_scale(float amax) {
  if (!(amax > 0.0f)) return 0.0f;
  const uint32_t u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);  // biased exponent of s
  e = max(e, 1);
  return __uint_as_float((uint32_t)e << 23);
}

__device__ __forceinline__ bool finite_f(float x) { return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u; }

// x / s as the stored code's value before rounding: NaN for what is not
// finite (inf must not meet an inverse scale of 0).
__device__ __forceinline__ float e4m3_in(float x, float inv) {
  return finite_f(x) ? x * inv : __uint_as_float(0x7FC00000u);
}

// cos and sin of the angle 2 pi * phase / 2^64.  The phase is reduced to a
// quadrant and a remainder of at most an eighth of a turn in integers, so far
// positions lose nothing; the remainder (|x| <= pi/4) goes through the Taylor
// series, whose next terms are below 2.5e-8.
__device__ __forceinline__ float2 rope_cos_sin(uint64_t phase) {
  const uint64_t u = phase + (1ull << 61);
  const int quad = (int)(u >> 62);
  const int32_t r = (int32_t)((int64_t)((u & ((1ull << 62) - 1)) - (1ull << 61)) >> 30);
  const float x = (float)r * (0.78539816339744831f / 2147483648.0f);
  const float x2 = x * x;
  float s = fmaf(x2, 1.0f / 362880.0f, -1.0f / 5040.0f);
  s = fmaf(x2, s, 1.0f / 120.0f);
  s = fmaf(x2, s, -1.0f / 6.0f);
  s = fmaf(x2 * x, s, x);
  float c = fmaf(x2, 1.0f / 40320.0f, -1.0f / 720.0f);
  c = fmaf(x2, c, 1.0f / 24.0f);
  c = fmaf(x2, c, -0.5f);
  c = fmaf(x2, c, 1.0f);
  const bool swap = quad & 1;
  const float cc = swap ? s : c, ss = swap ? c : s;
  return make_float2((quad == 1 || quad == 2) ? -cc : cc, quad >= 2 ? -ss : ss);
}

__device__ __forceinline__ float2 rope_cos_sin(int32_t pos, uint64_t turns, float magnitude) {
  float2 cs = rope_cos_sin((uint64_t)(int64_t)pos * turns);
  cs.x *= magnitude;
  cs.y *= magnitude;
  return cs;
}

// Counts thread blocks that share a request in *arrive; true, and the count
// zero again, for the last of `total`.  Acquire-release: what the others read
// before arriving was read before the last one goes on.
__device__ __forceinline__ bool arrive_last(int* arrive, int total) {
  int prev;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(prev) : "l"(arrive) : "memory");
  if (prev != total - 1) return false;
  *arrive = 0;
  return true;
}

// The rotated pair, rounded in one way wherever it is computed (the result
// does not depend on the rows' alignment).
__device__ __forceinline__ float rope_first(float a, float b, float2 c) { return fmaf(a, c.x, -__fmul_rn(b, c.y)); }
__device__ __forceinline__ float rope_second(float a, float b, float2 c) { return fmaf(b, c.x, __fmul_rn(a, c.y)); }

// Host check of a rotary table against a head width.
inline bool rope_table_ok(const mtp_rope_table* r, int head_dim) {
  return r && (r->layout == MTP_ROPE_HALF || r->layout == MTP_ROPE_INTERLEAVED) && r->rotary_dim >= 2 &&
         r->rotary_dim % 2 == 0 && r->rotary_dim <= head_dim;
}

inline bool kv8_ok(const mtp_kv8* kv) {
  return kv && kv->k_pool && kv->v_pool && kv->k_scale && kv->v_scale && kv->block_table && kv->seq_len &&
         kv->pending && kv->arrive && kv->num_blocks > 0 && kv->max_blocks > 0 && !((uintptr_t)kv->k_pool & 15) &&
         !((uintptr_t)kv->v_pool & 15);
}

}  // namespace mtp
