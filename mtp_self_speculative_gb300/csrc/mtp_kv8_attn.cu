// Attention of a request's new rows over its 8-bit cache (decode, draft
// verification, packed trees).
//
//   out[r, h] = sum_t p_t V[t, g] / sum_t p_t,  p_t = 2^(c s_t - m),
//   s_t = q[r, h] . K[t, g], c = scale * log2 e, m the running maximum.
//
// A warp owns one (row, query head): lanes hold head_dim / 32 dimensions,
// scores are summed across the lanes, and the softmax is online.
#include <math.h>

#include "mtp_kv8.cuh"

namespace mtp {

struct Attn8Args {
  const void* q;
  void* out;
  float* lse;
  const int32_t* row_offsets;
  const int32_t* mask;
  mtp_kv8 kv;
  int* err;
  long long q_stride;
  int B, T, max_rows, mask_words, n_kv, n_q;
  float qscale;  // scale * log2(e)
};

template <typename T, int HD>
__global__ void __launch_bounds__(128) kv8_attn_kernel(const Attn8Args a) {
  constexpr int DPL = HD / 32;
  __shared__ int sh[3];
  const int r = blockIdx.x;
  if (!find_request(a.row_offsets, a.B, a.T, r, a.err, sh, [](int o, int) { return o; })) return;
  const int b = sh[0], o0 = sh[1], n = sh[2] - o0;
  const int lane = threadIdx.x & 31, h = blockIdx.y * 4 + (threadIdx.x >> 5);
  const long long L = (long long)a.kv.seq_len[b] + a.kv.pending[b];
  if (n > a.max_rows || L < n || a.kv.seq_len[b] < 0 || a.kv.pending[b] < 0) {
    if (threadIdx.x == 0) set_error(a.err, MTP_ERR_DEVICE_ARGS);
    return;
  }
  if (L > (long long)a.kv.max_blocks * kBlk) {
    if (threadIdx.x == 0) set_error(a.err, MTP_ERR_CAPACITY);
    return;
  }
  if (h >= a.n_q) return;
  const int g = h / (a.n_q / a.n_kv), base = (int)L - n, i = r - o0;
  const int32_t* bits = a.mask ? a.mask + (long long)r * a.mask_words : nullptr;
  float q[DPL], o[DPL], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int e = 0; e < DPL; ++e) {
    q[e] = Elem<T>::load1((const T*)a.q + (long long)r * a.q_stride + h * HD + lane * DPL + e);
    o[e] = 0.0f;
  }
  for (int t = 0; t < (int)L; ++t) {
    const int j = t - base;
    if (j >= 0 && (bits ? !((uint32_t)bits[j >> 5] >> (j & 31) & 1u) : j > i)) continue;
    const int blk = a.kv.block_table[(long long)b * a.kv.max_blocks + (t >> 4)];
    float kx[DPL], vx[DPL];
#pragma unroll
    for (int e = 0; e < DPL; ++e) kx[e] = vx[e] = 0.0f;
    if (blk < 0 || blk >= a.kv.num_blocks) {
      if (lane == 0) set_error(a.err, MTP_ERR_CAPACITY);
    } else {
      const long long tile = (long long)blk * a.n_kv + g, at = (tile * kBlk + (t & 15)) * HD + lane * DPL;
      const float ks = a.kv.k_scale[tile], vs = a.kv.v_scale[tile];
#pragma unroll
      for (int e = 0; e < DPL; e += 2) {
        const float2 kk = e4m3_to_float2(*(const uint16_t*)((const uint8_t*)a.kv.k_pool + at + e));
        const float2 vv = e4m3_to_float2(*(const uint16_t*)((const uint8_t*)a.kv.v_pool + at + e));
        kx[e] = kk.x * ks; kx[e + 1] = kk.y * ks;
        vx[e] = vv.x * vs; vx[e + 1] = vv.y * vs;
      }
    }
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < DPL; ++e) s = fmaf(q[e], kx[e], s);
    s = warp_sum(s) * a.qscale;
    const float mn = fmaxf(m, s);
    const float f = m == -INFINITY ? 0.0f : exp2f(m - mn), p = exp2f(s - mn);
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < DPL; ++e) o[e] = o[e] * f + p * vx[e];
    m = mn;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int e = 0; e < DPL; ++e)
    Elem<T>::store1((T*)a.out + ((long long)r * a.n_q + h) * HD + lane * DPL + e, o[e] * inv);
  if (a.lse && lane == 0)
    a.lse[(long long)r * a.n_q + h] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace mtp

using namespace mtp;

extern "C" {

size_t mtp_kv8_attention_workspace_bytes(const mtp_ctx* ctx) { return ctx ? 256 : 0; }

mtp_status mtp_kv8_attention(mtp_ctx* ctx, void* stream, int B, int T, const int32_t* row_offsets, int max_rows,
                             const void* q, int64_t q_stride, const mtp_kv8* kv, const int32_t* mask, int mask_words,
                             float scale, void* out, float* lse, void* ws, size_t ws_bytes) {
  if (!ctx || B < 1 || B > ctx->cfg.max_batch || T < 0 || !row_offsets || !q || !out || !kv8_ok(kv))
    return MTP_ERR_INVALID;
  const mtp_config& c = ctx->cfg;
  if (max_rows < 1 || max_rows > 256 || q_stride < (int64_t)c.n_q_heads * c.head_dim) return MTP_ERR_INVALID;
  if (mask && mask_words < (max_rows + 31) / 32) return MTP_ERR_INVALID;
  if (!(scale > 0.0f) || !isfinite(scale)) return MTP_ERR_INVALID;
  if (!ws || ((uintptr_t)ws & 15) || ws_bytes < mtp_kv8_attention_workspace_bytes(ctx)) return MTP_ERR_INVALID;
  if (T == 0) return MTP_OK;
  DeviceGuard dev(ctx->device);
  if (!dev.ok) return MTP_ERR_CUDA;
  Attn8Args a{q, out, lse, row_offsets, mask, *kv, ctx->err, q_stride, B, T, max_rows, mask_words, c.n_kv_heads,
              c.n_q_heads, scale * 1.4426950408889634f};
  const dim3 grid(T, (c.n_q_heads + 3) / 4);
  cudaStream_t s = (cudaStream_t)stream;
  const bool bf = c.dtype == MTP_DTYPE_BF16;
  if (c.head_dim == 128) {
    if (bf) kv8_attn_kernel<uint16_t, 128><<<grid, 128, 0, s>>>(a);
    else kv8_attn_kernel<float, 128><<<grid, 128, 0, s>>>(a);
  } else {
    if (bf) kv8_attn_kernel<uint16_t, 64><<<grid, 128, 0, s>>>(a);
    else kv8_attn_kernel<float, 64><<<grid, 128, 0, s>>>(a);
  }
  ctx->launches++;
  return launch_status(cudaGetLastError());
}

}  // extern "C"
