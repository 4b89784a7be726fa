// Penalties for repeated tokens, biases and grammar masks on logits rows
// ("Speculative Decoding", "Overview": the target's rows that verification
// reads; row j of a request follows its first j drafts, so those count too).
//
//   z1 = z / r or z * r (z > 0 or not) where the token has occurred,
//   z2 = z1 - f c - p [c > 0],  z3 = z2 + bias,  -inf where the mask is clear.
//
// Memory bounds it: each logit is read and written once and each count read
// once for all rows of its request.  A thread block owns a range of the
// vocabulary for one request; its counts and biases stay in registers while
// it walks over the request's rows, a draft raising its token's count on the
// way.
#include "mtp_kv8.cuh"

namespace mtp {

constexpr int kLogitThreads = 128;
constexpr int kLogitPer = 8;                                // consecutive entries per thread
constexpr int kLogitRange = kLogitThreads * kLogitPer;

// Sum the biases that fall into [v0, v0 + kLogitRange) into acc.  One warp
// walks the list 32 entries at a time; entries of one step that name the same
// token are added by its first lane in list order, so the sum does not depend
// on timing.
__device__ __forceinline__ void gather_biases(const int32_t* tok, const float* val, int e0, int e1, int v0, int V,
                                              float* acc, int* err) {
  const int lane = threadIdx.x & 31;
  for (int e = e0; e < e1; e += 32) {
    const bool in = e + lane < e1;
    const int t = in ? tok[e + lane] : -1;
    const float x = in ? val[e + lane] : 0.0f;
    if (in && (t < 0 || t >= V) && v0 == 0) set_error(err, MTP_ERR_DEVICE_ARGS);
    const bool mine = in && t >= v0 && t < V && t < v0 + kLogitRange;
    if (!__any_sync(0xffffffffu, mine)) continue;
    const unsigned same = __match_any_sync(0xffffffffu, mine ? t : -1 - lane);
    float sum = 0.0f;
    for (int l = 0; l < 32; ++l) {
      const float y = __shfl_sync(0xffffffffu, x, l);
      if (same >> l & 1u) sum = (l == __ffs(same) - 1) ? (mine ? acc[t - v0] + y : 0.0f) : sum + y;
    }
    if (mine && lane == __ffs(same) - 1) acc[t - v0] = sum;
    __syncwarp();
  }
}

template <typename T>
__global__ void __launch_bounds__(kLogitThreads) logits_kernel(const mtp_logits_args a, int V, int* err) {
  __shared__ float bias[kLogitRange];
  const int b = blockIdx.y, v0 = blockIdx.x * kLogitRange, tid = threadIdx.x;
  const int o0 = a.row_offsets[b], o1 = a.row_offsets[b + 1];
  float rep = 1.0f, freq = 0.0f, pres = 0.0f;
  if (a.repetition) rep = a.repetition[b];
  if (a.frequency) freq = a.frequency[b];
  if (a.presence) pres = a.presence[b];
  int e0 = 0, e1 = 0;
  if (a.bias_offsets) {
    e0 = a.bias_offsets[b];
    e1 = a.bias_offsets[b + 1];
  }
  if (o0 < 0 || o1 < o0 || o1 > a.num_rows || (a.drafts && o1 - o0 > a.drafts_stride + 1) || !(rep > 0.0f) ||
      !finite_f(rep) || !finite_f(freq) || !finite_f(pres) || e0 < 0 || e1 < e0 || e1 > a.num_bias) {
    if (tid == 0) set_error(err, MTP_ERR_DEVICE_ARGS);
    return;
  }
  if (o0 == o1) return;
  if (e1 > e0) {
    for (int i = tid; i < kLogitRange; i += kLogitThreads) bias[i] = 0.0f;
    __syncthreads();
    if (tid < 32) gather_biases(a.bias_tokens, a.bias_values, e0, e1, v0, V, bias, err);
    __syncthreads();
  }
  const int base = v0 + tid * kLogitPer;
  if (base >= V) return;
  const int n = min(kLogitPer, V - base);
  const float inv = 1.0f / rep;
  const int words = (V + 31) / 32;
  uint32_t cnt[kLogitPer];
#pragma unroll
  for (int e = 0; e < kLogitPer; ++e)
    cnt[e] = a.counts && e < n ? (uint32_t)a.counts[(long long)b * V + base + e] : 0u;
  for (int j = 0; j < o1 - o0; ++j) {
    const long long row = o0 + j;
    if (j > 0 && a.drafts) {
      const int d = a.drafts[(long long)b * a.drafts_stride + j - 1] - base;
#pragma unroll
      for (int e = 0; e < kLogitPer; ++e) cnt[e] += e == d ? 1u : 0u;
    }
    uint32_t allow = 0xFFu;
    if (a.mask) {
      const int mi = a.mask_index[row];
      if (mi < -1 || mi >= a.num_masks) {
        set_error(err, MTP_ERR_DEVICE_ARGS);
        continue;
      }
      if (mi >= 0) allow = (uint32_t)a.mask[(long long)mi * words + (base >> 5)] >> (base & 31);
    }
#pragma unroll
    for (int e = 0; e < kLogitPer; ++e) {
      if (e >= n) break;
      float z = Elem<T>::loads((const T*)a.logits + row * V + base + e);
      const uint32_t c = cnt[e] & 0x7FFFFFFFu;
      if (cnt[e]) {
        z = z > 0.0f ? z * inv : z * rep;
        z = z - freq * (float)c - (c ? pres : 0.0f);
      }
      if (e1 > e0) z += bias[tid * kLogitPer + e];
      if (!(allow >> e & 1u)) z = -INFINITY;
      Elem<T>::store1((T*)a.out + row * V + base + e, z);
    }
  }
}

__global__ void __launch_bounds__(128) counts_add_kernel(const int32_t* tokens, int stride, const int32_t* n_tokens,
                                                         int in_prompt, int32_t* counts, int V, int* err) {
  const int b = blockIdx.y, n = n_tokens[b];
  if (n < 0 || n > stride) {
    if (threadIdx.x == 0) set_error(err, MTP_ERR_DEVICE_ARGS);
    return;
  }
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) {
    const int t = tokens[(long long)b * stride + i];
    if (t < 0 || t >= V) {
      set_error(err, MTP_ERR_DEVICE_ARGS);
      continue;
    }
    int32_t* c = counts + (long long)b * V + t;
    if (in_prompt) atomicOr(c, (int)0x80000000u); else atomicAdd(c, 1);
  }
}

}  // namespace mtp

using namespace mtp;

extern "C" {

mtp_status mtp_token_counts_add(mtp_ctx* ctx, void* stream, int B, const int32_t* tokens, int stride,
                                const int32_t* n_tokens, int in_prompt, int32_t* counts) {
  if (!ctx || B < 1 || B > ctx->cfg.max_batch || B > 65535 || !tokens || stride < 1 || !n_tokens || !counts ||
      (in_prompt != 0 && in_prompt != 1))
    return MTP_ERR_INVALID;
  DeviceGuard dev(ctx->device);
  if (!dev.ok) return MTP_ERR_CUDA;
  const int gx = stride < 64 * 128 ? (stride + 127) / 128 : 64;
  counts_add_kernel<<<dim3(gx, B), 128, 0, (cudaStream_t)stream>>>(tokens, stride, n_tokens, in_prompt, counts,
                                                                   ctx->cfg.vocab, ctx->err);
  ctx->launches++;
  return launch_status(cudaGetLastError());
}

mtp_status mtp_logits_process(mtp_ctx* ctx, void* stream, const mtp_logits_args* args) {
  if (!ctx || !args) return MTP_ERR_INVALID;
  const mtp_logits_args& a = *args;
  if (a.B < 1 || a.B > ctx->cfg.max_batch || a.B > 65535 || a.num_rows < 0 || !a.row_offsets || !a.logits || !a.out)
    return MTP_ERR_INVALID;
  if ((a.drafts || a.repetition || a.frequency || a.presence) && !a.counts) return MTP_ERR_INVALID;
  if (a.drafts && a.drafts_stride < 1) return MTP_ERR_INVALID;
  if (a.bias_offsets && (a.num_bias < 0 || (a.num_bias > 0 && (!a.bias_tokens || !a.bias_values))))
    return MTP_ERR_INVALID;
  if (a.mask && (!a.mask_index || a.num_masks < 1)) return MTP_ERR_INVALID;
  if (a.num_rows == 0) return MTP_OK;
  DeviceGuard dev(ctx->device);
  if (!dev.ok) return MTP_ERR_CUDA;
  const int V = ctx->cfg.vocab;
  const dim3 grid((V + kLogitRange - 1) / kLogitRange, a.B);
  if (ctx->cfg.dtype == MTP_DTYPE_BF16)
    logits_kernel<uint16_t><<<grid, kLogitThreads, 0, (cudaStream_t)stream>>>(a, V, ctx->err);
  else
    logits_kernel<float><<<grid, kLogitThreads, 0, (cudaStream_t)stream>>>(a, V, ctx->err);
  ctx->launches++;
  return launch_status(cudaGetLastError());
}

}  // extern "C"
