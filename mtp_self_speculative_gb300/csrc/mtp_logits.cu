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

// A thread's eight entries of a row: consecutive ones in 16-byte vectors
// (VEC: rows and outputs start on 16 bytes), else every 128th, which keeps a
// warp's accesses together whatever the row's alignment.
template <typename T, bool VEC>
struct LogitRow {
  float z[kLogitPer];
  __device__ static __forceinline__ int at(int v0, int tid, int e) {
    return VEC ? v0 + tid * kLogitPer + e : v0 + e * kLogitThreads + tid;
  }
  __device__ __forceinline__ void load(const T* row, int v0, int tid, int V) {
    if constexpr (VEC) {
      if (at(v0, tid, 0) >= V) return;  // V is a multiple of 8 here
      const uint4* p = reinterpret_cast<const uint4*>(row + at(v0, tid, 0));
      if constexpr (sizeof(T) == 2) {
        const uint4 x = *p;
        z[0] = bf16_lo(x.x); z[1] = bf16_hi(x.x); z[2] = bf16_lo(x.y); z[3] = bf16_hi(x.y);
        z[4] = bf16_lo(x.z); z[5] = bf16_hi(x.z); z[6] = bf16_lo(x.w); z[7] = bf16_hi(x.w);
      } else {
        const uint4 x = p[0], y = p[1];
        z[0] = __uint_as_float(x.x); z[1] = __uint_as_float(x.y); z[2] = __uint_as_float(x.z);
        z[3] = __uint_as_float(x.w); z[4] = __uint_as_float(y.x); z[5] = __uint_as_float(y.y);
        z[6] = __uint_as_float(y.z); z[7] = __uint_as_float(y.w);
      }
    } else {
#pragma unroll
      for (int e = 0; e < kLogitPer; ++e)
        if (at(v0, tid, e) < V) z[e] = Elem<T>::loads(row + at(v0, tid, e));
    }
  }
  __device__ __forceinline__ void store(T* row, int v0, int tid, int V) const {
    if constexpr (VEC) {
      if (at(v0, tid, 0) >= V) return;
      uint4* p = reinterpret_cast<uint4*>(row + at(v0, tid, 0));
      if constexpr (sizeof(T) == 2) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = (uint32_t)f32_to_bf16_rne(z[2 * i]) | ((uint32_t)f32_to_bf16_rne(z[2 * i + 1]) << 16);
        *p = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        p[0] = make_uint4(__float_as_uint(z[0]), __float_as_uint(z[1]), __float_as_uint(z[2]), __float_as_uint(z[3]));
        p[1] = make_uint4(__float_as_uint(z[4]), __float_as_uint(z[5]), __float_as_uint(z[6]), __float_as_uint(z[7]));
      }
    } else {
#pragma unroll
      for (int e = 0; e < kLogitPer; ++e)
        if (at(v0, tid, e) < V) Elem<T>::store1(row + at(v0, tid, e), z[e]);
    }
  }
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(kLogitThreads) logits_kernel(const mtp_logits_args a, int V, int* err) {
  using Row = LogitRow<T, VEC>;
  __shared__ float bias_s[kLogitRange];
  pdl_wait();
  pdl_trigger();
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
  const T* x = (const T*)a.logits;
  T* out = (T*)a.out;
  Row next;
  next.load(x + (long long)o0 * V, v0, tid, V);
  uint32_t cnt[kLogitPer], any = 0;
#pragma unroll
  for (int e = 0; e < kLogitPer; ++e) cnt[e] = 0;
  if (a.counts) {
    const int32_t* c = a.counts + (long long)b * V;
    if (VEC && !((uintptr_t)a.counts & 15)) {
      if (Row::at(v0, tid, 0) < V) {
        const uint4* p = reinterpret_cast<const uint4*>(c + Row::at(v0, tid, 0));
        const uint4 y = __ldg(p), w = __ldg(p + 1);
        cnt[0] = y.x; cnt[1] = y.y; cnt[2] = y.z; cnt[3] = y.w;
        cnt[4] = w.x; cnt[5] = w.y; cnt[6] = w.z; cnt[7] = w.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < kLogitPer; ++e)
        if (Row::at(v0, tid, e) < V) cnt[e] = (uint32_t)__ldg(c + Row::at(v0, tid, e));
    }
  }
  float bias[kLogitPer];
#pragma unroll
  for (int e = 0; e < kLogitPer; ++e) bias[e] = 0.0f;
  if (e1 > e0) {
    for (int i = tid; i < kLogitRange; i += kLogitThreads) bias_s[i] = 0.0f;
    __syncthreads();
    if (tid < 32) gather_biases(a.bias_tokens, a.bias_values, e0, e1, v0, V, bias_s, err);
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kLogitPer; ++e) bias[e] = bias_s[Row::at(0, tid, e)];
  }
#pragma unroll
  for (int e = 0; e < kLogitPer; ++e) any |= cnt[e];
  const float inv = 1.0f / rep;
  const int words = (V + 31) / 32;
  for (int j = 0; j < o1 - o0; ++j) {
    const long long row = o0 + j;
    Row z = next;
    if (j + 1 < o1 - o0) next.load(x + (row + 1) * V, v0, tid, V);
    if (j > 0 && a.drafts) {
      const int d = a.drafts[(long long)b * a.drafts_stride + j - 1];
      if (d >= v0 && d < v0 + kLogitRange) {
#pragma unroll
        for (int e = 0; e < kLogitPer; ++e)
          if (Row::at(v0, tid, e) == d) {
            cnt[e] += 1u;
            any |= 1u;
          }
      }
    }
    if (any) {
#pragma unroll
      for (int e = 0; e < kLogitPer; ++e) {
        const uint32_t c = cnt[e] & 0x7FFFFFFFu;
        const float met = z.z[e] * (z.z[e] > 0.0f ? inv : rep) - freq * (float)c;
        if (cnt[e]) z.z[e] = c ? met - pres : met;
      }
    }
    if (e1 > e0) {
#pragma unroll
      for (int e = 0; e < kLogitPer; ++e) z.z[e] += bias[e];
    }
    if (a.mask) {
      const int mi = a.mask_index[row];
      if (mi < -1 || mi >= a.num_masks) {
        set_error(err, MTP_ERR_DEVICE_ARGS);
        continue;
      }
      if (mi >= 0) {
        const int32_t* m = a.mask + (long long)mi * words;
        if constexpr (VEC) {
          const int v = Row::at(v0, tid, 0);
          const uint32_t ok = v < V ? (uint32_t)__ldg(m + (v >> 5)) >> (v & 31) : 0u;
#pragma unroll
          for (int e = 0; e < kLogitPer; ++e)
            if (!(ok >> e & 1u)) z.z[e] = -INFINITY;
        } else {
#pragma unroll
          for (int e = 0; e < kLogitPer; ++e) {
            const int v = Row::at(v0, tid, e);
            if (v < V && !((uint32_t)__ldg(m + (v >> 5)) >> (v & 31) & 1u)) z.z[e] = -INFINITY;
          }
        }
      }
    }
    if (MTP_IN_BOUNDS(err, row, a.num_rows)) z.store(out + row * V, v0, tid, V);
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
  const bool vec = V % 8 == 0 && !(((uintptr_t)a.logits | (uintptr_t)a.out) & 15);
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  if (ctx->cfg.dtype == MTP_DTYPE_BF16)
    e = vec ? launch_pdl(logits_kernel<uint16_t, true>, grid, dim3(kLogitThreads), 0, s, a, V, ctx->err)
            : launch_pdl(logits_kernel<uint16_t, false>, grid, dim3(kLogitThreads), 0, s, a, V, ctx->err);
  else
    e = vec ? launch_pdl(logits_kernel<float, true>, grid, dim3(kLogitThreads), 0, s, a, V, ctx->err)
            : launch_pdl(logits_kernel<float, false>, grid, dim3(kLogitThreads), 0, s, a, V, ctx->err);
  ctx->launches++;
  return launch_status(e);
}

}  // extern "C"
