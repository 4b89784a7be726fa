// Penalties for repeated tokens, biases and grammar masks on logits rows
// ("Speculative Decoding", "Overview": the target's rows that verification
// reads; row j of a request follows its first j drafts, so those count too).
//
//   z1 = z / r or z * r (z > 0 or not) where the token has occurred,
//   z2 = z1 - f c - p [c > 0],  z3 = z2 + bias,  -inf where the mask is clear.
//
// Each logit is read and written once and each count read once for all rows of
// its request.  A thread block owns a range of the vocabulary for one request;
// the factor and offset that its counts and biases make stay in registers while
// it walks over the request's rows, two of them in flight, and a draft changes
// its token's on the way.  Memory would bound it (64 requests x 6 rows of 151936
// with counts, biases and masks: 274 MB, 40 us); it takes 70 us, 3.9 TB/s, with
// nothing saturated: selects and bit tests keep the half-rate pipe half busy,
// 46 % of the warps are active at 64 registers a thread (bf16 vectors; 28 bytes
// are spilled, eight thread blocks per SM instead of six), and the loads of
// two rows ahead do not hide their latency.  1 x 6 rows: 4.5 us.
#include "mtp_kv8.cuh"

namespace mtp {

constexpr int kLogitThreads = 128;
constexpr int kLogitPer = 8;                                // consecutive entries per thread
constexpr int kLogitRange = kLogitThreads * kLogitPer;

// A thread's eight entries of a row, as loaded: consecutive ones in 16-byte
// vectors (VEC: rows and outputs start on 16 bytes and V is a multiple of 8),
// else every 32nd of its warp's 256, which keeps a warp's accesses together
// whatever the row's alignment.
template <typename T, bool VEC>
struct LogitRow {
  static constexpr int kWords = VEC && sizeof(T) == 2 ? 4 : 8;
  uint32_t w[kWords];
  // entry e of a lane, within the warp's 256
  __device__ static __forceinline__ int at(int lane, int e) { return VEC ? lane * kLogitPer + e : e * 32 + lane; }
  __device__ __forceinline__ void load(const T* row, int lane, int left) {
    if constexpr (VEC) {
      if (at(lane, 0) >= left) return;
      const uint4* p = reinterpret_cast<const uint4*>(row + at(lane, 0));
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 x = p[i / 4];
        w[i] = x.x; w[i + 1] = x.y; w[i + 2] = x.z; w[i + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < kLogitPer; ++e)
        if (at(lane, e) < left) w[e] = __float_as_uint(Elem<T>::loads(row + at(lane, e)));
    }
  }
  __device__ __forceinline__ float value(int e) const {
    return kWords == 8 ? __uint_as_float(w[e]) : (e & 1) ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
  }
  __device__ static __forceinline__ void store(T* row, const float (&z)[kLogitPer], int lane, int left) {
    if constexpr (VEC) {
      if (at(lane, 0) >= left) return;
      uint4* p = reinterpret_cast<uint4*>(row + at(lane, 0));
      uint32_t w[kWords];
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        if constexpr (kWords == 4) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(z[2 * i + 1]), "f"(z[2 * i]));
        else w[i] = __float_as_uint(z[i]);
      }
#pragma unroll
      for (int i = 0; i < kWords; i += 4) p[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    } else {
#pragma unroll
      for (int e = 0; e < kLogitPer; ++e)
        if (at(lane, e) < left) Elem<T>::store1(row + at(lane, e), z[e]);
    }
  }
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(kLogitThreads, (VEC && sizeof(T) == 2 ? 8 : 6)) logits_kernel(const mtp_logits_args a, int V, int* err) {
  using Row = LogitRow<T, VEC>;
  constexpr int kWarpRange = 32 * kLogitPer;
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int v0 = blockIdx.x * kLogitRange + warp * kWarpRange;     // the warp's first entry
  const int left = V - v0;                                         // entries from there on
  const int o0 = a.row_offsets[b], o1 = a.row_offsets[b + 1];
  uint32_t cnt[kLogitPer];
#pragma unroll
  for (int e = 0; e < kLogitPer; ++e) cnt[e] = 0;
  if (a.counts) {
    const int32_t* counts = a.counts + (long long)b * V + v0;
    if (VEC && !((uintptr_t)a.counts & 15)) {
      if (Row::at(lane, 0) < left) {
        const uint4* p = reinterpret_cast<const uint4*>(counts + Row::at(lane, 0));
        const uint4 y = __ldg(p), w = __ldg(p + 1);
        cnt[0] = y.x; cnt[1] = y.y; cnt[2] = y.z; cnt[3] = y.w;
        cnt[4] = w.x; cnt[5] = w.y; cnt[6] = w.z; cnt[7] = w.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < kLogitPer; ++e)
        if (Row::at(lane, e) < left) cnt[e] = (uint32_t)__ldg(counts + Row::at(lane, e));
    }
  }
  float rep = 1.0f, freq = 0.0f, pres = 0.0f;
  if (a.repetition) rep = a.repetition[b];
  if (a.frequency) freq = a.frequency[b];
  if (a.presence) pres = a.presence[b];
  int e0 = 0, e1 = 0;
  if (a.bias_offsets) {
    e0 = a.bias_offsets[b];
    e1 = a.bias_offsets[b + 1];
  }
  const int n = o1 - o0;
  if (o0 < 0 || o1 < o0 || o1 > a.num_rows || (a.drafts && n > a.drafts_stride + 1) || !(rep > 0.0f) ||
      !finite_f(rep) || !finite_f(freq) || !finite_f(pres) || e0 < 0 || e1 < e0 || e1 > a.num_bias) {
    if (threadIdx.x == 0) set_error(err, MTP_ERR_DEVICE_ARGS);
    return;
  }
  if (n == 0 || left <= 0) return;
  const T* x = (const T*)a.logits + (long long)o0 * V + v0;
  T* out = (T*)a.out + (long long)o0 * V + v0;
  const int32_t* drafts = a.drafts ? a.drafts + (long long)b * a.drafts_stride : nullptr;
  // the first two rows, and the first one's mask, on their way
  Row cur, next;
  cur.load(x, lane, left);
  if (n > 1) next.load(x + V, lane, left);
  const int words = (V + 31) / 32;
  const int32_t* mask = a.mask + (v0 >> 5);
  // the mask bits of the thread's entries in row j; 0x100: a bad index, the row is left as it was
  auto allowed = [&](int j) -> uint32_t {
    const int mi = a.mask_index[o0 + j];
    if (mi == -1) return 0xFFu;
    if (mi < -1 || mi >= a.num_masks) {
      set_error(err, MTP_ERR_DEVICE_ARGS);
      return 0x100u;
    }
    const int32_t* m = mask + (long long)mi * words;
    if constexpr (VEC) {
      return Row::at(lane, 0) < left ? (uint32_t)__ldg(m + (lane >> 2)) >> (8 * (lane & 3)) & 0xFFu : 0u;
    } else {
      uint32_t ok = 0;
#pragma unroll
      for (int e = 0; e < kLogitPer; ++e)
        if (Row::at(lane, e) < left) ok |= ((uint32_t)__ldg(m + e) >> lane & 1u) << e;
      return ok;
    }
  };
  uint32_t ok = a.mask ? allowed(0) : 0xFFu;
  // z <- z * (z > 0 ? up : down) - sub, sub = f c + p [c > 0] - bias.  Each warp
  // looks through the biases for its own entries; one that falls among them
  // is added by the thread that owns it, in the list's order.
  float up[kLogitPer], down[kLogitPer], sub[kLogitPer];
  bool any = false;
#pragma unroll
  for (int e = 0; e < kLogitPer; ++e) sub[e] = 0.0f;
  for (int at = e0; at < e1; at += 32) {
    const int t = at + lane < e1 ? a.bias_tokens[at + lane] : -1;
    if (v0 == 0 && at + lane < e1 && (t < 0 || t >= V)) set_error(err, MTP_ERR_DEVICE_ARGS);
    for (unsigned hit = __ballot_sync(0xffffffffu, t >= v0 && t < V && t - v0 < kWarpRange); hit; hit &= hit - 1) {
      const int l = __ffs(hit) - 1, k = __shfl_sync(0xffffffffu, t, l) - v0;
      const float y = a.bias_values[at + l];
#pragma unroll
      for (int e = 0; e < kLogitPer; ++e)
        if (Row::at(lane, e) == k) {
          sub[e] -= y;
          any = true;
        }
    }
  }
  const float inv = 1.0f / rep;
#pragma unroll
  for (int e = 0; e < kLogitPer; ++e) {
    const uint32_t c = cnt[e] & 0x7FFFFFFFu;
    up[e] = cnt[e] ? inv : 1.0f;
    down[e] = cnt[e] ? rep : 1.0f;
    sub[e] += fmaf(freq, (float)(int)c, c ? pres : 0.0f);
    any |= cnt[e] != 0;
  }
  int d_next = drafts && n > 1 ? drafts[0] : -1;
#pragma unroll 2
  for (int j = 0; j < n; ++j) {
    float z[kLogitPer];
#pragma unroll
    for (int e = 0; e < kLogitPer; ++e) z[e] = cur.value(e);
    cur = next;
    if (j + 2 < n) next.load(x + 2 * (long long)V, lane, left);
    x += V;
    const uint32_t ok_now = ok;
    if (a.mask && j + 1 < n) ok = allowed(j + 1);
    if (any) {
#pragma unroll
      for (int e = 0; e < kLogitPer; ++e) z[e] = fmaf(z[e], z[e] > 0.0f ? up[e] : down[e], -sub[e]);
    }
    if (ok_now != 0xFFu) {
#pragma unroll
      for (int e = 0; e < kLogitPer; ++e)
        if (!(ok_now & (1u << e))) z[e] = -INFINITY;
    }
    if (ok_now != 0x100u && MTP_IN_BOUNDS(err, o0 + j, a.num_rows)) Row::store(out, z, lane, left);
    out += V;
    // the draft between row j and row j + 1 counts from there on
    const int d = d_next - v0;
    if (drafts && j + 2 < n) d_next = drafts[j + 1];
    if (drafts && j + 1 < n && d >= 0 && d < kWarpRange && d < left) {
      const int32_t* counts = a.counts + (long long)b * V + v0;
      uint32_t c = (uint32_t)__ldg(counts + d) & 0x7FFFFFFFu;   // the token's count before this draft
      for (int k = 0; k < j; ++k) c += drafts[k] - v0 == d ? 1u : 0u;
#pragma unroll
      for (int e = 0; e < kLogitPer; ++e)
        if (Row::at(lane, e) == d) {
          up[e] = inv;
          down[e] = rep;
          sub[e] += c ? freq : freq + pres;
          any = true;
        }
    }
  }
}

// One atomic add (or or) per token; sums of whole numbers do not depend on
// their order.
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
  if (a.drafts && a.drafts_stride < 0) return MTP_ERR_INVALID;
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
