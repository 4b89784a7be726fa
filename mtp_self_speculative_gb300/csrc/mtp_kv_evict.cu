// Eviction from a paged cache by the attention weight that its entries have
// gathered: for each request and kv head the first `sink` entries, the last
// `recent` ones and, of those between, the ones with the largest weights stay,
// and move in their order to the blocks of another cache.
//
// Two kernels.  The first finds, per (request, kv head), the weight of the
// last entry that stays, digit by digit (11, 11 and 10 bits of the weights'
// ordered bit patterns, counted in shared memory), and lists the slots that
// stay in ascending order; equal weights stay from the lowest slot on, so the
// result depends on nothing but the weights.  The second copies: a thread block
// per (request, kv head, new cache block), 16 bytes a lane.
#include "mtp_kv16.cuh"

namespace mtp {

constexpr int kSelThreads = 1024;
constexpr int kSelBins = 2048;

struct EvictArgs {
  mtp_kv from, to;
  const float* weights;     // [from.num_blocks, n_kv, 16]
  float* to_weights;        // [to.num_blocks, n_kv, 16] or null
  const int32_t* budget;    // [B]
  int32_t* kept;            // [B, n_kv, width]
  int* err;
  int B, n_kv, hd, sink, recent, width;
  int cached;               // keys that the selection's shared memory holds
};

// A request's entries and how many stay; false (and the error) for one that
// is left out.
__device__ __forceinline__ bool evict_request(const EvictArgs& a, int b, int& L, int& n, bool report) {
  L = a.from.seq_len[b];
  const int budget = a.budget[b];
  int e = MTP_OK;
  if (L < 0 || a.from.pending[b] != 0 || budget < 0 || (long long)a.sink + a.recent > budget) e = MTP_ERR_DEVICE_ARGS;
  else if ((long long)L > (long long)a.from.max_blocks * kBlk) e = MTP_ERR_CAPACITY;
  n = min(L, budget);
  if (e == MTP_OK && (n > a.width || (long long)n > (long long)a.to.max_blocks * kBlk)) e = MTP_ERR_CAPACITY;
  if (e != MTP_OK && report) set_error(a.err, e);
  return e == MTP_OK;
}

// Larger weights have larger keys; -0 counts as 0 and NaN below everything.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  if (w == 0.0f) w = 0.0f;
  const uint32_t u = __float_as_uint(w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive sum over the block of each thread's value, and the total.
__device__ __forceinline__ int block_scan(int v, int* warps, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();   // (earlier readers of `warps` are done)
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int y = warps[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, y, d);
      if (lane >= d) y += z;
    }
    warps[lane] = y;
  }
  __syncthreads();
  total = warps[kSelThreads / 32 - 1];
  return x - v + (warp ? warps[warp - 1] : 0);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  extern __shared__ uint32_t keys[];
  __shared__ int bins[kSelBins];
  __shared__ int warps[kSelThreads / 32];
  __shared__ uint32_t digit_s;
  __shared__ int above_s;
  pdl_wait();
  pdl_trigger();
  const int g = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int L, n;
  if (!evict_request(a, b, L, n, g == 0 && tid == 0)) return;
  int32_t* kept = a.kept + ((long long)b * a.n_kv + g) * a.width;
  for (int j = n + tid; j < a.width; j += kSelThreads) kept[j] = -1;
  if (n == L) {
    for (int j = tid; j < n; j += kSelThreads) kept[j] = j;
    return;
  }
  // candidates: the slots [lo, hi); `want` of them stay (budget - sink - recent >= 0)
  const int lo = a.sink, hi = L - a.recent, want = n - a.sink - a.recent;
  const int32_t* row = a.from.block_table + (long long)b * a.from.max_blocks;
  int lost = 0;
  auto load_key = [&](int t) -> uint32_t {
    const int blk = row[t >> 4];
    if (blk < 0 || blk >= a.from.num_blocks) {
      lost = 1;
      return 0u;
    }
    return weight_key(a.weights[((long long)blk * a.n_kv + g) * kBlk + (t & 15)]);
  };
  auto key_of = [&](int t) -> uint32_t { return t - lo < a.cached ? keys[t - lo] : load_key(t); };
  for (int t = lo + tid; t < hi && t - lo < a.cached; t += kSelThreads) keys[t - lo] = load_key(t);
  if (lost) set_error(a.err, MTP_ERR_CAPACITY);
  // ---- the key of the last candidate that stays, from its high digits down
  uint32_t prefix = 0;
  int left = want;             // how many of the keys that share the prefix stay
  int shift = 32;
  if (want > 0) {
    for (int pass = 0; pass < 3; ++pass) {
      const int width = pass == 2 ? 10 : 11;
      const uint32_t high = shift == 32 ? 0u : ~0u << shift;   // the digits that are known
      shift -= width;
      for (int i = tid; i < kSelBins; i += kSelThreads) bins[i] = 0;
      __syncthreads();
      // the loop runs for whole warps, so that a warp whose keys agree adds once
      for (int t0 = lo + warp * 32; t0 < hi; t0 += kSelThreads) {
        const int t = t0 + lane;
        const uint32_t k = t < hi ? key_of(t) : 0u;
        const bool in = t < hi && (k & high) == prefix;
        const uint32_t d = in ? (k >> shift) & ((1u << width) - 1u) : 0xFFFFFFFFu;
        int same;
        __match_all_sync(0xffffffffu, d, &same);
        if (same) {
          if (in && lane == 0) atomicAdd(&bins[d], 32);
        } else if (in) {
          atomicAdd(&bins[d], 1);
        }
      }
      __syncthreads();
      // thread i looks at digits 2 i and 2 i + 1 counted from the top
      const int top = kSelBins - 1 - 2 * tid;
      const int c1 = bins[top], c0 = bins[top - 1];
      int total;
      const int before = block_scan(c1 + c0, warps, total);   // keys with a larger digit
      if (before < left && before + c1 >= left) {
        digit_s = (uint32_t)top;
        above_s = before;
      } else if (before + c1 < left && before + c1 + c0 >= left) {
        digit_s = (uint32_t)(top - 1);
        above_s = before + c1;
      }
      __syncthreads();
      prefix |= digit_s << shift;
      left -= above_s;
      __syncthreads();
    }
  }
  // ---- list: warp w takes a contiguous share of all slots
  const int per = ((L + kSelThreads / 32 - 1) / (kSelThreads / 32) + 31) / 32 * 32;
  const int s0 = warp * per, s1 = min(L, s0 + per);
  int n_more = 0, n_same = 0;   // slots that stay anyway or lie above, and those that equal the last key
  for (int t0 = s0; t0 < s1; t0 += 32) {
    const int t = t0 + lane;
    const bool cand = t < s1 && t >= lo && t < hi;
    const uint32_t k = cand && want > 0 ? key_of(t) : 0u;
    const bool more = t < s1 && (!cand || (want > 0 && k > prefix)), same = cand && want > 0 && k == prefix;
    n_more += __popc(__ballot_sync(0xffffffffu, more));
    n_same += __popc(__ballot_sync(0xffffffffu, same));
  }
  int total;
  const int more_before = block_scan(lane == 0 ? n_more : 0, warps, total);
  const int same_before = block_scan(lane == 0 ? n_same : 0, warps, total);
  int more_at = __shfl_sync(0xffffffffu, more_before, 0), same_at = __shfl_sync(0xffffffffu, same_before, 0);
  const uint32_t under = (1u << lane) - 1u;
  for (int t0 = s0; t0 < s1; t0 += 32) {
    const int t = t0 + lane;
    const bool cand = t < s1 && t >= lo && t < hi;
    const uint32_t k = cand && want > 0 ? key_of(t) : 0u;
    const bool more = t < s1 && (!cand || (want > 0 && k > prefix)), same = cand && want > 0 && k == prefix;
    const uint32_t mb = __ballot_sync(0xffffffffu, more), sb = __ballot_sync(0xffffffffu, same);
    const int equals = same_at + __popc(sb & under);          // equal keys before this slot
    const int at = more_at + __popc(mb & under) + min(equals, left);
    if ((more || (same && equals < left)) && at < n) kept[at] = t;
    more_at += __popc(mb);
    same_at += __popc(sb);
  }
}

template <typename T, int HD>
__global__ void __launch_bounds__(256) evict_copy_kernel(const EvictArgs a) {
  constexpr int VEC = HD * sizeof(T) / 16;   // 16-byte vectors of a row
  pdl_wait();
  pdl_trigger();
  const int j0 = blockIdx.x * kBlk, g = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  int L, n;
  if (!evict_request(a, b, L, n, false)) return;
  if (j0 == 0 && g == 0 && tid == 0) {
    a.to.seq_len[b] = n;
    a.to.pending[b] = 0;
  }
  if (j0 >= n) return;
  const int blk = a.to.block_table[(long long)b * a.to.max_blocks + blockIdx.x];
  if (blk < 0 || blk >= a.to.num_blocks) {
    if (tid == 0) set_error(a.err, MTP_ERR_CAPACITY);
    return;
  }
  const long long tile = ((long long)blk * a.n_kv + g) * kBlk;
  const int32_t* kept = a.kept + ((long long)b * a.n_kv + g) * a.width;
  const long long extent = (long long)a.to.num_blocks * a.n_kv * kBlk * VEC;
  (void)extent;   // bounds-checked builds only
  for (int i = tid; i < kBlk * VEC; i += 256) {
    const int r = i / VEC, e = i - r * VEC, j = j0 + r;
    if (j >= n) break;
    const int slot = kept[j];
    const int src = a.from.block_table[(long long)b * a.from.max_blocks + (slot >> 4)];
    uint4 k = make_uint4(0, 0, 0, 0), v = k;
    float w = 0.0f;
    if (src >= 0 && src < a.from.num_blocks) {
      const long long at = ((long long)src * a.n_kv + g) * kBlk + (slot & 15);
      k = ld_stream((const uint4*)a.from.k_pool + at * VEC + e);
      v = ld_stream((const uint4*)a.from.v_pool + at * VEC + e);
      if (e == 0 && a.to_weights) w = a.weights[at];
    } else {
      set_error(a.err, MTP_ERR_CAPACITY);
    }
    if (!MTP_IN_BOUNDS(a.err, (tile + r) * VEC + e, extent)) continue;
    ((uint4*)a.to.k_pool)[(tile + r) * VEC + e] = k;
    ((uint4*)a.to.v_pool)[(tile + r) * VEC + e] = v;
    if (e == 0 && a.to_weights) a.to_weights[tile + r] = w;
  }
}

}  // namespace mtp

using namespace mtp;

extern "C" {

mtp_status mtp_kv_evict(mtp_ctx* ctx, void* stream, int B, const mtp_kv* from, const float* weights,
                        const int32_t* budget, int sink, int recent, const mtp_kv* to, float* to_weights,
                        int32_t* kept, int kept_width) {
  if (!ctx || B < 1 || B > ctx->cfg.max_batch || B > 65535 || !kv16_ok(from) || !kv16_ok(to) || !weights || !budget ||
      !kept || kept_width < 1 || sink < 0 || recent < 0)
    return MTP_ERR_INVALID;
  // the new cache's lengths are written while the old ones are read
  if (from->seq_len == to->seq_len || from->pending == to->pending || from->block_table == to->block_table)
    return MTP_ERR_INVALID;
  const mtp_config& c = ctx->cfg;
  const long long blocks = ((long long)kept_width + kBlk - 1) / kBlk;
  if (c.n_kv_heads > 65535) return MTP_ERR_INVALID;
  DeviceGuard dev(ctx->device);
  if (!dev.ok) return MTP_ERR_CUDA;
  EvictArgs a{};
  a.from = *from;
  a.to = *to;
  a.weights = weights;
  a.to_weights = to_weights;
  a.budget = budget;
  a.kept = kept;
  a.err = ctx->err;
  a.B = B;
  a.n_kv = c.n_kv_heads;
  a.hd = c.head_dim;
  a.sink = sink;
  a.recent = recent;
  a.width = kept_width;
  const long long most = (long long)from->max_blocks * kBlk;
  a.cached = (int)(most < 49152 ? most : 49152);
  cudaStream_t s = (cudaStream_t)stream;
  const size_t smem = (size_t)a.cached * 4;
  cudaError_t e = ensure_smem((const void*)evict_select_kernel, smem);
  if (e == cudaSuccess) e = launch_pdl(evict_select_kernel, dim3(c.n_kv_heads, B), dim3(kSelThreads), smem, s, a);
  const dim3 grid((unsigned)(blocks < to->max_blocks ? blocks : to->max_blocks), c.n_kv_heads, B), block(256);
  if (e == cudaSuccess) {
    if (c.head_dim == 128)
      e = c.dtype == MTP_DTYPE_BF16 ? launch_pdl(evict_copy_kernel<uint16_t, 128>, grid, block, 0, s, a)
                                    : launch_pdl(evict_copy_kernel<float, 128>, grid, block, 0, s, a);
    else
      e = c.dtype == MTP_DTYPE_BF16 ? launch_pdl(evict_copy_kernel<uint16_t, 64>, grid, block, 0, s, a)
                                    : launch_pdl(evict_copy_kernel<float, 64>, grid, block, 0, s, a);
  }
  ctx->launches += 2;
  return launch_status(e);
}

}  // extern "C"
