// Eviction from a paged cache by the attention weight that its entries have
// gathered: for each request and kv head the first `sink` entries, the last
// `recent` ones and, of those between, the ones with the largest weights stay,
// and move in their order to the blocks of another cache.
//
// Two kernels.  The first finds, per (request, kv head), the weight of the
// last entry that stays, digit by digit (11, 11 and 10 bits of the weights'
// ordered bit patterns, counted in shared memory; where few entries share the
// digits so far they are ranked among one another at once), and lists the slots
// that stay in ascending order; equal weights stay from the lowest slot on, so the
// result depends on nothing but the weights.  A cluster of up to four thread
// blocks shares a long context's slots and adds up their counts through
// distributed shared memory.  The second kernel copies: a thread block per
// (request, kv head, new cache block), 16 bytes a lane.
//
// The copy is bound by memory; the selection by its chain of steps, each a pass
// over a few entries a thread and a barrier.  Four requests of 16384 entries to
// 2048, 8 heads of 128: 27 us, 10 of them the copy's bytes; 24 short ones 11 us.
// Clusters and shared memory are sized by the table, whose width the host knows, and
// not by the lengths: a short request leaves blocks of its clusters without slots.
#include <cooperative_groups.h>

#include "mtp_kv16.cuh"
#include "mtp_kv_evict_range.h"

namespace mtp {

constexpr int kSelThreads = 1024;
constexpr int kSelBins = 2048;
constexpr int kSelFew = 512;      // entries that are ranked at once
constexpr int kSelCluster = 4;    // thread blocks of a cluster at most

struct EvictArgs {
  mtp_kv from, to;
  const float* weights;     // [from.num_blocks, n_kv, 16]
  float* to_weights;        // [to.num_blocks, n_kv, 16] or null
  const int32_t* budget;    // [B]
  int32_t* kept;            // [B, n_kv, width]
  int* err;
  int B, n_kv, hd, sink, recent, width;
  int cached;               // keys that the selection's shared memory holds, in fours
  int vec;                  // weights on 16 bytes
};

// A request's entries and how many stay; false (and the error) for one that
// is left out.
__device__ __forceinline__ bool evict_request(const EvictArgs& a, int b, int& L, int& n, bool report) {
  L = a.from.seq_len[b];
  const int budget = a.budget[b];
  int e = MTP_OK;
  if (L < 0 || a.from.pending[b] != 0 || budget < 0 || (long long)a.sink + a.recent > budget) e = MTP_ERR_DEVICE_ARGS;
  else if ((long long)L > (long long)a.from.max_blocks * kBlk || L > kKvMaxSlots) e = MTP_ERR_CAPACITY;
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

// Exclusive sum over the block of each thread's value.
__device__ __forceinline__ long long block_scan(long long v, long long* warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  long long y = lane < warp ? warps[lane] : 0;   // every warp adds up those before it
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) y += __shfl_xor_sync(0xffffffffu, y, d);
  return x - v + y;
}

// Cluster (kv head, request); its blocks share the slots (mtp_kv_evict_range.h).
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ int bins_s[3][kSelBins];                // this block's counts, a pass each
  __shared__ long long warps[4][kSelThreads / 32];   // a scan each
  __shared__ uint32_t few_s[kSelFew];                // this block's keys to rank
  __shared__ uint32_t few[kSelFew];                  // the cluster's
  __shared__ long long count_s;                      // this block's slots that stay, and equals
  __shared__ uint32_t digit_s;
  __shared__ int above_s, here_s, few_n;
  const cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), c = (int)cluster.block_rank();
  auto sync_all = [&]() {
    if (C > 1) cluster.sync();
    else __syncthreads();
  };
  pdl_wait();
  pdl_trigger();
  const int g = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int L, n;
  if (!evict_request(a, b, L, n, g == 0 && c == 0 && tid == 0)) return;   // (the whole cluster)
  int32_t* kept = a.kept + ((long long)b * a.n_kv + g) * a.width;
  for (int j = n + c * kSelThreads + tid; j < a.width; j += C * kSelThreads) kept[j] = -1;
  if (n == L) {
    for (int j = c * kSelThreads + tid; j < n; j += C * kSelThreads) kept[j] = j;
    return;
  }
  // candidates: the slots [lo, hi); `want` of them stay (budget - sink - recent >= 0)
  const int lo = a.sink, hi = L - a.recent, want = n - a.sink - a.recent;
  const EvictRange own = evict_range(L, a.sink, a.recent, C, c);   // a short request leaves blocks without slots
  const int s0 = own.s0, s1 = own.s1, c0 = own.c0, c1 = own.c1, f0 = own.f0;
  const int32_t* row = a.from.block_table + (long long)b * a.from.max_blocks;
  int lost = 0;
  // slots go in fours, which lie in one cache block
  auto load4 = [&](int t, uint32_t (&k)[4]) {
    const int blk = row[t >> 4];
    const bool good = blk >= 0 && blk < a.from.num_blocks;
    const float* p = a.weights + ((long long)(good ? blk : 0) * a.n_kv + g) * kBlk + (t & 12);
    float4 w;
    if (a.vec) w = *reinterpret_cast<const float4*>(p);
    else w = make_float4(p[0], p[1], p[2], p[3]);
    if (!good) lost = 1;
    if (!good) w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);   // (as its entries are copied)
    k[0] = weight_key(w.x);
    k[1] = weight_key(w.y);
    k[2] = weight_key(w.z);
    k[3] = weight_key(w.w);
  };
  auto keys4 = [&](int t, uint32_t (&k)[4]) {
    if (t - s0 < a.cached) {
      const uint4 u = *reinterpret_cast<const uint4*>(keys + (t - s0));
      k[0] = u.x; k[1] = u.y; k[2] = u.z; k[3] = u.w;
    } else {
      load4(t, k);
    }
  };
  auto key_of = [&](int t) -> uint32_t {
    if (t - s0 < a.cached) return keys[t - s0];
    uint32_t k[4];
    load4(t & ~3, k);
    return t & 2 ? (t & 1 ? k[3] : k[2]) : (t & 1 ? k[1] : k[0]);
  };
#pragma unroll 2
  for (int t = f0 + 4 * tid; t < min(c1, s0 + a.cached); t += 4 * kSelThreads) {
    uint32_t k[4];
    load4(t, k);
    *reinterpret_cast<uint4*>(keys + (t - s0)) = make_uint4(k[0], k[1], k[2], k[3]);
  }
  // ---- the key of the last candidate that stays, from its high digits down
  uint32_t prefix = 0;
  int left = want;             // how many of the keys that share the prefix stay
  int shift = 32;
  for (int pass = 0; want > 0 && pass < 3; ++pass) {
    int* bins = bins_s[pass];
    const int width = pass == 2 ? 10 : 11;
    const uint32_t high = shift == 32 ? 0u : ~0u << shift;   // the digits that are known
    shift -= width;
    for (int i = tid; i < kSelBins; i += kSelThreads) bins[i] = 0;
    if (tid == 0) few_n = 0;
    __syncthreads();
    // whole warps go round, so that one whose keys agree (no weight yet) adds once
    for (int t0 = f0 + warp * 128; t0 < c1; t0 += 4 * kSelThreads) {
      const int t = t0 + 4 * lane;
      uint32_t k[4] = {0u, 0u, 0u, 0u};
      if (t < c1) keys4(t, k);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool in = t + i >= c0 && t + i < c1 && (k[i] & high) == prefix;
        const uint32_t d = in ? (k[i] >> shift) & ((1u << width) - 1u) : 0xFFFFFFFFu;
        if (__all_sync(0xffffffffu, d == __shfl_sync(0xffffffffu, d, 0))) {
          if (in && lane == 0) atomicAdd(&bins[d], 32);
        } else if (in) {
          atomicAdd(&bins[d], 1);
        }
      }
    }
    sync_all();
    // thread i looks at digits 2 i and 2 i + 1 counted from the top, over the cluster
    const int top = kSelBins - 1 - 2 * tid;
    int n1 = 0, n0 = 0;
    int2 u[kSelCluster];        // (all on their way together: a remote load takes half a microsecond)
#pragma unroll
    for (int x = 0; x < kSelCluster; ++x)
      if (x < C) u[x] = *reinterpret_cast<const int2*>(cluster.map_shared_rank(bins, x) + top - 1);
#pragma unroll
    for (int x = 0; x < kSelCluster; ++x)
      if (x < C) {
        n0 += u[x].x;
        n1 += u[x].y;
      }
    const int before = (int)block_scan(n1 + n0, warps[pass]);   // keys with a larger digit
    if (before < left && before + n1 >= left) {
      digit_s = (uint32_t)top;
      above_s = before;
      here_s = n1;
    } else if (before + n1 < left && before + n1 + n0 >= left) {
      digit_s = (uint32_t)(top - 1);
      above_s = before + n1;
      here_s = n0;
    }
    __syncthreads();
    prefix |= digit_s << shift;
    left -= above_s;
    const int here = here_s;
    __syncthreads();
    if (shift == 0 || here > kSelFew) continue;
    // few keys share these digits: rank them
    const uint32_t known = ~0u << shift;
    for (int t = f0 + 4 * tid; t < c1; t += 4 * kSelThreads) {
      uint32_t k[4];
      keys4(t, k);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (t + i >= c0 && t + i < c1 && (k[i] & known) == prefix) few_s[atomicAdd(&few_n, 1)] = k[i];
    }
    sync_all();
    if (warp < C) {   // warp x fetches block x's
      int m = lane < C ? *cluster.map_shared_rank(&few_n, lane) : 0;
      int at = lane < warp ? m : 0;
#pragma unroll
      for (int d = 2; d > 0; d >>= 1) at += __shfl_xor_sync(0xffffffffu, at, d);
      at = __shfl_sync(0xffffffffu, at, 0);
      m = __shfl_sync(0xffffffffu, m, warp);
      const uint32_t* src = cluster.map_shared_rank(few_s, warp);
      for (int i = lane; i < m; i += 32) few[at + i] = src[i];
    }
    __syncthreads();
    if (tid < here) {
      const uint32_t mine = few[tid];
      int more = 0, same = 0;
#pragma unroll 4
      for (int i = 0; i < here; ++i) {
        const uint32_t k = few[i];
        more += k > mine;
        same += k == mine;
      }
      if (more < left && more + same >= left) {   // (all threads with this key write the same)
        digit_s = mine;
        above_s = more;
      }
    }
    __syncthreads();
    prefix = digit_s;
    left -= above_s;
    break;
  }
  // ---- list: a warp takes a contiguous share of the block's slots
  const int per = ((s1 - s0 + kSelThreads / 32 - 1) / (kSelThreads / 32) + 31) / 32 * 32;
  const int w0 = min(s1, s0 + warp * per), w1 = min(s1, w0 + per);
  int n_more = 0, n_same = 0;   // slots that stay anyway or lie above, and those that equal the last key
  auto classes = [&](int t, bool& more, bool& same) {
    const bool cand = t < w1 && t >= lo && t < hi;
    const uint32_t k = cand && want > 0 ? key_of(t) : 0u;
    more = t < w1 && (!cand || (want > 0 && k > prefix));
    same = cand && want > 0 && k == prefix;
  };
#pragma unroll 4
  for (int t0 = w0; t0 < w1; t0 += 32) {
    bool more, same;
    classes(t0 + lane, more, same);
    n_more += __popc(__ballot_sync(0xffffffffu, more));
    n_same += __popc(__ballot_sync(0xffffffffu, same));
  }
  const long long mine = lane == 0 ? (long long)n_same << 32 | n_more : 0;
  long long at0 = block_scan(mine, warps[3]);
  if (tid == kSelThreads - 32) count_s = at0 + mine;      // (the last warp's first lane: the block's total)
  sync_all();
  long long first = __shfl_sync(0xffffffffu, at0, 0);
  long long others = lane < c ? *cluster.map_shared_rank(&count_s, lane) : 0;
#pragma unroll
  for (int d = 2; d > 0; d >>= 1) others += __shfl_xor_sync(0xffffffffu, others, d);
  first += __shfl_sync(0xffffffffu, others, 0);
  int more_at = (int)(first & 0xFFFFFFFF), same_at = (int)(first >> 32);
  const uint32_t under = (1u << lane) - 1u;
#pragma unroll 2
  for (int t0 = w0; t0 < w1; t0 += 32) {
    bool more, same;
    classes(t0 + lane, more, same);
    const uint32_t mb = __ballot_sync(0xffffffffu, more), sb = __ballot_sync(0xffffffffu, same);
    const int equals = same_at + __popc(sb & under);          // equal keys before this slot
    const int at = more_at + __popc(mb & under) + min(equals, left);
    if ((more || (same && equals < left)) && at < n) kept[at] = t0 + lane;
    more_at += __popc(mb);
    same_at += __popc(sb);
  }
  if (lost) set_error(a.err, MTP_ERR_CAPACITY);
  if (C > 1) cluster.sync();   // no block leaves while another reads its shared memory
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
      !kept || kept_width < 1 || kept_width > kKvMaxSlots || sink < 0 || recent < 0)
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
  // blocks of a cluster: about 2048 slots each, as long as the grid fits the GPU.
  // Four requests of up to 16384 entries, 8 heads, selection and copy: 34, 30 and 27
  // us with one, two and four; eight wait for one another (51 us).
  const long long most = (long long)from->max_blocks * kBlk, heads = (long long)B * c.n_kv_heads;
  int C = 1;
  while (C < kSelCluster && most > 2048ll * C && heads * 2 * C <= ctx->num_sms) C *= 2;
  const long long part = evict_share(most, C) + 4;
  a.cached = (int)(part < 49152 ? part : 49152) & ~3;
  a.vec = !((uintptr_t)weights & 15);
  cudaStream_t s = (cudaStream_t)stream;
  const size_t smem = (size_t)a.cached * 4;
  cudaError_t e = ensure_smem((const void*)evict_select_kernel, smem);
  if (e == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(C, c.n_kv_heads, B);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a);
  }
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
