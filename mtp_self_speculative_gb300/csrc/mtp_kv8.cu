// The paged 8-bit KV cache: append with rotary and quantization, read-back,
// commit / rollback / truncate and the commit of a packed tree's path.
//
// A block of 16 tokens and one kv head share a scale s, a power of two with
// max|x| <= 448 s; an entry's value is code * s.  With a power of two the
// rescaling that a growing block needs is exact (only values that fall under
// the format's smallest normal number are rounded again), and every value is
// a bf16 number.
#include "mtp_kv8.cuh"

namespace mtp {

constexpr int kAppendThreads = 128;

// ------------------------------------------------------------------ append
struct Append8Args {
  const void* k;
  const void* v;
  const void* q;
  void* q_out;
  long long k_stride, v_stride, q_stride, q_out_stride;
  const int32_t* row_offsets;
  const int32_t* positions;
  mtp_kv8 kv;
  int* err;
  int B, T, n_kv, n_q;
  int rope;
};

// A unit is one cache block that takes new rows.  Request b's units start at
// floor(off_b / 16) + 2 b, which leaves it floor(n_b / 16) + 2 at least: as
// many as n_b rows can touch.
struct UnitFirst {
  __device__ int operator()(int o, int b) const { return (o >> 4) + 2 * b; }
};

template <typename T> __device__ __forceinline__ float get1(const T* p);
template <> __device__ __forceinline__ float get1<float>(const float* p) { return *p; }
template <> __device__ __forceinline__ float get1<uint16_t>(const uint16_t* p) {
  return __uint_as_float((uint32_t)*p << 16);
}

// One rotated element e of a head row (cs: the row's cosines and sines, or
// null for no rotation).
template <typename T>
__device__ __forceinline__ float rotated(const T* row, int e, const float2* cs, int rd, int layout) {
  const float x = get1<T>(row + e);
  if (!cs || e >= rd) return x;
  if (layout == MTP_ROPE_HALF) {
    const int h = rd >> 1;
    if (e < h) return x * cs[e].x - get1<T>(row + e + h) * cs[e].y;
    return x * cs[e - h].x + get1<T>(row + e - h) * cs[e - h].y;
  }
  const float2 c = cs[e >> 1];
  if (!(e & 1)) return x * c.x - get1<T>(row + e + 1) * c.y;
  return x * c.x + get1<T>(row + e - 1) * c.y;
}

template <typename T, int HD>
__global__ void __launch_bounds__(kAppendThreads) kv8_append_kernel(const Append8Args a,
                                                                    const __grid_constant__ mtp_rope_table tab) {
  constexpr int W = kAppendThreads / 32;
  constexpr int RPW = kBlk / W;          // rows of a block per warp
  constexpr int DPL = HD / 32;           // elements of a row per lane
  __shared__ float2 cs[kBlk][HD / 2];
  __shared__ float red[2][W];
  __shared__ int sh[3], live_blk[3];
  const int u = blockIdx.x, g = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (!find_request(a.row_offsets, a.B, a.T, u, a.err, sh, UnitFirst())) return;
  const int b = sh[0], o0 = sh[1], n_new = sh[2] - o0;
  if (tid == 0) {
    const int L0 = a.kv.seq_len[b], P = a.kv.pending[b];
    int bi = -1, blk = -1, start = 0;
    if (L0 < 0 || P < 0 || L0 > INT32_MAX - P) {
      set_error(a.err, MTP_ERR_DEVICE_ARGS);
    } else if ((long long)L0 + P + n_new > (long long)a.kv.max_blocks * kBlk) {
      set_error(a.err, MTP_ERR_CAPACITY);
    } else {
      start = L0 + P;
      const int first = start >> 4, last = (start + n_new - 1) >> 4;
      bi = first + (u - UnitFirst()(o0, b));
      if (bi > last) {
        bi = -1;
      } else {
        blk = a.kv.block_table[(long long)b * a.kv.max_blocks + bi];
        if (blk < 0 || blk >= a.kv.num_blocks) {
          set_error(a.err, MTP_ERR_CAPACITY);
          blk = -1;
        }
        // the last of the request's thread blocks publishes the new length:
        // all have read the old one by then
        if (arrive_last(a.kv.arrive + b, (last - first + 1) * a.n_kv)) a.kv.pending[b] = P + n_new;
      }
    }
    live_blk[0] = bi;
    live_blk[1] = blk;
    live_blk[2] = start;
  }
  __syncthreads();
  const int bi = live_blk[0], blk = live_blk[1], start = live_blk[2];
  if (bi < 0) return;
  const int s0 = max(start - bi * kBlk, 0);                  // first new slot within the block
  const int s1 = min(start + n_new - bi * kBlk, kBlk);       // one past the last
  const int r0 = o0 + bi * kBlk + s0 - start;                // input row of slot s0
  const int rd = a.rope ? tab.rotary_dim : 0, half = rd >> 1;
  for (int i = tid; i < (s1 - s0) * half; i += kAppendThreads) {
    const int r = i / half, p = i - r * half;
    cs[r][p] = rope_cos_sin(a.positions[r0 + r], tab.turns[p], tab.magnitude);
  }
  __syncthreads();
  if (blk >= 0) {
    float val[2][RPW][DPL];
    float amax[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < RPW; ++j) {
      const int s = warp + j * W;  // slot within the block
      if (s < s0 || s >= s1) continue;
      const int r = r0 + s - s0;
      const T* kr = (const T*)a.k + (long long)r * a.k_stride + g * HD;
      const T* vr = (const T*)a.v + (long long)r * a.v_stride + g * HD;
#pragma unroll
      for (int e = 0; e < DPL; ++e) {
        val[0][j][e] = rotated<T>(kr, lane * DPL + e, rd ? cs[s - s0] : nullptr, rd, tab.layout);
        val[1][j][e] = get1<T>(vr + lane * DPL + e);
#pragma unroll
        for (int w = 0; w < 2; ++w)
          if (finite_f(val[w][j][e])) amax[w] = fmaxf(amax[w], fabsf(val[w][j][e]));
      }
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const float m = warp_max(amax[w]);
      if (lane == 0) red[w][warp] = m;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < W; ++i) m = fmaxf(m, red[w][i]);
      float* scale = (w ? a.kv.v_scale : a.kv.k_scale) + (long long)blk * a.n_kv + g;
      uint8_t* tile = (uint8_t*)(w ? a.kv.v_pool : a.kv.k_pool) + ((long long)blk * a.n_kv + g) * (kBlk * HD);
      const float was = s0 > 0 ? *scale : 0.0f;
      const float need = e4m3_scale(m);
      const float now = fmaxf(was, need);
      const float inv = now > 0.0f ? 1.0f / now : 0.0f;
      // entries of a block whose scale grows
      if (was > 0.0f && now > was) {
        const float f = was * inv;
        for (int i = tid; i < s0 * (HD / 2); i += kAppendThreads) {
          uint16_t* p = (uint16_t*)tile + i;
          const float2 x = e4m3_to_float2(*p);
          *p = (uint16_t)e4m3_pack2(x.x * f, x.y * f);
        }
      }
#pragma unroll
      for (int j = 0; j < RPW; ++j) {
        const int s = warp + j * W;
        if (s < s0 || s >= s1) continue;
        uint16_t* p = (uint16_t*)(tile + s * HD + lane * DPL);
#pragma unroll
        for (int e = 0; e < DPL; e += 2)
          p[e / 2] = (uint16_t)e4m3_pack2(e4m3_in(val[w][j][e], inv), e4m3_in(val[w][j][e + 1], inv));
      }
      __syncthreads();  // all have read the old scale
      if (tid == 0) *scale = now;
    }
  }
  if (a.q) {
    const int G = a.n_q / a.n_kv;
    const int width = G * HD;
    for (int i = tid; i < (s1 - s0) * (width / 2); i += kAppendThreads) {
      const int r = i / (width / 2), p = i - r * (width / 2);
      const int h = p / (HD / 2), pe = p - h * (HD / 2);
      const T* x = (const T*)a.q + (long long)(r0 + r) * a.q_stride + (g * G + h) * HD;
      T* o = (T*)a.q_out + (long long)(r0 + r) * a.q_out_stride + (g * G + h) * HD;
      // pe < half: a rotated pair; then the rest, two at a time
      const int ia = pe < half ? (tab.layout == MTP_ROPE_HALF ? pe : 2 * pe) : 2 * pe;
      const int ib = pe < half && tab.layout == MTP_ROPE_HALF ? pe + half : ia + 1;
      const float xa = get1<T>(x + ia), xb = get1<T>(x + ib);
      if (pe < half) {
        const float2 c = cs[r][pe];
        Elem<T>::store1(o + ia, xa * c.x - xb * c.y);
        Elem<T>::store1(o + ib, xb * c.x + xa * c.y);
      } else if (x != o) {
        o[ia] = x[ia];
        o[ib] = x[ib];
      }
    }
  }
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

template <int HD>
__global__ void __launch_bounds__(128) kv8_read_kernel(const Read8Args a) {
  const int r = blockIdx.x;
  __shared__ int sh[3], at[2];
  if (!find_request(a.row_offsets, a.B, a.T, r, a.err, sh, [](int o, int) { return o; })) return;
  if (threadIdx.x == 0) {
    const int b = sh[0], s = a.start[b];
    const long long L = (long long)a.kv.seq_len[b] + a.kv.pending[b];
    int blk = -1, slot = 0;
    if (s < 0 || (long long)s + (sh[2] - sh[1]) > L) {
      set_error(a.err, MTP_ERR_DEVICE_ARGS);
    } else {
      slot = s + (r - sh[1]);
      const int bi = slot >> 4;
      blk = bi < a.kv.max_blocks ? a.kv.block_table[(long long)b * a.kv.max_blocks + bi] : -1;
      if (blk < 0 || blk >= a.kv.num_blocks) {
        set_error(a.err, MTP_ERR_CAPACITY);
        blk = -1;
      }
    }
    at[0] = blk;
    at[1] = slot & 15;
  }
  __syncthreads();
  const int blk = at[0], off = at[1];
  if (blk < 0) return;
  const int per = a.n_kv * (HD / 2);
  for (int i = threadIdx.x; i < 2 * per; i += blockDim.x) {
    const int w = i >= per;
    const int j = i - w * per, g = j / (HD / 2), e = j - g * (HD / 2);
    const long long tile = (long long)blk * a.n_kv + g;
    const uint16_t c = ((const uint16_t*)(w ? a.kv.v_pool : a.kv.k_pool))[(tile * kBlk + off) * (HD / 2) + e];
    const float s = (w ? a.kv.v_scale : a.kv.k_scale)[tile];
    const float2 x = e4m3_to_float2(c);
    ((uint32_t*)(w ? a.v_out : a.k_out))[((long long)r * a.n_kv + g) * (HD / 2) + e] =
        (uint32_t)f32_to_bf16_rne(x.x * s) | ((uint32_t)f32_to_bf16_rne(x.y * s) << 16);
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
// their blocks' scales.
__global__ void __launch_bounds__(kEditThreads) kv8_edit_kernel(const Edit8Args a) {
  extern __shared__ __align__(16) uint8_t kept[];   // path: [n][hd] codes
  __shared__ float kept_scale[kPathMax];
  __shared__ float red[kEditThreads / 32];
  __shared__ int sh[4];
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
    // the last head's block publishes the lengths; all have read them
    if (good && arrive_last(a.kv.arrive + b, a.n_kv)) {
      a.kv.seq_len[b] = nl;
      a.kv.pending[b] = 0;
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
        ((uint4*)kept)[i] = t >= 0 ? pool[(t * kBlk + (slot & 15)) * vec + e] : make_uint4(0, 0, 0, 0);
        if (e == 0) kept_scale[j] = t >= 0 ? scale[t] : 0.0f;
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
        if (t >= 0) {
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
        }
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
  a.row_offsets = row_offsets;
  a.positions = positions;
  a.kv = *kv;
  a.err = ctx->err;
  a.B = B;
  a.T = T;
  a.n_kv = c.n_kv_heads;
  a.n_q = c.n_q_heads;
  a.rope = rope != nullptr;
  mtp_rope_table tab = {};
  if (rope) tab = *rope;
  const dim3 grid(T / 16 + 2 * B, c.n_kv_heads);
  cudaStream_t s = (cudaStream_t)stream;
  const bool bf = c.dtype == MTP_DTYPE_BF16;
  if (c.head_dim == 128) {
    if (bf) kv8_append_kernel<uint16_t, 128><<<grid, kAppendThreads, 0, s>>>(a, tab);
    else kv8_append_kernel<float, 128><<<grid, kAppendThreads, 0, s>>>(a, tab);
  } else {
    if (bf) kv8_append_kernel<uint16_t, 64><<<grid, kAppendThreads, 0, s>>>(a, tab);
    else kv8_append_kernel<float, 64><<<grid, kAppendThreads, 0, s>>>(a, tab);
  }
  ctx->launches++;
  return launch_status(cudaGetLastError());
}

mtp_status mtp_kv8_read(mtp_ctx* ctx, void* stream, int B, const mtp_kv8* kv, const int32_t* start, int T,
                        const int32_t* row_offsets, void* k_out, void* v_out) {
  if (!ctx || B < 1 || B > ctx->cfg.max_batch || T < 0 || !start || !row_offsets || !k_out || !v_out || !kv8_ok(kv))
    return MTP_ERR_INVALID;
  if (T == 0) return MTP_OK;
  DeviceGuard dev(ctx->device);
  if (!dev.ok) return MTP_ERR_CUDA;
  Read8Args a{*kv, start, row_offsets, (uint16_t*)k_out, (uint16_t*)v_out, ctx->err, B, T, ctx->cfg.n_kv_heads};
  if (ctx->cfg.head_dim == 128) kv8_read_kernel<128><<<T, 128, 0, (cudaStream_t)stream>>>(a);
  else kv8_read_kernel<64><<<T, 128, 0, (cudaStream_t)stream>>>(a);
  ctx->launches++;
  return launch_status(cudaGetLastError());
}

static mtp_status kv8_edit(mtp_ctx* ctx, void* stream, int B, const mtp_kv8* kv, int mode, const int32_t* arg,
                           int extra, const int32_t* keep, int keep_stride) {
  if (!ctx || B < 1 || B > ctx->cfg.max_batch || B > 65535 || !kv8_ok(kv)) return MTP_ERR_INVALID;
  if (mode != KV_ROLLBACK && !arg) return MTP_ERR_INVALID;
  DeviceGuard dev(ctx->device);
  if (!dev.ok) return MTP_ERR_CUDA;
  Edit8Args a{*kv, arg, keep, ctx->err, keep_stride, mode, extra, ctx->cfg.n_kv_heads, ctx->cfg.head_dim};
  const size_t smem = keep ? (size_t)kPathMax * ctx->cfg.head_dim : 0;  // at most 32 KB
  kv8_edit_kernel<<<dim3(ctx->cfg.n_kv_heads, B), kEditThreads, smem, (cudaStream_t)stream>>>(a);
  ctx->launches++;
  return launch_status(cudaGetLastError());
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
