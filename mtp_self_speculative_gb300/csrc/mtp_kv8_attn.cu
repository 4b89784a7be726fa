// Attention of a request's new rows over its 8-bit cache (decode, draft
// verification, packed trees).
//
//   out[r, h] = sum_t p_t V[t, g] / sum_t p_t,  p_t = 2^(c s_t - m),
//   s_t = q[r, h] . K[t, g], c = scale * log2 e, m a running
// reference near the maximum.
//
// The (row, query head) pairs that share a kv head are the columns of a tile
// (n_b * G of them, 8 NT per tile); both products run on the tensor cores with
// the cache as the A operand, so that a single decoding row wastes half of an
// 8-wide tile at most:
//   S^T[16 tokens, 8 cols] = K[16, d] Q^T          m16n8k16, fp16 in, fp32 out
//   O^T[16 dims, 8 cols]  += V^T[16, 16 tokens] P^T
// e4m3 codes convert to fp16 exactly; the block scales multiply the float32
// accumulators.  Queries are scaled per column by a power of two into fp16's
// range (bf16 queries are then exact).  P is held relative to the reference, 2^8
// to 2^15 at its largest (1 for scores beyond 2^20), in 11 bits down to 2^-22
// (2^-14) of the largest and in steps of 2^-32 (2^-24) of it below: fp16 has more
// bits than bf16 at the same rate, and codes become fp16 exactly.  Float32
// heads split both Q and P into a high and a low half (22 bits) and issue each
// product twice.  The normalising sum takes the weights unrounded.  P^T comes out of the S^T accumulators with one movmatrix per
// 8 x 8; V is read 4 tokens x 16 dims per lane and its bytes are interleaved
// in registers, so no transposed copy of V exists anywhere.
//
// Work is split over the flattened sequence (request, kv head, tile, step of
// 16 or 32 tokens): every thread block takes an equal contiguous share, whatever
// the lengths are (they are only known on the device), so ragged batches and
// a single long context both fill the machine.  Each warp streams every
// fourth step of its block's share through its own ring of shared memory
// (cp.async, 16 bytes a lane, swizzled so that the fragment reads are free of
// bank conflicts).  A segment (request, kv head, tile) costs a start and an end
// besides its steps, so it counts kLead steps more.  Pieces of a segment
// that spans blocks meet in the workspace, and a second, small kernel joins
// them in a fixed order: the joining of a long context (a piece from every
// block) is spread over the machine, where the last block to arrive took 42 of
// 72 us of a call.
//
// Memory bounds decoding batches: 64 requests of up to 8192 entries (494 MB)
// 88-94 us, 5.3-5.6 TB/s; 128 of up to 4096 (542 MB) 95 us.  One request of
// 32768 entries takes 21 us, of which 4 are the join and as much the way to the
// first data.  Draft rows add products: 16 x 6 rows over up to 4096 entries 30.6
// us, at two warps per scheduler bound by the products' latencies.  Many rows
// are far from what the machine can do (8 x 61 rows 108 us, 169 TFLOP/s, floor
// about 10 us): each tile of at most 32 columns reads and converts the cache
// again.
#include <math.h>

#include "mtp_kv8.cuh"

namespace mtp {

constexpr int kA8Warps = 4;
constexpr int kA8Threads = kA8Warps * 32;
constexpr int kA8MaxB = 1024;      // requests of a call (prefix sums in shared memory)
constexpr int kA8MinShare = 16;    // cache blocks of a thread block's share at least
constexpr int kA8MaxCols = 32;     // columns of a tile
constexpr float kA8Least = -3.4028235e38f;   // the reference of a column that has seen nothing
constexpr float kA8Coarse = 16777216.0f;     // from 2^24 on float32 holds scores in steps of two and more

struct Attn8Args {
  const void* q;
  void* out;
  uint16_t* out_bf16;   // a bf16 copy of float32 results, or null
  float* lse;
  const int32_t* row_offsets;
  const int32_t* mask;
  mtp_kv8 kv;
  int* err;
  float* part;     // [2 * grid][32][HD + 4]: o, then reference and sum
  int4* meta;      // [2 * grid]: what the join kernel joins, per segment (by_segment) or per first block
  int by_segment, max_tiles, tile_cols;   // few segments: the join kernel has a block for each; tiles of max_rows rows
  long long q_stride;
  int B, T, max_rows, mask_words, n_kv, g_shift;
  float qscale;    // scale * log2(e)
  int q_vec;       // query rows allow four elements per load
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same onto zero.
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// 16 (or 4) bytes global -> shared; bytes = 0 fills zeros.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
  return r;
}
__device__ __forceinline__ float lds32f(uint32_t a) {
  float r;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(r) : "r"(a));
  return r;
}
// 2^x to 2^-22 of its value; results below 2^-126 are zero.
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t u) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
// One bit (0x80 of the byte) per NaN code of a word.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// Byte offset of 16-byte chunk c of token row r (0..31) within a staged K or
// V tile.  Rows of 128 (64) bytes; K: the two rows that eight lanes read
// together swap halves; V: the four rows that eight lanes read together are
// spread over the banks.
template <int HD>
__device__ __forceinline__ uint32_t k_at(int r, int c) {
  if constexpr (HD == 128) return (uint32_t)(r * 128 + ((c ^ ((r & 1) << 2)) << 4));
  return (uint32_t)(r * 64 + (c << 4));
}
template <int HD>
__device__ __forceinline__ uint32_t v_at(int r, int c) {
  if constexpr (HD == 128) return (uint32_t)(r * 128 + ((c ^ (r & 6)) << 4));
  return (uint32_t)((r >> 1) * 128 + ((((r & 1) * 4 + c) ^ (r & 6)) << 4));
}

// Four consecutive elements as loaded, in one load where the alignment allows
// it, and later as floats (so that nothing waits for the load before then).
template <typename T> struct Quad;
template <> struct Quad<float> {
  float4 w;
  __device__ __forceinline__ void zero() { w = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  __device__ __forceinline__ void load(const float* p, int vec) {
    if (vec) w = *reinterpret_cast<const float4*>(p);
    else w = make_float4(p[0], p[1], p[2], p[3]);
  }
  __device__ __forceinline__ void get(float (&x)[4]) const { x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w; }
};
template <> struct Quad<uint16_t> {
  uint2 w;
  __device__ __forceinline__ void zero() { w = make_uint2(0u, 0u); }
  __device__ __forceinline__ void load(const uint16_t* p, int vec) {
    if (vec) w = *reinterpret_cast<const uint2*>(p);
    else w = make_uint2((uint32_t)p[0] | ((uint32_t)p[1] << 16), (uint32_t)p[2] | ((uint32_t)p[3] << 16));
  }
  __device__ __forceinline__ void get(float (&x)[4]) const {
    x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
  }
};

template <int HD, int NT, int SPLIT>
struct Attn8Shape {
  // Cache blocks of a step.  Wide tiles have the registers for one (two spill
  // more at NT = 3 and 4: 16 x 6 rows 52.6 -> 50.1 us; with one, NT = 3 and 4
  // of 128-wide heads still spill 8 and 24 bytes in bf16, 20 and 68 in
  // float32); one column tile gains from the longer softmax step.
  static constexpr int JB = NT == 1 ? 2 : 1;
  static constexpr int kStep = kBlk * JB;                  // tokens of a step
  static constexpr int kTile = kStep * HD;                 // bytes of a staged K (or V) tile
  static constexpr int kStage = 2 * kTile + 16;            // K, V, the blocks' scales
  // units that a segment's start and end count for: its queries, the first
  // stages' latency, the join of the warps.  8, 16, 24, 32 blocks for each
  // (one 16 x 6 call: 49.9, 42.6, 38.1, 38.4 us; 8 x 61: 211, 167, 139, 127;
  // 48: 115), so it grows with the width.  One column tile counts 24: over
  // twelve ragged batches (24 - 100 requests of up to 4096 - 12288 entries) 24,
  // 32, 40 and 48 agree within 1 %, while a single batch moves by up to 8 %
  // either way with where its shares happen to be cut.
  static constexpr int kLead = (16 + 8 * NT) / JB, kMinShare = kA8MinShare / JB;
  static constexpr int kBlocks = SPLIT == 1 && NT == 1 ? 3 : 2;   // thread blocks per SM (registers)
  // Stages of a warp's ring.  Two of 32 tokens for three blocks per SM; four
  // of 16 tokens for two: six (what the shared memory would hold) make the
  // start longer and gain nothing (16 x 6 rows 31.3 against 30.0 us, one
  // request of 6 rows on 32768 entries 28.1 against 26.0 us; three: 30.6, 26.5).
  static constexpr int kStages = NT == 1 ? 2 : 4;
  static constexpr int kRing = kA8Warps * kStages * kStage;
  static constexpr int kCols = 8 * NT;
  static constexpr int kPitch = HD + 4;                    // floats of a merged row
  static constexpr int kMerge = kA8Warps * kCols * kPitch * 4;
  static constexpr int kMain = kRing > kMerge ? kRing : kMerge;
  static constexpr int kQ = NT * (HD / 16) * 32 * 8 * SPLIT;
  static constexpr int kBytes = kMain + kQ;
};

// Request b's first row, rows and entries; false if the call leaves it out.
// L2: read past this SM's first-level cache.
template <bool L2 = false>
__device__ __forceinline__ bool attn8_request(const Attn8Args& a, int b, int& o0, int& n, int& L) {
  auto get = [](const int32_t* p) -> int { return L2 ? __ldcg(p) : *p; };
  o0 = get(a.row_offsets + b);
  const int o1 = get(a.row_offsets + b + 1), sl = get(a.kv.seq_len + b), pe = get(a.kv.pending + b);
  n = o1 - o0;
  const long long len = (long long)sl + pe;
  L = (int)len;
  return o0 >= 0 && o1 <= a.T && n > 0 && n <= a.max_rows && sl >= 0 && pe >= 0 && len >= n &&
         len <= min((long long)a.kv.max_blocks * kBlk, 1ll << 30);
}

// Write four elements of a column's result and its lse.
template <typename T, int HD>
__device__ __forceinline__ void attn8_finish(const Attn8Args& a, int o0, int col, int g, int d4, float4 x, float ref,
                                             float sum) {
  const int G = 1 << a.g_shift;
  const long long row = (long long)(o0 + (col >> a.g_shift)) * (a.n_kv << a.g_shift) + (long long)g * G + (col & (G - 1));
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  if (!MTP_IN_BOUNDS(a.err, row * HD + d4 * 4 + 3, (long long)a.T * (a.n_kv << a.g_shift) * HD)) return;
  T* op = (T*)a.out + row * HD + d4 * 4;
  Elem<T>::store1(op, x.x * inv);
  Elem<T>::store1(op + 1, x.y * inv);
  Elem<T>::store1(op + 2, x.z * inv);
  Elem<T>::store1(op + 3, x.w * inv);
  if (sizeof(T) == 4 && a.out_bf16)
    *reinterpret_cast<uint2*>(a.out_bf16 + row * HD + d4 * 4) =
        make_uint2((uint32_t)f32_to_bf16_rne(x.x * inv) | ((uint32_t)f32_to_bf16_rne(x.y * inv) << 16),
                   (uint32_t)f32_to_bf16_rne(x.z * inv) | ((uint32_t)f32_to_bf16_rne(x.w * inv) << 16));
  if (a.lse && d4 == 0) a.lse[row] = sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * 0.69314718055994531f;
}

// Take a partial result (reference m, sum l, o) into another.
__device__ __forceinline__ void attn8_take(float& M, float& Ls, float4& x, float m, float l, const float4& y) {
  const float mn = fmaxf(M, m);
  const float f0 = ex2(M - mn), f1 = ex2(m - mn);
  Ls = Ls * f0 + l * f1;
  x.x = x.x * f0 + y.x * f1;
  x.y = x.y * f0 + y.y * f1;
  x.z = x.z * f0 + y.z * f1;
  x.w = x.w * f0 + y.w * f1;
  M = mn;
}

// SPLIT: halves of Q and P (2 keeps 22 bits; 1 is for results that bf16
// arithmetic goes on with).
template <typename T, int HD, int NT, int SPLIT>
__global__ void __launch_bounds__(kA8Threads, (Attn8Shape<HD, NT, SPLIT>::kBlocks)) kv8_attn_kernel(const Attn8Args a) {
  using S = Attn8Shape<HD, NT, SPLIT>;
  constexpr int KS = HD / 16;                 // k-steps of Q K^T
  constexpr int MT = HD / 16;                 // m-tiles of V^T P^T
  constexpr int STEP = S::kStep, JB = S::JB, PER = 32 / JB;   // PER: steps whose blocks a warp looks up at a time
  constexpr bool kQReg = NT * SPLIT <= 2;     // query fragments stay in registers
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int pre[kA8MaxB + 1];            // units before each request
  __shared__ long long wsum[kA8Warps];
  __shared__ int piece_s[4];
  __shared__ float qfac_s[S::kCols];
  __shared__ float wm[kA8Warps][S::kCols], wl[kA8Warps][S::kCols];

  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gi = lane >> 2, ti = lane & 3;
  const int G = 1 << a.g_shift;

  // ---- the call's work: units (steps) before each request
  long long carry = 0;
  int bad = 0;
  int my_o0 = 0, my_n = 0, my_len = 0;              // request tid of a batch of at most kA8Threads:
  uint32_t my_first = 0, my_units = 0;              // its rows, length and units
  for (int b0 = 0; b0 < a.B; b0 += kA8Threads) {
    const int b = b0 + tid;
    long long units = 0;
    if (b < a.B) {
      const int o0 = a.row_offsets[b], o1 = a.row_offsets[b + 1];
      if (o0 < 0 || o1 < o0 || o1 > a.T) {
        bad = 1;
      } else if (o1 > o0) {
        if (attn8_request(a, b, my_o0, my_n, my_len)) {
          const int tiles = (my_n * G + S::kCols - 1) / S::kCols;
          units = (long long)((my_len + STEP - 1) / STEP + S::kLead) * tiles * a.n_kv;
        } else if (blockIdx.x == 0) {
          set_error(a.err, my_n <= a.max_rows && (long long)a.kv.seq_len[b] + a.kv.pending[b] > (long long)a.kv.max_blocks * kBlk
                               ? MTP_ERR_CAPACITY : MTP_ERR_DEVICE_ARGS);
        }
      }
    }
    long long x = units;  // inclusive scan over the block
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    long long add = carry, all = 0;
#pragma unroll
    for (int w = 0; w < kA8Warps; ++w) {
      if (w < warp) add += wsum[w];
      all += wsum[w];
    }
    if (b < a.B) pre[b + 1] = (int)(add + x);
    my_first = (uint32_t)(add + x - units);
    my_units = (uint32_t)units;
    carry += all;
    __syncthreads();
  }
  if (tid == 0) {
    pre[0] = 0;
    if (!a.by_segment) a.meta[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
  }
  const bool refused = __syncthreads_or(bad);
  const long long total = carry;
  if (refused || total > INT32_MAX) {  // (or more steps than a call can count: 16 TB of cache read)
    if (tid == 0) {
      a.meta[2 * blockIdx.x] = make_int4(0, 0, 0, 0);   // nothing to join, whichever way it looks
      if (blockIdx.x == 0) set_error(a.err, refused ? MTP_ERR_DEVICE_ARGS : MTP_ERR_CAPACITY);
    }
    return;
  }
  // units fit 31 bits, so the divisions below are 32-bit ones
  const uint32_t units = (uint32_t)total, share = max((units + gridDim.x - 1) / gridDim.x, (uint32_t)S::kMinShare);
  uint32_t u = min((unsigned long long)blockIdx.x * share, (unsigned long long)units);
  const uint32_t u_end = min(units - u, share) + u;

  const uint32_t ring = smem_addr(smem) + warp * (S::kStages * S::kStage);
  float* merge = reinterpret_cast<float*>(smem);
  unsigned char* qf = smem + S::kMain;

  while (u < u_end) {
    // ---- the piece: request b, kv head g, tile, steps [s_lo, s_hi)
    int b, o0, n, L;
    if (a.B <= kA8Threads) {
      // the thread that holds the request says so
      if (u - my_first < my_units) {
        piece_s[0] = tid; piece_s[1] = my_o0; piece_s[2] = my_n; piece_s[3] = my_len;
      }
      __syncthreads();  // (the last piece's shared memory is free, too)
      b = piece_s[0]; o0 = piece_s[1]; n = piece_s[2]; L = piece_s[3];
    } else {
      int lo = 0, hi = a.B - 1;  // the request with pre[b] <= u < pre[b + 1]
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((uint32_t)pre[mid] <= u) lo = mid; else hi = mid - 1;
      }
      b = lo;
      attn8_request(a, b, o0, n, L);
      __syncthreads();
    }
    const int base = L - n;
    const int steps = (L + STEP - 1) / STEP, tiles = (n * G + S::kCols - 1) / S::kCols;
    const uint32_t seg = (u - (uint32_t)pre[b]) / (uint32_t)(steps + S::kLead);
    const int g = (int)(seg / (uint32_t)tiles), tile = (int)seg - g * tiles;
    const uint32_t seg_u0 = (uint32_t)pre[b] + seg * (uint32_t)(steps + S::kLead) + S::kLead;   // the segment's first step
    if (u_end <= seg_u0) break;   // the share ends before it
    const int s_lo = u > seg_u0 ? (int)(u - seg_u0) : 0, s_hi = min(steps, (int)(u_end - seg_u0));
    const int col0 = tile * S::kCols, ncols = min(S::kCols, n * G - col0);

    // the queries' loads go first: behind the first stages' they would wait
    // for all of those
    const bool lane_on = lane < HD / 4;
    Quad<T> xq[2 * NT];
#pragma unroll
    for (int k = 0; k < 2 * NT; ++k) {
      const int c = warp + kA8Warps * k, cc = col0 + c;
      xq[k].zero();
      if (c < ncols && lane_on)
        xq[k].load((const T*)a.q + (long long)(o0 + (cc >> a.g_shift)) * a.q_stride +
                       ((long long)g * G + (cc & (G - 1))) * HD + lane * 4,
                   a.q_vec);
    }
    // ---- this warp's steps: s_lo + warp, + 4, ...
    const int n_my = s_hi - s_lo > warp ? (s_hi - s_lo - warp + kA8Warps - 1) / kA8Warps : 0;
    const int32_t* trow = a.kv.block_table + (long long)b * a.kv.max_blocks;
    // table entries of PER steps at a time: lane JB i + j holds block j of step i
    auto load_table = [&](int batch) -> int {
      const int i = batch * PER + lane / JB;
      const int bi = JB * (s_lo + warp + kA8Warps * i) + lane % JB;
      int id = -1;
      if (i < n_my && (long long)bi * kBlk < L) {
        id = trow[bi];
        if (id < 0 || id >= a.kv.num_blocks) {
          set_error(a.err, MTP_ERR_CAPACITY);
          id = -1;
        }
      }
      return id;
    };
    int tbl = -1, tnext = load_table(0);
    auto issue = [&](int i) {
      if (i < n_my) {
        if (i % PER == 0) {
          tbl = tnext;
          tnext = load_table(i / PER + 1);
        }
        const int tok0 = (s_lo + warp + kA8Warps * i) * STEP;
        const uint32_t st = ring + (uint32_t)(i % S::kStages) * S::kStage;
#pragma unroll
        for (int j = 0; j < JB; ++j) {
          const int id = __shfl_sync(0xffffffffu, tbl, JB * (i % PER) + j);
          const long long t = (long long)max(id, 0) * a.n_kv + g;
          const unsigned char* kp = (const unsigned char*)a.kv.k_pool + t * (kBlk * HD);
          const unsigned char* vp = (const unsigned char*)a.kv.v_pool + t * (kBlk * HD);
#pragma unroll
          for (int x = 0; x < HD / 32; ++x) {
            const int idx = x * 32 + lane, r = idx / (HD / 16), c = idx % (HD / 16);
            const int bytes = id >= 0 && tok0 + 16 * j + r < L ? 16 : 0;
            cp16(st + k_at<HD>(16 * j + r, c), kp + idx * 16, bytes);
            cp16(st + S::kTile + v_at<HD>(16 * j + r, c), vp + idx * 16, bytes);
          }
          if (lane < 2) cp4(st + 2 * S::kTile + (lane * JB + j) * 4, (lane ? a.kv.v_scale : a.kv.k_scale) + t, id >= 0 ? 4 : 0);
        }
      }
      cp_commit();
    };
    // two stages now, the others once the queries are in place
    issue(0);
    if constexpr (S::kStages > 2) issue(1);

    // ---- queries: per column a power of two that brings them into fp16's
    // range, then fragments in the order the lanes read them
#pragma unroll
    for (int k = 0; k < 2 * NT; ++k) {
      const int c = warp + kA8Warps * k;
      float x[4];
      xq[k].get(x);
      float m = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
      m = warp_max(m);
      int sh = 0;  // largest element to [2^14, 2^15)
      if (m > 0.0f && finite_f(m)) sh = min(126, 141 - (int)(__float_as_uint(m) >> 23));
      const float up = __uint_as_float((uint32_t)(127 + sh) << 23);
      if (lane == 0) qfac_s[c] = a.qscale * (1.0f / up);
      if (lane_on) {
        // element d = 4 lane: half d / 64, lane group (d % 64) / 16, word (d % 16) / 4
        // (two words' fragments, 16 bytes, lie together)
        const int ks = (lane >> 4) * 4 + (lane & 3), fl = (c & 7) * 4 + ((lane & 15) >> 2);
        uint2 hi;
        hi.x = pack_half2(x[0] * up, x[1] * up);
        hi.y = pack_half2(x[2] * up, x[3] * up);
        uint2* dst = reinterpret_cast<uint2*>(qf) + ((c >> 3) * KS + (ks & ~1)) * 32 + fl * 2 + (ks & 1);
        *dst = hi;
        if constexpr (SPLIT == 2) {
          const float2 h0 = unpack_half2(hi.x), h1 = unpack_half2(hi.y);
          dst[NT * KS * 32] = make_uint2(pack_half2(x[0] * up - h0.x, x[1] * up - h0.y),
                                                 pack_half2(x[2] * up - h1.x, x[3] * up - h1.y));
        }
      }
    }
    __syncthreads();
    // fragments of k-steps 2 i and 2 i + 1
    auto q_frag = [&](int sp, int nt, int i) -> uint4 {
      return lds128(smem_addr(qf) + (uint32_t)(((sp * NT + nt) * KS + 2 * i) * 256 + lane * 16));
    };
    uint4 qreg[kQReg ? SPLIT : 1][kQReg ? NT : 1][kQReg ? KS / 2 : 1];
    if constexpr (kQReg) {
#pragma unroll
      for (int sp = 0; sp < SPLIT; ++sp)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < KS / 2; ++i) qreg[sp][nt][i] = q_frag(sp, nt, i);
    }
    float qfac[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      qfac[nt][0] = qfac_s[nt * 8 + 2 * ti];
      qfac[nt][1] = qfac_s[nt * 8 + 2 * ti + 1];
    }

#pragma unroll
    for (int i = 2; i < S::kStages - 1; ++i) issue(i);

    float o[NT][MT][4], m_run[NT][2], l_run[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.0f;
      m_run[nt][0] = m_run[nt][1] = kA8Least;
      l_run[nt][0] = l_run[nt][1] = 0.0f;
    }

    // whether column c (of the tile) sees token t >= base
    auto sees = [&](int c, int t) -> bool {
      const int i = (col0 + c) >> a.g_shift, j = t - base;
      if (i >= n || j >= n) return false;
      if (!a.mask) return j <= i;
      return (uint32_t)a.mask[(long long)(o0 + i) * a.mask_words + (j >> 5)] >> (j & 31) & 1u;
    };

    bool coarse = false;   // some column's reference is kA8Coarse or more (the same for the whole warp)
    for (int it = 0; it < n_my; ++it) {
      cp_wait<S::kStages - 2>();
      __syncwarp();
      issue(it + S::kStages - 1);
      const uint32_t st = ring + (uint32_t)(it % S::kStages) * S::kStage;
      const int tok0 = (s_lo + warp + kA8Warps * it) * STEP;
      const bool edge = tok0 + STEP > base;   // some tokens are not seen by every column
      // ---- scores
      float sc[JB][NT][4];
#pragma unroll
      for (int j = 0; j < JB; ++j) {
#pragma unroll
        for (int hh = 0; hh < HD / 64; ++hh) {
          const uint4 lo = lds128(st + k_at<HD>(16 * j + gi, hh * 4 + ti));
          const uint4 hi = lds128(st + k_at<HD>(16 * j + gi + 8, hh * 4 + ti));
          const uint32_t lw[4] = {lo.x, lo.y, lo.z, lo.w}, hw[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
          for (int w = 0; w < 4; w += 2) {
            uint32_t f[2][4];   // the A fragments of two k-steps
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              e4m3_unpack4(lw[w + x], f[x][0], f[x][2]);
              e4m3_unpack4(hw[w + x], f[x][1], f[x][3]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int sp = 0; sp < SPLIT; ++sp) {
                uint4 qq;
                if constexpr (kQReg) qq = qreg[sp][nt][hh * 2 + w / 2];
                else qq = q_frag(sp, nt, hh * 2 + w / 2);
                if (hh == 0 && w == 0 && sp == 0) mma_f16_zero(sc[j][nt], f[0][0], f[0][1], f[0][2], f[0][3], qq.x, qq.y);
                else mma_f16(sc[j][nt], f[0][0], f[0][1], f[0][2], f[0][3], qq.x, qq.y);
                mma_f16(sc[j][nt], f[1][0], f[1][1], f[1][2], f[1][3], qq.z, qq.w);
              }
          }
        }
      }
      // ---- online softmax over the step's tokens
      float kscale[JB], vscale[JB];
#pragma unroll
      for (int j = 0; j < JB; ++j) {
        kscale[j] = lds32f(st + 2 * S::kTile + 4 * j);
        vscale[j] = lds32f(st + 2 * S::kTile + 4 * (JB + j));
      }
      // Weights are 2^(s - r).  The reference r of a column stays while every
      // score is at most r + 15 (fp16 holds 2^15.9), so most steps need no
      // maximum across the lanes and no rescaling.  When one is above, r
      // becomes 9 below the maximum, a whole number: fp16 then keeps 11 bits
      // of weights down to 2^-22 of the largest.  (Beyond 2^20 that sum would
      // round, and r is the maximum itself.)  That maximum is a product rounded
      // to float32, up to half a step off: from kA8Coarse on the scores are
      // rounded like it before r is taken off, and r follows every maximum;
      // else the largest weights would be 2^8, 2^16, .. and pass fp16's range.
      float fac[JB][NT][2];
      bool above = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int j = 0; j < JB; ++j) {
            // a zero scale stands for zero entries: a factor above zero keeps
            // -inf * f from becoming NaN
            const float f = fmaxf(kscale[j] * qfac[nt][e], 1e-37f);
            fac[j][nt][e] = f;
            if (edge) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int t = tok0 + 16 * j + 8 * h + gi;
                if (t >= L || (t >= base && !sees(nt * 8 + 2 * ti + e, t))) sc[j][nt][2 * h + e] = -INFINITY;
              }
            }
            above |= fmaf(fmaxf(sc[j][nt][e], sc[j][nt][2 + e]), f, -m_run[nt][e]) > 15.0f;
          }
      if (__any_sync(0xffffffffu, above) || coarse) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float alpha[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(sc[0][nt][e], sc[0][nt][2 + e]) * fac[0][nt][e];
            if constexpr (JB == 2) mx = fmaxf(mx, fmaxf(sc[JB - 1][nt][e], sc[JB - 1][nt][2 + e]) * fac[JB - 1][nt][e]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float ref = fabsf(mx) > 1048576.0f ? mx : ceilf(mx) - 9.0f;
            const float rn = fmaxf(m_run[nt][e], ref);
            alpha[e] = ex2(m_run[nt][e] - rn);
            m_run[nt][e] = rn;
            l_run[nt][e] *= alpha[e];
            coarse |= fabsf(rn) >= kA8Coarse && rn != kA8Least;
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            o[nt][mt][0] *= alpha[0];
            o[nt][mt][1] *= alpha[1];
            o[nt][mt][2] *= alpha[0];
            o[nt][mt][3] *= alpha[1];
          }
        }
        coarse = __any_sync(0xffffffffu, coarse);
        if (coarse) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (fabsf(m_run[nt][e]) >= kA8Coarse) {
#pragma unroll
                for (int j = 0; j < JB; ++j) {
                  sc[j][nt][e] = __fmul_rn(sc[j][nt][e], fac[j][nt][e]);
                  sc[j][nt][2 + e] = __fmul_rn(sc[j][nt][2 + e], fac[j][nt][e]);
                  fac[j][nt][e] = 1.0f;
                }
              }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int j = 0; j < JB; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float p = ex2(fmaf(sc[j][nt][2 * h + e], fac[j][nt][e], -m_run[nt][e]));
              sc[j][nt][2 * h + e] = p;
              l_run[nt][e] += p;
            }
      // ---- values
#pragma unroll
      for (int j = 0; j < JB; ++j) {
        uint32_t pb[SPLIT][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t h0 = pack_half2(sc[j][nt][0], sc[j][nt][1]), h1 = pack_half2(sc[j][nt][2], sc[j][nt][3]);
          pb[0][nt][0] = movmatrix(h0);
          pb[0][nt][1] = movmatrix(h1);
          if constexpr (SPLIT == 2) {
            const float2 f0 = unpack_half2(h0), f1 = unpack_half2(h1);
            pb[1][nt][0] = movmatrix(pack_half2(sc[j][nt][0] - f0.x, sc[j][nt][1] - f0.y));
            pb[1][nt][1] = movmatrix(pack_half2(sc[j][nt][2] - f1.x, sc[j][nt][3] - f1.y));
          }
        }
        // tokens 2 ti, 2 ti + 1, 2 ti + 8, 2 ti + 9; dims (HD / 8) gi ..
        constexpr int WD = HD / 32;  // words of a token per lane
        uint32_t v[4][WD];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int r = 16 * j + 2 * ti + (x & 1) + (x >> 1) * 8;
          if constexpr (HD == 128) {
            const uint4 y = lds128(st + S::kTile + v_at<HD>(r, gi));
            v[x][0] = y.x; v[x][1] = y.y; v[x][2] = y.z; v[x][3] = y.w;
          } else {
            const uint2 y = lds64(st + S::kTile + v_at<HD>(r, gi >> 1) + (gi & 1) * 8);
            v[x][0] = y.x; v[x][1] = y.y;
          }
        }
        if (edge) {
          // a NaN entry must not reach columns that do not see it through
          // 0 * NaN: take it out of the product and put it in by hand
          uint32_t any = 0;
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int w = 0; w < WD; ++w) {
              const uint32_t nb = nan_bytes(v[x][w]);
              any |= nb;
              v[x][w] &= ~((nb >> 7) * 0xFFu);
            }
          if (__any_sync(0xffffffffu, any != 0)) {
            for (int t = 0; t < 16; ++t) {
              uint32_t nb[WD];
#pragma unroll
              for (int w = 0; w < WD; ++w) {
                uint32_t y;
                const uint32_t at = st + S::kTile + (HD == 128 ? v_at<HD>(16 * j + t, gi) : v_at<HD>(16 * j + t, gi >> 1) + (gi & 1) * 8);
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(y) : "r"(at + 4 * w));
                nb[w] = nan_bytes(y);
              }
              const int tok = tok0 + 16 * j + t;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  if (!(tok < L && (tok < base || sees(nt * 8 + 2 * ti + e, tok)))) continue;
#pragma unroll
                  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                      if (nb[mt >> 1] >> (8 * (2 * (mt & 1) + h)) & 0x80u)
                        o[nt][mt][2 * h + e] = __uint_as_float(0x7FC00000u);
                }
            }
          }
        }
        const float vs = vscale[j];
#pragma unroll
        for (int w = 0; w < WD; ++w) {
          const uint32_t p01 = __byte_perm(v[0][w], v[1][w], 0x5140), q01 = __byte_perm(v[0][w], v[1][w], 0x7362);
          const uint32_t p23 = __byte_perm(v[2][w], v[3][w], 0x5140), q23 = __byte_perm(v[2][w], v[3][w], 0x7362);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int mt = 2 * w + h;
            const uint32_t x01 = h ? q01 : p01, x23 = h ? q23 : p23;
            uint32_t a0, a1, a2, a3;
            e4m3_unpack4(x01, a0, a1);
            e4m3_unpack4(x23, a2, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float pv[4];
              mma_f16_zero(pv, a0, a1, a2, a3, pb[0][nt][0], pb[0][nt][1]);
              if constexpr (SPLIT == 2) mma_f16(pv, a0, a1, a2, a3, pb[SPLIT - 1][nt][0], pb[SPLIT - 1][nt][1]);
#pragma unroll
              for (int e = 0; e < 4; ++e) o[nt][mt][e] = fmaf(pv[e], vs, o[nt][mt][e]);
            }
          }
        }
      }
    }

    // ---- join the warps: the ring becomes [warp][column][HD + 4]
    cp_wait<0>();
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = l_run[nt][e];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        const int c = nt * 8 + 2 * ti + e;
        if (gi == 0) {
          wm[warp][c] = m_run[nt][e];
          wl[warp][c] = l;
        }
        float* row = merge + (warp * S::kCols + c) * S::kPitch + gi * (HD / 8);
#pragma unroll
        for (int mt = 0; mt < MT; mt += 2)
          *reinterpret_cast<float4*>(row + 2 * mt) =
              make_float4(o[nt][mt][e], o[nt][mt][2 + e], o[nt][mt + 1][e], o[nt][mt + 1][2 + e]);
      }
    __syncthreads();
    const uint32_t c_first = seg_u0 / share, c_last = (seg_u0 + (uint32_t)steps - 1) / share;
    const bool whole = c_first == c_last;
    const int slot = blockIdx.x == c_first ? 1 : 0;
#pragma unroll 2
    for (int i = tid; i < ncols * (HD / 4); i += kA8Threads) {
      const int c = i / (HD / 4), d4 = i - c * (HD / 4);
      float M = kA8Least;
#pragma unroll
      for (int w = 0; w < kA8Warps; ++w) M = fmaxf(M, wm[w][c]);
      float Ls = 0.0f;
      float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kA8Warps; ++w) {
        const float f = ex2(wm[w][c] - M);
        const float4 y = *reinterpret_cast<const float4*>(merge + (w * S::kCols + c) * S::kPitch + d4 * 4);
        Ls += wl[w][c] * f;
        x.x = fmaf(y.x, f, x.x);
        x.y = fmaf(y.y, f, x.y);
        x.z = fmaf(y.z, f, x.z);
        x.w = fmaf(y.w, f, x.w);
      }
      if (whole) {
        attn8_finish<T, HD>(a, o0, col0 + c, g, d4, x, M, Ls);
      } else {
        const long long at = ((2ll * blockIdx.x + slot) * kA8MaxCols + c) * (HD + 4);
        if (!MTP_IN_BOUNDS(a.err, at + HD + 1, 2ll * gridDim.x * kA8MaxCols * (HD + 4))) continue;
        float* pr = a.part + at;
        *reinterpret_cast<float4*>(pr + d4 * 4) = x;
        if (d4 == 0) *reinterpret_cast<float2*>(pr + HD) = make_float2(M, Ls);
      }
    }
    if (tid == 0 && slot == 1 && (a.by_segment || !whole)) {
      int4* m = a.meta + 2 * (a.by_segment ? (b * a.n_kv + g) * a.max_tiles + tile : (int)blockIdx.x);
      m[0] = make_int4(whole ? 0 : (int)(c_last - c_first + 1), (int)c_first, ncols, g);
      m[1] = make_int4(o0, col0, 0, 0);
    }
    u = seg_u0 + (uint32_t)s_hi;
  }
}

// Joins the pieces of segments that span thread blocks.  Where a call has
// fewer segments than the first kernel has blocks, block x takes segment x;
// else the one that begins in the first kernel's block x.  A thread owns four
// elements of a column, or shares them with `ways - 1` others where there are
// many pieces; block (x, y) takes the y-th group of columns and every
// gridDim.y-th after it.
constexpr int kJoinThreads = 256;
constexpr int kJoinAhead = 4;   // pieces in flight per thread
// Threads that share an element's pieces.
__host__ __device__ __forceinline__ int join_ways(int count) {
  return count <= kJoinAhead ? 1 : count <= 2 * kJoinAhead ? 2 : count <= 4 * kJoinAhead ? 4 : 8;
}

template <typename T, int HD>
__global__ void __launch_bounds__(kJoinThreads) kv8_attn_join_kernel(const Attn8Args a) {
  __shared__ float4 xs[kJoinThreads];
  __shared__ float2 ms[kJoinThreads];
  if (a.by_segment) {
    // A request that the call leaves out has written nothing.  Its rows and
    // lengths do not change during the call, and what wrote them had ended when
    // the first kernel let this one start; that may be before this kernel's wait,
    // so they are read from the second-level cache.  (Behind the wait: 0.3 to
    // 0.9 us more a call.)
    const int b = blockIdx.x / (a.n_kv * a.max_tiles), tile = blockIdx.x % a.max_tiles;
    int o0, n, L;
    if (!attn8_request<true>(a, b, o0, n, L) || tile * a.tile_cols >= n << a.g_shift) {
      pdl_wait();   // this kernel must not end before the first one
      return;
    }
  }
  pdl_wait();
  pdl_trigger();
  const int4 seg = a.meta[2 * blockIdx.x], at = a.meta[2 * blockIdx.x + 1];
  const int count = seg.x, c_first = seg.y, ncols = seg.z;
  if (count == 0) return;
  const int ways = join_ways(count);
  static_assert(kJoinThreads / 8 >= HD / 4, "a block must hold a column at least, or the loop below stands still");
  const int items = kJoinThreads / ways, cols = items / (HD / 4);
  const int item = threadIdx.x % items, way = threadIdx.x / items;
  const int d4 = item % (HD / 4);
  for (int c0 = cols * blockIdx.y; c0 < ncols; c0 += cols * gridDim.y) {
    const int c = c0 + item / (HD / 4);
    float M = kA8Least, Ls = 0.0f;
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c < ncols) {
      for (int k0 = way; k0 < count; k0 += kJoinAhead * ways) {
        float2 ml[kJoinAhead];
        float4 y[kJoinAhead];
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k) {   // no branches: all loads go out together
          const int kk = min(k0 + k * ways, count - 1);
          const float* pr = a.part + ((2ll * (c_first + kk) + (kk == 0 ? 1 : 0)) * kA8MaxCols + c) * (HD + 4);
          ml[k] = __ldcg(reinterpret_cast<const float2*>(pr + HD));
          y[k] = __ldcg(reinterpret_cast<const float4*>(pr) + d4);
        }
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k)
          if (k0 + k * ways >= count) {
            ml[k] = make_float2(kA8Least, 0.0f);
            y[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          }
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k) attn8_take(M, Ls, x, ml[k].x, ml[k].y, y[k]);
      }
    }
    if (ways > 1) {
      __syncthreads();
      xs[threadIdx.x] = x;
      ms[threadIdx.x] = make_float2(M, Ls);
      __syncthreads();
      for (int w = 1; way == 0 && w < ways; ++w)
        attn8_take(M, Ls, x, ms[w * items + item].x, ms[w * items + item].y, xs[w * items + item]);
    }
    if (way == 0 && c < ncols) attn8_finish<T, HD>(a, at.x, at.y + c, seg.w, d4, x, M, Ls);
  }
}

// Blocks per SM of the widest grid: the workspace serves every tile width.
constexpr int kA8MaxBlocks = 3;
static size_t a8_meta_bytes(const mtp_ctx* ctx) { return (size_t)kA8MaxBlocks * ctx->num_sms * 2 * sizeof(int4); }

template <typename T, int HD, int NT, int SPLIT = sizeof(T) == 4 ? 2 : 1>
static cudaError_t attn8_launch(mtp_ctx* ctx, cudaStream_t s, Attn8Args a) {
  using S = Attn8Shape<HD, NT, SPLIT>;
  static_assert(S::kBlocks <= kA8MaxBlocks, "workspace");
  cudaError_t e = ensure_smem((const void*)kv8_attn_kernel<T, HD, NT, SPLIT>, S::kBytes);
  if (e != cudaSuccess) return e;
  const int grid = S::kBlocks * ctx->num_sms;
  const int cols = a.max_rows << a.g_shift;   // of the longest request
  a.tile_cols = S::kCols;
  a.max_tiles = (cols + S::kCols - 1) / S::kCols;
  const long long segments = (long long)a.B * a.n_kv * a.max_tiles;
  a.by_segment = segments <= grid;
  e = launch_pdl(kv8_attn_kernel<T, HD, NT, SPLIT>, dim3(grid), dim3(kA8Threads), S::kBytes, s, a);
  if (e != cudaSuccess) return e;
  // columns that a block joins at a time, for twice the average of pieces
  const int even = kJoinThreads / join_ways((int)(2 * grid / segments + 1)) / (HD / 4), per = even > 1 ? even : 1;
  const int gy = ((cols < S::kCols ? cols : S::kCols) + per - 1) / per;
  return launch_pdl(kv8_attn_join_kernel<T, HD>, dim3(a.by_segment ? (unsigned)segments : (unsigned)grid, gy),
                    dim3(kJoinThreads), 0, s, a);
}

template <typename T, int HD>
static cudaError_t attn8_pick(mtp_ctx* ctx, cudaStream_t s, const Attn8Args& a, int nt) {
  switch (nt) {
    case 1: return attn8_launch<T, HD, 1>(ctx, s, a);
    case 2: return attn8_launch<T, HD, 2>(ctx, s, a);
    case 3: return attn8_launch<T, HD, 3>(ctx, s, a);
    default: return attn8_launch<T, HD, 4>(ctx, s, a);
  }
}

// Fills in what follows from the context and the queries.
static void attn8_fill(const mtp_ctx* ctx, Attn8Args& a, size_t q_bytes, float scale) {
  const mtp_config& c = ctx->cfg;
  a.n_kv = c.n_kv_heads;
  const int G = c.n_q_heads / c.n_kv_heads;
  for (a.g_shift = 0; (1 << a.g_shift) < G; ++a.g_shift) {
  }
  a.qscale = scale * 1.4426950408889634f;
  a.q_vec = (uintptr_t)a.q % (4 * q_bytes) == 0 && a.q_stride % 4 == 0;
}

// --------------------------------------------- draft steps on an 8-bit cache
//
// The draft step's projection kernels write a step's key and value rows where
// they are told the cache is.  For an 8-bit cache that is a staging area of
// the call's workspace (a cache of max_k slots a request that starts empty);
// the kernel below quantizes the step's row into the request's real slot, and
// the attention above runs on the context's float32 queries.
struct Kv8Draft {
  mtp_kv8 kv;
  mtp_kv stage;
  const int32_t* positions;
  const int32_t* row_offsets;   // 0, 1, .. B
  void* attn_ws;
};

__global__ void __launch_bounds__(128) kv8_stage_kernel(int B, int blocks, int32_t* table, int32_t* seq_len,
                                                        int32_t* pending, int32_t* offsets,
                                                        const int32_t* kv_pending) {
  pdl_wait();
  pdl_trigger();
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i <= B; i += gridDim.x * blockDim.x) {
    offsets[i] = i;
    if (i == B) break;
    for (int j = 0; j < blocks; ++j) table[i * blocks + j] = i * blocks + j;
    seq_len[i] = 0;
    // a request with pending entries is refused by the first step's check
    pending[i] = kv_pending[i] != 0;
  }
}

// Thread block (kv head, request): warp 0 the key, warp 1 the value row of
// step k.  At a position outside the rotary table the projections write no
// staged row (its bytes are the workspace's), so the entry stays zero bits and
// the block's scale as it is; the request counts it as pending all the same,
// as on a 16-bit cache.
template <typename T, int HD>
__global__ void __launch_bounds__(64) kv8_stage_append_kernel(mtp_kv8 kv, mtp_kv stage, const int* req_bad, int* err,
                                                              const int32_t* positions, int max_pos, int n_kv, int k) {
  constexpr int DPL = HD / 32;
  pdl_wait();
  pdl_trigger();
  const int g = blockIdx.x, b = blockIdx.y, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (__ldcg(req_bad + b)) return;
  const long long slot = (long long)kv.seq_len[b] + k - 1;
  if (slot < k - 1 || slot >= (long long)kv.max_blocks * kBlk) {
    if (threadIdx.x == 0) set_error(err, slot < k - 1 ? MTP_ERR_DEVICE_ARGS : MTP_ERR_CAPACITY);
    return;
  }
  if (g == 0 && threadIdx.x == 0) kv.pending[b] = k;
  const long long pos = (long long)positions[b] + k - 1;
  if (pos < 0 || pos >= max_pos) {
    if (threadIdx.x == 0) set_error(err, MTP_ERR_CAPACITY);
    return;
  }
  const int blk = kv.block_table[(long long)b * kv.max_blocks + (slot >> 4)], off = (int)(slot & 15);
  if (blk < 0 || blk >= kv.num_blocks) {
    if (threadIdx.x == 0) set_error(err, MTP_ERR_CAPACITY);
    return;
  }
  const long long st = ((long long)b * stage.max_blocks + ((k - 1) >> 4)) * n_kv + g;
  const T* src = (const T*)(w ? stage.v_pool : stage.k_pool) + (st * kBlk + ((k - 1) & 15)) * HD + lane * DPL;
  float x[DPL], amax = 0.0f;
#pragma unroll
  for (int e = 0; e < DPL; ++e) {
    x[e] = Elem<T>::loads(src + e);
    if (finite_f(x[e])) amax = fmaxf(amax, fabsf(x[e]));
  }
  const long long t = (long long)blk * n_kv + g;
  float* scale = (w ? kv.v_scale : kv.k_scale) + t;
  uint8_t* tile = (uint8_t*)(w ? kv.v_pool : kv.k_pool) + t * (kBlk * HD);
  const float was = off > 0 ? *scale : 0.0f, now = fmaxf(was, e4m3_scale(warp_max(amax)));
  const float inv = now > 0.0f ? 1.0f / now : 0.0f;
  if (was > 0.0f && now > was) {
    for (int i = lane; i < off * (HD / 2); i += 32) {
      uint16_t* p = (uint16_t*)tile + i;
      const float2 y = e4m3_to_float2(*p);
      *p = (uint16_t)e4m3_pack2(y.x * (was * inv), y.y * (was * inv));
    }
  }
  if (!MTP_IN_BOUNDS(err, t * (kBlk * HD) + off * HD + HD - 1, (long long)kv.num_blocks * n_kv * kBlk * HD)) return;
#pragma unroll
  for (int e = 0; e < DPL; e += 2)
    *(uint16_t*)(tile + off * HD + lane * DPL + e) = (uint16_t)e4m3_pack2(e4m3_in(x[e], inv), e4m3_in(x[e + 1], inv));
  __syncwarp();   // all lanes have read the old scale
  if (lane == 0) *scale = now;
}

cudaError_t launch_attention_kv8(mtp_ctx* ctx, cudaStream_t s, int B, int k) {
  const Kv8Draft& d = *(const Kv8Draft*)ctx->kv8_draft;
  const mtp_config& c = ctx->cfg;
  const dim3 grid(c.n_kv_heads, B), block(64);
  const bool bf = c.dtype == MTP_DTYPE_BF16;
  const int* req_bad = ctx->req_bad;
  auto append = [&](auto kernel) {
    return launch_pdl(kernel, grid, block, 0, s, d.kv, d.stage, req_bad, ctx->err, d.positions, c.max_pos, c.n_kv_heads, k);
  };
  cudaError_t e = c.head_dim == 128 ? (bf ? append(kv8_stage_append_kernel<uint16_t, 128>) : append(kv8_stage_append_kernel<float, 128>))
                                    : (bf ? append(kv8_stage_append_kernel<uint16_t, 64>) : append(kv8_stage_append_kernel<float, 64>));
  if (e != cudaSuccess) return e;
  Attn8Args a{};
  a.q = ctx->q;
  a.out = ctx->attn;
  a.out_bf16 = tc_supported(ctx, B) ? ctx->tc_attn : nullptr;
  a.row_offsets = d.row_offsets;
  a.kv = d.kv;
  a.err = ctx->err;
  a.meta = (int4*)d.attn_ws;
  a.part = (float*)((char*)d.attn_ws + a8_meta_bytes(ctx));
  a.q_stride = ctx->q_dim;
  a.B = B;
  a.T = B;
  a.max_rows = 1;
  ctx->launches += 3;
  attn8_fill(ctx, a, 4, 1.0f / sqrtf((float)c.head_dim));
  // one row: at most 8 columns.  A bf16 head's next projection takes bf16, so
  // its queries and weights need no second half.
  if (bf) return c.head_dim == 128 ? attn8_launch<float, 128, 1, 1>(ctx, s, a) : attn8_launch<float, 64, 1, 1>(ctx, s, a);
  return c.head_dim == 128 ? attn8_launch<float, 128, 1>(ctx, s, a) : attn8_launch<float, 64, 1>(ctx, s, a);
}

// Workspace of a draft call: the attention's, then the staging cache.
struct DraftLayout {
  size_t attn, k, v, table, seq_len, pending, offsets, bytes;
  int blocks;
};
static DraftLayout draft_layout(const mtp_ctx* ctx) {
  const mtp_config& c = ctx->cfg;
  DraftLayout L{};
  L.blocks = (c.max_k + kBlk - 1) / kBlk;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = (off + bytes + 255) & ~(size_t)255;
    return o;
  };
  const size_t entries = (size_t)c.max_batch * L.blocks, pool = entries * kBlk * ctx->kv_dim * (c.dtype == MTP_DTYPE_BF16 ? 2 : 4);
  L.attn = take(mtp_kv8_attention_workspace_bytes(ctx));
  L.k = take(pool);
  L.v = take(pool);
  L.table = take(entries * 4);
  L.seq_len = take((size_t)c.max_batch * 4);
  L.pending = take((size_t)c.max_batch * 4);
  L.offsets = take(((size_t)c.max_batch + 1) * 4);
  L.bytes = off;
  return L;
}

}  // namespace mtp

using namespace mtp;

extern "C" {

size_t mtp_draft_kv8_workspace_bytes(const mtp_ctx* ctx) { return ctx && ctx->has_weights ? draft_layout(ctx).bytes : 0; }

mtp_status mtp_draft_kv8(mtp_ctx* ctx, void* stream, int B, const void* hidden, const void* embeds,
                         const int32_t* positions, const mtp_kv8* kv, int K, const int32_t* chain_ids,
                         int32_t* draft_ids, float* logits, float* hidden_out, void* ws, size_t ws_bytes) {
  if (!ctx || !ctx->has_weights) return MTP_ERR_INVALID;
  if (B < 1 || B > ctx->cfg.max_batch || B > kA8MaxB || K < 1 || K > ctx->cfg.max_k) return MTP_ERR_INVALID;
  if (!hidden || !embeds || !positions || !draft_ids || !kv8_ok(kv)) return MTP_ERR_INVALID;
  const DraftLayout L = draft_layout(ctx);
  if (!ws || ((uintptr_t)ws & 255) || ws_bytes < L.bytes) return MTP_ERR_INVALID;
  DeviceGuard dev(ctx->device);
  if (!dev.ok) return MTP_ERR_CUDA;
  cudaStream_t s = (cudaStream_t)stream;
  char* base = (char*)ws;
  Kv8Draft d{};
  d.kv = *kv;
  d.stage.k_pool = base + L.k;
  d.stage.v_pool = base + L.v;
  d.stage.block_table = (int32_t*)(base + L.table);
  d.stage.seq_len = (int32_t*)(base + L.seq_len);
  d.stage.pending = (int32_t*)(base + L.pending);
  d.stage.num_blocks = ctx->cfg.max_batch * L.blocks;
  d.stage.max_blocks = L.blocks;
  d.positions = positions;
  d.row_offsets = (const int32_t*)(base + L.offsets);
  d.attn_ws = base + L.attn;
  cudaError_t e = launch_pdl(kv8_stage_kernel, dim3((B + 128) / 128), dim3(128), 0, s, B, L.blocks, d.stage.block_table,
                             d.stage.seq_len, d.stage.pending, (int32_t*)(base + L.offsets),
                             (const int32_t*)kv->pending);
  ctx->launches++;
  ctx->kv8_draft = &d;
  for (int k = 1; k <= K && e == cudaSuccess; ++k)
    e = draft_one_step(ctx, s, B, k, K, hidden, embeds, positions, &d.stage, chain_ids, draft_ids, logits, hidden_out);
  ctx->kv8_draft = nullptr;
  return launch_status(e);
}

size_t mtp_kv8_attention_workspace_bytes(const mtp_ctx* ctx) {
  if (!ctx) return 0;
  return a8_meta_bytes(ctx) + (size_t)2 * kA8MaxBlocks * ctx->num_sms * kA8MaxCols * (ctx->cfg.head_dim + 4) * 4;
}

mtp_status mtp_kv8_attention(mtp_ctx* ctx, void* stream, int B, int T, const int32_t* row_offsets, int max_rows,
                             const void* q, int64_t q_stride, const mtp_kv8* kv, const int32_t* mask, int mask_words,
                             float scale, void* out, float* lse, void* ws, size_t ws_bytes) {
  if (!ctx || B < 1 || B > ctx->cfg.max_batch || B > kA8MaxB || T < 0 || !row_offsets || !q || !out || !kv8_ok(kv))
    return MTP_ERR_INVALID;
  const mtp_config& c = ctx->cfg;
  if (max_rows < 1 || max_rows > 256 || q_stride < (int64_t)c.n_q_heads * c.head_dim) return MTP_ERR_INVALID;
  if (mask && mask_words < (max_rows + 31) / 32) return MTP_ERR_INVALID;
  if (!(scale > 0.0f) || !isfinite(scale)) return MTP_ERR_INVALID;
  if (!ws || ((uintptr_t)ws & 15) || ws_bytes < mtp_kv8_attention_workspace_bytes(ctx)) return MTP_ERR_INVALID;
  if (T == 0) return MTP_OK;
  DeviceGuard dev(ctx->device);
  if (!dev.ok) return MTP_ERR_CUDA;
  Attn8Args a{};
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.row_offsets = row_offsets;
  a.mask = mask;
  a.kv = *kv;
  a.err = ctx->err;
  a.meta = (int4*)ws;
  a.part = (float*)((char*)ws + a8_meta_bytes(ctx));
  a.q_stride = q_stride;
  a.B = B;
  a.T = T;
  a.max_rows = max_rows;
  a.mask_words = mask_words;
  const bool bf = c.dtype == MTP_DTYPE_BF16;
  attn8_fill(ctx, a, bf ? 2 : 4, scale);
  // columns per tile: the fewest tiles of at most 32 columns, evenly filled
  const int cols = max_rows << a.g_shift, tiles = (cols + kA8MaxCols - 1) / kA8MaxCols;
  const int nt = (cols + 8 * tiles - 1) / (8 * tiles);
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e =
      c.head_dim == 128 ? (bf ? attn8_pick<uint16_t, 128>(ctx, s, a, nt) : attn8_pick<float, 128>(ctx, s, a, nt))
                        : (bf ? attn8_pick<uint16_t, 64>(ctx, s, a, nt) : attn8_pick<float, 64>(ctx, s, a, nt));
  ctx->launches += 2;
  return launch_status(e);
}

}  // extern "C"
