// Last step of decode attention: the states that several clusters left of a
// row's keys are joined, and every row goes through W_UV of its head,
//   w_i = e^{lse_i - m} / sum_j e^{lse_j - m},  o = sum_i w_i o_i,  lse = m + ln sum_j e^{lse_j - m}
//   out[t][h] = out_scale o W_UV,h
// A CTA takes some tokens of one head: up to 64, fewer where the grid would not
// fill the GPU.  Its 32 warps join the fp32 states of their rows (few rows:
// several warps a row, each some of the pieces) into one K-major swizzled
// operand of 512 columns, each value as its bf16 and, in other rows, the bf16 of
// what that leaves, so that one chain of M = 128, N = 128 MMAs multiplies o to
// 2^-16; the two products are added at the end.  W_UV,h comes by TMA in chunks
// of 128 rows, two buffers deep; where there are 32 tokens at most, their rows
// leave room for all four chunks, which are there before the states (the rows of
// the MMA that no token has read what lies behind), and with 16 also for partial
// sums of warps that share a row.
// Latency-bound: a row is two dependent loads from L2 (weights, states), so the
// rows are spread over many warps (8 warps took 30 us for 64 tokens of 128
// heads).
#include <atomic>

#include "serving.cuh"

namespace mla {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr uint32_t kBlk = 16384;                   // [128 rows x 128 B] swizzled block
constexpr int kMaxPieces = kDecodeClusters;        // of one item

struct RowOf {
  int x;           // unit of the item's first tile
  int n;           // pieces: -1 no request's row, 0 no keys, 1 a whole item
  int c0;          // cluster of the first piece
  int ridx;        // row within the item
  float lse;
};
static_assert(sizeof(RowOf) == 20, "row table");

template <int kTokens>   // at most, of a CTA: 16, 32 or 64
struct Lay {
  static constexpr int kRest = kTokens;                            // row of a state's rest: this many below
  static constexpr uint32_t kABlk = 2 * kRest * 128;               // 64 columns of the rows that tokens have
  static constexpr int kChunks = kTokens <= 32 ? 4 : 2;            // buffers of [128 c x 128 j] in two blocks
  static constexpr bool kShared = kTokens <= 16;                   // warps may share a row
  static constexpr uint32_t kA = 0;                                // 8 blocks of 64 columns
  static constexpr uint32_t kB = 8 * kABlk;
  static constexpr uint32_t kShare = kB + kChunks * 2 * kBlk;      // partial sums of warps that share rows, 2 KB each
  static constexpr uint32_t kRows = kShare + (kShared ? kWarps * 2048 : 0);
  static constexpr uint32_t kBegin = kRows + kTokens * 20;         // first unit of each cluster
  static constexpr uint32_t kBars = (kBegin + 4 * (kDecodeClusters + 1) + 15) & ~15u;   // B landed, MMAs done x 2, TMEM address
  static constexpr uint32_t kSmem = kBars + 8 * (kChunks + 2) + 16;
  static_assert(kSmem <= 232448, "more than 227 KB of shared memory per CTA");
};
constexpr uint32_t kIdesc = idesc_bf16(128, 128, false, true);
__device__ __forceinline__ bool wait(uint32_t* err, uint32_t bar, uint32_t parity) {
  if (mbar_wait(bar, parity)) return true;
  atomicOr(err, kErrTimeout);
  return false;
}

// Request of row x by one thread (ascending cu_q).
__device__ __forceinline__ int find_request(const BatchRows& b, int x) {
  if (b.cu_q == nullptr) return x / b.per_req;
  int lo = 0, hi = b.num_reqs - 1;   // the last request that starts at or before x
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldcg(b.cu_q + mid) <= x) lo = mid; else hi = mid - 1;
  }
  const int2 rr = request_rows<true>(b, lo);
  return x >= rr.x && x < rr.y ? lo : -1;
}

// 4 columns 4 lane + 128 k of row i into the operand: their bf16, and that of the rest.
template <class L>
__device__ __forceinline__ void put4(uint32_t a, int i, int lane, int k, float4 v) {
  const int c = 4 * lane + 128 * k;
  const uint32_t addr = a + (uint32_t)(c >> 6) * L::kABlk + sw128_off((uint32_t)i, (uint32_t)((c & 63) >> 3)) + (c & 4) * 2;
  const uint32_t h0 = pack_bf16(v.x, v.y), h1 = pack_bf16(v.z, v.w);
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(h0), "r"(h1) : "memory");
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr + L::kRest * 128), "r"(pack_bf16(v.x - bf16_lo(h0), v.y - bf16_hi(h0))),
               "r"(pack_bf16(v.z - bf16_lo(h1), v.w - bf16_hi(h1)))
               : "memory");
}

template <int kTokens>
__global__ void __launch_bounds__(kThreads, 1) decode_out_kernel(const __grid_constant__ DecodeOutParams p) {
  using L = Lay<kTokens>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  const uint32_t bars = sb + L::kBars, done = bars + 8 * L::kChunks;
  RowOf* rows = reinterpret_cast<RowOf*>(smem + L::kRows);
  int* begin = reinterpret_cast<int*>(smem + L::kBegin);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kBars + 8 * (L::kChunks + 2));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = p.batch.num_heads, h = blockIdx.z, r0 = blockIdx.x * p.tile;
  const int R = min(p.tile, p.batch.rows.rows - r0);

  auto load_w = [&](int ch) {
    const uint32_t b = ch % L::kChunks, dst = sb + L::kB + b * 2 * kBlk;
    mbar_arrive_expect_tx(bars + 8 * b, 2 * kBlk);
    tma_load_2d(dst, &p.tm_w, 128 * H + 128 * h, 128 * ch, bars + 8 * b);
    tma_load_2d(dst + kBlk, &p.tm_w, 128 * H + 128 * h + 64, 128 * ch, bars + 8 * b);
  };
  if (tid == 0) {
    prefetch_tensormap(&p.tm_w);
#pragma unroll
    for (int i = 0; i < L::kChunks + 2; ++i) mbar_init(bars + 8 * i, 1);
    fence_mbar_init();
    for (int ch = 0; ch < L::kChunks; ++ch) load_w(ch);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 128);
    tmem_relinquish();
  }
  const int B = p.batch.rows.num_reqs;
  int r = -1;
  int2 rr = make_int2(0, 0);
  if (tid < R) {
    r = find_request(p.batch.rows, r0 + tid);
    if (r >= 0) rr = request_rows<true>(p.batch.rows, r);
  }
  grid_wait();      // the attention kernel's states are there
  grid_trigger();
  const int total = p.ws.first[B], n_clusters = p.ws.first[B + 1];
  if (tid < R) {
    RowOf o;
    o.n = -1;
    o.c0 = o.ridx = o.x = 0;
    o.lse = -INFINITY;
    if (r >= 0) {
      const int f = p.ws.first[r];
      const int items = ((rr.y - rr.x) * H + kItemRows - 1) / kItemRows;
      const int u = (p.ws.first[r + 1] - f) / items;
      const int idx = (r0 + tid - rr.x) * H + h;
      o.ridx = idx & (kItemRows - 1);
      o.n = 0;
      if (u > 0) {
        o.x = f + (idx / kItemRows) * u + kItemUnits;
        // (clamped: a cu_q that does not ascend must not lead outside the tables)
        o.c0 = min(max(cluster_of(o.x, n_clusters, max(total, 1)), 0), kDecodeClusters - 1);
        o.n = cluster_of(o.x + u - kItemUnits - 1, n_clusters, max(total, 1)) - o.c0 + 1;
        o.n = min(max(o.n, 0), kDecodeClusters - o.c0);
        if (o.n == 1) o.lse = p.ws.lat_lse[(int64_t)(r0 + tid) * H + h];
      }
    }
    rows[tid] = o;
  } else if (tid >= 512 && tid - 512 < n_clusters) {
    begin[tid - 512] = unit_begin(tid - 512, n_clusters, total);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // ---------------------------------------------------------------- the rows' states
  int G = 1;        // warps a row
  if (L::kShared)
    while (2 * G * R <= kWarps) G *= 2;
  const int part = warp % G;
  for (int i = warp / G; i < R; i += kWarps / G) {
    const RowOf o = rows[i];
    if (o.n == 1) {
      if (part == 0) {
        const float4* src = reinterpret_cast<const float4*>(p.ws.lat + ((int64_t)(r0 + i) * H + h) * kDc) + lane;
        float4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = src[32 * k];
#pragma unroll
        for (int k = 0; k < 4; ++k) put4<L>(sb + L::kA, i, lane, k, v[k]);
      }
      continue;
    }
    float4 acc[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (o.n > 1) {
      // lane l has the weights and slots of pieces l, l + 32, l + 64
      constexpr int kPerLane = (kMaxPieces + 31) / 32;
      float w[kPerLane], m = -INFINITY;
      int at[kPerLane];   // row of the states
#pragma unroll
      for (int k = 0; k < kPerLane; ++k) {
        const int c = o.c0 + lane + 32 * k;
        const bool have = lane + 32 * k < o.n;
        at[k] = have ? piece_slot(c, begin[c] <= o.x) * kItemRows + o.ridx : 0;
        w[k] = have ? p.ws.part_lse[at[k]] : -INFINITY;
        m = fmaxf(m, w[k]);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < kPerLane; ++k) {
        w[k] = w[k] == -INFINITY ? 0.f : __expf(w[k] - m);   // a NaN stays one
        sum += w[k];
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      const float inv = sum != 0.f ? 1.f / sum : 0.f;
      if (part == 0 && lane == 0) rows[i].lse = sum != 0.f ? m + __logf(sum) : -INFINITY;
      static_assert(kPerLane == 3, "the pieces of three lane groups");
#pragma unroll 2
      for (int l = part; l < o.n; l += G) {
        const float wi = __shfl_sync(0xffffffffu, l < 32 ? w[0] : l < 64 ? w[1] : w[2], l & 31) * inv;
        const int row = __shfl_sync(0xffffffffu, l < 32 ? at[0] : l < 64 ? at[1] : at[2], l & 31);
        const float4* src = reinterpret_cast<const float4*>(p.ws.part + (int64_t)row * kDc) + lane;
        float4 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = src[32 * q];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          acc[q].x = fmaf(wi, v[q].x, acc[q].x);
          acc[q].y = fmaf(wi, v[q].y, acc[q].y);
          acc[q].z = fmaf(wi, v[q].z, acc[q].z);
          acc[q].w = fmaf(wi, v[q].w, acc[q].w);
        }
      }
    }
    if (G == 1) {
#pragma unroll
      for (int k = 0; k < 4; ++k) put4<L>(sb + L::kA, i, lane, k, acc[k]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) reinterpret_cast<float4*>(smem + L::kShare + 2048 * warp)[lane + 32 * k] = acc[k];
    }
  }
  if (G > 1) {
    __syncthreads();
    for (int x = warp; x < 4 * R; x += kWarps) {   // columns 128 k .. of row i
      const int i = x >> 2, k = x & 3, n = rows[i].n;
      if (n != 1) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int g = 0; g < min(G, n); ++g) {
          const float4 v = reinterpret_cast<const float4*>(smem + L::kShare + 2048 * (i * G + g))[lane + 32 * k];
          s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
        }
        put4<L>(sb + L::kA, i, lane, k, s);
      }
    }
  }
  fence_proxy_async_smem();
  __syncthreads();

  // ---------------------------------------------------------------- out = o W_UV,h
  bool ok = true;
  if (tid == 0) {
    for (int ch = 0; ch < 4 && ok; ++ch) {
      const uint32_t b = ch % L::kChunks;
      ok = wait(p.ws.err, bars + 8 * b, (ch / L::kChunks) & 1);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        mma_bf16(tmem, sdesc_sw128(sb + L::kA + (2 * ch + (kk >> 2)) * L::kABlk + (kk & 3) * 32, 16, 1024),
                 sdesc_sw128(sb + L::kB + b * 2 * kBlk + kk * 2048, kBlk, 1024), kIdesc, (ch | kk) ? 1u : 0u);
      if (L::kChunks == 2 || ch >= 2) mma_commit(done + 8 * (ch & 1));
      if (L::kChunks == 2 && ch < 2) {
        ok = wait(p.ws.err, done + 8 * b, 0);
        if (ok) load_w(ch + 2);
      }
    }
  }
  ok = __syncthreads_and(ok);
  if (ok) ok = wait(p.ws.err, done, L::kChunks == 4 ? 0 : 1) && wait(p.ws.err, done + 8, L::kChunks == 4 ? 0 : 1);
  ok = __syncthreads_and(ok);
  tc_fence_after();
  if (ok) {
    // sixteen warps: TMEM lanes 32 (w mod 4) .., columns 32 (w / 4) ..; the products of the rests, in as many lanes
    // behind those of the tokens, pass through shared memory (the weights' buffers)
    const int q = warp & 3, i = (32 * q + lane) % L::kRest, cb = 32 * (warp >> 2);
    const bool of_rest = 32 * q + lane >= L::kRest;   // (of lanes below 2 kRest)
    float* rest = reinterpret_cast<float*>(smem + L::kB) + i * 132 + cb;   // rows of 128, padded
    const bool rows_here = warp < 16 && 32 * q < 2 * L::kRest && 32 * q % L::kRest < R;
    uint32_t v[32];
    if (rows_here) {
      tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + cb, v);
      if (of_rest) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          reinterpret_cast<uint4*>(rest)[k] = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
      }
    }
    __syncthreads();
    if (rows_here && !of_rest && i < R && rows[i].n >= 0) {
      const int64_t orow = (int64_t)(r0 + i) * H + h, o = orow * kDv + cb;
      const bool empty = rows[i].lse == -INFINITY;   // no key seen: 0
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float4 x = reinterpret_cast<const float4*>(rest)[k];
        const float f[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[4 * k + e] = empty ? 0u : __float_as_uint((__uint_as_float(v[4 * k + e]) + f[e]) * p.out_scale);
      }
      if (p.out_bf16) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + o);
        auto o2 = [&](int k) { return pack_bf16(__uint_as_float(v[k]), __uint_as_float(v[k + 1])); };
#pragma unroll
        for (int k = 0; k < 4; ++k) dst[k] = make_uint4(o2(8 * k), o2(8 * k + 2), o2(8 * k + 4), o2(8 * k + 6));
      } else {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<float*>(p.out) + o);
#pragma unroll
        for (int k = 0; k < 8; ++k) dst[k] = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
      }
      if (p.lse != nullptr && warp < 4) p.lse[orow] = rows[i].lse;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 128);
  }
}

}  // namespace

cudaError_t launch_decode_out(const DecodeOutParams& p, cudaStream_t s) {
  static std::atomic<bool> configured[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev].load()) {
    e = cudaFuncSetAttribute(decode_out_kernel<16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay<16>::kSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(decode_out_kernel<32>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay<32>::kSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(decode_out_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay<64>::kSmem);
    if (e != cudaSuccess) return e;
    configured[dev].store(true);
  }
  const dim3 grid((p.batch.rows.rows + p.tile - 1) / p.tile, 1, p.batch.num_heads);
  if (p.tile <= 16) return launch_dependent(decode_out_kernel<16>, grid, kThreads, Lay<16>::kSmem, p, s);
  if (p.tile <= 32) return launch_dependent(decode_out_kernel<32>, grid, kThreads, Lay<32>::kSmem, p, s);
  return launch_dependent(decode_out_kernel<64>, grid, kThreads, Lay<64>::kSmem, p, s);
}

}  // namespace mla
