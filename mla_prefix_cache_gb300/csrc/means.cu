// Means of the cache blocks that new rows fill: for every block j of request r
// with (len - n) / 64 <= j < len / 64 (n its new rows, already in the cache),
//   means[block] = 1/64 sum_i [c | k_rope]_i        (FP8 rows: kv_scale e4m3)
// summed in fp32 and rounded to bf16 once.  HBM-bound: 73,728 B (bf16) or 40,960
// (FP8) read and 1152 written a block.
//
// The host does not know how many blocks fill up: request r has the candidates
// [cu_r / 64 + r, cu_{r+1} / 64 + r + 1), at least the ceil(n / 64) blocks that n
// new rows can fill (floor((c + n) / 64) - floor(c / 64) + 1 is no less for any first
// row c), and those that are none are passed over.  The launch before may be the one
// that wrote the block table: what is looked up ahead of the wait for it is looked at
// again behind it (64 requests, a few blocks filled: 2.9 us, all looked up
// behind it 3.3).
//  - Few candidates (two an SM at most): a CTA each, every thread one 16-byte
//    column of some rows with all its loads in flight at once.
//  - Many: a CTA an SM, whose producer warp looks up 32 candidates at a time and
//    has blocks copied whole into a ring (three of 72 KB, or five of 40), so that
//    an SM always has that much in flight; the other warps add up from shared
//    memory.  62,818 rows (984 blocks, 74 MB, 10.8 us at the copy rate): 14.2 us;
//    with a CTA each 17.6, 2.4 waves whose look-ups and sums have nothing in flight.
#include <atomic>

#include "serving.cuh"
#include "sparse.h"

namespace mla {
namespace {

template <bool kFp8>
struct MeanShape {
  static constexpr int kCols = kFp8 ? 40 : 72;      // 16-byte columns of a row
  static constexpr int kGroups = kFp8 ? 8 : 4;      // row groups
  static constexpr int kThreads = kCols * kGroups;  // 320, 288
  static constexpr int kRows = kBlock / kGroups;
};

// First row of request r's new rows, clamped to the batch.
__device__ __forceinline__ int first_row(const BatchRows& b, int r) {
  return b.cu_q == nullptr ? r * b.per_req : min(max(__ldcg(b.cu_q + r), 0), b.rows);
}

// Candidate i: of request r, the last one whose candidates start at or before i, block j of its table (-1: none).
struct Candidate {
  int r, j;
};
__device__ __forceinline__ bool starts_by(const BatchRows& b, int r, int i) { return first_row(b, r) / kBlock + r <= i; }
__device__ __forceinline__ Candidate candidate_of(const MeansParams& p, int i, int r) {
  const int c0 = first_row(p.batch, r), n = first_row(p.batch, r + 1) - c0, len = __ldcg(p.batch.seq_lens + r);
  const int k = i - (c0 / kBlock + r), j = max(len - n, 0) / kBlock + k;
  return {r, n <= 0 || k < 0 || j >= len / kBlock ? -1 : j};
}
__device__ __forceinline__ int entry(const MeansParams& p, Candidate c) {
  return c.j >= 0 && c.j < p.max_blocks ? __ldcg(p.block_table + (int64_t)c.r * p.max_blocks + c.j) : -1;
}
// Its cache block, -1 for none, -2 for one to be reported.
__device__ __forceinline__ int taken(const MeansParams& p, Candidate c, int id) {
  return c.j < 0 ? -1 : id >= 0 && id < p.num_blocks ? id : -2;
}
// The same behind the wait, by what find(i) gave ahead of it.
template <class Find>
__device__ __forceinline__ int block_of(const MeansParams& p, int i, Candidate before, Find find) {
  // (loads that do not wait for one another)
  int id = entry(p, before);
  Candidate c = candidate_of(p, i, before.r);
  const bool same = starts_by(p.batch, c.r, i) && (c.r + 1 == p.batch.num_reqs || !starts_by(p.batch, c.r + 1, i));
  if (!same) c = find(i);
  if (c.r != before.r || c.j != before.j) id = entry(p, c);
  return taken(p, c, id);
}

// A 16-byte column of kRows rows added up: its values, 8 of bf16 or 16 of E4M3.
template <bool kFp8>
__device__ __forceinline__ void add_column(int col, const uint4 (&v)[MeanShape<kFp8>::kRows], float (&a)[kFp8 ? 16 : 8]) {
  using M = MeanShape<kFp8>;
#pragma unroll
  for (int e = 0; e < (kFp8 ? 16 : 8); ++e) a[e] = 0.f;
#pragma unroll
  for (int k = 0; k < M::kRows; ++k) {
    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
    if (!kFp8 || col >= kDc / 16) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[2 * e] += bf16_lo(w[e]);
        a[2 * e + 1] += bf16_hi(w[e]);
      }
    } else if constexpr (kFp8) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 lo = e4m3x2_floats(w[e] & 0xFFFFu), hi = e4m3x2_floats(w[e] >> 16);
        a[4 * e] += lo.x;
        a[4 * e + 1] += lo.y;
        a[4 * e + 2] += hi.x;
        a[4 * e + 3] += hi.y;
      }
    }
  }
}
template <bool kFp8>
__device__ __forceinline__ void put_column(float* sums, int col, const float (&a)[kFp8 ? 16 : 8]) {
  const bool rope = kFp8 && col >= kDc / 16;
  float* to = sums + (kFp8 ? (rope ? kDc + 8 * (col - kDc / 16) : 16 * col) : 8 * col);
#pragma unroll
  for (int e = 0; e < (kFp8 ? 16 : 8); e += 4)
    if (e < 8 || !rope) *reinterpret_cast<float4*>(to + e) = make_float4(a[e], a[e + 1], a[e + 2], a[e + 3]);
}
// Values 2 t, 2 t + 1 of the mean, from the groups' sums.
template <bool kFp8>
__device__ __forceinline__ void write_mean(const MeansParams& p, const float (*sums)[kRowBf16], int id, int t) {
  float x = 0.f, y = 0.f;
#pragma unroll
  for (int g = 0; g < MeanShape<kFp8>::kGroups; ++g) {
    const float2 s = *reinterpret_cast<const float2*>(&sums[g][2 * t]);
    x += s.x;
    y += s.y;
  }
  const float f = (kFp8 && t < kDc / 2 ? p.kv_scale : 1.f) / kBlock;
  reinterpret_cast<uint32_t*>(p.means)[(int64_t)id * (kRowBf16 / 2) + t] = pack_bf16(x * f, y * f);
}

template <bool kFp8>
__global__ void __launch_bounds__(MeanShape<kFp8>::kThreads) block_means_kernel(const __grid_constant__ MeansParams p) {
  using M = MeanShape<kFp8>;
  __shared__ __align__(16) float sums[M::kGroups][kRowBf16];
  const int tid = threadIdx.x, lane = tid & 31, i = blockIdx.x;
  auto find = [&](int i) {      // 32 tries a step
    int r = 0;
    for (int n = p.batch.num_reqs; n > 1;) {
      const int step = (n + 31) / 32, at = lane * step;
      const bool ok = lane == 0 || (at < n && starts_by(p.batch, r + at, i));
      const int k = 31 - __clz(__ballot_sync(0xffffffffu, ok));
      r += k * step;
      n = min(step, n - k * step);
    }
    return candidate_of(p, i, r);
  };
  const Candidate before = find(i);
  const int guess = taken(p, before, entry(p, before));
  grid_wait();      // the new rows are in the cache, their blocks in the table
  grid_trigger();
  const int col = tid % M::kCols, group = tid / M::kCols;
  uint4 v[M::kRows];
  auto load = [&](int id) {
    const uint4* src = reinterpret_cast<const uint4*>(p.cache) + ((int64_t)id * kBlock + group * M::kRows) * M::kCols + col;
#pragma unroll
    for (int k = 0; k < M::kRows; ++k) v[k] = __ldg(src + k * M::kCols);
  };
  if (guess >= 0) load(guess);      // on its way beside the second look
  const int id = block_of(p, i, before, find);
  if (id >= 0 && id != guess) load(id);
  if (id < 0) {
    if (id == -2 && tid == 0 && p.err != nullptr) atomicOr(p.err, kErrBadBlock);
    return;
  }
  float a[kFp8 ? 16 : 8];
  add_column<kFp8>(col, v, a);
  put_column<kFp8>(sums[group], col, a);
  __syncthreads();
  if (tid < kRowBf16 / 2) write_mean<kFp8>(p, sums, id, tid);
}

template <bool kFp8>
struct RingShape : MeanShape<kFp8> {
  static constexpr uint32_t kBytes = kBlock * (kFp8 ? kRowBytesFp8 : kRowBytesBf16);
  static constexpr int kStages = kFp8 ? 5 : 3;
  static constexpr int kAdders = MeanShape<kFp8>::kThreads;      // then the producer warp
  static constexpr uint32_t kSums = kStages * kBytes;
  static constexpr uint32_t kBars = kSums + MeanShape<kFp8>::kGroups * kRowBf16 * 4;      // full, empty, the stages' block ids
  static constexpr uint32_t kSmem = kBars + kStages * 24;
  static_assert(kSmem <= 232448, "shared memory per CTA");
};

template <bool kFp8>
__global__ void __launch_bounds__(RingShape<kFp8>::kAdders + 32, 1) block_means_ring_kernel(const __grid_constant__ MeansParams p) {
  using M = RingShape<kFp8>;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  float(*sums)[kRowBf16] = reinterpret_cast<float(*)[kRowBf16]>(smem + M::kSums);
  volatile int* ids = reinterpret_cast<volatile int*>(smem + M::kBars + 16 * M::kStages);
  auto full = [&](int s) { return sb + M::kBars + 8u * s; };
  auto empty = [&](int s) { return sb + M::kBars + 8u * (M::kStages + s); };
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < M::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), M::kAdders / 32);
    }
    fence_mbar_init();
  }
  __syncthreads();
  auto await = [&](uint32_t bar, uint32_t parity) {
    if (mbar_wait(bar, parity, p.wait_limit_ns)) return true;
    if (p.err != nullptr) atomicOr(p.err, kErrTimeout);
    return false;
  };
  if (tid >= M::kAdders) {
    // ---- producer: 32 candidates looked up at a time, their blocks asked for one by one
    const int total = p.batch.rows / kBlock + p.batch.num_reqs;
    auto find = [&](int i) {
      int r = 0;
      for (int n = p.batch.num_reqs; n > 1;) {
        const int half = n >> 1;
        if (starts_by(p.batch, r + half, i)) { r += half; n -= half; }
        else n = half;
      }
      return candidate_of(p, i, r);
    };
    bool ok = true, waited = false;
    int g = 0;
    for (int64_t base = blockIdx.x; ok && base < total; base += 32 * (int64_t)gridDim.x) {
      const int64_t i = base + lane * (int64_t)gridDim.x;
      Candidate c = {0, -1};
      if (i < total) c = find((int)i);
      int id = -1;
      if (waited) {
        id = taken(p, c, entry(p, c));
      } else {
        grid_wait();      // the new rows are in the cache, their blocks in the table
        grid_trigger();
        waited = true;
        if (i < total) id = block_of(p, (int)i, c, find);
      }
      if (id == -2 && p.err != nullptr) atomicOr(p.err, kErrBadBlock);
      for (uint32_t rest = __ballot_sync(0xffffffffu, id >= 0); ok && rest; rest &= rest - 1, ++g) {
        const int next = __shfl_sync(0xffffffffu, id, __ffs(rest) - 1), s = g % M::kStages;
        if (g >= M::kStages && !(ok = __all_sync(0xffffffffu, await(empty(s), (g / M::kStages - 1) & 1)))) break;
        if (lane == 0) {
          ids[s] = next;
          mbar_arrive_expect_tx(full(s), M::kBytes);
          bulk_load(sb + s * M::kBytes, p.cache + (int64_t)next * M::kBytes, M::kBytes, full(s));
        }
      }
    }
    // the end: an id of -1 (on a wait that gave up the adders give up too)
    const int s = g % M::kStages;
    int v = max(0, g - M::kStages);      // loads before this one have landed
    if (ok && g >= M::kStages) {
      ok = __all_sync(0xffffffffu, await(empty(s), (g / M::kStages - 1) & 1));
      v += ok;                           // its stage's barrier goes on to the end's phase
    }
    if (ok && lane == 0) {
      ids[s] = -1;
      mbar_arrive(full(s));
    }
    for (; v < g; ++v) await(full(v % M::kStages), (v / M::kStages) & 1);   // no copy is in flight when the CTA ends
  } else {
    // ---- adders
    grid_wait();
    grid_trigger();
    const int col = tid % M::kCols, group = tid / M::kCols;
    for (int g = 0; (int)blockIdx.x != p.withhold; ++g) {
      const int s = g % M::kStages;
      if (named_bar_or(1, M::kAdders, !await(full(s), (g / M::kStages) & 1))) break;      // (the sums of the block before have been read too)
      const int id = ids[s];
      if (id < 0) break;
      uint4 v[M::kRows];
      float a[kFp8 ? 16 : 8];
      const uint32_t src = sb + s * M::kBytes + ((group * M::kRows) * M::kCols + col) * 16;
#pragma unroll
      for (int k = 0; k < M::kRows; ++k) {
        uint32_t w[4];
        lds128(src + k * M::kCols * 16, w);
        v[k] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      add_column<kFp8>(col, v, a);
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(s));
      put_column<kFp8>(sums[group], col, a);
      named_bar_sync(2, M::kAdders);
      if (tid < kRowBf16 / 2) write_mean<kFp8>(p, sums, id, tid);
    }
  }
}

template <bool kFp8>
cudaError_t launch(const MeansParams& p, cudaStream_t s) {
  constexpr int kSms = 2 * kDecodeClusters;
  const int candidates = p.batch.rows / kBlock + p.batch.num_reqs;
  if (candidates <= 2 * kSms) return launch_dependent(block_means_kernel<kFp8>, dim3(candidates), MeanShape<kFp8>::kThreads, 0, p, s);
  static std::atomic<uint64_t> configured;   // devices
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(configured.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(block_means_ring_kernel<kFp8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)RingShape<kFp8>::kSmem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(1ull << dev);
  }
  return launch_dependent(block_means_ring_kernel<kFp8>, dim3(kSms), RingShape<kFp8>::kAdders + 32, RingShape<kFp8>::kSmem, p, s);
}

}  // namespace

cudaError_t launch_block_means(const MeansParams& p, bool fp8, cudaStream_t s) {
  if (p.batch.rows == 0) return cudaSuccess;
  return fp8 ? launch<true>(p, s) : launch<false>(p, s);
}

}  // namespace mla
