// Scores of cache blocks for a query: the share of its attention that the blocks'
// mean rows would take, over the heads that share them (all, with one latent row
// for every head):
//   s_hj = scale (qlat_h . c_j + R(pos) q_rope_h . k_j)    [c_j | k_j] the mean row of block j
//   score_j = 1/H sum_h e^{s_hj} / sum_i e^{s_hi}          over the blocks before the query's own
// in three launches, each dependent on the one before: the query absorption
// (headproj.cu), which also turns q_rope, score_kernel, which leaves s with the
// maximum and sum of each 32 blocks per head, and join_kernel, which adds up the heads.
//
// score_kernel.  The (query, head) rows of a request form items of whole queries,
// 128 rows at most; an item's blocks form tiles of 64.  The tiles of all items are
// cut evenly over a persistent grid of one CTA an SM, on the device from the
// lengths: every CTA makes the prefix sum over the requests for itself.  Q [128 x
// 576] of an item sits in TMEM (by TMA in four groups of blocks through two places,
// the next item's ahead of time), which leaves shared memory to a ring of two tiles
// of mean rows; S [128 x 64] of each tile goes to one of two TMEM buffers.  The rows of a tile lie anywhere in the pool: they are gathered by
// cp.async, whose copies the loading threads turn into the MMAs' swizzle.  Mean
// rows do not depend on the query absorption, so their loads start before it ends.
//
// S leaves in f16, less the largest of its 32 blocks, which is kept in fp32 with the
// sum of 2^(s - maximum): that moves s by 2^-11 of the difference at most, and half
// the bytes go to L2 and back.  Of the fp32 shares' error against 64 bits (32 queries
// of 2048 blocks, 2.44e-4 of their norm) the bf16 operands alone make 2.43e-4, the
// f16 alone 2.5e-5.
#include <atomic>

#include "scores.cuh"

namespace mla {
namespace {

// warps 0-3: loads of mean rows; 4: MMA; 5: loads of Q; 8-15: Q into TMEM and scores, two threads a row
constexpr int kThreads = 512;
constexpr int kGrid = 2 * kDecodeClusters;         // one CTA on each of a GB300's 152 SMs
constexpr int kBlocksQ = kRowBf16 / 64;            // 64-column blocks of a row
constexpr uint32_t kQBlk = 16384;                  // [128 rows x 128 B]
// Q is staged in groups of blocks, 0-2 and 5-7 in one place, 3-4 and 8 in another; every thread that takes blocks out
// waits for every group.  (Staging blocks that passed between groups of threads would have phases that one of them does
// not wait for, and a wait for the phase after one that is not over returns at once.)
constexpr int kQStages = 5, kQPlaces = 2, kQGroups = 4;
__device__ __forceinline__ constexpr int group_first(int g) { return g == 0 ? 0 : g == 1 ? 3 : g == 2 ? 5 : g == 3 ? 8 : 9; }
__device__ __forceinline__ constexpr uint32_t group_place(int g) { return (g & 1 ? 3 : 0) * 16384u; }
constexpr uint32_t kBlk = kScoreTile * 128;        // [64 rows x 128 B]
constexpr int kStageBlks = 3, kTileStages = kBlocksQ / kStageBlks, kStages = 2 * kTileStages;
constexpr uint32_t kStage = kStageBlks * kBlk;
constexpr uint32_t kRing = kQStages * kQBlk;
constexpr uint32_t kBars = kRing + kStages * kStage;
enum : uint32_t {
  kF = 0,                 // 6: stage landed (128 threads)
  kE = kF + kStages,      // 6: its MMAs are done
  kQT = kE + kStages,     // 2: a place's group of Q's blocks landed
  kQS = kQT + kQPlaces,   // 2: it is in TMEM (8 warps)
  kQR = kQS + kQPlaces,   // 3: the blocks that a stage's MMAs read are in TMEM (8 warps)
  kSF = kQR + kTileStages,   // 2: S buffer written
  kSR = kSF + 2,          // 2: S buffer read (8 warps)
  kNBars = kSR + 2
};
constexpr uint32_t kShared = kBars + 8 * kNBars;   // TMEM address, warps' sums, where the CTA begins
constexpr uint32_t kSums = kShared + 16;
constexpr uint32_t kFlags = kSums + 3 * 4 * (kThreads / 32);
constexpr uint32_t kBegin = kFlags + 4 * (kThreads / 32);
constexpr uint32_t kSmem = kBegin + 8 + 24 * 32;   // (struct Begin)
constexpr uint32_t kTmemS = 32 * kBlocksQ;         // columns of Q, then the S buffers
constexpr uint32_t kIdesc = idesc_bf16(128, kScoreTile, false, false);
static_assert(kScoreTile == 64 && kSmem <= 232448, "shared memory per CTA");

// What a request adds to the work: items of `per_item` whole queries, tiles of each.
struct Work {
  int q0, n, len, items, tiles;
};
__device__ __forceinline__ Work work_of(const ScoreParams& p, int r) {
  Work w;
  const int2 rr = request_rows<true>(p.batch, r);
  w.q0 = rr.x;
  w.n = rr.y - rr.x;
  w.len = min(max(__ldcg(p.batch.seq_lens + r), 0), p.max_blocks * kBlock);
  w.items = (w.n + p.per_item - 1) / p.per_item;
  w.tiles = (max(w.len - 1, 0) / kBlock + kScoreTile - 1) / kScoreTile;   // blocks before the last token's
  return w;
}

// What the CTA's threads found out about its first requests, for its roles: request r is entry r % 32, if that says so.
constexpr int kKept = 32;
struct Begin {
  int r, first;      // first request, its first unit
  int req[kKept];
  Work w[kKept];
};
static_assert(kBegin + sizeof(Begin) == kSmem, "shared memory");

// A CTA's run of units (item, tile), walked alike by every role.
struct Units {
  int left, r;             // units, request
  Work w;
  int item, tile;          // the present unit
  bool head;               // the first unit of its item here
  __device__ __forceinline__ void look_up(const ScoreParams& p, const Begin& b) {
    const int i = r % kKept;
    w = b.req[i] == r ? b.w[i] : work_of(p, r);
  }
  // units [at, end), or piece `at` of items cut into pieces of `per` tiles
  __device__ __forceinline__ bool start(const ScoreParams& p, const Begin& b, int at, int end, int per) {
    left = end - at;
    if (left <= 0) return false;
    r = b.r;
    look_up(p, b);
    const int of_item = per ? (w.tiles + per - 1) / per : w.tiles;
    item = (at - b.first) / of_item;
    tile = at - b.first - item * of_item;
    if (per) {
      tile *= per;
      left = min(per, w.tiles - tile);
    }
    head = true;
    return true;
  }
  __device__ __forceinline__ bool next(const ScoreParams& p, const Begin& b) {
    if (--left <= 0) return false;
    head = ++tile == w.tiles;
    if (!head) return true;
    tile = 0;
    if (++item == w.items) {
      item = 0;
      do {
        ++r;
        look_up(p, b);
      } while (w.items == 0 || w.tiles == 0);
    }
    return true;
  }
  // the block that the token of the item's query i lies in
  __device__ __forceinline__ int own(const ScoreParams& p, int i) const {
    return max(w.len - w.n + item * p.per_item + i, 0) / kBlock;
  }
  __device__ __forceinline__ int queries(const ScoreParams& p) const { return min(p.per_item, w.n - item * p.per_item); }
};

__device__ __forceinline__ bool await(const ScoreParams& p, uint32_t bar, uint32_t parity) {
  if (mbar_wait(bar, parity, p.wait_limit_ns)) return true;
  grid_wait();     // (the launch before clears the word)
  atomicOr(p.err, kErrTimeout);
  return false;
}
__device__ __forceinline__ bool await_warp(const ScoreParams& p, uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, await(p, bar, parity));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {   // the rest of the 16 is 0
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// An arrival on the barrier once the thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__global__ void __launch_bounds__(kThreads, 1) score_kernel(const __grid_constant__ ScoreParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto bar = [&](uint32_t i) { return sb + kBars + 8u * i; };
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + kShared);
  int* sums = reinterpret_cast<int*>(smem + kSums);
  uint32_t* warp_flags = reinterpret_cast<uint32_t*>(smem + kFlags);
  Begin* begin = reinterpret_cast<Begin*>(smem + kBegin);
  const int H = p.num_heads;

  if (tid == 0) {
    prefetch_tensormap(&p.tm_q);
    for (uint32_t i = 0; i < kNBars; ++i)
      mbar_init(bar(i), i < kE ? 128 : (i >= kQS && i < kSF) || i >= kSR ? 8 : 1);
    fence_mbar_init();
  }
  if (tid < kKept) begin->req[tid] = -1;
  if (warp == 5) {
    tmem_alloc(smem_u32(smem + kShared), 512);
    tmem_relinquish();
  }

  // ---- this CTA's units: thread t has requests [t k, (t + 1) k)
  const int B = p.batch.num_reqs, k = (B + kThreads - 1) / kThreads;
  const int r0 = min(B, tid * k), r1 = min(B, r0 + k);
  Work mine;                         // of the last one
  int sum = 0;
  bool mixed = false, cut = false;   // a request that ends before it starts, a sequence longer than its table
  for (int r = r0; r < r1; ++r) {
    mine = work_of(p, r);
    sum += mine.items * mine.tiles;
    cut |= __ldcg(p.batch.seq_lens + r) > p.max_blocks * kBlock;
    if (p.batch.cu_q != nullptr) mixed |= __ldcg(p.batch.cu_q + r + 1) < __ldcg(p.batch.cu_q + r);
  }
  // prefix sum over the threads, and the total, through `sums` (16 more words of it a call)
  int slot = 0;
  auto scan = [&](int v, int* before) {
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    int* w = sums + (kThreads / 32) * slot++;
    if (lane == 31) w[warp] = x;
    __syncthreads();
    const int of = lane < kThreads / 32 ? w[lane] : 0;
    *before = x - v + __reduce_add_sync(0xffffffffu, lane < warp ? of : 0);
    return __reduce_add_sync(0xffffffffu, of);
  };
  const uint32_t flags = __reduce_or_sync(0xffffffffu, (mixed ? 1u : 0u) | (cut ? 2u : 0u));
  if (lane == 0) warp_flags[warp] = flags;
  int pre = 0;
  int total = scan(sum, &pre);      // (its barrier is the first one: the mbarriers are there)
  const uint32_t all_flags = __reduce_or_sync(0xffffffffu, lane < kThreads / 32 ? warp_flags[lane] : 0u);
  mixed = all_flags & 1;
  cut = all_flags & 2;
  if (mixed) total = 0;      // (it could count rows twice and pass 31 bits)
  const int grid = gridDim.x, c = blockIdx.x;
  // A second item costs a CTA about two tiles (its Q takes 3.5 us to come).  So where the items, cut into pieces of as many
  // tiles as an even share has, or one more, are no more than the CTAs, each CTA has one piece: 64 queries of up to 512
  // blocks 20.7 us, cut evenly 22.1.  Else the units are cut evenly, and a CTA's run may pass from item to item.
  int per = 0;               // tiles of a piece
  if (total > grid) {
    const int t0 = (total + grid - 1) / grid;
    int n0 = 0, n1 = 0, before0, before1;
    for (int r = r0; r < r1; ++r) {
      const Work w = k == 1 ? mine : work_of(p, r);
      n0 += w.items * ((w.tiles + t0 - 1) / t0);
      n1 += w.items * ((w.tiles + t0) / (t0 + 1));
    }
    const int all0 = scan(n0, &before0);
    if (all0 <= grid) {
      per = t0;
      pre = before0;
      sum = n0;
      total = all0;
    } else if (const int all1 = scan(n1, &before1); all1 <= grid) {
      per = t0 + 1;
      pre = before1;
      sum = n1;
      total = all1;
    }
  }
  // the first total % grid CTAs have one unit (or piece) more than the others
  const int each = total / grid, more_of = total - each * grid;
  const int at = c * each + min(c, more_of), end = at + each + (c < more_of ? 1 : 0);
  auto parts = [&](const Work& w) { return w.items * (per ? (w.tiles + per - 1) / per : w.tiles); };
  if (at < end && pre <= at && at < pre + sum) {
    int r = r0, first = pre;
    if (k > 1)
      for (;; ++r) {
        mine = work_of(p, r);
        if (at < first + parts(mine)) break;
        first += parts(mine);
      }
    begin->r = r;
    begin->first = first;
  }
  if (k == 1 && r0 < r1 && pre < end && pre + sum >= at && atomicCAS(&begin->req[r0 % kKept], -1, r0) == -1) begin->w[r0 % kKept] = mine;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Units u;
  bool more = u.start(p, *begin, at, end, per);
  if (warp >= 4) {
    grid_wait();      // qlat is there
    grid_trigger();
    if (c == 0 && tid == 128) {
      *p.state = mixed;
      if (mixed || cut) atomicOr(p.err, kErrBadBlock);
    }
  }

  if (warp < 4) {
    // ------------------------------------------------------------ mean rows: 16 B of rows tid / 8 + 16 i a thread.  The
    // arrival of its copies is left to the copies; the next tile's block ids are on their way meanwhile.
    const int row = tid >> 3, chunk = tid & 7;
    bool ok = true, bad = false;
    if (c == p.withhold) more = false;
    int ids[4], seen = 0;
    auto look_up = [&]() {
      seen = u.own(p, u.queries(p) - 1) - u.tile * kScoreTile - row;      // the thread's rows 16 i < seen count
#pragma unroll
      for (int i = 0; i < 4; ++i)
        ids[i] = 16 * i < seen ? __ldcg(p.block_table + (int64_t)u.r * p.max_blocks + u.tile * kScoreTile + row + 16 * i) : 0;
    };
    if (more) look_up();
    int g = 0;                    // stages
    while (ok && more) {
      const uint8_t* src[4];
      uint32_t bytes[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool there = ids[i] >= 0 && ids[i] < p.num_blocks && 16 * i < seen;
        bad |= 16 * i < seen && !there;
        src[i] = reinterpret_cast<const uint8_t*>(p.means) + (there ? (int64_t)ids[i] * (2 * kRowBf16) : 0) + 16 * chunk;
        bytes[i] = there ? 16u : 0u;
      }
      more = u.next(p, *begin);
      if (more) look_up();
#pragma unroll 1
      for (int i = 0; i < kTileStages; ++i, ++g) {
        const int s = g % kStages;
        if (g >= kStages && !(ok = await_warp(p, bar(kE + s), (g / kStages - 1) & 1))) break;
#pragma unroll
        for (int b = 0; b < kStageBlks; ++b)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            cp_async16(sb + kRing + s * kStage + b * kBlk + sw128_off(row + 16 * k, chunk), src[k] + 128 * (kStageBlks * i + b), bytes[k]);
        cp_async_arrive(bar(kF + s));
      }
    }
    cp_async_wait_all();
    for (int v = max(0, g - kStages); v < g && ok; ++v) ok = await_warp(p, bar(kE + v % kStages), (v / kStages) & 1);   // before this CTA ends
    if (bad) {
      grid_wait();
      atomicOr(p.err, kErrBadBlock);
    }
  } else if (warp == 4) {
    // ------------------------------------------------------------ S = Q [c | k]^T
    const uint64_t cd0 = sdesc_sw128(sb + kRing, 16, 1024);
    bool ok = true;
    int t = 0, e = 0;             // tiles, items
    while (ok && more) {
      const int b = t & 1;
      const bool head = u.head;
      if (head) ++e;
      if (t >= 2) ok = await_warp(p, bar(kSR + b), ((t >> 1) - 1) & 1);
#pragma unroll
      for (int i = 0; i < kTileStages && ok; ++i) {
        const int s = kTileStages * b + i;
        ok = await_warp(p, bar(kF + s), (t >> 1) & 1) && (!head || await_warp(p, bar(kQR + i), (e - 1) & 1));
        if (!ok) break;
        fence_proxy_async_smem();   // written by the threads' copies, read by the MMAs as operands
        tc_fence_after();
        const uint64_t cd = sdesc_add(cd0, s * kStage);
#pragma unroll
        for (int k = 0; k < kStageBlks; ++k)
          mma_ts4_elect(tmem + kTmemS + kScoreTile * b, tmem + 32 * (kStageBlks * i + k), sdesc_add(cd, k * kBlk), kIdesc, i + k ? 1u : 0u);
        mma_commit_elect(bar(kE + s));
      }
      if (ok) mma_commit_elect(bar(kSF + b));
      ++t;
      more = u.next(p, *begin);
    }
  } else if (warp == 5 && lane == 0) {
    // ------------------------------------------------------------ Q of each item, a group of blocks at a time (with a barrier
    // a block, 350 cycles each, the loads paced a CTA's first tile)
    bool ok = true;
    int groups = 0;
    for (; ok && more; more = u.next(p, *begin)) {
      if (!u.head) continue;
      const int row = (u.w.q0 + u.item * p.per_item) * H;
#pragma unroll
      for (int g = 0; g < kQGroups; ++g) {
        const int pl = g & 1, use = groups >> 1;      // the place, its earlier groups
        if (ok && use > 0) ok = await(p, bar(kQS + pl), (use - 1) & 1);
        if (!ok) break;
        mbar_arrive_expect_tx(bar(kQT + pl), (group_first(g + 1) - group_first(g)) * kQBlk);
#pragma unroll
        for (int b = group_first(g); b < group_first(g + 1); ++b)
          tma_load_2d(sb + group_place(g) + (b - group_first(g)) * kQBlk, &p.tm_q, 64 * b, row, bar(kQT + pl));
        ++groups;
      }
    }
    for (int v = max(0, groups - kQPlaces); v < groups; ++v) await(p, bar(kQT + (v & 1)), (v >> 1) & 1);   // its loads land
  } else if (warp >= 8) {
    // ------------------------------------------------------------ Q: blocks of the half's parity; scores: columns 32 half .. of
    // a row a thread
    const int half = (warp - 8) >> 2, r = 32 * (warp & 3) + lane;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16), cols = lanes + kTmemS + 32 * half;
    const int64_t rows = (int64_t)p.batch.rows * H;
    bool ok = true;
    int t = 0, groups = 0, own = 0;      // tiles, groups of Q's blocks
    for (; ok && more; more = u.next(p, *begin)) {
      const int x0 = u.w.q0 + u.item * p.per_item;
      const bool live = r < u.queries(p) * H;
      const int64_t row = (int64_t)x0 * H + r;
      if (u.head) {
        // the last S buffer has been seen: no MMA reads the Q before this
        own = u.own(p, r / H);
        tc_fence_after();
#pragma unroll 1
        for (int g = 0; g < kQGroups; ++g, ++groups) {
          if (ok) ok = await_warp(p, bar(kQT + (g & 1)), (groups >> 1) & 1);
          const int b0 = group_first(g);
#pragma unroll 1
          for (int i = b0 + ((b0 ^ half) & 1); i < group_first(g + 1); i += 2) {
            uint32_t w[32];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              uint32_t w4[4];
              lds128(sb + group_place(g) + (i - b0) * kQBlk + sw128_off((uint32_t)r, (uint32_t)c), w4);
              w[4 * c] = w4[0]; w[4 * c + 1] = w4[1]; w[4 * c + 2] = w4[2]; w[4 * c + 3] = w4[3];
            }
            tmem_st32(lanes + 32 * i, w);
          }
          __syncwarp();
          if (lane == 0 && ok) mbar_arrive(bar(kQS + (g & 1)));
          if (g == 1) continue;      // groups 0, 2 and 3 complete the blocks of the stages 0, 1 and 2
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0 && ok) mbar_arrive(bar(kQR + max(0, g - 1)));
        }
        if (!ok) break;
      }
      const int b = t & 1;
      if (!(ok = await_warp(p, bar(kSF + b), (t >> 1) & 1))) break;
      ++t;
      tc_fence_after();
      uint32_t v[32];
      tmem_ld32(cols + kScoreTile * b, v);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kSR + b));
      const int sub = 2 * u.tile + half, seen = own - 32 * sub;      // columns that the row sees
      if (!live || seen <= 0) continue;
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float s = __uint_as_float(v[i]) * p.scale_log2;
        v[i] = __float_as_uint(s);
        if (i < seen) m = fmaxf(m, s);
      }
      if (m != -INFINITY) {
#pragma unroll
        for (int i = 0; i < 32; ++i) l += i < seen ? ex2(__uint_as_float(v[i]) - m) : 0.f;
      } else {      // only NaN, or only -infinite
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i < seen && __uint_as_float(v[i]) != __uint_as_float(v[i])) l = __uint_as_float(v[i]);
      }
      p.ml[sub * rows + row] = make_float2(m, l);
      const float top = m == -INFINITY ? 0.f : m;
      uint4* dst = p.s + (int64_t)sub * 4 * rows + row;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = pack_f16(__uint_as_float(v[8 * i + 2 * e]) - top, __uint_as_float(v[8 * i + 2 * e + 1]) - top);
        dst[i * rows] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

__device__ __forceinline__ float2 f16x2_floats(uint32_t a) {
  float2 f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}" : "=f"(f.x), "=f"(f.y) : "r"(a));
  return f;
}

// A maximum and the sum of 2^(s - maximum) joined with another one's; (-infinite, 0) is nothing.
__device__ __forceinline__ void add_part(float& m, float& l, float2 a) {
  if (a.x == -INFINITY && a.y == 0.f) return;
  const float top = fmaxf(m, a.x);
  l = l * ex2(m - top) + a.y * ex2(a.x - top);
  m = top;
}

// A CTA has 128 blocks of one query, or four times as many: each head's maximum and sum over all blocks, the warps
// taking every 16th entry of all heads, then the heads' shares of eight blocks a step and warp, 32 heads at a time.  The
// scores are asked for before the sums.
constexpr int kJoinWarps = 16, kJoinBlocks = 8 * kJoinWarps;
template <int kSteps>
__global__ void __launch_bounds__(32 * kJoinWarps, kSteps == 1 ? 2 : 1) join_kernel(const __grid_constant__ ScoreParams p) {
  __shared__ float2 part[kJoinWarps][kMaxHeads];
  __shared__ float2 head[kMaxHeads];   // maximum, 1 / (sum H)
  const int x = blockIdx.y, j0 = blockIdx.x * kSteps * kJoinBlocks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kGroups = kMaxHeads / 32;
  const Query o = query_of_row(p.batch, p.max_blocks, x, lane);
  grid_wait();
  grid_trigger();
  const bool mixed = __ldcg(p.state) != 0;
  if (p.lens != nullptr && blockIdx.x == 0 && tid == 0) p.lens[x] = mixed ? 0 : chosen_length(o, p.keep);
  if (p.cu != nullptr && blockIdx.x == 0 && tid == 0) {      // the requests' rows, one each
    const int lo = request_rows(p.batch, 0).x, hi = request_rows(p.batch, p.batch.num_reqs - 1).y;
    p.cu[x] = mixed ? 0 : min(max(x, lo), hi);
    if (x == p.batch.rows - 1) p.cu[x + 1] = mixed ? 0 : hi;
  }
  if (o.req < 0) return;
  const int H = p.num_heads, seen = mixed ? 0 : o.block;
  const int64_t n = (int64_t)p.batch.rows * H, row0 = (int64_t)x * H + lane;
  uint4 v[kSteps][kGroups];
  float m8[kSteps][kGroups];           // what the scores are less than
#pragma unroll
  for (int c = 0; c < kSteps; ++c)
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      const int j = j0 + kJoinBlocks * c + 8 * warp;
      const bool there = j < seen && lane + 32 * k < H;
      v[c][k] = there ? __ldcg(p.s + (int64_t)(j / 8) * n + row0 + 32 * k) : make_uint4(0, 0, 0, 0);
      m8[c][k] = there ? __ldcg(&p.ml[(int64_t)(j / 32) * n + row0 + 32 * k].x) : 0.f;
    }
  if (j0 < seen) {
    const int subs = (seen + 31) / 32;
    float m[kGroups], l[kGroups];
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      m[k] = -INFINITY;
      l[k] = 0.f;
    }
#pragma unroll 1
    for (int t = warp; t < subs; t += 2 * kJoinWarps) {
      float2 a[2][kGroups];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < kGroups; ++k)
          a[i][k] = t + i * kJoinWarps < subs && lane + 32 * k < H ? __ldcg(p.ml + (t + i * kJoinWarps) * n + row0 + 32 * k)
                                                                   : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < kGroups; ++k) add_part(m[k], l[k], a[i][k]);
    }
#pragma unroll
    for (int k = 0; k < kGroups; ++k) part[warp][lane + 32 * k] = make_float2(m[k], l[k]);
    __syncthreads();
    if (tid < H) {
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) add_part(top, sum, part[w][tid]);
      head[tid] = make_float2(top, 1.f / (sum * H));
    }
    __syncthreads();
  }
#pragma unroll
  for (int c = 0; c < kSteps; ++c) {
    const int j = j0 + kJoinBlocks * c + 8 * warp;
    if (j >= p.max_blocks) return;
    float sum[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = 0.f;
    if (j < seen) {
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        if (lane + 32 * k >= H) break;
        const float2 b = head[lane + 32 * k];
        // (a tile of -infinite scores only: they are less than 0)
        const float d = (m8[c][k] == -INFINITY ? 0.f : m8[c][k]) - b.x;
        const uint32_t w[4] = {v[c][k].x, v[c][k].y, v[c][k].z, v[c][k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = f16x2_floats(w[i]);
          sum[2 * i] = fmaf(ex2(f.x + d), b.y, sum[2 * i]);
          sum[2 * i + 1] = fmaf(ex2(f.y + d), b.y, sum[2 * i + 1]);
        }
      }
      __syncwarp();
      // lane l is left with block l / 4's sum
#pragma unroll
      for (int k = 0; k < 3; ++k) {
#pragma unroll
        for (int i = 0; i < (4 >> k); ++i) {
          const bool up = lane >> (4 - k) & 1;
          const float give = up ? sum[i] : sum[i + (4 >> k)], keep = up ? sum[i + (4 >> k)] : sum[i];
          sum[i] = keep + __shfl_xor_sync(0xffffffffu, give, 16 >> k);
        }
      }
      sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], 2);
      sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], 1);
    }
    const int jj = j + lane / 4;
    if ((lane & 3) == 0 && jj < p.max_blocks) {
      const float y = jj < seen ? sum[0] : -INFINITY;
      const int64_t at = (int64_t)x * p.max_blocks + jj;
      if (p.out_bf16) static_cast<uint16_t*>(p.out)[at] = (uint16_t)pack_bf16(y, 0.f);
      else static_cast<float*>(p.out)[at] = y;
    }
  }
}

}  // namespace

cudaError_t launch_block_scores(const ScoreParams& p, cudaStream_t s) {
  static std::atomic<uint64_t> configured;   // devices
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(configured.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(score_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(1ull << dev);
  }
  e = launch_dependent(score_kernel, dim3(kGrid), kThreads, kSmem, p, s);
  if (e != cudaSuccess) return e;
  // wider CTAs, which make the heads' sums less often, where narrow ones are more than two an SM (the whole call for 32
  // queries of 2048 blocks: 35.9 us, with 128 blocks a CTA 38.8; for 64 queries of 512 at most 22.5 and 20.7)
  const int spans = (p.max_blocks + kJoinBlocks - 1) / kJoinBlocks;
  if ((int64_t)spans * p.batch.rows <= 2 * kGrid) return launch_dependent(join_kernel<1>, dim3(spans, p.batch.rows), 32 * kJoinWarps, 0, p, s);
  return launch_dependent(join_kernel<4>, dim3((spans + 3) / 4, p.batch.rows), 32 * kJoinWarps, 0, p, s);
}

}  // namespace mla
