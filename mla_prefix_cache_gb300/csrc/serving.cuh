// Device helpers of the serving operators: the request of a row, a request's
// key ranges, E4M3 values.
#pragma once

#include "serving.h"
#include "serving_ptx.cuh"

namespace mla {

// Programmatic dependent launch: a kernel launched by launch_dependent may
// start once every CTA of the kernel before it in the stream has called
// grid_trigger() (or ended); grid_wait() in it returns when that one is done and
// its memory visible.  Each kernel here waits before it triggers, and every CTA
// waits: so what a dependent kernel reads before its own wait was there before
// the kernel that it depends on, and one wait covers all earlier kernels.  Nothing
// says that an SM's L1, which may hold what an earlier call found at the same
// address, is cleared before the wait: reads before it go to L2 (kL2).
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <class Params>
cudaError_t launch_dependent(void (*kernel)(Params), dim3 grid, int threads, size_t smem, const Params& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// First row of request r and one past its last, clamped to the batch's rows; kL2: see grid_wait.
template <bool kL2 = false>
__device__ __forceinline__ int2 request_rows(const BatchRows& b, int r) {
  if (b.cu_q == nullptr) return make_int2(r * b.per_req, (r + 1) * b.per_req);
  const int c0 = kL2 ? __ldcg(b.cu_q + r) : __ldg(b.cu_q + r), c1 = kL2 ? __ldcg(b.cu_q + r + 1) : __ldg(b.cu_q + r + 1);
  const int lo = min(max(c0, 0), b.rows);
  return make_int2(lo, min(max(c1, lo), b.rows));
}

// The request that row `row` belongs to, or -1 (behind the last request).  A
// whole warp searches the ascending cu_q 32 entries at a time: two dependent
// loads for up to 1024 requests.
__device__ __forceinline__ int request_of_row(const BatchRows& b, int row, int lane) {
  if (b.cu_q == nullptr) return row / b.per_req;
  int lo = 0, n = b.num_reqs;            // the request is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lane * step;
    // lane 0 always holds: the last lane whose request starts at or before the row
    const bool at = lane == 0 || (i < n && __ldg(b.cu_q + lo + i) <= row);
    const int k = 31 - __clz(__ballot_sync(0xffffffffu, at));
    lo += k * step;
    n = min(step, n - k * step);
  }
  const int2 rr = request_rows(b, lo);
  return row >= rr.x && row < rr.y ? lo : -1;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// A key range of a request that is attended with one RoPE offset.
struct KeyRange {
  int lo, hi;
  int64_t offset;
};
// Ranges of a request: its segments in order, then the keys behind the last
// segment's end (offset 0).
__device__ __forceinline__ int2 request_segments(const DecodeBatch& b, int r) {
  if (b.segments == nullptr) return make_int2(0, 0);
  const int lo = min(max(__ldg(b.seg_ptr + r), 0), b.num_segments);
  return make_int2(lo, min(max(__ldg(b.seg_ptr + r + 1), lo), b.num_segments));
}
// Range i of [sg.x, sg.y] (i == sg.y: the tail, from `end` on), clamped to
// [end, len): a segment never reaches back over the ones before it.
__device__ __forceinline__ KeyRange request_range(const DecodeBatch& b, int2 sg, int i, int end, int len) {
  KeyRange k;
  if (i >= sg.y) {
    k.lo = min(end, len);
    k.hi = len;
    k.offset = 0;
    return k;
  }
  const int64_t s = __ldg(b.segments + 3 * (int64_t)i), n = __ldg(b.segments + 3 * (int64_t)i + 1);
  k.offset = __ldg(b.segments + 3 * (int64_t)i + 2);
  const int64_t lo = s < end ? (int64_t)end : s;
  // neither sum leaves 64 bits: s >= 0 in the first, s < 0 < n or s + n <= len in the second
  const int64_t e = n <= 0 ? lo : (s >= 0 && n > (int64_t)len - s) ? (int64_t)len : s + n;
  k.lo = (int)(lo < len ? lo : len);
  k.hi = (int)(e < k.lo ? k.lo : e < len ? e : len);
  return k;
}
// 128-key tiles of a range: they start at the cache block that holds its first key.
__device__ __forceinline__ int range_tiles(const KeyRange& k) {
  return k.hi > k.lo ? (k.hi - (k.lo & ~(kBlock - 1)) + 127) >> 7 : 0;
}

// A request's share of the decode work.  Its rows (token * H + head) form items
// of 128 rows; an item has `tiles` key tiles and counts `units` = tiles +
// kItemUnits in the schedule (none if it has no keys).
constexpr int kItemUnits = 2;   // an item's start and end cost about as much as this many tiles
struct RequestWork {
  int q_begin, q_count, len, tiles, items;
  int2 sg;
  __device__ __forceinline__ int units() const { return tiles > 0 ? tiles + kItemUnits : 0; }
};
__device__ __forceinline__ RequestWork request_work(const DecodeBatch& b, int r) {
  RequestWork w;
  const int2 rr = request_rows(b.rows, r);
  w.q_begin = rr.x;
  w.q_count = rr.y - rr.x;
  w.len = min(max(__ldg(b.rows.seq_lens + r), 0), b.max_blocks * kBlock);
  w.sg = request_segments(b, r);
  w.items = (w.q_count * b.num_heads + kItemRows - 1) / kItemRows;
  if (w.sg.x == w.sg.y) {
    w.tiles = (w.len + 127) >> 7;
    return w;
  }
  w.tiles = 0;
  int end = 0;
#pragma unroll 1
  for (int g = w.sg.x; g <= w.sg.y; ++g) {
    const KeyRange k = request_range(b, w.sg, g, end, w.len);
    end = k.hi;
    w.tiles += range_tiles(k);
  }
  return w;
}

// The units [0, total) of the batch are cut evenly: cluster c of n has
// [unit_begin(c), unit_begin(c + 1)); cluster_of(x) is the one that has unit x.
// (The host keeps total below 2^31.)
__device__ __forceinline__ int unit_begin(int c, int n, int total) {   // floor(c total / n) in 32 bits: c <= n is small
  const int q = total / n;
  return c * q + c * (total - q * n) / n;
}
__device__ __forceinline__ int cluster_of(int x, int n, int total) { return (int)(((uint64_t)(x + 1) * (uint32_t)n - 1) / (uint32_t)total); }
// The slot of the state that cluster c has of a shared item, by whether it has
// the item's first tile: each cluster shares one item with the clusters before it
// at most, and one with those after it.
__device__ __forceinline__ int piece_slot(int c, bool first_tile) { return 2 * c + (first_tile ? 1 : 0); }

// A cluster's run of units, walked alike by every role, as ranges of key tiles
// with one RoPE offset: tiles j = 0 .. n - 1 of 128 keys from key t0 on, of
// which [k_lo, k_hi) count.  The ranges of a piece (a run of one item's tiles)
// follow one another, the first marked `head`, the last `tail`.  The query
// absorption's launch leaves each cluster's walk at its first range; a role's
// copy sits in shared memory, advanced by one of its threads.
struct Walk {
  // range
  int64_t offset;
  int t0, n, k_lo, k_hi;
  // its piece
  int r, row0, slot, rows;   // request, first row of the item, slot of its state (-1: a whole item), the request's rows
  RequestWork w;             // of request r
  // where the walk is
  int cluster, at, end, first;        // next unit, one past the run's last, first unit of request r
  int lo, hi, g, last_key, acc;   // the piece's tiles; next range, end of the keys so far, tiles so far
  bool more, head, tail;          // of the range (last here: they fill up a word)
  // run [begin, stop) of units, which begins in request q with its first unit f and work u
  __device__ __forceinline__ void start(int c, int begin, int stop, int q, int f, const RequestWork& u) {
    cluster = c;
    at = begin;
    end = stop;
    r = q;
    first = f;
    w = u;
    lo = hi = acc = 0;
  }
};
constexpr int kWalkWords = sizeof(Walk) / 4;
static_assert(sizeof(Walk) % 8 == 0 && sizeof(Walk) <= kWalkBytes, "a warp copies a walk in one step");

// Advances a walk to its next range; false at its end.
__device__ __forceinline__ bool next_range(const DecodeBatch& b, Walk& k) {
  k.head = false;
  while (k.acc >= k.hi) {   // the next piece
    while (true) {
      if (k.at >= k.end || k.r >= b.rows.num_reqs) return false;
      const int u = k.w.units();
      const int past = k.first + u * k.w.items;
      if (k.at >= past) {   // also a request without units
        k.first = past;
        if (++k.r < b.rows.num_reqs) k.w = request_work(b, k.r);
        continue;
      }
      const int item = k.at - k.first < u ? 0 : (k.at - k.first) / u;
      const int base = k.first + item * u;
      const int stop = min(base + u, k.end);
      k.lo = max(0, k.at - base - kItemUnits);
      k.hi = max(0, stop - base - kItemUnits);
      k.at = stop;
      if (k.hi <= k.lo) continue;   // only units of the item's start
      k.row0 = item * kItemRows;
      k.slot = (k.lo == 0 && k.hi == k.w.tiles) ? -1 : piece_slot(k.cluster, k.lo == 0);
      break;
    }
    k.head = true;
    k.rows = k.w.q_count * b.num_heads;
    if (k.w.sg.x == k.w.sg.y) {   // no segments: one range
      k.t0 = 128 * k.lo;
      k.n = k.hi - k.lo;
      k.k_lo = 0;
      k.k_hi = k.w.len;
      k.offset = 0;
      k.tail = true;
      k.acc = k.hi;
      return true;
    }
    // ranges before the piece's first tile
    int g = k.w.sg.x, last = 0, acc = 0;
    const int len = k.w.len, lo = k.lo;
    const int2 sg = k.w.sg;
#pragma unroll 1
    for (; g <= sg.y; ++g) {
      const KeyRange kr = request_range(b, sg, g, last, len);
      const int t = range_tiles(kr);
      if (acc + t > lo) break;
      acc += t;
      last = kr.hi;
    }
    k.g = g;
    k.last_key = last;
    k.acc = acc;
  }
  while (true) {   // the next range with tiles: the piece's tiles say there is one
    const KeyRange kr = request_range(b, k.w.sg, k.g, k.last_key, k.w.len);
    const int t = range_tiles(kr), from = k.acc;
    k.last_key = kr.hi;
    k.acc += t;
    ++k.g;
    const int lo = max(from, k.lo), hi = min(k.acc, k.hi);
    if (lo >= hi) continue;
    k.t0 = (kr.lo & ~(kBlock - 1)) + 128 * (lo - from);
    k.n = hi - lo;
    k.k_lo = kr.lo;
    k.k_hi = kr.hi;
    k.offset = kr.offset;
    k.tail = k.acc >= k.hi;
    return true;
  }
}

}  // namespace mla
