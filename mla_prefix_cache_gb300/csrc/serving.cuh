// Device helpers of the serving operators: the request of a row, a request's
// key ranges, E4M3 values.
#pragma once

#include "ptx.cuh"
#include "serving.h"

namespace mla {

// First row of request r and one past its last, clamped to the batch's rows.
__device__ __forceinline__ int2 request_rows(const BatchRows& b, int r) {
  if (b.cu_q == nullptr) return make_int2(r * b.per_req, (r + 1) * b.per_req);
  const int lo = min(max(__ldg(b.cu_q + r), 0), b.rows);
  return make_int2(lo, min(max(__ldg(b.cu_q + r + 1), lo), b.rows));
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

// Two E4M3 codes (low 16 bits) to floats, exactly.
__device__ __forceinline__ float2 e4m3x2_floats(uint32_t pair) {
  float2 f;
  asm("{\n\t.reg .b16 in, l, h;\n\t.reg .b32 hx;\n\t"
      "cvt.u16.u32 in, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 hx, in;\n\t"
      "mov.b32 {l, h}, hx;\n\t"
      "cvt.f32.f16 %0, l;\n\t"
      "cvt.f32.f16 %1, h;\n\t}"
      : "=f"(f.x), "=f"(f.y) : "r"(pair));
  return f;
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
__device__ __forceinline__ int2 request_segments(const DecodeParams& p, int r) {
  if (p.segments == nullptr) return make_int2(0, 0);
  const int lo = min(max(__ldg(p.seg_ptr + r), 0), p.num_segments);
  return make_int2(lo, min(max(__ldg(p.seg_ptr + r + 1), lo), p.num_segments));
}
// Range i of [sg.x, sg.y] (i == sg.y: the tail, from `end` on), clamped to
// [end, len): a segment never reaches back over the ones before it.
__device__ __forceinline__ KeyRange request_range(const DecodeParams& p, int2 sg, int i, int end, int len) {
  KeyRange k;
  if (i >= sg.y) {
    k.lo = min(end, len);
    k.hi = len;
    k.offset = 0;
    return k;
  }
  const int64_t s = __ldg(p.segments + 3 * (int64_t)i), n = __ldg(p.segments + 3 * (int64_t)i + 1);
  k.offset = __ldg(p.segments + 3 * (int64_t)i + 2);
  const int64_t lo = s < end ? (int64_t)end : s;
  const int64_t e = n <= 0 ? lo : (n > (int64_t)len - s ? (int64_t)len : s + n);   // no overflow for any s, n
  k.lo = (int)(lo < len ? lo : len);
  k.hi = (int)(e < k.lo ? k.lo : e);
  return k;
}

}  // namespace mla
