// Appending rows to the paged latent cache: the row [c_kv 512 | k_rope 64] of
// the down-projection becomes the cache row that attention reads,
//   c = x[0:512] / sqrt(mean(x[0:512]^2) + eps) * w     (w optional: x as it is)
//   k = R(pos) x[512:576], interleaved pairs (2k, 2k + 1) turned by pos theta^(-2k/64)
// stored as bf16 [c | k], or as E4M3 codes of c / kv_scale and bf16 k, at token
// seq_lens[r] - n_r + i of request r for its row i of n_r.  Sums and products
// are fp32; every stored value is rounded once, to nearest even.
//
// One warp takes some consecutive rows (one in a small batch), 16 latent values
// and one RoPE pair a lane, in 16-byte and 4-byte accesses that are contiguous
// over the warp.  The next row's loads are in flight while a row is computed,
// and a request and a block are looked up when they change only (a row with its
// own five dependent loads took 39 us for 62,731 FP8 rows, four rows a warp with
// all loads first and 100 registers 35).  HBM-bound: 1152 B read and 1152 (bf16)
// or 640 B (FP8) written a row.
#include "serving.cuh"

namespace mla {
namespace {

constexpr int kWarps = 8;
constexpr int kBlocksPerSm = 4;

struct Row {   // latent values 8 l .. 8 l + 7 and 256 + 8 l .., RoPE pair l
  uint4 a, b;
  uint32_t kr;
  int pos;
};
__device__ __forceinline__ Row load_row(const AppendParams& p, int row, int lane) {
  const uint16_t* x = p.kv + (int64_t)row * p.row_stride;
  Row r;
  r.a = __ldg(reinterpret_cast<const uint4*>(x) + lane);
  r.b = __ldg(reinterpret_cast<const uint4*>(x) + 32 + lane);
  r.kr = __ldg(reinterpret_cast<const uint32_t*>(x + kDc) + lane);
  r.pos = __ldg(p.pos + row);
  return r;
}

template <bool kFp8>
__global__ void __launch_bounds__(32 * kWarps, kBlocksPerSm) cache_append_kernel(const __grid_constant__ AppendParams p) {
  const int lane = threadIdx.x & 31;
  const int first = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * p.per_warp;
  const int end = min(first + p.per_warp, p.batch.rows);
  if (first >= end) {
    grid_wait();    // every CTA: the next dependent kernel counts on this grid's wait
    return;
  }
  grid_wait();      // launched dependently: the inputs are there
  grid_trigger();
  Row next = load_row(p, first, lane);
  uint4 ga = make_uint4(0, 0, 0, 0), gb = ga;
  const bool norm = p.norm_weight != nullptr;
  if (norm) {
    ga = __ldg(reinterpret_cast<const uint4*>(p.norm_weight) + lane);
    gb = __ldg(reinterpret_cast<const uint4*>(p.norm_weight) + 32 + lane);
  }
  const uint64_t frac = p.rope_frac[lane];
  int r = -1, past = first, len = 0;        // request, one past its last row, its tokens
  int lb = -1, id = -1;                     // block of the request, and its id
  for (int row = first; row < end; ++row) {
    const Row x = next;
    if (row + 1 < end) next = load_row(p, row + 1, lane);
    if (row >= past) {
      r = request_of_row(p.batch, row, lane);
      if (r < 0) {                          // no request's row: before the first one, or behind the last
        past = row + 1;
        id = -1;
        len = 0;
        lb = 0;
        continue;
      }
      past = request_rows(p.batch, r).y;
      len = __ldg(p.batch.seq_lens + r);
      lb = -1;
    }
    const int tok = len - (past - row);
    if (tok < 0) continue;                  // a padded request: its length does not hold this row
    if (tok >> 6 != lb) {
      lb = tok >> 6;
      id = lb < p.max_blocks ? __ldg(p.block_table + (int64_t)r * p.max_blocks + lb) : -1;
      if (id < 0 || id >= p.num_blocks) {
        id = -1;
        if (lane == 0 && p.err != nullptr) atomicOr(p.err, kErrBadBlock);
      }
    }
    if (id < 0) continue;
    const uint32_t w[8] = {x.a.x, x.a.y, x.a.z, x.a.w, x.b.x, x.b.y, x.b.z, x.b.w};
    float v[16];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[2 * k] = bf16_lo(w[k]);
      v[2 * k + 1] = bf16_hi(w[k]);
    }
    // E4M3 codes are of c times the reciprocal of kv_scale: the factor joins the norm's
    float f = kFp8 ? p.inv_scale : 1.f;
    if (norm) {
      const uint32_t g[8] = {ga.x, ga.y, ga.z, ga.w, gb.x, gb.y, gb.z, gb.w};
      float ss = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) ss = fmaf(v[k], v[k], ss);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      f *= rsqrtf(ss * (1.f / kDc) + p.norm_eps);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[2 * k] *= f * bf16_lo(g[k]);
        v[2 * k + 1] *= f * bf16_hi(g[k]);
      }
    } else if (kFp8) {
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] *= f;
    }
    float sn, cs;
    rope_sincos_sfu(x.pos, frac, &sn, &cs);
    const float x0 = bf16_lo(x.kr), x1 = bf16_hi(x.kr);
    const uint32_t k2 = pack_bf16(x0 * cs - x1 * sn, x0 * sn + x1 * cs);

    uint8_t* dst = p.cache + ((int64_t)id * kBlock + (tok & (kBlock - 1))) * (kFp8 ? kRowBytesFp8 : kRowBytesBf16);
    if constexpr (kFp8) {
      uint32_t c[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        c[k] = (uint32_t)pack_e4m3x2(v[4 * k], v[4 * k + 1]) | ((uint32_t)pack_e4m3x2(v[4 * k + 2], v[4 * k + 3]) << 16);
      reinterpret_cast<uint2*>(dst)[lane] = make_uint2(c[0], c[1]);
      reinterpret_cast<uint2*>(dst)[32 + lane] = make_uint2(c[2], c[3]);
      reinterpret_cast<uint32_t*>(dst + kDc)[lane] = k2;
    } else {
      reinterpret_cast<uint4*>(dst)[lane] = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                       pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
      reinterpret_cast<uint4*>(dst)[32 + lane] = make_uint4(pack_bf16(v[8], v[9]), pack_bf16(v[10], v[11]),
                                                            pack_bf16(v[12], v[13]), pack_bf16(v[14], v[15]));
      reinterpret_cast<uint32_t*>(dst + 2 * kDc)[lane] = k2;
    }
  }
}

}  // namespace

cudaError_t launch_cache_append(AppendParams p, bool fp8, cudaStream_t s) {
  if (p.batch.rows == 0) return cudaSuccess;
  // as many rows a warp as one wave of CTAs on a GB300's 152 SMs leaves it
  constexpr int kMostWarps = 152 * kBlocksPerSm * kWarps;
  p.per_warp = (p.batch.rows + kMostWarps - 1) / kMostWarps;
  const int grid = ((p.batch.rows + p.per_warp - 1) / p.per_warp + kWarps - 1) / kWarps;
  return launch_dependent(fp8 ? cache_append_kernel<true> : cache_append_kernel<false>, dim3(grid), 32 * kWarps, 0, p, s);
}

}  // namespace mla
