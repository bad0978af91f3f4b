// Appending rows to the paged latent cache: the row [c_kv 512 | k_rope 64] of
// the down-projection becomes the cache row that attention reads,
//   c = x[0:512] / sqrt(mean(x[0:512]^2) + eps) * w     (w optional: x as it is)
//   k = R(pos) x[512:576], interleaved pairs (2k, 2k + 1) turned by pos theta^(-2k/64)
// stored as bf16 [c | k], or as E4M3 codes of c / kv_scale and bf16 k, at token
// seq_lens[r] - n_r + i of request r for its row i of n_r.  Sums and products
// are fp32; every stored value is rounded once, to nearest even.
//
// One warp takes a row, 16 latent values and one RoPE pair a lane, in 16-byte
// and 4-byte accesses that are contiguous over the warp; large batches give a
// warp four rows, all of whose loads are issued before the first row's request
// and block are looked up (five dependent loads, which a wave of short warps
// would pay each).  HBM-bound: 1152 B read and 1152 (bf16) or 640 B (FP8)
// written a row.
#include "serving.cuh"

namespace mla {
namespace {

constexpr int kWarps = 8;
constexpr int kManyRows = 8192;   // from here on a warp takes four rows

template <bool kFp8, int kRows>
__global__ void __launch_bounds__(32 * kWarps) cache_append_kernel(const __grid_constant__ AppendParams p) {
  const int lane = threadIdx.x & 31;
  const int row0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * kRows;
  const int n = min(kRows, p.batch.rows - row0);
  if (n <= 0) return;
  // latent values 8 l .. 8 l + 7 and 256 + 8 l .., RoPE pair l
  uint4 a[kRows], b[kRows];
  uint32_t kr[kRows];
  int pos[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (i < n) {
      const uint16_t* x = p.kv + (int64_t)(row0 + i) * p.row_stride;
      a[i] = __ldg(reinterpret_cast<const uint4*>(x) + lane);
      b[i] = __ldg(reinterpret_cast<const uint4*>(x) + 32 + lane);
      kr[i] = __ldg(reinterpret_cast<const uint32_t*>(x + kDc) + lane);
      pos[i] = __ldg(p.pos + row0 + i);
    }
  }
  uint4 ga = make_uint4(0, 0, 0, 0), gb = ga;
  const bool norm = p.norm_weight != nullptr;
  if (norm) {
    ga = __ldg(reinterpret_cast<const uint4*>(p.norm_weight) + lane);
    gb = __ldg(reinterpret_cast<const uint4*>(p.norm_weight) + 32 + lane);
  }
  int r = request_of_row(p.batch, row0, lane);
  int2 rr = r >= 0 ? request_rows(p.batch, r) : make_int2(0, 0);
  int len = r >= 0 ? __ldg(p.batch.seq_lens + r) : 0;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int row = row0 + i;
    if (i >= n) break;
    if (i > 0 && row >= rr.y) {   // the next row's request
      r = request_of_row(p.batch, row, lane);
      if (r >= 0) {
        rr = request_rows(p.batch, r);
        len = __ldg(p.batch.seq_lens + r);
      }
    }
    if (r < 0) return;            // behind the last request, and so are the rows after it
    const int tok = len - (rr.y - row);
    if (tok < 0) continue;        // a padded request: its length does not hold this row
    const int lb = tok >> 6;
    const int id = lb < p.max_blocks ? __ldg(p.block_table + (int64_t)r * p.max_blocks + lb) : -1;
    if (id < 0 || id >= p.num_blocks) {
      if (lane == 0 && p.err != nullptr) atomicOr(p.err, kErrBadBlock);
      continue;
    }
    const uint32_t w[8] = {a[i].x, a[i].y, a[i].z, a[i].w, b[i].x, b[i].y, b[i].z, b[i].w};
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
    rope_sincos_sfu(pos[i], p.rope_frac[lane], &sn, &cs);
    const float x0 = bf16_lo(kr[i]), x1 = bf16_hi(kr[i]);
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

template <bool kFp8, int kRows>
void launch(const AppendParams& p, cudaStream_t s) {
  const int grid = (p.batch.rows + kWarps * kRows - 1) / (kWarps * kRows);
  cache_append_kernel<kFp8, kRows><<<grid, 32 * kWarps, 0, s>>>(p);
}

}  // namespace

cudaError_t launch_cache_append(const AppendParams& p, bool fp8, cudaStream_t s) {
  if (p.batch.rows == 0) return cudaSuccess;
  const bool many = p.batch.rows >= kManyRows;
  if (fp8) many ? launch<true, 4>(p, s) : launch<true, 1>(p, s);
  else many ? launch<false, 4>(p, s) : launch<false, 1>(p, s);
  count_launch();
  return cudaGetLastError();
}

}  // namespace mla
