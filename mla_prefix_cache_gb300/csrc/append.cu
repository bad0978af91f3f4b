// Appending rows to the paged latent cache: the row [c_kv 512 | k_rope 64] of
// the down-projection becomes the cache row that attention reads,
//   c = x[0:512] / sqrt(mean(x[0:512]^2) + eps) * w     (w optional: x as it is)
//   k = R(pos) x[512:576], interleaved pairs (2k, 2k + 1) turned by pos theta^(-2k/64)
// stored as bf16 [c | k], or as E4M3 codes of c / kv_scale and bf16 k, at token
// seq_lens[r] - n_r + i of request r for its row i of n_r.  Sums and products
// are fp32; every stored value is rounded once, to nearest even.
//
// One warp takes a row: 16 latent values and one RoPE pair a lane, in 16-byte
// and 4-byte accesses that are contiguous over the warp.  HBM-bound: 1152 B
// read and 1152 (bf16) or 640 B (FP8) written a row.
#include "serving.cuh"

namespace mla {
namespace {

constexpr int kWarps = 8;

template <bool kFp8>
__global__ void __launch_bounds__(32 * kWarps) cache_append_kernel(const __grid_constant__ AppendParams p) {
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= p.batch.rows) return;
  const uint16_t* x = p.kv + (int64_t)row * p.row_stride;
  // latent values 8 l .. 8 l + 7 and 256 + 8 l .., RoPE pair l
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(x) + lane);
  const uint4 b = __ldg(reinterpret_cast<const uint4*>(x) + 32 + lane);
  const uint32_t kr = __ldg(reinterpret_cast<const uint32_t*>(x + kDc) + lane);
  const int pos = __ldg(p.pos + row);
  const int r = request_of_row(p.batch, row, lane);
  if (r < 0) return;
  const int2 rr = request_rows(p.batch, r);
  const int tok = __ldg(p.batch.seq_lens + r) - (rr.y - row);
  if (tok < 0) return;   // a padded request: its length does not hold this row
  const int lb = tok >> 6;
  const int id = lb < p.max_blocks ? __ldg(p.block_table + (int64_t)r * p.max_blocks + lb) : -1;
  if (id < 0 || id >= p.num_blocks) {
    if (lane == 0 && p.err != nullptr) atomicOr(p.err, kErrBadBlock);
    return;
  }

  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float v[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
  if (p.norm_weight != nullptr) {
    const uint4 ga = __ldg(reinterpret_cast<const uint4*>(p.norm_weight) + lane);
    const uint4 gb = __ldg(reinterpret_cast<const uint4*>(p.norm_weight) + 32 + lane);
    const uint32_t g[8] = {ga.x, ga.y, ga.z, ga.w, gb.x, gb.y, gb.z, gb.w};
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = fmaf(v[i], v[i], ss);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float inv = 1.f / sqrtf(ss * (1.f / kDc) + p.norm_eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[2 * i] *= inv * bf16_lo(g[i]);
      v[2 * i + 1] *= inv * bf16_hi(g[i]);
    }
  }
  float sn, cs;
  rope_sincos(pos, p.rope_frac[lane], &sn, &cs);
  const float x0 = bf16_lo(kr), x1 = bf16_hi(kr);
  const uint32_t k2 = pack_bf16(x0 * cs - x1 * sn, x0 * sn + x1 * cs);

  uint8_t* dst = p.cache + ((int64_t)id * kBlock + (tok & (kBlock - 1))) * (kFp8 ? kRowBytesFp8 : kRowBytesBf16);
  if constexpr (kFp8) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = (uint32_t)pack_e4m3x2(v[4 * i] / p.kv_scale, v[4 * i + 1] / p.kv_scale) |
             ((uint32_t)pack_e4m3x2(v[4 * i + 2] / p.kv_scale, v[4 * i + 3] / p.kv_scale) << 16);
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

}  // namespace

cudaError_t launch_cache_append(const AppendParams& p, bool fp8, cudaStream_t s) {
  if (p.batch.rows == 0) return cudaSuccess;
  const int grid = (p.batch.rows + kWarps - 1) / kWarps;
  if (fp8) cache_append_kernel<true><<<grid, 32 * kWarps, 0, s>>>(p);
  else cache_append_kernel<false><<<grid, 32 * kWarps, 0, s>>>(p);
  count_launch();
  return cudaGetLastError();
}

}  // namespace mla
