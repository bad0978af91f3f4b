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
// over the warp, with the next row's loads in flight while a row is computed.
// Rows of one block of one request are a run: the request and the block are
// looked up between runs, and the loop over a run's rows reads no parameters.
// HBM-bound in principle: 1152 B read and 1152 (bf16) or 640 B (FP8) written a
// row.  62,731 FP8 rows (112 MB, 16.6 us at the copy rate) take 20.9 us, 5.4
// TB/s; what it takes beyond that is issue slots (about 200 instructions a row
// and warp) and the rows' latency:
//   a row a warp, its five loads dependent                              39 us
//   four rows a warp, all loads first (100 registers)                   35
//   consecutive rows, the next one in flight, look-ups when they change 27
//   runs (their loop had waited for parameters)                         22
//   norm weights as floats in shared memory, packed arithmetic          20.9
// Two rows in flight, or five through shared memory, gained nothing (23.5, 28
// against 22, 27); 3 and 5 CTAs an SM take 23.1 and 22.2.
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
// x: the row's element 8 l
__device__ __forceinline__ Row load_row(const uint16_t* x, const int32_t* pos, int lane) {
  Row r;
  r.a = __ldg(reinterpret_cast<const uint4*>(x));
  r.b = __ldg(reinterpret_cast<const uint4*>(x + 256));
  r.kr = __ldg(reinterpret_cast<const uint32_t*>(x + kDc - 6 * lane));
  r.pos = __ldg(pos);
  return r;
}

template <bool kFp8>
__global__ void __launch_bounds__(32 * kWarps, kBlocksPerSm) cache_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kRow = kFp8 ? kRowBytesFp8 : kRowBytesBf16;
  const int lane = threadIdx.x & 31;
  const int first = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * p.per_warp;
  const int end = min(first + p.per_warp, p.batch.rows);
  if (first >= end) {
    grid_wait();    // every CTA: the next dependent kernel counts on this grid's wait
    return;
  }
  grid_wait();      // launched dependently: the inputs are there
  grid_trigger();
  const int64_t stride = p.row_stride;
  const uint16_t* x = p.kv + first * stride + 8 * lane;    // of the next row to load
  const int32_t* xpos = p.pos + first;
  Row next = load_row(x, xpos, lane);
  const bool norm = p.norm_weight != nullptr;
  // the lane's 16 norm weights (1 without a norm) as floats, in places that only it uses
  __shared__ float4 weights[kWarps][4][32];
  float4(&g)[4][32] = weights[threadIdx.x >> 5];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint4 w = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
    if (norm) w = __ldg(reinterpret_cast<const uint4*>(p.norm_weight) + 32 * k + lane);
    g[2 * k][lane] = make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
    g[2 * k + 1][lane] = make_float4(bf16_lo(w.z), bf16_hi(w.z), bf16_lo(w.w), bf16_hi(w.w));
  }
  const uint64_t frac = p.rope_frac[lane];
  // E4M3 codes are of c times the reciprocal of kv_scale: the factor joins the norm's
  const float scale = kFp8 ? p.inv_scale : 1.f, eps = p.norm_eps;
  int r = -1, past = first, len = 0;        // request, one past its last row, its tokens
  for (int row = first; row < end;) {
    // the rows up to `stop` go to one block of one request, or nowhere
    if (row >= past) {
      r = request_of_row(p.batch, row, lane);
      past = row + 1;                       // no request's row: before the first one, or behind the last
      if (r >= 0) {
        past = request_rows(p.batch, r).y;
        len = max(__ldg(p.batch.seq_lens + r), 0);   // (so that no token index below leaves 32 bits)
      }
    }
    int stop = min(past, end);
    const int tok = len - (past - row);
    uint8_t* dst = nullptr;
    if (r >= 0 && tok >= 0) {               // (a padded request: its length does not hold this row)
      stop = min(stop, row + kBlock - (tok & (kBlock - 1)));
      const int lb = tok >> 6;
      const int id = lb < p.max_blocks ? __ldg(p.block_table + (int64_t)r * p.max_blocks + lb) : -1;
      if (id >= 0 && id < p.num_blocks) dst = p.cache + ((int64_t)id * kBlock + (tok & (kBlock - 1))) * kRow;
      else if (lane == 0 && p.err != nullptr) atomicOr(p.err, kErrBadBlock);
    } else if (r >= 0) {
      stop = min(stop, row - tok);
    }
    if (dst == nullptr) {                   // left out
      const int n = stop - row;
      row = stop;
      if (row < end) {
        x += n * stride;
        xpos += n;
        next = load_row(x, xpos, lane);
      }
      continue;
    }
    dst += (kFp8 ? 8 : 16) * lane;
#pragma unroll 1
    for (; row < stop; ++row, dst += kRow) {
      const Row q = next;
      if (row + 1 < end) {
        x += stride;
        ++xpos;
        next = load_row(x, xpos, lane);
      }
      const uint32_t w[8] = {q.a.x, q.a.y, q.a.z, q.a.w, q.b.x, q.b.y, q.b.z, q.b.w};
      uint64_t v2[8];                       // pairs
#pragma unroll
      for (int k = 0; k < 8; ++k) v2[k] = f2pack(bf16_lo(w[k]), bf16_hi(w[k]));
      float f = scale;
      if (norm) {
        uint64_t s2 = 0ull;
#pragma unroll
        for (int k = 0; k < 8; ++k) s2 = ffma2(v2[k], v2[k], s2);
        float ss, s1;
        f2unpack(s2, ss, s1);
        ss += s1;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        f *= rsqrtf(ss * (1.f / kDc) + eps);
      }
      float v[16];
#pragma unroll
      for (int k = 0; k < 4; ++k) {         // without a norm, times 1
        const float4 gk = g[k][lane];
        f2unpack(fmul2(v2[2 * k], fmul2(f2pack(gk.x, gk.y), f2pack(f, f))), v[4 * k], v[4 * k + 1]);
        f2unpack(fmul2(v2[2 * k + 1], fmul2(f2pack(gk.z, gk.w), f2pack(f, f))), v[4 * k + 2], v[4 * k + 3]);
      }
      float sn, cs;
      rope_sincos_sfu(q.pos, frac, &sn, &cs);
      const float x0 = bf16_lo(q.kr), x1 = bf16_hi(q.kr);
      const uint32_t k2 = pack_bf16(x0 * cs - x1 * sn, x0 * sn + x1 * cs);
      if constexpr (kFp8) {
        uint32_t c[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          c[k] = (uint32_t)pack_e4m3x2(v[4 * k], v[4 * k + 1]) | ((uint32_t)pack_e4m3x2(v[4 * k + 2], v[4 * k + 3]) << 16);
        *reinterpret_cast<uint2*>(dst) = make_uint2(c[0], c[1]);
        *reinterpret_cast<uint2*>(dst + 256) = make_uint2(c[2], c[3]);
        *reinterpret_cast<uint32_t*>(dst + kDc - 4 * lane) = k2;
      } else {
        *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                    pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
        *reinterpret_cast<uint4*>(dst + 512) = make_uint4(pack_bf16(v[8], v[9]), pack_bf16(v[10], v[11]),
                                                          pack_bf16(v[12], v[13]), pack_bf16(v[14], v[15]));
        *reinterpret_cast<uint32_t*>(dst + 2 * kDc - 12 * lane) = k2;
      }
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
