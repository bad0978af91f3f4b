// Decode attention over the paged latent cache: one or a few new queries per
// request, lengths and block table on the device.  In latent space
// ("DeepSeek MLA — Prefix Cache 与 Chunked Prefill 深度解析", section 3):
//   qlat_h = q_nope_h W_UK,h^T;  s_t = scale (qlat_h . c_t + R(pos - offset) q_rope_h . k_rope_t)
//   o_h = sum_t softmax(s)_t c_t;  out_h = o_h W_UV,h;  lse = ln sum_t e^{s_t}
//
// The simple form: a CTA of four warps takes one (row, head), its warps take
// the keys in turn and keep a running maximum, sum and latent state each,
// joined at the end.  Every key is read from L2 once per head.
#include "serving.cuh"

namespace mla {
namespace {

constexpr int kDecodeWarps = 4;

template <bool kFp8>
__global__ void __launch_bounds__(32 * kDecodeWarps) decode_simple_kernel(const __grid_constant__ DecodeParams p) {
  __shared__ float q_s[kDqk], lat_s[kDc], rot_s[kDr];
  __shared__ float o_s[kDecodeWarps][kDc], m_s[kDecodeWarps], l_s[kDecodeWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x, row = blockIdx.y, H = p.num_heads;
  const int r = request_of_row(p.batch, row, lane);
  if (r < 0) return;
  const int2 rr = request_rows(p.batch, r);
  int len = __ldg(p.batch.seq_lens + r);
  if (len > p.max_blocks * kBlock) {
    if (tid == 0) atomicOr(p.err, kErrBadBlock);
    len = p.max_blocks * kBlock;
  }
  const int tok = len - (rr.y - row);      // this row's token: the last key it sees
  const int64_t orow = (int64_t)row * H + h;
  for (int i = tid; i < kDqk; i += 32 * kDecodeWarps)
    q_s[i] = __uint_as_float((uint32_t)__ldg(p.q + orow * kDqk + i) << 16);
  __syncthreads();
  const int64_t wcols = (int64_t)H * (kDnope + kDv);
  for (int c = tid; c < kDc; c += 32 * kDecodeWarps) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(p.kv_b_proj + c * wcols + h * kDnope);
    float a = 0.f;
    for (int d = 0; d < kDnope / 2; ++d) {
      const uint32_t w2 = __ldg(w + d);
      a = fmaf(q_s[2 * d], bf16_lo(w2), a);
      a = fmaf(q_s[2 * d + 1], bf16_hi(w2), a);
    }
    lat_s[c] = a;
  }
  float m = -INFINITY, l = 0.f, o[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = 0.f;
  const float vs = kFp8 ? p.kv_scale : 1.f;
  const int2 sg = request_segments(p, r);
  int end = 0;
  for (int g = sg.x; g <= sg.y; ++g) {
    const KeyRange kr = request_range(p, sg, g, end, max(len, 0));
    end = kr.hi;
    __syncthreads();
    if (tid < kDr / 2) {
      float sn, cs;
      rope_sincos((int64_t)__ldg(p.q_pos + row) - kr.offset, p.rope_frac[tid], &sn, &cs);
      const float x0 = q_s[kDnope + 2 * tid], x1 = q_s[kDnope + 2 * tid + 1];
      rot_s[2 * tid] = x0 * cs - x1 * sn;
      rot_s[2 * tid + 1] = x0 * sn + x1 * cs;
    }
    __syncthreads();
    for (int t = kr.lo + warp; t < min(kr.hi, tok + 1); t += kDecodeWarps) {
      const int id = __ldg(p.block_table + (int64_t)r * p.max_blocks + (t >> 6));
      const bool ok = id >= 0 && id < p.num_blocks;
      if (!ok && lane == 0) atomicOr(p.err, kErrBadBlock);
      const uint8_t* src = p.cache + ((int64_t)(ok ? id : 0) * kBlock + (t & 63)) * (kFp8 ? kRowBytesFp8 : kRowBytesBf16);
      float c[16], s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {        // pair 32 i + l of the latent
        float2 f;
        if constexpr (kFp8) {
          f = e4m3x2_floats(__ldg(reinterpret_cast<const uint16_t*>(src) + 32 * i + lane));
        } else {
          const uint32_t w2 = __ldg(reinterpret_cast<const uint32_t*>(src) + 32 * i + lane);
          f = make_float2(bf16_lo(w2), bf16_hi(w2));
        }
        c[2 * i] = ok ? f.x * vs : 0.f;
        c[2 * i + 1] = ok ? f.y * vs : 0.f;
        s = fmaf(c[2 * i], lat_s[64 * i + 2 * lane], s);
        s = fmaf(c[2 * i + 1], lat_s[64 * i + 2 * lane + 1], s);
      }
      const uint32_t k2 = ok ? __ldg(reinterpret_cast<const uint32_t*>(src + (kFp8 ? kDc : 2 * kDc)) + lane) : 0u;
      s = fmaf(bf16_lo(k2), rot_s[2 * lane], s);
      s = fmaf(bf16_hi(k2), rot_s[2 * lane + 1], s);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      s *= p.scale;
      const float mn = fmaxf(m, s);
      const float a = m == -INFINITY ? 0.f : expf(m - mn), e = mn == -INFINITY ? 0.f : expf(s - mn);
      m = mn;
      l = l * a + e;
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] = fmaf(e, c[i], o[i] * a);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    o_s[warp][64 * i + 2 * lane] = o[2 * i];
    o_s[warp][64 * i + 2 * lane + 1] = o[2 * i + 1];
  }
  if (lane == 0) {
    m_s[warp] = m;
    l_s[warp] = l;
  }
  __syncthreads();
  float mm = -INFINITY, ll = 0.f, f[kDecodeWarps];
  for (int w = 0; w < kDecodeWarps; ++w) mm = fmaxf(mm, m_s[w]);
  for (int w = 0; w < kDecodeWarps; ++w) {
    f[w] = m_s[w] == -INFINITY ? 0.f : expf(m_s[w] - mm);
    ll += f[w] * l_s[w];
  }
  const float inv = ll > 0.f ? 1.f / ll : 0.f;
  for (int c = tid; c < kDc; c += 32 * kDecodeWarps) {
    float a = 0.f;
    for (int w = 0; w < kDecodeWarps; ++w) a = fmaf(f[w], o_s[w][c], a);
    lat_s[c] = a * inv;
  }
  __syncthreads();
  float a = 0.f;
  const uint16_t* wv = p.kv_b_proj + (int64_t)H * kDnope + h * kDv + tid;
  for (int c = 0; c < kDc; ++c) a = fmaf(lat_s[c], __uint_as_float((uint32_t)__ldg(wv + c * wcols) << 16), a);
  if (p.out_bf16) reinterpret_cast<uint16_t*>(p.out)[orow * kDv + tid] = (uint16_t)pack_bf16(a, 0.f);
  else reinterpret_cast<float*>(p.out)[orow * kDv + tid] = a;
  if (p.lse != nullptr && tid == 0) p.lse[orow] = ll > 0.f ? mm + logf(ll) : -INFINITY;
}

}  // namespace

cudaError_t launch_decode(const DecodeParams& p, bool fp8, cudaStream_t s) {
  if (p.batch.rows == 0) return cudaSuccess;
  const dim3 grid(p.num_heads, p.batch.rows);
  if (fp8) decode_simple_kernel<true><<<grid, 32 * kDecodeWarps, 0, s>>>(p);
  else decode_simple_kernel<false><<<grid, 32 * kDecodeWarps, 0, s>>>(p);
  count_launch();
  return cudaGetLastError();
}

}  // namespace mla
