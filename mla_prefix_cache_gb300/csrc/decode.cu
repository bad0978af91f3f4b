// Decode attention over the paged latent cache: one or a few new queries per
// request, lengths, block table and segments on the device.  In latent space
// ("DeepSeek MLA — Prefix Cache 与 Chunked Prefill 深度解析", section 3):
//   qlat_h = q_nope_h W_UK,h^T                                   (qabsorb_kernel, headproj.cu)
//   s_t = scale (qlat_h . c_t + R(pos - offset) q_rope_h . k_rope_t)
//   o_h = sum_t softmax(s)_t c_t                                  (decode_attn_kernel, here)
//   out_h = o_h W_UV,h;  lse = ln sum_t e^{s_t}                   (decode_out_kernel, decode_out.cu)
// so every cached row is read for all heads at once: 2 * 1088 FLOP per (row,
// query, key) against 1152 (bf16) or 640 B (FP8) per key.
//
// Work.  A request's (token, head) rows form items of 128 rows, an item's keys
// tiles of 128.  The tiles of all items, in order, with a few units for each
// item's start and end, are cut evenly over the clusters of a persistent grid,
// whatever the lengths are: a cluster has one contiguous run of tiles, the last
// part of one item, whole items, the first part of another.  A piece that is a
// whole item leaves its state as bf16 rows; the others leave fp32 states in the
// cluster's two slots, which decode_out_kernel joins.  The cut is computed by
// every CTA from the lengths (one pass of its threads over the requests), so no
// launch waits for a plan.
//
// A cluster is two CTAs, split by operation because O [128 x 512] fp32 fills a
// CTA's TMEM and Q [128 x 512] half of another's:
//  - CTA 0 (scores): Q in TMEM, its rotated q_rope in shared memory; per tile
//    S = Q [c | k_rope]^T (M = 128, N = 128) into one of two TMEM buffers, the
//    running softmax of one row a thread, and P with the rows' rescale factors
//    staged and copied in bulk into the other CTA.
//  - CTA 1 (values): O += P c (M = 128, N = 256 twice), rows rescaled in TMEM
//    when their maximum rose by more than 2^8; at a piece's end O / l leaves.
// Each CTA reads the cache's blocks in place by TMA, the scores as rows of all
// 128 keys in blocks of 128 B, the values 32 KB at a time.
//
// An FP8 cache is multiplied as it is stored, on kind::f8f6f4, without a
// conversion: what would be bf16 operands are two 8-bit terms each.  qlat is
// q8 + q8', E4M3 codes by the row's scale and of what they leave (relative
// error below 2^-8).  P is its value rounded to 2 mantissa bits in E5M2, whose
// range keeps weights down to 2^-24 of the largest, and the rest in E4M3
// (together below 2^-7, 1.3e-3 in the mean).  Two 8-bit MMAs take the time of
// one bf16 MMA on a cache of half the bytes.
#include "serving.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;   // warp 0: loads (scores: first half of a tile); 1: MMA; 2: TMEM; 3: loads of the
                                // second half (scores), P landed (values); 4-7: softmax or rescale and epilogue
constexpr uint32_t kBlk = 16384;                 // [128 rows x 128 B] swizzled block
// scores CTA: rotated q_rope, two P staging buffers, the ring
constexpr uint32_t kQR = 0;
constexpr uint32_t kPS = kBlk;
constexpr uint32_t kPBytes = 2 * kBlk;           // P of a tile: [128 x 128] bf16, or two 8-bit terms
constexpr uint32_t kSRing = kPS + 2 * kPBytes;
constexpr int kSStages = 3;
constexpr uint32_t kSStage = 3 * kBlk;           // three 128-byte blocks of 128 rows
// values CTA: two P tiles, the ring, two boxes for the epilogue
constexpr uint32_t kOP = 0;
constexpr uint32_t kORing = 2 * kPBytes;
constexpr int kOStages = 4;
constexpr uint32_t kOStage = 32768;              // 32 bf16 rows or 64 FP8 rows, without k_rope
constexpr uint32_t kOBox = kORing + kOStages * kOStage;
// both: per P buffer the rows' factors, sums and four rescale flags (staged and copied like P), then barriers
constexpr uint32_t kFac = kSRing + kSStages * kSStage;
static_assert(kFac == kOBox + 2 * kBlk, "the factors sit at one offset in both CTAs");
constexpr uint32_t kFacSum = 512, kFacFlags = 1024, kFacBytes = 1040;
constexpr uint32_t kBars = kFac + 2 * kFacBytes;
enum : uint32_t {
  // scores
  kSF = 0,      // 3: stage landed (two loading threads)
  kSE = 3,      // 3: the stage's MMAs are done
  kSSF = 6,     // 2: S buffer written
  kSSR = 8,     // 2: the 4 softmax warps have read the S buffer
  kQRd = 10,    // Q of the range in place (4 warps)
  kPFR = 11,    // 2: the PV of the P tile is done (from the values CTA)
  kSTF = 13,    // 2: a staging buffer's last copy landed (from the values CTA)
  // values
  kCF = 15,     // 4: stage landed
  kCE = 19,     // 4: the stage's MMAs are done
  kPF = 23,     // 2: P tile, factors and flags landed
  kPVD = 25,    // 2: PV of the tile done
  kCN = 27,     // the control warp handed a tile, or a piece's end, to the correction warps
  kCD = 28,     // the 4 correction warps rescaled their rows (piece's end: have read the sums)
  kEP = 29,     // the 4 correction warps have read the piece's O
  kNBars = 30
};
constexpr uint32_t kShared = kBars + 8 * kNBars;   // Start, then the hand-over word
constexpr uint32_t kHand = kShared + 64;
constexpr uint32_t kSmem = kHand + 16;
static_assert(kSmem <= 232448, "more than 227 KB of shared memory per CTA");
constexpr uint32_t kTxP = kPBytes + kFacBytes;

constexpr uint32_t kIdS = idesc_bf16(128, 128, false, false);
constexpr uint32_t kIdPV = idesc_bf16(128, 256, false, true);
constexpr uint32_t kIdS8 = idesc_8bit(128, 128, 0, 0, false);
constexpr uint32_t kIdPV8 = idesc_8bit(128, 256, 1, 0, true);     // E5M2 P
constexpr uint32_t kIdPV8r = idesc_8bit(128, 256, 0, 0, true);    // E4M3 rest of P
constexpr float kRescale = 8.f;   // log2 units: P stays <= 256

// Where a cluster's run of units begins: in request r, whose first unit is `first`.
struct Start {
  int64_t begin, end, first, total;
  int r, n;      // n: clusters in use
  uint32_t tmem;
};

// The units of all requests, and this cluster's run.  Every thread of the CTA;
// thread t takes requests [t k, (t + 1) k).  CTA 0 of the grid leaves the
// requests' first units for decode_out_kernel and reports cut sequences.
__device__ void schedule(const DecodeParams& p, Start* st, int64_t* scratch, int cluster) {
  const int B = p.batch.rows.num_reqs, k = (B + kThreads - 1) / kThreads;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r0 = min(B, tid * k), r1 = min(B, r0 + k);
  int64_t sum = 0;
  for (int r = r0; r < r1; ++r) {
    const RequestWork w = request_work(p.batch, r);
    sum += (int64_t)w.units() * w.items;
    if (blockIdx.x == 0 && __ldg(p.batch.rows.seq_lens + r) > p.batch.max_blocks * kBlock) atomicOr(p.ws.err, kErrBadBlock);
  }
  int64_t pre = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, pre, o);
    if (lane >= o) pre += v;
  }
  if (lane == 31) scratch[warp] = pre;
  __syncthreads();
  int64_t total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) pre += scratch[w];
    total += scratch[w];
  }
  pre -= sum;   // units of the requests before r0
  const int64_t n = total < (int64_t)(gridDim.x / 2) ? total : (int64_t)(gridDim.x / 2);
  const int64_t begin = cluster < n ? unit_begin(cluster, n, total) : total;
  if (tid == 0) {
    st->begin = begin;
    st->end = cluster < n ? unit_begin(cluster + 1, n, total) : total;
    st->total = total;
    st->n = (int)n;
    st->r = B;
    if (blockIdx.x == 0) {
      p.ws.first[B] = total;
      p.ws.first[B + 1] = total;
      p.ws.first[B + 2] = n;
    }
  }
  __syncthreads();
  const bool mine = begin >= pre && begin < pre + sum;
  if (mine || blockIdx.x == 0) {
    int64_t at = pre;
    bool found = false;
    for (int r = r0; r < r1; ++r) {
      const RequestWork w = request_work(p.batch, r);
      if (blockIdx.x == 0) p.ws.first[r] = at;
      const int64_t next = at + (int64_t)w.units() * w.items;
      if (mine && !found && begin < next) {
        found = true;
        st->r = r;
        st->first = at;
      }
      at = next;
    }
  }
  __syncthreads();
}

// A piece: tiles [lo, hi) of one item.
struct Piece {
  RequestWork w;
  int r, row0, lo, hi, slot;   // slot -1: the whole item
};
// The pieces of a cluster's run in order, walked alike by every role.
struct Pieces {
  RequestWork w;
  int64_t at, end;   // next unit, one past the run's last
  int64_t first;     // first unit of request r
  int r, cluster;
  bool loaded;
  __device__ Pieces(const Start& s, int cluster_) : at(s.begin), end(s.end), first(s.first), r(s.r), cluster(cluster_), loaded(false) {}
  __device__ bool next(const DecodeParams& p, Piece& o) {
    while (at < end && r < p.batch.rows.num_reqs) {
      if (!loaded) {
        w = request_work(p.batch, r);
        loaded = true;
      }
      const int u = w.units();
      const int64_t past = first + (int64_t)u * w.items;
      if (at >= past) {   // also a request without units
        first = past;
        ++r;
        loaded = false;
        continue;
      }
      const int item = (int)((at - first) / u);
      const int64_t base = first + (int64_t)item * u;
      const int64_t stop = min(base + u, end);
      o.lo = (int)max((int64_t)0, at - base - kItemUnits);
      o.hi = (int)max((int64_t)0, stop - base - kItemUnits);
      at = stop;
      if (o.hi <= o.lo) continue;   // only units of the item's start
      o.w = w;
      o.r = r;
      o.row0 = item * kItemRows;
      o.slot = (o.lo == 0 && o.hi == w.tiles) ? -1 : 2 * cluster + (o.lo == 0 ? 1 : 0);
      return true;
    }
    return false;
  }
};

// The part of a piece with one RoPE offset: tiles j = 0 .. n - 1 from key t0 on, keys [k_lo, k_hi).
struct Run {
  int t0, n, k_lo, k_hi;
  int64_t offset;
};
struct Runs {
  int g, end, acc;
  __device__ explicit Runs(const Piece& o) : g(o.w.sg.x), end(0), acc(0) {}
  __device__ bool next(const DecodeParams& p, const Piece& o, Run& u) {
    while (g <= o.w.sg.y && acc < o.hi) {
      const KeyRange k = request_range(p.batch, o.w.sg, g, end, o.w.len);
      const int from = acc;
      end = k.hi;
      acc += range_tiles(k);
      ++g;
      const int lo = max(from, o.lo), hi = min(acc, o.hi);
      if (lo >= hi) continue;
      u.t0 = (k.lo & ~(kBlock - 1)) + 128 * (lo - from);
      u.n = hi - lo;
      u.k_lo = k.lo;
      u.k_hi = k.hi;
      u.offset = k.offset;
      return true;
    }
    return false;
  }
};

__device__ __forceinline__ bool await(const DecodeParams& p, uint32_t bar, uint32_t parity) {
  if (mbar_wait(bar, parity)) return true;
  atomicOr(p.ws.err, kErrTimeout);
  return false;
}
__device__ __forceinline__ bool await_warp(const DecodeParams& p, uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, await(p, bar, parity));
}

// The cache row of key token kt (in a block of its own: a multiple of the
// load's rows): a row before the map, which TMA reads as zeros, behind the
// run's last key and for a bad block id, which is reported.
__device__ __forceinline__ int cache_row(const DecodeParams& p, int r, int kt, int k_hi) {
  if (kt >= k_hi) return -kBlock;
  const int lb = kt >> 6;
  const int id = lb < p.batch.max_blocks ? __ldg(p.block_table + (int64_t)r * p.batch.max_blocks + lb) : -1;
  if (id < 0 || id >= p.num_blocks) {
    atomicOr(p.ws.err, kErrBadBlock);
    return -kBlock;
  }
  return id * kBlock + (kt & (kBlock - 1));
}

template <bool kFp8>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    decode_attn_kernel(const __grid_constant__ DecodeParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool scores = cluster_rank() == 0;
  const int cluster = blockIdx.x >> 1;
  const int H = p.batch.num_heads;
  auto bar = [&](uint32_t i) { return sb + kBars + 8u * i; };
  Start* start = reinterpret_cast<Start*>(smem + kShared);
  constexpr int kTileStages = kFp8 ? 2 : 3;   // scores: 128-byte blocks 3 m .. of [c | k_rope] a stage (9 or 5 in all)
  constexpr int kBlocks = kFp8 ? 5 : 9, kLatBlocks = kFp8 ? 4 : 8;
  constexpr int kORows = kFp8 ? 64 : 32, kOPerTile = 128 / kORows;

  if (tid == 0) {
    prefetch_tensormap(scores ? &p.tm_s : &p.tm_o);
    for (uint32_t i = 0; i < kNBars; ++i) {
      uint32_t cnt = 1;
      if (i < kSE) cnt = 2;
      else if (i == kSSR || i == kSSR + 1 || i == kQRd || i == kCD || i == kEP) cnt = 4;
      mbar_init(bar(i), cnt);
    }
    fence_mbar_init();
  }
  schedule(p, start, reinterpret_cast<int64_t*>(smem), cluster);
  cluster_sync_all();   // both CTAs' barriers exist before either is signalled
  if (warp == 2) {
    tmem_alloc(smem_u32(&start->tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&start->tmem);
  Pieces pieces(*start, cluster);
  Piece pc;
  Run run;

  if (scores) {
    if ((warp == 0 || warp == 3) && lane == 0) {
      // ---------------------------------------------------------- loads: 64 keys of each tile, all its blocks
      const int half = warp == 3 ? 1 : 0;
      bool ok = true;
      int u = 0;
      while (ok && pieces.next(p, pc)) {
        Runs runs(pc);
        while (ok && runs.next(p, pc, run)) {
          for (int j = 0; j < run.n && ok; ++j) {
            const int row = cache_row(p, pc.r, run.t0 + 128 * j + 64 * half, run.k_hi);
            for (int m = 0; m < kTileStages; ++m, ++u) {
              const int s = u % kSStages;
              if (u >= kSStages && !await(p, bar(kSE + s), ((u / kSStages) - 1) & 1)) {
                ok = false;
                break;
              }
              const int nb = min(3, kBlocks - 3 * m);
              mbar_arrive_expect_tx(bar(kSF + s), (uint32_t)nb * (kBlk / 2));
              for (int b = 0; b < nb; ++b)
                tma_load_3d(sb + kSRing + s * kSStage + b * kBlk + half * (kBlk / 2), &p.tm_s, 0, row, 3 * m + b,
                            bar(kSF + s));
            }
          }
        }
      }
      // the last commits land before this CTA exits
      for (int v = max(0, u - kSStages); v < u && ok; ++v) ok = await(p, bar(kSE + v % kSStages), (v / kSStages) & 1);
    } else if (warp == 1) {
      // ---------------------------------------------------------- S = Q [c | k_rope]^T
      bool ok = true;
      const uint64_t qd = sdesc_sw128(sb + kQR, 16, 1024);
      const uint64_t sd0 = sdesc_sw128(sb + kSRing, 16, 1024);
      int g = 0, s = 0, e = 0;
      uint32_t ph = 0;
      while (ok && pieces.next(p, pc)) {
        Runs runs(pc);
        while (ok && runs.next(p, pc, run)) {
          if (!await_warp(p, bar(kQRd), e++ & 1)) { ok = false; break; }
          for (int j = 0; j < run.n && ok; ++j, ++g) {
            const int b = g & 1;
            if (g >= 2 && !await_warp(p, bar(kSSR + b), ((g >> 1) - 1) & 1)) { ok = false; break; }
            const uint32_t d = tmem + 256 + 128 * b;
#pragma unroll
            for (int m = 0; m < kTileStages; ++m) {
              if (!await_warp(p, bar(kSF + s), ph)) { ok = false; break; }
              tc_fence_after();
              const uint64_t sd = sdesc_add(sd0, s * kSStage);
#pragma unroll
              for (int kb = 0; kb < 3; ++kb) {
                const int blk = 3 * m + kb;
                if (blk >= kBlocks) break;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                  const uint64_t bd = sdesc_add(sd, kb * kBlk + kk * 32);
                  const uint32_t acc = (blk | kk) ? 1u : 0u;
                  if (blk >= kLatBlocks) {
                    mma_ss_elect(d, sdesc_add(qd, kk * 32), bd, kIdS, 1u);
                  } else if (kFp8) {
                    mma_ts_8bit_elect(d, tmem + 32 * blk + 8 * kk, bd, kIdS8, acc);
                    mma_ts_8bit_elect(d, tmem + 128 + 32 * blk + 8 * kk, bd, kIdS8, 1u);
                  } else {
                    mma_ts_elect(d, tmem + 32 * blk + 8 * kk, bd, kIdS, acc);
                  }
                }
              }
              mma_commit_elect(bar(kSE + s));
              if (++s == kSStages) { s = 0; ph ^= 1u; }
            }
            if (ok) mma_commit_elect(bar(kSSF + b));
          }
        }
      }
    } else if (warp >= 4) {
      // ---------------------------------------------------------- Q into TMEM and shared memory; softmax
      const int r = tid - 128;
      const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t o_p = mapa_shared(sb + kOP, 1u), o_fac = mapa_shared(sb + kFac, 1u), o_pf = mapa_shared(bar(kPF), 1u);
      bool ok = true;
      int g = 0;
      while (ok && pieces.next(p, pc)) {
        const int prow = pc.row0 + r;
        const bool live = prow < pc.w.q_count * H;
        const int tl = live ? prow / H : 0;
        const int64_t grow = (int64_t)pc.w.q_begin + tl;
        const int64_t orow = (int64_t)pc.w.q_begin * H + prow;
        const float qs = kFp8 ? (live ? p.ws.qscale[orow] : 1.f) * p.kv_scale : 1.f;
        // qlat: every earlier score MMA is done (this warp has seen the last S buffer of the piece before)
        {
          const uint8_t* src = p.ws.qlat + orow * (kFp8 ? kDc : 2 * kDc);
          const int64_t second = kFp8 ? (int64_t)p.batch.rows.rows * H * kDc : kDc;   // TMEM columns 128 .. 255
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            const uint4* v4 = reinterpret_cast<const uint4*>(src + (i >> 1) * second + (i & 1) * 256);
            uint4 v[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) v[c] = live ? v4[c] : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              uint32_t w[32];
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                w[4 * c] = v[8 * hh + c].x; w[4 * c + 1] = v[8 * hh + c].y;
                w[4 * c + 2] = v[8 * hh + c].z; w[4 * c + 3] = v[8 * hh + c].w;
              }
              tmem_st32(tmem + lane_off + 64 * i + 32 * hh, w);
            }
          }
          tmem_wait_st();
        }
        const int qk = live ? pc.w.len - pc.w.q_count + tl : -1;   // the last key token the row sees
        const float sl2 = p.scale_log2 * qs;
        float m_used = -INFINITY, l = 0.f;
        Runs runs(pc);
        while (ok && runs.next(p, pc, run)) {
          {
            // q_rope turned by pos - offset, as a K-major swizzled block; FP8 scores count in units of qs,
            // so it is divided by that
            const uint4* qr = reinterpret_cast<const uint4*>(p.q + orow * kDqk + kDnope);
            const int64_t delta = live ? (int64_t)__ldg(p.q_pos + grow) - run.offset : 0;
            const float rq = 1.f / qs;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const uint4 qv = live ? __ldg(qr + c) : make_uint4(0, 0, 0, 0);
              const uint32_t w4[4] = {qv.x, qv.y, qv.z, qv.w};
              uint32_t o4[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float sn, cs;
                rope_sincos_sfu(delta, p.rope_frac[4 * c + i], &sn, &cs);
                const float x0 = bf16_lo(w4[i]), x1 = bf16_hi(w4[i]);
                o4[i] = pack_bf16((x0 * cs - x1 * sn) * rq, (x0 * sn + x1 * cs) * rq);
              }
              sts128(sb + kQR + sw128_off((uint32_t)r, (uint32_t)c), o4[0], o4[1], o4[2], o4[3]);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kQRd));
          }
          for (int j = 0; j < run.n; ++j, ++g) {
            const int b = g & 1;
            uint32_t v0[64], v1[64];
            float mx = -INFINITY;
            bool wok = await_warp(p, bar(kSSF + b), (g >> 1) & 1);
            tc_fence_after();
            if (wok) {
              const float m0 = tmem_ld64_max(tmem + lane_off + 256 + 128 * b, v0);
              const float m1 = tmem_ld64_max(tmem + lane_off + 256 + 128 * b + 64, v1);
              mx = fmaxf(m0, m1);
            }
            tc_fence_before();
            __syncwarp();
            // relaxed: the reads are ordered for the next MMAs by the tcgen05 fences around it
            if (lane == 0 && wok) mbar_arrive_relaxed(bar(kSSR + b));
            const int kt0 = run.t0 + 128 * j;
            if (!(kt0 >= run.k_lo && kt0 + 127 < run.k_hi && kt0 + 127 <= qk)) {
              const int hi = min(run.k_hi - 1, qk) - kt0, lo = run.k_lo - kt0;   // visible columns lo .. hi
              float m8[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) m8[i] = -INFINITY;
#pragma unroll
              for (int c = 0; c < 64; ++c) {
                const float xa = (c >= lo && c <= hi) ? __uint_as_float(v0[c]) : -INFINITY;
                const float xb = (c + 64 >= lo && c + 64 <= hi) ? __uint_as_float(v1[c]) : -INFINITY;
                v0[c] = __float_as_uint(xa);
                v1[c] = __float_as_uint(xb);
                m8[c & 7] = fmax3(m8[c & 7], xa, xb);
              }
              mx = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])), fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
            }
            const float m_tile = mx * sl2;
            float alpha = 1.f;
            if (m_tile > m_used + kRescale) {
              alpha = ex2(m_used - m_tile);   // 0 when m_used = -inf
              m_used = m_tile;
            }
            const float mref = (m_used == -INFINITY) ? 0.f : m_used;
            const uint64_t sc2 = f2pack(sl2, sl2), nm2 = f2pack(-mref, -mref);
            // P in registers while the previous tile's copy is still in flight: bf16 pairs, or per four keys a
            // word of E5M2 and a word of E4M3 codes
            uint64_t s4[4] = {0ull, 0ull, 0ull, 0ull};
            uint32_t pk[64];
            if (wok) {
#pragma unroll
              for (int c = 0; c < 64; ++c) {
                const uint32_t x0u = c < 32 ? v0[2 * c] : v1[2 * c - 64], x1u = c < 32 ? v0[2 * c + 1] : v1[2 * c - 63];
                float x0, x1;
                f2unpack(ffma2(f2pack(__uint_as_float(x0u), __uint_as_float(x1u)), sc2, nm2), x0, x1);
                const float a = ex2(x0), bb = ex2(x1);
                s4[c & 3] = fadd2(s4[c & 3], f2pack(a, bb));
                if constexpr (kFp8) {
                  // a value to 2 mantissa bits (half up), exact in E5M2 above 2^-14, and the rest
                  const float ah = __uint_as_float((__float_as_uint(a) + 0x00100000u) & 0xFFE00000u);
                  const float bh = __uint_as_float((__float_as_uint(bb) + 0x00100000u) & 0xFFE00000u);
                  const uint32_t h2 = pack_e5m2x2(ah, bh), r2 = pack_e4m3x2(a - ah, bb - bh);
                  if (c & 1) {
                    pk[c >> 1] |= h2 << 16;
                    pk[32 + (c >> 1)] |= r2 << 16;
                  } else {
                    pk[c >> 1] = h2;
                    pk[32 + (c >> 1)] = r2;
                  }
                } else {
                  pk[c] = pack_bf16(a, bb);
                }
              }
            }
            // the staging buffer is free once the copy it held two tiles ago landed; the four warps go on, or
            // leave, together
            if (wok && g >= 2) wok = await_warp(p, bar(kSTF + b), ((g - 2) >> 1) & 1);
            if (named_bar_or(1, 128, !wok)) { ok = false; break; }
            const uint32_t stg = sb + kPS + b * kPBytes;
#pragma unroll
            for (int hk = 0; hk < 2; ++hk)
#pragma unroll
              for (int c = 0; c < 8; ++c)
                sts128(stg + hk * kBlk + sw128_off((uint32_t)r, (uint32_t)c), pk[32 * hk + 4 * c],
                       pk[32 * hk + 4 * c + 1], pk[32 * hk + 4 * c + 2], pk[32 * hk + 4 * c + 3]);
            float s8[4];
            f2unpack(fadd2(s4[0], s4[1]), s8[0], s8[1]);
            f2unpack(fadd2(s4[2], s4[3]), s8[2], s8[3]);
            l = l * alpha + ((s8[0] + s8[2]) + (s8[1] + s8[3]));
            uint8_t* fac = smem + kFac + b * kFacBytes;
            reinterpret_cast<float*>(fac)[r] = alpha;
            reinterpret_cast<float*>(fac + kFacSum)[r] = l;
            const uint32_t any_rescale = __any_sync(0xffffffffu, alpha != 1.f) ? 1u : 0u;
            if (lane == 0) reinterpret_cast<uint32_t*>(fac + kFacFlags)[warp & 3] = any_rescale;
            fence_proxy_async_smem();   // the staged tile is read by the bulk copies (async proxy)
            named_bar_sync(1, 128);
            if (r == 0) {
              // P tile b of the values CTA is free once the PV of tile g - 2 is done
              if (g >= 2 && !await(p, bar(kPFR + b), ((g - 2) >> 1) & 1)) continue;   // the others time out next tile
              bulk_copy_to_peer(o_p + b * kPBytes, stg, kPBytes, o_pf + 8u * b);
              bulk_copy_to_peer(o_fac + b * kFacBytes, sb + kFac + b * kFacBytes, kFacBytes, o_pf + 8u * b);
            }
          }
        }
        if (live) {
          const float lse = (ok && l > 0.f) ? (m_used + __log2f(l)) * 0.6931471805599453f : -INFINITY;
          if (pc.slot < 0) p.ws.lat_lse[orow] = lse;
          else p.ws.part_lse[pc.slot * kItemRows + r] = lse;
        }
      }
      // the last two PV commits land before this CTA exits
      for (int v = max(0, g - 2); v < g && ok; ++v) ok = await_warp(p, bar(kPFR + (v & 1)), (v >> 1) & 1);
    }
  } else {
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- loads: latent columns of 32 (64) keys a stage
      bool ok = true;
      int u = 0;
      while (ok && pieces.next(p, pc)) {
        Runs runs(pc);
        while (ok && runs.next(p, pc, run)) {
          const int stages = kOPerTile * run.n;
          for (int i = 0; i < stages; ++i, ++u) {
            const int s = u % kOStages;
            const int row = cache_row(p, pc.r, run.t0 + kORows * i, run.k_hi);
            if (u >= kOStages && !await(p, bar(kCE + s), ((u / kOStages) - 1) & 1)) { ok = false; break; }
            mbar_arrive_expect_tx(bar(kCF + s), kOStage);
            tma_load_3d(sb + kORing + s * kOStage, &p.tm_o, 0, row, 0, bar(kCF + s));
          }
        }
      }
      for (int v = max(0, u - kOStages); v < u && ok; ++v) ok = await(p, bar(kCE + v % kOStages), (v / kOStages) & 1);
    } else if (warp == 1) {
      // ---------------------------------------------------------- P landed, rows rescaled, O += P c
      volatile int* hand = reinterpret_cast<volatile int*>(smem + kHand);
      const uint64_t pd0 = sdesc_sw128(sb + kOP, 16, 1024);                        // P, K-major
      const uint64_t cd0 = sdesc_sw128(sb + kORing, kORows * 128, 1024);           // latent stages, MN-major
      bool ok = true;
      int g = 0, u = 0, events = 0, done = 0;   // tiles, stages, hand-overs, finished pieces
      if (lane == 0)
        for (int b = 0; b < 2; ++b) mbar_arrive_expect_tx(bar(kPF + b), kTxP);
      while (ok && pieces.next(p, pc)) {
        Runs runs(pc);
        int left = pc.hi - pc.lo;
        bool head = true;
        while (ok && runs.next(p, pc, run)) {
          for (int j = 0; j < run.n && ok; ++j, ++g, --left) {
            const int b = g & 1;
            if (!await_warp(p, bar(kPF + b), (g >> 1) & 1)) { ok = false; break; }
            if (!head) {
              uint32_t f[4];
              lds128(sb + kFac + b * kFacBytes + kFacFlags, f);
              if (f[0] | f[1] | f[2] | f[3]) {
                // O must hold the PV of every earlier tile before its rows are rescaled
                if (!await_warp(p, bar(kPVD + ((g - 1) & 1)), ((g - 1) >> 1) & 1)) { ok = false; break; }
                if (lane == 0) {
                  *hand = b;
                  mbar_arrive(bar(kCN));
                }
                if (!await_warp(p, bar(kCD), events++ & 1)) { ok = false; break; }
              }
            } else if (done > 0) {
              // the piece before has been read out of O
              if (!await_warp(p, bar(kEP), (done - 1) & 1)) { ok = false; break; }
            }
            if (left == 1) {
              // the row sums sit beside this P tile: read before the next tiles may replace them
              if (lane == 0) {
                *hand = 2 + b;
                mbar_arrive(bar(kCN));
              }
              if (!await_warp(p, bar(kCD), events++ & 1)) { ok = false; break; }
            }
            fence_proxy_async_smem();   // P was written by the other CTA's copy, the MMA reads it as an operand
            if (lane == 0) mbar_arrive_expect_tx_relaxed(bar(kPF + b), kTxP);
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < kOPerTile; ++i, ++u) {
              const int s = u & (kOStages - 1);
              if (!await_warp(p, bar(kCF + s), (u / kOStages) & 1)) { ok = false; break; }
              // rows outside the run meet P = 0, but may hold anything: they are zeroed
              const int kt = run.t0 + 128 * j + kORows * i;
              const int lo = max(0, run.k_lo - kt), hi = min(kORows, run.k_hi - kt);
              if ((lo > 0 || hi < kORows) && hi > 0) {
                for (int row = 0; row < kORows; ++row) {
                  if (row >= lo && row < hi) continue;
                  for (int c = lane; c < (int)(kOStage / kORows / 16); c += 32)
                    sts128(sb + kORing + s * kOStage + (c >> 3) * (kORows * 128) + row * 128 + (c & 7) * 16, 0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                __syncwarp();
              }
              tc_fence_after();
              const uint64_t cd = sdesc_add(cd0, s * kOStage);
#pragma unroll
              for (int kk = 0; kk < 2; ++kk) {
                const int k = 2 * i + kk;   // the tile's k-step: 16 keys (bf16) or 32 (FP8)
                const uint32_t acc = (head && k == 0) ? 0u : 1u;
#pragma unroll
                for (int nh = 0; nh < 2; ++nh) {
                  const uint64_t bd = sdesc_add(cd, nh * (kOStage / 2) + kk * (kORows * 64));
                  if (kFp8) {
                    mma_ss_8bit_elect(tmem + 256 * nh, sdesc_add(pd0, b * kPBytes + k * 32), bd, kIdPV8, acc);
                    mma_ss_8bit_elect(tmem + 256 * nh, sdesc_add(pd0, b * kPBytes + kBlk + k * 32), bd, kIdPV8r, 1u);
                  } else {
                    mma_ss_elect(tmem + 256 * nh, sdesc_add(pd0, b * kPBytes + (k >> 2) * kBlk + (k & 3) * 32), bd,
                                 kIdPV, acc);
                  }
                }
              }
              mma_commit_elect(bar(kCE + s));
            }
            if (!ok) break;
            head = false;
            mma_commit_elect(bar(kPVD + b));
            mma_commit_mc_elect(bar(kPFR + b), 0x1);
          }
        }
        ++done;
      }
      if (!ok && lane == 0) {
        *hand = -1;
        mbar_arrive(bar(kCN));
      }
    } else if (warp == 3 && lane == 0) {
      // ---------------------------------------------------------- each P tile landed: the scores CTA may stage the
      // tile after next.  The copy of tile g + 2 waits for this thread's signal of tile g, so the barrier's
      // phases never run ahead of this loop.
      const uint32_t stf = mapa_shared(bar(kSTF), 0u);
      int g = 0;
      bool ok = true;
      while (ok && pieces.next(p, pc))
        for (int j = pc.lo; j < pc.hi && ok; ++j, ++g) {
          ok = await(p, bar(kPF + (g & 1)), (g >> 1) & 1);
          if (ok) mbar_arrive_cluster_relaxed(stf + 8u * (g & 1));   // relaxed: a landed copy has read its source
        }
    } else if (warp >= 4) {
      // ---------------------------------------------------------- rescale O rows; epilogue
      const int r = tid - 128;
      const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
      const volatile int* hand = reinterpret_cast<const volatile int*>(smem + kHand);
      bool ok = true;
      int g = 0, ev = 0;
      while (pieces.next(p, pc)) {
        g += pc.hi - pc.lo;
        float lsum = 0.f;
        while (ok) {
          if (!await_warp(p, bar(kCN), ev++ & 1)) { ok = false; break; }
          const int h = *hand;
          if (h < 0) { ok = false; break; }
          if (h >= 2) {
            lsum = reinterpret_cast<const float*>(smem + kFac + (h - 2) * kFacBytes + kFacSum)[r];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kCD));
            break;
          }
          tc_fence_after();
          const float a = reinterpret_cast<const float*>(smem + kFac + h * kFacBytes)[r];
          if (__any_sync(0xffffffffu, a != 1.f)) {
#pragma unroll 1
            for (int cc = 0; cc < 16; ++cc) {
              uint32_t o[32];
              tmem_ld32(tmem + lane_off + 32 * cc, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
              tmem_st32(tmem + lane_off + 32 * cc, o);
            }
            tmem_wait_st();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kCD));
        }
        if (ok) ok = await_warp(p, bar(kPVD + ((g - 1) & 1)), ((g - 1) >> 1) & 1);
        if (named_bar_or(2, 128, !ok)) {   // the four warps leave together
          ok = false;
          break;
        }
        tc_fence_after();
        const float inv = lsum > 0.f ? 1.f / lsum : 0.f;
        const int prow = pc.row0 + r;
        const int rows = pc.w.q_count * H - pc.row0;      // live rows of the item
        const int64_t orow0 = (int64_t)pc.w.q_begin * H + pc.row0;
        const bool whole = pc.slot < 0;
        const bool full = rows >= kItemRows;
        // 128 live rows leave by TMA stores of staged 128-byte columns, fewer by their threads
#pragma unroll 1
        for (int cc = 0; cc < 16; ++cc) {
          uint32_t o[32];
          tmem_ld32(tmem + lane_off + 32 * cc, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
          if (cc == 15) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kEP));   // O has been read: the next piece may begin
          }
          if (whole) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = pack_bf16(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
            if (full) {
              const uint32_t box = sb + kOBox + (uint32_t)((cc >> 1) & 1) * kBlk;
              if ((cc & 1) == 0) {   // a box of 64 columns: its last store has read it
                if (r == 0) bulk_wait_read<1>();
                named_bar_sync(2, 128);
              }
#pragma unroll
              for (int c = 0; c < 4; ++c)
                sts128(box + sw128_off((uint32_t)r, (uint32_t)(4 * (cc & 1) + c)), w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
              if (cc & 1) {
                fence_proxy_async_smem();
                named_bar_sync(2, 128);
                if (r == 0) {
                  tma_store_2d(&p.tm_lat, box, 64 * (cc >> 1), (int)orow0);
                  bulk_commit();
                }
              }
            } else if (prow < pc.w.q_count * H) {
              uint4* dst = reinterpret_cast<uint4*>(p.ws.lat + (orow0 + r) * kDc + 32 * cc);
#pragma unroll
              for (int c = 0; c < 4; ++c) dst[c] = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
            }
          } else if (full) {
            const uint32_t box = sb + kOBox + (uint32_t)(cc & 1) * kBlk;
            if (r == 0) bulk_wait_read<1>();
            named_bar_sync(2, 128);
#pragma unroll
            for (int c = 0; c < 8; ++c)
              sts128(box + sw128_off((uint32_t)r, (uint32_t)c), o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
            fence_proxy_async_smem();
            named_bar_sync(2, 128);
            if (r == 0) {
              tma_store_2d(&p.tm_part, box, 32 * cc, pc.slot * kItemRows);
              bulk_commit();
            }
          } else if (r < rows) {
            uint4* dst = reinterpret_cast<uint4*>(p.ws.part + ((int64_t)pc.slot * kItemRows + r) * kDc + 32 * cc);
#pragma unroll
            for (int c = 0; c < 8; ++c) dst[c] = make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
          }
        }
      }
      if (r == 0) bulk_wait0();   // every store complete before the CTA's shared memory goes
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // nothing of the other CTA is under way into this one
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_decode_attn(const DecodeParams& p, bool fp8, cudaStream_t s) {
  static int configured = -1;
  static int clusters = kDecodeClusters;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured != dev) {
    e = cudaFuncSetAttribute(decode_attn_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(decode_attn_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    // as many clusters as are resident at once: the work is cut evenly over them
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(2 * kDecodeClusters);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int resident = 0;
    e = cudaOccupancyMaxActiveClusters(&resident, decode_attn_kernel<false>, &cfg);
    if (e != cudaSuccess) return e;
    clusters = resident < 1 ? 1 : resident < kDecodeClusters ? resident : kDecodeClusters;
    configured = dev;
  }
  if (fp8) decode_attn_kernel<true><<<2 * clusters, kThreads, kSmem, s>>>(p);
  else decode_attn_kernel<false><<<2 * clusters, kThreads, kSmem, s>>>(p);
  count_launch();
  return cudaGetLastError();
}

}  // namespace mla
