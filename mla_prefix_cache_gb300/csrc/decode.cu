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
// part of one item, whole items, the first part of another.  A piece leaves the
// fp32 states of its rows, a whole item's in the rows' own place, the others in
// the cluster's two slots, which decode_out_kernel joins.  The cut is computed on
// the device from the lengths, by a CTA of the query absorption's launch.
//
// A cluster is two CTAs, split by operation because O [128 x 512] fp32 fills a
// CTA's TMEM and Q [128 x 512] half of another's:
//  - CTA 0 (scores): Q in TMEM, its rotated q_rope in shared memory; per tile
//    S = Q [c | k_rope]^T (M = 128, N = 128) into one of two TMEM buffers, the
//    running softmax (two threads a row), and P with the rows' rescale factors
//    staged and copied in bulk into the other CTA.
//  - CTA 1 (values): O += P c (M = 128, N = 256 twice), rows rescaled in TMEM
//    when their maximum rose by more than 2^8 (FP8 2^4); at a piece's end O / l
//    leaves.
// Each CTA reads the cache's blocks in place by TMA, 16 KB a stage: the scores a
// block of 128 B of all 128 keys, the values half the columns of 32 or 64 keys.
//
// An FP8 cache is multiplied as it is stored, on kind::f8f6f4, without a
// conversion: what would be bf16 operands are two 8-bit terms each.  qlat is
// q8 + q8', E4M3 codes by the row's scale and of what they leave (relative
// error below 2^-8).  P is p + p', both E5M2, in units of 2^-11 of the largest
// weight: its value rounded to f16 and then to 2 mantissa bits, and what that
// leaves, together within 2^-7 of a weight (2.5e-3 rms) down to 2^-21 of the
// largest and 2^-28 of the largest below.  (An E4M3 p' halves that error, but its
// least step of 2^-9 leaves weights below 2^-10 of the largest with p alone, off
// by 5% rms: rows whose output is many small weights beside one of a small value
// were off by as much.)  O is divided by the sum of the weights as they are
// multiplied, so that an error that equal weights share does not stay; lse is
// made of their sum in fp32.  Two 8-bit MMAs take the time of one bf16 MMA on a
// cache of half the bytes.
//
// A bf16 cache's operands are qlat, q_rope and P rounded to bf16 once each: 2.0e-3
// of the output's norm together, where a bf16 output's own rounding is 1.7e-3.
// Second terms of Q (whose MMAs read every block of keys again) would add 1.1 us
// to a tile of 2.0, of P as much and 32 KB to copy.
//
// What bounds it.  A bf16 tile takes 1.9 to 2.0 us against 1.2 us of MMAs (36 of
// 64 cycles in one CTA, 16 of 128 in the other): in the scores CTA every tile
// moves about 375 KB through shared memory (147 KB written by TMA, read by the
// MMAs, P staged and copied), 76 clusters draw 5.4 TB/s of rows, and with the
// cache in L2 a tile is 8% faster only.  An FP8 tile takes 1.4 to 1.55 us, the
// MMAs 1.2 of them (tensor pipes busy 60% of a launch of 104 us, the start, the
// end and the handoffs the rest).  A launch begins with 4.3 us from its plan to
// the first scores (Q through registers into TMEM, then the first keys) and ends
// with 4 us for the last tile's chain and 6 us for 256 KB of fp32 states, at the
// 30 B a cycle that an SM stores to L2.  64 requests of 2K to 32K bf16 tokens, 128
// heads: 189 us with the kernels before and after; 64 of 4K to 16K FP8 tokens:
// 139 us.
#include <atomic>

#include "serving.cuh"

namespace mla {
namespace {

// Scores: warps 0, 3 load; 1: MMA; 2: TMEM, then the copies of P; 4-11: softmax,
// two threads a row; 12-15: Q.  Values: warps 0, 2 load; 1: MMA; 3: P landed;
// 4-11: rescale and epilogue, half the columns each.
constexpr int kThreads = 512;
constexpr uint32_t kBlk = 16384;                 // [128 rows x 128 B] swizzled block
// scores CTA: rotated q_rope, two P staging buffers, the ring
constexpr uint32_t kQR = 0;
constexpr uint32_t kPS = kBlk;
constexpr uint32_t kPBytes = 2 * kBlk;           // P of a tile: [128 x 128] bf16, or two 8-bit terms
constexpr uint32_t kSRing = kPS + 2 * kPBytes;
constexpr int kSStages = 9;                      // of one 128-byte block of 128 rows
// values CTA: two P tiles, the ring (whose stages also take the states that leave)
constexpr uint32_t kOP = 0;
constexpr uint32_t kORing = 2 * kPBytes;
constexpr int kOStages = 10;                     // even ones for columns 0 .. 255, odd ones for 256 .. 511
constexpr uint32_t kOStage = 16384;              // 256 latent columns of 32 bf16 rows or 64 FP8 rows
// both: per P buffer the rows' factors, sums and four rescale flags (staged and copied like P), then barriers
constexpr uint32_t kFac = kSRing + kSStages * kBlk;
static_assert(kFac == kORing + kOStages * kOStage, "the factors sit at one offset in both CTAs");
// (a flag word has the 32 rows' rescaling in its low byte, a key that is not finite in the others)
constexpr uint32_t kFacSum = 512, kFacFlags = 1024, kFacBytes = 1040;
constexpr uint32_t kBars = kFac + 2 * kFacBytes;
enum : uint32_t {
  // scores
  kSF = 0,      // 9: stage landed
  kSE = 9,      // 9: the stage has been read (its MMAs are done, or Q is in TMEM)
  kSSF = 18,    // 2: S buffer written
  kSSR = 20,    // 2: the 8 softmax warps have read the S buffer
  kQRd = 22,    // Q of the range in place (4 warps: qlat, 8 warps: q_rope)
  kQE = 23,     // the MMAs that read it are done
  kPST = 24,    // 2: P staged (8 warps)
  kPFR = 26,    // 2: the PV of the P tile is done (from the values CTA)
  kSTF = 28,    // 2: a staging buffer's last copy landed (from the values CTA)
  // values
  kCF = 0,      // 10: stage landed (or free for a box of states)
  kCE = 10,     // 10: the stage's MMAs are done (or its box has been read)
  kPF = 20,     // 2: P tile, factors and flags landed
  kPVD = 22,    // 2: PV of the tile done
  kCN = 24,     // the control warp handed a tile, or a piece's end, to the correction warps
  kCD = 25,     // the 8 correction warps rescaled their rows (piece's end: have read the sums)
  kEP = 26,     // the 8 correction warps have read the piece's O
  kNBars = 30
};
constexpr uint32_t kShared = kBars + 8 * kNBars;   // TMEM address, then the hand-over word
constexpr uint32_t kHand = kShared + 16;
constexpr uint32_t kWalks = kHand + 16;            // the roles' walks
constexpr int kRoles = 6;

constexpr uint32_t kIdS = idesc_bf16(128, 128, false, false);
constexpr uint32_t kIdPV = idesc_bf16(128, 256, false, true);
constexpr uint32_t kIdS8 = idesc_8bit(128, 128, 0, 0, false);
constexpr uint32_t kIdPV8 = idesc_8bit(128, 256, 1, 0, true);     // E5M2 terms of P
// Rows are rescaled when their maximum rises by more than this (log2 units).
// 8-bit terms of P: P counts in units of 2^-11, so that it spans 2^15, below
// E5M2's and f16's largest, down to E5M2's least step 2^-16.
constexpr float kRescaleBf16 = 8.f, kRescaleFp8 = 4.f;
constexpr float kPBiasFp8 = 11.f;

// Stages of each half of the columns that a piece's states leave through, if it has 32 live rows (fewer are written by
// their threads).
constexpr int kBoxes = 4;
__device__ __forceinline__ int boxes_of(const Walk& k) { return k.rows - k.row0 < 32 ? 0 : kBoxes; }

constexpr uint32_t kSmem = kWalks + kRoles * sizeof(Walk);
static_assert(kWalks % alignof(Walk) == 0 && kSmem <= 232448, "shared memory per CTA");

// One copy of this code serves every role: inlined into each, the kernel's code
// was 170 KB and its roles waited for instructions (1.5 times the time).
__device__ __noinline__ bool next(const DecodeParams& p, Walk& k) { return next_range(p.batch, k); }
// The next range of a walk (the first one is there already): by the one thread
// of a role, by a warp, by `count` threads at named barrier `id` (everyone is
// done with the range before).
__device__ __forceinline__ bool next_of_one(const DecodeParams& p, Walk& k, bool& first) {
  if (!first) return next(p, k);
  first = false;
  return *const_cast<volatile bool*>(&k.more);
}
__device__ __forceinline__ bool next_of_warp(const DecodeParams& p, Walk& k, bool& first, int lane) {
  if (!first) {
    __syncwarp();
    if (lane == 0) k.more = next(p, k);
    __syncwarp();
  }
  first = false;
  return *const_cast<volatile bool*>(&k.more);
}
__device__ __forceinline__ bool next_of_group(const DecodeParams& p, Walk& k, bool& first, bool leader, uint32_t id,
                                              uint32_t count) {
  if (!first) {
    named_bar_sync(id, count);
    if (leader) k.more = next(p, k);
  }
  first = false;
  named_bar_sync(id, count);
  return *const_cast<volatile bool*>(&k.more);
}

// Waits for a barrier's phase; false, and the error word, when it gives up.
__device__ __noinline__ bool await_long(const DecodeParams& p, uint32_t bar, uint32_t parity) {
  if (mbar_wait(bar, parity, p.wait_limit_ns)) return true;
  atomicOr(p.ws.err, kErrTimeout);
  return false;
}
__device__ __forceinline__ bool await(const DecodeParams& p, uint32_t bar, uint32_t parity) {
  return mbar_try_wait(bar, parity) || await_long(p, bar, parity);
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

// Zeroes all but rows [lo, hi) of a values stage, for the MMAs that this warp issues next.
template <int kRows>
__device__ __noinline__ void zero_rows(uint32_t stage, int lo, int hi, int lane) {
  for (int row = 0; row < kRows; ++row) {
    if (row >= lo && row < hi) continue;
    for (int c = lane; c < (int)(kOStage / kRows / 16); c += 32)
      sts128(stage + (c >> 3) * (kRows * 128) + row * 128 + (c & 7) * 16, 0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// The last key token that live row i of a request's rows sees.
__device__ __forceinline__ int last_key(const Walk& k, int i, int H) { return k.w.len - (k.rows - 1 - i) / H - 1; }

// Tile j of a range, whose P is in buffer b and whose values stages begin at s, of parity ph, may hold a key that is not
// finite and that some rows do not see: the 16-byte pieces of its latents that are not finite are zeroed, and bf16 rows
// that see such a key have NaN as its weight (an infinity with a score of -infinite has weight 0 so far; E4M3 has NaN
// only, which is in the score).  The ring holds a whole tile.
template <bool kFp8>
__device__ __noinline__ bool zero_not_finite(const DecodeParams& p, const Walk& k, int j, int b, uint32_t sb, int s,
                                             uint32_t ph, int lane) {
  constexpr uint32_t kOnes = kFp8 ? 0x7F7F7F7Fu : 0x7F807F80u;   // E4M3's NaN, bf16's exponent
  constexpr int kStages = 128 * 1024 / (kFp8 ? 2 : 1) / kOStage, kRows = kFp8 ? 64 : 32;
  static_assert(kStages <= kOStages, "a tile's stages");
  bool ok = true;
#pragma unroll 1
  for (int i = 0; i < kStages && ok; i += 2) {   // both halves of the columns of the same keys
    uint32_t bad = 0;                            // of the keys, 32 of them (bf16)
#pragma unroll 1
    for (int nh = 0; nh < 2 && ok; ++nh) {
      ok = await_warp(p, sb + kBars + 8 * (kCF + s), ph);
      const uint32_t stage = sb + kORing + s * kOStage;
#pragma unroll 1
      for (uint32_t at = 16 * lane; ok && at < kOStage; at += 512) {
        uint32_t w[4], any = 0;
        lds128(stage + at, w);
#pragma unroll
        for (int q = 0; q < 4; ++q) any |= kFp8 ? __vcmpeq4(w[q] & kOnes, kOnes) : __vcmpeq2(w[q] & kOnes, kOnes);
        if (any) {
          sts128(stage + at, 0u, 0u, 0u, 0u);
          bad |= 1u << ((at >> 7) % kRows & 31);
        }
      }
      if (++s == kOStages) { s = 0; ph ^= 1u; }
    }
    if (!kFp8) {
      bad = __reduce_or_sync(0xffffffffu, bad);
#pragma unroll 1
      for (; ok && bad; bad &= bad - 1) {
        const int key = (i >> 1) * kRows + __ffs(bad) - 1, kt = k.t0 + 128 * j + key;   // in the tile, its token
#pragma unroll 1
        for (int r = lane; kt >= k.k_lo && kt < k.k_hi && r < min(kItemRows, k.rows - k.row0); r += 32)
          if (kt <= last_key(k, k.row0 + r, p.batch.num_heads))
            asm volatile("st.shared.b16 [%0], %1;" ::"r"(sb + kOP + b * kPBytes + (key >> 6) * kBlk +
                                                         sw128_off((uint32_t)r, (uint32_t)(key & 63) >> 3) + 2 * (key & 7)),
                         "h"((uint16_t)0x7FC0)
                         : "memory");
      }
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
  return ok;
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
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kShared);
  constexpr int kBlocks = kFp8 ? 5 : 9, kLatBlocks = kFp8 ? 4 : 8;   // 128-byte blocks of a row [c | k_rope], of c
  constexpr int kQBoxes = 8;                                         // and of an item's Q
  constexpr int kORows = kFp8 ? 64 : 32, kOPerTile = 128 / kORows;   // key rows of a values stage

  if (tid == 0) {
    prefetch_tensormap(scores ? &p.tm_s : &p.tm_o);
    prefetch_tensormap(scores ? &p.tm_q : &p.tm_part);
    if (!scores) prefetch_tensormap(&p.tm_lat);
    for (uint32_t i = 0; i < kNBars; ++i) {
      uint32_t cnt = 1;
      if (scores) {
        if (i == kSSR || i == kSSR + 1 || i == kPST || i == kPST + 1) cnt = 8;
        else if (i == kQRd) cnt = 12;
      } else if (i == kCD || i == kEP) {
        cnt = 8;
      }
      mbar_init(bar(i), cnt);
    }
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  cluster_sync_all();   // both CTAs' barriers exist before either is signalled
  tc_fence_after();
  const uint32_t tmem = *const_cast<volatile uint32_t*>(tmem_slot);
  grid_wait();      // the plan, qlat and the inputs are there
  grid_trigger();   // decode_out_kernel may take SMs as they fall free
  // scores: loads 0, 1, MMA, copies, Q, softmax; values: loads 0, 1, MMA, P landed, -, rescale
  const int role = warp == 0 ? 0 : warp == (scores ? 3 : 2) ? 1 : warp == 1 ? 2 : warp < 4 ? 3 : warp >= 12 ? 4 : 5;
  Walk& k = reinterpret_cast<Walk*>(smem + kWalks)[role];
  bool first = true;
  if (lane < kWalkWords && (warp <= 4 || warp == 12))
    reinterpret_cast<uint32_t*>(&k)[lane] = __ldcg(p.ws.walks + kWalkBytes / 4 * cluster + lane);
  __syncwarp();

  if (scores) {
    if ((warp == 0 || warp == 3) && lane == 0) {
      // ---------------------------------------------------------- loads: an item's Q, then the blocks of its tiles,
      // every other stage a thread
      const int mine = warp == 3 ? 1 : 0;
      bool ok = true;
      int u = 0;
      // stage u's slot is free: arms its barrier
      auto open = [&]() {
        const int s = u % kSStages;
        if (u >= kSStages && !await(p, bar(kSE + s), ((u / kSStages) - 1) & 1)) return false;
        mbar_arrive_expect_tx(bar(kSF + s), kBlk);
        return true;
      };
      while (ok && cluster != p.withhold && next_of_one(p, k, first)) {
        const int qrow = k.w.q_begin * H + k.row0;
        for (int i = 0; k.head && i < kQBoxes; ++i, ++u) {
          if ((u & 1) != mine) continue;
          if (!(ok = open())) break;
          const int s = u % kSStages;
          if (kFp8) tma_load_2d(sb + kSRing + s * kBlk, &p.tm_q, 128 * (i & 3), qrow + (i >> 2) * p.batch.rows.rows * H, bar(kSF + s));
          else tma_load_2d(sb + kSRing + s * kBlk, &p.tm_q, 64 * i, qrow, bar(kSF + s));
        }
        for (int j = 0; j < k.n && ok; ++j) {
          const int kt = k.t0 + 128 * j;
          const int row0 = cache_row(p, k.r, kt, k.k_hi), row1 = cache_row(p, k.r, kt + 64, k.k_hi);
#pragma unroll 1
          for (int b = 0; b < kBlocks; ++b, ++u) {
            if ((u & 1) != mine) continue;
            if (!(ok = open())) break;
            const int s = u % kSStages;
            tma_load_3d(sb + kSRing + s * kBlk, &p.tm_s, 0, row0, b, bar(kSF + s));
            tma_load_3d(sb + kSRing + s * kBlk + kBlk / 2, &p.tm_s, 0, row1, b, bar(kSF + s));
          }
        }
      }
      // the last reads are signalled before this CTA exits
      for (int v = max(0, u - kSStages); v < u && ok; ++v) ok = await(p, bar(kSE + v % kSStages), (v / kSStages) & 1);
      // a wait gave up: the loads in flight land first
      for (int v = max(0, u - kSStages); v < u && !ok; ++v)
        if ((v & 1) == mine) await(p, bar(kSF + v % kSStages), (v / kSStages) & 1);
    } else if (warp == 1) {
      // ---------------------------------------------------------- S = Q [c | k_rope]^T
      bool ok = true;
      const uint64_t qd = sdesc_sw128(sb + kQR, 16, 1024);
      const uint64_t sd0 = sdesc_sw128(sb + kSRing, 16, 1024);
      int g = 0, s = 0, e = 0;
      uint32_t ph = 0;
      while (ok && next_of_warp(p, k, first, lane)) {
        if (k.head) {
          s += kQBoxes;   // the Q stages
          if (s >= kSStages) { s -= kSStages; ph ^= 1u; }
        }
        const int n = k.n;
        if (!await_warp(p, bar(kQRd), e++ & 1)) { ok = false; break; }
        for (int j = 0; j < n && ok; ++j, ++g) {
          const int b = g & 1;
          if (g >= 2 && !await_warp(p, bar(kSSR + b), ((g >> 1) - 1) & 1)) { ok = false; break; }
          const uint32_t d = tmem + 256 + 128 * b;
          // unrolled: with the block in a register, every MMA took 130 cycles to issue
#pragma unroll
          for (int blk = 0; blk < kBlocks; ++blk) {
            if (!await_warp(p, bar(kSF + s), ph)) { ok = false; break; }
            tc_fence_after();
            const uint64_t sd = sdesc_add(sd0, s * kBlk);
            const uint32_t qa = tmem + 32 * blk;
            if (blk >= kLatBlocks) mma_ss4_elect(d, qd, sd, kIdS, 1u);
            else if (kFp8) mma_ts4x2_8bit_elect(d, qa, sd, kIdS8, blk ? 1u : 0u);
            else mma_ts4_elect(d, qa, sd, kIdS, blk ? 1u : 0u);
            mma_commit_elect(bar(kSE + s));
            if (++s == kSStages) { s = 0; ph ^= 1u; }
          }
          if (ok) mma_commit_elect(bar(kSSF + b));
        }
        if (ok) mma_commit_elect(bar(kQE));
      }
    } else if (warp == 2) {
      // ---------------------------------------------------------- staged P and its factors into the values CTA
      constexpr int kPieceRows = kFp8 ? 16 : 8;
      constexpr uint32_t kPiece = 128 * kPieceRows;
      const uint32_t o_p = mapa_shared(sb + kOP, 1u), o_fac = mapa_shared(sb + kFac, 1u), o_pf = mapa_shared(bar(kPF), 1u);
      bool ok = true;
      int g = 0;
      while (ok && next_of_warp(p, k, first, lane)) {
        // Pieces of a block down to the item's last live rows (16 of 128 live: a copy of all of them made the whole
        // launch 8% longer; what the other rows of P hold ends in rows of O that none reads), one a lane.  In pieces
        // the copy passes between this CTA's loads: with one of 32 KB, 64 bf16 requests took 200 us, with 2 KB 192.5,
        // with 1 KB 189.5 (FP8, whose loads are fewer: 139, 137.5, 140).
        const uint32_t live = (uint32_t)(min(128, k.rows - k.row0) + kPieceRows - 1) / kPieceRows;   // pieces of a block
        const uint32_t mine = lane % (128 / kPieceRows), at = lane / (128 / kPieceRows) * kBlk + mine * kPiece;
        for (int j = 0; j < k.n && ok; ++j, ++g) {
          const int b = g & 1;
          // P tile b of the values CTA is free once the PV of tile g - 2 is done
          ok = await_warp(p, bar(kPST + b), (g >> 1) & 1) && (g < 2 || await_warp(p, bar(kPFR + b), ((g - 2) >> 1) & 1));
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx_cluster(o_pf + 8u * b, 2 * live * kPiece + kFacBytes);
            bulk_copy_to_peer(o_fac + b * kFacBytes, sb + kFac + b * kFacBytes, kFacBytes, o_pf + 8u * b);
          }
          if (lane < 256 / kPieceRows && mine < live) bulk_copy_to_peer(o_p + b * kPBytes + at, sb + kPS + b * kPBytes + at, kPiece, o_pf + 8u * b);
        }
      }
      // the last two PV commits land before this CTA exits
      for (int v = max(0, g - 2); v < g && ok; ++v) ok = await_warp(p, bar(kPFR + (v & 1)), (v >> 1) & 1);
      for (int v = max(0, g - 2); v < g && !ok; ++v) await_warp(p, bar(kSTF + (v & 1)), (v >> 1) & 1);   // as above, the copies
    } else if (warp >= 12) {
      // ---------------------------------------------------------- Q: qlat from its stages into TMEM
      const int r = tid - 384;
      const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
      bool ok = true;
      int e = 0, u = 0;
      while (next_of_group(p, k, first, r == 0, 7, 128)) {
        // the MMAs that read the Q before this are done
        if (ok && e > 0) ok = await_warp(p, bar(kQE), (e - 1) & 1);
        ++e;
        tc_fence_after();
        if (k.head) {
#pragma unroll 1
          for (int i = 0; i < kQBoxes; i += 2, u += 2) {
            const int sa = u % kSStages, sc = (u + 1) % kSStages;
            if (ok) ok = await_warp(p, bar(kSF + sa), (u / kSStages) & 1);
            if (ok) ok = await_warp(p, bar(kSF + sc), ((u + 1) / kSStages) & 1);
            uint32_t w[2][32];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                uint32_t w4[4];
                lds128(sb + kSRing + (hh ? sc : sa) * kBlk + sw128_off((uint32_t)r, (uint32_t)c), w4);
                w[hh][4 * c] = w4[0]; w[hh][4 * c + 1] = w4[1]; w[hh][4 * c + 2] = w4[2]; w[hh][4 * c + 3] = w4[3];
              }
            tmem_st32(tmem + lane_off + 32 * i, w[0]);
            tmem_st32(tmem + lane_off + 32 * i + 32, w[1]);
            named_bar_sync(6, 128);   // all rows of the stages are read
            if (r == 0 && ok) {
              mbar_arrive(bar(kSE + sa));
              mbar_arrive(bar(kSE + sc));
            }
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(bar(kQRd));
        u += kBlocks * k.n;   // the stages of its tiles
      }
      if (ok && e > 0) await_warp(p, bar(kQE), (e - 1) & 1);   // the last commit lands before this CTA exits
    } else if (warp >= 4) {
      // ---------------------------------------------------------- softmax: columns 64 half .. of a row a thread
      const int half = (warp - 4) >> 2, r = 32 * (warp & 3) + lane;
      const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t pair = 1 + (warp & 3);   // barrier of the two warps that share 32 rows
      // a warp whose wait gave up goes on without waits and signals: its barriers with the other warp of its rows
      // are met
      bool ok = true;
      int g = 0;
      float m_used = -INFINITY, l = 0.f, lt = 0.f, lsum = 0.f;   // lt: of P as its terms hold it
      while (next_of_group(p, k, first, tid == 128, 5, 256)) {
        const int prow = k.row0 + r;
        const bool live = prow < k.rows;
        const int64_t orow = (int64_t)k.w.q_begin * H + prow;
        const float qs = kFp8 && live ? p.ws.qscale[orow] * p.kv_scale : 1.f, sl2 = p.scale_log2 * qs;
        {
          // q_rope turned by pos - offset, as a K-major swizzled block: chunks 4 half .. of the row.  This warp has
          // seen the last S buffer of the range before, so no MMA reads the block.  FP8 scores count in units of
          // the row's scale, so q_rope is divided by that.
          const uint4* qr = reinterpret_cast<const uint4*>(p.q + orow * kDqk + kDnope) + 4 * half;
          const int64_t delta = live ? (int64_t)__ldg(p.q_pos + k.w.q_begin + prow / H) - k.offset : 0;
          const float rq = 1.f / qs;
          uint4 x[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) x[c] = live ? __ldg(qr + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t w4[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float sn, cs;
              rope_sincos_sfu(delta, p.rope_frac[16 * half + 4 * c + i], &sn, &cs);
              const float x0 = bf16_lo(w4[i]), x1 = bf16_hi(w4[i]);
              w4[i] = pack_bf16((x0 * cs - x1 * sn) * rq, (x0 * sn + x1 * cs) * rq);
            }
            sts128(sb + kQR + sw128_off((uint32_t)r, (uint32_t)(4 * half + c)), w4[0], w4[1], w4[2], w4[3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && ok) mbar_arrive(bar(kQRd));
        }
        const int qk = live ? last_key(k, prow, H) : -1;
        const int n = k.n, t0 = k.t0, k_lo = k.k_lo, k_hi = k.k_hi, slot = k.slot;
        const bool tail = k.tail;
        if (k.head) {
          m_used = -INFINITY;
          l = lt = lsum = 0.f;
        }
#pragma unroll 1
        for (int j = 0; j < n; ++j, ++g) {
          const int b = g & 1;
          uint32_t v[64];
          float mx;
          // the staging buffer is free once the copy it held two tiles ago landed
          if (ok && g >= 2) ok = await_warp(p, bar(kSTF + b), ((g - 2) >> 1) & 1);
          if (ok) ok = await_warp(p, bar(kSSF + b), (g >> 1) & 1);
          tc_fence_after();
          mx = tmem_ld64_max(tmem + lane_off + 256 + 128 * b + 64 * half, v);
          tc_fence_before();
          __syncwarp();
          // relaxed: the reads are ordered for the next MMAs by the tcgen05 fences around it
          if (lane == 0 && ok) mbar_arrive_relaxed(bar(kSSR + b));
          const int kt0 = t0 + 128 * j + 64 * half;
          float odd = 0.f;   // NaN: a score that is not finite among columns that may be hidden from the row
          if (!(kt0 >= k_lo && kt0 + 63 < k_hi && kt0 + 63 <= qk)) {
            const int hi = min(k_hi - 1, qk) - kt0, lo = k_lo - kt0;   // visible columns lo .. hi
            float m4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) m4[i] = -INFINITY;
#pragma unroll
            for (int c = 0; c < 64; c += 2) {
              odd = fmaf(__uint_as_float(v[c]), 0.f, fmaf(__uint_as_float(v[c + 1]), 0.f, odd));
              const float xa = (c >= lo && c <= hi) ? __uint_as_float(v[c]) : -INFINITY;
              const float xb = (c + 1 >= lo && c + 1 <= hi) ? __uint_as_float(v[c + 1]) : -INFINITY;
              v[c] = __float_as_uint(xa);
              v[c + 1] = __float_as_uint(xb);
              m4[(c >> 1) & 3] = fmax3(m4[(c >> 1) & 3], xa, xb);
            }
            mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          }
          // The row's maximum over both halves, in fp32: a reference some bits above it would lose P where the scores
          // are large.  Each thread leaves its own in the staging buffer, in a chunk that the other one reads behind
          // the barrier and only then writes its P to.
          const uint32_t stg = sb + kPS + b * kPBytes;
          // chunk c of a half of the row.  bf16: 64 keys are the half's own block; 8-bit: 4 chunks of each term's block
          auto chunk = [&](int hh, int c) {
            return kFp8 ? stg + (c >> 2) * kBlk + sw128_off((uint32_t)r, (uint32_t)(4 * hh + (c & 3)))
                        : stg + hh * kBlk + sw128_off((uint32_t)r, (uint32_t)c);
          };
          const uint32_t word = 4 * ((lane >> 3) & 3);   // the 32 rows in 32 banks
          sts32(chunk(half ^ 1, 0) + word, __float_as_uint(mx));
          named_bar_sync(pair, 64);
          const float m_tile = fmaxf(mx, __uint_as_float(lds32(chunk(half, 0) + word))) * sl2;
          uint8_t* fac = smem + kFac + b * kFacBytes;
          float alpha = 1.f;
          if (m_tile > m_used + (kFp8 ? kRescaleFp8 : kRescaleBf16)) {
            alpha = ex2(m_used - m_tile);   // 0 when m_used = -inf
            m_used = m_tile;
          }
          const float mref = ((m_used == -INFINITY) ? 0.f : m_used) - (kFp8 ? kPBiasFp8 : 0.f);
          const uint64_t sc2 = f2pack(sl2, sl2), nm2 = f2pack(-mref, -mref);
          // P in registers while the previous tile's copy is still in flight: bf16 pairs, or per four keys a
          // word of each term's codes
          uint64_t s2[2] = {0ull, 0ull};
          float t0 = 0.f, t1 = 0.f;   // 8-bit: the sums of the two terms
          uint32_t pk[32];
          {
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              float x0, x1;
              f2unpack(ffma2(f2pack(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1])), sc2, nm2), x0, x1);
              const float a = ex2(x0), bb = ex2(x1);
              s2[c & 1] = fadd2(s2[c & 1], f2pack(a, bb));
              if constexpr (kFp8) {
                // f16 (2^-11), its nearest E5M2, the rest of it, which f16 holds exactly, and that in E5M2 too
                const uint32_t h16 = pack_f16(a, bb);
                const uint32_t h2 = e5m2x2_of_f16x2(h16), hw = __byte_perm(h2, 0u, 0x1404);   // (E5M2: f16's high byte)
                const uint32_t r2 = e5m2x2_of_f16x2(sub_f16x2(h16, hw));
                add_f16x2(t0, t1, fadd_f16x2(hw, __byte_perm(r2, 0u, 0x1404)));               // their sum: exact in f16
                if (c & 1) {
                  pk[c >> 1] = __byte_perm(pk[c >> 1], h2, 0x5410);
                  pk[16 + (c >> 1)] = __byte_perm(pk[16 + (c >> 1)], r2, 0x5410);
                } else {
                  pk[c >> 1] = h2;
                  pk[16 + (c >> 1)] = r2;
                }
              } else {
                pk[c] = pack_bf16(a, bb);
              }
            }
          }
          float s4[4];
          f2unpack(s2[0], s4[0], s4[1]);
          f2unpack(s2[1], s4[2], s4[3]);
          l = l * alpha + ((s4[0] + s4[2]) + (s4[1] + s4[3]));
          if (kFp8) lt = lt * alpha + (t0 + t1);
          if (tail && j == n - 1) {   // the piece's last tile: the row's sums over both halves
            if (half) {
              sts32(chunk(0, 1) + word, __float_as_uint(l));
              if (kFp8) sts32(chunk(0, 2) + word, __float_as_uint(lt));
            }
            named_bar_sync(pair, 64);
            if (half == 0) {
              lsum = l + __uint_as_float(lds32(chunk(0, 1) + word));
              reinterpret_cast<float*>(fac + kFacSum)[r] = kFp8 ? lt + __uint_as_float(lds32(chunk(0, 2) + word)) : lsum;
            }
          }
#pragma unroll
          for (int c = 0; c < 8; ++c) sts128(chunk(half, c), pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
          // P = 0 does not hide a key that is not finite from O: a query before it would have NaN
          const uint32_t any_odd = __any_sync(0xffffffffu, odd != 0.f) ? 0x100u : 0u;
          uint16_t* flag = reinterpret_cast<uint16_t*>(fac + kFacFlags + 4 * (warp & 3)) + half;
          if (half == 0) {
            reinterpret_cast<float*>(fac)[r] = alpha;
            const uint32_t any_rescale = __any_sync(0xffffffffu, alpha != 1.f) ? 1u : 0u;
            if (lane == 0) *flag = (uint16_t)(any_odd | any_rescale);
          } else if (lane == 0) {
            *flag = (uint16_t)any_odd;
          }
          fence_proxy_async_smem();   // the staged tile is read by the bulk copies (async proxy)
          __syncwarp();
          if (lane == 0 && ok) mbar_arrive(bar(kPST + b));
        }
        if (tail && live && half == 0) {
          const float lse = (ok && lsum != 0.f) ? (m_used - (kFp8 ? kPBiasFp8 : 0.f) + __log2f(lsum)) * 0.6931471805599453f
                                              : -INFINITY;
          if (slot < 0) p.ws.lat_lse[orow] = lse;
          else p.ws.part_lse[slot * kItemRows + r] = lse;
        }
      }
    }
  } else {
    if ((warp == 0 || warp == 2) && lane == 0) {
      // ---------------------------------------------------------- loads: 256 latent columns of 32 (64) keys a stage,
      // each half of the columns by its thread
      const int nh = warp >> 1;
      bool ok = true;
      int u = nh;
      while (ok && next_of_one(p, k, first)) {
        const int stages = kOPerTile * k.n, boxes = k.tail ? boxes_of(k) : 0;
        for (int i = 0; i < stages + boxes; ++i, u += 2) {
          const int s = u % kOStages;
          const int row = i < stages ? cache_row(p, k.r, k.t0 + kORows * i, k.k_hi) : 0;
          if (u >= kOStages && !await(p, bar(kCE + s), ((u / kOStages) - 1) & 1)) { ok = false; break; }
          if (i < stages) {
            mbar_arrive_expect_tx(bar(kCF + s), kOStage);
            tma_load_3d(sb + kORing + s * kOStage, &p.tm_o, 0, row, (kLatBlocks / 2) * nh, bar(kCF + s));
          } else {
            mbar_arrive(bar(kCF + s));   // the stage is the correction warps'
          }
        }
      }
      const int last = u - kOStages < nh ? nh : u - kOStages;
      for (int v = last; v < u && ok; v += 2) ok = await(p, bar(kCE + v % kOStages), (v / kOStages) & 1);
      for (int v = last; v < u && !ok; v += 2) await(p, bar(kCF + v % kOStages), (v / kOStages) & 1);   // as above
    } else if (warp == 1) {
      // ---------------------------------------------------------- P landed, rows rescaled, O += P c
      volatile int* hand = reinterpret_cast<volatile int*>(smem + kHand);
      const uint64_t pd0 = sdesc_sw128(sb + kOP, 16, 1024);                        // P, K-major
      const uint64_t cd0 = sdesc_sw128(sb + kORing, kORows * 128, 1024);           // latent stages, MN-major
      bool ok = true;
      int g = 0, events = 0, done = 0;   // tiles, hand-overs, finished pieces
      int s = 0;                         // next stage, and the parity of its fill
      uint32_t ph = 0;
      auto advance = [&](int n) {
        s += n;
        while (s >= kOStages) { s -= kOStages; ph ^= 1u; }
      };
      bool head = true;
      while (ok && next_of_warp(p, k, first, lane)) {
        if (k.head) head = true;
#pragma unroll 1
        for (int j = 0; j < k.n && ok; ++j, ++g) {
          const int b = g & 1;
          if (!await_warp(p, bar(kPF + b), (g >> 1) & 1)) { ok = false; break; }
          uint32_t f[4];
          lds128(sb + kFac + b * kFacBytes + kFacFlags, f);
          const uint32_t flags = f[0] | f[1] | f[2] | f[3];
          if (!head) {
            if (flags & 0xFFu) {
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
          if (k.tail && j == k.n - 1) {
            // the row sums sit beside this P tile: read before the next tiles may replace them
            if (lane == 0) {
              *hand = 2 + b;
              mbar_arrive(bar(kCN));
            }
            if (!await_warp(p, bar(kCD), events++ & 1)) { ok = false; break; }
          }
          if ((flags & ~0xFFu) && !zero_not_finite<kFp8>(p, k, j, b, sb, s, ph, lane)) { ok = false; break; }
          fence_proxy_async_smem();   // P was written by the other CTA's copy, the MMA reads it as an operand
          tc_fence_after();
#pragma unroll 1
          for (int i = 0; i < kOPerTile; ++i) {
            if (!ok) break;
#pragma unroll
            for (int nh = 0; nh < 2; ++nh) {
              if (!await_warp(p, bar(kCF + s), ph)) { ok = false; break; }
              // rows outside the run meet P = 0, but may hold anything: they are zeroed
              const int kt = k.t0 + 128 * j + kORows * i;
              const int lo = max(0, k.k_lo - kt), hi = min(kORows, k.k_hi - kt);
              if ((lo > 0 || hi < kORows) && hi > 0) zero_rows<kORows>(sb + kORing + s * kOStage, lo, hi, lane);
              tc_fence_after();
              const uint64_t cd = sdesc_add(cd0, s * kOStage);
              // k-steps 2 i, 2 i + 1 of the tile: 16 keys (bf16) or 32 (FP8) each
              const uint32_t acc = (head && i == 0) ? 0u : 1u;
              const uint64_t pd = sdesc_add(pd0, b * kPBytes + (kFp8 ? i * 64 : (i >> 1) * kBlk + (i & 1) * 64));
              if (kFp8) mma_ss2x2_mn_8bit_elect(tmem + 256 * nh, pd, cd, kIdPV8, acc);
              else mma_ss2_mn_elect(tmem + 256 * nh, pd, cd, kIdPV, acc);
              mma_commit_elect(bar(kCE + s));
              advance(1);
            }
          }
          if (!ok) break;
          head = false;
          mma_commit_elect(bar(kPVD + b));
          mma_commit_mc_elect(bar(kPFR + b), 0x1);
        }
        if (k.tail) {
          ++done;
          advance(2 * boxes_of(k));
        }
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
      while (ok && next_of_one(p, k, first))
        for (int j = 0; j < k.n && ok; ++j, ++g) {
          ok = await(p, bar(kPF + (g & 1)), (g >> 1) & 1);
          if (ok) mbar_arrive_cluster_relaxed(stf + 8u * (g & 1));   // relaxed: a landed copy has read its source
        }
    } else if (warp >= 4 && warp < 12) {
      // ---------------------------------------------------------- rescale O rows; epilogue: columns 256 half ..
      const int half = (warp - 4) >> 2, r = 32 * (warp & 3) + lane;
      const uint32_t o_cols = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 256 * half;
      const volatile int* hand = reinterpret_cast<const volatile int*>(smem + kHand);
      bool ok = true;
      int g = 0, ev = 0, u = half;   // tiles, hand-overs, this half's next stage
      while (next_of_group(p, k, first, tid == 128, 5, 256)) {
        g += k.n;
        u += 2 * kOPerTile * k.n;
        if (!k.tail) continue;   // a piece's states leave at its end
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
            for (int cc = 0; cc < 8; ++cc) {
              uint32_t o[32];
              tmem_ld32(o_cols + 32 * cc, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
              tmem_st32(o_cols + 32 * cc, o);
            }
            tmem_wait_st();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kCD));
        }
        if (ok) ok = await_warp(p, bar(kPVD + ((g - 1) & 1)), ((g - 1) >> 1) & 1);
        if (named_bar_or(2, 256, !ok)) {   // the eight warps leave together
          ok = false;
          break;
        }
        tc_fence_after();
        const float inv = lsum != 0.f ? 1.f / lsum : 0.f;   // no key seen: 0; a NaN stays one
        const int rows = k.rows - k.row0;      // live rows of the item
        const bool whole = k.slot < 0;
        const int row0 = whole ? k.w.q_begin * H + k.row0 : k.slot * kItemRows;   // first row of the states
        const int boxes = boxes_of(k);
        // A warp of 32 live rows stages 32 columns of them in its quarter of a box and stores them by TMA, four
        // boxes in turn, at its own pace; a warp with fewer writes them by its threads.  256 KB in 4.6 us: the SM's
        // stores to L2 pace it, about 30 B a cycle (contiguous 4 KB copies, loads of the next columns started
        // before, or 64 columns a step took as long).
        const bool tma = 32 * (warp & 3) + 32 <= rows;
        if (boxes > 0 && ok) {   // the loading thread hands the stages over in order
#pragma unroll 1
          for (int b = 0; b < kBoxes; ++b) ok = ok && await_warp(p, bar(kCF + (u + 2 * b) % kOStages), ((u + 2 * b) / kOStages) & 1);
        }
#pragma unroll 1
        for (int cc = 0; cc < 8; ++cc) {
          uint32_t o[32];
          tmem_ld32(o_cols + 32 * cc, o);
          if (cc == 7) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kEP));   // O has been read: the next piece may begin
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
          const int col = 256 * half + 32 * cc;
          if (tma) {
            const uint32_t box = sb + kORing + (uint32_t)((u + 2 * (cc & 3)) % kOStages) * kOStage + (uint32_t)(warp & 3) * 4096;
            if (cc >= 4) {   // the box's store of four steps ago has read it
              if (lane == 0) bulk_wait_read<3>();
              __syncwarp();
            }
#pragma unroll
            for (int c = 0; c < 8; ++c)
              sts128(box + sw128_off((uint32_t)lane, (uint32_t)c), o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && ok) {
              tma_store_2d(whole ? &p.tm_lat : &p.tm_part, box, col, row0 + 32 * (warp & 3));
              bulk_commit();
            }
          } else if (r < rows) {
            uint4* dst = reinterpret_cast<uint4*>((whole ? p.ws.lat : p.ws.part) + (int64_t)(row0 + r) * kDc + col);
#pragma unroll
            for (int c = 0; c < 8; ++c) dst[c] = make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
          }
        }
        if (boxes > 0) {   // the stages go back once every warp's stores have read them
          if (lane == 0) bulk_wait_read0();
          named_bar_sync(3 + half, 128);
          if (r < kBoxes && ok) mbar_arrive(bar(kCE + (u + 2 * r) % kOStages));
          u += 2 * kBoxes;
        }
      }
      if (lane == 0) bulk_wait0();   // every store complete before the CTA's shared memory goes
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

cudaError_t decode_clusters(int* out) {
  static std::atomic<int> resident_on[64];   // per device, 0: not configured yet
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int clusters = resident_on[dev].load();
  if (clusters == 0) {
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
    resident_on[dev].store(clusters);
  }
  *out = clusters;
  return cudaSuccess;
}

cudaError_t launch_decode_attn(const DecodeParams& p, bool fp8, int clusters, cudaStream_t s) {
  return launch_dependent(fp8 ? decode_attn_kernel<true> : decode_attn_kernel<false>, dim3(2 * clusters), kThreads, kSmem,
                          p, s);
}

}  // namespace mla
