// Block tables and slot maps from the requests' lengths.  With need = ceil(len /
// 64) and held blocks so far, request r
//   gives back  j in [max(need, shared), held)   (shared ones only leave the table)
//   asks for    j in [held, need)
// (where held < shared, what it gets below shared is its own: shared becomes held)
// and both, over all requests in (r, j) order, are one run on the stack of free
// blocks of height n: entry e of the R given back goes to place n + R - 1 - e,
// then entry e of those taken comes from place n + R - 1 - e.  So what is given
// back and what is taken undo one another, and no two entries depend on another
// but by two prefix sums over the requests.  A request is served if the demands
// up to and with its own fit; the others stay as they are.
//
// One cluster: every CTA makes the prefix sums of all requests for itself, the
// entries and the rows of the slot map are shared out over the cluster's warps in
// runs, a warp finding the request of its first entry by a search in shared memory
// and the others from there.  A barrier of the cluster lies between what is pushed
// and what is popped.  Bound by latency and by the few SMs of a cluster: 512
// requests, 16,000 to 20,000 entries each way and 19,000 to 36,000 rows 9.2 us (on
// 8 SMs, each entry searched for by its thread, 12.2); 64 requests, a few entries,
// 320 rows 4.7 us, of which a launch is 2.2.
#include <atomic>

#include "serving.cuh"
#include "sparse.h"

namespace mla {
namespace {

constexpr int kThreads = 1024, kAtOnce = 4;

struct Req {
  int held, len;     // blocks; tokens wanted
  int from;          // first entry to give back
  int back, more;    // entries given back and asked for by the requests before
};

__global__ void __launch_bounds__(kThreads, 1) assign_blocks_kernel(const __grid_constant__ AssignParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int B = p.batch.num_reqs;
  Req* req = reinterpret_cast<Req*>(smem);              // [B]
  int* cu = reinterpret_cast<int*>(req + B);            // [B + 1]: first rows
  __shared__ int warp_back[32], warp_more[32], warp_served[32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t rank, ctas;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  const bool report = p.err != nullptr && rank == 0;
  grid_wait();
  grid_trigger();

  // ---- prefix sums: thread t has requests [t k, (t + 1) k)
  const int k = (B + kThreads - 1) / kThreads;
  const int r0 = min(B, tid * k), r1 = min(B, r0 + k);
  auto need = [&](const Req& q) { return q.len > p.max_blocks * kBlock ? p.max_blocks : (q.len + kBlock - 1) / kBlock; };
  int back = 0, more = 0;
  bool bad = false;
  uint32_t below = 0;    // bit r - r0: it holds less than its shared blocks
  static_assert(kMaxAssignReqs <= 32 * kThreads, "a bit a request of a thread");
  for (int r = r0; r < r1; ++r) {
    const int h = __ldcg(p.held + r), sh = p.shared == nullptr ? 0 : __ldcg(p.shared + r);      // (an earlier call may have written both)
    Req q;
    q.len = max(__ldg(p.batch.seq_lens + r), 0);
    q.held = min(max(h, 0), p.max_blocks);
    q.from = max(need(q), min(sh, q.held));
    below |= sh > q.held ? 1u << (r - r0) : 0u;
    q.back = back;
    q.more = more;
    bad |= q.len > p.max_blocks * kBlock || h != q.held;
    back += max(0, q.held - q.from);
    more += max(0, need(q) - q.held);
    req[r] = q;
    if (p.batch.cu_q != nullptr) cu[r] = __ldg(p.batch.cu_q + r);
  }
  if (tid == 0 && p.batch.cu_q != nullptr) cu[B] = __ldg(p.batch.cu_q + B);
  int ib = back, im = more;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int b = __shfl_up_sync(0xffffffffu, ib, o), m = __shfl_up_sync(0xffffffffu, im, o);
    if (lane >= o) { ib += b; im += m; }
  }
  if (lane == 31) { warp_back[warp] = ib; warp_more[warp] = im; }
  __syncthreads();
  const int wb = warp_back[lane], wm = warp_more[lane];
  const int all_back = __reduce_add_sync(0xffffffffu, wb);
  const int pb = __reduce_add_sync(0xffffffffu, lane < warp ? wb : 0) + ib - back;
  const int pm = __reduce_add_sync(0xffffffffu, lane < warp ? wm : 0) + im - more;
  const int count = __ldcg(p.free_count);
  const int pushed = min(max(count, 0), p.capacity) + all_back, top = min(pushed, p.capacity);   // (what outgrows the stack is lost)
  bad |= tid == 0 && (count < 0 || pushed > top || count > p.capacity);
  int served = 0;                        // entries taken: the last demand that fits
  bool left = false;
  for (int r = r0; r < r1; ++r) {
    Req q = req[r];
    q.back += pb;
    q.more += pm;
    const int end = q.more + max(0, need(q) - q.held);
    if (end <= top) served = max(served, end);
    else left |= need(q) > q.held;
    req[r] = q;
  }
  served = __reduce_max_sync(0xffffffffu, served);
  if (lane == 0) warp_served[warp] = served;
  if (report && bad) atomicOr(p.err, kErrBadBlock);
  if (report && left) atomicOr(p.err, kErrNoBlocks);
  __syncthreads();
  served = __reduce_max_sync(0xffffffffu, warp_served[lane]);

  // a warp's run of n entries or rows, 32 at a time and four times that under way: store(e, r, load(e, r)) with the last
  // request r that starts at or before e
  const int id_warp = rank * (kThreads / 32) + warp, warps = ctas * (kThreads / 32);
  auto share = [&](int n, auto starts, auto load, auto store) {
    const int each = (n + 32 * warps - 1) / (32 * warps) * 32;
    const int begin = (int)min((int64_t)n, (int64_t)id_warp * each), end = min(n, begin + each);
    if (begin >= end) return;
    int r = 0;
    for (int k = B; k > 1;) {            // of the first entry, 32 tries a step
      const int step = (k + 31) / 32, at = lane * step;
      const bool ok = lane == 0 || (at < k && starts(r + at) <= begin);
      const int i = 31 - __clz(__ballot_sync(0xffffffffu, ok));
      r += i * step;
      k = min(step, k - i * step);
    }
    for (int e0 = begin; e0 < end; e0 += 32 * kAtOnce) {
      int of[kAtOnce], v[kAtOnce];
#pragma unroll
      for (int c = 0; c < kAtOnce; ++c) {
        if (e0 + 32 * c >= end) break;
        const int e = min(e0 + 32 * c + lane, end - 1);
        for (int i = 0; i < 4; ++i) r += r + 1 < B && starts(r + 1) <= e;
        if (r + 1 < B && starts(r + 1) <= e) {      // behind many requests without entries
          for (int k = B - r; k > 1;) {
            const int half = k >> 1;
            if (starts(r + half) <= e) { r += half; k -= half; }
            else k = half;
          }
        }
        of[c] = r;
        v[c] = load(e, r);
        r = __shfl_sync(0xffffffffu, r, 31);
      }
#pragma unroll
      for (int c = 0; c < kAtOnce; ++c)
        if (e0 + 32 * c + lane < end) store(e0 + 32 * c + lane, of[c], v[c]);
    }
  };
  const int first = rank * kThreads + tid, step = ctas * kThreads;

  // ---- blocks given back
  auto given = [&](int e, int r) { return p.table + (int64_t)r * p.max_blocks + req[r].from + (e - req[r].back); };
  share(all_back, [&](int k) { return req[k].back; }, [&](int e, int r) { return __ldcg(given(e, r)); }, [&](int e, int r, int id) {
    if (pushed - 1 - e < p.capacity) p.free_blocks[pushed - 1 - e] = id;
    *given(e, r) = -1;
  });
  if (p.shared != nullptr)
    for (int k = id_warp; k < B; k += warps) {      // dropped ones
      const Req q = req[k];
      for (int j = need(q) + lane; j < min(q.from, q.held); j += 32) p.table[(int64_t)k * p.max_blocks + j] = -1;
    }
  cluster_sync_all();      // pushed before it is popped; everyone has read held, shared and free_count

  // ---- blocks taken
  auto popped = [&](int k) { return __ldcg(p.free_blocks + top - 1 - k); };      // k < served <= top
  share(served, [&](int k) { return req[k].more; }, [&](int e, int) { return popped(e); }, [&](int e, int r, int id) {
    p.table[(int64_t)r * p.max_blocks + req[r].held + (e - req[r].more)] = id;
  });
  auto kept = [&](const Req& q) { return need(q) <= q.held || q.more + (need(q) - q.held) <= top ? need(q) : q.held; };
  for (int k = first; k < B; k += step) p.held[k] = kept(req[k]);
  if (below != 0 && rank == 0)      // blocks popped below the shared ones are given back like the others
    for (int r = r0; r < r1; ++r)
      if ((below >> (r - r0) & 1) && kept(req[r]) > req[r].held) p.shared[r] = req[r].held;
  if (first == 0) *p.free_count = top - served;

  // ---- slots of the new rows
  const bool even = p.batch.cu_q == nullptr;
  auto begins = [&](int k) { return even ? k * p.batch.per_req : cu[k]; };
  auto token = [&](int x, int r) { return req[r].len - (even ? begins(r + 1) - x : min(cu[r + 1], p.batch.rows) - x); };
  share(p.batch.rows, begins, [&](int x, int r) {
    const Req q = req[r];
    const int t = token(x, r), b = t >> 6;
    if (x < begins(r) || (!even && x >= cu[r + 1]) || t < 0 || b >= kept(q)) return -1;
    return b < q.held ? __ldcg(p.table + (int64_t)r * p.max_blocks + b) : popped(q.more + (b - q.held));
  }, [&](int x, int r, int id) { p.slots[x] = id >= 0 ? (int64_t)id * kBlock + (token(x, r) & (kBlock - 1)) : -1; });
}

}  // namespace

cudaError_t launch_assign_blocks(const AssignParams& p, cudaStream_t s) {
  // 16 CTAs where the device takes such a cluster, else 8 (512_mixed 9.2 us, with 8 11.3, with 4 15; small batches alike)
  static std::atomic<int> ctas_of[64];   // per device, 0: not configured yet
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(kThreads);
  cfg.attrs = attr;
  int ctas = ctas_of[dev].load();
  if (ctas == 0) {
    constexpr int kMostSmem = 24 * kMaxAssignReqs + 16;
    e = cudaFuncSetAttribute(assign_blocks_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(assign_blocks_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    int resident = 0;
    attr[0].val.clusterDim.x = 16;
    cfg.gridDim = dim3(16);
    cfg.dynamicSmemBytes = kMostSmem;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&resident, assign_blocks_kernel, &cfg);
    if (e != cudaSuccess) return e;
    ctas = resident > 0 ? 16 : 8;
    ctas_of[dev].store(ctas);
  }
  attr[0].val.clusterDim.x = ctas;
  cfg.gridDim = dim3(ctas);
  cfg.dynamicSmemBytes = 24 * (size_t)p.batch.num_reqs + 16;
  cfg.stream = s;
  cfg.numAttrs = 2;
  count_launch();
  return cudaLaunchKernelEx(&cfg, assign_blocks_kernel, p);
}

}  // namespace mla
