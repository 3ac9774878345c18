// tables.cu — block tables, slot map and lengths of a batch from the requests'
// lengths, on the GPU.
//
// Request b holds ctx_b tokens and adds new_b.  Its pages 0 .. ceil(ctx_b / 16) - 1
// are in its block-table row already; pages first_b = ceil(ctx_b / 16) up to
// last_b = ceil((ctx_b + new_b) / 16) come from the free list:
//   page_start_b = sum of last - first over the requests before b
//   table[b][first_b + k] = free[head + page_start_b + k]
//   slot of token t of the step's new tokens (request b, position p = ctx_b + t -
//   query_start_b) = table[b][p / 16] * 16 + p % 16, and -1 behind the last token.
//
// What bounds it: latency.  The bytes (8 a slot, 4 a page) are 0.0003 to 1.3 us of
// the copy rate, a launch and two dependent loads ~4 us in a CUDA graph.  So it is one kernel:
// every CTA scans all the lengths itself (a few hundred values from L2) into
// shared memory and then fills its share of the table entries and slots, with no
// second launch and no wait between CTAs.  ctx_lens may be seq_lens and free_head
// may be free_head_out (a captured step then advances its own lengths): only the
// CTA that is the last to have read them writes the two, which a counter in the
// workspace tells (reset by that CTA, so that the next call finds it zero).
// Measured (CUDA graph): 64 sequences of one new token 4.0 us, 8 of 1,024 new tokens
// 4.0 us, 251 prompts of about 1M tokens in all 7.5 us (1.1 TB/s of slots).
#include <algorithm>

#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kTabThreads = 512;
constexpr int kTabWarps = kTabThreads / 32;
constexpr int kTabPage = 16;

struct Scanned {  // per request, in shared memory
  int32_t* qs;    // [B + 1] first new token
  int32_t* ps;    // [B + 1] first new page
  int32_t* ctx;   // [B] tokens before the step
};

// last b with start[b] <= i (start is non-decreasing, start[0] = 0 <= i)
__device__ __forceinline__ int owner(const int32_t* start, int n, int i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// VEC slots a thread, stored together (16-byte stores for VEC = 4).
template <int VEC>
__global__ void __launch_bounds__(kTabThreads) build_tables_kernel(const TablesParams p) {
  extern __shared__ int32_t tab_smem[];
  __shared__ int32_t wsum[2][kTabWarps];
  __shared__ int32_t s_last;
  Scanned s;
  s.qs = tab_smem;
  s.ps = s.qs + p.batch + 1;
  s.ctx = s.ps + p.batch + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int32_t flags = 0;
  int head = *p.free_head;
  if (head < 0 || head > p.num_free) {
    flags |= KVQ_DEV_NO_PAGE;
    head = head < 0 ? 0 : p.num_free;
  }
  // ---- lengths -> exclusive sums of new tokens and new pages
  const int cap = p.max_pages * kTabPage;
  int carry_q = 0, carry_p = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kTabThreads) {
    const int b = b0 + tid;
    int ctx = 0, add = 0;
    if (b < p.batch) {
      ctx = p.ctx_lens[b];
      add = p.new_lens[b];
      if (ctx < 0 || add < 0 || ctx > cap || add > cap - ctx) {  // a request that does not fit adds nothing
        flags |= KVQ_DEV_BAD_SEQLEN;
        ctx = min(max(ctx, 0), cap);
        add = 0;
      }
    }
    const int want = (ctx + add + kTabPage - 1) / kTabPage - (ctx + kTabPage - 1) / kTabPage;
    int iq = add, ip = want;  // inclusive sums over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int uq = __shfl_up_sync(0xffffffffu, iq, o), up = __shfl_up_sync(0xffffffffu, ip, o);
      if (lane >= o) {
        iq += uq;
        ip += up;
      }
    }
    if (lane == 31) {
      wsum[0][warp] = iq;
      wsum[1][warp] = ip;
    }
    __syncthreads();
    int bq = carry_q, bp = carry_p;
    int tq = 0, tp = 0;
#pragma unroll
    for (int w = 0; w < kTabWarps; ++w) {
      const int vq = wsum[0][w], vp = wsum[1][w];
      if (w < warp) {
        bq += vq;
        bp += vp;
      }
      tq += vq;
      tp += vp;
    }
    if (b < p.batch) {
      s.qs[b] = bq + iq - add;
      s.ps[b] = bp + ip - want;
      s.ctx[b] = ctx;
    }
    carry_q += tq;
    carry_p += tp;
    __syncthreads();
  }
  if (tid == 0) {
    s.qs[p.batch] = carry_q;
    s.ps[p.batch] = carry_p;
    // every thread of this CTA has read its lengths and the head (the barriers
    // above): count the CTA, and the last one may overwrite them
    __threadfence();
    const uint32_t seen = atomicAdd(p.counter, 1u);
    s_last = seen == gridDim.x - 1 ? 1 : 0;
  }
  __syncthreads();
  const bool last = s_last != 0;
  if (blockIdx.x == 0) {
    for (int b = tid; b <= p.batch; b += kTabThreads) {
      p.query_start[b] = s.qs[b];
      p.page_start[b] = s.ps[b];
    }
  }
  if (last) {
    __threadfence();
    for (int b = tid; b < p.batch; b += kTabThreads) p.seq_lens[b] = s.ctx[b] + s.qs[b + 1] - s.qs[b];
    if (tid == 0) {
      *p.free_head_out = carry_p > p.num_free - head ? p.num_free : head + carry_p;
      *p.counter = 0;
    }
  }
  if (carry_q > p.num_slots) flags |= KVQ_DEV_BAD_SLOT;
  if (carry_p > p.num_free - head) flags |= KVQ_DEV_NO_PAGE;

  const int64_t first_thread = (int64_t)blockIdx.x * kTabThreads + tid;
  const int64_t threads = (int64_t)gridDim.x * kTabThreads;
  // ---- table entries of the new pages
  for (int64_t k = first_thread; k < carry_p; k += threads) {
    const int b = owner(s.ps, p.batch, static_cast<int>(k));
    const int col = (s.ctx[b] + kTabPage - 1) / kTabPage + static_cast<int>(k) - s.ps[b];
    const int64_t f = head + k;
    p.block_tables[(size_t)b * p.max_pages + col] = f < p.num_free ? p.free_pages[f] : -1;
  }
  // ---- slots
  for (int64_t t0 = first_thread * VEC; t0 < p.num_slots; t0 += threads * VEC) {
    int64_t slot[VEC];
    int b = t0 < carry_q ? owner(s.qs, p.batch, static_cast<int>(t0)) : 0;
    int seen_page = -1, seen_b = -1, id = -1;
#pragma unroll
    for (int u = 0; u < VEC; ++u) {
      const int64_t t = t0 + u;
      slot[u] = -1;
      if (t < carry_q) {
        while (t >= s.qs[b + 1]) ++b;
        const int ctx = s.ctx[b];
        const int pos = ctx + static_cast<int>(t) - s.qs[b];
        const int page = pos / kTabPage, first = (ctx + kTabPage - 1) / kTabPage;
        if (page != seen_page || b != seen_b) {
          if (page < first) {
            id = p.block_tables[(size_t)b * p.max_pages + page];
          } else {
            const int64_t f = (int64_t)head + s.ps[b] + page - first;
            id = f < p.num_free ? p.free_pages[f] : -1;
          }
          if (id < 0 || id >= p.num_pages) {
            flags |= KVQ_DEV_BAD_PAGE;
            id = -1;
          }
          seen_page = page;
          seen_b = b;
        }
        if (id >= 0) slot[u] = (int64_t)id * kTabPage + pos % kTabPage;
      }
    }
    if (VEC == 4 && t0 + VEC <= p.num_slots) {
      longlong2* o = reinterpret_cast<longlong2*>(p.slot_mapping + t0);
      o[0] = make_longlong2(slot[0], slot[VEC > 1 ? 1 : 0]);
      o[1] = make_longlong2(slot[VEC > 2 ? 2 : 0], slot[VEC > 3 ? 3 : 0]);
    } else {
#pragma unroll
      for (int u = 0; u < VEC; ++u)
        if (t0 + u < p.num_slots) p.slot_mapping[t0 + u] = slot[u];
    }
  }
  if (flags) atomicOr(p.status, flags);
}

template <int VEC>
cudaError_t launch_t(const TablesParams& p, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kTabThreads);
  cfg.dynamicSmemBytes = tables_smem_bytes(p.batch);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, build_tables_kernel<VEC>, p);
}

}  // namespace

int tables_smem_bytes(int batch) { return (3 * batch + 2) * static_cast<int>(sizeof(int32_t)); }

void tables_kernels(const void* (&kernels)[2]) {
  kernels[0] = reinterpret_cast<const void*>(&build_tables_kernel<1>);
  kernels[1] = reinterpret_cast<const void*>(&build_tables_kernel<4>);
}

cudaError_t launch_tables(const TablesParams& p, int sms, cudaStream_t stream) {
  // One slot a thread while a few CTAs hold them all (the shortest path to the last
  // slot), four a thread above.
  if (p.num_slots <= 8 * kTabThreads) {
    const int grid = static_cast<int>(std::max<int64_t>(1, (p.num_slots + kTabThreads - 1) / kTabThreads));
    return launch_t<1>(p, grid, stream);
  }
  const int64_t blocks = (p.num_slots + 4 * kTabThreads - 1) / (4 * kTabThreads);
  return launch_t<4>(p, static_cast<int>(std::min<int64_t>(blocks, 2 * (int64_t)sms)), stream);
}

}  // namespace kvq
