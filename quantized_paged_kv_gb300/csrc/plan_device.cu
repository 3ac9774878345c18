// plan_device.cu — the split plan of a decode, verify or prefix call, made on the
// GPU from the device lengths (the host planner of kvq_plan_splits needs them on
// the host, which a captured step with lengths of its own does not have).
//
// With V = batch * q_len launch sequences, n_v pages of sequence v's own (its
// visible pages less its group's shared ones) and T splits to give:
//   x   = the smallest page count with sum_v max(1, ceil(n_v / x)) <= T
//   S_v = max(1, ceil(n_v / x)), the splits left over going in order to the
//         sequences that x - 1 would split further (x = 1: evenly), so that
//         sum S_v = T whatever the lengths are — the launch's size is fixed
//   split k of v = its own pages [k n_v / S_v, (k + 1) n_v / S_v)
//   items (split, head group) sorted by size, largest first (stable), dealt to the
//   C CTAs in rounds of alternating direction, so that a CTA's long item of one
//   round meets a short one of the next.  Simulated on the repository's workloads
//   this packing's longest CTA is within 0..2 % of longest-first greedy packing,
//   which is sequential; the splits of kvq_plan_splits (twelve candidates tried)
//   are 0..7 % better at mixed lengths (serving mix: 263 pages either way).
//
// What bounds it: latency, in one CTA.  A sequence's items have two sizes only (floor
// and ceil of n_v / S_v), so the sort is over 2 V keys instead of the items, and by their
// sizes' bits alone (at most x + 1): two radix passes of five bits up to 1,022 pages.
// x is found by 32 candidates a round (fewer for many sequences, so that a lane adds up
// 16 of them), inside the bracket [total / T, total / (T - V)];
// splits, leftover and partial slots come from one scan of three packed sums.
// Measured (CUDA graph): one sequence of 2,048 pages 5.7 us, 64 sequences 7.8 us, 256
// sequences of six query tokens in five prefix groups 17.6 us (a bitonic
// network in place of the radix passes, and conversions and divisions: 6.1, 8.4, 26.0).
#include <algorithm>

#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kPlThreads = 1024;
constexpr int kPlWarps = kPlThreads / 32;
constexpr int kPlPage = 16;

int pow2_at_least(int n) {
  int p = 32;
  while (p < n) p <<= 1;
  return p;
}

// floor(a / x) for a = an integer + 0.5 below 2^22 and an integer x >= 1, with rx = 1 / x to
// 2^-23: a / x lies at least 0.5 / x from every integer and the product is off by less, so
// a / x - 0.5 rounds to the floor, which the sum with 2^23 leaves in the low bits (a
// conversion to int takes four times as long).  Below 2^23 the sum has halves: a floor of 0
// may come out as -1, which callers lift.
__device__ __forceinline__ int floor_half(float a, float rx) {
  return __float_as_int(fmaf(a, rx, 8388607.5f)) - 0x4B000000;
}
__device__ __forceinline__ int ceil_div_pages(float n, float x, float rx) {  // ceil(n / x), integers n, x < 2^21
  return floor_half(n + x - 0.5f, rx);  // 0 (n = 0) may come out as -1: the caller takes at least 1
}
__device__ __forceinline__ float reciprocal(int s) {  // to 2^-23
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(static_cast<float>(s)));
  return r;
}
__device__ __forceinline__ int div_pages(float n, int s) {  // n / s, integer n < 2^21
  return max(0, floor_half(n + 0.5f, reciprocal(s)));
}

// Inclusive sum over the CTA of one value a thread; *total = the whole sum.
template <class V>
__device__ __forceinline__ V block_scan(V v, V* wsum, V* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) wsum[warp] = v;
  __syncthreads();
  V w = wsum[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const V before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  __syncthreads();  // wsum is used again
  return v + (warp > 0 ? before : 0);
}

// Stable ascending sort of n keys in shared memory by the `bits` bits from bit `low` up,
// five a pass (least significant first); keys, other: n words each, used in turn; at: n
// halfwords; hist: 32 x 33 words.  Returns the array that holds the result.
// Warp w takes the w-th part of the keys, 32 at a time; lane d counts digit d.  Which
// lanes share a digit follows from five ballots, so a pass needs no atomics: a key's
// place is (keys of smaller digits) + (its digit's keys in earlier warps) + (in this warp).
__device__ uint32_t* sort_keys(uint32_t* keys, uint32_t* other, uint16_t* at, int* hist, int* wsum, int n, int low,
                               int bits) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = (n + kPlThreads - 1) / kPlThreads * 32;
  const int i0 = warp * part + lane, i1 = min(n, (warp + 1) * part);  // this lane's keys: i0, i0 + 32, ...
#pragma unroll 1
  for (int b = low; b < low + bits; b += 5) {
    int count = 0;  // keys with digit `lane` so far
#pragma unroll 1
    for (int i = i0; i - lane < i1; i += 32) {
      const bool in = i < i1;
      const uint32_t d = in ? (keys[i] >> b) & 31u : 0u;
      uint32_t same = __ballot_sync(0xffffffffu, in), mine = same;  // lanes with this lane's digit; with digit `lane`
#pragma unroll
      for (int x = 0; x < 5; ++x) {
        const uint32_t set = __ballot_sync(0xffffffffu, (d >> x) & 1u);
        same &= (d >> x) & 1u ? set : ~set;
        mine &= (lane >> x) & 1 ? set : ~set;
      }
      const int before = __shfl_sync(0xffffffffu, count, d);
      if (in) at[i] = static_cast<uint16_t>(before + __popc(same & ((1u << lane) - 1)));
      count += __popc(mine);
    }
    hist[lane * 33 + warp] = count;
    __syncthreads();
    const int v = hist[warp * 33 + lane];  // digit `warp`, the keys of warp `lane`
    int total;
    const int inc = block_scan<int>(v, wsum, &total);
    hist[warp * 33 + lane] = inc - v;
    __syncthreads();
#pragma unroll 1
    for (int i = i0; i < i1; i += 32) {
      const uint32_t k = keys[i];
      other[hist[((k >> b) & 31u) * 33 + warp] + at[i]] = k;
    }
    __syncthreads();
    uint32_t* t = keys;
    keys = other;
    other = t;
  }
  return keys;
}

__global__ void __launch_bounds__(kPlThreads) plan_device_kernel(const PlanParams p) {
  extern __shared__ __align__(16) uint32_t pl_smem[];
  __shared__ int wsum[kPlWarps];
  __shared__ unsigned long long wsum3[kPlWarps];
  __shared__ int csum[3][kPlWarps];
  __shared__ int hist[32 * 33];
  __shared__ int s_max;
  __shared__ unsigned long long s_total;
  const int V = p.batch * p.q_len;
  uint32_t* keys = pl_smem;                                // [2][2 V]
  float* nf = reinterpret_cast<float*>(keys + 4 * V);      // [V] own pages
  int* S = reinterpret_cast<int*>(nf + V);                 // [V] splits
  int* skip = S + V;                                       // [V] shared pages
  int* start = skip + V;                                   // [V + 1] first split (items without the head groups)
  int* off = start + V + 1;                                // [V + 1] first partial slot
  int* rk = off + V + 1;                                   // [2 V] first rank of (v, size class)
  uint16_t* at = reinterpret_cast<uint16_t*>(rk + 2 * V);  // [2 V] a key's place in its warp
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid < 3 * kPlWarps) csum[tid / kPlWarps][tid % kPlWarps] = 0;
  if (tid == 0) {
    s_max = 1;
    s_total = 0;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int32_t flags = 0;
  // the groups must be ranges in order; otherwise no sequence has a shared prefix
  int groups = p.num_groups;
  {
    bool bad = false;
    for (int g = tid; g < groups; g += kPlThreads) {
      const int a = p.group_offsets[g], e = p.group_offsets[g + 1];
      if (a < 0 || e < a || e > p.batch) bad = true;
      start[g] = a;  // start and off: the groups' first sequences and pages for now
      if (g == groups - 1) start[groups] = e;
      off[g] = min(max(p.prefix_lens[g], 0) / kPlPage, p.max_pages);
    }
    if (__syncthreads_or(bad ? 1 : 0)) {
      flags |= KVQ_DEV_BAD_PLAN;
      groups = 0;
    }
  }
  // ---- own pages
  int my_max = 1;
  unsigned long long my_total = 0;
  for (int v = tid; v < V; v += kPlThreads) {
    const int b = v / p.q_len, i = v - b * p.q_len;
    int L = p.seq_lens[b];
    if (L < 0 || L > p.max_pages * kPlPage) {
      flags |= KVQ_DEV_BAD_SEQLEN;
      L = L < 0 ? 0 : p.max_pages * kPlPage;
    }
    const int vis = max(0, L - p.q_len + 1 + i);
    int sk = 0;
    if (groups > 0 && b >= start[0] && b < start[groups]) {
      int lo = 0, hi = groups - 1;  // last group that starts at or before b (behind empty ones)
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= b) lo = mid;
        else hi = mid - 1;
      }
      sk = off[lo];
    }
    const int n = max(0, (vis + kPlPage - 1) / kPlPage - sk);
    nf[v] = static_cast<float>(n);
    skip[v] = sk;
    my_max = max(my_max, n);
    my_total += n;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    my_max = max(my_max, __shfl_xor_sync(0xffffffffu, my_max, o));
    my_total += __shfl_xor_sync(0xffffffffu, my_total, o);
  }
  if (lane == 0 && my_total) {
    atomicMax(&s_max, my_max);
    atomicAdd(&s_total, my_total);
  }
  __syncthreads();
  // ---- x: rounds of 32 >> cs candidates, 2^cs warps each
  // An item costs a CTA about as much as 8 pages besides its own, so where the splits would
  // be short one wave of them is faster (prefix call, us, one wave / two: 64 sequences, 8 KV
  // heads of 128, INT8, own lengths below 256 21.6 / 25.4, 1,024 31.5 / 33.3, 2,048 (27 pages
  // a split) 51.2 / 48.1, 8,192 161.9 / 107.3; 100 sequences, 4 heads of 256: 36.2 / 43.0,
  // 55.9 / 60.7, 76.5 / 77.5, 193 / 168).
  const int T = p.few_splits > 0 && s_total <= 14ull * p.items_splits ? p.few_splits : p.items_splits;
  // ceil(total / T) <= x, and x <= ceil(total / (T - V)); the factors cover the quotients' rounding (2^-22)
  const float total = static_cast<float>(s_total);
  int lo = max(1, static_cast<int>(ceilf(total * reciprocal(T) * (1.f - 0x1p-21f))));
  int hi = s_max;
  if (T > V) hi = static_cast<int>(fminf(static_cast<float>(hi), ceilf(total * reciprocal(T - V) * (1.f + 0x1p-21f))));
  hi = max(hi, lo);
  int cs = 0;
  while (cs < 4 && (512 << cs) < V) ++cs;
  const int lc = 5 - cs;  // log2 of the candidates
  auto candidate = [&](int c) { return lo + static_cast<int>((int64_t)(hi - lo) * c >> lc); };
  // three buffers of sums: the one cleared in a round was read in the round before
  for (int round = 0; lo < hi; round = round == 2 ? 0 : round + 1) {
    const int xc = candidate(warp >> cs);
    const float x = static_cast<float>(xc), rx = reciprocal(xc);
    int sum = 0;
#pragma unroll 4
    for (int v = lane + 32 * (warp & ((1 << cs) - 1)); v < V; v += 32 << cs) sum += max(1, ceil_div_pages(nf[v], x, rx));
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (lane == 0) atomicAdd(&csum[round][warp >> cs], sum);
    __syncthreads();
    const unsigned ok = __ballot_sync(0xffffffffu, lane < (1 << lc) && csum[round][lane] <= T);
    if (tid < 32) csum[round == 0 ? 2 : round - 1][lane] = 0;
    const int w = ok ? __ffs(ok) - 1 : 1 << lc;  // first candidate that fits (larger ones do too)
    const int c_prev = w > 0 ? candidate(w - 1) : lo - 1;
    const int c_at = w < (1 << lc) ? candidate(w) : hi;
    lo = c_prev + 1;
    hi = c_at;
  }
  // ---- splits, the leftover in order, partial slots: one scan of (S, what x - 1 would
  // give more, sequences with shared pages), 20 + 28 + 16 bits: sum S <= T <= 2^15, and
  // sum ceil(n / (x - 1)) <= 2 sum ceil(n / x) + V
  const float x = static_cast<float>(lo), rx = reciprocal(lo);
  const float x1 = static_cast<float>(max(1, lo - 1)), rx1 = reciprocal(max(1, lo - 1));
  unsigned long long carry3 = 0;
  for (int v0 = 0; v0 < V; v0 += kPlThreads) {
    const int v = v0 + tid;
    unsigned long long mine = 0;
    if (v < V) {
      const int s = max(1, ceil_div_pages(nf[v], x, rx));
      const int d = lo > 1 ? max(1, ceil_div_pages(nf[v], x1, rx1)) - s : 0;
      mine = (unsigned long long)s | ((unsigned long long)d << 20) | (skip[v] > 0 ? 1ull << 48 : 0ull);
    }
    unsigned long long tot;
    const unsigned long long inc = block_scan<unsigned long long>(mine, wsum3, &tot);
    if (v < V) {
      const unsigned long long ex = carry3 + inc - mine;
      S[v] = static_cast<int>(mine & 0xFFFFF);
      start[v] = static_cast<int>(ex & 0xFFFFF);               // the leftover is added below
      rk[v] = static_cast<int>((ex >> 20) & 0xFFFFFFF);        // sum of d before v
      off[v] = static_cast<int>(ex >> 48);
    }
    carry3 += tot;
  }
  const int left = T - static_cast<int>(carry3 & 0xFFFFF);
  const int sum_d = static_cast<int>((carry3 >> 20) & 0xFFFFFFF);
  __syncthreads();
  const int even = left / V, odd = left - even * V;  // x = 1: all take `even`, the first `odd` one more
  // extra splits before sequence v (v = V: all of them)
  auto extra_before = [&](int v) {
    return lo > 1 ? min(left, v < V ? rk[v] : sum_d) : v * even + min(v, odd);
  };
  // (start and off still hold the sums before v; each thread rewrites its own)
  int ib = 0;  // bits of a key's place
  while ((1 << ib) < 2 * V) ++ib;
  for (int v = tid; v < V; v += kPlThreads) {
    // size classes, largest first: class 0 of v (key 2 v) has floor + 1, class 1 floor; no
    // split has more than x = lo pages, so a size is at most lo + 1
    const int s = S[v] + extra_before(v + 1) - extra_before(v);
    const uint32_t size = static_cast<uint32_t>(div_pages(nf[v], s));
    *reinterpret_cast<uint2*>(keys + 2 * v) = make_uint2((lo - size) << ib | 2 * v, (lo + 1 - size) << ib | (2 * v + 1));
  }
  __syncthreads();
  for (int v = tid; v < V; v += kPlThreads) {
    const int e = extra_before(v);
    const int st = start[v] + e;
    S[v] += extra_before(v + 1) - e;
    start[v] = st;
    off[v] = st + off[v] * p.prefix_splits;
  }
  if (tid == 0) {
    start[V] = T;
    off[V] = T + static_cast<int>(carry3 >> 48) * p.prefix_splits;
  }
  __syncthreads();
  const uint32_t* sorted = sort_keys(keys, keys + 2 * V, at, hist, wsum, 2 * V, ib, 32 - __clz(lo + 1));
  // ---- first rank of each size class
  int carry_r = 0;
  for (int k0 = 0; k0 < 2 * V; k0 += kPlThreads) {
    const int k = k0 + tid;
    int cnt = 0, id = 0;
    if (k < 2 * V) {
      id = static_cast<int>(sorted[k] & ((1u << ib) - 1));
      const int v = id >> 1;
      const int big = static_cast<int>(nf[v]) - div_pages(nf[v], S[v]) * S[v];  // splits of the larger size
      cnt = (id & 1) == 0 ? big : S[v] - big;
    }
    int tot;
    const int inc = block_scan<int>(cnt, wsum, &tot);
    if (k < 2 * V) rk[id] = carry_r + inc - cnt;
    carry_r += tot;
  }
  __syncthreads();
  // ---- the plan
  const int C = p.num_ctas, N = T * p.head_groups;
  const int A = (V + 2 + 3) & ~3;
  const int rest_at = (A + 5 * C + 1 + 3) & ~3;
  const int full = N / C, rem = N - full * C;
  int32_t* plan = p.plan;
  for (int v = tid; v <= V; v += kPlThreads) plan[v] = off[v];
  for (int i = V + 1 + tid; i < A; i += kPlThreads) plan[i] = i == V + 1 ? C : 0;
  auto rest_of = [&](int c) {  // rest entries of the CTAs before c
    return c * (full - 1) + ((full & 1) ? max(0, c - (C - rem)) : min(c, rem));
  };
  for (int c = tid; c <= C; c += kPlThreads) plan[A + 4 * C + c] = rest_of(c);
  for (int i = A + 5 * C + 1 + tid; i < rest_at; i += kPlThreads) plan[i] = 0;
  int4* firsts = reinterpret_cast<int4*>(plan + A);
  int4* rest = reinterpret_cast<int4*>(plan + rest_at);
  for (int it = tid; it < T; it += kPlThreads) {
    int l = 0, h = V - 1;
    while (l < h) {
      const int mid = (l + h + 1) >> 1;
      if (start[mid] <= it) l = mid;
      else h = mid - 1;
    }
    const int v = l, k = it - start[v], n = static_cast<int>(nf[v]), s = S[v];
    const int f = div_pages(nf[v], s), r = n - f * s;
    const int extra = static_cast<int>(static_cast<uint32_t>(k) * r / s);  // larger splits before k
    const int size = f + (k * r - extra * s + r >= s ? 1 : 0);
    const int shared = skip[v] > 0 ? p.prefix_splits : 0;
    const int rank0 = (size > f ? rk[2 * v] + extra : rk[2 * v + 1] + k - extra);
    int4 d;
    d.x = v;
    d.y = off[v] + shared + k;
    d.z = skip[v] + k * f + extra;
    const int w = size | ((s + shared == 1 ? 1 : 0) << 23);
    for (int g = 0; g < p.head_groups; ++g) {
      const int rank = rank0 * p.head_groups + g;
      const int rnd = static_cast<int>(static_cast<uint32_t>(rank) / C), j = rank - rnd * C;
      const int c = (rnd & 1) ? C - 1 - j : j;
      d.w = w | (g << 24);
      if (rnd == 0) firsts[c] = d;
      else rest[rest_of(c) + rnd - 1] = d;
    }
  }
  if (flags) atomicOr(p.status, flags);
  // A decode with KVQ_EARLY_START behind another call of this library may read the plan
  // before this grid counts as complete: the plan is in global memory when this block ends.
  asm volatile("fence.acq_rel.gpu;" ::: "memory");
}

}  // namespace

int plan_device_keys(int v) { return pow2_at_least(2 * v); }

int plan_device_smem_bytes(int v) { return 4 * (12 * v + 2); }

const void* plan_device_kernel_fn() { return reinterpret_cast<const void*>(&plan_device_kernel); }

cudaError_t launch_plan_device(const PlanParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kPlThreads);
  cfg.dynamicSmemBytes = plan_device_smem_bytes(p.batch * p.q_len);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, plan_device_kernel, p);
}

}  // namespace kvq
