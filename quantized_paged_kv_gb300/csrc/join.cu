// join.cu — the log-sum-exp join of a prefix call's partials: the shared pages' (one a
// key range) and the own pages' (one a split) of every query row.
//
//   M = max_s lse_s,  w_s = exp(lse_s - M),  out = sum_s w_s o_s / sum_s w_s,
//   lse = M + ln(sum_s w_s);  a partial with lse = -inf (no visible token) has weight 0,
//   one with lse = NaN (a NaN logit among the shared tokens) makes the row NaN.
//
// The same combination as the merge kernel's, shaped for what a prefix call leaves:
// hundreds to thousands of rows of 10 to 40 partials (the merge kernel serves one long
// sequence's ~150 as well, with few rows in flight).  The partials come from L2 (a few
// to 20 MB, written just before), so it is bound by how many loads are under way: a
// warp takes 128 columns of a row, lane s reads partial s's lse, and 8 or 16 partials of a
// row are in flight a warp; the slot offsets are read before the wait for the
// kernels that write the partials (the prefix kernel, or a decode on its own, has waited
// for whatever wrote them before it lets this grid start).  With few rows several warps share one (a row's
// partials in turn) and combine through shared memory.
// Measured as what a whole prefix call takes less (24 query heads of 256, CUDA graph,
// against the merge kernel in its place, 10.8, 10.5 and 8.2 us of the call there): 32
// sequences on 32K shared tokens 79.8 -> 76 us, 48 on 16K in NVFP4 49.2 -> 46, 16 of
// four query tokens on 8K 44.4 -> 42 (the converters' earlier loads had a part in it).
#include <algorithm>

#include "kvq_internal.h"
#include "kvq_ptx.cuh"

namespace kvq {
namespace {

constexpr int kJoinWarps = 8;

template <int kJoinFlight>  // partials in flight a warp
__global__ void __launch_bounds__(kJoinWarps * 32)
    join_kernel(const float* __restrict__ o_part, const float* __restrict__ lse_part,
                const int32_t* __restrict__ offs, int total_splits, int rows, int num_q_heads, int D, int wpr, void* out,
                int out_bf16, float* lse_out, int32_t* status) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float4 red_o[kJoinWarps][32];
  __shared__ float red_w[kJoinWarps], red_m[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slices = D / 128;
  // task = (row, slice), the slice fastest; wpr warps a task
  const int64_t task = ((int64_t)blockIdx.x * kJoinWarps + warp) / wpr;
  const int sub = warp % wpr;
  const int row = static_cast<int>(task / slices), slice = static_cast<int>(task - (int64_t)row * slices);
  int n = 0, base = 0, g = 0;
  if (row < rows) {
    const int v = row / num_q_heads;  // launch sequence
    g = row - v * num_q_heads;
    base = offs[v];
    n = offs[v + 1] - base;
    if (base < 0 || n < 1 || n > total_splits || base > total_splits - n) {  // not a plan for this call
      n = 0;
      base = 0;
      if (lane == 0) atomicOr(status, KVQ_DEV_BAD_PLAN);
    }
  }
  const bool active = n > 1;  // a single partial was written directly
  const float* lrow = lse_part + (size_t)base * num_q_heads + g;
  const float4* orow = reinterpret_cast<const float4*>(o_part + ((size_t)base * num_q_heads + g) * D + slice * 128) + lane;
  const size_t ostep = (size_t)num_q_heads * D / 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, wsum = 0.f;
  if (active) {
    // this warp's partials are sub, sub + wpr, ...; 32 of them a round (a lane each)
    const int mine = (n - sub + wpr - 1) / wpr;
    orow += (size_t)sub * ostep;
    lrow += (size_t)sub * num_q_heads;
#pragma unroll 1
    for (int s0 = 0; s0 < mine; s0 += 32) {
      const int left = min(32, mine - s0);
      const float l = lane < left ? __ldcg(lrow + (size_t)((s0 + lane) * wpr) * num_q_heads) : -INFINITY;
      float4 v[kJoinFlight];
      auto load = [&](int u0) {
#pragma unroll
        for (int u = 0; u < kJoinFlight; ++u)
          if (u0 + u < left) v[u] = __ldcg(orow + (size_t)((s0 + u0 + u) * wpr) * ostep);
      };
      load(0);
      float mn = fmaxf(m, l);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      const float w = l == -INFINITY ? 0.f : expf(l - mn);
      const float sc = m == -INFINITY ? 0.f : expf(m - mn);
      wsum = wsum * sc + w;  // a lane's part
      m = mn;
      acc.x *= sc;
      acc.y *= sc;
      acc.z *= sc;
      acc.w *= sc;
#pragma unroll 1
      for (int u0 = 0;;) {
#pragma unroll
        for (int u = 0; u < kJoinFlight; ++u) {
          const float wu = __shfl_sync(0xffffffffu, w, u0 + u);
          if (wu != 0.f) {  // also leaves out what was not loaded
            acc.x += wu * v[u].x;
            acc.y += wu * v[u].y;
            acc.z += wu * v[u].z;
            acc.w += wu * v[u].w;
          }
        }
        u0 += kJoinFlight;
        if (u0 >= left) break;
        load(u0);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) wsum += __shfl_xor_sync(0xffffffffu, wsum, o);
  }
  if (wpr > 1) {
    red_o[warp][lane] = acc;
    if (lane == 0) {
      red_w[warp] = wsum;
      red_m[warp] = m;
    }
    __syncthreads();
    if (sub != 0) return;
    float mn = m;
    for (int j = 1; j < wpr; ++j) mn = fmaxf(mn, red_m[warp + j]);
    const float s0 = mn == -INFINITY ? 0.f : expf(m - mn);
    wsum *= s0;
    acc.x *= s0;
    acc.y *= s0;
    acc.z *= s0;
    acc.w *= s0;
    for (int j = 1; j < wpr; ++j) {
      const float sj = mn == -INFINITY ? 0.f : expf(red_m[warp + j] - mn);
      const float4 v = red_o[warp + j][lane];
      wsum += red_w[warp + j] * sj;
      acc.x += v.x * sj;
      acc.y += v.y * sj;
      acc.z += v.z * sj;
      acc.w += v.w * sj;
    }
    m = mn;
  }
  if (!active) return;
  const float inv = wsum != 0.f ? 1.f / wsum : 0.f;  // NaN stays NaN
  acc.x *= inv;
  acc.y *= inv;
  acc.z *= inv;
  acc.w *= inv;
  const size_t at = (size_t)row * D + slice * 128 + 4 * lane;
  if (out_bf16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x, acc.y), b = __floats2bfloat162_rn(acc.z, acc.w);
    uint2 w;
    w.x = *reinterpret_cast<const uint32_t*>(&a);
    w.y = *reinterpret_cast<const uint32_t*>(&b);
    *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(out) + at) = w;
  } else {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + at) = acc;
  }
  if (lse_out && slice == 0 && lane == 0) lse_out[row] = wsum != 0.f ? m + logf(wsum) : -INFINITY;
}

}  // namespace

cudaError_t launch_join(const float* o_part, const float* lse_part, const int32_t* offsets, int batch, int total_splits,
                        int num_q_heads, int head_dim, void* out, int out_bf16, float* lse_out,
                        int32_t* status, int sms, cudaStream_t stream) {
  const int64_t rows = (int64_t)batch * num_q_heads;
  const int64_t tasks = rows * (head_dim / 128);
  // warps a row: doubled while they all fit in two blocks an SM and each is left four partials
  // or more; in four blocks an SM if each is left eight (one against two warps a row: 768
  // rows of 24 partials 77.2 -> 74.7 us of the prefix call, 1,152 rows of 15 47.4 -> 49.1)
  // Against all of 1, 2, 4, 8 warps x 8, 16 in flight on eleven other shapes (8 to 128 rows of
  // 5 to 64 heads, 6 to 66 partials, D 128 and 256): within 3 % of the call's best on ten, 8 % above
  // it on the other (40 x 24 rows of 19 partials, D = 256: 26.6 us, 24.6 with one warp a row and 16).
  const int n = total_splits / batch;
  int wpr = 1;
  while (wpr < kJoinWarps && n >= 8 * wpr && 2 * wpr * tasks <= (int64_t)(n >= 16 * wpr ? 4 : 2) * sms * kJoinWarps) wpr *= 2;
  const int64_t blocks = (tasks * wpr + kJoinWarps - 1) / kJoinWarps;
  // 16 partials in flight a warp while two blocks an SM (their registers) hold all rows, 8 above
  // (8 against 16: 256 blocks of 10 partials 34.1 -> 33.3 us of the prefix call, 180 of 9 39.5 ->
  // 38.5, 384 blocks of 14 and 24 partials 41.4 -> 43.2 and 74.9 -> 77.3)
  const auto kernel = blocks <= 2 * (int64_t)sms ? &join_kernel<16> : &join_kernel<8>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, o_part, lse_part, offsets, total_splits, static_cast<int>(rows),
                            num_q_heads, head_dim, wpr, out, out_bf16, lse_out, status);
}

}  // namespace kvq
