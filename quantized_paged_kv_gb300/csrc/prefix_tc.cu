// prefix_tc.cu — attention of a batch over the pages its sequences share (a common
// prompt), each page read once for its group, on the fifth-generation tensor cores
// (tcgen05.mma, accumulators in TMEM).
//
// A softmax over (shared tokens, own tokens) splits into partials (o, lse) that the
// log-sum-exp merge joins exactly, as it joins the splits of one sequence:
//   o = sum_j exp(z_j - m) v_j / l,  lse = m + ln l,  l = sum_j exp(z_j - m).
// This kernel makes the partials of the shared pages; the decode kernel makes those
// of each sequence's own pages; the join kernel combines them.
//
// The rows of a group are its (sequence, query token, query head) triples of one KV
// head: with tens of sequences a page serves hundreds of rows, so the contraction is
// GEMM-shaped (2 D multiply-adds a (row, key) against D code bytes a key) and bound
// by the tensor cores, not by HBM as a decode is.
//
// Work item (one CTA): 128 rows of one KV head of one group against one range of the
// group's shared pages, in tiles of 64 keys.  Warp roles (16 warps, the most that
// leave a thread 128 registers):
//   * warps 0..3 and 4..7 (softmax): two groups take alternate tiles, so that one
//     tile's exponentials run while the tensor cores and the other group work on its
//     neighbours.  One row a thread: S from TMEM, the online softmax, P over S(i) in
//     TMEM as the A operand of the P V product (hi + lo terms when the call's output
//     is fp32, or the cache BF16).  The groups share the rows' running references (they scale one O): the
//     reference after tile i goes from warp to warp through shared memory, each row's
//     sum stays with its group (two partial sums, joined at the end).
//   * warp 8 (MMA): S(i) = Q K(i)^T into one of three (D = 128: four) TMEM
//     buffers, two (three) tiles ahead of O += P(i) V(i), so that a group finds its
//     next tile ready; each group of MMAs is committed to an mbarrier.
//   * warps 9..12 and 13..15 (converters of K and of V): take half tiles (32 keys) in
//     turn.  Eight lanes read 128 contiguous bytes of a row: with one row a thread every load
//     instruction touched 32 cache lines, whose lookups alone took ~2,000 cycles a
//     tile.  Codes -> fp16, the whole half in flight at once; BF16 rows go to shared
//     memory by cp.async, unconverted.
// The code is kept short (loops where registers allow): the roles run different code at
// once, and instruction fetch was a third of the warps' stalls.
// Measured (the kernel alone, nothing in L2): INT8, 4 heads of 256, fp32 output, 192 rows a
// head on 32K tokens 46.6 us, 553 TFLOP/s of q K and P V and 1,106 with P's lo terms and the
// empty rows of the second block (measured bf16 rate 1,951); INT8, 8 heads of 128, bf16 output,
// 256 rows a head on 2,048 tokens 11.7 us, 184 TFLOP/s: mostly a CTA's start and end.
// Every wait is bounded (%globaltimer); a timeout sets KVQ_DEV_TIMEOUT, the CTA waits
// for its issued MMAs, frees its TMEM and returns.
#include "tc_tile.cuh"

namespace kvq {
namespace {

constexpr int kPxRows = 128;               // query rows of an item (the MMA's M)
constexpr int kPxKeys = 64;                // keys of a tile
constexpr int kPxPages = kPxKeys / kPage;  // pages of a tile
constexpr int kPxSoft = 256;               // softmax threads
constexpr int kPxMmaWarp = 8;
constexpr int kPxConvK = 9, kPxConvV = 13, kPxWarps = 16;  // first converter warp of K, of V
constexpr int kPxThreads = 16 * 32;
constexpr float kPxRescale = 8.0f;  // log2 of the largest p a stale maximum may give
constexpr int kPxScaleRise = 4;     // log2 of the growth of V scales within one unit
constexpr int kNoScale = -10000;

template <int FMT, int D>
struct PxLayout {
  static constexpr int kAtoms = D / 64;                  // 128-byte swizzle atoms along D (fp16)
  // a K or V tile: [8-key group][d atom of 64][8 keys][128 B], 128-byte swizzle, read
  // K-major (K: rows = keys) or MN-major (V: rows of d); one layout, one converter
  static constexpr int kKBytes = kPxKeys * D * 2;
  static constexpr int kVBytes = kPxKeys * D * 2;
  static constexpr uint32_t kAtomBytes = 1024, kGroupBytes = kAtoms * 1024;
  // five tiles fit at D = 256: S runs ahead, so K(i+2) has two tiles' time to be converted
  // once S(i) has left its stage, V(i+2) only one
  static constexpr int kKStages = D == 256 ? 2 : 3;
  static constexpr int kVStages = 3;
  static constexpr int kKAt = 0;                         // K tiles
  static constexpr int kVAt = kKAt + kKStages * kKBytes;   // V tiles
  static constexpr int kTilesEnd = kVAt + kVStages * kVBytes;
  // q rows on their way to TMEM, padded so that a thread a row reads without
  // conflicts: over the tiles, whose converters wait until q is read
  static constexpr int kQRow = 2 * D + 16;
  static constexpr int kQAt = kTilesEnd - (kPxRows * kQRow + 1023) / 1024 * 1024;
  static constexpr bool kQOverK = kQAt < kVAt;
  static_assert(kQAt >= kVAt - kKBytes, "q staging covers V tiles and at most the last K tile");
  // the epilogue's patches of 32 rows x 32 columns of O, one a softmax warp, over the
  // tiles (all MMAs are done then); padded against bank conflicts
  static constexpr int kORow = 128 + 16;
  static constexpr int kOPatch = 32 * kORow;
  static constexpr int kOAt = 0;
  static_assert(8 * kOPatch <= kTilesEnd, "staging");
  // Q's elements from kQTmem on, as a K-major A operand [atom][128 rows][128 B]: at D =
  // 256 half of Q leaves TMEM to a third S buffer
  static constexpr int kQTmem = D == 256 ? 128 : D;
  static constexpr int kQSmemAt = kTilesEnd;
  static constexpr int kQSmemBytes = (D - kQTmem) * 2 * kPxRows;
  // a slot of the scale ring is written for tile i once S(i-3) (D = 256: S(i-2)) is done,
  // which was issued after P(i-7) V(i-7) at the latest: the softmax of tile i-8, the slot's
  // last tile, has read it
  static constexpr int kScRing = 8;
  static constexpr int kScAt = kQSmemAt + kQSmemBytes;   // float k scales [8][64], v scales [8][64]
  static constexpr int kBadAt = kScAt + 2 * kScRing * kPxKeys * 4;  // uint32 [8][2]: bit j = page j of the half not read
  static constexpr int kExpAt = kBadAt + 8 * kScRing;    // int32 [8][2]: exponent of the half's largest V scale
  static constexpr int kMaxAt = kExpAt + 8 * kScRing;    // float [2][128] running maxima, [2][128] sums
  static constexpr int kQOffAt = kMaxAt + 4 * kPxRows * 4;    // int32 [128] q row index (-1: no live row)
  static constexpr int kLimAt = kQOffAt + kPxRows * 4;        // int32 [128] tokens each row sees
  static constexpr int kORowAt = kLimAt + kPxRows * 4;        // int32 [128] partial row
  static constexpr int kBarAt = kORowAt + kPxRows * 4;
  static constexpr int kNumBars = 32;
  static constexpr int kSlotAt = kBarAt + kNumBars * 8;
  static constexpr int kSmemBytes = 1024 + kSlotAt + 16;
  static_assert(kSmemBytes <= 226 * 1024, "shared memory budget");
  // TMEM columns: O (D), the S buffers of 64, and Q (pairs of f16 / bf16).  P(i) is
  // written over S(i) once the softmax has read S(i): for each 16 keys 8 columns of hi
  // pairs, then 8 of lo pairs, the A operand of O += P V.  Q's part is the A operand of
  // S = Q K^T.
  static constexpr int kSBufs = D == 256 ? 3 : 4;
  static constexpr int kLook = kSBufs - 1;  // tiles that S runs ahead of P V
  static constexpr uint32_t kTmemO = 0;
  static constexpr uint32_t kTmemS = D;
  static constexpr uint32_t kTmemQ = D + kSBufs * kPxKeys;
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kTmemQ + kQTmem / 2 <= kTmemCols, "TMEM columns");
  // converters: LPR lanes share a row's 128 bytes (64 bytes: NVFP4 at D = 128), a warp
  // covers RPP rows a pass; its chunks of a page go out and are converted together
  static constexpr int kRow = DecodeTraits<FMT, D>::kRow;
  static constexpr int kCpr = kRow / 16;               // 16-byte chunks of a row
  static constexpr int kLpr = kCpr < 8 ? kCpr : 8;
  static constexpr int kSets = kCpr / kLpr;            // chunks of a row a lane takes
  static constexpr int kRpp = 32 / kLpr;
  static constexpr int kPasses = kPage / kRpp;         // of a page
  static constexpr int kPer = kSets * kPasses;         // chunks a lane takes of a page
  static constexpr int kPhases = 8 / kRpp;             // passes of an 8-key group
};

// A parity wait tells a phase from its neighbours only, so a waiter must know that the
// phase before the one it waits for is over, and that the next cannot end without it.
// Hence a barrier for every stage and buffer, and: a converter's previous wait covered a
// tile at most two back, which is past the phase before (stages 3, or 2 for K); a
// softmax warp has seen S(i), which was issued after P(i-4) V(i-4).  V(i) shares the
// barrier of P(i) (one wait fewer for the MMA warp): the buffer's next V comes after
// P(i) V(i), which its stage waits for.
enum : int {
  kBarQ = 0,             // q in TMEM and shared memory (softmax warps)
  kBarP0,                // [4] P(i) written over S(i) (four softmax warps), V(i) converted (two half tiles)
  kBarK0 = kBarP0 + 4,   // [3] K(i) converted (two half tiles)
  kBarKF0 = kBarK0 + 3,  // [3] S(i) done (commit): K stage free
  kBarVF0 = kBarKF0 + 3, // [3] P(i) V(i) done (commit): V stage free
  kBarS0 = kBarVF0 + 3,  // [4] S(i) done (commit): readable
  kBarO0 = kBarS0 + 4,   // [4] P(i) V(i) done (commit): O holds it
  kBarM0 = kBarO0 + 4,   // [2][4] row references after tile i, one a softmax warp
  kBarFinal = kBarM0 + 8,
  kBarCount
};

// packed fp32 pairs: two IEEE round-to-nearest operations in one instruction
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) { return pair(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float ex2(float x) {  // ex2.approx.ftz: results below 2^-126 are 0, of -inf exactly 0
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void st_shared16(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void l2_prefetch(const void* src, uint32_t bytes) {  // both multiples of 16
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Element d of a pool row.
template <int FMT, int D>
__device__ __forceinline__ float pool_value(const uint8_t* codes, const uint8_t* scales, int64_t row, int d) {
  if constexpr (FMT == KVQ_FMT_BF16) {
    return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(codes)[row * D + d] << 16);
  } else if constexpr (FMT == KVQ_FMT_INT8) {
    return static_cast<float>(reinterpret_cast<const int8_t*>(codes)[row * D + d]) *
           reinterpret_cast<const float*>(scales)[row];
  } else {
    const uint32_t n = codes[row * (D / 2) + d / 2] >> (4 * (d & 1));
    const uint32_t two = n & 6u;  // E2M1: 0, 0.5, then (1 + half the low bit) x 2^((n & 6) / 2 - 1)
    const float mag = two ? (1.f + 0.5f * static_cast<float>(n & 1u)) * pow2f(static_cast<int>(two >> 1) - 1)
                          : 0.5f * static_cast<float>(n & 1u);
    const float s = __low2float(u32_as_h2(e4m3x2_to_h2(scales[row * (D / 16) + d / 16])));
    return ((n & 8u) ? -mag : mag) * s;
  }
}

// One row's result over keys [16 pg0, kend) of a range, key after key by a whole warp:
// columns [col, col + D / 2), given the row's m and 1 / l (x 1 / gs_V).  For rows whose O a
// NaN or an infinity spoiled that lies behind their last key (0 x NaN in the P V product),
// which no pool of finite values brings here: it is out of line, and slow.
template <int FMT, int D>
__device__ __noinline__ void redo_row(const uint16_t* q, const uint8_t* k_codes, const uint8_t* k_scales,
                                      const uint8_t* v_codes, const uint8_t* v_scales, const int32_t* btab, int num_pages,
                                      int num_kv_heads, int h, int pg0, int kend, int col, float scale, float m,
                                      float inv, float* out) {
  constexpr int EK = D / 32, EV = D / 64;  // elements of K and of V a lane
  const int lane = threadIdx.x & 31;
  float qv[EK], acc[EV];
#pragma unroll
  for (int e = 0; e < EK; ++e) qv[e] = __uint_as_float((uint32_t)q[EK * lane + e] << 16);
#pragma unroll
  for (int e = 0; e < EV; ++e) acc[e] = 0.f;
  for (int key = pg0 * kPage; key < kend; ++key) {
    const int id = btab[key / kPage];
    if (id < 0 || id >= num_pages) continue;  // left out, as in the tiles
    const int64_t row = ((int64_t)id * num_kv_heads + h) * kPage + key % kPage;
    float z = 0.f;
#pragma unroll
    for (int e = 0; e < EK; ++e) z = fmaf(qv[e], pool_value<FMT, D>(k_codes, k_scales, row, EK * lane + e), z);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    const float pr = ex2(z * scale - m);
#pragma unroll
    for (int e = 0; e < EV; ++e) acc[e] = fmaf(pr, pool_value<FMT, D>(v_codes, v_scales, row, col + EV * lane + e), acc[e]);
  }
#pragma unroll
  for (int e = 0; e < EV; ++e) out[col + EV * lane + e] = acc[e] * inv;
}
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kPxSoft) : "memory"); }

template <int FMT, int D, bool PLO>
__global__ void __launch_bounds__(kPxThreads, 1)
    prefix_tc_kernel(const PrefixParams p) {
  using T = DecodeTraits<FMT, D>;
  using Lo = PxLayout<FMT, D>;
  constexpr bool kBf16 = T::kBf16Mma;
  constexpr int KS = D / 16;  // k-steps of S
  // INT8 with bf16 output: V's scales go into the V tile, fp16(code x scale 2^-e) (two
  // roundings of 2^-11, an eighth of the output's own 2^-8; P has one more), which spares the
  // softmax a multiplication and a shared-memory read a key.  2^e is the unit of 32 keys: a
  // scale below 2^-14 of their largest is subnormal in fp16, its key's V off by up to 2^-24 of
  // the largest |V| among them, as P' is with the scales folded into it (see the softmax).
  // With fp32 output the tile holds the exact codes and the scales are folded into P.
  constexpr bool kFoldV = FMT == KVQ_FMT_INT8 && !PLO;
  constexpr uint32_t kIdescS = umma_idesc_f16(kPxRows, kPxKeys, kBf16, false);
  constexpr uint32_t kIdescPV = umma_idesc_f16(kPxRows, D, kBf16, true);
  static_assert(kBarCount <= Lo::kNumBars, "barriers");
  static_assert(PLO || !kBf16, "a BF16 cache always takes two terms");

  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lo::kBarAt);
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + Lo::kSlotAt);  // [0] TMEM base, [1] abort flag
  float* ksc = reinterpret_cast<float*>(smem + Lo::kScAt);            // [8][64]
  float* vsc = ksc + Lo::kScRing * kPxKeys;                           // [8][64]
  uint32_t* bad_pages = reinterpret_cast<uint32_t*>(smem + Lo::kBadAt);
  [[maybe_unused]] int32_t* vexp = reinterpret_cast<int32_t*>(smem + Lo::kExpAt);
  float* m_sh = reinterpret_cast<float*>(smem + Lo::kMaxAt);          // [2][128]
  float* l_sh = m_sh + 2 * kPxRows;                                   // [2][128]
  int32_t* qoff = reinterpret_cast<int32_t*>(smem + Lo::kQOffAt);
  int32_t* lims = reinterpret_cast<int32_t*>(smem + Lo::kLimAt);
  int32_t* orow_at = reinterpret_cast<int32_t*>(smem + Lo::kORowAt);
  const uint32_t sbase = smem_addr(smem);

  __shared__ int wlim[4];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int b = 0; b < kBarCount; ++b) {
      const int count = b == kBarQ ? 8 : b < kBarK0 ? 6 : b < kBarKF0 ? 2 : 1;
      mbar_init(&bars[b], count);
    }
    slot[1] = 0;
    fence_mbar_init();
  }
  if (warp == kPxMmaWarp) {
    tmem_alloc(slot, Lo::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // The launch is a programmatic dependent of the preceding kernel: the barriers
  // and the TMEM are set up while that kernel drains, and nothing it may write
  // (q, the block table, the sequence length, the pool) is read before it completes.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // nothing below depends on the grid that follows (it may be scheduled now)
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // work item: key range s, KV head h, flat row block k of all groups
  const int s = blockIdx.x, h = blockIdx.y, k = blockIdx.z;
  const int G = p.num_q_heads / p.num_kv_heads;
  // Row block k lies in group gi: 32 groups a step, blocks of a group = rows / 128
  // rounded up (none for a group without shared pages).  The groups must be ranges in
  // order (as for the plan): otherwise no sequence has a shared prefix and there is
  // nothing to do.  Every warp scans them all, so that none waits for another.
  int gi = -1, rb = 0, pages = 0, seq0 = 0, rows = 0;
  {
    int before = 0;
    bool bad = false;
    for (int g0 = 0; g0 < p.num_groups; g0 += 32) {
      const int g = g0 + lane;
      int off = 0, n = 0, pg = 0;
      if (g < p.num_groups) {
        off = p.group_offsets[g];
        const int end = p.group_offsets[g + 1];
        bad |= off < 0 || end < off || end > p.batch;
        pg = min(max(p.prefix_lens[g], 0) / kPage, p.max_pages);
        n = pg > 0 ? (end - off) * p.q_len * G : 0;
      }
      int inc = (n + kPxRows - 1) / kPxRows;
      const int mine = inc;
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, k < before + inc);
      if (hit && gi < 0) {
        const int src = __ffs(hit) - 1;
        gi = g0 + src;
        rb = k - before - __shfl_sync(0xffffffffu, inc - mine, src);
        pages = __shfl_sync(0xffffffffu, pg, src);
        seq0 = __shfl_sync(0xffffffffu, off, src);
        rows = __shfl_sync(0xffffffffu, n, src);
      }
      before += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (__any_sync(0xffffffffu, bad)) {
      if (threadIdx.x == 0) atomicOr(p.status, KVQ_DEV_BAD_PLAN);
      gi = -1;
      pages = 0;
    }
  }
  // Row threadIdx.x of the block (threads 0 .. 127): launch sequence vb (token i of
  // sequence vb / q_len) and query head; lim = the tokens that it sees
  const int rl = threadIdx.x & (kPxRows - 1);
  if (warp < 4) {
    const int row = rb * kPxRows + rl;
    int lim = 0, at = -1, slot_row = 0;  // slot_row: the row's place in the partials
    if (gi >= 0 && row < rows) {
      const int dv = row / G, qh = h * G + row - dv * G;
      const int di = p.q_len > 1 ? dv / p.q_len : dv;  // sequence of the group
      const int vb = seq0 * p.q_len + dv, b = seq0 + di;
      // partial slot: the sequence's first ones.  A plan made for other groups or
      // splits would put this elsewhere: such a row is left out, and flagged
      const int a = p.plan[vb], e = p.plan[vb + 1];
      int L = p.seq_lens[b];
      int flag = 0;
      if (L < 0 || L > p.max_pages * kPage) {
        flag = KVQ_DEV_BAD_SEQLEN;
        L = L < 0 ? 0 : p.max_pages * kPage;
      }
      if (a >= 0 && e <= p.total_splits && e - a > p.splits) {
        lim = max(0, L - p.q_len + 1 + dv - di * p.q_len);
        at = vb * p.num_q_heads + qh;
        slot_row = (a + s) * p.num_q_heads + qh;  // total_splits x Hq fits in 31 bits (checked by the host)
      } else {
        flag |= KVQ_DEV_BAD_PLAN;
      }
      if (flag) atomicOr(p.status, flag);
    }
    lims[rl] = lim;
    orow_at[rl] = slot_row;
    qoff[rl] = at;
    const int m = __reduce_max_sync(0xffffffffu, lim);
    if (lane == 0) wlim[warp] = m;
  }
  // this group's shared pages: the first entries of its first sequence's table row
  const int32_t* btab = p.block_tables + (size_t)seq0 * p.max_pages;
  const int pg0 = s * pages / p.splits, pg1 = (s + 1) * pages / p.splits;  // s < 64, pages < 2^21
  __syncthreads();
  // the block's furthest limit: keys past it are in no row's sequence, may never have
  // been written, and are not read
  const int blim = max(max(wlim[0], wlim[1]), max(wlim[2], wlim[3]));
  const int npg = max(0, min(pg1, (blim + kPage - 1) / kPage) - pg0);
  const int nt = (npg + kPxPages - 1) / kPxPages;
  const int key_end = min(blim, (pg0 + npg) * kPage);  // keys of this range (exclusive)
  const uint32_t tmem = slot[0];
  volatile uint32_t* abort_flag = slot + 1;
  auto wait = [&](int b, uint32_t parity) -> bool {  // one thread
    if (mbar_try_wait(&bars[b], parity)) return true;
    if (*abort_flag) return false;
    if (mbar_wait(&bars[b], parity, kWaitLimitNs)) return true;
    atomicOr(p.status, KVQ_DEV_TIMEOUT);
    *abort_flag = 1;
    return false;
  };
  auto wait_warp = [&](int b, uint32_t parity) -> bool {  // a whole warp, one answer for all its lanes
    return __all_sync(0xffffffffu, wait(b, parity));
  };

  if (warp == kPxMmaWarp) {
    // ================================================================== MMA issue
    // The whole warp runs the loop and one elected lane issues: addresses and
    // descriptors are then uniform over the warp, which the instructions want (issued
    // from a single lane's registers an MMA took ~80 cycles, whatever its size).
    if (nt > 0) {
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const bool leader = elect_one();
      bool ok = wait_warp(kBarQ, 0);
      tc_fence_after();
      // step i: S(i) (K(i) ready), then P(j) V(j) for j = i - kLook
      int ks = 0, vs = 0, sb = 0, pb = 0;  // stages of K(i) and V(j), buffers of S(i) and P(j)
      uint32_t kph = 0, pph = 0;           // the phases of K(i) and P(j)
      for (int i = 0; ok && i < nt + Lo::kLook; ++i) {
        if (i < nt) {
          if (!wait_warp(kBarK0 + ks, kph)) break;
          tc_fence_after();
          if (leader) {
            const uint32_t ds = tm + Lo::kTmemS + (uint32_t)sb * kPxKeys;
            // descriptors of a tile differ in the start address (a 14-bit field of 16 bytes)
            const uint64_t kd = umma_desc_sw128(sbase + Lo::kKAt + (uint32_t)ks * Lo::kKBytes, 16, Lo::kGroupBytes);
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) {  // k-step of 16 elements: 8 columns of Q
              const uint64_t bd = kd + (((kk >> 2) * Lo::kAtomBytes + 32 * (kk & 3)) >> 4);
              if (16 * kk < Lo::kQTmem) {
                umma_f16_ta(ds, tm + Lo::kTmemQ + 8 * kk, bd, kIdescS, kk > 0 ? 1u : 0u);
              } else {
                const int k2 = kk - Lo::kQTmem / 16;
                const uint64_t ad = umma_desc_sw128(sbase + Lo::kQSmemAt, 16, 1024) +
                                    (((k2 >> 2) * kPxRows * 128 + 32 * (k2 & 3)) >> 4);
                umma_f16(ds, ad, bd, kIdescS, 1u);
              }
            }
            umma_commit(&bars[kBarS0 + sb]);
            umma_commit(&bars[kBarKF0 + ks]);
          }
          __syncwarp();
          if (++ks == Lo::kKStages) {
            ks = 0;
            kph ^= 1;
          }
          if (++sb == Lo::kSBufs) sb = 0;
        }
        const int j = i - Lo::kLook;
        if (j >= 0) {
          if (!wait_warp(kBarP0 + pb, pph)) break;
          tc_fence_after();
          if (leader) {
            const uint64_t vd =
                umma_desc_sw128(sbase + Lo::kVAt + (uint32_t)vs * Lo::kVBytes, Lo::kAtomBytes, Lo::kGroupBytes);
            const uint32_t pa = tm + Lo::kTmemS + (uint32_t)pb * kPxKeys;  // P(j) over S(j), see the softmax
#pragma unroll
            for (int kk = 0; kk < kPxKeys / 16; ++kk)
              umma_f16_ta(tm + Lo::kTmemO, pa + 16 * kk, vd + (2 * kk * Lo::kGroupBytes >> 4), kIdescPV,
                          (j > 0 || kk > 0) ? 1u : 0u);
            if constexpr (PLO) {
#pragma unroll
              for (int kk = 0; kk < kPxKeys / 16; ++kk)
                umma_f16_ta(tm + Lo::kTmemO, pa + 16 * kk + 8, vd + (2 * kk * Lo::kGroupBytes >> 4), kIdescPV, 1u);
            }
            umma_commit(&bars[kBarO0 + (j & 3)]);
            umma_commit(&bars[kBarVF0 + vs]);
          }
          __syncwarp();
          if (++vs == Lo::kVStages) vs = 0;
          if (++pb == Lo::kSBufs) {
            pb = 0;
            pph ^= 1;
          }
        }
      }
      // every MMA that the leader issued has completed before the TMEM is freed
      if (leader) {
        umma_commit(&bars[kBarFinal]);
        if (!mbar_wait(&bars[kBarFinal], 0, kWaitLimitNs)) atomicOr(p.status, KVQ_DEV_TIMEOUT);
      }
      __syncwarp();
    }
  } else if (warp >= kPxConvK) {
    // ================================================================== converters
    // Unit u = (tile u / 2, half u % 2) of K or of V, its warps in turn.  The half's two
    // pages go to the tile's keys 32 half .. + 31.
    const bool is_v = warp >= kPxConvV;
    const int warps = is_v ? kPxWarps - kPxConvV : kPxConvV - kPxConvK;
    // This lane's chunk u0 and row rsub of a pass.  A 16-byte access is served eight lanes
    // at a time.  The lanes are dealt so that eight neighbours write to the eight
    // different 16-byte columns of the swizzled 128 bytes (a BF16 chunk is one column, so
    // eight chunks of a row; an INT8 chunk two, four chunks of two rows; an NVFP4 chunk
    // four, two chunks of four rows) and, by the XOR, read different 16-byte columns too.
    int rsub, u0;
    if constexpr (FMT == KVQ_FMT_BF16) {
      u0 = lane & 7;
      rsub = lane >> 3;
    } else if constexpr (FMT == KVQ_FMT_INT8) {
      rsub = ((lane >> 2) & 1) | ((lane >> 3) & 2);
      u0 = ((lane & 3) | ((lane >> 1) & 4)) ^ ((rsub & 1) << 2);
    } else if constexpr (Lo::kLpr == 8) {
      rsub = (lane >> 1) & 3;
      u0 = ((lane & 1) | ((lane >> 2) & 6)) ^ (rsub << 1);
    } else {
      rsub = ((lane >> 1) & 3) | ((lane >> 2) & 4);
      u0 = ((lane & 1) | ((lane >> 2) & 2)) ^ (rsub & 2);
    }
    // where this lane's eight-element blocks go in an 8-key group's pass (set 0)
    constexpr int NB = chunk_elems<FMT>() / 8;
    uint32_t at[Lo::kPhases][NB];
#pragma unroll
    for (int ps = 0; ps < Lo::kPhases; ++ps)
#pragma unroll
      for (int x = 0; x < NB; ++x)
        at[ps][x] = vtile_off<D>(ps * Lo::kRpp + rsub, chunk_elems<FMT>() * u0 + 8 * x);
    // block x of chunk (pass ps, set) of the half's page j: 8-key group 2 j + ps / kPhases
    auto place = [&](int j, int ps, int set, int x) -> uint32_t {
      return at[ps % Lo::kPhases][x] + (uint32_t)(2 * j + ps / Lo::kPhases) * Lo::kGroupBytes +
             (uint32_t)(set * chunk_elems<FMT>() / 8) * Lo::kAtomBytes;
    };
    // lane j holds the id of page j of the warp's next unit (-1: past the range)
    auto id_of = [&](int u) {
      const int jp = 2 * u + lane;
      return lane < 2 && jp < npg ? __ldg(btab + pg0 + jp) : -1;
    };
    const uint8_t* codes = (is_v ? p.v_codes : p.k_codes) + u0 * 16;
    const int stages = is_v ? Lo::kVStages : Lo::kKStages;
    // A unit's two pages as lane j sees page j: first pool row, readable rows, and which
    // ids lie outside the pool (left out and flagged).  A page that is not read takes
    // row 0 of the pool: its keys are masked, and whatever codes they hold decode to
    // finite values.
    struct Unit {
      int row, ok;
      uint32_t bad;
    };
    auto unit_of = [&](int u, int id) {
      const int nkeys = key_end - (pg0 + 2 * u) * kPage;  // keys of the half that are read
      const bool in_pool = id >= 0 && id < p.num_pages;
      Unit n;
      n.bad = __ballot_sync(0xffffffffu, !in_pool && lane < 2 && 2 * u + lane < npg);
      if (n.bad && lane == 0) atomicOr(p.status, KVQ_DEV_BAD_PAGE);
      n.row = in_pool ? (id * p.num_kv_heads + h) * kPage : 0;  // a pool has fewer than 2^31 rows
      n.ok = in_pool ? min(kPage, max(0, nkeys - kPage * lane)) : 0;
      return n;
    };
    auto wait_stage = [&](int i) -> bool {  // the stage's last tile is consumed, or (first round) q has left it
      const int stage = i % stages, round = i / stages;
      if (round == 0) return !(is_v || (Lo::kQOverK && stage == Lo::kKStages - 1)) || wait_warp(kBarQ, 0);
      return wait_warp((is_v ? kBarVF0 : kBarKF0) + stage, (round - 1) & 1);
    };
    int u = warp - (is_v ? kPxConvV : kPxConvK);
    const int units = 2 * nt;
    if constexpr (FMT == KVQ_FMT_NVFP4) {
      // A warp's registers hold half as many bytes in flight as with 8-bit rows, too few
      // for HBM, so the first units are fetched into L2 ahead (48 sequences on 16K
      // tokens, nothing in L2: 57 -> 53 us; 8-bit and 16-bit rows: 0 to 2 us slower).
      const int jp = 2 * (u + (lane >> 1) * warps) + (lane & 1);  // lanes 2 x, 2 x + 1: the warp's x-th unit
      const int id = jp < npg ? __ldg(btab + pg0 + jp) : -1;
      if (id >= 0 && id < p.num_pages) {
        const int64_t r0 = ((int64_t)id * p.num_kv_heads + h) * kPage;
        l2_prefetch((is_v ? p.v_codes : p.k_codes) + r0 * Lo::kRow, kPage * Lo::kRow);
        l2_prefetch((is_v ? p.v_scales : p.k_scales) + r0 * T::kScaleRow, kPage * T::kScaleRow);
      }
    }
    int my_id = id_of(u);
    if constexpr (FMT == KVQ_FMT_BF16) {
      for (; u < units; u += warps) {
        const int i = u >> 1, half = u & 1, stage = i % stages;
        const Unit n = unit_of(u, my_id);
        my_id = id_of(u + warps);
        const uint32_t tile = sbase + (is_v ? Lo::kVAt : Lo::kKAt) + stage * Lo::kKBytes + half * 4 * Lo::kGroupBytes;
        if (!wait_stage(i)) break;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int ok = __shfl_sync(0xffffffffu, n.ok, j);
          const uint8_t* src = codes + (int64_t)(__shfl_sync(0xffffffffu, n.row, j) + rsub) * Lo::kRow;
#pragma unroll
          for (int c = 0; c < Lo::kPer; ++c) {
            const int ps = c / Lo::kSets, set = c % Lo::kSets;
            cp_async16(tile + place(j, ps, set, 0), src + ps * Lo::kRpp * Lo::kRow + set * 128,
                       ps * Lo::kRpp + rsub < ok);
          }
        }
        cp_async_wait_all();
        if (!is_v && lane == 0) bad_pages[2 * (i & (Lo::kScRing - 1)) + half] = n.bad;
        fence_proxy_async_smem();  // the half's bytes become visible to the tensor cores
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[is_v ? kBarP0 + i % Lo::kSBufs : kBarK0 + stage]);
      }
    } else {
      static_assert(FMT != KVQ_FMT_NVFP4 || Lo::kSets == 1, "NVFP4 rows are at most 128 bytes");
      // The next unit's first page is loaded once this unit's is converted, its second
      // page (and scales) behind the proxy fence, which waits for loads in flight: a
      // load has the conversion of the other page, and the wait for the stage, to land.
      uint4 raw[2][Lo::kPer];
      uint32_t gs[2][FMT == KVQ_FMT_NVFP4 ? Lo::kPer : 1];
      float ksv = 0.f, vsv = 0.f;                    // INT8, K: key `lane` of the half
      float sc[kFoldV ? 2 * Lo::kPasses : 1] = {};   // INT8, V folded: this lane's rows
      auto load = [&](int j, const Unit& n) {
        const int64_t ro = (int64_t)__shfl_sync(0xffffffffu, n.row, j) + rsub;
        const uint8_t* src = codes + ro * Lo::kRow;
#pragma unroll
        for (int c = 0; c < Lo::kPer; ++c)
          raw[j][c] = __ldg(reinterpret_cast<const uint4*>(src + (c / Lo::kSets) * Lo::kRpp * Lo::kRow +
                                                           (c % Lo::kSets) * 128));
        if constexpr (FMT == KVQ_FMT_NVFP4) {  // a chunk's two group scales; 0 where they may be NaN
          const int ok = __shfl_sync(0xffffffffu, n.ok, j);
          const uint8_t* gsrc = (is_v ? p.v_scales : p.k_scales) + ro * (D / 16) + u0 * 2;
#pragma unroll
          for (int c = 0; c < Lo::kPer; ++c)
            gs[j][c] = c * Lo::kRpp + rsub < ok
                           ? __ldg(reinterpret_cast<const uint16_t*>(gsrc + c * Lo::kRpp * (D / 16)))
                           : 0u;
        }
      };
      auto load_scales = [&](const Unit& n) {
        if constexpr (FMT == KVQ_FMT_INT8) {
          if (!is_v) {
            const int r = lane & 15;
            const int64_t ro = (int64_t)__shfl_sync(0xffffffffu, n.row, lane >> 4) + r;
            const bool in = r < __shfl_sync(0xffffffffu, n.ok, lane >> 4);
            ksv = in ? __ldg(reinterpret_cast<const float*>(p.k_scales) + ro) : 0.f;
            vsv = in ? __ldg(reinterpret_cast<const float*>(p.v_scales) + ro) : 0.f;
          } else if constexpr (kFoldV) {
#pragma unroll
            for (int x = 0; x < 2 * Lo::kPasses; ++x) {
              const int j = x / Lo::kPasses, r = (x % Lo::kPasses) * Lo::kRpp + rsub;
              const int64_t ro = (int64_t)__shfl_sync(0xffffffffu, n.row, j) + r;
              sc[x] = r < __shfl_sync(0xffffffffu, n.ok, j)
                          ? __ldg(reinterpret_cast<const float*>(p.v_scales) + ro)
                          : 0.f;
            }
          }
        }
      };
      Unit cur = unit_of(u, u < units ? my_id : -1);
      my_id = id_of(u + warps);
      if (u < units) {
        load(0, cur);
        load(1, cur);
        load_scales(cur);
      }
      for (; u < units; u += warps) {
        const int i = u >> 1, half = u & 1, stage = i % stages;
        const uint32_t tile = sbase + (is_v ? Lo::kVAt : Lo::kKAt) + stage * Lo::kKBytes + half * 4 * Lo::kGroupBytes;
        const bool more = u + warps < units;
        const Unit next = unit_of(u + warps, my_id);
        my_id = id_of(u + 2 * warps);
        if (!wait_stage(i)) break;
        // V folded: the half's largest scale fixes the tile's unit 2^e, as published with
        // K(i) (from the same 32 scales); one factor a row of this lane
        [[maybe_unused]] uint32_t vfac[kFoldV ? 2 * Lo::kPasses : 1];
        if constexpr (kFoldV) {
          if (is_v) {
            float vm = 0.f;
#pragma unroll
            for (int x = 0; x < 2 * Lo::kPasses; ++x) vm = fmaxf(vm, fabsf(sc[x]));
            const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(vm));
            const int ex = m ? static_cast<int>(m >> 23) - 126 : 0;
            const float dn = pow2f(max(-126, min(126, -ex)));
#pragma unroll
            for (int x = 0; x < 2 * Lo::kPasses; ++x) vfac[x] = h2_as_u32(__float2half2_rn(sc[x] * dn));
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int c = 0; c < Lo::kPer; ++c)
            convert_chunk<FMT>(raw[j][c], gs[j][FMT == KVQ_FMT_NVFP4 ? c : 0], 0, [&](int el, uint4 v) {
              if constexpr (kFoldV) {
                if (is_v) {
                  const __half2 f = u32_as_h2(vfac[j * Lo::kPasses + c / Lo::kSets]);
                  v.x = h2_as_u32(__hmul2(u32_as_h2(v.x), f));
                  v.y = h2_as_u32(__hmul2(u32_as_h2(v.y), f));
                  v.z = h2_as_u32(__hmul2(u32_as_h2(v.z), f));
                  v.w = h2_as_u32(__hmul2(u32_as_h2(v.w), f));
                }
              }
              st_shared16(tile + place(j, c / Lo::kSets, c % Lo::kSets, el / 8), v);
            });
          if (j == 0 && more) load(0, next);
        }
        if (!is_v) {  // published with K(i): the softmax reads them once S(i) is done
          const int sl = i & (Lo::kScRing - 1);
          if constexpr (FMT == KVQ_FMT_INT8) {
            ksc[sl * kPxKeys + 32 * half + lane] = ksv * p.sm_scale_log2;  // the softmax's log2 factor folded in
            // 2^e above the half's V scales (kNoScale: all zero), which the softmax gets as scale x 2^-e
            const uint32_t vm = __reduce_max_sync(0xffffffffu, __float_as_uint(vsv) & 0x7FFFFFFFu);
            const int ex = vm ? static_cast<int>(vm >> 23) - 126 : kNoScale;
            if constexpr (!kFoldV) vsc[sl * kPxKeys + 32 * half + lane] = vsv * pow2f(max(-126, min(126, -ex)));
            if (lane == 0) vexp[2 * sl + half] = ex;
          }
          if (lane == 0) bad_pages[2 * sl + half] = cur.bad;
        }
        fence_proxy_async_smem();  // the half's bytes become visible to the tensor cores
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[is_v ? kBarP0 + i % Lo::kSBufs : kBarK0 + stage]);
        cur = next;
        if (more) {
          load(1, next);
          load_scales(next);
        }
      }
    }
  } else {
    // ================================================================== softmax
    const int grp = warp >> 2, w4 = warp & 3;
    const uint32_t tq = tmem + ((uint32_t)(32 * w4) << 16);  // this warp's TMEM lanes
    // ---- q -> TMEM.  Warp w copies rows 16 w .. 16 w + 15 of the block (whole rows,
    // coalesced) to shared memory; then a thread has half a row: its part of the row's
    // maximum, and (INT8 / NVFP4) q x 2^k, k such that the largest |q| of the row lies
    // in [2^14, 2^15), which makes q exact in fp16.  Column c of TMEM holds elements 2c
    // (low half) and 2c + 1.
    {
      constexpr int kLq = D / 8, kRq = 32 / kLq;  // lanes of a row, rows a copy
      const int sub = lane / kLq, c = lane % kLq;
#pragma unroll
      for (int j = 0; j < 16 / kRq; ++j) {
        const int r = warp * 16 + j * kRq + sub;
        const int at = qoff[r];
        cp_async16(sbase + Lo::kQAt + r * Lo::kQRow + 16 * c,
                   reinterpret_cast<const uint8_t*>(p.q) + (size_t)max(at, 0) * (2 * D) + 16 * c, at >= 0);
      }
      cp_async_wait_all();
    }
    soft_sync();
    const uint8_t* qr = smem + Lo::kQAt + rl * Lo::kQRow + grp * D;  // half a row: D / 2 elements
    float up = 1.f;
    if constexpr (!kBf16) {
      uint32_t a2 = 0;  // largest |q| of the half row's even and odd elements, as bits (ordered like the values)
#pragma unroll 4
      for (int c = 0; c < D / 16; ++c) {
        const uint4 v = *reinterpret_cast<const uint4*>(qr + 16 * c);
        a2 = __vmaxu2(a2, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                   __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
      }
      uint32_t a = max(a2 << 16, a2 & 0xFFFF0000u);
      uint32_t* half_max = reinterpret_cast<uint32_t*>(l_sh);
      half_max[grp * kPxRows + rl] = a;
      soft_sync();
      a = max(half_max[rl], half_max[kPxRows + rl]);
      // |q| < 2^(e - 126) with e the exponent field (0 for a zero row: any power will do)
      up = pow2f(min(126, max(-126, 15 + 126 - static_cast<int>(a >> 23))));
    }
    // logit (log2 units) = S x kfac x rs with rs = 1 / up: INT8 kfac = the key's scale
    // x sm_scale x log2(e) (folded in by the converters), otherwise kfac = sm_scale x
    // log2(e) (NVFP4: x 1 / gs_K, the tiles hold values x gs).  kfac carries the sign
    // of sm_scale and rs > 0, so max(S x kfac) x rs is the maximum logit.
    const float rs = 1.f / up;  // a power of two: exact
    {
#pragma unroll 2
      for (int c16 = 0; c16 < D / 32; ++c16) {  // 16 elements: 8 columns
        uint32_t cols[8];
#pragma unroll
        for (int h8 = 0; h8 < 2; ++h8) {
          const uint4 v = *reinterpret_cast<const uint4*>(qr + 32 * c16 + 16 * h8);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int x = 0; x < 4; ++x)
            cols[4 * h8 + x] = kBf16 ? w[x]
                                     : h2_as_u32(__floats2half2_rn(__uint_as_float(w[x] << 16) * up,
                                                                   __uint_as_float(w[x] & 0xFFFF0000u) * up));
        }
        if (D == 256 && grp == 1) {  // the second half: shared memory
          const uint32_t qs = sbase + Lo::kQSmemAt;
          st_shared16(qs + kmajor_off(rl, 16 * c16, kPxRows), make_uint4(cols[0], cols[1], cols[2], cols[3]));
          st_shared16(qs + kmajor_off(rl, 16 * c16 + 8, kPxRows), make_uint4(cols[4], cols[5], cols[6], cols[7]));
        } else {
          tmem_st8(tq + Lo::kTmemQ + grp * (D / 4) + 8 * c16, cols);
        }
      }
      fence_proxy_async_smem();
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kBarQ]);
    }
    const int kend = min(lims[rl], key_end);
    const float kconst = p.sm_scale_log2 * p.k_gs_inv;  // kfac of the non-INT8 formats
    [[maybe_unused]] const uint64_t kconst2 = pair(kconst, kconst);
    // The row's reference is m, its running maximum (a stale one: raised only by more
    // than 2^8, so that O is seldom rescaled): l = sum of 2^(z - m).  O (INT8) has a unit
    // of its own besides, 2^E, E the exponent of the tiles' V scales (raised by more than
    // 2^4), so that P' = 2^(z - m) x v_scale x 2^-E <= 2^12 fits fp16 whatever the size of
    // V; the epilogue gives 2^E back.  Keys whose P' is below 2^-14 are off by up to 2^-25,
    // that is 2^-24 of the range's largest |V| a key of weight 1.  INT8 rounds m up to a whole
    // number: the differences of m and E, and the rescaling of O and l, are then exact.
    float m_ref = -INFINITY, l_run = 0.f;  // l_run = this group's sum of 2^(z - m_ref)
    [[maybe_unused]] int e_run = kNoScale;
    auto raise_scale = [&](int sl) {
      const int e = max(vexp[2 * sl], vexp[2 * sl + 1]);
      if (e != kNoScale && (e_run == kNoScale || e > e_run + kPxScaleRise)) e_run = e;
    };

    bool ok = true;
    for (int i = grp; i < nt; i += 2) {
      const int sb = i % Lo::kSBufs;
      if (!wait_warp(kBarS0 + sb, (i / Lo::kSBufs) & 1)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t ts = tq + Lo::kTmemS + (uint32_t)sb * kPxKeys;
      uint32_t sv[64];
      tmem_ld64(ts, sv);
      const int sl = i & (Lo::kScRing - 1);
      const float* ks = ksc + sl * kPxKeys;
      const float* vs = vsc + sl * kPxKeys;
      const int nvis = kend - (pg0 + i * kPxPages) * kPage;  // visible keys of this tile for this row
      const uint32_t bad = bad_pages[2 * sl] | bad_pages[2 * sl + 1] << 2;
      [[maybe_unused]] int e_old = 0;
      if constexpr (FMT == KVQ_FMT_INT8) {  // the tiles in order: the other group's, then this one
        if (i > 0) raise_scale((i - 1) & (Lo::kScRing - 1));
        e_old = e_run;
        raise_scale(sl);
      }
      tmem_ld_wait();
      // pass 1: z = S x kfac (the logit before the row factor rs > 0), two keys an
      // operation, and the tile maximum (four independent chains)
      uint64_t z[kPxKeys / 2];
      float mxs[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c4 = 0; c4 < kPxKeys / 4; ++c4) {
        uint64_t ka = kconst2, kb = kconst2;
        if constexpr (FMT == KVQ_FMT_INT8) {
          const float4 k4 = *reinterpret_cast<const float4*>(ks + 4 * c4);
          ka = pair(k4.x, k4.y);
          kb = pair(k4.z, k4.w);
        }
        z[2 * c4] = mul2(pair(sv[4 * c4], sv[4 * c4 + 1]), ka);
        z[2 * c4 + 1] = mul2(pair(sv[4 * c4 + 2], sv[4 * c4 + 3]), kb);
        const float2 za = unpair(z[2 * c4]), zb = unpair(z[2 * c4 + 1]);
        mxs[2 * (c4 & 1)] = fmaxf(mxs[2 * (c4 & 1)], fmaxf(za.x, za.y));
        mxs[2 * (c4 & 1) + 1] = fmaxf(mxs[2 * (c4 & 1) + 1], fmaxf(zb.x, zb.y));
      }
      if (__any_sync(0xffffffffu, nvis < kPxKeys || bad != 0)) {
        // A tile that ends inside for a row, or holds pages that were not read: those
        // keys out, and the maximum again.  At most a tile or two of a range come here,
        // so it is a short loop through TMEM (z over S), not another unrolled pass.
        mxs[0] = mxs[1] = mxs[2] = mxs[3] = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < kPxKeys / 8; ++c) {
          uint32_t v[8];
          tmem_ld8(ts + 8 * c, v);
          tmem_ld_wait();
          const bool off = (bad >> (c >> 1)) & 1u;
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const float f = FMT == KVQ_FMT_INT8 ? ks[8 * c + x] : kconst;
            const float zz = !off && 8 * c + x < nvis ? __uint_as_float(v[x]) * f : -INFINITY;
            mxs[x & 3] = fmaxf(mxs[x & 3], zz);
            v[x] = __float_as_uint(zz);
          }
          tmem_st8(ts + 8 * c, v);
        }
        tmem_st_wait();
        tmem_ld64(ts, sv);
        tmem_ld_wait();
#pragma unroll
        for (int t2 = 0; t2 < kPxKeys / 2; ++t2) z[t2] = pair(sv[2 * t2], sv[2 * t2 + 1]);
      }
      float mx = fmaxf(fmaxf(mxs[0], mxs[1]), fmaxf(mxs[2], mxs[3])) * rs;  // log2 units
      if constexpr (FMT == KVQ_FMT_INT8) mx = ceilf(mx);
      // the row's reference after tile i - 1, from the other group; this tile's goes on
      float m_prev = -INFINITY;
      if (i > 0) {
        if (!wait_warp(kBarM0 + 4 * ((i - 1) & 1) + w4, ((i - 1) >> 1) & 1)) {
          ok = false;
          break;
        }
        m_prev = m_sh[((i - 1) & 1) * kPxRows + rl];
      }
      // how far O's unit rises (from no unit at all: O is 0)
      const int e_up = FMT == KVQ_FMT_INT8 && e_old != kNoScale ? e_run - e_old : 0;
      const float m = m_prev == -INFINITY || mx > m_prev + kPxRescale ? mx : m_prev;
      m_sh[(i & 1) * kPxRows + rl] = m;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kBarM0 + 4 * (i & 1) + w4]);
      const bool resc = m_prev != -INFINITY && (m != m_prev || e_up != 0);
      if (__any_sync(0xffffffffu, resc)) {
        // O is rescaled once it holds P(i-1) V(i-1), before P(i) V(i) adds to it
        if (!wait_warp(kBarO0 + ((i - 1) & 3), ((i - 1) >> 2) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float alpha = resc ? ex2(m_prev - m - static_cast<float>(e_up)) : 1.f;
#pragma unroll 1
        for (int c = 0; c < D / 8; ++c) {
          uint32_t ov[8];
          tmem_ld8(tq + Lo::kTmemO + 8 * c, ov);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 8; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
          tmem_st8(tq + Lo::kTmemO + 8 * c, ov);
        }
        tmem_st_wait();
      }
      if (m != m_ref) {  // raised here or by the other group since this group's last tile
        l_run *= ex2(m_ref - m);  // m_ref = -inf: 0
        m_ref = m;
      }
      // P(i) goes over S(i), which this thread has read.  The last reader of those
      // columns before S(i), the P V product of the buffer's previous tile, was issued
      // before S(i), so the commit that reported S(i) done covered it too.
      // pass 2: p = 2^(z - m + d), d = (the half's exponent) - E (a masked key's z = -inf
      // gives exactly 0), packed hi (+ lo).  The V scales that the half's tile or vs holds
      // carry 2^-(its exponent), so p x v is P' x code in O's unit; the half's sum takes
      // 2^-d.  A half far below the others keeps its place in the sum (d >= -60), whatever
      // is left of it in fp16; one of zeros may take any d.
      uint64_t ps[2] = {0, 0};
      const float nm = m == -INFINITY ? 0.f : -m;  // a row with no visible key: every z is -inf
      const uint64_t rs2 = pair(rs, rs);
      uint64_t nr2 = pair(nm, nm);
      [[maybe_unused]] int dh[2] = {0, 0};
      if constexpr (FMT == KVQ_FMT_INT8) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int e = vexp[2 * sl + x];
          dh[x] = e == kNoScale ? 0 : max(-60, e - e_run);
        }
      }
#pragma unroll
      for (int c16 = 0; c16 < kPxKeys / 16; ++c16) {  // 16 keys: 8 columns
        uint32_t ph[8], pl[8];
        [[maybe_unused]] float4 v4;  // V scales of four keys
        if constexpr (FMT == KVQ_FMT_INT8) {
          if ((c16 & 1) == 0) {
            const float nd = nm + static_cast<float>(dh[c16 >> 1]);
            nr2 = pair(nd, nd);
          }
        }
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int t2 = 8 * c16 + x;
          if constexpr (FMT == KVQ_FMT_INT8 && !kFoldV)
            if ((x & 1) == 0) v4 = *reinterpret_cast<const float4*>(vs + 2 * t2);
          const float2 a = unpair(fma2(z[t2], rs2, nr2));
          const float2 pr = make_float2(ex2(a.x), ex2(a.y));
          uint64_t pv = pair(pr.x, pr.y);
          constexpr bool kHalves = FMT == KVQ_FMT_INT8;
          ps[kHalves ? c16 >> 1 : x & 1] = add2(ps[kHalves ? c16 >> 1 : x & 1], pv);
          if constexpr (FMT == KVQ_FMT_INT8 && !kFoldV)  // finite scales, 0 for a key that was not read
            pv = mul2(pv, (x & 1) ? pair(v4.z, v4.w) : pair(v4.x, v4.y));
          const float2 v = unpair(pv);
          if constexpr (!PLO) {
            ph[x] = h2_as_u32(__floats2half2_rn(v.x, v.y));
          } else {
            // hi + lo, lo = what hi leaves of p', rounded: fp16 hi cut off to 11 bits (22 kept
            // in all), bf16 hi rounded to 8 (the rest is then half as large, and both
            // roundings leave 2^-18 of p')
            float2 hi;
            if constexpr (kBf16) {
              const __nv_bfloat162 hv = __floats2bfloat162_rn(v.x, v.y);
              ph[x] = *reinterpret_cast<const uint32_t*>(&hv);
              hi = make_float2(__uint_as_float(ph[x] << 16), __uint_as_float(ph[x] & 0xFFFF0000u));
            } else {
              hi = make_float2(__uint_as_float(__float_as_uint(v.x) & 0xFFFFE000u),
                               __uint_as_float(__float_as_uint(v.y) & 0xFFFFE000u));
              ph[x] = h2_as_u32(__floats2half2_rn(hi.x, hi.y));
            }
            const float2 lo = unpair(sub2(pv, pair(hi.x, hi.y)));
            if constexpr (kBf16) {
              const __nv_bfloat162 lv = __floats2bfloat162_rn(lo.x, lo.y);
              pl[x] = *reinterpret_cast<const uint32_t*>(&lv);
            } else {
              pl[x] = h2_as_u32(__floats2half2_rn(lo.x, lo.y));
            }
          }
        }
        // 16 columns of S become 8 of hi pairs and 8 of lo pairs
        tmem_st8(ts + 16 * c16, ph);
        if constexpr (PLO) tmem_st8(ts + 16 * c16 + 8, pl);
      }
      if constexpr (FMT == KVQ_FMT_INT8) {
        const float2 s0 = unpair(ps[0]), s1 = unpair(ps[1]);
        l_run += (s0.x + s0.y) * pow2f(-dh[0]) + (s1.x + s1.y) * pow2f(-dh[1]);
      } else {
        const float2 sum = unpair(add2(ps[0], ps[1]));
        l_run += sum.x + sum.y;
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kBarP0 + sb]);
    }
    // ================================================================ epilogue
    // the last tile's reference is the row's; both groups bring their sums to it
    float m_fin = m_ref;
    if (ok && nt > 0) {
      ok = wait_warp(kBarM0 + 4 * ((nt - 1) & 1) + w4, ((nt - 1) >> 1) & 1) &&
           wait_warp(kBarO0 + ((nt - 1) & 3), ((nt - 1) >> 2) & 1);
      tc_fence_after();
      m_fin = m_sh[((nt - 1) & 1) * kPxRows + rl];
      if (m_fin != m_ref) l_run *= ex2(m_ref - m_fin);
      if constexpr (FMT == KVQ_FMT_INT8)  // O's unit after the last tile
        if (((nt - 1) & 1) != grp) raise_scale((nt - 1) & (Lo::kScRing - 1));
    }
    l_sh[grp * kPxRows + rl] = l_run;
    soft_sync();
    ok = ok && *abort_flag == 0;  // a group that gave up leaves the row without a result
    const float l = l_sh[rl] + l_sh[kPxRows + rl];
    constexpr float kLn2 = 0.69314718055994530942f;
    // l = 0: no visible token (or only logits of -inf).  A NaN logit among the visible
    // ones makes l, and so the row's partial, NaN
    const bool any = ok && nt > 0 && l != 0.f;
    const float inv_l = any ? p.v_gs_inv / l : 0.f;
    float inv = inv_l, unit = 1.f;
    if constexpr (FMT == KVQ_FMT_INT8) {  // 2^E in two factors: E reaches beyond one's exponents
      const int e = e_run == kNoScale ? 0 : e_run;
      inv *= pow2f(e / 2);
      unit = pow2f(e - e / 2);
    }
    if (grp == 0 && qoff[rl] >= 0) p.lse_part[orow_at[rl]] = any ? (m_fin + log2f(l)) * kLn2 : -INFINITY;
    // rows that end inside the range: a key behind their last one has weight 0, but 0 x NaN is
    // NaN, so their O is looked at (odd stays 0 while all of it is finite).  A row whose l is
    // NaN is NaN anyway
    const bool ends = any && l == l && kend < key_end && qoff[rl] >= 0;
    const bool look = __any_sync(0xffffffffu, ends);
    float odd = 0.f;
    // Each warp writes its 32 rows' half of the columns, 32 columns at a time, through a
    // patch of shared memory of its own: 128 contiguous bytes of four rows a store.
    uint8_t* patch = smem + Lo::kOAt + warp * Lo::kOPatch;
    const int sub = lane >> 3, c4 = lane & 7;  // row of four, 16 bytes of the 128
    int at[8];  // partial row of patch row 4 x + sub (-1: no live row)
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int r = 32 * w4 + 4 * x + sub;
      at[x] = qoff[r] >= 0 ? orow_at[r] : -1;
    }
#pragma unroll 1
    for (int c = 0; c < D / 64; ++c) {
      const int col = grp * (D / 2) + 32 * c;
      uint32_t ov[32];
      if (ok && nt > 0) {  // the same for the warp's lanes
        tmem_ld32(tq + Lo::kTmemO + col, ov);
        tmem_ld_wait();
      }
      __syncwarp();  // the patch has been read
      if (look) {
#pragma unroll
        for (int e = 0; e < 32; ++e) odd = fmaf(__uint_as_float(ov[e]), 0.f, odd);
      }
#pragma unroll
      for (int v4 = 0; v4 < 8; ++v4) {
        float4 o;
        o.x = any ? __uint_as_float(ov[4 * v4]) * inv * unit : 0.f;
        o.y = any ? __uint_as_float(ov[4 * v4 + 1]) * inv * unit : 0.f;
        o.z = any ? __uint_as_float(ov[4 * v4 + 2]) * inv * unit : 0.f;
        o.w = any ? __uint_as_float(ov[4 * v4 + 3]) * inv * unit : 0.f;
        *reinterpret_cast<float4*>(patch + lane * Lo::kORow + 16 * v4) = o;
      }
      __syncwarp();
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const float4 o = *reinterpret_cast<const float4*>(patch + (4 * x + sub) * Lo::kORow + 16 * c4);
        if (at[x] >= 0) *reinterpret_cast<float4*>(p.o_part + (size_t)at[x] * D + col + 4 * c4) = o;
      }
    }
    __syncwarp();  // a row that is made again is written after this
    for (unsigned redo = __ballot_sync(0xffffffffu, ends && odd != 0.f); redo; redo &= redo - 1) {
      const int src = __ffs(redo) - 1, r = 32 * w4 + src;
      redo_row<FMT, D>(reinterpret_cast<const uint16_t*>(p.q) + (size_t)qoff[r] * D, p.k_codes, p.k_scales, p.v_codes,
                       p.v_scales, btab, p.num_pages, p.num_kv_heads, h, pg0, __shfl_sync(0xffffffffu, kend, src),
                       grp * (D / 2), p.sm_scale_log2 * p.k_gs_inv, __shfl_sync(0xffffffffu, m_fin, src),
                       __shfl_sync(0xffffffffu, inv_l, src), p.o_part + (size_t)orow_at[r] * D);
    }
  }
  // all TMEM reads and MMAs are complete: free the columns
  tc_fence_before();
  __syncthreads();
  if (warp == kPxMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, Lo::kTmemCols);
  }
}

// P as hi + lo terms: with fp32 output, and on a BF16 cache always (one bf16 term is off by up
// to 2^-8 a weight, as much as bf16 output by its own rounding: rms 2.3e-3 in all against 1.7e-3;
// the lo terms here and on the own pages cost 1.3 of 38.6 us with 45 sequences in three groups
// on up to 4,096 tokens)
template <int FMT>
constexpr bool two_terms(bool out_f32) {
  return out_f32 || FMT == KVQ_FMT_BF16;
}

template <int FMT, int D>
cudaError_t launch_px_t(const PrefixParams& p, int blocks, cudaStream_t stream) {
  using Lo = PxLayout<FMT, D>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.splits, p.num_kv_heads, blocks);
  cfg.blockDim = dim3(kPxThreads);
  cfg.dynamicSmemBytes = Lo::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.out_bf16 ? cudaLaunchKernelEx(&cfg, prefix_tc_kernel<FMT, D, two_terms<FMT>(false)>, p)
                    : cudaLaunchKernelEx(&cfg, prefix_tc_kernel<FMT, D, true>, p);
}

template <int FMT, int D>
PrefixInstance px_instance_of() {
  using Lo = PxLayout<FMT, D>;
  return PrefixInstance{{reinterpret_cast<const void*>(&prefix_tc_kernel<FMT, D, true>),
                         reinterpret_cast<const void*>(&prefix_tc_kernel<FMT, D, two_terms<FMT>(false)>)},
                        Lo::kSmemBytes,
                        kPxThreads,
                        kPxRows};
}

}  // namespace

bool prefix_tc_instance(int format, int head_dim, PrefixInstance* out) {
  if (format == KVQ_FMT_NVFP4 && head_dim == 256) *out = px_instance_of<KVQ_FMT_NVFP4, 256>();
  else if (format == KVQ_FMT_NVFP4 && head_dim == 128) *out = px_instance_of<KVQ_FMT_NVFP4, 128>();
  else if (format == KVQ_FMT_INT8 && head_dim == 256) *out = px_instance_of<KVQ_FMT_INT8, 256>();
  else if (format == KVQ_FMT_INT8 && head_dim == 128) *out = px_instance_of<KVQ_FMT_INT8, 128>();
  else if (format == KVQ_FMT_BF16 && head_dim == 256) *out = px_instance_of<KVQ_FMT_BF16, 256>();
  else if (format == KVQ_FMT_BF16 && head_dim == 128) *out = px_instance_of<KVQ_FMT_BF16, 128>();
  else return false;
  return true;
}

cudaError_t launch_prefix_tc(int format, int head_dim, const PrefixParams& p, int blocks, cudaStream_t stream) {
  if (format == KVQ_FMT_NVFP4 && head_dim == 256) return launch_px_t<KVQ_FMT_NVFP4, 256>(p, blocks, stream);
  if (format == KVQ_FMT_NVFP4 && head_dim == 128) return launch_px_t<KVQ_FMT_NVFP4, 128>(p, blocks, stream);
  if (format == KVQ_FMT_INT8 && head_dim == 256) return launch_px_t<KVQ_FMT_INT8, 256>(p, blocks, stream);
  if (format == KVQ_FMT_INT8 && head_dim == 128) return launch_px_t<KVQ_FMT_INT8, 128>(p, blocks, stream);
  if (format == KVQ_FMT_BF16 && head_dim == 256) return launch_px_t<KVQ_FMT_BF16, 256>(p, blocks, stream);
  if (format == KVQ_FMT_BF16 && head_dim == 128) return launch_px_t<KVQ_FMT_BF16, 128>(p, blocks, stream);
  return cudaErrorInvalidValue;
}

}  // namespace kvq
