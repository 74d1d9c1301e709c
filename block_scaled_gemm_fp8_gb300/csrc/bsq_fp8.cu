// bsq_fp8.cu -- products of E4M3 operands on their own codes (tcgen05 kind::f8f6f4), with the
// scales applied to every 128-deep partial sum:
//
//   forward  y[m, n]  = sum_b xs[m, b] ws[n/128, b] sum_{k in b} xc[m, k] wc[n, k]
//   dgrad    gx[m, k] = sum_b gs[m, b] ws[b, k/128] sum_{n in b} gc[m, n] wc[n, k]
//
// The first operand has one float32 scale per row and 128 columns, W one per 128 x 128
// block, so within one contraction block b an output element's scale is one number: the
// tensor cores sum the codes' products of a block, and the promotion warps add the partial
// sum times xs * ws to an FP32 accumulator in registers.  The product is rounded to BF16
// once, at the end.  Grouped calls take the token rows of expert e against W[e]; an
// expert's rows need no alignment, its last tile's foreign rows are computed and dropped.
//
// W is stored [N][K].  The forward contracts over its contiguous axis (a K-major B
// operand), dgrad over its rows (MN-major): one kernel, two descriptors, no transpose.
//
// Tile: 128 rows by BN output columns, one CTA per SM, 12 warps:
//   warps 0-7   promotion and epilogue: TMEM lanes 32 (w % 4).., output columns half w / 4
//   warp 8      TMA producer: 128 x 128 bytes of the first operand, BN x 128 of W's
//   warp 9      MMA issuer
//   warps 10-11 scales: xs * ws of each k-block's rows and column halves, into shared memory
// A 128-deep block of BN = 256 takes 512 tensor-core cycles per SM; its promotion is 64 packed
// FMAs and 4 TMEM loads per thread, 256 cycles of each SM quarter's FMA pipe.  Measured, M =
// 8192, N = 14336, K = 5120: 480 us as calls on inputs beyond L2, 2.5 PFLOP/s (1.32 of the
// measured BF16 burst rate); on the same operands 436 over 20 calls back to back, 468 over 400.
// Over 1 to 16 tiles a CTA and 4 to 64 k-blocks a call takes about 10 us + 1.0 a tile + 0.45 a
// k-block (within 6 %): the k-block is what counts, and the MMAs alone would take 0.35.
// With parts left out, 20 calls back to back take 399 us without output, 385 without the
// promotion's loads and FMAs, 385 without TMA loads, 334 with the MMAs alone and 334 with the
// promotion alone (438 with all of them).  MMAs and promotion share the SM: the operands alone
// are 48 KB of writes and as many reads of its shared memory a k-block.  Which of the shared
// parts holds the other up is not settled; loading W's tile once for two CTAs (multicast)
// changed nothing (437 us), so L2 does not bound it.
// Tried and slower, back to back: CTA pairs of 256 x 256, which halve W's part (509 us, 354 without
// promotion: an accumulator's hand-over then crosses SMs; 658 in half accumulators); two
// 128-column accumulators a k-block with an issuer each (501); 16 promotion warps (513); one
// scale load per thread in the promotion loop instead of the scale warps (531); scalar FMAs
// (500); L2 prefetch of operands 6 or 16 k-blocks ahead (456, 458); consecutive tiles to one
// CTA (545).  A fourth ring stage changed nothing.
#include <atomic>
#include <cstdlib>

#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include "bsq_fp8_internal.h"
#include "bsq_internal.h"
#include "bsq_pipe.cuh"
#include "bsq_ptx.cuh"
#include "../../include/bsq.h"

namespace bsq {

bool encode_map(CUtensorMap* m, CUtensorMapDataType dt, uint32_t rank, const void* base, const uint64_t* dims,
                const uint64_t* strides, const uint32_t* box, CUtensorMapSwizzle sw);

namespace {

constexpr int kThreads8 = 384;
constexpr int kLaunchRegs = 168;            // registers per thread at launch (65536 / 384, in eights)
constexpr int kPromoteRegs = 216, kOtherRegs = 72;
static_assert(256 * kPromoteRegs + 128 * kOtherRegs <= kThreads8 * kLaunchRegs, "register split");
constexpr int kRows8 = 128;                 // rows of the first operand per CTA
constexpr int kDepth = 128;                 // contraction per k-block: one scale block, 128 bytes of codes
constexpr int kABytes = kRows8 * kDepth;    // 16 KB
constexpr int kTmemCols8 = 512;
constexpr int kPromoteWarps = 8, kScaleWarps = 2;
constexpr int kBoxBytes8 = 32 * 128;        // output box: 32 rows of 64 columns
// Of the first operand: what stays in L2 beside W and the output (dgrad of 8192 x 14336 x 5120,
// 117 MB of gradient codes: 465 us in groups, 492 in one; groups of 8 or 16 row tiles where
// 42 MB fit: 468 and 452 us against 440).
constexpr int64_t kRasterBytes = 48 << 20;
constexpr int kMaxSplit = 4;                // clusters of 8 do not all fit the SMs at once

constexpr int BN = 256;                     // output columns of a tile
struct Fp8Cfg {
  static constexpr int kBBytes = BN * kDepth;
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kStages = 3;
  static constexpr int kBufs = kTmemCols8 / BN;         // accumulators in TMEM
  static constexpr int kCols = BN / 2;                  // output columns of one promotion warp
  static constexpr int kRing = kStages * kStage;
  static constexpr int kOutWarp = kCols / 64 * kBoxBytes8;   // output staging of one promotion warp
  static constexpr int kOutBytes = kPromoteWarps * kOutWarp;
};

struct Fp8Params {
  const float* xs;             // [S][xs_ld] scales of the first operand
  const float* ws;             // W's scales; element (e, output block, contraction block) at
  int64_t ws_e;                //   e * ws_e + ob * ws_o + cb * ws_c
  int32_t ws_o, ws_c, xs_ld;
  __nv_bfloat16* y;            // [S][O]
  const int32_t* offsets;      // device cumulative ends [E], or null: one group of S rows
  int32_t* err;
  int32_t S, O, E;
  int32_t kblocks, num_nt;
  int32_t raster;              // row tiles of a group
  int32_t split;               // CTAs of a cluster that share a tile's contraction; 1: none
  uint64_t timeout_ns;
  int32_t drop_announce;       // test hook: 1, the producer never requests a stage's operands; 2, not a CTA's last ones
};

struct Fp8Shared {
  uint64_t full[Fp8Cfg::kStages];
  uint64_t empty[Fp8Cfg::kStages];
  uint64_t tmem_full[Fp8Cfg::kBufs];    // the accumulator is complete and its scales are stored
  uint64_t tmem_empty[Fp8Cfg::kBufs];
  uint64_t drain;
  float scale[Fp8Cfg::kBufs][2][kRows8];   // of an accumulator: column half, row
  uint32_t tmem_base;
  uint32_t abort_flag;
  int32_t total_mt;                 // row tiles of all experts; none when the offsets are bad
  int32_t mt_start[kMaxExperts + 1];   // row tiles before expert e
};

// kind::f8f6f4, E4M3 x E4M3 -> F32.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(uint32_t M, uint32_t N, bool b_mn_major) {
  return (1u << 4)                              // D format: F32; A and B formats 0: E4M3
         | ((b_mn_major ? 1u : 0u) << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// Whole-warp roles leave their loops together: a lane that left alone would leave the others at
// an instruction that wants all 32.  No lane branches on how a wait ended.  Promotion and scale
// lanes remember a failure, wait no more and go on with the others, and the warp votes once a
// tile; the MMA warp votes behind each k-block's MMAs, between its two announcements (8192 x
// 14336 x 5120: 487 us, as without agreement; a vote before the first announcement 489, behind
// the second 492, right after every wait 500).
__device__ __forceinline__ bool all_lanes(bool ok) { return __all_sync(0xffffffffu, ok); }

// One lane of a converged warp.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e;
}

// The four MMAs (K = 32 each) of one 128-deep block into a fresh accumulator: A K-major,
// advancing 32 bytes a step; B by BSTEP descriptor units.  Called by a converged warp, issued
// by its elected lane: the operands stay in uniform registers.
template <uint32_t BSTEP>
__device__ __forceinline__ void umma_e4m3_k128(uint32_t elected, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                    uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred e, p, q;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "setp.ne.b32 e, %7, 0;\n\t"
      "setp.ne.b32 p, %3, %3;\n\t"
      "setp.eq.b32 q, %3, %3;\n\t"
      "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
      "add.s64 b1, %2, %4;\n\tadd.s64 b2, %2, %5;\n\tadd.s64 b3, %2, %6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, q;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "n"(BSTEP), "n"(2 * BSTEP), "n"(3 * BSTEP), "r"(elected)
      : "memory");
}
// Arrive on the CTA's barrier when every MMA the elected lane issued so far has completed.
__device__ __forceinline__ void umma_commit(uint32_t elected, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// As tmem_ld_32x32b_x16_wait, 32 columns.
__device__ __forceinline__ void tmem_ld_32x32b_x32_wait(uint32_t taddr, uint32_t (&r)[32]) {
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// Bounded wait; false when the CTA aborted or the limit ran out, which then aborts it.  The
// first polls come without a timer read, and nothing here is a call, around which the
// promotion warps' accumulators would be spilled.
__device__ __forceinline__ bool wait8(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, int32_t* err,
                                      uint64_t limit_ns) {
#pragma unroll 1
  for (int i = 0; i < 32; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 16; ++i)
      if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
    if (*abort_flag) return false;
    if (global_timer_ns() - t0 > limit_ns) {
      *abort_flag = 1u;
      record_error(err, BSQ_DEVERR_TIMEOUT);
      return false;
    }
  }
}
// The promotion warps' wait, in a few instructions.  What they wait for is the MMA warp's and
// the scale warps', whose own waits keep the time: they leave when the CTA has aborted, or
// after a poll count that no run reaches.
__device__ __forceinline__ bool wait8_promote(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag) {
#pragma unroll 1
  for (uint32_t i = 1; i < (1u << 28); ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 1023u) == 0 && *abort_flag) break;
  }
  return false;
}

// acc += p * s on a pair of FP32 values.
__device__ __forceinline__ void fma_f32x2(uint64_t& acc, uint32_t p0, uint32_t p1, uint64_t s2) {
  asm volatile("{\n\t.reg .b64 p;\n\tmov.b64 p, {%1, %2};\n\tfma.rn.f32x2 %0, p, %3, %0;\n\t}"
      : "+l"(acc)
      : "r"(p0), "r"(p1), "l"(s2));
}

// Load the next 32 columns from TMEM and, while they fly, acc += cur * s over the current
// ones.  One statement, ended by the wait, for the reason tmem_ld_32x32b_x16_wait gives.
__device__ __forceinline__ void tmem_ld_x32_fma(uint32_t taddr, uint32_t (&next)[32], uint64_t* acc, const uint32_t (&cur)[32],
                                                uint64_t s2) {
  asm volatile(
      "{\n\t.reg .b64 p;\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%80];\n\t"
      "mov.b64 p, {%48, %49};\n\tfma.rn.f32x2 %32, p, %81, %32;\n\t"
      "mov.b64 p, {%50, %51};\n\tfma.rn.f32x2 %33, p, %81, %33;\n\t"
      "mov.b64 p, {%52, %53};\n\tfma.rn.f32x2 %34, p, %81, %34;\n\t"
      "mov.b64 p, {%54, %55};\n\tfma.rn.f32x2 %35, p, %81, %35;\n\t"
      "mov.b64 p, {%56, %57};\n\tfma.rn.f32x2 %36, p, %81, %36;\n\t"
      "mov.b64 p, {%58, %59};\n\tfma.rn.f32x2 %37, p, %81, %37;\n\t"
      "mov.b64 p, {%60, %61};\n\tfma.rn.f32x2 %38, p, %81, %38;\n\t"
      "mov.b64 p, {%62, %63};\n\tfma.rn.f32x2 %39, p, %81, %39;\n\t"
      "mov.b64 p, {%64, %65};\n\tfma.rn.f32x2 %40, p, %81, %40;\n\t"
      "mov.b64 p, {%66, %67};\n\tfma.rn.f32x2 %41, p, %81, %41;\n\t"
      "mov.b64 p, {%68, %69};\n\tfma.rn.f32x2 %42, p, %81, %42;\n\t"
      "mov.b64 p, {%70, %71};\n\tfma.rn.f32x2 %43, p, %81, %43;\n\t"
      "mov.b64 p, {%72, %73};\n\tfma.rn.f32x2 %44, p, %81, %44;\n\t"
      "mov.b64 p, {%74, %75};\n\tfma.rn.f32x2 %45, p, %81, %45;\n\t"
      "mov.b64 p, {%76, %77};\n\tfma.rn.f32x2 %46, p, %81, %46;\n\t"
      "mov.b64 p, {%78, %79};\n\tfma.rn.f32x2 %47, p, %81, %47;\n\t"
      "tcgen05.wait::ld.sync.aligned;\n\t}"
      : "=&r"(next[0]), "=&r"(next[1]), "=&r"(next[2]), "=&r"(next[3]), "=&r"(next[4]), "=&r"(next[5]), "=&r"(next[6]), "=&r"(next[7]),
        "=&r"(next[8]), "=&r"(next[9]), "=&r"(next[10]), "=&r"(next[11]), "=&r"(next[12]), "=&r"(next[13]), "=&r"(next[14]), "=&r"(next[15]),
        "=&r"(next[16]), "=&r"(next[17]), "=&r"(next[18]), "=&r"(next[19]), "=&r"(next[20]), "=&r"(next[21]), "=&r"(next[22]), "=&r"(next[23]),
        "=&r"(next[24]), "=&r"(next[25]), "=&r"(next[26]), "=&r"(next[27]), "=&r"(next[28]), "=&r"(next[29]), "=&r"(next[30]), "=&r"(next[31]),
        "+l"(acc[0]), "+l"(acc[1]), "+l"(acc[2]), "+l"(acc[3]), "+l"(acc[4]), "+l"(acc[5]), "+l"(acc[6]), "+l"(acc[7]),
        "+l"(acc[8]), "+l"(acc[9]), "+l"(acc[10]), "+l"(acc[11]), "+l"(acc[12]), "+l"(acc[13]), "+l"(acc[14]), "+l"(acc[15])
      : "r"(cur[0]), "r"(cur[1]), "r"(cur[2]), "r"(cur[3]), "r"(cur[4]), "r"(cur[5]), "r"(cur[6]), "r"(cur[7]),
        "r"(cur[8]), "r"(cur[9]), "r"(cur[10]), "r"(cur[11]), "r"(cur[12]), "r"(cur[13]), "r"(cur[14]), "r"(cur[15]),
        "r"(cur[16]), "r"(cur[17]), "r"(cur[18]), "r"(cur[19]), "r"(cur[20]), "r"(cur[21]), "r"(cur[22]), "r"(cur[23]),
        "r"(cur[24]), "r"(cur[25]), "r"(cur[26]), "r"(cur[27]), "r"(cur[28]), "r"(cur[29]), "r"(cur[30]), "r"(cur[31]), "r"(taddr), "l"(s2)
      : "memory");
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map), "r"(src), "r"(x), "r"(y)
               : "memory");
}

// One tile: the expert and its rows, and the first output column.
struct Tile8 {
  int e, row0, row_end, n0;
};

// MN: W is contracted over its rows (dgrad).
template <bool MN>
__global__ void __launch_bounds__(kThreads8, 1)
    bsq_fp8_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                   const __grid_constant__ CUtensorMap tm_y, const Fp8Params p) {
  using C = Fp8Cfg;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Fp8Shared& sh = *reinterpret_cast<Fp8Shared*>(smem + C::kRing + C::kOutBytes);
  volatile uint32_t* abort_flag = &sh.abort_flag;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // known to be the same in every lane
  const uint32_t elected = elect_one();

  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&sh.full[s]), 1);
      mbar_init(smem_u32(&sh.empty[s]), 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      mbar_init(smem_u32(&sh.tmem_full[b]), 1 + kScaleWarps);
      mbar_init(smem_u32(&sh.tmem_empty[b]), kPromoteWarps);
    }
    mbar_init(smem_u32(&sh.drain), 1);
    sh.abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_map(&tm_x);
    tma_prefetch_map(&tm_w);
  }
  if (warp == 9) tmem_alloc(smem_u32(&sh.tmem_base), kTmemCols8);
  if (warp == 0) {
    // Row tiles before each expert, and the offsets' validity: lane l takes experts
    // [l * per, (l + 1) * per).
    const int per = (p.E + 31) / 32;
    const int e0 = min(p.E, lane * per), e1 = min(p.E, e0 + per);
    auto end = [&](int e) { return p.offsets ? __ldg(p.offsets + e) : p.S; };
    const int first = e0 == 0 ? 0 : end(e0 - 1);
    int a = first, bad = 0, sum = 0;
    for (int e = e0; e < e1; ++e) {
      const int b = end(e);
      if (a < 0 || b < a || b > p.S) bad = 1;
      sum += (max(b - a, 0) + kRows8 - 1) / kRows8;
      a = b;
    }
    bad = __any_sync(0xffffffffu, bad);
    int at = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int o = __shfl_up_sync(0xffffffffu, at, d);
      if (lane >= d) at += o;
    }
    if (lane == 31) {
      sh.total_mt = bad ? 0 : at;
      sh.mt_start[p.E] = at;
      if (bad && blockIdx.x == 0) record_error(p.err, BSQ_DEVERR_BAD_OFFSETS);
    }
    at -= sum;
    a = first;
    for (int e = e0; e < e1; ++e) {
      const int b = end(e);
      sh.mt_start[e] = at;
      at += (max(b - a, 0) + kRows8 - 1) / kRows8;
      a = b;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = sh.tmem_base;
  const uint64_t limit = p.timeout_ns;
  const int total_tiles = sh.total_mt * p.num_nt;
  // With a split, the CTAs of a cluster take one tile, each a part of its k-blocks; without,
  // a CTA takes tiles until none is left.
  const int rank = p.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile0 = blockIdx.x / p.split, tile_step = p.split > 1 ? total_tiles : gridDim.x;
  const int kb0 = p.kblocks * rank / p.split, kb1 = p.kblocks * (rank + 1) / p.split;

  // Tile t: experts in order; within one, groups of p.raster row tiles; in a group, row tiles
  // vary fastest, so that concurrent CTAs share W tiles in L2.
  auto tile_of = [&](int t) {
    int lo = 0, hi = p.E - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sh.mt_start[mid] * p.num_nt <= t) lo = mid;
      else hi = mid - 1;
    }
    const int mts = sh.mt_start[lo + 1] - sh.mt_start[lo];
    int l = t - sh.mt_start[lo] * p.num_nt;
    const int r0 = l / (p.raster * p.num_nt) * p.raster, many = min(p.raster, mts - r0);
    l -= r0 * p.num_nt;
    const int begin = p.offsets && lo > 0 ? __ldg(p.offsets + lo - 1) : 0;
    return Tile8{lo, begin + (r0 + l % many) * kRows8, p.offsets ? __ldg(p.offsets + lo) : p.S, (l / many) * BN};
  };

  uint32_t pend_mask = 0, pend_par = 0;   // the producer's: stages it requested, parity of each one's last request
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8) {
      // ===== TMA producer =====
      if (lane == 0) {
        uint32_t st = 0, sp = 0;
        for (int t = tile0; t < total_tiles && !*abort_flag; t += tile_step) {
          const Tile8 tl = tile_of(t);
          bool ok = true;
#pragma unroll 1
          for (int kb = kb0; kb < kb1; ++kb) {
            if (!wait8(smem_u32(&sh.empty[st]), sp ^ 1u, abort_flag, p.err, limit)) { ok = false; break; }
            const uint32_t full = smem_u32(&sh.full[st]);
            if (p.drop_announce == 1 || (p.drop_announce == 2 && kb == kb1 - 1 && t + tile_step >= total_tiles)) continue;
            mbar_arrive_expect_tx(full, C::kStage);
            const uint32_t dst = smem_u32(smem + st * C::kStage);
            tma_load_2d(dst, &tm_x, full, kb * kDepth, tl.row0);
            if (MN) {
              for (int c = 0; c < BN; c += 128)   // 128 columns a box: one swizzle atom wide
                tma_load_3d(dst + kABytes + c * kDepth, &tm_w, full, tl.n0 + c, kb * kDepth, tl.e);
            } else {
              tma_load_3d(dst + kABytes, &tm_w, full, kb * kDepth, tl.n0, tl.e);
            }
            pend_mask |= 1u << st;
            pend_par = (pend_par & ~(1u << st)) | (sp << st);
            if (++st == C::kStages) {
              st = 0;
              sp ^= 1u;
            }
          }
          if (!ok) break;
        }
      }
    } else if (warp == 9) {
      // ===== MMA issuer: the whole warp walks the loop, its elected lane issues =====
      const uint32_t idesc = idesc_e4m3_f32(kRows8, BN, MN);
      const uint64_t adesc0 = sdesc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t bdesc0 = sdesc_sw128(smem_u32(smem + kABytes), 128 * kDepth, 1024);
      const uint32_t full0 = smem_u32(&sh.full[0]), empty0 = smem_u32(&sh.empty[0]);
      const uint32_t tfull0 = smem_u32(&sh.tmem_full[0]), tempty0 = smem_u32(&sh.tmem_empty[0]);
      uint32_t st = 0, sp = 0, bi = 0, bp = 1;   // stage and its parity, TMEM buffer and its empty parity
      bool ok = true;
      for (int t = tile0; t < total_tiles && all_lanes(ok && !*abort_flag); t += tile_step) {
#pragma unroll 1
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = wait8(tempty0 + 8 * bi, bp, abort_flag, p.err, limit) && wait8(full0 + 8 * st, sp, abort_flag, p.err, limit);
          __syncwarp();
          tc_fence_after();
          umma_e4m3_k128<MN ? 256 : 2>(elected, tmem_base + bi * BN, adesc0 + st * (C::kStage >> 4),
                                       bdesc0 + st * (C::kStage >> 4), idesc);
          umma_commit(elected, tfull0 + 8 * bi);
          if (!all_lanes(ok)) break;   // after a failure no operands are asked for
          umma_commit(elected, empty0 + 8 * st);
          if (++bi == C::kBufs) {
            bi = 0;
            bp ^= 1u;
          }
          if (++st == C::kStages) {
            st = 0;
            sp ^= 1u;
          }
        }
      }
    } else {
      // ===== scales: two rows a thread; a k-block ahead of its accumulator =====
      const int i = (warp - 10) * 32 + lane;
      const uint32_t tempty0 = smem_u32(&sh.tmem_empty[0]), tfull0 = smem_u32(&sh.tmem_full[0]);
      uint32_t bi = 0, bp = 1;
      bool ok = true;
      for (int t = tile0; t < total_tiles && all_lanes(ok && !*abort_flag); t += tile_step) {
        const Tile8 tl = tile_of(t);
        // rows past the expert's last and columns past the last block: not stored, any scale does
        const float* xs0 = p.xs + static_cast<int64_t>(min(tl.row0 + i, tl.row_end - 1)) * p.xs_ld;
        const float* xs1 = p.xs + static_cast<int64_t>(min(tl.row0 + i + 64, tl.row_end - 1)) * p.xs_ld;
        const float* ws0 = p.ws + tl.e * p.ws_e + static_cast<int64_t>(tl.n0 >> 7) * p.ws_o +
                           static_cast<int64_t>(kb0) * p.ws_c;
        const float* ws1 = p.ws + tl.e * p.ws_e + static_cast<int64_t>(min(tl.n0 + C::kCols, p.O - 1) >> 7) * p.ws_o +
                           static_cast<int64_t>(kb0) * p.ws_c;
#pragma unroll 1
        for (int kb = kb0; kb < kb1; ++kb) {
          const float x0 = __ldg(xs0 + kb), x1 = __ldg(xs1 + kb);
          const float w0 = __ldg(ws0), w1 = __ldg(ws1);
          ws0 += p.ws_c;
          ws1 += p.ws_c;
          ok = ok && wait8(tempty0 + 8 * bi, bp, abort_flag, p.err, limit);
          sh.scale[bi][0][i] = x0 * w0;
          sh.scale[bi][0][i + 64] = x1 * w0;
          sh.scale[bi][1][i] = x0 * w1;
          sh.scale[bi][1][i + 64] = x1 * w1;
          __syncwarp();
          if (elected && ok) mbar_arrive(tfull0 + 8 * bi);
          if (++bi == C::kBufs) {
            bi = 0;
            bp ^= 1u;
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPromoteRegs));
    // ===== promotion and epilogue: lane = output row, kCols consecutive columns =====
    const int q = warp & 3, h = warp >> 2;
    constexpr int kChunks = C::kCols / 32;   // loads of 32 columns; even, so that v[0] starts every k-block
    static_assert(kChunks % 2 == 0, "register double buffer");
    uint32_t bi = 0, bp = 0;   // TMEM buffer and its parity
    const uint32_t scale0 = smem_u32(&sh.scale[0][h][q * 32 + lane]);
    const uint32_t stage = smem_u32(smem + C::kRing) + warp * C::kOutWarp;
    const uint32_t tfull0 = smem_u32(&sh.tmem_full[0]), tempty0 = smem_u32(&sh.tmem_empty[0]);
    const uint32_t trow = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + h * C::kCols;
    bool ok = true;
    for (int t = tile0; t < total_tiles && all_lanes(!*abort_flag); t += tile_step) {
      const Tile8 tl = tile_of(t);
      const int col0 = tl.n0 + h * C::kCols;
      uint64_t acc[C::kCols / 2];
#pragma unroll
      for (int j = 0; j < C::kCols / 2; ++j) acc[j] = 0;
      uint32_t v[2][32];
      uint64_t s2;   // the k-block's scale, twice
      // the next accumulator and its scale
      auto arrived = [&]() {
        ok = ok && wait8_promote(tfull0 + 8 * bi, bp, abort_flag);
        __syncwarp();
        tc_fence_after();
        asm volatile("{\n\t.reg .b32 s;\n\tld.shared.b32 s, [%1];\n\tmov.b64 %0, {s, s};\n\t}"
                     : "=l"(s2)
                     : "r"(scale0 + bi * (2 * kRows8 * 4))
                     : "memory");
      };
      arrived();
      tmem_ld_32x32b_x32_wait(trow + bi * BN, v[0]);
#pragma unroll 1
      for (int left = kb1 - kb0; left > 0; --left) {
        const uint32_t at = trow + bi * BN;
#pragma unroll
        for (int c = 0; c + 1 < kChunks; ++c) tmem_ld_x32_fma(at + (c + 1) * 32, v[(c + 1) & 1], acc + c * 16, v[c & 1], s2);
        // every column is in registers: the TMEM is free before the last are used
        const uint64_t s = s2;
        tc_fence_before();
        __syncwarp();
        if (elected) mbar_arrive(tempty0 + 8 * bi);
        if (++bi == C::kBufs) {
          bi = 0;
          bp ^= 1u;
        }
        if (left > 1) {
          arrived();
          tmem_ld_x32_fma(trow + bi * BN, v[0], acc + (kChunks - 1) * 16, v[1], s);
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) fma_f32x2(acc[(kChunks - 1) * 16 + j], v[1][2 * j], v[1][2 * j + 1], s);
        }
      }
      if (!all_lanes(ok && !*abort_flag)) break;   // aborted: nothing is stored
      if (p.split > 1) {
        // this part of the sum, [column][row] over the operand ring: every load into it has
        // been multiplied, and a split CTA takes no further tile
        float* part = reinterpret_cast<float*>(smem) + h * C::kCols * kRows8 + q * 32 + lane;
#pragma unroll
        for (int j = 0; j < C::kCols / 2; ++j) {
          part[(2 * j) * kRows8] = __uint_as_float(static_cast<uint32_t>(acc[j]));
          part[(2 * j + 1) * kRows8] = __uint_as_float(static_cast<uint32_t>(acc[j] >> 32));
        }
      } else {
        // The warp's 32 rows x kCols columns go through shared memory (64-column boxes, 128-byte
        // swizzled) and from there by TMA, which writes them while the next tile is multiplied.
        if (lane == 0) bulk_wait_read0();   // the last tile's have been read
        __syncwarp();
#pragma unroll
        for (int c = 0; c < C::kCols / 8; ++c) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            w[j] = pack_bf16x2(static_cast<uint32_t>(acc[4 * c + j]), static_cast<uint32_t>(acc[4 * c + j] >> 32));
          sts128(stage + (c / 8) * kBoxBytes8 + lane * 128 + (((c % 8) ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
        }
        const int row0 = tl.row0 + q * 32;
        if (row0 + 32 <= tl.row_end || !p.offsets) {
          // rows past S and columns past O are clipped
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
#pragma unroll
            for (int c = 0; c < C::kCols; c += 64)
              if (row0 < p.S && col0 + c < p.O) tma_store_2d(&tm_y, stage + (c / 64) * kBoxBytes8, col0 + c, row0);
            bulk_commit();
          }
        } else {
          // the next expert's rows begin within these 32: plain stores of this one's
          __syncwarp();
#pragma unroll 4
          for (int i = lane; i < 32 * (C::kCols / 8); i += 32) {
            const int r = i / (C::kCols / 8), c = i % (C::kCols / 8);
            const uint4 o = lds128(stage + (c / 8) * kBoxBytes8 + r * 128 + (((c % 8) ^ (r & 7)) << 4));
            if (row0 + r < tl.row_end && col0 + 8 * c < p.O)   // O % 8 == 0: whole 16-byte pieces
              *reinterpret_cast<uint4*>(p.y + static_cast<int64_t>(row0 + r) * p.O + col0 + 8 * c) = o;
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all0();   // this warp's stores have been performed
  }

  if (p.split > 1) {
    // ---------------------------------------------------------------- join the parts
    // Each CTA of the cluster adds the parts of its share of the tile's columns, in rank
    // order, and writes them.  An aborted CTA's part is garbage, as the call's result is.
    __syncwarp();
    cluster_sync();
    if (warp < 8 && tile0 < total_tiles) {
      const Tile8 tl = tile_of(tile0);
      const int q = warp & 3, h = warp >> 2;
      const int row = tl.row0 + q * 32 + lane;
      const int share = BN / p.split;   // 32 columns at least: two warps of 16
      for (int c = rank * share + h * (share / 2); c < rank * share + (h + 1) * (share / 2); c += 8) {
        float sum[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = 0.f;
        const uint32_t at = smem_u32(smem) + (c * kRows8 + q * 32 + lane) * 4;
        for (int r = 0; r < p.split; ++r) {
          const uint32_t from = map_to_rank(at, r);
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = ld_shared_cluster_f32(from + j * kRows8 * 4);
#pragma unroll
          for (int j = 0; j < 8; ++j) sum[j] += v[j];
        }
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(__float_as_uint(sum[2 * i]), __float_as_uint(sum[2 * i + 1]));
        if (row < tl.row_end && tl.n0 + c < p.O)
          *reinterpret_cast<uint4*>(p.y + static_cast<int64_t>(row) * p.O + tl.n0 + c) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    __syncwarp();
    cluster_sync();   // no CTA leaves while another reads its part
  }

  // ---------------------------------------------------------------- teardown
  __syncthreads();
  // Every role has left.  After an abort copies may be in flight, also when the producer had
  // ended before it: they land before the CTA's shared memory is another's.
  if (pend_mask && *abort_flag) drain_pending<C::kStages>(sh.full, pend_mask, pend_par, kDrainLimitNs);
  if (warp == 9 && elected) {   // the lane that issued the MMAs: all of them have completed
    const uint32_t drain = smem_u32(&sh.drain);
    umma_commit(1u, drain);
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(drain, 0) && global_timer_ns() - t0 < kDrainLimitNs) {
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem_base, kTmemCols8);
}

template <bool MN>
int launch_fp8_typed(const Fp8Args& a, const char** msg) {
  using C = Fp8Cfg;
  const int64_t inner = MN ? a.N : a.K, outer = MN ? a.K : a.N;
  CUtensorMap tm_x, tm_w, tm_y;
  {
    const uint64_t dims[2] = {static_cast<uint64_t>(inner), static_cast<uint64_t>(a.S)};
    const uint64_t strides[1] = {static_cast<uint64_t>(inner)};
    const uint32_t box[2] = {kDepth, kRows8};
    if (!encode_map(&tm_x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.x, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) {
      *msg = "tensor map encoding failed for the first operand";
      return -1;
    }
  }
  {
    const uint64_t dims[3] = {static_cast<uint64_t>(a.K), static_cast<uint64_t>(a.N), static_cast<uint64_t>(a.E)};
    const uint64_t strides[2] = {static_cast<uint64_t>(a.K), static_cast<uint64_t>(a.K) * static_cast<uint64_t>(a.N)};
    const uint32_t box[3] = {128, MN ? kDepth : BN, 1};
    if (!encode_map(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, a.w, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) {
      *msg = "tensor map encoding failed for W";
      return -1;
    }
  }
  {
    const uint64_t dims[2] = {static_cast<uint64_t>(outer), static_cast<uint64_t>(a.S)};
    const uint64_t strides[1] = {static_cast<uint64_t>(outer) * 2};
    const uint32_t box[2] = {64, 32};
    if (!encode_map(&tm_y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.y, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) {
      *msg = "tensor map encoding failed for the output";
      return -1;
    }
  }
  const int64_t nb = (a.N + 127) / 128, kb = (a.K + 127) / 128;
  Fp8Params p;
  p.xs = a.x_scale;
  p.ws = a.w_scale;
  p.ws_e = nb * kb;
  p.ws_o = static_cast<int32_t>(MN ? 1 : kb);
  p.ws_c = static_cast<int32_t>(MN ? kb : 1);
  p.xs_ld = static_cast<int32_t>((inner + 127) / 128);
  p.y = static_cast<__nv_bfloat16*>(a.y);
  p.offsets = a.offsets;
  p.err = a.err;
  p.S = static_cast<int32_t>(a.S);
  p.O = static_cast<int32_t>(outer);
  p.E = static_cast<int32_t>(a.E);
  p.kblocks = static_cast<int32_t>((inner + kDepth - 1) / kDepth);
  p.num_nt = static_cast<int32_t>((outer + BN - 1) / BN);
  p.timeout_ns = wait_limit_ns();
  const char* drop = std::getenv("BSQ_TEST_DROP_ANNOUNCE");
  p.drop_announce = drop && (drop[0] == '1' || drop[0] == '2') ? drop[0] - '0' : 0;
  // an upper bound of the row tiles: the exact count depends on the offsets
  int64_t mt = (a.S + kRows8 - 1) / kRows8;
  if (a.offsets) mt += a.E < a.S ? a.E : a.S;
  if (mt * p.num_nt > INT32_MAX - 4096) {
    *msg = "too many output tiles";
    return -1;
  }
  // Every column of tiles reads the group's rows again: from L2, if they stay there.
  const int64_t groups = a.S * inner / kRasterBytes + 1;
  p.raster = static_cast<int32_t>((mt + groups - 1) / groups);
  static_assert(C::kRing + C::kOutBytes + sizeof(Fp8Shared) + 1024 <= 232448, "rings exceed the shared memory of a CTA");
  const size_t smem = static_cast<size_t>(C::kRing) + C::kOutBytes + sizeof(Fp8Shared) + 1024;
  auto kern = bsq_fp8_kernel<MN>;
  static std::atomic<uint64_t> ready;   // devices (one bit each) on which the kernel is set up
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev < 0 || dev >= kMaxDevices)) e = cudaErrorInvalidDevice;
  if (e == cudaSuccess && !(ready.load() >> dev & 1u)) {
    // the promotion warps' registers come from the launch's: a build that took fewer would
    // leave them waiting
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, kern);
    if (e == cudaSuccess && attr.numRegs != kLaunchRegs) {
      *msg = "built with another register count than its split needs";
      return -1;
    }
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e == cudaSuccess) ready.fetch_or(uint64_t(1) << dev);
  }
  // Tiles that leave more than half of the SMs without work are split over the contraction, as
  // often as fits the SMs, if it is long enough: joining the parts takes about 3 us, a k-block
  // 0.4 to 0.5 (128 x 512 x 7168, 56 k-blocks: 29 us whole, 15 in four; 8 k-blocks: 9.0 whole,
  // 9.9 in two).
  const int64_t tiles = mt * p.num_nt;
  p.split = 1;
  if (p.kblocks >= 12)
    while (p.split < kMaxSplit && tiles * p.split * 2 <= a.num_sms && p.kblocks >= p.split * 8) p.split *= 2;
  static_assert(BN * kRows8 * 4 <= C::kRing && BN / kMaxSplit % 16 == 0, "parts of a split");
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.split);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kThreads8);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = a.stream;
  cfg.attrs = attr;
  cfg.numAttrs = p.split > 1 ? 1 : 0;
  cfg.gridDim = dim3(static_cast<unsigned>(p.split > 1 ? tiles * p.split : tiles < a.num_sms ? tiles : a.num_sms));
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kern, tm_x, tm_w, tm_y, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    *msg = cudaGetErrorString(e);
    return static_cast<int>(e);
  }
  return 0;
}

}  // namespace

int launch_fp8(const Fp8Args& a, const char** msg) {
  return a.dgrad ? launch_fp8_typed<true>(a, msg) : launch_fp8_typed<false>(a, msg);
}

}  // namespace bsq
