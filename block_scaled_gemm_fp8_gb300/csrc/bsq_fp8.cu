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
// Pair tile: 256 rows (128 per CTA of a cta_group::2 pair) by BN output columns.  Per CTA,
// 10 warps:
//   warps 0-7   promotion and epilogue: TMEM lanes 32 (w % 4).., output columns half w / 4
//   warp 8      TMA producer: 128 x 128 bytes of the first operand, BN/2 x 128 of W's
//   warp 9      even CTA: MMA issuer; odd CTA: relays "operands landed" to it
// A 128-deep block of BN = 256 takes 512 tensor-core cycles per SM at the FP8 rate; its
// promotion is 64 packed FMAs and 4 TMEM loads per thread, about half of that, so two
// TMEM buffers keep the tensor cores fed.
#include <atomic>
#include <cstdlib>

#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include "bsq_internal.h"
#include "bsq_pipe.cuh"
#include "bsq_ptx.cuh"
#include "../../include/bsq.h"

namespace bsq {

bool encode_map(CUtensorMap* m, CUtensorMapDataType dt, uint32_t rank, const void* base, const uint64_t* dims,
                const uint64_t* strides, const uint32_t* box, CUtensorMapSwizzle sw);

namespace {

constexpr int kThreads8 = 320;
constexpr int kPair8 = 2;
constexpr uint16_t kPairMask8 = 3;
constexpr int kRows8 = 128;                 // rows of the first operand per CTA
constexpr int kDepth = 128;                 // contraction per k-block: one scale block, 128 bytes of codes
constexpr int kABytes = kRows8 * kDepth;    // 16 KB
constexpr int kTmemCols8 = 512;
constexpr int kPromoteWarps = 8;
constexpr int kMaxStages8 = 8;
constexpr int kMaxBufs8 = 4;

// BN: output columns of a pair tile.  MN: W is contracted over its rows (dgrad).
template <int BN, bool MN>
struct Fp8Cfg {
  static constexpr int kBBytes = MN ? kDepth * 128 : (BN / 2) * kDepth;   // this CTA's half of W's tile
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kStages = BN == 256 ? 6 : 8;
  static constexpr int kBufs = kTmemCols8 / BN < kMaxBufs8 ? kTmemCols8 / BN : kMaxBufs8;
  static constexpr int kCols = BN / 2;               // output columns of one promotion warp
  static constexpr int kRing = kStages * kStage;
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
  uint64_t timeout_ns;
  int32_t drop_announce;       // test hook: the odd CTA's relay never announces a stage
};

struct Fp8Shared {
  uint64_t full[kMaxStages8];       // this CTA's tiles of the stage have landed
  uint64_t peer_full[kMaxStages8];  // even CTA: the odd CTA's have
  uint64_t empty[kMaxStages8];
  uint64_t tmem_full[kMaxBufs8];
  uint64_t tmem_empty[kMaxBufs8];   // even CTA: 8 arrivals, and 4 bytes from each of the odd CTA's 8 warps
  uint64_t drain;
  uint32_t tmem_base;
  uint32_t sink;
  uint32_t abort_flag;
  int32_t total_mt;                 // row tiles of all experts; -1: bad offsets
  int32_t mt_start[kMaxExperts + 1];   // row tiles before expert e
};

// kind::f8f6f4, E4M3 x E4M3 -> F32.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(uint32_t M, uint32_t N, bool b_mn_major) {
  return (1u << 4)                              // D format: F32; A and B formats 0: E4M3
         | ((b_mn_major ? 1u : 0u) << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// The four MMAs (K = 32 each) of one 128-deep block into a fresh accumulator: A K-major,
// advancing 32 bytes a step; B by BSTEP descriptor units.
template <uint32_t BSTEP>
__device__ __forceinline__ void umma_e4m3_pair_k128(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "setp.ne.b32 p, %3, %3;\n\t"
      "setp.eq.b32 q, %3, %3;\n\t"
      "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
      "add.s64 b1, %2, %4;\n\tadd.s64 b2, %2, %5;\n\tadd.s64 b3, %2, %6;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a1, b1, %3, q;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a2, b2, %3, q;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a3, b3, %3, q;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "n"(BSTEP), "n"(2 * BSTEP), "n"(3 * BSTEP)
      : "memory");
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

// acc += p * s on a pair of FP32 values.
__device__ __forceinline__ void fma_f32x2(uint64_t& acc, uint32_t p0, uint32_t p1, uint64_t s2) {
  asm("{\n\t.reg .b64 p;\n\tmov.b64 p, {%1, %2};\n\tfma.rn.f32x2 %0, p, %3, %0;\n\t}"
      : "+l"(acc)
      : "r"(p0), "r"(p1), "l"(s2));
}

// One pair tile: the expert and its rows, and the first output column.
struct Tile8 {
  int e, row0, row_end, n0;
};

template <int BN, bool MN>
__global__ void __launch_bounds__(kThreads8, 1)
    bsq_fp8_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w, const Fp8Params p) {
  using C = Fp8Cfg<BN, MN>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Fp8Shared& sh = *reinterpret_cast<Fp8Shared*>(smem + C::kRing);
  volatile uint32_t* abort_flag = &sh.abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&sh.full[s]), 1);
      mbar_init(smem_u32(&sh.peer_full[s]), 1);
      mbar_init(smem_u32(&sh.empty[s]), 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      mbar_init(smem_u32(&sh.tmem_full[b]), 1);
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
  if (warp == 9) {
    tmem_alloc_pair(smem_u32(&sh.tmem_base), kTmemCols8);
    tmem_relinquish_pair();
  }
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
      sum += (max(b - a, 0) + kPair8 * kRows8 - 1) / (kPair8 * kRows8);
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
      at += (max(b - a, 0) + kPair8 * kRows8 - 1) / (kPair8 * kRows8);
      a = b;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();
  const uint32_t tmem_base = sh.tmem_base;
  const uint64_t limit = p.timeout_ns;
  const int rank = static_cast<int>(cluster_ctarank());
  const int cl_id = blockIdx.x / kPair8, n_cl = gridDim.x / kPair8;
  const int total_tiles = sh.total_mt * p.num_nt;
  uint32_t mma_uses = 0;   // MMA thread: k-blocks issued

  // Tile t: experts in order; within one, row tiles vary fastest, so that concurrent pairs
  // share W tiles in L2.
  auto tile_of = [&](int t) {
    int lo = 0, hi = p.E - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sh.mt_start[mid] * p.num_nt <= t) lo = mid;
      else hi = mid - 1;
    }
    const int mts = sh.mt_start[lo + 1] - sh.mt_start[lo];
    const int l = t - sh.mt_start[lo] * p.num_nt;
    const int begin = p.offsets && lo > 0 ? __ldg(p.offsets + lo - 1) : 0;
    return Tile8{lo, begin + (l % mts) * (kPair8 * kRows8), p.offsets ? __ldg(p.offsets + lo) : p.S, (l / mts) * BN};
  };

  if (warp == 8) {
    // ===== TMA producer =====
    if (lane == 0) {
      uint32_t uc = 0, pend_mask = 0, pend_par = 0;
      for (int t = cl_id; t < total_tiles && !*abort_flag; t += n_cl) {
        const Tile8 tl = tile_of(t);
        const int xrow = tl.row0 + rank * kRows8;
        const int o0 = tl.n0 + rank * (BN / 2);
        bool ok = true;
        for (int kb = 0; kb < p.kblocks; ++kb, ++uc) {
          const Slot sl = ring_slot<C::kStages>(uc);
          if (!wait_phase(smem_u32(&sh.empty[sl.idx]), sl.par ^ 1u, abort_flag, p.err, limit)) { ok = false; break; }
          const uint32_t full = smem_u32(&sh.full[sl.idx]);
          mbar_arrive_expect_tx(full, C::kStage);
          pend_mask |= 1u << sl.idx;
          pend_par = (pend_par & ~(1u << sl.idx)) | (sl.par << sl.idx);
          const uint32_t dst = smem_u32(smem + sl.idx * C::kStage);
          tma_load_2d(dst, &tm_x, full, kb * kDepth, xrow);
          if (MN) tma_load_3d(dst + kABytes, &tm_w, full, o0, kb * kDepth, tl.e);
          else tma_load_3d(dst + kABytes, &tm_w, full, kb * kDepth, o0, tl.e);
        }
        if (!ok) break;
      }
      if (*abort_flag) drain_pending<C::kStages>(sh.full, pend_mask, pend_par, kDrainLimitNs);
    }
  } else if (warp == 9) {
    if (lane == 0 && rank == 0) {
      // ===== MMA issuer =====
      const uint32_t idesc = idesc_e4m3_f32(kPair8 * kRows8, BN, MN);
      const uint64_t adesc0 = sdesc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t bdesc0 = sdesc_sw128(smem_u32(smem + kABytes), 16, 1024);
      uint32_t uc = 0;
      bool ok = true;
      for (int t = cl_id; ok && t < total_tiles && !*abort_flag; t += n_cl) {
        for (int kb = 0; kb < p.kblocks; ++kb, ++uc) {
          const Slot sl = ring_slot<C::kStages>(uc);
          const Slot sb = ring_slot<C::kBufs>(uc);
          const uint32_t peer = smem_u32(&sh.peer_full[sl.idx]);
          mbar_arrive_expect_tx(peer, 4);
          if (!wait_phase<true>(smem_u32(&sh.tmem_empty[sb.idx]), sb.par ^ 1u, abort_flag, p.err, limit) ||
              !wait_phase(smem_u32(&sh.full[sl.idx]), sl.par, abort_flag, p.err, limit) ||
              !wait_phase<true>(peer, sl.par, abort_flag, p.err, limit)) {
            ok = false;
            break;
          }
          tc_fence_after();
          umma_e4m3_pair_k128<MN ? 256 : 2>(tmem_base + sb.idx * BN, adesc0 + sl.idx * (C::kStage >> 4),
                                            bdesc0 + sl.idx * (C::kStage >> 4), idesc);
          umma_commit_pair(smem_u32(&sh.tmem_full[sb.idx]), kPairMask8);
          umma_commit_pair(smem_u32(&sh.empty[sl.idx]), kPairMask8);
          ++mma_uses;
        }
      }
    } else if (lane == 0) {
      // ===== operands-landed relay of the odd CTA =====
      uint32_t uc = 0;
      bool ok = true;
      for (int t = cl_id; ok && t < total_tiles && !*abort_flag; t += n_cl)
        for (int kb = 0; kb < p.kblocks; ++kb, ++uc) {
          const Slot sl = ring_slot<C::kStages>(uc);
          if (!wait_phase(smem_u32(&sh.full[sl.idx]), sl.par, abort_flag, p.err, limit)) { ok = false; break; }
          if (!p.drop_announce) st_async_tx_rank(smem_u32(&sh.sink), smem_u32(&sh.peer_full[sl.idx]), 0);
        }
    }
  } else {
    // ===== promotion and epilogue: lane = output row, kCols consecutive columns =====
    const int q = warp & 3, h = warp >> 2;
    uint32_t uc = 0;
    bool ok = true;
    for (int t = cl_id; t < total_tiles && !*abort_flag; t += n_cl) {
      const Tile8 tl = tile_of(t);
      const int row = tl.row0 + rank * kRows8 + q * 32 + lane;
      const int col0 = tl.n0 + h * C::kCols;
      const bool valid = row < tl.row_end;
      const float* xs = p.xs + static_cast<int64_t>(valid ? row : tl.row_end - 1) * p.xs_ld;
      // columns past the last scale block are not stored: any scale does
      const int ob = min(col0, p.O - 1) >> 7;
      const float* ws = p.ws + tl.e * p.ws_e + static_cast<int64_t>(ob) * p.ws_o;
      uint64_t acc[C::kCols / 2];
#pragma unroll
      for (int j = 0; j < C::kCols / 2; ++j) acc[j] = 0;
      float sx = __ldg(xs), sw = __ldg(ws);
      for (int kb = 0; kb < p.kblocks; ++kb, ++uc) {
        const Slot sb = ring_slot<C::kBufs>(uc);
        const float s = sx * sw;
        if (kb + 1 < p.kblocks) {
          sx = __ldg(xs + kb + 1);
          sw = __ldg(ws + static_cast<int64_t>(kb + 1) * p.ws_c);
        }
        uint64_t s2;
        asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "r"(__float_as_uint(s)));
        ok = wait_phase(smem_u32(&sh.tmem_full[sb.idx]), sb.par, abort_flag, p.err, limit);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + sb.idx * BN + h * C::kCols;
#pragma unroll
        for (int c = 0; c < C::kCols / 32; ++c) {
          uint32_t v[32];
          tmem_ld_32x32b_x32_wait(taddr + c * 32, v);
          if (c + 1 == C::kCols / 32) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if (rank == 0) mbar_arrive_expect_tx(smem_u32(&sh.tmem_empty[sb.idx]), 4);
              else st_async_tx_rank(smem_u32(&sh.sink), smem_u32(&sh.tmem_empty[sb.idx]), 0);
            }
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) fma_f32x2(acc[c * 16 + j], v[2 * j], v[2 * j + 1], s2);
        }
      }
      if (!ok) break;
      if (valid) {
        uint4* o4 = reinterpret_cast<uint4*>(p.y + static_cast<int64_t>(row) * p.O + col0);   // O % 8 == 0: 16-byte aligned
#pragma unroll
        for (int j = 0; j < C::kCols / 8; ++j) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = pack_bf16x2(static_cast<uint32_t>(acc[4 * j + i]), static_cast<uint32_t>(acc[4 * j + i] >> 32));
          if (col0 + 8 * j < p.O) o4[j] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  __syncthreads();
  if (warp == 9 && lane == 0 && rank == 0) {
    umma_commit_pair(smem_u32(&sh.drain), 1);
    uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(smem_u32(&sh.drain), 0) && global_timer_ns() - t0 < kDrainLimitNs) {
    }
    if (!*abort_flag) {
      // the odd CTA's last asynchronous stores have landed
      for (uint32_t b = 0; b < static_cast<uint32_t>(C::kBufs); ++b) {
        const uint32_t uses = (mma_uses + C::kBufs - 1u - b) / C::kBufs;
        if (uses == 0) continue;
        t0 = global_timer_ns();
        while (!mbar_try_wait(smem_u32(&sh.tmem_empty[b]), (uses - 1u) & 1u) && global_timer_ns() - t0 < kDrainLimitNs) {
        }
      }
    }
  }
  if (rank == 0 && *abort_flag) {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < kAbortSettleNs) {
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();
  if (warp == 9) tmem_dealloc_pair(tmem_base, kTmemCols8);
}

template <int BN, bool MN>
int launch_fp8_typed(const Fp8Args& a, const char** msg) {
  using C = Fp8Cfg<BN, MN>;
  const int64_t inner = MN ? a.N : a.K, outer = MN ? a.K : a.N;
  CUtensorMap tm_x, tm_w;
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
    const uint32_t box[3] = {128, MN ? kDepth : BN / 2, 1};
    if (!encode_map(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, a.w, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) {
      *msg = "tensor map encoding failed for W";
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
  p.drop_announce = drop && drop[0] == '1' ? 1 : 0;
  // an upper bound of the row tiles: the exact count depends on the offsets
  int64_t mt = (a.S + kPair8 * kRows8 - 1) / (kPair8 * kRows8);
  if (a.offsets) mt += a.E < a.S ? a.E : a.S;
  if (mt * p.num_nt > INT32_MAX - 4096) {
    *msg = "too many output tiles";
    return -1;
  }
  static_assert(C::kRing + sizeof(Fp8Shared) + 1024 <= 232448, "rings exceed the shared memory of a CTA");
  const size_t smem = static_cast<size_t>(C::kRing) + sizeof(Fp8Shared) + 1024;
  auto kern = bsq_fp8_kernel<BN, MN>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kPair8;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kThreads8);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = a.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static std::atomic<int> max_clusters_of[kMaxDevices];
  int dev = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev < 0 || dev >= kMaxDevices)) e = cudaErrorInvalidDevice;
  int max_clusters = e == cudaSuccess ? max_clusters_of[dev].load() : 0;
  if (e == cudaSuccess && max_clusters == 0) {
    cfg.gridDim = dim3(kPair8 * (a.num_sms / kPair8));
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
    max_clusters = n > 0 ? n : a.num_sms / kPair8;
    max_clusters_of[dev].store(max_clusters);
  }
  int64_t clusters = mt * p.num_nt < max_clusters ? mt * p.num_nt : max_clusters;
  if (clusters < 1) clusters = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * kPair8));
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kern, tm_x, tm_w, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    *msg = cudaGetErrorString(e);
    return static_cast<int>(e);
  }
  return 0;
}

}  // namespace

int launch_fp8(const Fp8Args& a, const char** msg) {
  return a.dgrad ? launch_fp8_typed<256, true>(a, msg) : launch_fp8_typed<256, false>(a, msg);
}

}  // namespace bsq
