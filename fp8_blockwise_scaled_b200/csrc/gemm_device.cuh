// Device side shared by the blockwise-scaled GEMM kernels (gemm.cu and
// gemm_grouped.cu): tile and ring constants, the control block in shared
// memory, TMEM loads, the per-K-block promotion and the tile order.
#pragma once

#include <cuda_bf16.h>

#include <cstddef>

#include "device.cuh"

namespace fp8blk {

constexpr int BM = 128;
constexpr int BK = 128;
constexpr int kThreads = 384;
constexpr int kPromoWarps = 8;
constexpr int kPromoWarp0 = 4;
constexpr int kScaleWarp = 2;
constexpr int kBWarp = 3;
constexpr int kSRing = 8;        // scale ring depth (K-blocks)
// Register split: warpgroup 0 (producers, MMA issuer) drops to kLowRegs and
// the two promotion warpgroups rise to kHighRegs; the launch allocates 168
// per thread (ptxas pins it when setmaxnreg is used), and the split must not
// exceed what the launch holds.
constexpr int kLowRegs = 80;
constexpr int kHighRegs = 208;
static_assert(128 * kLowRegs + 256 * kHighRegs <= kThreads * 168, "register split exceeds the launch allocation");
static_assert(kLowRegs % 8 == 0 && kHighRegs % 8 == 0, "setmaxnreg takes multiples of 8");

// kTensor: the one-scale-per-operand variant (no per-K-block promotion).
template <int BN, bool kTensor = false>
struct Cfg {
  // The blockwise kernel with BN = 256 stages its bf16 tile in shared memory
  // for TMA stores and keeps 3 operand stages beside it (measured on the
  // layer's GEMMs, a fourth stage gains less than the staged epilogue does).
  // BN = 128 stores from registers and keeps 6 stages; so does the
  // one-scale variant with 4 (its K loop, with no promotion, runs ahead of 3
  // stages: measured 10% slower with the staged epilogue).
  static constexpr bool kStagedOut = BN == 256 && !kTensor;
  static constexpr int kStages = kStagedOut ? 3 : (BN == 256 ? 4 : 6);
  static constexpr int kOutBytes = kStagedOut ? BM * BN * 2 : 0;
  static constexpr int kABytes = BM * BK;
  static constexpr int kBBytes = BN * BK;
  static constexpr int kStageBytes = kABytes + kBBytes;
  // TMEM accumulators: 2 x 256 columns for BN=256; 4 x 128 for BN=128.
  static constexpr int kAccBufs = (BN == 256) ? 2 : 4;
  static constexpr int kTmemCols = kAccBufs * BN;
};

// One K-block's scales for one tile.
struct ScaleSlot {
  float sa[BM];       // sa[kb][m0 + r]
  float sb[256];      // WGRAD: sb[kb][n0 + c];  FWD/DGRAD: sb[n-block][kb] in sb[0], sb[1]
};

struct Ctrl {
  uint64_t full[8];
  uint64_t empty[8];
  uint64_t tfull[4];
  uint64_t tempty[4];
  uint64_t sfull[kSRing];
  uint64_t sempty[kSRing];
  uint64_t mma_done;
  uint64_t never;         // completed by nothing: the stall test waits on it
  uint32_t tmem_base;
  int abort;
  alignas(16) ScaleSlot slots[kSRing];
};
static_assert(offsetof(Ctrl, slots) % 16 == 0, "scale slots are filled with 16-byte copies");

template <int BN, bool kTensor>
constexpr int smem_bytes() {
  using C = Cfg<BN, kTensor>;
  return 1024 + C::kStages * C::kStageBytes + C::kOutBytes + static_cast<int>(sizeof(Ctrl));
}
static_assert(smem_bytes<256, false>() <= 227 * 1024 && smem_bytes<128, false>() <= 227 * 1024 &&
                  smem_bytes<256, true>() <= 227 * 1024 && smem_bytes<128, true>() <= 227 * 1024,
              "shared memory per CTA");

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// tcgen05.wait::ld, tied to the registers it makes valid so that the
// compiler cannot read them before the wait.
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                 "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld_32x32b_x32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// tcgen05.wait::ld tied to all 32 registers of a 32-column load.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// Promotion of 16 columns of one row with packed f32x2 FMAs:
//   FWD/DGRAD: acc += P * f           (f = sa[m] * sb[n-block])
//   WGRAD    : acc += (P * sb[n]) * sa[m]
template <bool kWgrad>
__device__ __forceinline__ void promote16(float2* acc, const uint32_t* r, float f, const float* sbc, float sa) {
  const float2 f2 = make_float2(f, f), sa2 = make_float2(sa, sa);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 pj = make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
    if constexpr (kWgrad)
      acc[j] = __ffma2_rn(__fmul2_rn(pj, *reinterpret_cast<const float2*>(sbc + 2 * j)), sa2, acc[j]);
    else
      acc[j] = __ffma2_rn(pj, f2, acc[j]);
  }
}

__device__ __forceinline__ void st_global_v8(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Rounds kCols fp32 sums of one row to bf16 and stores them (32-byte stores).
template <int kCols>
__device__ __forceinline__ void store_row_bf16(uint16_t* drow, const float2* acc) {
#pragma unroll
  for (int j = 0; j < kCols; j += 16) {
    uint32_t v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = pack_bf16x2(acc[j / 2 + q].x, acc[j / 2 + q].y);
    st_global_v8(drow + j, v);
  }
}

// Stores kCols fp32 sums of one row unrounded (32-byte stores): the output of a
// partial product that is summed further (the data-parallel weight gradient).
template <int kCols>
__device__ __forceinline__ void store_row_f32(float* drow, const float2* acc) {
#pragma unroll
  for (int j = 0; j < kCols; j += 8) {
    uint32_t v[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = __float_as_uint(acc[j / 2 + q].x);
      v[2 * q + 1] = __float_as_uint(acc[j / 2 + q].y);
    }
    st_global_v8(drow + j, v);
  }
}

// Ring position: an index into a ring of N slots and the parity of its use.
template <int N>
struct Ring {
  int idx = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++idx == N) {
      idx = 0;
      phase ^= 1u;
    }
  }
};

// One promotion warp's K loop over one output tile: its 32 TMEM lanes (rows)
// times kCols = BN/2 columns starting at col0.  `release(buf)` hands TMEM
// buffer buf back to the MMA issuer.  Params: the kernel's parameters (its
// timeout_ns and err bound the waits).  Returns false when a wait gave up.
template <int BN, bool kWgrad, typename Params, typename Release>
__device__ __forceinline__ bool promote_tile(Ctrl* ctrl, const Params& p, float2 (&acc)[BN / 4], int kblocks,
                                             uint32_t tmem_lanes, int row, int col0, Ring<Cfg<BN>::kAccBufs>& tbuf,
                                             Ring<kSRing>& sring, volatile int* abort, int lane, Release release) {
  constexpr int kCols = BN / 2;
#pragma unroll
  for (int j = 0; j < kCols / 2; ++j) acc[j] = make_float2(0.0f, 0.0f);
  for (int kb = 0; kb < kblocks; ++kb) {
    // The scale producer runs up to kSRing K-blocks ahead: this wait normally
    // finds the slot filled, and the scales are in registers before the
    // accumulator arrives.
    if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded<false>(&ctrl->sfull[sring.idx], sring.phase, abort,
                                                          p.timeout_ns, p.err)))
      return false;
    const ScaleSlot& ss = ctrl->slots[sring.idx];
    const float sa = ss.sa[row];
    float f = 0.0f;
    if constexpr (!kWgrad) {
      f = sa * ss.sb[col0 / 128];          // the column slice's n-block
      __syncwarp();                        // every lane has its scales: the slot can be refilled
      if (lane == 0) mbar_arrive(&ctrl->sempty[sring.idx]);
    }
    if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded<false>(&ctrl->tfull[tbuf.idx], tbuf.phase, abort, p.timeout_ns,
                                                          p.err)))
      return false;
    tc_fence_after_sync();
    const uint32_t taddr = tmem_lanes + tbuf.idx * BN;
    const float* sbc = ss.sb + col0;
    // 32-column TMEM loads, each in flight while the FMAs of the previous
    // chunk run; the buffer goes back to the MMA issuer as soon as the last
    // load has landed, before the FMAs that consume it.
    uint32_t ra[32], rb[32];
    tmem_ld_32x32b_x32(taddr, ra);
    tmem_wait_ld32(ra);
#pragma unroll
    for (int c = 0; c < kCols; c += 64) {
      tmem_ld_32x32b_x32(taddr + c + 32, rb);
      promote16<kWgrad>(acc + c / 2, ra, f, sbc + c, sa);
      promote16<kWgrad>(acc + c / 2 + 8, ra + 16, f, sbc + c + 16, sa);
      tmem_wait_ld32(rb);
      if (c + 64 < kCols)
        tmem_ld_32x32b_x32(taddr + c + 64, ra);
      else
        release(tbuf.idx);
      promote16<kWgrad>(acc + c / 2 + 16, rb, f, sbc + c + 32, sa);
      promote16<kWgrad>(acc + c / 2 + 24, rb + 16, f, sbc + c + 48, sa);
      if (c + 64 < kCols) tmem_wait_ld32(ra);
    }
    if constexpr (kWgrad) {
      __syncwarp();                        // the column scales were read during the FMAs
      if (lane == 0) mbar_arrive(&ctrl->sempty[sring.idx]);
    }
    tbuf.next();
    sring.next();
  }
  return true;
}

// Tile order: groups of `group_m` M-blocks, N-blocks inside a group, M-blocks
// fastest inside that.  The CTAs running at the same time then share each A tile
// among ~#SMs/group_m CTAs and each B tile among group_m CTAs, instead of all
// M-blocks asking for the same B tile at once.
__device__ __forceinline__ void tile_coords(int tile, int num_mb, int num_nb, int group_m, int& mb, int& nb) {
  const int per_group = group_m * num_nb;
  const int g = tile / per_group, r = tile - g * per_group;
  const int gm = min(group_m, num_mb - g * group_m);   // the last group may be short
  mb = g * group_m + r % gm;
  nb = r / gm;
}

}  // namespace fp8blk
