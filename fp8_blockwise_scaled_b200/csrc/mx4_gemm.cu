// Products of 4-bit microscaled operands for sm_100a (tcgen05 block-scaled MMA).
//
//   D[m][n] = ga gb sum_k a[m][k] sfa(m, block of k) b[n][k] sfb(n, block of k)
//
// The tensor cores apply the block scales themselves, so a tile's whole K loop
// accumulates in TMEM in fp32 and the epilogue multiplies once by the tensors'
// scales and rounds once.  What is left to feed is the operands (128 bytes of
// codes a row and stage: 256 values of K) and their scales: a stage's scale
// atoms arrive by TMA next to the codes and are copied from shared memory to
// TMEM by tcgen05.cp, in the order of the MMAs that read them.  Two sets of
// scale columns alternate; a set is rewritten once the MMAs that read it have
// completed (their commit).  Measured against it on 8192^3: four warps that
// write the scales with tcgen05.st run MXFP4 equally fast and NVFP4 12% slower,
// copies of half the size one step ahead of the MMAs 58% slower.
//
// Warp roles (256 threads): warp 0 loads, warp 1 owns TMEM and issues copies
// and MMAs, warps 4-7 drain the accumulators (two of them alternate, so a
// tile's epilogue runs under the next tile's K loop).
//
// gemm_mx4_kernel: persistent, one CTA per SM, 128 x 128 tiles.
// gemm_mx4_pair_kernel: 256 x 256 tiles on pairs of SMs, for large outputs.
// gemm_mx4_few_kernel: few rows of a (decoding), K split over a cluster.
//
// Every wait is bounded as in gemm.cu.
#include <cudaTypedefs.h>

#include "gemm_device.cuh"
#include "gemm_host.h"
#include "kernels.h"
#include "mx4_device.cuh"

namespace fp8blk {

namespace {

constexpr int kMxThreads = 256;
constexpr int kMxPairThreads = 384;      // eight epilogue warps
constexpr int kStageK = 256;             // values of K in a stage: 128 bytes of codes
constexpr int kEpiWarp0 = 4;

struct Mx4Params {
  int64_t M, N, K;          // rows of a, rows of b, contraction
  const float* tsa;         // NVFP4: tensor scales (null = 1)
  const float* tsb;
  void* d;
  int64_t ldd;
  int out_f32;
  int group_m;
  uint64_t timeout_ns;
  unsigned int* err;
  int inject_stall;
};

constexpr int kBN = 128;                 // columns of gemm_mx4_kernel's tile: one block of scale rows

template <bool kNv>
struct MxCfg {
  static constexpr int kAtoms = kNv ? 4 : 2;              // scale atoms of 128 rows in a stage
  static constexpr int kABytes = 128 * 128;
  static constexpr int kBBytes = kBN * 128;
  static constexpr int kSfBytes = kAtoms * kMx4AtomBytes;    // of each operand
  static constexpr int kStageBytes = kABytes + kBBytes + 2 * kSfBytes;
  static constexpr int kStages = 5;
  static constexpr int kOutBytes = 4 * 2 * 4096;          // two 32-row boxes of 128 bytes for each epilogue warp
  static constexpr int kSetCols = 2 * kAtoms * 4;         // TMEM columns of one set of scales
  static constexpr int kTmemCols = 512;                   // a power of two that holds two accumulators and two sets
  static_assert(2 * kBN + 2 * kSetCols <= kTmemCols && 2 * kBN + 2 * kSetCols > kTmemCols / 2, "tensor memory");
  static_assert(kStageBytes % 1024 == 0, "swizzled tiles start on 1024-byte boundaries");
};

struct MxCtrl {
  uint64_t full[8], empty[8];
  uint64_t tfull[2], tempty[2];
  uint64_t sfree[2];                     // the MMAs that read this set of scale columns are done
  uint64_t mma_done;
  uint64_t never;
  uint32_t tmem_base;
  int abort;
};

template <bool kNv>
constexpr int mx_smem_bytes() {
  using C = MxCfg<kNv>;
  return 1024 + C::kStages * C::kStageBytes + C::kOutBytes + static_cast<int>(sizeof(MxCtrl));
}

// Waits until the oldest of a thread's kBoxes staging boxes has been read by its store.
template <int kBoxes>
__device__ __forceinline__ void bulk_wait_box_free() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kBoxes - 1) : "memory");
}

// 64 columns of one warp's 32 accumulator rows.
__device__ __forceinline__ void load_chunk(uint32_t taddr, uint32_t (&r)[2][32]) {
  tmem_ld_32x32b_x32(taddr, r[0]);
  tmem_ld_32x32b_x32(taddr + 32, r[1]);
  tmem_wait_ld32(r[0]);
  tmem_wait_ld32(r[1]);
}

// Those columns to d (row, col: the chunk's first): times alpha, rounded to bf16
// (one box of 64 columns) or as fp32 (two boxes of 32), through the warp's
// kBoxes staging boxes and TMA stores, which clip at d's last row and column.  A TMA
// store clips columns in units of 16 bytes: where N is no multiple of them, the
// last columns are stored one by one, so that nothing behind column N is
// written.  `stores`: boxes this warp has staged.
template <int kBoxes>
__device__ __forceinline__ void store_chunk(const Mx4Params& p, const CUtensorMap* tm_d, uint8_t* stg,
                                            const uint32_t (&r)[2][32], float alpha, int64_t row, int64_t col, int lane,
                                            uint32_t& stores) {
  if (col >= p.N) return;
  const bool inside = row < p.M;         // a box starts inside d or is not stored
  if (col + 64 > p.N && p.N % (p.out_f32 ? 4 : 8) != 0) {
    if (row + lane < p.M) {
      const int64_t at = (row + lane) * p.ldd + col;
#pragma unroll
      for (int j = 0; j < 64; ++j) {
        if (col + j < p.N) {
          const float v = __uint_as_float(r[j >> 5][j & 31]) * alpha;
          if (p.out_f32)
            static_cast<float*>(p.d)[at + j] = v;
          else
            static_cast<__nv_bfloat16*>(p.d)[at + j] = __float2bfloat16_rn(v);
        }
      }
    }
    __syncwarp();
  } else if (p.out_f32) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint8_t* box = stg + (stores % kBoxes) * 4096;
      if (lane == 0) bulk_wait_box_free<kBoxes>();
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<float4*>(box + lane * 128 + ((j ^ (lane & 7)) << 4)) =
            make_float4(__uint_as_float(r[h][4 * j]) * alpha, __uint_as_float(r[h][4 * j + 1]) * alpha,
                        __uint_as_float(r[h][4 * j + 2]) * alpha, __uint_as_float(r[h][4 * j + 3]) * alpha);
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) {
        if (inside && col + 32 * h < p.N)
          tma_store_2d(tm_d, box, static_cast<int>(col) + 32 * h, static_cast<int>(row));
        bulk_commit_group();
      }
      ++stores;
    }
  } else {
    uint8_t* box = stg + (stores % kBoxes) * 4096;
    if (lane == 0) bulk_wait_box_free<kBoxes>();
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t* q = r[j >> 2] + 8 * (j & 3);
      *reinterpret_cast<uint4*>(box + lane * 128 + ((j ^ (lane & 7)) << 4)) = make_uint4(
          pack_bf16x2(__uint_as_float(q[0]) * alpha, __uint_as_float(q[1]) * alpha),
          pack_bf16x2(__uint_as_float(q[2]) * alpha, __uint_as_float(q[3]) * alpha),
          pack_bf16x2(__uint_as_float(q[4]) * alpha, __uint_as_float(q[5]) * alpha),
          pack_bf16x2(__uint_as_float(q[6]) * alpha, __uint_as_float(q[7]) * alpha));
    }
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) {
      if (inside) tma_store_2d(tm_d, box, static_cast<int>(col), static_cast<int>(row));
      bulk_commit_group();
    }
    ++stores;
  }
}

}  // namespace

template <bool kNv>
__global__ void __launch_bounds__(kMxThreads, 1)
    gemm_mx4_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                    const __grid_constant__ CUtensorMap tm_sa, const __grid_constant__ CUtensorMap tm_sb,
                    const __grid_constant__ CUtensorMap tm_d, const Mx4Params p) {
  using C = MxCfg<kNv>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* smem_out = smem + C::kStages * C::kStageBytes;
  MxCtrl* ctrl = reinterpret_cast<MxCtrl*>(smem_out + C::kOutBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int num_mb = static_cast<int>((p.M + 127) / 128), num_nb = static_cast<int>((p.N + kBN - 1) / kBN);
  const int kblocks = static_cast<int>((p.K + kStageK - 1) / kStageK);
  const int tiles = num_mb * num_nb;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&ctrl->full[s], 1);
      mbar_init(&ctrl->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctrl->tfull[b], 1);
      mbar_init(&ctrl->tempty[b], 4);
      mbar_init(&ctrl->sfree[b], 1);
    }
    mbar_init(&ctrl->mma_done, 1);
    mbar_init(&ctrl->never, 1);
    ctrl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctrl->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const uint32_t tmem_base = ctrl->tmem_base;
  volatile int* abort = &ctrl->abort;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_map(&tm_a);
      tma_prefetch_map(&tm_b);
      tma_prefetch_map(&tm_sa);
      tma_prefetch_map(&tm_sb);
      Ring<C::kStages> st;
      int64_t issued = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < tiles; u += gridDim.x) {
        int mb, nb;
        tile_coords(u, num_mb, num_nb, p.group_m, mb, nb);
        for (int kb = 0; kb < kblocks; ++kb) {
          if (!mbar_wait_bounded(&ctrl->empty[st.idx], st.phase ^ 1u, abort, p.timeout_ns, p.err)) {
            ok = false;
            break;
          }
          uint8_t* stage = smem + st.idx * C::kStageBytes;
          uint64_t* full = &ctrl->full[st.idx];
          mbar_arrive_expect_tx(full, C::kStageBytes);
          tma_load_2d(stage, &tm_a, full, kb * 128, mb * 128);
          tma_load_2d(stage + C::kABytes, &tm_b, full, kb * 128, nb * kBN);
          // Scale maps: rows of 128-row blocks, columns of 8-byte words, 64 to an atom.
          tma_load_2d(stage + C::kABytes + C::kBBytes, &tm_sa, full, kb * C::kAtoms * 64, mb);
          tma_load_2d(stage + C::kABytes + C::kBBytes + C::kSfBytes, &tm_sb, full, kb * C::kAtoms * 64, nb);
          ++issued;
          st.next();
        }
      }
      const int64_t first = issued > C::kStages ? issued - C::kStages : 0;
      for (int64_t j = first; j < issued; ++j)
        mbar_wait_bounded(&ctrl->full[j % C::kStages], static_cast<uint32_t>((j / C::kStages) & 1), nullptr,
                          p.timeout_ns, p.err);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = elect_one();
    constexpr uint32_t idesc = idesc_mx4(128, kBN, kNv);
    const uint32_t smem0 = smem_addr(smem);
    Ring<C::kStages> st;
    Ring<2> acc, set;
    bool ok = true;
    if (p.inject_stall) ok = mbar_wait_bounded(&ctrl->never, 0, abort, p.timeout_ns, p.err);
    ok = __all_sync(0xFFFFFFFFu, ok);
    for (int u = blockIdx.x; ok && u < tiles; u += gridDim.x) {
      if (!__all_sync(0xFFFFFFFFu,
                      mbar_wait_hot(&ctrl->tempty[acc.idx], acc.phase ^ 1u, abort, 0, p.timeout_ns, p.err)))
        break;
      const uint32_t d_tmem = tmem_base + acc.idx * kBN;
      for (int kb = 0; kb < kblocks; ++kb) {
        const bool got = mbar_wait_hot(&ctrl->full[st.idx], st.phase, abort, 0, p.timeout_ns, p.err) &&
                         mbar_wait_hot(&ctrl->sfree[set.idx], set.phase ^ 1u, abort, 0, p.timeout_ns, p.err);
        if (!__all_sync(0xFFFFFFFFu, got)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t a_addr = smem0 + st.idx * C::kStageBytes;
        const uint32_t sf_addr = a_addr + C::kABytes + C::kBBytes;
        const uint64_t adesc = smem_desc_kmajor_sw128(a_addr);
        const uint64_t bdesc = smem_desc_kmajor_sw128(a_addr + C::kABytes);
        const uint64_t sfdesc = smem_desc_atom(sf_addr);
        const uint32_t sfa = tmem_base + 2 * kBN + set.idx * C::kSetCols, sfb = sfa + C::kAtoms * 4;
        const int steps = static_cast<int>(min((p.K - static_cast<int64_t>(kb) * kStageK + 63) / 64, int64_t{4}));
        if (leader) {
#pragma unroll
          for (int i = 0; i < C::kAtoms; ++i) {
            tmem_cp_atom(sfa + 4 * i, sfdesc + i * (kMx4AtomBytes >> 4));
            tmem_cp_atom(sfb + 4 * i, sfdesc + ((C::kSfBytes + i * kMx4AtomBytes) >> 4));
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k < steps) {
              const int atom = kNv ? k : k >> 1;
              umma_mx4<kNv>(d_tmem, adesc + 2 * k, bdesc + 2 * k, idesc | idesc_scale_id(kNv ? 0 : 2 * (k & 1)),
                            sfa + 4 * atom, sfb + 4 * atom, (kb | k) != 0);
            }
          }
          umma_commit(&ctrl->empty[st.idx]);
          umma_commit(&ctrl->sfree[set.idx]);
          if (kb == kblocks - 1) umma_commit(&ctrl->tfull[acc.idx]);
        }
        __syncwarp();
        st.next();
        set.next();
      }
      acc.next();
    }
    if (leader) umma_commit(&ctrl->mma_done);
    __syncwarp();
    mbar_wait_bounded(&ctrl->mma_done, 0, nullptr, p.timeout_ns, p.err);
  } else if (warp >= kEpiWarp0) {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;
    const uint32_t lanes = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    uint8_t* stg = smem_out + quarter * 8192;
    const float alpha = (p.tsa ? __ldg(p.tsa) : 1.0f) * (p.tsb ? __ldg(p.tsb) : 1.0f);
    Ring<2> acc;
    uint32_t stores = 0;
    for (int u = blockIdx.x; u < tiles; u += gridDim.x) {
      int mb, nb;
      tile_coords(u, num_mb, num_nb, p.group_m, mb, nb);
      if (!__all_sync(0xFFFFFFFFu,
                      mbar_wait_bounded(&ctrl->tfull[acc.idx], acc.phase, abort, p.timeout_ns, p.err)))
        break;
      tc_fence_after_sync();
      const uint32_t taddr = lanes + acc.idx * kBN;
#pragma unroll 1
      for (int c = 0; c < kBN; c += 64) {
        uint32_t r[2][32];
        load_chunk(taddr + c, r);
        store_chunk<2>(p, &tm_d, stg, r, alpha, static_cast<int64_t>(mb) * 128 + quarter * 32,
                       static_cast<int64_t>(nb) * kBN + c, lane, stores);
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctrl->tempty[acc.idx]);
      acc.next();
    }
    if (lane == 0) bulk_wait_group0();
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// Pair kernel: a cluster of two CTAs computes a 256 x 256 tile with
// tcgen05.mma.cta_group::2.  Each CTA loads its own 128 rows of a and half of
// the 256 rows of b, so a stage moves 32 KB of codes into each SM for 256 x 256 x
// 256 products (the 1-CTA kernel moves 32 KB for 128 x 128 x 256), which is what
// the SMs' share of L2 bandwidth asks for at the 4-bit rate; and, in its own
// TMEM, holds its rows' sums, the scales of its rows of a and those of all 256
// rows of b.
//
// TMEM: two accumulators of 256 columns and two sets of scale columns do not fit
// 512 columns, so the accumulators overlap by kOverlap columns.  A tile's
// epilogue drains those first and then lets the issuer start the next tile,
// whose other columns were drained a tile earlier.
//
// What bounds it: power.  A stage takes 735 (MXFP4) or 768 cycles (NVFP4) where
// its MMAs alone take 512, but the SMs run at 1.6 GHz under it, and variants that
// need fewer cycles ran at lower clocks for the same time.  8192^3 alone: 211 to 213
// us, 5.2 PFLOP/s (MXFP4), 222 to 227 us (NVFP4); call after call 240 us at a median
// of 1.56 GHz, 258 us at 1.51.  With K = 1536 another 1500 cycles a tile go
// to the hand-over between tiles.
namespace {

template <bool kNv>
struct MxPairCfg {
  static constexpr int kAtoms = kNv ? 4 : 2;
  static constexpr int kHalfBytes = 128 * 128;            // own rows of a, or own half of b
  static constexpr int kSfBytes = kAtoms * kMx4AtomBytes; // of 128 rows
  static constexpr int kStageBytes = 2 * kHalfBytes + 3 * kSfBytes;
  static constexpr int kStages = 5;
  static constexpr int kOutBytes = 8 * 4096;              // one 32-row box of 128 bytes for each epilogue warp
  static constexpr int kSetCols = 3 * kAtoms * 4;
  static constexpr int kScaleCol = 512 - 2 * kSetCols;
  static constexpr int kAcc1 = kScaleCol - 256;           // first column of the second accumulator
  static constexpr int kOverlap = 256 - kAcc1;
  static_assert(kOverlap <= 128, "an epilogue drains half of its columns before the next tile starts");
  static_assert(kStageBytes % 1024 == 0, "swizzled tiles start on 1024-byte boundaries");
  static constexpr int kSmem = 1024 + kStages * kStageBytes + kOutBytes + static_cast<int>(sizeof(MxCtrl));
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
};

}  // namespace

template <bool kNv>
__global__ void __launch_bounds__(kMxPairThreads, 1)
    gemm_mx4_pair_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                         const __grid_constant__ CUtensorMap tm_sa, const __grid_constant__ CUtensorMap tm_sb,
                         const __grid_constant__ CUtensorMap tm_d, const Mx4Params p) {
  using C = MxPairCfg<kNv>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* smem_out = smem + C::kStages * C::kStageBytes;
  MxCtrl* ctrl = reinterpret_cast<MxCtrl*>(smem_out + C::kOutBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int num_mb = static_cast<int>((p.M + 255) / 256), num_nb = static_cast<int>((p.N + 255) / 256);
  const int kblocks = static_cast<int>((p.K + kStageK - 1) / kStageK);
  const int tiles = num_mb * num_nb;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&ctrl->full[s], 1);      // the leader's arrive + the bytes of both CTAs
      mbar_init(&ctrl->empty[s], 1);     // the leader's MMA commit
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctrl->tfull[b], 1);
      mbar_init(&ctrl->sfree[b], 1);
    }
    mbar_init(&ctrl->tempty[0], 16);     // the epilogue warps of both CTAs: the overlap is drained
    mbar_init(&ctrl->mma_done, 1);
    mbar_init(&ctrl->never, 1);
    ctrl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(&ctrl->tmem_base, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before any cross-CTA signal
  tc_fence_after_sync();
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const uint32_t tmem_base = ctrl->tmem_base;
  volatile int* abort = &ctrl->abort;
  const uint32_t peer_abort = mapa_shared(smem_addr(&ctrl->abort), rank ^ 1u);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_map(&tm_a);
      tma_prefetch_map(&tm_b);
      tma_prefetch_map(&tm_sa);
      tma_prefetch_map(&tm_sb);
      Ring<C::kStages> st;
      int64_t issued = 0;
      bool ok = true;
      for (int u = pair; ok && u < tiles; u += npairs) {
        int mb, nb;
        tile_coords(u, num_mb, num_nb, p.group_m, mb, nb);
        for (int kb = 0; kb < kblocks; ++kb) {
          if (!mbar_wait_bounded_pair(&ctrl->empty[st.idx], st.phase ^ 1u, abort, peer_abort, p.timeout_ns, p.err)) {
            ok = false;
            break;
          }
          uint8_t* stage = smem + st.idx * C::kStageBytes;
          const uint32_t full = mapa_shared(smem_addr(&ctrl->full[st.idx]), 0);
          if (leader) mbar_arrive_expect_tx(&ctrl->full[st.idx], 2 * C::kStageBytes);
          tma_load_2d_pair(stage, &tm_a, full, kb * 128, mb * 256 + static_cast<int>(rank) * 128);
          tma_load_2d_pair(stage + C::kHalfBytes, &tm_b, full, kb * 128, nb * 256 + static_cast<int>(rank) * 128);
          tma_load_2d_pair(stage + 2 * C::kHalfBytes, &tm_sa, full, kb * C::kAtoms * 64, mb * 2 + static_cast<int>(rank));
          tma_load_2d_pair(stage + 2 * C::kHalfBytes + C::kSfBytes, &tm_sb, full, kb * C::kAtoms * 64, nb * 2);
          ++issued;
          st.next();
        }
      }
      if (leader) {
        // The leader's full barriers count the bytes of both CTAs.
        const int64_t first = issued > C::kStages ? issued - C::kStages : 0;
        for (int64_t j = first; j < issued; ++j)
          mbar_wait_bounded(&ctrl->full[j % C::kStages], static_cast<uint32_t>((j / C::kStages) & 1), nullptr,
                            p.timeout_ns, p.err);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (of the leader CTA)
    if (leader) {
      const bool issuer = elect_one();
      constexpr uint32_t idesc = idesc_mx4(256, 256, kNv);
      const uint32_t smem0 = smem_addr(smem);
      Ring<C::kStages> st;
      Ring<2> acc, set;
      uint32_t drained = 1;              // parity of the last tile's drain (the first tile waits for none)
      bool ok = true;
      if (p.inject_stall) ok = mbar_wait_bounded_pair(&ctrl->never, 0, abort, peer_abort, p.timeout_ns, p.err);
      ok = __all_sync(0xFFFFFFFFu, ok);
      for (int u = pair; ok && u < tiles; u += npairs) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_hot(&ctrl->tempty[0], drained, abort, peer_abort,
                                                                   p.timeout_ns, p.err)))
          break;
        drained ^= 1u;
        const uint32_t d_tmem = tmem_base + acc.idx * C::kAcc1;
        for (int kb = 0; kb < kblocks; ++kb) {
          const bool got =
              mbar_wait_hot(&ctrl->full[st.idx], st.phase, abort, peer_abort, p.timeout_ns, p.err) &&
              mbar_wait_hot(&ctrl->sfree[set.idx], set.phase ^ 1u, abort, peer_abort, p.timeout_ns,
                                            p.err);
          if (!__all_sync(0xFFFFFFFFu, got)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t a_addr = smem0 + st.idx * C::kStageBytes;
          const uint64_t adesc = smem_desc_kmajor_sw128(a_addr);
          const uint64_t bdesc = smem_desc_kmajor_sw128(a_addr + C::kHalfBytes);
          const uint64_t sfdesc = smem_desc_atom(a_addr + 2 * C::kHalfBytes);
          const uint32_t sfa = tmem_base + C::kScaleCol + set.idx * C::kSetCols, sfb = sfa + C::kAtoms * 4;
          const int steps = static_cast<int>(min((p.K - static_cast<int64_t>(kb) * kStageK + 63) / 64, int64_t{4}));
          if (issuer) {
#pragma unroll
            for (int i = 0; i < C::kAtoms; ++i) {
              constexpr int kSf = C::kSfBytes >> 4, kAtom = kMx4AtomBytes >> 4;
              tmem_cp_atom_pair(sfa + 4 * i, sfdesc + i * kAtom);
              tmem_cp_atom_pair(sfb + 8 * i, sfdesc + kSf + i * kAtom);
              tmem_cp_atom_pair(sfb + 8 * i + 4, sfdesc + 2 * kSf + i * kAtom);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (k < steps) {
                const int atom = kNv ? k : k >> 1;
                umma_mx4_pair<kNv>(d_tmem, adesc + 2 * k, bdesc + 2 * k, idesc | idesc_scale_id(kNv ? 0 : 2 * (k & 1)),
                                   sfa + 4 * atom, sfb + 8 * atom, (kb | k) != 0);
              }
            }
            umma_commit_pair(&ctrl->empty[st.idx], 0x3);
            umma_commit_pair(&ctrl->sfree[set.idx], 0x1);
            if (kb == kblocks - 1) umma_commit_pair(&ctrl->tfull[acc.idx], 0x3);
          }
          __syncwarp();
          st.next();
          set.next();
        }
        acc.next();
      }
      if (issuer) umma_commit_pair(&ctrl->mma_done, 0x1);
      __syncwarp();
      mbar_wait_bounded(&ctrl->mma_done, 0, nullptr, p.timeout_ns, p.err);
    }
  } else if (warp >= kEpiWarp0) {
    // ------------------------------------------------------------ epilogue
    // Two warpgroups: of each half of the columns a warp takes 64.
    const int quarter = warp & 3, part = 64 * ((warp - kEpiWarp0) >> 2);
    const uint32_t lanes = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    uint8_t* stg = smem_out + (warp - kEpiWarp0) * 4096;
    const float alpha = (p.tsa ? __ldg(p.tsa) : 1.0f) * (p.tsb ? __ldg(p.tsb) : 1.0f);
    const uint32_t tempty = mapa_shared(smem_addr(&ctrl->tempty[0]), 0);
    Ring<2> acc;
    uint32_t stores = 0;
    for (int u = pair; u < tiles; u += npairs) {
      int mb, nb;
      tile_coords(u, num_mb, num_nb, p.group_m, mb, nb);
      if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded_pair(&ctrl->tfull[acc.idx], acc.phase, abort, peer_abort,
                                                                 p.timeout_ns, p.err)))
        break;
      tc_fence_after_sync();
      const uint32_t taddr = lanes + acc.idx * C::kAcc1;
      const int64_t row = static_cast<int64_t>(mb) * 256 + rank * 128 + quarter * 32, col = static_cast<int64_t>(nb) * 256;
      // The half that overlaps the other accumulator first; once it is in
      // registers the next tile may start.
      const int first = (acc.idx == 0 ? 128 : 0) + part, second = first ^ 128;
      uint32_t r[2][32];
      load_chunk(taddr + first, r);
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if (leader)
          mbar_arrive(&ctrl->tempty[0]);
        else
          mbar_arrive_remote(tempty);
      }
      store_chunk<1>(p, &tm_d, stg, r, alpha, row, col + first, lane, stores);
      load_chunk(taddr + second, r);
      store_chunk<1>(p, &tm_d, stg, r, alpha, row, col + second, lane, stores);
      tc_fence_before_sync();
      acc.next();
    }
    if (lane == 0) bulk_wait_group0();
  }

  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();  // every MMA of the pair is done and no signal is left in flight
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// ---------------------------------------------------------------------------
// Few rows of a (M <= BN = 16, 32 or 64: decoding).  The operands' roles are
// exchanged: 128 rows of b are the MMA's M side and all rows of a its N side, so
// the tile is D transposed and the work is one read of b.  That read is bound by
// HBM where b is large and by latency where it is not, so the K loop of a tile is
// split over the CTAs of a cluster (1 to 8): each sums its stages in TMEM and
// leaves the fp32 partial tile in its shared memory; after a cluster barrier
// each adds its share of the columns over the partials in the order of their
// ranks (always the same sum) and stores it.  N = 1536, K = 8960, one row: 15.8 us
// unsplit, 6.4 us split.
//
// kQuant: a is not codes but up to 16 rows of bf16 x, quantised on the way by the
// epilogue's warps (which have nothing else to do yet): a thread turns 32 values
// of a row into the 16 bytes of codes and the scale bytes that TMA would have
// brought.  Every CTA of a K range does that again, for a few KB from L2; a launch
// and a round trip of codes through memory are saved.
namespace {

// x of a product that quantises on the way.
struct FewInput {
  const uint16_t* x;
  int64_t ldx;
};

template <int BN, bool kNv>
struct FewCfg {
  static constexpr int kAtoms = kNv ? 4 : 2;
  static constexpr int kABytes = 128 * 128;               // b: the MMA's A operand
  static constexpr int kBBytes = BN * 128;
  static constexpr int kSfBytes = kAtoms * kMx4AtomBytes;
  static constexpr int kStageBytes = kABytes + kBBytes + 2 * kSfBytes;
  static constexpr int kStages = BN == 64 ? 3 : 4;        // two CTAs per SM
  static constexpr int kSetCols = 2 * kAtoms * 4;
  static constexpr int kScaleCol = BN < 32 ? 32 : BN;
  static constexpr int kTmemCols = 128;
  static_assert(kScaleCol + 2 * kSetCols <= kTmemCols, "accumulator and two sets of scales");
  static_assert(kStageBytes % 1024 == 0, "swizzled tiles start on 1024-byte boundaries");
  static_assert(BN * 128 * 4 <= kStages * kStageBytes, "the partial tile takes the stages' place");
};

template <int BN, bool kNv>
constexpr int few_smem_bytes() {
  return 1024 + FewCfg<BN, kNv>::kStages * FewCfg<BN, kNv>::kStageBytes + static_cast<int>(sizeof(MxCtrl));
}
static_assert(2 * (few_smem_bytes<64, true>() + 1024) <= 227 * 1024 && 2 * (few_smem_bytes<32, true>() + 1024) <= 227 * 1024,
              "two CTAs per SM");

__device__ __forceinline__ float4 ld_shared_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

}  // namespace

// The scale of 16 or 32 values, and their codes: w[0 .. 7] bf16 pairs -> two words a
// block of 16.
template <bool kNv>
__device__ __forceinline__ uint32_t quant_block(const uint4* w, int n, float g, float rg, uint32_t* codes) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < n; ++i)
    m = __vmaxu2(m, __vmaxu2(__vmaxu2(w[i].x & kAbs2, w[i].y & kAbs2), __vmaxu2(w[i].z & kAbs2, w[i].w & kAbs2)));
  QScale q;
  const uint32_t byte = block_scale<kNv>(__uint_as_float(max(m << 16, m & 0xFFFF0000u)), g, rg, q);
#pragma unroll
  for (int i = 0; i < n; ++i) {
    float x[8], v[8];
    unpack8(w[i], x);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 r = scaled2<kNv>(make_float2(x[j], x[j + 1]), make_float2(q.s, q.s), make_float2(q.nr, q.nr));
      v[j] = r.x;
      v[j + 1] = r.y;
    }
    codes[i] = finish_codes<kNv>(cvt8_e2m1(v), q.nr);
  }
  return byte;
}

template <int BN, bool kNv, bool kQuant>
__global__ void __launch_bounds__(kMxThreads, 2)
    gemm_mx4_few_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                        const __grid_constant__ CUtensorMap tm_sa, const __grid_constant__ CUtensorMap tm_sb,
                        const Mx4Params p, int splits, const FewInput in) {
  static_assert(!kQuant || BN == 16, "128 threads quantise 16 rows x 256 values, 32 each");
  using C = FewCfg<BN, kNv>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  MxCtrl* ctrl = reinterpret_cast<MxCtrl*>(smem + C::kStages * C::kStageBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = static_cast<int>(blockIdx.x) / splits, rank = static_cast<int>(blockIdx.x) - tile * splits;
  const int64_t all = (p.K + kStageK - 1) / kStageK;
  const int kb0 = static_cast<int>(rank * all / splits), kb1 = static_cast<int>((rank + 1) * all / splits);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&ctrl->full[s], kQuant ? 5 : 1);   // the producer, and the warps that quantise
      mbar_init(&ctrl->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) mbar_init(&ctrl->sfree[b], 1);
    mbar_init(&ctrl->mma_done, 1);
    mbar_init(&ctrl->never, 1);
    ctrl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctrl->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const uint32_t tmem_base = ctrl->tmem_base;
  volatile int* abort = &ctrl->abort;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int issued = 0;
      Ring<C::kStages> st;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait_bounded(&ctrl->empty[st.idx], st.phase ^ 1u, abort, p.timeout_ns, p.err)) break;
        uint8_t* stage = smem + st.idx * C::kStageBytes;
        uint64_t* full = &ctrl->full[st.idx];
        mbar_arrive_expect_tx(full, kQuant ? C::kABytes + C::kSfBytes : C::kStageBytes);
        tma_load_2d(stage, &tm_b, full, kb * 128, tile * 128);
        tma_load_2d(stage + C::kABytes + C::kBBytes, &tm_sb, full, kb * C::kAtoms * 64, tile);
        if constexpr (!kQuant) {
          tma_load_2d(stage + C::kABytes, &tm_a, full, kb * 128, 0);
          tma_load_2d(stage + C::kABytes + C::kBBytes + C::kSfBytes, &tm_sa, full, kb * C::kAtoms * 64, 0);
        }
        ++issued;
        st.next();
      }
      for (int j = issued > C::kStages ? issued - C::kStages : 0; j < issued; ++j)
        mbar_wait_bounded(&ctrl->full[j % C::kStages], static_cast<uint32_t>((j / C::kStages) & 1), nullptr,
                          p.timeout_ns, p.err);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = elect_one();
    constexpr uint32_t idesc = idesc_mx4(128, BN, kNv);
    const uint32_t smem0 = smem_addr(smem);
    Ring<C::kStages> st;
    Ring<2> set;
    bool ok = true;
    if (p.inject_stall) ok = mbar_wait_bounded(&ctrl->never, 0, abort, p.timeout_ns, p.err);
    ok = __all_sync(0xFFFFFFFFu, ok);
    for (int kb = kb0; ok && kb < kb1; ++kb) {
      const bool got = mbar_wait_hot(&ctrl->full[st.idx], st.phase, abort, 0, p.timeout_ns, p.err) &&
                       mbar_wait_hot(&ctrl->sfree[set.idx], set.phase ^ 1u, abort, 0, p.timeout_ns, p.err);
      ok = __all_sync(0xFFFFFFFFu, got);
      if (!ok) break;
      tc_fence_after_sync();
      const uint32_t a_addr = smem0 + st.idx * C::kStageBytes;
      const uint64_t adesc = smem_desc_kmajor_sw128(a_addr), bdesc = smem_desc_kmajor_sw128(a_addr + C::kABytes);
      const uint64_t sfdesc = smem_desc_atom(a_addr + C::kABytes + C::kBBytes);
      const uint32_t sfa = tmem_base + C::kScaleCol + set.idx * C::kSetCols, sfb = sfa + C::kAtoms * 4;
      const int steps = static_cast<int>(min((p.K - static_cast<int64_t>(kb) * kStageK + 63) / 64, int64_t{4}));
      if (leader) {
#pragma unroll
        for (int i = 0; i < C::kAtoms; ++i) {
          tmem_cp_atom(sfa + 4 * i, sfdesc + i * (kMx4AtomBytes >> 4));
          tmem_cp_atom(sfb + 4 * i, sfdesc + ((C::kSfBytes + i * kMx4AtomBytes) >> 4));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k < steps) {
            const int atom = kNv ? k : k >> 1;
            umma_mx4<kNv>(tmem_base, adesc + 2 * k, bdesc + 2 * k, idesc | idesc_scale_id(kNv ? 0 : 2 * (k & 1)),
                          sfa + 4 * atom, sfb + 4 * atom, (kb != kb0) | (k != 0));
          }
        }
        umma_commit(&ctrl->empty[st.idx]);
        umma_commit(&ctrl->sfree[set.idx]);
      }
      __syncwarp();
      st.next();
      set.next();
    }
    if (leader) umma_commit(&ctrl->mma_done);
    __syncwarp();
    // The partial tile takes the stages' place: only when every stage has arrived and been read.
    if (!mbar_wait_bounded(&ctrl->mma_done, 0, nullptr, p.timeout_ns, p.err) || !ok) *abort = 1;
  } else if (kQuant && warp >= kEpiWarp0) {
    // ------------------------------------------------------------ x to codes, in the stages' layout
    const int q = threadIdx.x - 32 * kEpiWarp0, row = q >> 3, part = q & 7;   // values 32 part .. of the stage
    const float g = kNv && p.tsa ? __ldg(p.tsa) : 1.0f, rg = __frcp_rn(g);
    const uint16_t* xr = in.x + static_cast<int64_t>(row < p.M ? row : 0) * in.ldx + 32 * part;
    auto load = [&](int kb, uint4 (&w)[4]) {
      const int64_t k = static_cast<int64_t>(kb) * kStageK;
      const bool inside = kb < kb1 && row < p.M && k + 32 * part < p.K;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = inside ? __ldg(reinterpret_cast<const uint4*>(xr + k) + i) : make_uint4(0, 0, 0, 0);
    };
    Ring<C::kStages> st;
    uint4 w[4], next[4];
    load(kb0, w);
    for (int kb = kb0; kb < kb1; ++kb) {
      load(kb + 1, next);                // in flight while this stage's values are turned into codes
      if (!__all_sync(0xFFFFFFFFu,
                      mbar_wait_bounded(&ctrl->empty[st.idx], st.phase ^ 1u, abort, p.timeout_ns, p.err)))
        break;
      uint8_t* codes = smem + st.idx * C::kStageBytes + C::kABytes;
      uint8_t* scales = codes + C::kBBytes + C::kSfBytes;
      uint32_t c[4];
      if constexpr (kNv) {
        const uint32_t b0 = quant_block<kNv>(w, 2, g, rg, c), b1 = quant_block<kNv>(w + 2, 2, g, rg, c + 2);
        *reinterpret_cast<uint16_t*>(scales + (part >> 1) * kMx4AtomBytes + row * 16 + 2 * (part & 1)) =
            static_cast<uint16_t>(b0 | (b1 << 8));
      } else {
        scales[(part >> 2) * kMx4AtomBytes + row * 16 + (part & 3)] =
            static_cast<uint8_t>(finish_scales<kNv>(quant_block<kNv>(w, 4, g, rg, c)));
      }
      *reinterpret_cast<uint4*>(codes + row * 128 + ((part ^ (row & 7)) << 4)) = make_uint4(c[0], c[1], c[2], c[3]);
      fence_proxy_async_shared();        // the writes above, then the tensor cores' reads
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctrl->full[st.idx]);
      st.next();
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = next[i];
    }
  }
  tc_fence_before_sync();
  __syncthreads();                       // the sums are complete (or a role gave up)
  const bool done = *abort == 0;
  const int rows = static_cast<int>(p.M);
  float* part = reinterpret_cast<float*>(smem);   // [rows][128]
  if (done && warp >= kEpiWarp0) {
    tc_fence_after_sync();
    const int quarter = warp & 3;
    const uint32_t lanes = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    for (int c = 0; c < rows; c += 16) {
      uint32_t r[16];
      tmem_ld_32x32b_x16(lanes + c, r);
      tmem_wait_ld16(r);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (c + j < rows) part[(c + j) * 128 + quarter * 32 + lane] = __uint_as_float(r[j]);
    }
  }
  tc_fence_before_sync();
  if (splits > 1) {
    cluster_sync();
  } else {
    __syncthreads();
  }
  // Column n of the tile: this CTA's share is 128 / splits of them.
  if (done) {
    const float alpha = (p.tsa ? __ldg(p.tsa) : 1.0f) * (p.tsb ? __ldg(p.tsb) : 1.0f);
    // Four columns a thread and step; the partials of all ranks are loaded before any is added.
    const int share = 128 / splits, quads = share / 4;
    const uint32_t part0 = smem_addr(part);
    for (int i = threadIdx.x; i < rows * quads; i += kMxThreads) {
      const int m = i / quads, n = rank * share + 4 * (i - m * quads);
      const uint32_t at = part0 + static_cast<uint32_t>(m * 128 + n) * 4;
      float4 v[8];
#pragma unroll
      for (int s = 0; s < 8; ++s)
        if (s < splits) v[s] = ld_shared_cluster_v4(mapa_shared(at, s));
      float4 sum = v[0];
#pragma unroll
      for (int s = 1; s < 8; ++s) {
        if (s < splits) {
          sum.x += v[s].x;
          sum.y += v[s].y;
          sum.z += v[s].z;
          sum.w += v[s].w;
        }
      }
      const float out[4] = {sum.x * alpha, sum.y * alpha, sum.z * alpha, sum.w * alpha};
      const int64_t col = static_cast<int64_t>(tile) * 128 + n;
      float* df = static_cast<float*>(p.d) + m * p.ldd + col;
      __nv_bfloat16* db = static_cast<__nv_bfloat16*>(p.d) + m * p.ldd + col;
      if (col + 4 <= p.N) {
        if (p.out_f32)
          *reinterpret_cast<float4*>(df) = make_float4(out[0], out[1], out[2], out[3]);
        else
          *reinterpret_cast<uint2*>(db) = make_uint2(pack_bf16x2(out[0], out[1]), pack_bf16x2(out[2], out[3]));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (col + j < p.N) {
            if (p.out_f32)
              df[j] = out[j];
            else
              db[j] = __float2bfloat16_rn(out[j]);
          }
        }
      }
    }
  }
  if (splits > 1) cluster_sync();        // no CTA leaves while its partials are read
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

namespace {

bool encode_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t inner, int64_t outer,
                int64_t pitch_bytes, int box_inner, int box_outer, CUtensorMapSwizzle swizzle,
                CUtensorMapL2promotion promotion) {
  auto encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch_bytes)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_inner), static_cast<cuuint32_t>(box_outer)};
  const cuuint32_t estr[2] = {1, 1};
  return encode(map, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                swizzle, promotion, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Codes [rows][k/2 bytes], boxes of 128 bytes x box_rows in the 128-byte swizzle.
bool codes_map(CUtensorMap* map, const uint8_t* q, int64_t rows, int64_t k, int box_rows) {
  return encode_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, q, k / 2, rows, k / 2, 128, box_rows,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// Scale atoms [rows/128][atoms][512 bytes] as 8-byte words; a box is one stage's atoms of row_blocks blocks.
bool scales_map(CUtensorMap* map, const uint8_t* s, int64_t rows, int64_t k, bool nv, int row_blocks) {
  const int64_t atoms = nv ? (k + 63) / 64 : (k + 127) / 128;
  return encode_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT64, s, atoms * 64, (rows + 127) / 128, atoms * kMx4AtomBytes,
                    (nv ? 4 : 2) * 64, row_blocks, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// The output, boxes of 32 rows x 128 bytes in the 128-byte swizzle.
bool mx_out_map(CUtensorMap* map, const Mx4GemmArgs& g) {
  const int size = g.out_f32 ? 4 : 2;
  return encode_map(map, g.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g.d, g.N, g.M,
                    g.ldd * size, 128 / size, 32, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

Mx4Params mx_params(const Mx4GemmArgs& g, int64_t num_mb) {
  Mx4Params p{g.M, g.N, g.K, g.tsa, g.tsb, g.d, g.ldd, g.out_f32, 0, g.timeout_ns, g.err, g.inject_stall};
  p.group_m = static_cast<int>(num_mb < 8 ? num_mb : (g.group_m > 0 ? g.group_m : 8));
  return p;
}

template <bool kNv>
cudaError_t launch_mx4(const Mx4GemmArgs& g, cudaStream_t stream) {
  static PerContext<int> smem_set;
  constexpr int kSmem = mx_smem_bytes<kNv>();
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
  if (cudaError_t e = set_smem_once(smem_set, gemm_mx4_kernel<kNv>, kSmem); e != cudaSuccess) return e;
  CUtensorMap ta, tb, tsa, tsb, td;
  if (!codes_map(&ta, g.a, g.M, g.K, 128) || !codes_map(&tb, g.b, g.N, g.K, kBN) ||
      !scales_map(&tsa, g.sa, g.M, g.K, kNv, 1) || !scales_map(&tsb, g.sb, g.N, g.K, kNv, 1) || !mx_out_map(&td, g))
    return cudaErrorInvalidValue;
  const int64_t num_mb = (g.M + 127) / 128, num_nb = (g.N + kBN - 1) / kBN;
  const Mx4Params p = mx_params(g, num_mb);
  int64_t ctas = num_sms();
  if (g.max_ctas > 0 && g.max_ctas < ctas) ctas = g.max_ctas;
  if (num_mb * num_nb < ctas) ctas = num_mb * num_nb;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
  cfg.blockDim = dim3(kMxThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  cfg.numAttrs = set_pdl_attr(attr, g.pdl);
  cfg.attrs = attr;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, gemm_mx4_kernel<kNv>, ta, tb, tsa, tsb, td, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int BN, bool kNv, bool kQuant>
cudaError_t launch_mx4_few(const Mx4GemmArgs& g, const FewInput& in, cudaStream_t stream) {
  static PerContext<int> smem_set;
  constexpr int kSmem = few_smem_bytes<BN, kNv>();
  if (cudaError_t e = set_smem_once(smem_set, gemm_mx4_few_kernel<BN, kNv, kQuant>, kSmem); e != cudaSuccess) return e;
  CUtensorMap ta, tb, tsa, tsb;
  if (!codes_map(&tb, g.b, g.N, g.K, 128) || !scales_map(&tsb, g.sb, g.N, g.K, kNv, 1)) return cudaErrorInvalidValue;
  if constexpr (kQuant) {
    ta = tb;                             // not used
    tsa = tsb;
  } else if (!codes_map(&ta, g.a, g.M, g.K, BN) || !scales_map(&tsa, g.sa, g.M, g.K, kNv, 1)) {
    return cudaErrorInvalidValue;
  }
  const int64_t tiles = (g.N + 127) / 128, kblocks = (g.K + kStageK - 1) / kStageK;
  // As many CTAs as the SMs hold (two each), every one with at least two stages.
  int splits = 1;
  while (splits < 8 && 2 * splits * tiles <= 2 * num_sms() && kblocks >= 4 * splits) splits *= 2;
  // It is not persistent: a cap on the CTAs is kept by the 1-CTA kernel.
  if constexpr (!kQuant) {
    if (g.max_ctas > 0 && tiles * splits > g.max_ctas) return launch_mx4<kNv>(g, stream);
  }
  const Mx4Params p = mx_params(g, 1);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * splits), 1, 1);
  cfg.blockDim = dim3(kMxThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1 + set_pdl_attr(attr + 1, g.pdl);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, gemm_mx4_few_kernel<BN, kNv, kQuant>, ta, tb, tsa, tsb, p, splits, in);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool kNv>
cudaError_t launch_mx4_pair(const Mx4GemmArgs& g, cudaStream_t stream) {
  static PerContext<int> smem_set;
  using C = MxPairCfg<kNv>;
  if (cudaError_t e = set_smem_once(smem_set, gemm_mx4_pair_kernel<kNv>, C::kSmem); e != cudaSuccess) return e;
  CUtensorMap ta, tb, tsa, tsb, td;
  if (!codes_map(&ta, g.a, g.M, g.K, 128) || !codes_map(&tb, g.b, g.N, g.K, 128) ||
      !scales_map(&tsa, g.sa, g.M, g.K, kNv, 1) || !scales_map(&tsb, g.sb, g.N, g.K, kNv, 2) || !mx_out_map(&td, g))
    return cudaErrorInvalidValue;
  const int64_t num_mb = (g.M + 255) / 256, tiles = num_mb * ((g.N + 255) / 256);
  const Mx4Params p = mx_params(g, num_mb);
  int64_t pairs = num_sms() / 2;
  if (g.max_ctas > 1 && g.max_ctas / 2 < pairs) pairs = g.max_ctas / 2;
  if (tiles < pairs) pairs = tiles;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs), 1, 1);
  cfg.blockDim = dim3(kMxPairThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1 + set_pdl_attr(attr + 1, g.pdl);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, gemm_mx4_pair_kernel<kNv>, ta, tb, tsa, tsb, td, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool kNv>
cudaError_t launch_mx4_fmt(const Mx4GemmArgs& g, cudaStream_t stream) {
  // Up to 64 rows: 17920 x 8960 NVFP4 with 16 rows 14.5 us (128 x 128 tiles: 24.8), with 64 rows 17.5 (22.0); 8960 x
  // 4096 with 64 rows 10.2 (11.5).
  if (g.M <= 16) return launch_mx4_few<16, kNv, false>(g, {}, stream);
  if (g.M <= 32) return launch_mx4_few<32, kNv, false>(g, {}, stream);
  if (g.M <= 64) return launch_mx4_few<64, kNv, false>(g, {}, stream);
  const int64_t pair_tiles = ((g.M + 255) / 256) * ((g.N + 255) / 256);
  // Pairs once there is a tile for every pair of SMs (alone; 16384 x 17920 x 1536 NVFP4: 234 to 238 us, in 128 x 128
  // tiles 396 us; 1536 x 8960 x 16384 MXFP4: 92 to 94 us and 187 us).
  if (pair_tiles >= num_sms() / 2 && g.max_ctas != 1) return launch_mx4_pair<kNv>(g, stream);
  return launch_mx4<kNv>(g, stream);
}

}  // namespace

// Few rows: 1 x 1536 x 8960 9.7 us for the two launches, 7.3 us in one; 16 x 17920 x
// 8960 the same either way.
bool mx4_quantizes_on_the_way(int64_t M) { return M <= 16; }

cudaError_t launch_linear_mx4(const Mx4GemmArgs& g, const uint16_t* x, int64_t ldx, cudaStream_t stream) {
  const FewInput in{x, ldx};
  return g.nv ? launch_mx4_few<16, true, true>(g, in, stream) : launch_mx4_few<16, false, true>(g, in, stream);
}

cudaError_t launch_gemm_mx4(const Mx4GemmArgs& g, cudaStream_t stream) {
  return g.nv ? launch_mx4_fmt<true>(g, stream) : launch_mx4_fmt<false>(g, stream);
}

}  // namespace fp8blk
