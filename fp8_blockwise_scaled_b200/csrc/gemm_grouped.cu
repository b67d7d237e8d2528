// Blockwise-scaled GEMMs of a layer with one weight per group (expert), over
// rows sorted by group.  With T rows, group e owning rows off[e] .. off[e+1]-1:
//
//   FWD    D[t][n]    = sum_k A[t][k] W_e[n][k]        (t a row of group e)
//   DGRAD  D[t][k]    = sum_n A[t][n] W_e[n][k]
//   WGRAD  D[e][n][k] = sum over the rows t of e  A[n][t] B[k][t]
//
// with the operands, the per-128-block scales and the promotion of
// gemm.cu: per K-block the tensor cores make one fp32 partial product, scaled
// into fp32 running sums in registers, rounded once.
//
// The kernel has gemm_blockwise_kernel's roles (two operand producers, MMA
// issuer, scale producer, eight promotion warps, one persistent CTA per SM)
// and differs in its tiles, which the host cannot know:
//   - every CTA builds the groups' 128-row block counts from the offsets; tile u is looked up in them (a step or a binary search);
//   - FWD / DGRAD tiles start at a group's own rows.  The TMA load of A takes
//     any first row and may bring rows of the next group or, behind the last
//     row, zeros; those rows are computed and not stored.  The rows' scales are
//     not 16-byte aligned there, so they come by 4-byte cp.async into the
//     scale ring instead of by bulk copies;
//   - WGRAD tiles run over their group's own 128-token blocks (the quantiser
//     pads each group to whole blocks with zero codes) and write zeros for a
//     group without rows.
// A tile of whole 32-row quarters leaves by TMA stores as in gemm.cu; a quarter
// that the group's last row cuts is stored row by row.
#include <cudaTypedefs.h>

#include "gemm_device.cuh"
#include "gemm_host.h"
#include "groups.cuh"
#include "kernels.h"
#include "qmath.cuh"

namespace fp8blk {

namespace {

struct GroupedParams {
  const int* offsets;
  int groups;
  int rows;               // T
  int n;                  // columns of the output (of each group's output for WGRAD)
  int m;                  // WGRAD: rows of each group's output
  int kblocks;            // FWD / DGRAD: K-blocks of the contraction;  WGRAD: blocks of all padded rows
  int b_step_x, b_step_y; // B coordinates advance by these from group to group
  int sb_step;            // FWD / DGRAD: scales of B advance by this from group to group ...
  int sb_row;             // ... and by this from one block of 128 output columns to the next
  int b_rows;             // WGRAD: rows of B (pitch of its scales)
  const float* sa;
  const float* sb;
  void* d;
  int64_t ldd;
  int out_f32;
  uint64_t timeout_ns;
  unsigned int* err;
  int inject_stall;
  int group_m;
  uint32_t fmt_bits;
};

// Where tile u is: its group, its rows and columns in the operands and in the
// output, its K-blocks and the number of its rows that are stored.
struct GroupedTile {
  int e;
  int a_row, out_col, valid;
  int64_t out_row;
  int kb0, kb1;
};

// Finds tile u (tiles in group order; within a group as tile_coords orders
// them).  e: the group of this role's previous tile.
template <int BN, bool kWgrad>
__device__ __forceinline__ GroupedTile grouped_tile(const GroupedParams& p, const int* ends, int u, int& e) {
  const int num_nb = p.n / BN;
  GroupedTile w;
  int mb, nb;
  if constexpr (kWgrad) {
    const int num_mb = p.m / BM, per_group = num_mb * num_nb;
    e = u / per_group;
    tile_coords(u - e * per_group, num_mb, num_nb, p.group_m, mb, nb);
    w.a_row = mb * BM;
    w.out_row = static_cast<int64_t>(e) * p.m + w.a_row;
    w.valid = BM;
    w.kb1 = min(ends[e], p.kblocks);
    w.kb0 = min(e ? ends[e - 1] : 0, w.kb1);
  } else {
    e = find_group(ends, p.groups, u / num_nb, e);
    const int first = e ? ends[e - 1] : 0, num_mb = ends[e] - first;
    tile_coords(u - first * num_nb, num_mb, num_nb, min(p.group_m, num_mb), mb, nb);
    int size;
    w.a_row = group_rows(p.offsets, e, p.rows, &size) + mb * BM;
    w.out_row = w.a_row;
    w.valid = min(size - mb * BM, BM);
    w.kb0 = 0;
    w.kb1 = p.kblocks;
  }
  w.e = e;
  w.out_col = nb * BN;
  return w;
}

// The number of K-blocks of tile u alone (what the promotion needs before its loop).
template <int BN, bool kWgrad>
__device__ __forceinline__ int grouped_kblocks(const GroupedParams& p, const int* ends, int u) {
  if constexpr (!kWgrad) return p.kblocks;
  const int e = u / ((p.m / BM) * (p.n / BN));
  const int kb1 = min(ends[e], p.kblocks);
  return kb1 - min(e ? ends[e - 1] : 0, kb1);
}

__device__ __forceinline__ void cp_async4(void* smem_dst, const void* gsrc, bool real) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(smem_dst)), "l"(gsrc), "r"(real ? 4 : 0)
               : "memory");
}

// Arrives once on `bar` (one of its expected arrivals) when this thread's cp.async so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Register split of the warpgroups (as kLowRegs and kHighRegs).  With 256-column
// tiles of rows the scale producer needs more than 80 registers and the promotion
// no more than 200: 88 / 200 spills nothing, 80 / 208 does (65536 x 8960 x 1536 over
// 8 groups: 8% more time).
template <int BN, bool kWgrad>
struct RegSplit {
  static constexpr int kLow = BN == 256 && !kWgrad ? 88 : kLowRegs;
  static constexpr int kHigh = BN == 256 && !kWgrad ? 200 : kHighRegs;
  static_assert(128 * kLow + 256 * kHigh <= kThreads * 168, "register split exceeds the launch allocation");
};

// Where the promotion warps store a tile, published by the scale producer with
// the tile's first scales (they have no registers left to find it).  The scale producer is at most kSRing
// K-blocks, so at most kSRing tiles, ahead of the slowest promotion warp.
struct TilePlace {
  int row, col, valid;
};
constexpr int kPlaces = 16;
static_assert(kPlaces > kSRing + 1, "a place is rewritten only after every promotion warp has left its tile");

template <int BN>
constexpr int grouped_smem_bytes() {
  return smem_bytes<BN, false>() + kPlaces * static_cast<int>(sizeof(TilePlace)) + kMaxGroups * 4;
}
static_assert(grouped_smem_bytes<256>() <= 227 * 1024 && grouped_smem_bytes<128>() <= 227 * 1024,
              "shared memory per CTA");

}  // namespace

template <int BN, bool kWgrad>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_grouped_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                        const __grid_constant__ CUtensorMap tm_d, const GroupedParams p) {
  using C = Cfg<BN>;
  constexpr int kCols = BN / 2;   // columns per promotion warp
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* smem_out = smem + C::kStages * C::kStageBytes;
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem_out + C::kOutBytes);
  TilePlace* places = reinterpret_cast<TilePlace*>(ctrl + 1);
  int* ends = reinterpret_cast<int*>(places + kPlaces);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&ctrl->full[s], 1);
      mbar_init(&ctrl->empty[s], 1);
    }
    for (int b = 0; b < C::kAccBufs; ++b) {
      mbar_init(&ctrl->tfull[b], 1);
      mbar_init(&ctrl->tempty[b], kPromoWarps);
    }
    for (int s = 0; s < kSRing; ++s) {
      // WGRAD: the scale producer's arrive + the bytes of its copies;  FWD / DGRAD: an arrive of
      // every lane once its copies have landed, and one for the B scales.
      mbar_init(&ctrl->sfull[s], kWgrad ? 1 : 33);
      mbar_init(&ctrl->sempty[s], kPromoWarps);
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
  griddep_wait();   // the offsets may come from the previous kernel
  build_block_ends(ends, nullptr, p.offsets, p.groups, p.rows, threadIdx.x, kThreads);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const uint32_t tmem_base = ctrl->tmem_base;
  volatile int* abort = &ctrl->abort;
  const int tiles = kWgrad ? p.groups * (p.m / BM) * (p.n / BN) : ends[p.groups - 1] * (p.n / BN);

  if (warp < kPromoWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(RegSplit<BN, kWgrad>::kLow));
    if (warp == 0 || warp == kBWarp) {
      // ---------------------------------------------------------- operand producers (A: warp 0, B: warp 3)
      const bool is_a = warp == 0;
      if (lane == 0) {
        tma_prefetch_map(is_a ? &tm_a : &tm_b);
        Ring<C::kStages> st;
        int64_t issued = 0;
        bool ok = true;
        int e = 0;
        for (int u = blockIdx.x; ok && u < tiles; u += gridDim.x) {
          const GroupedTile w = grouped_tile<BN, kWgrad>(p, ends, u, e);
          const int bx = kWgrad ? 0 : w.e * p.b_step_x, by = w.out_col + (kWgrad ? 0 : w.e * p.b_step_y);
          for (int kb = w.kb0; kb < w.kb1; ++kb) {
            if (!mbar_wait_bounded(&ctrl->empty[st.idx], st.phase ^ 1u, abort, p.timeout_ns, p.err)) {
              ok = false;
              break;
            }
            uint8_t* stage = smem + st.idx * C::kStageBytes;
            if (is_a) {
              mbar_arrive_expect_tx(&ctrl->full[st.idx], C::kStageBytes);
              tma_load_2d(stage, &tm_a, &ctrl->full[st.idx], kb * BK, w.a_row);
            } else {
              tma_load_2d(stage + C::kABytes, &tm_b, &ctrl->full[st.idx], bx + kb * BK, by);
            }
            ++issued;
            st.next();
          }
        }
        // Let the copies still in flight land before the CTA's smem goes away.
        const int64_t first = issued > C::kStages ? issued - C::kStages : 0;
        for (int64_t j = first; j < issued; ++j)
          mbar_wait_bounded(&ctrl->full[j % C::kStages], static_cast<uint32_t>((j / C::kStages) & 1), nullptr,
                            p.timeout_ns, p.err);
      }
    } else if (warp == kScaleWarp) {
      // ---------------------------------------------------------- scale producer (whole warp)
      Ring<kSRing> ring;
      int64_t issued = 0;
      bool ok = true;
      int e = 0;
      [[maybe_unused]] float sb0 = 0.0f, sb1 = 0.0f;   // FWD/DGRAD: B scales of K-blocks 32 i + lane
      int n = 0;
      for (int u = blockIdx.x; ok && u < tiles; u += gridDim.x, ++n) {
        const GroupedTile w = grouped_tile<BN, kWgrad>(p, ends, u, e);
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if constexpr (!kWgrad) {
            if ((kb & 31) == 0) {
              const int k = kb + lane;
              const float* row = p.sb + static_cast<int64_t>(w.e) * p.sb_step +
                                 static_cast<int64_t>(w.out_col / 128) * p.sb_row;
              sb0 = k < w.kb1 ? __ldg(row + k) : 0.0f;
              if constexpr (BN == 256) sb1 = k < w.kb1 ? __ldg(row + p.sb_row + k) : 0.0f;
            }
          }
          if (!__all_sync(0xFFFFFFFFu,
                          mbar_wait_bounded(&ctrl->sempty[ring.idx], ring.phase ^ 1u, abort, p.timeout_ns, p.err))) {
            ok = false;
            break;
          }
          ScaleSlot& ss = ctrl->slots[ring.idx];
          uint64_t* full = &ctrl->sfull[ring.idx];
          if constexpr (!kWgrad) {
            const float* src = p.sa + static_cast<int64_t>(kb) * p.rows + w.a_row;
#pragma unroll
            for (int i = 0; i < BM / 32; ++i) {
              const int r = i * 32 + lane;
              cp_async4(&ss.sa[r], src + (r < w.valid ? r : 0), r < w.valid);
            }
            cp_async_arrive(full);
            const float v0 = __shfl_sync(0xFFFFFFFFu, sb0, kb & 31);
            const float v1 = __shfl_sync(0xFFFFFFFFu, sb1, kb & 31);
            if (lane == 0) {
              ss.sb[0] = v0;
              if constexpr (BN == 256) ss.sb[1] = v1;
              if (kb == 0) places[n % kPlaces] = TilePlace{w.a_row, w.out_col, w.valid};
              mbar_arrive(full);                         // releases the stores above
            }
          } else if (lane == 0) {
            // The promotion warps read this slot through the generic proxy; the
            // bulk copies below write it through the async proxy: order them.
            fence_proxy_async_shared();
            mbar_arrive_expect_tx(full, (BM + BN) * 4);
            bulk_load(ss.sa, p.sa + static_cast<int64_t>(kb) * p.m + w.a_row, BM * 4, full);
            bulk_load(ss.sb, p.sb + static_cast<int64_t>(kb) * p.b_rows + w.out_col, BN * 4, full);
          }
          ++issued;
          ring.next();
        }
      }
      for (int64_t j = issued > kSRing ? issued - kSRing : 0; j < issued; ++j)
        mbar_wait_bounded(&ctrl->sfull[j % kSRing], static_cast<uint32_t>((j / kSRing) & 1), nullptr, p.timeout_ns,
                          p.err);
    } else {
      // ---------------------------------------------------------- MMA issuer (warp 1)
      const bool leader = elect_one();
      const uint32_t idesc = idesc_e4m3_f32(BM, BN) | p.fmt_bits;
      const uint32_t smem0 = smem_addr(smem);
      Ring<C::kStages> st;
      Ring<C::kAccBufs> acc;
      bool ok = true;
      if (p.inject_stall) ok = mbar_wait_bounded(&ctrl->never, 0, abort, p.timeout_ns, p.err);
      ok = __all_sync(0xFFFFFFFFu, ok);
      for (int u = blockIdx.x; ok && u < tiles; u += gridDim.x) {
        const int kblocks = grouped_kblocks<BN, kWgrad>(p, ends, u);
        for (int kb = 0; kb < kblocks; ++kb) {
          const bool got =
              mbar_wait_hot(&ctrl->full[st.idx], st.phase, abort, 0, p.timeout_ns, p.err) &&
              mbar_wait_hot(&ctrl->tempty[acc.idx], acc.phase ^ 1u, abort, 0, p.timeout_ns, p.err);
          if (!__all_sync(0xFFFFFFFFu, got)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t a_addr = smem0 + st.idx * C::kStageBytes;
          const uint64_t adesc = smem_desc_kmajor_sw128(a_addr);
          const uint64_t bdesc = smem_desc_kmajor_sw128(a_addr + C::kABytes);
          const uint32_t d_tmem = tmem_base + acc.idx * BN;
          if (leader) {
            umma_e4m3(d_tmem, adesc, bdesc, idesc, 0u);
#pragma unroll
            for (int k = 1; k < BK / 32; ++k)
              umma_e4m3(d_tmem, adesc + 2 * k, bdesc + 2 * k, idesc, 1u);
            umma_commit(&ctrl->empty[st.idx]);
            umma_commit(&ctrl->tfull[acc.idx]);
          }
          __syncwarp();
          st.next();
          acc.next();
        }
      }
      if (leader) umma_commit(&ctrl->mma_done);
      __syncwarp();
      mbar_wait_bounded(&ctrl->mma_done, 0, nullptr, p.timeout_ns, p.err);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(RegSplit<BN, kWgrad>::kHigh));
    // ------------------------------------------------------------ promotion + epilogue
    const int ew = warp - kPromoWarp0;  // 0 .. 7
    const int wg = ew >> 2;             // which half of the tile's columns
    const int quarter = warp & 3;       // TMEM lanes this warp may read
    const int row = quarter * 32 + lane;
    const int col0 = wg * kCols;
    const uint32_t tmem_lanes = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + col0;
    Ring<C::kAccBufs> tbuf;
    Ring<kSRing> sring;
    float2 acc[BN / 4];
    int e = 0;
    auto release = [&](int b) {
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctrl->tempty[b]);
    };
    // Read from shared memory in every round, so that no register holds it over the K loop.
    auto num_tiles = [&]() {
      if constexpr (kWgrad) return tiles;
      int blocks;
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(blocks) : "r"(smem_addr(ends + p.groups - 1)) : "memory");
      return blocks * (p.n / BN);
    };
    for (int u = blockIdx.x; u < num_tiles(); u += gridDim.x) {
      if (!promote_tile<BN, kWgrad>(ctrl, p, acc, grouped_kblocks<BN, kWgrad>(p, ends, u), tmem_lanes, row, col0, tbuf,
                                    sring, abort, lane, release))
        break;
      GroupedTile w;
      if constexpr (kWgrad) {
        w = grouped_tile<BN, kWgrad>(p, ends, u, e);
      } else {
        const TilePlace at = places[(u / gridDim.x) % kPlaces];
        w.out_row = at.row;
        w.out_col = at.col;
        w.valid = at.valid;
      }
      const int64_t off = (w.out_row + row) * p.ldd + w.out_col + col0;
      if (p.out_f32) {
        if (kWgrad || row < w.valid) store_row_f32<kCols>(static_cast<float*>(p.d) + off, acc);
      } else if constexpr (!C::kStagedOut) {
        if (kWgrad || row < w.valid) store_row_bf16<kCols>(static_cast<uint16_t*>(p.d) + off, acc);
      } else {
        // As in gemm_blockwise_kernel: the warp's 32 rows x kCols columns in the
        // 128-byte swizzle of the output map, then TMA stores by one lane; or, of a
        // quarter that the group's last row cuts, its rows by the warp.
        uint8_t* stg = smem_out + ew * (32 * kCols * 2);
        if (lane == 0) bulk_wait_group_read0();   // the last tile's stores have read the staging area
        __syncwarp();
#pragma unroll
        for (int b = 0; b < kCols / 64; ++b) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2* a = acc + b * 32 + j * 4;
            *reinterpret_cast<uint4*>(stg + b * 4096 + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                make_uint4(pack_bf16x2(a[0].x, a[0].y), pack_bf16x2(a[1].x, a[1].y), pack_bf16x2(a[2].x, a[2].y),
                           pack_bf16x2(a[3].x, a[3].y));
          }
        }
        if (kWgrad || quarter * 32 + 32 <= w.valid) {
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) {
#pragma unroll
            for (int b = 0; b < kCols / 64; ++b)
              tma_store_2d(&tm_d, stg + b * 4096, w.out_col + col0 + b * 64, static_cast<int>(w.out_row) + quarter * 32);
            bulk_commit_group();
          }
        } else {
          __syncwarp();
          const int chunk = lane & 15, box = chunk >> 3;       // 16 bytes of a row: two rows a step
          for (int r = lane >> 4; r < w.valid - quarter * 32; r += 2)
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.d) + (w.out_row + quarter * 32 + r) * p.ldd + w.out_col +
                                      col0 + chunk * 8) =
                *reinterpret_cast<const uint4*>(stg + box * 4096 + r * 128 + (((chunk & 7) ^ (r & 7)) << 4));
          __syncwarp();
        }
      }
    }
    if constexpr (C::kStagedOut) {
      if (lane == 0) bulk_wait_group0();
    }
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
// Few rows a group (decoding).  The work is one read of the weights of the
// groups that have rows, so the operands' roles are exchanged: 128 rows of the
// weight (output columns) are the MMA's M side and 16 rows of A its N side.  A
// K-block then brings 16 KB of weight and only 2 KB of rows into the SM, and the
// promotion folds 16 columns, not 128 or 256, into registers (one output column a
// thread: acc[t] += P[n][t] * (sa[t] * sb)).  Two persistent CTAs per SM keep 180 KB
// of loads in flight per SM and fill the SMs when there are few tiles.  A group
// with more than 16 rows takes several tiles of the same weight next to each
// other, which L2 serves.
//
// kQuant: A is bf16 x, quantised on the way by four more warps: per K-block 128
// threads take 16 values each, reduce a row's 128 over eight lanes, and write the
// codes in the stage's swizzled layout and the scales into the scale ring, where
// TMA and cp.async would have put them.  Every column block of a tile's rows does
// that again, for 4 KB a K-block from L2; a launch and a round trip of codes
// through memory are saved.
namespace {

constexpr int kFewThreads = 256;
constexpr int kFewQuantThreads = 384;    // with the warps that quantise
constexpr int kFewWarps = 4;             // promotion warps
constexpr int kFewRows = 16;             // rows of A in a tile

struct FewCfg {
  static constexpr int kABytes = 128 * BK;                // weight rows
  static constexpr int kBBytes = kFewRows * BK;           // rows of A
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = 5;
  static constexpr int kAccBufs = 4;
  static constexpr int kTmemCols = kAccBufs * kFewRows;
};

struct FewSlot {
  float sa[kFewRows];
  float sb;
  float pad[3];
};

struct FewCtrl {
  uint64_t full[8], empty[8];
  uint64_t tfull[4], tempty[4];
  uint64_t sfull[kSRing], sempty[kSRing];
  uint64_t mma_done, never;
  uint32_t tmem_base;
  int abort;
  alignas(16) FewSlot slots[kSRing];
};

constexpr int kFewSmem =
    1024 + FewCfg::kStages * FewCfg::kStageBytes + static_cast<int>(sizeof(FewCtrl)) + kMaxGroups * 4;
static_assert(2 * (kFewSmem + 1024) <= 227 * 1024, "two CTAs per SM");

struct FewTile {
  int e, row, col, valid;
};

// x of a product that quantises on the way.
struct FewInput {
  const uint16_t* x;
  int64_t ldx;
};

__device__ __forceinline__ FewTile few_tile(const GroupedParams& p, const int* ends, int u, int& e) {
  const int num_nb = p.n / 128;
  e = find_group(ends, p.groups, u / num_nb, e);
  const int first = e ? ends[e - 1] : 0, blocks = ends[e] - first, local = u - first * num_nb;
  const int nb = local / blocks, tb = local - nb * blocks;
  FewTile w;
  int size;
  w.e = e;
  w.row = group_rows(p.offsets, e, p.rows, &size) + tb * kFewRows;
  w.col = nb * 128;
  w.valid = min(size - tb * kFewRows, kFewRows);
  return w;
}

}  // namespace

template <bool kQuant>
__global__ void __launch_bounds__(kQuant ? kFewQuantThreads : kFewThreads, 2)
    gemm_grouped_few_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                            const GroupedParams p, const FewInput in) {
  using C = FewCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  FewCtrl* ctrl = reinterpret_cast<FewCtrl*>(smem + C::kStages * C::kStageBytes);
  int* ends = reinterpret_cast<int*>(ctrl + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&ctrl->full[s], kQuant ? 5 : 1);   // the producer, and the warps that quantise
      mbar_init(&ctrl->empty[s], 1);
    }
    for (int b = 0; b < C::kAccBufs; ++b) {
      mbar_init(&ctrl->tfull[b], 1);
      mbar_init(&ctrl->tempty[b], kFewWarps);
    }
    for (int s = 0; s < kSRing; ++s) {
      mbar_init(&ctrl->sfull[s], kQuant ? 5 : 33);   // the warps that quantise (every lane's copies), and the B scale
      mbar_init(&ctrl->sempty[s], kFewWarps);
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
  griddep_wait();
  build_block_ends(ends, nullptr, p.offsets, p.groups, p.rows, threadIdx.x, kQuant ? kFewQuantThreads : kFewThreads,
                   kFewRows);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const uint32_t tmem_base = ctrl->tmem_base;
  volatile int* abort = &ctrl->abort;
  const int tiles = ends[p.groups - 1] * (p.n / 128);
  int e = 0;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_map(&tm_a);
      tma_prefetch_map(&tm_b);
      Ring<C::kStages> st;
      int64_t issued = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < tiles; u += gridDim.x) {
        const FewTile w = few_tile(p, ends, u, e);
        const int bx = w.e * p.b_step_x, by = w.col + w.e * p.b_step_y;
        for (int kb = 0; kb < p.kblocks; ++kb) {
          if (!mbar_wait_bounded(&ctrl->empty[st.idx], st.phase ^ 1u, abort, p.timeout_ns, p.err)) {
            ok = false;
            break;
          }
          uint8_t* stage = smem + st.idx * C::kStageBytes;
          mbar_arrive_expect_tx(&ctrl->full[st.idx], kQuant ? C::kABytes : C::kStageBytes);
          tma_load_2d(stage, &tm_b, &ctrl->full[st.idx], bx + kb * BK, by);
          if constexpr (!kQuant) tma_load_2d(stage + C::kABytes, &tm_a, &ctrl->full[st.idx], kb * BK, w.row);
          ++issued;
          st.next();
        }
      }
      const int64_t first = issued > C::kStages ? issued - C::kStages : 0;
      for (int64_t j = first; j < issued; ++j)
        mbar_wait_bounded(&ctrl->full[j % C::kStages], static_cast<uint32_t>((j / C::kStages) & 1), nullptr,
                          p.timeout_ns, p.err);
    }
  } else if (warp == kScaleWarp) {
    // ------------------------------------------------------------ scale producer (whole warp)
    Ring<kSRing> ring;
    int64_t issued = 0;
    bool ok = true;
    float sb0 = 0.0f;                    // B scales of K-blocks 32 i + lane
    for (int u = blockIdx.x; ok && u < tiles; u += gridDim.x) {
      const FewTile w = few_tile(p, ends, u, e);
      const float* row = p.sb + static_cast<int64_t>(w.e) * p.sb_step + static_cast<int64_t>(w.col / 128) * p.sb_row;
      for (int kb = 0; kb < p.kblocks; ++kb) {
        if ((kb & 31) == 0) sb0 = kb + lane < p.kblocks ? __ldg(row + kb + lane) : 0.0f;
        if (!__all_sync(0xFFFFFFFFu,
                        mbar_wait_bounded(&ctrl->sempty[ring.idx], ring.phase ^ 1u, abort, p.timeout_ns, p.err))) {
          ok = false;
          break;
        }
        FewSlot& ss = ctrl->slots[ring.idx];
        uint64_t* full = &ctrl->sfull[ring.idx];
        if constexpr (!kQuant) {
          const float* src = p.sa + static_cast<int64_t>(kb) * p.rows + w.row;
          if (lane < kFewRows) cp_async4(&ss.sa[lane], src + (lane < w.valid ? lane : 0), lane < w.valid);
          cp_async_arrive(full);
        }
        const float v = __shfl_sync(0xFFFFFFFFu, sb0, kb & 31);
        if (lane == 0) {
          ss.sb = v;
          mbar_arrive(full);
        }
        ++issued;
        ring.next();
      }
    }
    for (int64_t j = issued > kSRing ? issued - kSRing : 0; j < issued; ++j)
      mbar_wait_bounded(&ctrl->sfull[j % kSRing], static_cast<uint32_t>((j / kSRing) & 1), nullptr, p.timeout_ns, p.err);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = elect_one();
    const uint32_t idesc = idesc_e4m3_f32(128, kFewRows) | p.fmt_bits;
    const uint32_t smem0 = smem_addr(smem);
    Ring<C::kStages> st;
    Ring<C::kAccBufs> acc;
    bool ok = true;
    if (p.inject_stall) ok = mbar_wait_bounded(&ctrl->never, 0, abort, p.timeout_ns, p.err);
    ok = __all_sync(0xFFFFFFFFu, ok);
    for (int u = blockIdx.x; ok && u < tiles; u += gridDim.x) {
      for (int kb = 0; kb < p.kblocks; ++kb) {
        const bool got = mbar_wait_hot(&ctrl->full[st.idx], st.phase, abort, 0, p.timeout_ns, p.err) &&
                         mbar_wait_hot(&ctrl->tempty[acc.idx], acc.phase ^ 1u, abort, 0, p.timeout_ns, p.err);
        if (!__all_sync(0xFFFFFFFFu, got)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t a_addr = smem0 + st.idx * C::kStageBytes;
        const uint64_t adesc = smem_desc_kmajor_sw128(a_addr);
        const uint64_t bdesc = smem_desc_kmajor_sw128(a_addr + C::kABytes);
        const uint32_t d_tmem = tmem_base + acc.idx * kFewRows;
        if (leader) {
          umma_e4m3(d_tmem, adesc, bdesc, idesc, 0u);
#pragma unroll
          for (int k = 1; k < BK / 32; ++k) umma_e4m3(d_tmem, adesc + 2 * k, bdesc + 2 * k, idesc, 1u);
          umma_commit(&ctrl->empty[st.idx]);
          umma_commit(&ctrl->tfull[acc.idx]);
        }
        __syncwarp();
        st.next();
        acc.next();
      }
    }
    if (leader) umma_commit(&ctrl->mma_done);
    __syncwarp();
    mbar_wait_bounded(&ctrl->mma_done, 0, nullptr, p.timeout_ns, p.err);
  } else if (kQuant && warp >= 8) {
    // ------------------------------------------------------------ x to codes, in the stages' layout
    const int q = threadIdx.x - 256, row = q >> 3, part = q & 7;      // values 16 part .. of the K-block
    Ring<C::kStages> st;
    Ring<kSRing> ring;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < tiles; u += gridDim.x) {
      const FewTile w = few_tile(p, ends, u, e);
      const bool inside = row < w.valid;
      const uint4* src = reinterpret_cast<const uint4*>(in.x + (w.row + static_cast<int64_t>(inside ? row : 0)) * in.ldx +
                                                        16 * part);
      const uint4 zero = make_uint4(0, 0, 0, 0);
      uint4 v0 = inside ? __ldg(src) : zero, v1 = inside ? __ldg(src + 1) : zero;
      for (int kb = 0; kb < p.kblocks; ++kb) {
        const bool more = inside && kb + 1 < p.kblocks;               // in flight while this block becomes codes
        const uint4* ahead = src + 16 * (kb + 1);
        const uint4 n0 = more ? __ldg(ahead) : zero, n1 = more ? __ldg(ahead + 1) : zero;
        uint32_t m = __vmaxu2(__vmaxu2(__vmaxu2(v0.x & kAbs2, v0.y & kAbs2), __vmaxu2(v0.z & kAbs2, v0.w & kAbs2)),
                              __vmaxu2(__vmaxu2(v1.x & kAbs2, v1.y & kAbs2), __vmaxu2(v1.z & kAbs2, v1.w & kAbs2)));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const QScale s = make_qscale<false>(__uint_as_float(max(m << 16, m & 0xFFFF0000u)));
        float x[8];
        unpack8(v0, x);
        const uint2 c0 = quant8<false>(x, s);
        unpack8(v1, x);
        const uint2 c1 = quant8<false>(x, s);
        const bool got = mbar_wait_bounded(&ctrl->empty[st.idx], st.phase ^ 1u, abort, p.timeout_ns, p.err) &&
                         mbar_wait_bounded(&ctrl->sempty[ring.idx], ring.phase ^ 1u, abort, p.timeout_ns, p.err);
        if (!__all_sync(0xFFFFFFFFu, got)) {
          ok = false;
          break;
        }
        *reinterpret_cast<uint4*>(smem + st.idx * C::kStageBytes + C::kABytes + row * 128 + ((part ^ (row & 7)) << 4)) =
            make_uint4(c0.x, c0.y, c1.x, c1.y);
        if (part == 0) ctrl->slots[ring.idx].sa[row] = s.s;
        fence_proxy_async_shared();      // the codes above, then the tensor cores' reads
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&ctrl->full[st.idx]);
          mbar_arrive(&ctrl->sfull[ring.idx]);
        }
        st.next();
        ring.next();
        v0 = n0;
        v1 = n1;
      }
    }
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------ promotion + epilogue
    const int quarter = warp & 3;
    const uint32_t lanes = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    Ring<C::kAccBufs> tbuf;
    Ring<kSRing> sring;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < tiles; u += gridDim.x) {
      float2 acc[kFewRows / 2];
#pragma unroll
      for (int j = 0; j < kFewRows / 2; ++j) acc[j] = make_float2(0.0f, 0.0f);
      for (int kb = 0; kb < p.kblocks; ++kb) {
        const bool got = mbar_wait_bounded(&ctrl->sfull[sring.idx], sring.phase, abort, p.timeout_ns, p.err) &&
                         mbar_wait_bounded(&ctrl->tfull[tbuf.idx], tbuf.phase, abort, p.timeout_ns, p.err);
        if (!__all_sync(0xFFFFFFFFu, got)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const FewSlot& ss = ctrl->slots[sring.idx];
        const float2 sb = make_float2(ss.sb, ss.sb);
#pragma unroll
        for (int c = 0; c < kFewRows; c += 16) {
          uint32_t r[16];
          tmem_ld_32x32b_x16(lanes + tbuf.idx * kFewRows + c, r);
          tmem_wait_ld16(r);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 f = __fmul2_rn(*reinterpret_cast<const float2*>(&ss.sa[c + 2 * j]), sb);
            acc[c / 2 + j] = __ffma2_rn(make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), f,
                                        acc[c / 2 + j]);
          }
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&ctrl->tempty[tbuf.idx]);
          mbar_arrive(&ctrl->sempty[sring.idx]);
        }
        tbuf.next();
        sring.next();
      }
      if (!ok) break;
      const FewTile w = few_tile(p, ends, u, e);
      const int64_t at = static_cast<int64_t>(w.row) * p.ldd + w.col + quarter * 32 + lane;
#pragma unroll
      for (int t = 0; t < kFewRows; ++t) {
        if (t < w.valid) {
          const float v = t & 1 ? acc[t / 2].y : acc[t / 2].x;
          if (p.out_f32)
            static_cast<float*>(p.d)[at + t * p.ldd] = v;
          else
            static_cast<__nv_bfloat16*>(p.d)[at + t * p.ldd] = __float2bfloat16_rn(v);
        }
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

namespace {

GroupedParams grouped_params(const GroupedGemmArgs& g, int64_t contraction) {
  GroupedParams p{};
  p.offsets = g.offsets;
  p.groups = static_cast<int>(g.groups);
  p.rows = static_cast<int>(g.rows);
  p.n = static_cast<int>(g.n);
  p.m = static_cast<int>(g.m);
  p.kblocks = static_cast<int>(contraction / BK);
  p.b_step_x = g.layout == 1 ? static_cast<int>(g.k) : 0;
  p.b_step_y = g.layout == 0 ? static_cast<int>(g.n) : 0;
  p.sb_step = static_cast<int>(g.layout == 0 ? (g.n / 128) * (g.k / BK) : g.k / BK);
  p.sb_row = static_cast<int>(g.layout == 0 ? g.k / BK : g.groups * (g.k / BK));
  p.b_rows = static_cast<int>(g.n);
  p.sa = g.sa;
  p.sb = g.sb;
  p.d = g.d;
  p.ldd = g.ldd;
  p.out_f32 = g.out_f32;
  p.timeout_ns = g.timeout_ns;
  p.err = g.err;
  p.inject_stall = g.inject_stall;
  p.fmt_bits = (static_cast<uint32_t>(g.a_e5m2 != 0) << 7) | (static_cast<uint32_t>(g.b_e5m2 != 0) << 10);
  return p;
}

template <int BN, bool kWgrad>
cudaError_t launch_grouped(const GroupedGemmArgs& g, cudaStream_t stream) {
  static PerContext<int> smem_set;
  constexpr int kSmem = grouped_smem_bytes<BN>();
  if (cudaError_t e = set_smem_once(smem_set, gemm_grouped_kernel<BN, kWgrad>, kSmem); e != cudaSuccess) return e;
  const int64_t out_rows = kWgrad ? g.groups * g.m : g.rows;
  const int64_t a_rows = kWgrad ? g.m : g.rows;
  const int64_t contraction = kWgrad ? g.padded_rows : g.k;
  // B: FWD [groups * n][k], DGRAD [n][groups * k] (the transposed weights), WGRAD [n][padded rows].
  const int64_t b_rows = g.layout == 0 ? g.groups * g.n : g.n;
  const int64_t b_cols = g.layout == 1 ? g.groups * g.k : contraction;
  CUtensorMap ta, tb, td;
  const bool empty = contraction == 0;   // WGRAD of no rows: zeros, nothing is loaded (the maps only have to be valid)
  if (!make_map(&ta, empty ? g.d : g.a, a_rows, empty ? BK : contraction, BM) ||
      !make_map(&tb, empty ? g.d : g.b, b_rows, empty ? BK : b_cols, BN) ||
      !make_out_map(&td, g.d, out_rows, g.n, g.ldd, g.out_f32 != 0))
    return cudaErrorInvalidValue;
  GroupedParams p = grouped_params(g, contraction);
  p.group_m = g.group_m > 0 ? g.group_m : 8;
  if (kWgrad && p.group_m > g.m / BM) p.group_m = static_cast<int>(g.m / BM);
  // The number of tiles is known on the device only: at most this many.
  const int64_t blocks = kWgrad ? g.groups * (g.m / BM) : g.rows / BM + (g.groups < g.rows ? g.groups : g.rows);
  const int64_t most = blocks * (g.n / BN);
  int64_t ctas = num_sms();
  if (g.max_ctas > 0 && g.max_ctas < ctas) ctas = g.max_ctas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(most < ctas ? most : ctas), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  cfg.numAttrs = set_pdl_attr(attr, g.pdl);
  cfg.attrs = attr;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, gemm_grouped_kernel<BN, kWgrad>, ta, tb, td, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool kQuant>
cudaError_t launch_grouped_few(const GroupedGemmArgs& g, const FewInput& in, cudaStream_t stream) {
  static PerContext<int> smem_set;
  if (cudaError_t e = set_smem_once(smem_set, gemm_grouped_few_kernel<kQuant>, kFewSmem); e != cudaSuccess) return e;
  const int64_t b_rows = g.layout == 0 ? g.groups * g.n : g.n, b_cols = g.layout == 1 ? g.groups * g.k : g.k;
  CUtensorMap ta, tb;
  if (!make_map(&tb, g.b, b_rows, b_cols, 128)) return cudaErrorInvalidValue;
  if constexpr (kQuant) {
    ta = tb;                             // not used
  } else if (!make_map(&ta, g.a, g.rows, g.k, kFewRows)) {
    return cudaErrorInvalidValue;
  }
  GroupedParams p = grouped_params(g, g.k);
  // The operands' roles are exchanged: the rows' format is the MMA's B format.
  p.fmt_bits = (static_cast<uint32_t>(g.b_e5m2 != 0) << 7) | (static_cast<uint32_t>(g.a_e5m2 != 0) << 10);
  const int64_t most = (g.rows / kFewRows + (g.groups < g.rows ? g.groups : g.rows)) * (g.n / 128);
  int64_t ctas = 2 * static_cast<int64_t>(num_sms());
  if (g.max_ctas > 0 && g.max_ctas < ctas) ctas = g.max_ctas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(most < ctas ? most : ctas), 1, 1);
  cfg.blockDim = dim3(kQuant ? kFewQuantThreads : kFewThreads, 1, 1);
  cfg.dynamicSmemBytes = kFewSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  cfg.numAttrs = set_pdl_attr(attr, g.pdl);
  cfg.attrs = attr;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, gemm_grouped_few_kernel<kQuant>, ta, tb, p, in);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

namespace {

// Up to 12 rows a group on average go to gemm_grouped_few_kernel; measured with 64
// groups of 2560 x 1536: 8 rows 44.4 us against 50.5 us (128-row tiles), 12 rows 44.7
// to 47.8 us (evenly spread to skewed) against 50.7, 16 rows 50.3 to 51.2 against 50.9.
constexpr int64_t kFewRowsPerGroup = 12;

bool grouped_few_rows(const GroupedGemmArgs& g) {
  return g.layout != 2 && g.block_n == 0 && g.rows <= kFewRowsPerGroup * g.groups;
}

}  // namespace

// Up to 16 rows; then the codes cost more than the launch.  64 groups of 2560 x 1536:
// 8 rows 11.8 us against 12.8 us for the two launches, 16 rows 17.7 against 17.1,
// 64 rows 44.4 against 41.0 (the fence between the codes and the tensor cores' reads
// waits for the loads ahead of it, so every K-block waits for L2).
bool grouped_quantizes_on_the_way(int64_t rows, int64_t groups) { return rows <= 16 && rows <= kFewRowsPerGroup * groups; }

cudaError_t launch_linear_grouped(const GroupedGemmArgs& g, const uint16_t* x, int64_t ldx, cudaStream_t stream) {
  return launch_grouped_few<true>(g, FewInput{x, ldx}, stream);
}

cudaError_t launch_gemm_grouped(const GroupedGemmArgs& g, cudaStream_t stream) {
  const bool wgrad = g.layout == 2;
  if (grouped_few_rows(g)) return launch_grouped_few<false>(g, {}, stream);
  // 256-column tiles, unless even the most tiles that the rows can make leave SMs
  // idle (64 groups of 2560 x 1536, 1024 to 24576 rows: within 4% of 128-column
  // tiles while the weights' read bounds both, 12 to 15% faster from 12288 rows on).
  const int64_t most = (wgrad ? g.groups * (g.m / BM) : g.rows / BM + (g.groups < g.rows ? g.groups : g.rows)) * (g.n / 256);
  if (g.n % 256 != 0 || g.block_n == 128 || (g.block_n == 0 && most < num_sms()))
    return wgrad ? launch_grouped<128, true>(g, stream) : launch_grouped<128, false>(g, stream);
  return wgrad ? launch_grouped<256, true>(g, stream) : launch_grouped<256, false>(g, stream);
}

}  // namespace fp8blk
