// 4-bit microscaled quantisation (E2M1 codes, one scale for 32 or 16 values)
// and the values back in bf16.
//
//   MXFP4  scale = 2^clamp(floor(log2 amax) - 2, -127, 127), q = E2M1_RNE(clamp(x / scale, -6, 6))
//   NVFP4  sf = E4M3_RNE(min(fl32(fl32(amax / 6) / g), 448)), d = fl32(sf * g),
//          q = E2M1_RNE(clamp(fl32(x / d), -6, 6)), zeros where sf is zero
// with amax over the block and g the tensor's scale.  (The MXFP4 rule is the OCP
// Microscaling specification's; NVFP4's quotient x / d is reached exactly as
// qmath.cuh describes.)
//
// The quantiser walks 128 x 128 tiles: 128 columns are one (MXFP4) or two
// (NVFP4) scale atoms of 128 rows, so a tile owns whole atoms in both
// directions.  Persistent CTAs, two per SM, a ring of stages filled by TMA as in
// quant.cu; rows and columns behind the input arrive as zeros, which give zero
// codes and zero scales where the padded outputs need them.
//
// A warp covers 32 rows x 64 columns, a thread 8 x 8 of them: row blocks are 2
// or 4 neighbouring lanes, column blocks (the transposed direction) lanes 8 or
// 8 and 16 apart, so every block maximum is one or two shuffles and no warp
// waits for another before the outputs are staged: the scale bytes in the
// atoms' order, and the transposed codes as 64-byte lines (16-byte chunks XORed
// with the column block, two lanes a bank).  Per element 2 B read, 1/2 B of codes
// and 1/32 or 1/16 B of scales written per direction: HBM bound in one direction
// (16384 x 8960: 66 us MXFP4, 70 to 78 us NVFP4, 4.8 to 5.6 TB/s), bound by the code
// arithmetic in both (96 us and 127 us; 20 instructions an element at 60% of the
// issue slots).
#include <cudaTypedefs.h>

#include <algorithm>

#include "gemm_host.h"
#include "kernels.h"
#include "mx4_device.cuh"
#include "qmath.cuh"

namespace fp8blk {

namespace {

constexpr int kTile = 128;
constexpr int kThreads = 256;
constexpr uint32_t kTileBytes = kTile * kTile * 2;
constexpr int kStages = 3;

struct Mx4Ctrl {
  uint64_t full[kStages], empty[kStages];
  int abort;
  alignas(16) float2 divisor[128];                 // NVFP4: (d, -1/d) of every scale byte
  alignas(16) uint8_t atoms[2 * kMx4AtomBytes];    // row scales of a tile
  alignas(16) uint8_t atoms_t[2 * kMx4AtomBytes];     // column scales
  alignas(16) uint8_t codes_t[kTile * kTile / 2];  // transposed codes: 128 lines of 64 bytes
};

constexpr int kSmem = 1024 + kStages * static_cast<int>(kTileBytes) + static_cast<int>(sizeof(Mx4Ctrl));
static_assert(2 * (kSmem + 1024) <= 227 * 1024, "two CTAs per SM");

}  // namespace

template <bool kNv, bool kRow, bool kColT>
__global__ void __launch_bounds__(kThreads, 2) mx4_quant_kernel(const __grid_constant__ CUtensorMap tm,
                                                                 const __grid_constant__ Mx4QuantArgs a) {
  constexpr int kAtoms = kNv ? 2 : 1;       // atoms of a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Mx4Ctrl* ctrl = reinterpret_cast<Mx4Ctrl*>(smem + kStages * kTileBytes);
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const uint32_t tiles_r = static_cast<uint32_t>((a.rows + kTile - 1) / kTile);
  const uint32_t tiles = tiles_r * static_cast<uint32_t>((a.cols + kTile - 1) / kTile);
  volatile int* abort = &ctrl->abort;

  auto load = [&](int stage, uint32_t tile) {
    mbar_arrive_expect_tx(&ctrl->full[stage], kTileBytes);
    tma_load_2d(smem + stage * kTileBytes, &tm, &ctrl->full[stage], static_cast<int>(tile / tiles_r) * kTile,
                static_cast<int>(tile % tiles_r) * kTile);
  };
  uint32_t issued = 0;
  if (t == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&ctrl->full[s], 1);
      mbar_init(&ctrl->empty[s], kThreads / 32);
    }
    ctrl->abort = 0;
    fence_mbar_init();
    tma_prefetch_map(&tm);
    griddep_wait();
    for (uint32_t j = blockIdx.x; issued < kStages && j < tiles; j += gridDim.x) load(issued++, j);
  }
  __syncthreads();
  griddep_wait();
  if (t == 0) griddep_launch_dependents();
  const float g = kNv && a.tensor_scale ? __ldg(a.tensor_scale) : 1.0f, rg = __frcp_rn(g);
  if (kNv && t < 128) {                    // read after the first tile's barrier
    const QScale q = nvfp4_divisor(t, g);
    ctrl->divisor[t] = make_float2(q.s, q.nr);
  }

  // This thread's 8 x 8: rows 32 (warp / 2) + 8 (lane / 8) .., columns 64 (warp % 2) + 8 (lane % 8) ..
  const int r0 = 32 * (warp >> 1) + 8 * (lane >> 3), bj = lane & 7, c0 = 64 * (warp & 1) + 8 * bj;
  uint32_t it = 0;
  for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, ++it) {
    const int s = it % kStages;
    const uint32_t ph = (it / kStages) & 1;
    const bool ok = mbar_wait_bounded<false>(&ctrl->full[s], ph, abort, a.timeout_ns, a.err);
    if (!__syncthreads_and(ok)) break;     // also: the last tile's staged outputs have been read
    const uint32_t tc = tile / tiles_r, tr = tile - tc * tiles_r;
    const int64_t row0 = static_cast<int64_t>(tr) * kTile, col0 = static_cast<int64_t>(tc) * kTile;
    uint4 v[8];
    {
      const uint8_t* xs = smem + s * kTileBytes + r0 * 256 + c0 * 2;
#pragma unroll
      for (int r = 0; r < 8; ++r) v[r] = *reinterpret_cast<const uint4*>(xs + r * 256);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctrl->empty[s]);
    if (t == 0) {
      const uint32_t next = tile + kStages * gridDim.x;
      if (next < tiles && mbar_wait_bounded<false>(&ctrl->empty[s], ph, abort, a.timeout_ns, a.err)) {
        fence_proxy_async_shared();        // the warps' reads, then the TMA's writes
        load(s, next);
        ++issued;
      }
    }

    // Maxima of |x| on raw bits, two to a word: rm[p] rows 2p and 2p + 1 over this
    // thread's 8 columns, cm[j] columns 2j and 2j + 1 over its 8 rows; then over
    // the lanes that share the blocks.
    [[maybe_unused]] uint32_t rm[4], cm[4] = {0, 0, 0, 0};
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      uint32_t m[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 w = v[2 * p + h];
        const uint32_t a0 = w.x & kAbs2, a1 = w.y & kAbs2, a2 = w.z & kAbs2, a3 = w.w & kAbs2;
        if constexpr (kRow) m[h] = __vmaxu2(__vmaxu2(a0, a1), __vmaxu2(a2, a3));
        if constexpr (kColT) {
          cm[0] = __vmaxu2(cm[0], a0);
          cm[1] = __vmaxu2(cm[1], a1);
          cm[2] = __vmaxu2(cm[2], a2);
          cm[3] = __vmaxu2(cm[3], a3);
        }
      }
      if constexpr (kRow) {
        uint32_t k = __vmaxu2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
        k = __vmaxu2(k, __shfl_xor_sync(0xFFFFFFFFu, k, 1));
        if constexpr (!kNv) k = __vmaxu2(k, __shfl_xor_sync(0xFFFFFFFFu, k, 2));
        rm[p] = k;
      }
    }

    // Column scales.  NVFP4: lanes 8 apart share their 8 blocks; each computes those
    // of one parity and hands them over.
    [[maybe_unused]] float cs[8], cn[8];
    if constexpr (kColT) {
      uint8_t* atoms = ctrl->atoms_t;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        cm[j] = __vmaxu2(cm[j], __shfl_xor_sync(0xFFFFFFFFu, cm[j], 8));
        if constexpr (!kNv) cm[j] = __vmaxu2(cm[j], __shfl_xor_sync(0xFFFFFFFFu, cm[j], 16));
      }
      // 32 rows of the warp: block warp / 2 of the one atom (MXFP4), or blocks 2 (warp / 2) and the next of eight.
      const int block = kNv ? 2 * (warp >> 1) + (lane >> 4) : warp >> 1;
      auto put = [&](int col, uint32_t byte) {
        atoms[(block >> 2) * kMx4AtomBytes + (col & 31) * 16 + (col >> 5) * 4 + (block & 3)] = static_cast<uint8_t>(byte);
      };
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float lo = __uint_as_float(cm[j] << 16), hi = __uint_as_float(cm[j] & 0xFFFF0000u);
        if constexpr (kNv) {
          const bool odd = lane & 8;
          const uint32_t byte = nvfp4_scale(odd ? hi : lo, g, rg), other = __shfl_xor_sync(0xFFFFFFFFu, byte, 8);
          put(c0 + 2 * j + odd, byte);
          const float2 q0 = ctrl->divisor[odd ? other : byte], q1 = ctrl->divisor[odd ? byte : other];
          cs[2 * j] = q0.x;
          cs[2 * j + 1] = q1.x;
          cn[2 * j] = q0.y;
          cn[2 * j + 1] = q1.y;
        } else {
          QScale q0, q1;
          const uint32_t b0 = block_scale<kNv>(lo, g, rg, q0), b1 = block_scale<kNv>(hi, g, rg, q1);
          if ((lane & 24) == 0) {
            put(c0 + 2 * j, b0);
            put(c0 + 2 * j + 1, b1);
          }
          cn[2 * j] = q0.nr;
          cn[2 * j + 1] = q1.nr;
          cs[2 * j] = cs[2 * j + 1] = 0.0f;
        }
      }
    }

    // Codes, two rows at a time: a column's values of rows 2p and 2p + 1 form one
    // pair, divided in one packed step by the rows' scales and by the column's.
    // Transposed: of each column, the scaled values of the rows 2p and 2p + 1 for even
    // p, and the codes of this thread's rows so far, four rows to a half word.
    [[maybe_unused]] float2 pend[8];
    [[maybe_unused]] uint16_t half[8];
    [[maybe_unused]] uint32_t line[8];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      float2 x[8];
      {
        const uint4 a0 = v[2 * p], a1 = v[2 * p + 1];
        x[0] = make_float2(bf16lo(a0.x), bf16lo(a1.x));
        x[1] = make_float2(bf16hi(a0.x), bf16hi(a1.x));
        x[2] = make_float2(bf16lo(a0.y), bf16lo(a1.y));
        x[3] = make_float2(bf16hi(a0.y), bf16hi(a1.y));
        x[4] = make_float2(bf16lo(a0.z), bf16lo(a1.z));
        x[5] = make_float2(bf16hi(a0.z), bf16hi(a1.z));
        x[6] = make_float2(bf16lo(a0.w), bf16lo(a1.w));
        x[7] = make_float2(bf16hi(a0.w), bf16hi(a1.w));
      }
      if constexpr (kRow) {
        // 64 columns of the warp: one atom's four blocks (NVFP4), or two of an atom's (MXFP4).
        auto put = [&](int row, uint32_t byte) {
          const int atom = kNv ? warp & 1 : 0, j = kNv ? bj >> 1 : 2 * (warp & 1) + (bj >> 2);
          ctrl->atoms[atom * kMx4AtomBytes + (row & 31) * 16 + (row >> 5) * 4 + j] = static_cast<uint8_t>(byte);
        };
        const float lo = __uint_as_float(rm[p] << 16), hi = __uint_as_float(rm[p] & 0xFFFF0000u);
        float2 s2, nr2;
        if constexpr (kNv) {               // neighbouring lanes share the two rows' blocks: one row each
          const bool odd = lane & 1;
          QScale q;
          put(r0 + 2 * p + odd, block_scale<kNv>(odd ? hi : lo, g, rg, q));
          const float os = __shfl_xor_sync(0xFFFFFFFFu, q.s, 1), on = __shfl_xor_sync(0xFFFFFFFFu, q.nr, 1);
          s2 = odd ? make_float2(os, q.s) : make_float2(q.s, os);
          nr2 = odd ? make_float2(on, q.nr) : make_float2(q.nr, on);
        } else {
          QScale q0, q1;
          const uint32_t b0 = block_scale<kNv>(lo, g, rg, q0), b1 = block_scale<kNv>(hi, g, rg, q1);
          if ((lane & 3) == 0) {
            put(r0 + 2 * p, b0);
            put(r0 + 2 * p + 1, b1);
          }
          s2 = make_float2(0.0f, 0.0f);
          nr2 = make_float2(q0.nr, q1.nr);
        }
        float lo8[8], hi8[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float2 w = scaled2<kNv>(x[c], s2, nr2);
          lo8[c] = w.x;
          hi8[c] = w.y;
        }
        // Neighbouring lanes exchange halves: the even lane stores 16 columns of row 2p, the odd one of row 2p + 1.
        const uint32_t lo_c = finish_codes<kNv>(cvt8_e2m1(lo8), nr2.x), hi_c = finish_codes<kNv>(cvt8_e2m1(hi8), nr2.y);
        const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, (lane & 1) ? lo_c : hi_c, 1);
        const int64_t row = row0 + r0 + 2 * p + (lane & 1);
        const int64_t col = col0 + c0 - 8 * (lane & 1);
        if (row < a.rows && col < a.cols)
          *reinterpret_cast<uint2*>(a.q_row + row * (a.cols / 2) + col / 2) =
              (lane & 1) ? make_uint2(got, hi_c) : make_uint2(lo_c, got);
      }
      if constexpr (kColT) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float2 w = scaled2<kNv>(x[c], make_float2(cs[c], cs[c]), make_float2(cn[c], cn[c]));
          if ((p & 1) == 0) {
            pend[c] = w;
          } else {
            const uint16_t codes = cvt4_e2m1(pend[c].x, pend[c].y, w.x, w.y);
            if (p == 1) half[c] = codes;
            else line[c] = half[c] | (static_cast<uint32_t>(codes) << 16);
          }
        }
      }
    }
    if constexpr (kColT) {
      // Line c0 + c, 4-byte unit r0 / 8; the line's 16-byte chunk r0 / 32 goes to chunk (r0 / 32) ^ (bj % 4).
#pragma unroll
      for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint32_t*>(ctrl->codes_t + (c0 + c) * 64 + (((warp >> 1) ^ (bj & 3)) << 4) +
                                     ((lane >> 3) << 2)) = finish_codes<kNv>(line[c], cn[c]);
    }
    __syncthreads();                       // the staged scales and lines are complete
    if constexpr (kRow) {
      const int64_t atoms_k = (a.cols + mx4_atom_elems<kNv>() - 1) / mx4_atom_elems<kNv>();
      const int i = t >> 5;                // one warp an atom
      const int64_t ka = static_cast<int64_t>(tc) * kAtoms + i;
      if (i < kAtoms && ka < atoms_k)
        *reinterpret_cast<uint4*>(a.s_row + (tr * atoms_k + ka) * kMx4AtomBytes + lane * 16) =
            finish_scales<kNv>(*reinterpret_cast<const uint4*>(ctrl->atoms + i * kMx4AtomBytes + lane * 16));
    }
    if constexpr (kColT) {
      const int64_t padded = (a.rows + 31) / 32 * 32;
      const int64_t atoms_k = (padded + mx4_atom_elems<kNv>() - 1) / mx4_atom_elems<kNv>();
      const int i = (t >> 5) - 2;          // other warps than the row scales'
      const int64_t ka = static_cast<int64_t>(tr) * kAtoms + i;
      if (i >= 0 && i < kAtoms && ka < atoms_k)
        *reinterpret_cast<uint4*>(a.s_t + (tc * atoms_k + ka) * kMx4AtomBytes + lane * 16) =
            finish_scales<kNv>(*reinterpret_cast<const uint4*>(ctrl->atoms_t + i * kMx4AtomBytes + lane * 16));
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int k = t + kThreads * j, col = k >> 2, m = k & 3;
        if (col0 + col < a.cols && row0 + 32 * m < padded)
          *reinterpret_cast<uint4*>(a.q_t + (col0 + col) * (padded / 2) + row0 / 2 + m * 16) =
              *reinterpret_cast<const uint4*>(ctrl->codes_t + col * 64 + ((m ^ ((col >> 3) & 3)) << 4));
      }
    }
  }
  if (t == 0) {
    for (uint32_t j = it; j < issued; ++j)
      mbar_wait_bounded(&ctrl->full[j % kStages], (j / kStages) & 1, nullptr, a.timeout_ns, a.err);
  }
}

// Codes to bf16 values: y = bf16(fl32(code * d)), d the block's scale (times the
// tensor's, in fp32).  HBM bound: 1/2 + 1/32 or 1/16 B read and 2 B written per
// element.  A block covers 32 rows x 256 columns, a thread 8 columns of four rows,
// whose loads are all in flight together.
constexpr int kDequantRows = 4;          // rows of a thread, 8 apart

template <bool kNv>
__global__ void __launch_bounds__(256) mx4_dequant_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s,
                                                          const float* __restrict__ tensor_scale, int64_t rows,
                                                          int64_t cols, uint16_t* __restrict__ y, int64_t ldy) {
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const float g = kNv && tensor_scale ? __ldg(tensor_scale) : 1.0f;
  const int64_t atoms_k = (cols + mx4_atom_elems<kNv>() - 1) / mx4_atom_elems<kNv>();
  const int64_t row0 = blockIdx.x * static_cast<int64_t>(8 * kDequantRows) + threadIdx.y;
  const int64_t col = 8 * (blockIdx.y * static_cast<int64_t>(blockDim.x) + threadIdx.x);
  if (col >= cols) return;
  const int64_t block = col / mx4_block<kNv>();
  uint32_t code[kDequantRows], byte[kDequantRows];
#pragma unroll
  for (int i = 0; i < kDequantRows; ++i) {
    const int64_t row = row0 + 8 * i;
    if (row >= rows) break;
    code[i] = __ldg(reinterpret_cast<const uint32_t*>(q + (row * cols + col) / 2));
    byte[i] = __ldg(s + ((row / 128) * atoms_k + block / 4) * kMx4AtomBytes + (row & 31) * 16 + ((row >> 5) & 3) * 4 +
                    (block & 3));
  }
#pragma unroll
  for (int i = 0; i < kDequantRows; ++i) {
    const int64_t row = row0 + 8 * i;
    if (row >= rows) break;
    const float d = kNv ? e4m3_value(byte[i]) * g : e8m0_value(byte[i]);
    uint32_t h[4];                         // eight f16 values (exact)
    asm("{\n\t.reg .b8 a, b, c, e;\n\t"
        "mov.b32 {a, b, c, e}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, e;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(code[i]));
    uint32_t out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float lo, hi;
      asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
          : "=f"(lo), "=f"(hi)
          : "r"(h[j]));
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(out[j]) : "f"(hi * d), "f"(lo * d));
    }
    *reinterpret_cast<uint4*>(y + row * ldy + col) = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

namespace {

template <bool kNv, bool kRow, bool kColT>
cudaError_t launch_mx4_mode(const Mx4QuantArgs& a, cudaStream_t stream) {
  static PerContext<int> smem_set;
  if (cudaError_t e = set_smem_once(smem_set, mx4_quant_kernel<kNv, kRow, kColT>, kSmem); e != cudaSuccess) return e;
  auto encode = tensor_map_encoder();
  if (!encode) return cudaErrorInvalidValue;
  CUtensorMap tm;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.cols), static_cast<cuuint64_t>(a.rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(a.ldx) * 2};
  const cuuint32_t box[2] = {kTile, kTile};
  const cuuint32_t estr[2] = {1, 1};
  if (encode(&tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(a.x), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  const int64_t tiles = ((a.rows + kTile - 1) / kTile) * ((a.cols + kTile - 1) / kTile);
  int64_t ctas = 2 * static_cast<int64_t>(num_sms());
  if (a.max_ctas > 0 && a.max_ctas < ctas) ctas = a.max_ctas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min(tiles, ctas)), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  cfg.numAttrs = set_pdl_attr(attr, a.pdl);
  cfg.attrs = attr;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, mx4_quant_kernel<kNv, kRow, kColT>, tm, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool kNv>
cudaError_t launch_mx4_fmt(const Mx4QuantArgs& a, cudaStream_t stream) {
  if (a.q_row && a.q_t) return launch_mx4_mode<kNv, true, true>(a, stream);
  return a.q_row ? launch_mx4_mode<kNv, true, false>(a, stream) : launch_mx4_mode<kNv, false, true>(a, stream);
}

}  // namespace

cudaError_t launch_mx4_quant(const Mx4QuantArgs& a, cudaStream_t stream) {
  return a.nv ? launch_mx4_fmt<true>(a, stream) : launch_mx4_fmt<false>(a, stream);
}

cudaError_t launch_mx4_dequant(const Mx4DequantArgs& a, cudaStream_t stream) {
  const dim3 block(32, 8);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.rows + 8 * kDequantRows - 1) / (8 * kDequantRows)),
                     static_cast<unsigned>((a.cols + 255) / 256), 1);
  cfg.blockDim = block;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  cfg.numAttrs = set_pdl_attr(attr, a.pdl);
  cfg.attrs = attr;
  const cudaError_t e =
      a.nv ? cudaLaunchKernelEx(&cfg, mx4_dequant_kernel<true>, a.q, a.s, a.tensor_scale, a.rows, a.cols, a.y, a.ldy)
           : cudaLaunchKernelEx(&cfg, mx4_dequant_kernel<false>, a.q, a.s, a.tensor_scale, a.rows, a.cols, a.y, a.ldy);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace fp8blk
