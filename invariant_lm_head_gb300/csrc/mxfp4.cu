// The 4-bit head (sm_103a): microscaled quantisation to e2m1 and bf16 logits from
// two operands in that format.
//
// The format. 32 consecutive elements of a row share a power of two 2^(b - 127), held
// as the byte b; an element is e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives).
// b leaves the block's largest magnitude in [3.5, 7): nothing is off by more than half
// a step of its own binade, as 7 and above would be when cut to 6. (Relative error of
// normal values 0.112; with the largest in (3, 6] 0.115, in [4, 8) 0.115.) The division
// by a power of two is exact, so each element is rounded once.
//
// Scales lie in memory as the tensor cores read them: 128 rows x 4 blocks (128
// columns) are 512 bytes, byte (row % 32) * 16 + (row / 32 % 4) * 4 + block % 4. A
// tile's scales are then one contiguous copy, and 16 bytes a TMEM lane.
//
// Logits. logits[t][v] = sum_b 2^(hb - 127) 2^(wb - 127) sum_{k in b} hq[t][k] wq[v][k]
// on the tensor cores with the scales applied there (tcgen05 kind::mxf4, K = 64 an
// MMA), fp32 accumulators in TMEM over the whole K, one rounding to bf16.
//
// Batch invariance: a row's products and their order depend on H alone.
#include <atomic>
#include <cstdint>
#include <cstdio>

#include <cuda_bf16.h>

#include "internal.h"
#include "launch.cuh"
#include "lmhead.h"
#include "out_rows.cuh"
#include "ptx.cuh"

namespace lmh {

namespace {

constexpr int kXBlock = 32;     // elements of a scale
constexpr int kXAtomRows = 128; // rows and
constexpr int kXAtomCols = 128; // columns of 512 bytes of scales
constexpr int kXAtomBytes = 512;
constexpr uint32_t kXPad = 127; // the scale 1, in the atoms' unused places

// ------------------------------------------------------------ quantisation
// The byte of a block whose largest magnitude has these bf16 bits: its exponent,
// rounded up from 1.75 on, less two; NaN (255) where the block holds an infinity or
// a NaN.
__device__ __forceinline__ uint32_t mx_scale(uint32_t amax_bits16) {
  if (amax_bits16 >= 0x7f80u) return 255u;
  const uint32_t e = (amax_bits16 + 0x20u) >> 7;
  return e > 2u ? e - 2u : 0u;
}

// Eight bf16 values times 2^(127 - b) as eight e2m1 codes, the first in the lowest bits.
__device__ __forceinline__ uint32_t mx_codes(const uint4& v, uint32_t b) {
  const float inv = __uint_as_float(b == 255u ? 0u : (254u - b) << 23);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f2_unpack(f2_mul(f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)),
                     f2_pack(inv, inv)),
              y[2 * i], y[2 * i + 1]);
  uint32_t out;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(out)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return out;
}

constexpr int kXThreads = 512;
constexpr int kXGridPerSm = 12;  // (152064 x 3584: 3 an SM 223 us, 6 216, 12 212, a tile each 236)
constexpr int kXRows = kXAtomRows / (kXThreads / 16);  // rows of a thread: 4, 32 apart
static_assert(kXRows == 4, "the four rows that share 16 bytes of scales");

// A CTA takes 128 rows x 128 columns: 16 lanes a row (16 bytes each), four rows a thread,
// all loaded before the first is used. A block is four lanes; a row's four scales meet
// in one word, and the words of a thread's four rows are the 16 bytes that they share.
// Bound by HBM: 209 us for a weight of 152064 x 3584, 6.6 TB/s, 0.99 of the copy rate
// (with 256 threads of eight rows 250 us). 64 x 3584 takes 4 us, most of it one load.
__global__ void __launch_bounds__(kXThreads, 3)
    quantize_mxfp4_kernel(const uint16_t* __restrict__ x, int64_t rows, int64_t cols, int64_t ld,
                          int64_t kb, int64_t n_tiles, uint8_t* __restrict__ q,
                          uint8_t* __restrict__ scale) {
  ahead_done();
  const int sub = threadIdx.x & 15, r32 = threadIdx.x >> 4;
  for (int64_t b = blockIdx.x; b < n_tiles; b += gridDim.x) {
    if (b + gridDim.x >= n_tiles) nearly_done();
    const int64_t rb = b / kb;
    const int64_t col = (b - rb * kb) * kXAtomCols + sub * 8;
    const int64_t row0 = rb * kXAtomRows + r32;
    // of this thread's rows, how many there are
    const int n = col < cols ? static_cast<int>(min(int64_t{kXRows}, (rows - row0 + 31) >> 5)) : 0;
    const uint16_t* src = x + row0 * ld + col;
    uint4 v[kXRows];
#pragma unroll
    for (int i = 0; i < kXRows; ++i) {
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (i < n) v[i] = *reinterpret_cast<const uint4*>(src + i * 32 * ld);
    }
    uint8_t* dst = q + (row0 * cols + col) / 2;
    uint32_t words[kXRows];
#pragma unroll
    for (int i = 0; i < kXRows; ++i) {
      uint32_t m = __vmaxu2(__vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu),
                            __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu));
      m = max(m & 0xffffu, m >> 16);
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const uint32_t s = mx_scale(m);
      if (i < n) *reinterpret_cast<uint32_t*>(dst + i * 16 * cols) = mx_codes(v[i], s);
      uint32_t w = (i < n ? s : kXPad) << (8 * (sub >> 2));
      w |= __shfl_xor_sync(0xffffffffu, w, 4);
      words[i] = w | __shfl_xor_sync(0xffffffffu, w, 8);
    }
    if (sub == 0)
      reinterpret_cast<uint4*>(scale + b * kXAtomBytes)[r32] =
          make_uint4(words[0], words[1], words[2], words[3]);
  }
}

// The scale of byte b in fp32.
__device__ __forceinline__ float mx_value(uint32_t b) {
  if (b == 0u) return 0x1p-127f;
  return __uint_as_float(b == 255u ? 0x7fffffffu : b << 23);
}

// The same tiles back to bf16: 218 us for 152064 x 3584, 6.3 TB/s, 0.94 of the copy rate.
__global__ void __launch_bounds__(kXThreads, 3)
    dequantize_mxfp4_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ scale,
                            int64_t rows, int64_t cols, int64_t kb, int64_t n_tiles,
                            uint16_t* __restrict__ out, int64_t ld) {
  ahead_done();
  const int sub = threadIdx.x & 15, r32 = threadIdx.x >> 4;
  for (int64_t b = blockIdx.x; b < n_tiles; b += gridDim.x) {
    if (b + gridDim.x >= n_tiles) nearly_done();
    const int64_t rb = b / kb;
    const int64_t col = (b - rb * kb) * kXAtomCols + sub * 8;
    const int64_t row0 = rb * kXAtomRows + r32;
    const int n = col < cols ? static_cast<int>(min(int64_t{kXRows}, (rows - row0 + 31) >> 5)) : 0;
    const uint8_t* src = q + (row0 * cols + col) / 2;
    uint32_t codes[kXRows];
#pragma unroll
    for (int i = 0; i < kXRows; ++i) {
      codes[i] = 0u;
      if (i < n) codes[i] = *reinterpret_cast<const uint32_t*>(src + i * 16 * cols);
    }
    const uint4 s = reinterpret_cast<const uint4*>(scale + b * kXAtomBytes)[r32];
    const uint32_t words[kXRows] = {s.x, s.y, s.z, s.w};
    uint16_t* dst = out + row0 * ld + col;
#pragma unroll
    for (int i = 0; i < kXRows; ++i) {
      const float f = mx_value((words[i] >> (8 * (sub >> 2))) & 0xffu);
      uint32_t h[4], o[4];
      asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
          "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
          "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
          : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
          : "r"(codes[i]));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
        o[j] = bf16x2_of(p.x * f, p.y * f);
      }
      if (i < n) *reinterpret_cast<uint4*>(dst + i * 32 * ld) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// ------------------------------------------------------------ 4-bit logits
// A CTA alone takes a tile of 128 x 256, a pair of CTAs (cta_group::2) one of 256 x 256:
// each holds its 128 rows of A and half of B, so an MMA reads 8 KB of each SM's shared
// memory instead of 12, and L2 delivers 35 KB a stage and CTA instead of 51.
constexpr int kXM = 128;              // token rows of a CTA
constexpr int kXN = 256;              // vocabulary columns of a tile
constexpr int kXK = 256;              // elements of a ring stage: 128 bytes a row
constexpr int kXSteps = kXK / 64;     // MMAs of a stage
constexpr int kXBox = 32;             // columns of an output box
constexpr int kXBoxes = kXN / kXBox;
constexpr int kXMaxStages = 8;
constexpr int kXEpiWarps = 4;
constexpr int kXLogitsThreads = 64 + 32 * kXEpiWarps;  // warp 0 loads, warp 1 issues
constexpr int kXStagingWarp = 4096;   // of rows at any address
constexpr int kXStagingBytes = kXEpiWarps * kXStagingWarp;
constexpr int kXBarBytes = 512;
constexpr int kXSmemBytes = 232448;
constexpr int kXRingBytes = (kXSmemBytes - 1024 - kXBarBytes - kXStagingBytes) / 1024 * 1024;
constexpr int kXStageAtoms = kXK / kXAtomCols;             // atoms of a stage's scales: 2
constexpr int kXSetBytes = kXStageAtoms * kXAtomBytes;     // a stage's scales of 128 rows
constexpr int kXScaleBytes = (1 + kXN / kXAtomRows) * kXSetBytes;  // A's, then B's
// TMEM's 512 columns: two accumulators, of which the second starts before the first
// ends (the columns [208, 256) are in both), and two stages' scales.
constexpr uint32_t kXScaleCol = 464;  // where the scales begin
constexpr uint32_t kXScaleSet = 24;   // a stage's: 2 x 4 columns for A, 2 x 8 for B
constexpr uint32_t kXAcc1 = kXScaleCol - kXN;  // the second accumulator's first column
constexpr int kXShared = 2;           // output boxes that touch the shared columns
static_assert(kXScaleCol + 2 * kXScaleSet <= 512, "TMEM columns");
static_assert(kXN - kXAcc1 <= kXShared * kXBox, "shared columns");

struct Mxfp4Params {
  int T, V, KB;           // rows, vocabulary, ring stages of K
  int k_steps;            // MMAs of K: ceil(H / 64)
  int n_m, n_n, n_units;  // tiles (of 128 or 256 rows)
  int group_m;
  int a_rows;             // rows of an A box (T <= 128: T rounded up to 8)
  uint16_t* out;
  int64_t ld;
  int wide;               // rows on 32 (2) or 16 (1) bytes: stored in such parts
  unsigned* status;
};

// D[tmem] (+)= A[smem] * B[smem]^T, e2m1 inputs with a scale for 32 of K each, K = 64.
template <bool kPair>
__device__ __forceinline__ void tc_mma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t sfa_tmem, uint32_t sfb_tmem,
                                            uint32_t accumulate) {
  if constexpr (kPair)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
}

// 512 bytes of scales (32 rows of 16 bytes) into four TMEM columns, to the lanes of all
// four warps; a pair's form does so in each CTA from its own shared memory. Runs in
// order with the MMAs that the same thread issues.
template <bool kPair>
__device__ __forceinline__ void tc_copy_scales(uint32_t tmem, uint64_t desc) {
  if constexpr (kPair)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
                 : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
                 : "memory");
}

// Shared-memory descriptor of such an atom: no swizzle, 8 rows of 16 bytes together,
// 128 bytes from one such group to the next.
__device__ __forceinline__ uint64_t scales_desc(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(128u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  return d;
}

// Instruction descriptor for kind::mxf4: A and B e2m1 (format 1 in bits 7 and 10), both
// K-major, [17,23) N >> 3, bit 23 scales are powers of two, [24,29) M >> 4; `half`: which two
// of an atom's four scales ([4,6) for B, [29,31) for A: 0 or 2).
__device__ constexpr uint32_t idesc_mxf4(uint32_t M, uint32_t N, uint32_t half) {
  return (half << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | (1u << 23) | ((M >> 4) << 24) |
         (half << 29);
}

__device__ __forceinline__ void mx_unit(const Mxfp4Params& p, int u, int& m, int& n) {
  const int per_group = p.group_m * p.n_n;
  const int g = u / per_group;
  const int first = g * p.group_m;
  const int gm = min(p.group_m, p.n_m - first);
  const int r = u - g * per_group;
  n = r / gm;
  m = first + (r - n * gm);
}

// 32 finished columns of this lane's row, the first n - col of them, in parts of 32 or 16
// bytes. Straight from the registers: a box in shared memory on the way to a TMA store
// costs the loads and the MMAs, which share its bandwidth, more than 64-byte pieces of
// rows cost L2.
__device__ __forceinline__ void store_box(uint16_t* row, int col, int n, const uint32_t (&d)[32],
                                          int wide) {
  uint32_t w[16];
#pragma unroll
  for (int j = 0; j < 16; ++j)
    w[j] = bf16x2_of(__uint_as_float(d[2 * j]), __uint_as_float(d[2 * j + 1]));
  uint16_t* o = row + col;
  const int left = n - col;
  if (left >= kXBox && wide == 2) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o + 16 * j),
                   "r"(w[8 * j]), "r"(w[8 * j + 1]), "r"(w[8 * j + 2]), "r"(w[8 * j + 3]),
                   "r"(w[8 * j + 4]), "r"(w[8 * j + 5]), "r"(w[8 * j + 6]), "r"(w[8 * j + 7])
                   : "memory");
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (8 * j + 8 <= left) {
      *reinterpret_cast<uint4*>(o + 8 * j) =
          make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    } else {  // the vocabulary's end
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (8 * j + e < left) o[8 * j + e] = static_cast<uint16_t>(w[4 * j + e / 2] >> (16 * (e & 1)));
    }
  }
}

// Warp 0 loads, warp 1 copies the scales to TMEM and issues the MMAs (CTA 0 of a pair for
// both), the others turn finished tiles to bf16. Tokens are the MMA's rows, the
// vocabulary its columns.
//
// What bounds it. A short batch reads the weight once: 46 us at T=1 H=3584 V=152064, 6.3
// TB/s, 0.94 of the copy rate; 14.8 us at T=64 H=4096 V=32000, where first loads and the
// single wave's end take 5 us beside 10 of bytes. A long batch takes 314 us at T=2048
// H=3584 V=152064 (7.1 PFLOP/s; 360, 6.2, in a loop that runs into the power cap): MMAs
// and scale copies alone take 259, with the loads 272 (17.5 TB/s out of L2, near what it
// gives), and the stores, which share L2 and HBM with the loads, the rest. Of the 259 us
// 218 are MMAs at their rate (128 cycles for 256 x 256 x 64 of a pair) and the others the
// gap between two tiles, about 1000 cycles: the accumulators share columns, and the next
// tile's MMAs wait until those are read.
// In between: T=200 V=32000 takes 19.0 us at H=3584 (two waves of pairs, the second of 50 of
// 76), 22.1 at H=3616: where H / 32 is odd, rows of q start between two 32-byte sectors of
// L2 (T=300 24.2 us at H=3840, 33.8 at 3616). Rows of V=32003 one behind the other take
// 1.3 us more than on 16 bytes.
// Tried and slower at T=2048: eight warps for the finished tiles (349 us), groups of 4
// and 2 row blocks in the raster (340, 365), boxes of shared memory and TMA stores for
// the output (as fast there, 18.1 us at T=64).
template <bool kPair>
__device__ __forceinline__ void logits_mxfp4_body(const CUtensorMap& tmA, const CUtensorMap& tmB,
                                                  const CUtensorMap& tmSA, const CUtensorMap& tmSB,
                                                  const Mxfp4Params& p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t base = smem_u32(smem);
  const uint32_t staging = base + kXRingBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kXRingBytes + kXStagingBytes);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (kXMaxStages + s); };
  const uint32_t tfull_bar = bar0 + 8u * (2 * kXMaxStages);
  const uint32_t tfree_bar = bar0 + 8u * (2 * kXMaxStages + 1);
  const uint32_t final_bar = bar0 + 8u * (2 * kXMaxStages + 2);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kXMaxStages + 3);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // pair: the number of stages that CTA 1 loaded, told to CTA 0 at the end
  volatile uint32_t* peer_issued = tmem_slot + 2;
  static_assert(8 * (2 * kXMaxStages + 3) + 12 <= kXBarBytes, "barrier area");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = kPair ? cluster_ctarank() : 0u;
  const int first_unit = kPair ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
  const int unit_stride = kPair ? static_cast<int>(cluster_nid_x()) : static_cast<int>(gridDim.x);
  const uint32_t a_bytes = static_cast<uint32_t>(p.a_rows) * (kXK / 2);
  constexpr uint32_t kBBytes = (kPair ? kXN / 2 : kXN) * (kXK / 2);
  const uint32_t stage_bytes = a_bytes + kBBytes + kXScaleBytes;
  // the last stage's A operand may reach 128 rows on, past a short stage
  const uint32_t n_st =
      min(static_cast<uint32_t>(kXMaxStages),
          (kXRingBytes - (kXM * kXK / 2 - min(stage_bytes, static_cast<uint32_t>(kXM * kXK / 2)))) /
              stage_bytes);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kXMaxStages; ++s) {
      mbar_init(full_bar(s), 1);  // a pair's CTA 0: one arrive, both CTAs' bytes
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(tfull_bar, 1);
    mbar_init(tfree_bar, (kPair ? 2 : 1) * kXEpiWarps);  // a pair's: CTA 0's
    mbar_init(final_bar, 1);
    *abort_flag = 0;
    *peer_issued = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSA);
    tma_prefetch_desc(&tmSB);
  }
  if (warp == 1) {
    if constexpr (kPair) {
      tmem_alloc_pair(smem_u32(tmem_slot), 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if constexpr (kPair) {
    __syncwarp();
    cluster_sync();  // the peer's barriers are initialised before any arrive on them
  } else {
    __syncthreads();
  }
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  long long issued = 0;  // stages loaded by this CTA
  ahead_done();

  // Warps 0 and 1 run their loops as whole warps and act by one elected lane: with the
  // loops in one lane's branch the issue of a stage's 11 instructions took 1450 cycles
  // (CTAs alone at T=2048 H=3584 V=152064: 673 us for 438).
  if (warp == 0) {
    const bool one = elect_one();
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    for (int u = first_unit; u < p.n_units && ok; u += unit_stride) {
      int m, n;
      mx_unit(p, u, m, n);
      const int row_blk = kPair ? 2 * m + static_cast<int>(rank) : m;
      const int b_row = n * kXN + (kPair ? static_cast<int>(rank) * (kXN / 2) : 0);
      for (int kb = 0; kb < p.KB; ++kb) {
        if (!__all_sync(0xffffffffu, mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.status))) {
          ok = false;
          break;
        }
        const uint32_t sA = base + stage * stage_bytes;
        const uint32_t sS = sA + a_bytes + kBBytes;
        if (one) {
          if (rank == 0)
            mbar_arrive_expect_tx(full_bar(stage), (kPair ? 2u : 1u) * stage_bytes);
          if constexpr (kPair) {
            const uint32_t bar = mapa_shared(full_bar(stage), 0);
            tma_load_2d_pair(sA + a_bytes, &tmB, bar, kb * (kXK / 2), b_row);
            tma_load_2d_pair(sA, &tmA, bar, kb * (kXK / 2), row_blk * kXM);
            tma_load_2d_pair(sS, &tmSA, bar, kb * (kXSetBytes / 4), row_blk);
            tma_load_2d_pair(sS + kXSetBytes, &tmSB, bar, kb * (kXSetBytes / 4),
                             n * (kXN / kXAtomRows));
          } else {
            tma_load_2d(sA + a_bytes, &tmB, full_bar(stage), kb * (kXK / 2), b_row);
            tma_load_2d(sA, &tmA, full_bar(stage), kb * (kXK / 2), row_blk * kXM);
            tma_load_2d(sS, &tmSA, full_bar(stage), kb * (kXSetBytes / 4), row_blk);
            tma_load_2d(sS + kXSetBytes, &tmSB, full_bar(stage), kb * (kXSetBytes / 4),
                        n * (kXN / kXAtomRows));
          }
        }
        ++issued;
        if (++stage == n_st) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    nearly_done();
    if constexpr (kPair) {
      if (rank != 0 && one)  // CTA 0 waits for this CTA's copies too, at the end
        st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<uint32_t*>(peer_issued)), 0),
                              static_cast<uint32_t>(issued));
    } else {
      // Wait (bounded) for the copies still in flight, so that none lands after the
      // CTA exits: in every case, as another role may give up after the last was issued.
      volatile int no_abort = 0;
      for (long long i = issued > n_st ? issued - n_st : 0; i < issued; ++i)
        mbar_wait(full_bar(static_cast<uint32_t>(i % n_st)),
                  static_cast<uint32_t>((i / n_st) & 1), &no_abort, p.status);
    }
  } else if (warp == 1) {
    const bool one = elect_one();
    volatile int no_abort = 0;
    if (rank == 0) {
      constexpr uint32_t kM = kPair ? 2 * kXM : kXM;
      const uint64_t a0 = sw128_kmajor_desc(base), b0 = sw128_kmajor_desc(base + a_bytes);
      const uint64_t s0 = scales_desc(base + a_bytes + kBBytes);
      uint32_t stage = 0, phase = 0, set = 0, tile = 0;
      bool ok = true;
      auto commit = [&](uint32_t bar) {
        if (one) {
          if constexpr (kPair)
            tc_commit_pair(bar, 0x3);
          else
            tc_commit(bar);
        }
      };
      for (int u = first_unit; u < p.n_units && ok; u += unit_stride, ++tile) {
        const uint32_t acc = tmem + ((tile & 1u) ? kXAcc1 : 0u);
        for (int kb = 0; kb < p.KB; ++kb) {
          if (!__all_sync(0xffffffffu, mbar_wait(full_bar(stage), phase, abort_flag, p.status))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t off = (stage * stage_bytes) >> 4;
          const uint64_t ad = a0 + off, bd = b0 + off, sd = s0 + off;
          const uint32_t sfa = tmem + kXScaleCol + set * kXScaleSet, sfb = sfa + 8;
          const int now = p.k_steps - kb * kXSteps;  // MMAs up to the end of K
          if (one) {
#pragma unroll
            for (int a = 0; a < kXStageAtoms; ++a) {  // past K's end too: zeros
              tc_copy_scales<kPair>(sfa + 4 * a, sd + a * (kXAtomBytes >> 4));
#pragma unroll
              for (int i = 0; i < kXN / kXAtomRows; ++i)
                tc_copy_scales<kPair>(sfb + 8 * a + 4 * i,
                                      sd + ((1 + i) * kXSetBytes + a * kXAtomBytes) / 16);
            }
          }
          if (kb == 0) {
            // the tile before has left the columns that both accumulators hold (and the
            // one before that has left this one)
            if (!__all_sync(0xffffffffu, mbar_wait<kPair>(tfree_bar, (tile & 1u) ^ 1u, abort_flag,
                                                          p.status))) {
              ok = false;
              break;
            }
            tc_fence_after();
          }
          if (one) {
#pragma unroll
            for (int k = 0; k < kXSteps; ++k)  // 32 bytes on in each 128-byte row
              if (k == 0 || k < now)
                tc_mma_mxf4<kPair>(acc, ad + 2 * k, bd + 2 * k, idesc_mxf4(kM, kXN, 2u * (k & 1)),
                                   sfa + 4 * (k >> 1), sfb + 8 * (k >> 1),
                                   k > 0 || kb > 0 ? 1u : 0u);
          }
          commit(empty_bar(stage));
          if (kb == p.KB - 1) commit(tfull_bar);
          set ^= 1u;
          if (++stage == n_st) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // Every MMA ends before TMEM is released, also where a role gave up.
      commit(final_bar);
    }
    mbar_wait(final_bar, 0, &no_abort, p.status);
  } else {
    const int ew = warp - 2;
    const int lanes0 = 32 * (warp & 3);  // the TMEM lanes this warp may read
    const uint32_t lane_addr = static_cast<uint32_t>(lanes0) << 16;
    const uint32_t stg = staging + ew * kXStagingWarp;
    uint32_t tile = 0;
    for (int u = first_unit; u < p.n_units; u += unit_stride, ++tile) {
      int m, n;
      mx_unit(p, u, m, n);
      const int row0 = (kPair ? 2 * m + static_cast<int>(rank) : m) * kXM + lanes0;
      const int row = row0 + lane;
      const bool warp_on = row0 < p.T;
      const int64_t col0 = static_cast<int64_t>(n) * kXN;
      const uint32_t src = tmem + lane_addr + ((tile & 1u) ? kXAcc1 : 0u);
      const bool ready = mbar_wait<kPair>(tfull_bar, tile & 1u, abort_flag, p.status);
      if (!__all_sync(0xffffffffu, ready)) break;
      tc_fence_after();
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (kPair)
            mbar_arrive_remote(mapa_shared(tfree_bar, 0));
          else
            mbar_arrive(tfree_bar);
        }
      };
      if (!warp_on) {  // no row of this warp's is stored
        release();
        continue;
      }
      // the shared columns first (the last boxes of the first accumulator, the first of
      // the second): the next tile's MMAs wait for no more than these reads
      if (p.wide > 0) {
        uint16_t* const o = p.out + static_cast<int64_t>(row) * p.ld + col0;
        const int n_cols = row < p.T ? static_cast<int>(min(int64_t{kXN}, p.V - col0)) : 0;
        const int first = (tile & 1u) ? 0 : kXBoxes - kXShared;
        uint32_t d0[32], d1[32];
        tmem_ld32_issue(src + first * kXBox, d0);
        tmem_ld32_issue(src + (first + 1) * kXBox, d1);
        tmem_ld_wait(d0);
        tmem_ld_wait(d1);
        release();
        store_box(o, first * kXBox, n_cols, d0, p.wide);
        store_box(o, (first + 1) * kXBox, n_cols, d1, p.wide);
#pragma unroll 1
        for (int i = kXShared; i < kXBoxes; ++i) {
          const int b = (first + i) & (kXBoxes - 1);
          // the stores part the lanes (rows past T, the vocabulary's end), and TMEM is read
          // by whole warps only
          __syncwarp();
          tmem_ld32_issue(src + b * kXBox, d0);
          tmem_ld_wait(d0);
          store_box(o, b * kXBox, n_cols, d0, p.wide);
        }
        __syncwarp();  // and so is the next tile
        continue;
      }
      // rows at any address leave through shared memory, half a tile's columns at a time
#pragma unroll 1
      for (int i = 0; i < 2; ++i) {
        const int h = (tile & 1u) ? i : 1 - i;
        const int64_t colb = col0 + h * (kXN / 2);
        uint32_t words[kXN / 4];
#pragma unroll
        for (int b = 0; b < kXBoxes / 2; ++b) {
          uint32_t d[32];
          tmem_ld32_issue(src + h * (kXN / 2) + b * kXBox, d);
          tmem_ld_wait(d);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            words[16 * b + j] = bf16x2_of(__uint_as_float(d[2 * j]), __uint_as_float(d[2 * j + 1]));
        }
        if (i == 0) release();
        if (colb < p.V)
          store_rows(stg, lane, words, p.out + static_cast<int64_t>(row0) * p.ld + colb, p.ld,
                     min(32, p.T - row0),
                     static_cast<int>(min(int64_t{kXN / 2}, p.V - colb)));
      }
    }
  }

  tc_fence_before();
  if constexpr (kPair) {
    // Neither CTA leaves (or frees TMEM) while the other may still touch its barriers,
    // shared memory or TMEM. In between CTA 0 waits (bounded) for every stage still in
    // flight in either CTA: the stages before the last n_st of the CTA further ahead were
    // consumed by MMAs. A stage that one CTA did not load gets that CTA's share settled
    // here (CTA 0's arrive, or CTA 1's bytes as done).
    __syncwarp();
    cluster_sync();
    if (rank == 0 && warp == 0 && lane == 0) {
      const long long n0 = issued, n1 = static_cast<long long>(*peer_issued);
      const long long hi = n0 > n1 ? n0 : n1;
      volatile int no_abort = 0;
      for (long long i = hi > n_st ? hi - n_st : 0; i < hi; ++i) {
        const uint32_t s = static_cast<uint32_t>(i % n_st);
        if (i < n0 && i >= n1)
          mbar_complete_tx(full_bar(s), stage_bytes);
        else if (i >= n0 && i < n1)
          mbar_arrive_expect_tx(full_bar(s), stage_bytes);
        mbar_wait(full_bar(s), static_cast<uint32_t>((i / n_st) & 1), &no_abort, p.status);
      }
    }
    __syncwarp();
    cluster_sync();
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if constexpr (kPair)
      tmem_dealloc_pair(tmem, 512);
    else
      tmem_dealloc(tmem, 512);
  }
}

__global__ void __launch_bounds__(kXLogitsThreads, 1)
    logits_mxfp4_kernel(const __grid_constant__ CUtensorMap tmA,
                        const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ CUtensorMap tmSA,
                        const __grid_constant__ CUtensorMap tmSB,
                        const Mxfp4Params p) {
  logits_mxfp4_body<false>(tmA, tmB, tmSA, tmSB, p);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kXLogitsThreads, 1)
    logits_mxfp4_pair_kernel(const __grid_constant__ CUtensorMap tmA,
                             const __grid_constant__ CUtensorMap tmB,
                             const __grid_constant__ CUtensorMap tmSA,
                             const __grid_constant__ CUtensorMap tmSB,
                             const Mxfp4Params p) {
  logits_mxfp4_body<true>(tmA, tmB, tmSA, tmSB, p);
}

// The kernels' shared-memory attribute belongs to the device: set by its first call. *pairs:
// the CTA pairs that the device holds at once.
cudaError_t mxfp4_setup(int sms, int* pairs) {
  static std::atomic<int> done[64];  // pairs + 1
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int n = done[dev].load(std::memory_order_acquire);
  if (n == 0) {
    if ((e = cudaFuncSetAttribute(logits_mxfp4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  kXSmemBytes)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(logits_mxfp4_pair_kernel,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize, kXSmemBytes)) !=
            cudaSuccess)
      return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(sms & ~1));
    cfg.blockDim = dim3(kXLogitsThreads);
    cfg.dynamicSmemBytes = kXSmemBytes;
    if ((e = cudaOccupancyMaxActiveClusters(&n, logits_mxfp4_pair_kernel, &cfg)) != cudaSuccess)
      return e;
    n = (n < sms / 2 ? n : sms / 2) + 1;
    done[dev].store(n, std::memory_order_release);
  }
  *pairs = n - 1;
  return cudaSuccess;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

// Whether n_m row blocks of 128 go to pairs of CTAs. A wave of CTAs alone takes 1.15 to
// 1.4 times a wave of pairs (at one and two row blocks they are the same), so an odd
// last block, which leaves half of a pair idle, can make the pairs slower. H=3584 (us for a
// few calls, alone / pairs): V=152064 200 rows 64 / 60, 384 rows 85 / 90, 512 rows 108 / 96,
// 640 rows 129 / 125, 768 rows 152 / 131, 896 rows 175 / 165, 1152 rows 219 / 198, 2048
// rows 438 / 314; V=32000 384 rows 25.2 / 27.5, 640 rows 36.7 / 32.2. At the power cap
// pairs are the hotter: 640 rows of V=152064, a tie of the rule's, 136 / 141 in a loop, 896
// rows 185 / 184.
bool mxfp4_pairs(int64_t n_m, int64_t n_n, int sms, int pairs) {
  if (n_m < 2 || pairs < 1) return false;
  const int64_t alone = (n_m * n_n + sms - 1) / sms;
  const int64_t paired = ((n_m + 1) / 2 * n_n + pairs - 1) / pairs;
  return alone * 6 >= paired * 5;
}

int launch_error(cudaError_t e, const char* what) {
  char msg[256];
  snprintf(msg, sizeof(msg), "%s: %s", what, cudaGetErrorString(e));
  return api_set_error(LMH_ERR_LAUNCH, msg);
}

// What the quantiser and its inverse ask of a matrix.
int check_matrix(int64_t rows, int64_t cols, int64_t ld) {
  if (rows < 0 || rows > LMH_MAX_DIM || cols < 1 || cols > LMH_MAX_DIM)
    return api_set_error(LMH_ERR_INVALID_ARG, "rows or cols out of range");
  if (ld < cols) return api_set_error(LMH_ERR_INVALID_ARG, "ld must be at least cols");
  if (cols % kXBlock != 0 || ld % 8 != 0)
    return api_set_error(LMH_ERR_ALIGNMENT, "cols must be a multiple of 32 and ld of 8");
  return LMH_OK;
}

}  // namespace

}  // namespace lmh

extern "C" int lmhead_quantize_mxfp4(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld,
                                     uint8_t* q, uint8_t* scale, struct CUstream_st* stream) {
  using namespace lmh;
  int rc = check_matrix(rows, cols, ld);
  if (rc != LMH_OK) return rc;
  if (rows == 0) return api_set_error(LMH_OK, "");
  if (!x || !q || !scale)
    return api_set_error(LMH_ERR_INVALID_ARG, "x, q and scale are required");
  if (misaligned(x, 16) || misaligned(q, 16) || misaligned(scale, 16))
    return api_set_error(LMH_ERR_ALIGNMENT, "x, q and scale need 16-byte alignment");
  int sms = 0;
  unsigned* status = nullptr;
  rc = api_device(&sms, &status);
  if (rc != LMH_OK) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int64_t kb = ceil_div(cols, kXAtomCols);
  const int64_t tiles = ceil_div(rows, kXAtomRows) * kb;
  cudaError_t e;
  {
    KernelTimer timer(K_QUANTIZE_MXFP4, st);
    const int grid = static_cast<int>(tiles < kXGridPerSm * sms ? tiles : kXGridPerSm * sms);
    e = launch_early(quantize_mxfp4_kernel, grid, kXThreads, 0, st, 1, x, rows, cols, ld, kb, tiles,
                     q, scale);
    if (e == cudaSuccess) note_launch();
  }
  if (e != cudaSuccess) return launch_error(e, "4-bit quantisation");
  return api_set_error(LMH_OK, "");
}

extern "C" int lmhead_dequantize_mxfp4(const uint8_t* q, const uint8_t* scale, int64_t rows,
                                       int64_t cols, uint16_t* out, int64_t ld_out,
                                       struct CUstream_st* stream) {
  using namespace lmh;
  int rc = check_matrix(rows, cols, ld_out);
  if (rc != LMH_OK) return rc;
  if (rows == 0) return api_set_error(LMH_OK, "");
  if (!q || !scale || !out)
    return api_set_error(LMH_ERR_INVALID_ARG, "q, scale and out are required");
  if (misaligned(q, 16) || misaligned(scale, 16) || misaligned(out, 16))
    return api_set_error(LMH_ERR_ALIGNMENT, "q, scale and out need 16-byte alignment");
  int sms = 0;
  unsigned* status = nullptr;
  rc = api_device(&sms, &status);
  if (rc != LMH_OK) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int64_t kb = ceil_div(cols, kXAtomCols);
  const int64_t tiles = ceil_div(rows, kXAtomRows) * kb;
  cudaError_t e;
  {
    KernelTimer timer(K_DEQUANTIZE_MXFP4, st);
    const int grid = static_cast<int>(tiles < kXGridPerSm * sms ? tiles : kXGridPerSm * sms);
    e = launch_early(dequantize_mxfp4_kernel, grid, kXThreads, 0, st, 1, q, scale, rows, cols, kb,
                     tiles, out, ld_out);
    if (e == cudaSuccess) note_launch();
  }
  if (e != cudaSuccess) return launch_error(e, "4-bit dequantisation");
  return api_set_error(LMH_OK, "");
}

extern "C" int lmhead_logits_mxfp4(const uint8_t* hidden_q, const uint8_t* hidden_scale,
                                   const uint8_t* weight_q, const uint8_t* weight_scale, int64_t T,
                                   int64_t H, int64_t V, uint16_t* logits, int64_t ld_logits,
                                   struct CUstream_st* stream) {
  using namespace lmh;
  if (T < 0 || T > LMH_MAX_DIM || V < 1 || V > LMH_MAX_DIM || H < 1 || H > LMH_MAX_DIM)
    return api_set_error(LMH_ERR_INVALID_ARG, "T, H or V out of range");
  if (H % kXBlock != 0) return api_set_error(LMH_ERR_ALIGNMENT, "H must be a multiple of 32");
  if (ld_logits < V)
    return api_set_error(LMH_ERR_INVALID_ARG, "ld_logits must be at least V");
  if (ceil_div(T, kXM) * ceil_div(V, kXAtomRows) > (1LL << 30))
    return api_set_error(LMH_ERR_INVALID_ARG, "T x V has too many tiles");
  if (T == 0) return api_set_error(LMH_OK, "");
  if (!hidden_q || !hidden_scale || !weight_q || !weight_scale || !logits)
    return api_set_error(LMH_ERR_INVALID_ARG, "every pointer is required");
  if (misaligned(hidden_q, 16) || misaligned(weight_q, 16) || misaligned(hidden_scale, 16) ||
      misaligned(weight_scale, 16) || misaligned(logits, 2))
    return api_set_error(LMH_ERR_ALIGNMENT,
                         "the operands and scales need 16-byte, logits 2-byte alignment");
  int sms = 0;
  unsigned* status = nullptr;
  int rc = api_device(&sms, &status);
  if (rc != LMH_OK) return rc;
  int pairs = 0;
  cudaError_t e = mxfp4_setup(sms, &pairs);
  if (e != cudaSuccess) return launch_error(e, "4-bit logits");
  const int64_t n_n = ceil_div(V, kXN);
  const bool pair = mxfp4_pairs(ceil_div(T, kXM), n_n, sms, pairs);
  const int64_t n_m = ceil_div(T, pair ? 2 * kXM : kXM);
  const int64_t k_words = ceil_div(H, kXAtomCols) * (kXAtomBytes / 4);
  Mxfp4Params p{};
  p.T = static_cast<int>(T);
  p.V = static_cast<int>(V);
  p.KB = static_cast<int>(ceil_div(H, kXK));
  p.k_steps = static_cast<int>(ceil_div(H, 64));
  p.n_m = static_cast<int>(n_m);
  p.n_n = static_cast<int>(n_n);
  p.n_units = static_cast<int>(n_m * n_n);
  p.group_m = pair ? 8 : 16;
  p.a_rows = T < kXM ? static_cast<int>((T + 7) / 8 * 8) : kXM;
  p.out = logits;
  p.ld = ld_logits;
  // one row has no distance to the next
  p.wide = (T == 1 || ld_logits % 16 == 0) && !misaligned(logits, 32) ? 2
           : (T == 1 || ld_logits % 8 == 0) && !misaligned(logits, 16) ? 1 : 0;
  p.status = status;
  CUtensorMap ta, tb, tsa, tsb;
  if ((rc = api_make_tmap_u8(&ta, hidden_q, H / 2, T, H / 2, kXK / 2, p.a_rows)) != LMH_OK ||
      (rc = api_make_tmap_u8(&tb, weight_q, H / 2, V, H / 2, kXK / 2, pair ? kXN / 2 : kXN)) !=
          LMH_OK ||
      (rc = api_make_tmap_scales(&tsa, hidden_scale, k_words, ceil_div(T, kXAtomRows),
                                 kXSetBytes / 4, 1)) != LMH_OK ||
      (rc = api_make_tmap_scales(&tsb, weight_scale, k_words, ceil_div(V, kXAtomRows),
                                 kXSetBytes / 4, kXN / kXAtomRows)) != LMH_OK)
    return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  {
    KernelTimer timer(K_LOGITS_MXFP4, st);
    if (pair) {
      const int grid = 2 * (p.n_units < pairs ? p.n_units : pairs);
      e = launch_early(logits_mxfp4_pair_kernel, grid, kXLogitsThreads, kXSmemBytes, st, 1, ta, tb,
                       tsa, tsb, p);
    } else {
      const int grid = p.n_units < sms ? p.n_units : sms;
      e = launch_early(logits_mxfp4_kernel, grid, kXLogitsThreads, kXSmemBytes, st, 1, ta, tb, tsa,
                       tsb, p);
    }
    if (e == cudaSuccess) note_launch();
  }
  if (e != cudaSuccess) return launch_error(e, "4-bit logits");
  return api_set_error(LMH_OK, "");
}
