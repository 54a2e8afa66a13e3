// The fp8 head (sm_103a): block quantisation to e4m3 and bf16 logits from
// block-scaled e4m3 operands.
//
// Quantisation. For a block (1 x 128 for activations, 128 x 128 for the
// weight) a = max(max |x|, 2^-60), scale = a / 448 rounded once, and
// q = e4m3(x * 448 / a). The quotient is the correctly rounded fp32 one, which
// settles every e4m3 rounding as exact arithmetic would: x * 448 has 11
// significant bits and a has 8, so a quotient that is not halfway between two
// e4m3 values is at least 2^-14 away from halfway, relatively, and one that is
// halfway is an fp32 number and comes out exactly.
//
// Logits. With 128-wide K blocks b,
//   logits[t][v] = sum_b (hs[t][b] * ws[v / 128][b]) * sum_{k in b} hq[t][k] * wq[v][k]
// The inner sums run on the tensor cores (tcgen05 kind::f8f6f4, fp32
// accumulators in TMEM, one accumulator per K block); the outer sum runs in
// fp32 registers, one FMA per block in ascending order, and is rounded once to
// bf16. A scale differs per row and block, so it cannot be folded into the
// operands, and the accumulator has to leave TMEM once per block.
//
// Batch invariance: a row's products and their order depend on H alone.
#include <atomic>
#include <cstdint>
#include <cstdio>
#include <type_traits>

#include <cuda_bf16.h>

#include "fp8_block.cuh"
#include "internal.h"
#include "lmhead.h"
#include "out_rows.cuh"
#include "ptx.cuh"

namespace lmh {

namespace {

constexpr int kQBlock = 128;  // elements of a scale block along K (and along V)

// ------------------------------------------------------------ quantisation
__device__ __forceinline__ BlockScale block_scale_of(uint32_t amax_bits16) {
  // amax_bits16: the largest |x| as bf16 bits (the order of magnitudes is the
  // order of their bits; a NaN is above inf)
  const uint32_t bits = amax_bits16 << 16;
  if (bits >= 0x7f800000u) return block_scale_nan(__uint_as_float(bits));
  return block_scale(fmaxf(__uint_as_float(bits), 0x1p-60f));
}

__device__ __forceinline__ uint32_t amax_u16x2(uint32_t m, uint32_t w) {
  return __vmaxu2(m, w & 0x7fff7fffu);
}

__device__ __forceinline__ uint32_t quantize2(uint32_t w, const BlockScale& s) {
  return quantize2(f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)), s);
}

__device__ __forceinline__ uint2 quantize8(const uint4& v, const BlockScale& s) {
  uint2 o;
  o.x = quantize2(v.x, s) | (quantize2(v.y, s) << 16);
  o.y = quantize2(v.z, s) | (quantize2(v.w, s) << 16);
  return o;
}

__device__ __forceinline__ uint32_t amax8(uint32_t m, const uint4& v) {
  m = amax_u16x2(m, v.x);
  m = amax_u16x2(m, v.y);
  m = amax_u16x2(m, v.z);
  return amax_u16x2(m, v.w);
}

constexpr int kQuantThreads = 256;
constexpr int kQuantBlocks = 8;  // 1 x 128 blocks of a warp

// 1 x 128 blocks: 8 lanes hold one block, two runs of 8 elements (16 bytes) each, so
// a block's scale is worked out once for 16 elements of a lane; a warp takes two
// times four consecutive blocks of a row, all loaded before the first is used.
// At 16384 x 5120: one load in flight and a division for each 67 us, four loads
// 44 us (16 lanes a block), this 39.7 us.
__global__ void __launch_bounds__(kQuantThreads)
    quantize_rows_kernel(const uint16_t* __restrict__ x, int64_t rows, int64_t cols, int64_t ld,
                         int64_t kb, int64_t parts, uint8_t* __restrict__ q,
                         float* __restrict__ scale) {
  const int sub = threadIdx.x & 7, quarter = (threadIdx.x >> 3) & 3;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kQuantThreads / 32) + (threadIdx.x >> 5);
  const int64_t row = unit / parts;
  if (row >= rows) return;
  const int64_t blk0 = (unit - row * parts) * kQuantBlocks + quarter;
  const uint16_t* xr = x + row * ld;
  uint4 v[kQuantBlocks / 4][2];
#pragma unroll
  for (int i = 0; i < kQuantBlocks / 4; ++i) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t col = (blk0 + 4 * i) * kQBlock + h * 64 + sub * 8;
      v[i][h] = make_uint4(0u, 0u, 0u, 0u);
      if (col < cols) v[i][h] = *reinterpret_cast<const uint4*>(xr + col);
    }
  }
#pragma unroll
  for (int i = 0; i < kQuantBlocks / 4; ++i) {
    const int64_t blk = blk0 + 4 * i;
    uint32_t m = amax8(amax8(0u, v[i][0]), v[i][1]);
    m = max(m & 0xffffu, m >> 16);
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
    const BlockScale s = block_scale_of(m);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t col = blk * kQBlock + h * 64 + sub * 8;
      if (col < cols) *reinterpret_cast<uint2*>(q + row * cols + col) = quantize8(v[i][h], s);
    }
    if (blk < kb && sub == 0) scale[row * kb + blk] = s.scale;
  }
}

// 128 x 128 blocks: a CTA keeps one block in registers, 8 rows of 16 bytes
// per thread.
__global__ void __launch_bounds__(kQuantThreads)
    quantize_tiles_kernel(const uint16_t* __restrict__ x, int64_t rows, int64_t cols, int64_t ld,
                          int64_t kb, int64_t n_tiles, uint8_t* __restrict__ q,
                          float* __restrict__ scale) {
  __shared__ uint32_t warp_max[2][kQuantThreads / 32];
  const int sub = threadIdx.x & 15;
  int parity = 0;
  for (int64_t b = blockIdx.x; b < n_tiles; b += gridDim.x, parity ^= 1) {
    const int64_t rb = b / kb;
    const int64_t col = (b - rb * kb) * kQBlock + sub * 8;
    const int64_t row0 = rb * kQBlock + (threadIdx.x >> 4);
    uint4 v[8];
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t row = row0 + 16 * i;
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (row < rows && col < cols) v[i] = *reinterpret_cast<const uint4*>(x + row * ld + col);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) m = amax8(m, v[i]);
    m = max(m & 0xffffu, m >> 16);
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) warp_max[parity][threadIdx.x >> 5] = m;
    __syncthreads();  // the other parity's words are free: every thread has read them by now
#pragma unroll
    for (int w = 0; w < kQuantThreads / 32; ++w) m = max(m, warp_max[parity][w]);
    const BlockScale s = block_scale_of(m);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t row = row0 + 16 * i;
      if (row < rows && col < cols)
        *reinterpret_cast<uint2*>(q + row * cols + col) = quantize8(v[i], s);
    }
    if (threadIdx.x == 0) scale[b] = s.scale;
  }
}

// ------------------------------------------------------------ fp8 logits
constexpr int kFM = 128;               // token rows of one CTA's tile
constexpr int kFMaxN = 256;            // most vocabulary columns of a tile
constexpr int kFK = kQBlock;           // one K block per ring stage: 128 bytes per row
constexpr int kFChunk = 16;            // columns read from TMEM at once
constexpr int kFBox = 32;              // columns of an output box; tile widths are multiples
constexpr int kFGroups = 2;            // promote groups of four warps; a warp reads its lane quarter
constexpr int kFMaxAccs = 4;
constexpr int kFMaxStages = 12;
constexpr int kFPromoteWarps = 4 * kFGroups;
constexpr int kFThreads = 128 + 32 * kFPromoteWarps;  // warps 0-3: load, issue, two idle
// Registers: 384 threads start with 168 each. The first warpgroup gives most
// of its own back and the promote groups take 232 for their 128 sums and two
// chunks in flight: 128 * 40 + 256 * 232 = 384 * 168.
constexpr int kFRegsFew = 40, kFRegsMany = 232;
static_assert(128 * kFRegsFew + 32 * kFPromoteWarps * kFRegsMany <= kFThreads * 168, "registers");
constexpr int kFStagingWarp = 4096;    // output staging of a warp: two 32 x 32 bf16 boxes
constexpr int kFStagingBytes = kFPromoteWarps * kFStagingWarp;
constexpr int kFBarBytes = 512;
constexpr int kFSmemBytes = 232448;    // all that a CTA can have
constexpr int kFRingBytes = (kFSmemBytes - 1024 - kFBarBytes - kFStagingBytes) / 1024 * 1024;

struct Fp8Params {
  int T, V, KB;          // rows, vocabulary, K blocks
  int tile_n;            // columns of a tile
  int n_m, n_n, n_units; // tiles
  int group_m;           // m tiles that share a vocabulary tile in the raster
  int a_rows;            // rows of an A box (T <= 128: T rounded up to 8)
  const float* hs;       // [T][KB]
  const float* ws;       // [ceil(V / 128)][KB]
  uint16_t* out;
  int64_t ld;
  int tma_out;           // rows on 16-byte boundaries: the output leaves by TMA,
  int v_tma;             // which writes whole 16-byte chunks: its columns, V / 8 * 8
  unsigned* status;
};

// D[tmem] (+)= A[smem] * B[smem]^T, e4m3 inputs, fp32 accumulate, K = 32.
__device__ __forceinline__ void tc_mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor for kind::f8f6f4: D f32 (bit 4), A and B e4m3 (format
// 0 in bits 7 and 10), both K-major, [17,23) N >> 3, [24,29) M >> 4.
__device__ __forceinline__ uint32_t idesc_e4m3_f32(uint32_t M, uint32_t N) {
  return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// Unit u -> (m tile, n tile): groups of group_m m tiles, vocabulary tiles
// inside, so that the CTAs at work share a vocabulary tile in L2.
__device__ __forceinline__ void fp8_unit(const Fp8Params& p, int u, int& m, int& n) {
  const int per_group = p.group_m * p.n_n;
  const int g = u / per_group;
  const int first = g * p.group_m;
  const int gm = min(p.group_m, p.n_m - first);
  const int r = u - g * per_group;
  n = r / gm;
  m = first + (r - n * gm);
}

// Warp 0 loads, warp 1 issues the MMAs, the others scale and add each K block's
// accumulator into registers and store the finished tile. Tokens are the MMA's
// rows (one TMEM lane each, so a thread's hidden scale is one number), the
// vocabulary its columns (128 of them share one weight scale).
//
// A short batch loads only its own rows: the rest of the 128-row A operand reads
// whatever the stage holds next (its own vocabulary rows), which only feeds
// lanes that no one reads.
//
// What bounds it. A short batch reads the weight once and is bound by that: 82-84
// us at T=1 H=3584 V=152064, 6.6 TB/s; 26.0 us at T=64 H=4096 V=32000, 5.2 TB/s
// (one wave: its start and end show). A long one is bound by the promote groups:
// a K block's 128 x 256 accumulator is read out of TMEM beside the MMAs, which
// use TMEM as well (about 500 cycles, against 190 with no MMA running), scaled,
// added and handed back, about 1100 cycles in all for 512 of MMAs. 982-999 us at
// T=2048 H=3584 V=152064, 2.24-2.27 PFLOP/s (the same loop with one hand-over a tile
// runs at 3.15, but sums unscaled blocks).
// Tried and slower at T=2048 H=3584 V=38912 (253 us): CTA pairs sharing 256 x 256
// tiles (276 us: half the weight traffic, but the hand-over crosses two CTAs);
// three promote groups (276 us, spills) and four (293 us); halves of 128 columns
// with their own MMAs and buffers (336 us: the MMAs read the A tile twice); 64
// columns read before they are added (261 us). The additions themselves are 35 us
// of it: without them the loop takes 218.
__global__ void __launch_bounds__(kFThreads, 1)
    logits_fp8_kernel(const __grid_constant__ CUtensorMap tmA,
                      const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmC, const Fp8Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t base = smem_u32(smem);
  const uint32_t staging = base + kFRingBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kFRingBytes + kFStagingBytes);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (kFMaxStages + s); };
  auto tfull_bar = [&](uint32_t a) { return bar0 + 8u * (2 * kFMaxStages + a); };
  auto tempty_bar = [&](uint32_t a) { return bar0 + 8u * (2 * kFMaxStages + kFMaxAccs + a); };
  const uint32_t final_bar = bar0 + 8u * (2 * kFMaxStages + 2 * kFMaxAccs);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kFMaxStages + 2 * kFMaxAccs + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert(8 * (2 * kFMaxStages + 2 * kFMaxAccs + 1) + 8 <= kFBarBytes, "barrier area");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t a_bytes = static_cast<uint32_t>(p.a_rows) * kFK;
  const uint32_t stage_bytes = a_bytes + static_cast<uint32_t>(p.tile_n) * kFK;
  // the last stage's A operand may reach 128 rows on, past a short stage
  const uint32_t n_st = min(static_cast<uint32_t>(kFMaxStages),
                            (kFRingBytes - (kFM * kFK - min(stage_bytes, kFM * kFK))) / stage_bytes);
  // accumulators side by side in the 512 columns
  const uint32_t acc_cols = p.tile_n > 128 ? 256u : 128u;
  const uint32_t n_acc = 512u / acc_cols;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kFMaxStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < kFMaxAccs; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), kFPromoteWarps);
    }
    mbar_init(final_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    if (p.tma_out) tma_prefetch_desc(&tmC);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFRegsFew));
    if (warp == 0 && lane == 0) {
      uint32_t stage = 0, phase = 0;
      long long issued = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < p.n_units && ok; u += gridDim.x) {
        int m, n;
        fp8_unit(p, u, m, n);
        for (int kb = 0; kb < p.KB; ++kb) {
          if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          const uint32_t sA = base + stage * stage_bytes;
          mbar_arrive_expect_tx(full_bar(stage), stage_bytes);
          tma_load_2d(sA + a_bytes, &tmB, full_bar(stage), kb * kFK, n * p.tile_n);
          tma_load_2d(sA, &tmA, full_bar(stage), kb * kFK, m * kFM);
          ++issued;
          if (++stage == n_st) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // Wait (bounded) for the copies still in flight, so that none lands after the
      // CTA exits: in every case, as another role may give up after the last was issued.
      volatile int no_abort = 0;
      for (long long i = issued > n_st ? issued - n_st : 0; i < issued; ++i)
        mbar_wait(full_bar(static_cast<uint32_t>(i % n_st)),
                  static_cast<uint32_t>((i / n_st) & 1), &no_abort, p.status);
    }
    if (warp == 1 && lane == 0) {
      const uint32_t idesc = idesc_e4m3_f32(kFM, static_cast<uint32_t>(p.tile_n));
      uint32_t stage = 0, phase = 0, acc = 0, aphase = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < p.n_units && ok; u += gridDim.x) {
        for (int kb = 0; kb < p.KB; ++kb) {
          if (!mbar_wait(tempty_bar(acc), aphase ^ 1u, abort_flag, p.status) ||
              !mbar_wait(full_bar(stage), phase, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sA = base + stage * stage_bytes;
          const uint64_t ad = sw128_kmajor_desc(sA), bd = sw128_kmajor_desc(sA + a_bytes);
#pragma unroll
          for (int k = 0; k < kFK / 32; ++k)  // 32 bytes on in each 128-byte row
            tc_mma_e4m3(tmem + acc * acc_cols, ad + 2 * k, bd + 2 * k, idesc, k > 0 ? 1u : 0u);
          tc_commit(empty_bar(stage));
          tc_commit(tfull_bar(acc));
          if (++stage == n_st) {
            stage = 0;
            phase ^= 1u;
          }
          if (++acc == n_acc) {
            acc = 0;
            aphase ^= 1u;
          }
        }
      }
      // Every MMA of this thread ends before TMEM is released, also where a role gave up.
      volatile int no_abort = 0;
      tc_commit(final_bar);
      mbar_wait(final_bar, 0, &no_abort, p.status);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kFRegsMany));
    const int pw = warp - 4;
    const int lanes0 = 32 * (warp & 3);  // the TMEM lanes this warp may read
    const uint32_t lane_addr = static_cast<uint32_t>(lanes0) << 16;
    const uint32_t stg = staging + pw * kFStagingWarp;
    // this group's part of a tile's columns: whole output boxes, in chunks
    const int boxes = p.tile_n / kFBox;
    const int per = (boxes + kFGroups - 1) / kFGroups;
    const int box0 = (pw >> 2) * per;
    const int chunk0 = box0 * (kFBox / kFChunk);
    const int my = max(0, min(per, boxes - box0)) * (kFBox / kFChunk);
    const int last_vb = (p.V - 1) / kQBlock;
    uint32_t acc = 0, aphase = 0, obuf = 0;
    // One tile, kCh chunks of it this group's: branch-free inside a K block (with
    // a test at each chunk the reads and sums of a block took 870 cycles).
    auto tile = [&](auto chunk_count, int u) -> bool {
      constexpr int kCh = decltype(chunk_count)::value;
      int m, n;
      fp8_unit(p, u, m, n);
      const int row0 = m * kFM + lanes0;
      const int row = row0 + lane;
      const bool warp_on = row0 < p.T;
      const int64_t col0 = static_cast<int64_t>(n) * p.tile_n + chunk0 * kFChunk;
      // the group's columns (at most 128) meet at most two weight scales:
      // chunks below `cut` take the first
      const int vb0 = static_cast<int>(col0 / kQBlock);
      const int cut = static_cast<int>((static_cast<int64_t>(vb0 + 1) * kQBlock - col0) / kFChunk);
      const float* hs = p.hs + static_cast<int64_t>(min(row, p.T - 1)) * p.KB;
      const float* ws0 = p.ws + static_cast<int64_t>(min(vb0, last_vb)) * p.KB;
      const float* ws1 = p.ws + static_cast<int64_t>(min(vb0 + 1, last_vb)) * p.KB;
      float sum[kCh > 0 ? kCh * kFChunk : 1];
#pragma unroll
      for (int i = 0; i < kCh * kFChunk; ++i) sum[i] = 0.f;
      float h = hs[0], w0 = ws0[0], w1 = ws1[0];
      for (int kb = 0; kb < p.KB; ++kb) {
        const float s0 = __fmul_rn(h, w0), s1 = __fmul_rn(h, w1);
        if (kb + 1 < p.KB) {  // the next block's scales arrive during this one
          ++hs;
          ++ws0;
          ++ws1;
        }
        h = *hs;
        w0 = *ws0;
        w1 = *ws1;
        const bool ready = mbar_wait(tfull_bar(acc), aphase, abort_flag, p.status);
        if (!__all_sync(0xffffffffu, ready)) return false;
        tc_fence_after();
        if (warp_on) {
          // the next chunk's load is under way while one chunk is added
          const uint32_t src = tmem + lane_addr + acc * acc_cols + chunk0 * kFChunk;
          uint32_t d[2][kFChunk];
          if (kCh > 0) tmem_ld16_issue(src, d[0]);
#pragma unroll
          for (int c = 0; c < kCh; ++c) {
            tmem_ld_wait(d[c & 1]);
            if (c + 1 < kCh) tmem_ld16_issue(src + (c + 1) * kFChunk, d[(c + 1) & 1]);
            const float s = c < cut ? s0 : s1;
#pragma unroll
            for (int i = 0; i < kFChunk; i += 2) {
              float* o = sum + c * kFChunk + i;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(d[c & 1][i]), __uint_as_float(d[c & 1][i + 1])),
                               f2_pack(s, s), f2_pack(o[0], o[1])),
                        o[0], o[1]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty_bar(acc));
        if (++acc == n_acc) {
          acc = 0;
          aphase ^= 1u;
        }
      }
      if (!warp_on || kCh == 0 || col0 >= p.V) return true;
      if (!p.tma_out) {
        uint32_t words[kCh > 0 ? kCh * kFChunk / 2 : 4];
#pragma unroll
        for (int i = 0; i < kCh * kFChunk / 2; ++i) words[i] = bf16x2_of(sum[2 * i], sum[2 * i + 1]);
        const int64_t left = p.V - col0;
        store_rows(stg, lane, words, p.out + static_cast<int64_t>(row0) * p.ld + col0, p.ld,
                   min(32, p.T - row0),
                   static_cast<int>(min(static_cast<int64_t>(kCh * kFChunk), left)));
        return true;
      }
#pragma unroll
      for (int b = 0; b < kCh * kFChunk / kFBox; ++b) {
        const int64_t colb = col0 + b * kFBox;
        if (colb >= p.V) break;
        // a warp's 32 rows leave in boxes of 32 columns, through two buffers in turn
        const uint32_t obox = stg + obuf;
        obuf ^= kFStagingWarp / 2;
        if (lane == 0) bulk_wait_group_read<1>();  // the box before the last has left
        __syncwarp();
        stage_box_row(obox, lane, sum + b * kFBox);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (colb < p.v_tma) tma_store_2d(&tmC, obox, static_cast<int32_t>(colb), row0);
          bulk_commit_group();  // an empty one too: the buffers' turns are counted in groups
        }
        if (p.v_tma < p.V && p.v_tma < colb + kFBox && row < p.T) {
          // the vocabulary's last columns (at most seven): a chunk that TMA would fill
          // with zeros past the row's end
          const int j = (p.v_tma - static_cast<int>(colb)) >> 3;
          const uint4 v = ld_shared_v4(obox + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint16_t* o = p.out + static_cast<int64_t>(row) * p.ld + p.v_tma;
#pragma unroll
          for (int i = 0; i < 7; ++i)
            st_global_u16_if(o + i, static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1))),
                             p.v_tma + i < p.V);
        }
      }
      return true;
    };
    // this group's boxes: the same number in every tile, possibly none
    for (int u = blockIdx.x; u < p.n_units; u += gridDim.x) {
      bool more = true;
      switch (my / (kFBox / kFChunk)) {
        case 4: more = tile(std::integral_constant<int, 8>{}, u); break;
        case 3: more = tile(std::integral_constant<int, 6>{}, u); break;
        case 2: more = tile(std::integral_constant<int, 4>{}, u); break;
        case 1: more = tile(std::integral_constant<int, 2>{}, u); break;
        default: more = tile(std::integral_constant<int, 0>{}, u); break;
      }
      if (!more) break;
    }
    if (lane == 0) bulk_wait_group<0>();  // every output box of this warp has been written
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The kernel's shared-memory attribute belongs to the device: set by its first call.
cudaError_t fp8_setup() {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(logits_fp8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kFSmemBytes);
  if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
  return e;
}

// Columns of a tile when `sms` CTAs share the vocabulary m_tiles times over: as
// few waves as 256-column tiles need, each tile just wide enough to fill them (one
// 64-row tile of H=4096 V=32000, one wave of 152: 224 columns on 143 CTAs 26.0 us,
// 128 columns in two waves 32.1 us).
int fp8_tile_n(int64_t V, int64_t m_tiles, int sms) {
  const int64_t units = m_tiles * ((V + kFMaxN - 1) / kFMaxN);
  const int64_t waves = (units + sms - 1) / sms;
  const int64_t per_m = waves * sms / m_tiles;  // vocabulary tiles in that many waves
  if (per_m < 1) return kFMaxN;
  const int64_t n = ((V + per_m - 1) / per_m + kFBox - 1) / kFBox * kFBox;
  return static_cast<int>(n < kFMaxN ? n : kFMaxN);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

int launch_error(cudaError_t e, const char* what) {
  char msg[256];
  snprintf(msg, sizeof(msg), "%s: %s", what, cudaGetErrorString(e));
  return api_set_error(LMH_ERR_LAUNCH, msg);
}

}  // namespace

}  // namespace lmh

extern "C" int lmhead_quantize_fp8(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld,
                                   int block_rows, uint8_t* q, float* scale,
                                   struct CUstream_st* stream) {
  using namespace lmh;
  if (rows < 0 || rows > LMH_MAX_DIM || cols < 1 || cols > LMH_MAX_DIM)
    return api_set_error(LMH_ERR_INVALID_ARG, "rows or cols out of range");
  if (block_rows != 1 && block_rows != kQBlock)
    return api_set_error(LMH_ERR_INVALID_ARG, "block_rows must be 1 or 128");
  if (ld < cols) return api_set_error(LMH_ERR_INVALID_ARG, "ld must be at least cols");
  if (cols % 16 != 0 || ld % 8 != 0)
    return api_set_error(LMH_ERR_ALIGNMENT, "cols must be a multiple of 16 and ld of 8");
  if (ceil_div(rows, 8) * ceil_div(cols, kQBlock) > 0x7fffffffLL)
    return api_set_error(LMH_ERR_INVALID_ARG, "rows x cols has too many blocks");
  if (rows == 0) return api_set_error(LMH_OK, "");
  if (!x || !q || !scale)
    return api_set_error(LMH_ERR_INVALID_ARG, "x, q and scale are required");
  if (misaligned(x, 16) || misaligned(q, 16) || misaligned(scale, 4))
    return api_set_error(LMH_ERR_ALIGNMENT, "x and q need 16-byte, scale 4-byte alignment");
  int sms = 0;
  unsigned* status = nullptr;
  const int rc = api_device(&sms, &status);
  if (rc != LMH_OK) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int64_t kb = ceil_div(cols, kQBlock);
  cudaError_t e;
  {
    KernelTimer timer(K_QUANTIZE_FP8, st);
    if (block_rows == 1) {
      const int64_t parts = ceil_div(kb, kQuantBlocks);
      const int64_t grid = ceil_div(rows * parts, kQuantThreads / 32);
      quantize_rows_kernel<<<static_cast<unsigned>(grid), kQuantThreads, 0, st>>>(
          x, rows, cols, ld, kb, parts, q, scale);
    } else {
      const int64_t tiles = ceil_div(rows, kQBlock) * kb;
      const int grid = static_cast<int>(tiles < 8 * sms ? tiles : 8 * sms);
      quantize_tiles_kernel<<<grid, kQuantThreads, 0, st>>>(x, rows, cols, ld, kb, tiles, q, scale);
    }
    e = cudaGetLastError();
    if (e == cudaSuccess) note_launch();
  }
  if (e != cudaSuccess) return launch_error(e, "fp8 quantisation");
  return api_set_error(LMH_OK, "");
}

extern "C" int lmhead_logits_fp8(const uint8_t* hidden_q, const float* hidden_scale,
                                 const uint8_t* weight_q, const float* weight_scale, int64_t T,
                                 int64_t H, int64_t V, uint16_t* logits, int64_t ld_logits,
                                 struct CUstream_st* stream) {
  using namespace lmh;
  if (T < 0 || T > LMH_MAX_DIM || V < 1 || V > LMH_MAX_DIM || H < 1 || H > LMH_MAX_DIM)
    return api_set_error(LMH_ERR_INVALID_ARG, "T, H or V out of range");
  if (H % 16 != 0) return api_set_error(LMH_ERR_ALIGNMENT, "H must be a multiple of 16");
  if (ld_logits < V)
    return api_set_error(LMH_ERR_INVALID_ARG, "ld_logits must be at least V");
  if (ceil_div(T, kFM) * ceil_div(V, kFBox) > (1LL << 30))
    return api_set_error(LMH_ERR_INVALID_ARG, "T x V has too many tiles");
  if (T == 0) return api_set_error(LMH_OK, "");
  if (!hidden_q || !hidden_scale || !weight_q || !weight_scale || !logits)
    return api_set_error(LMH_ERR_INVALID_ARG, "every pointer is required");
  if (misaligned(hidden_q, 16) || misaligned(weight_q, 16) || misaligned(hidden_scale, 4) ||
      misaligned(weight_scale, 4) || misaligned(logits, 2))
    return api_set_error(LMH_ERR_ALIGNMENT,
                         "hidden_q and weight_q need 16-byte, the scales 4-byte, logits 2-byte "
                         "alignment");
  int sms = 0;
  unsigned* status = nullptr;
  int rc = api_device(&sms, &status);
  if (rc != LMH_OK) return rc;
  cudaError_t e = fp8_setup();
  if (e != cudaSuccess) return launch_error(e, "fp8 logits");
  const int64_t n_m = ceil_div(T, kFM);
  Fp8Params p{};
  p.tile_n = fp8_tile_n(V, n_m, sms);
  const int64_t n_n = ceil_div(V, p.tile_n);
  p.T = static_cast<int>(T);
  p.V = static_cast<int>(V);
  p.KB = static_cast<int>(ceil_div(H, kFK));
  p.n_m = static_cast<int>(n_m);
  p.n_n = static_cast<int>(n_n);
  p.n_units = static_cast<int>(n_m * n_n);
  p.group_m = 16;
  p.a_rows = T < kFM ? static_cast<int>((T + 7) / 8 * 8) : kFM;
  p.hs = hidden_scale;
  p.ws = weight_scale;
  p.out = logits;
  p.ld = ld_logits;
  p.v_tma = static_cast<int>(V / 8 * 8);
  p.tma_out = (ld_logits % 8 == 0 && !misaligned(logits, 16) && p.v_tma > 0) ? 1 : 0;
  p.status = status;
  CUtensorMap ta, tb, tc{};
  if (p.tma_out && (rc = api_make_out_tmap_bf16(&tc, logits, p.v_tma, T, ld_logits * 2)) != LMH_OK)
    return rc;
  if ((rc = api_make_tmap_u8(&ta, hidden_q, H, T, H, kFK, p.a_rows)) != LMH_OK) return rc;
  if ((rc = api_make_tmap_u8(&tb, weight_q, H, V, H, kFK, p.tile_n)) !=
      LMH_OK)
    return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  {
    KernelTimer timer(K_LOGITS_FP8, st);
    const int grid = p.n_units < sms ? p.n_units : sms;
    logits_fp8_kernel<<<grid, kFThreads, kFSmemBytes, st>>>(ta, tb, tc, p);
    e = cudaGetLastError();
    if (e == cudaSuccess) note_launch();
  }
  if (e != cudaSuccess) return launch_error(e, "fp8 logits");
  return api_set_error(LMH_OK, "");
}
