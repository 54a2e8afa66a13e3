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

#include <cuda_bf16.h>

#include "internal.h"
#include "lmhead.h"
#include "ptx.cuh"

namespace lmh {

namespace {

constexpr int kQBlock = 128;  // elements of a scale block along K (and along V)

// ------------------------------------------------------------ quantisation
// A block's quotient x * 448 / a in parts that stay clear of overflow and
// underflow: with a = am * 2^e (1 <= am < 2), c = 448 * 2^-e and r = 1 / am
// rounded to nearest, y = x * c is exact wherever q does not round to zero, and
// y / am is corrected from y * r by its exact remainder (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// IBM J. Res. Dev. 34(1), 1990).
struct BlockScale {
  float c, neg_am, r, scale;
};

__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits16) {
  // amax_bits16: the largest |x| as bf16 bits (the order of magnitudes is the
  // order of their bits; a NaN is above inf)
  const uint32_t bits = amax_bits16 << 16;
  BlockScale s;
  if (bits >= 0x7f800000u) {  // inf or NaN in the block: every q becomes NaN
    s.scale = __uint_as_float(bits);
    s.c = 0.f;
    s.neg_am = -1.f;
    s.r = __uint_as_float(0x7fffffffu);
    return s;
  }
  const float a = fmaxf(__uint_as_float(bits), 0x1p-60f);
  const uint32_t ab = __float_as_uint(a);
  const int e = static_cast<int>(ab >> 23) - 127;
  const float am = __uint_as_float((ab & 0x007fffffu) | 0x3f800000u);
  s.c = 448.f * __uint_as_float(static_cast<uint32_t>(127 - (e < 127 ? e : 126)) << 23);
  if (e == 127) s.c *= 0.5f;
  s.neg_am = -am;
  s.r = __frcp_rn(am);
  s.scale = __fdiv_rn(a, 448.f);
  return s;
}

__device__ __forceinline__ uint32_t amax_u16x2(uint32_t m, uint32_t w) {
  return __vmaxu2(m, w & 0x7fff7fffu);
}

// Two quotients to a pair of e4m3 bytes (low half first).
__device__ __forceinline__ uint32_t quantize2(uint32_t w, const BlockScale& s) {
  const f32x2 x = f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  const f32x2 y = f2_mul(x, f2_pack(s.c, s.c));
  const f32x2 r2 = f2_pack(s.r, s.r);
  const f32x2 q0 = f2_mul(y, r2);
  const f32x2 rem = f2_fma(q0, f2_pack(s.neg_am, s.neg_am), y);
  float lo, hi;
  f2_unpack(f2_fma(rem, r2, q0), lo, hi);
  uint16_t out;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(out) : "f"(hi), "f"(lo));
  return out;
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

// 1 x 128 blocks: 16 lanes hold one block, 8 elements (16 bytes) each.
__global__ void __launch_bounds__(kQuantThreads)
    quantize_rows_kernel(const uint16_t* __restrict__ x, int64_t rows, int64_t cols, int64_t ld,
                         int64_t kb, uint8_t* __restrict__ q, float* __restrict__ scale) {
  const int sub = threadIdx.x & 15;
  const int64_t n = rows * kb;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (kQuantThreads / 16);
  for (int64_t b = static_cast<int64_t>(blockIdx.x) * (kQuantThreads / 16) + (threadIdx.x >> 4);
       b - (threadIdx.x >> 4) % 2 < n; b += stride) {  // both halves of a warp take part
    const int64_t row = b / kb;
    const int64_t blk = b - row * kb;
    const int64_t col = blk * kQBlock + sub * 8;
    const bool on = b < n && col < cols;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (on) v = *reinterpret_cast<const uint4*>(x + row * ld + col);
    uint32_t m = amax8(0u, v);
    m = max(m & 0xffffu, m >> 16);
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
    const BlockScale s = block_scale(m);
    if (on) *reinterpret_cast<uint2*>(q + row * cols + col) = quantize8(v, s);
    if (b < n && sub == 0) scale[b] = s.scale;
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
    const BlockScale s = block_scale(m);
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
constexpr int kFM = 128;               // token rows of a tile
constexpr int kFN = 128;               // vocabulary columns of a tile
constexpr int kFK = kQBlock;           // one K block per ring stage: 128 bytes per row
constexpr int kFAccs = 512 / kFN;      // accumulators in TMEM
constexpr int kFMaxStages = 12;
constexpr int kFRingBytes = 208 * 1024;
constexpr int kFBBytes = kFN * kFK;
constexpr int kFPromoteWarps = 8;      // two groups of four: a warp reads its quarter of the lanes
constexpr int kFThreads = 64 + 32 * kFPromoteWarps;
constexpr int kFCols = kFN / 2;        // columns of one promote group
constexpr int kFStageRow = 17;         // 32-bit words per staged row of 32 bf16 (odd: no conflicts)
constexpr int kFStagingBytes = kFPromoteWarps * 32 * kFStageRow * 4;
constexpr int kFBarBytes = 1024;
constexpr int kFSmemBytes = kFRingBytes + kFStagingBytes + kFBarBytes + 1024;
static_assert(kFSmemBytes <= 232448, "exceeds the 227 KB shared-memory limit per CTA");

struct Fp8Params {
  int T, V, KB;          // rows, vocabulary, K blocks
  int n_m, n_n, n_units; // tiles
  int a_rows;            // rows of an A box (T <= 128: T rounded up to 8)
  const float* hs;       // [T][KB]
  const float* ws;       // [ceil(V / 128)][KB]
  uint16_t* out;
  int64_t ld;
  int vec;               // 16-byte stores are aligned
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
constexpr uint32_t idesc_e4m3_f32(uint32_t M, uint32_t N) {
  return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Warp 0 loads, warp 1 issues the MMAs, warps 2-9 scale and add each K block's
// accumulator into registers and store the finished tile. Tokens are the MMA's
// rows (one TMEM lane each, so a thread's hidden scale is one number), the
// vocabulary its columns (128 of them share one weight scale). A short batch
// loads only its own rows: the rest of the 128-row A operand reads whatever the
// stage holds next (its own B rows), which only feeds lanes that no one reads.
__global__ void __launch_bounds__(kFThreads, 1)
    logits_fp8_kernel(const __grid_constant__ CUtensorMap tmA,
                      const __grid_constant__ CUtensorMap tmB, const Fp8Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t base = smem_u32(smem);
  uint32_t* staging = reinterpret_cast<uint32_t*>(smem + kFRingBytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kFRingBytes + kFStagingBytes);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (kFMaxStages + s); };
  auto tfull_bar = [&](uint32_t a) { return bar0 + 8u * (2 * kFMaxStages + a); };
  auto tempty_bar = [&](uint32_t a) { return bar0 + 8u * (2 * kFMaxStages + kFAccs + a); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kFMaxStages + 2 * kFAccs);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t a_bytes = static_cast<uint32_t>(p.a_rows) * kFK;
  const uint32_t stage_bytes = a_bytes + kFBBytes;
  const uint32_t n_st = min(static_cast<uint32_t>(kFMaxStages), kFRingBytes / stage_bytes);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kFMaxStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < kFAccs; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), kFPromoteWarps);
    }
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      long long issued = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < p.n_units && ok; u += gridDim.x) {
        const int n_tile = u / p.n_m, m_tile = u - n_tile * p.n_m;
        for (int kb = 0; kb < p.KB; ++kb) {
          if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          const uint32_t sA = base + stage * stage_bytes;
          mbar_arrive_expect_tx(full_bar(stage), stage_bytes);
          tma_load_2d(sA + a_bytes, &tmB, full_bar(stage), kb * kFK, n_tile * kFN);
          tma_load_2d(sA, &tmA, full_bar(stage), kb * kFK, m_tile * kFM);
          ++issued;
          if (++stage == n_st) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        // wait for the copies still in flight, so that none lands after the CTA exits
        volatile int no_abort = 0;
        for (long long i = issued > n_st ? issued - n_st : 0; i < issued; ++i)
          mbar_wait(full_bar(static_cast<uint32_t>(i % n_st)),
                    static_cast<uint32_t>((i / n_st) & 1), &no_abort, p.status);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(kFM, kFN);
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
            tc_mma_e4m3(tmem + acc * kFN, ad + 2 * k, bd + 2 * k, idesc, k > 0 ? 1u : 0u);
          tc_commit(empty_bar(stage));
          tc_commit(tfull_bar(acc));
          if (++stage == n_st) {
            stage = 0;
            phase ^= 1u;
          }
          if (++acc == kFAccs) {
            acc = 0;
            aphase ^= 1u;
          }
        }
      }
    }
  } else {
    const int pw = warp - 2;
    const int grp = pw >> 2;
    const int lanes0 = 32 * (warp & 3);  // the TMEM lanes this warp may read
    uint32_t* stg = staging + pw * 32 * kFStageRow;
    uint32_t acc = 0, aphase = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < p.n_units && ok; u += gridDim.x) {
      const int n_tile = u / p.n_m, m_tile = u - n_tile * p.n_m;
      const int row0 = m_tile * kFM + lanes0;
      const int row = row0 + lane;
      const bool warp_on = row0 < p.T;
      const float* hs = p.hs + static_cast<int64_t>(min(row, p.T - 1)) * p.KB;
      const float* ws = p.ws + static_cast<int64_t>(n_tile) * p.KB;
      float sum[kFCols];
#pragma unroll
      for (int i = 0; i < kFCols; ++i) sum[i] = 0.f;
      for (int kb = 0; kb < p.KB; ++kb) {
        const float s = __fmul_rn(hs[kb], ws[kb]);
        ok = mbar_wait(tfull_bar(acc), aphase, abort_flag, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (warp_on) {
#pragma unroll
          for (int c = 0; c < kFCols / 32; ++c) {
            uint32_t d[32];
            tmem_ld32_issue(tmem + (static_cast<uint32_t>(lanes0) << 16) + acc * kFN + grp * kFCols +
                                c * 32,
                            d);
            tmem_ld_wait(d);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              sum[c * 32 + i] = __fmaf_rn(__uint_as_float(d[i]), s, sum[c * 32 + i]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty_bar(acc));
        if (++acc == kFAccs) {
          acc = 0;
          aphase ^= 1u;
        }
      }
      if (!ok || !warp_on) continue;
      const int64_t col0 = static_cast<int64_t>(n_tile) * kFN + grp * kFCols;
      if (p.vec) {
        uint16_t* o = p.out + static_cast<int64_t>(row) * p.ld + col0;
#pragma unroll
        for (int j = 0; j < kFCols / 8; ++j) {
          if (row < p.T && col0 + 8 * j + 8 <= p.V) {
            *reinterpret_cast<uint4*>(o + 8 * j) =
                make_uint4(bf16x2_of(sum[8 * j], sum[8 * j + 1]),
                           bf16x2_of(sum[8 * j + 2], sum[8 * j + 3]),
                           bf16x2_of(sum[8 * j + 4], sum[8 * j + 5]),
                           bf16x2_of(sum[8 * j + 6], sum[8 * j + 7]));
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (row < p.T && col0 + 8 * j + i < p.V)
                o[8 * j + i] = static_cast<uint16_t>(bf16x2_of(sum[8 * j + i], 0.f));
          }
        }
      } else {
        // rows at odd addresses: turn 32 columns at a time through shared
        // memory, so that a warp writes consecutive elements of one row
#pragma unroll
        for (int c = 0; c < kFCols / 32; ++c) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            stg[lane * kFStageRow + i] = bf16x2_of(sum[c * 32 + 2 * i], sum[c * 32 + 2 * i + 1]);
          __syncwarp();
          const int64_t col = col0 + c * 32 + lane;
          if (col < p.V) {
            const int n = min(32, p.T - row0);
            for (int r = 0; r < n; ++r)
              p.out[static_cast<int64_t>(row0 + r) * p.ld + col] =
                  reinterpret_cast<const uint16_t*>(stg + r * kFStageRow)[lane];
          }
          __syncwarp();
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
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
      const int64_t want = ceil_div(rows * kb, kQuantThreads / 16);
      const int grid = static_cast<int>(want < 8 * sms ? want : 8 * sms);
      quantize_rows_kernel<<<grid, kQuantThreads, 0, st>>>(x, rows, cols, ld, kb, q, scale);
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
  if (T == 0) return api_set_error(LMH_OK, "");
  if (!hidden_q || !hidden_scale || !weight_q || !weight_scale || !logits)
    return api_set_error(LMH_ERR_INVALID_ARG, "every pointer is required");
  if (misaligned(hidden_q, 16) || misaligned(weight_q, 16) || misaligned(hidden_scale, 4) ||
      misaligned(weight_scale, 4) || misaligned(logits, 2))
    return api_set_error(LMH_ERR_ALIGNMENT,
                         "hidden_q and weight_q need 16-byte, the scales 4-byte, logits 2-byte "
                         "alignment");
  const int64_t n_m = ceil_div(T, kFM), n_n = ceil_div(V, kFN);
  if (n_m * n_n > (1LL << 30))
    return api_set_error(LMH_ERR_INVALID_ARG, "T x V has too many tiles");
  int sms = 0;
  unsigned* status = nullptr;
  int rc = api_device(&sms, &status);
  if (rc != LMH_OK) return rc;
  Fp8Params p{};
  p.T = static_cast<int>(T);
  p.V = static_cast<int>(V);
  p.KB = static_cast<int>(ceil_div(H, kFK));
  p.n_m = static_cast<int>(n_m);
  p.n_n = static_cast<int>(n_n);
  p.n_units = static_cast<int>(n_m * n_n);
  p.a_rows = T < kFM ? static_cast<int>((T + 7) / 8 * 8) : kFM;
  p.hs = hidden_scale;
  p.ws = weight_scale;
  p.out = logits;
  p.ld = ld_logits;
  p.vec = (ld_logits % 8 == 0 && !misaligned(logits, 16)) ? 1 : 0;
  p.status = status;
  CUtensorMap ta, tb;
  if ((rc = api_make_tmap_u8(&ta, hidden_q, H, T, H, kFK, p.a_rows)) != LMH_OK) return rc;
  if ((rc = api_make_tmap_u8(&tb, weight_q, H, V, H, kFK, kFN)) != LMH_OK) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  {
    KernelTimer timer(K_LOGITS_FP8, st);
    e = cudaFuncSetAttribute(logits_fp8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kFSmemBytes);
    if (e == cudaSuccess) {
      const int grid = p.n_units < sms ? p.n_units : sms;
      logits_fp8_kernel<<<grid, kFThreads, kFSmemBytes, st>>>(ta, tb, p);
      e = cudaGetLastError();
    }
    if (e == cudaSuccess) note_launch();
  }
  if (e != cudaSuccess) return launch_error(e, "fp8 logits");
  return api_set_error(LMH_OK, "");
}
