// The norm before the head (sm_103a): residual addition, RMS norm and block
// quantisation to e4m3 in one pass, as lmhead_logits_fp8 takes its hidden states.
//
// For a row, with w the norm's weight,
//   h = bf16(x + residual)   (h = x without a residual)
//   r = 1 / sqrt(mean(h^2) + eps)
//   y = h * r * w
// and per 128 columns a = max(max |y|, 2^-60), scale = a / 448, q = e4m3(y * 448 / a).
//
// The row's factor r is in both y and a and cancels: q = e4m3(u * 448 / max |u|) with u
// = h * w, which is exact in fp32 (8 + 8 bits). u * 448 has 19 significant bits and max
// |u| 16, so a quotient that is not halfway between two e4m3 values (5 bits) is at least
// 2^-21 away from halfway, relatively, and the correctly rounded fp32 quotient settles
// every rounding as exact arithmetic would. Only the scale carries r's error. Blocks
// outside that argument's range (below the floor, products that leave fp32's normal
// range, infinities, NaN) take y itself, rounded.
//
// Batch invariance: the order of a row's sum depends on H alone.
#include <atomic>
#include <cstdint>
#include <cstdio>

#include <cuda_bf16.h>

#include "fp8_block.cuh"
#include "internal.h"
#include "launch.cuh"
#include "lmhead.h"
#include "out_rows.cuh"
#include "ptx.cuh"

namespace lmh {

namespace {

constexpr int kNBlock = 128;   // columns of a scale
constexpr int kNLanes = 8;     // lanes of a block, 16 elements each
constexpr int kNMaxSmem = 131072;  // 32768 columns one row at a time, 16384 two
constexpr int kNMaxCols = 32768;  // four units of each of 512 threads

struct NormParams {
  const uint16_t *x, *residual, *weight;
  int64_t rows, ld_x, ld_res, ld_out;
  int cols, kb;
  float eps;
  float low;  // smaller sums of squares are taken again in smaller units
  uint16_t* out_residual;
  uint8_t* q;
  float* scale;
};

__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  return bf16x2_of(__uint_as_float(a << 16) + __uint_as_float(b << 16),
                   __uint_as_float(a & 0xffff0000u) + __uint_as_float(b & 0xffff0000u));
}

__device__ __forceinline__ f32x2 widen(uint32_t w) {
  return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// The sum over the CTA, in every thread: within each warp, then the warps in order.
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  const int warps = blockDim.x >> 5;
  for (int w = 0; w < warps; ++w) s += part[w];
  return s;
}

// One row a CTA at a time, in a grid that stays. Thread t holds, for unit i < kU, 16
// elements of block (t + i * blockDim.x) / 8: two runs of 8 (16 bytes), 64 columns apart,
// so that a block's scale is worked out by 8 lanes. Each thread copies its own share of
// the CTA's next kD - 1 rows to shared memory while it works on one (no barrier: no
// other thread reads it), since the barrier of the row's sum would leave the memory idle.
//
// What bounds it: HBM. 90 us at 16384 x 5120 with a residual (7 bytes an element), 6.5
// TB/s, 0.97 of the copy rate (94 to 97 where nothing is launched behind it); loads into
// registers at each row's start 104 us, the same with 16 elements a thread and 320
// threads 119. The grid is what the SMs hold at once: one CTA an SM more 117 us. One row
// of 4096 takes 4.3 us, a load, a sum and a store one after the other. Past 16384 columns
// a row fills the shared memory (kD = 1: none ahead) and 64 elements a thread spill: 4096 x
// 20000 158 us, 3.6 TB/s, 2048 x 32768 100 us, 4.7 TB/s; 4096 x 16384 70 us, 6.7.
template <int kU, int kD>
__global__ void __launch_bounds__(kU == 1 ? 256 : 512) norm_fp8_kernel(const NormParams p) {
  extern __shared__ __align__(16) uint8_t ahead[];
  __shared__ float part[3][32];
  ahead_done();
  const int sub = threadIdx.x & (kNLanes - 1);
  int col[kU];
  uint4 w[kU][2];
#pragma unroll
  for (int i = 0; i < kU; ++i) {
    const int blk = (threadIdx.x + i * blockDim.x) / kNLanes;
    col[i] = blk < p.kb ? blk * kNBlock + sub * 8 : p.cols;
  }
  const uint32_t slots = smem_u32(ahead) + threadIdx.x * 16;
  auto slot = [&](int d, int which, int i, int h) {
    return slots + static_cast<uint32_t>((((d * 2 + which) * kU + i) * 2 + h) * blockDim.x * 16);
  };
  auto fetch = [&](int64_t row, int d) {
    if (row < p.rows) {
#pragma unroll
      for (int i = 0; i < kU; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (col[i] + 64 * h < p.cols) {
            copy16_async(slot(d, 0, i, h), p.x + row * p.ld_x + col[i] + 64 * h);
            if (p.residual)
              copy16_async(slot(d, 1, i, h), p.residual + row * p.ld_res + col[i] + 64 * h);
          }
    }
    copies_commit();  // an empty one too: the groups are counted
  };
#pragma unroll
  for (int d = 0; d < kD - 1; ++d) fetch(blockIdx.x + static_cast<int64_t>(d) * gridDim.x, d);
#pragma unroll
  for (int i = 0; i < kU; ++i) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w[i][h] = make_uint4(0u, 0u, 0u, 0u);
      if (col[i] + 64 * h < p.cols)
        w[i][h] = *reinterpret_cast<const uint4*>(p.weight + col[i] + 64 * h);
    }
  }
  int parity = 0, depth = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, parity ^= 1) {
    if (row + gridDim.x >= p.rows) nearly_done();
    fetch(row + static_cast<int64_t>(kD - 1) * gridDim.x, depth == 0 ? kD - 1 : depth - 1);
    copies_wait<kD - 1>();
    uint4 v[kU][2];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        v[i][h] = make_uint4(0u, 0u, 0u, 0u);
        if (col[i] + 64 * h < p.cols) {
          v[i][h] = ld_shared_v4(slot(depth, 0, i, h));
          if (p.residual) {
            const uint4 r = ld_shared_v4(slot(depth, 1, i, h));
            v[i][h].x = add_bf16x2(v[i][h].x, r.x);
            v[i][h].y = add_bf16x2(v[i][h].y, r.y);
            v[i][h].z = add_bf16x2(v[i][h].z, r.z);
            v[i][h].w = add_bf16x2(v[i][h].w, r.w);
            if (p.out_residual)
              *reinterpret_cast<uint4*>(p.out_residual + row * p.ld_out + col[i] + 64 * h) = v[i][h];
          }
        }
      }
    }
    if (++depth == kD) depth = 0;
    auto squares = [&](float factor) {
      f32x2 s2 = f2_pack(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kU; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t ws[4] = {v[i][h].x, v[i][h].y, v[i][h].z, v[i][h].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const f32x2 f = f2_mul(widen(ws[k]), f2_pack(factor, factor));
            s2 = f2_fma(f, f, s2);
          }
        }
      }
      float lo, hi;
      f2_unpack(s2, lo, hi);
      return lo + hi;
    };
    const float n = static_cast<float>(p.cols);
    const float sum = row_sum(squares(1.f), part[parity]);
    float r;
    if (sum >= p.low && sum < INFINITY) {
      r = __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, n), p.eps));
    } else {
      // squares past fp32 (or an infinity or a NaN): the row in units of 2^80; squares that
      // underflow beside an eps that is no normal number: in units of 2^-64
      const float unit = sum < p.low ? 0x1p64f : 0x1p-80f;
      const float scaled = row_sum(squares(unit), part[2]);
      r = __frsqrt_rn(__fadd_rn(__fdiv_rn(scaled, n), p.eps * unit * unit)) * unit;
      __syncthreads();  // part[2] is free for the next such row
    }
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      f32x2 u[8];
      uint32_t most = 0u;  // the largest |u|, as bits (a NaN is above inf)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t hs[4] = {v[i][h].x, v[i][h].y, v[i][h].z, v[i][h].w};
        const uint32_t ws[4] = {w[i][h].x, w[i][h].y, w[i][h].z, w[i][h].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          u[4 * h + k] = f2_mul(widen(hs[k]), widen(ws[k]));
          float lo, hi;
          f2_unpack(u[4 * h + k], lo, hi);
          most = max(most, max(__float_as_uint(lo) & 0x7fffffffu, __float_as_uint(hi) & 0x7fffffffu));
        }
      }
#pragma unroll
      for (int off = kNLanes / 2; off > 0; off >>= 1)
        most = max(most, __shfl_xor_sync(0xffffffffu, most, off));
      const float au = __uint_as_float(most), a = __fmul_rn(au, r);
      const bool usual = au >= 0x1p-100f && au <= 0x1p100f && a >= 0x1p-60f && a <= 0x1p100f;
      BlockScale s;
      if (usual) {
        s = block_scale(au);
        s.scale = __fdiv_rn(a, 448.f);
      }
      if (__any_sync(0xffffffffu, !usual)) {
        uint32_t top = 0u;
        f32x2 y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint4& hv = v[i][k >> 2];
          const uint4& wv = w[i][k >> 2];
          const uint32_t hw = (k & 3) == 0 ? hv.x : (k & 3) == 1 ? hv.y : (k & 3) == 2 ? hv.z : hv.w;
          const uint32_t ww = (k & 3) == 0 ? wv.x : (k & 3) == 1 ? wv.y : (k & 3) == 2 ? wv.z : wv.w;
          y[k] = f2_mul(f2_mul(widen(hw), f2_pack(r, r)), widen(ww));
          float lo, hi;
          f2_unpack(y[k], lo, hi);
          top = max(top, max(__float_as_uint(lo) & 0x7fffffffu, __float_as_uint(hi) & 0x7fffffffu));
        }
#pragma unroll
        for (int off = kNLanes / 2; off > 0; off >>= 1)
          top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
        if (!usual) {
          s = top >= 0x7f800000u ? block_scale_nan(__uint_as_float(top))
                                 : block_scale(fmaxf(__uint_as_float(top), 0x1p-60f));
#pragma unroll
          for (int k = 0; k < 8; ++k) u[k] = y[k];
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint2 o;
        o.x = quantize2(u[4 * h], s) | (quantize2(u[4 * h + 1], s) << 16);
        o.y = quantize2(u[4 * h + 2], s) | (quantize2(u[4 * h + 3], s) << 16);
        if (col[i] + 64 * h < p.cols)
          *reinterpret_cast<uint2*>(p.q + row * p.cols + col[i] + 64 * h) = o;
      }
      if (sub == 0 && col[i] < p.cols) p.scale[row * p.kb + col[i] / kNBlock] = s.scale;
    }
  }
}

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

// Units of 16 elements of a thread, by the row's length alone: the sum's order follows.
template <int kU, int kD>
cudaError_t launch_norm(const NormParams& p, int sms, cudaStream_t st) {
  const int units = p.kb * kNLanes;
  const int warps = ((units + kU - 1) / kU + 31) / 32, threads = 32 * warps;
  const int bytes = kD * 2 * kU * 2 * threads * 16;
  // CTAs that an SM holds, by the CTA's warps, and the kernel's shared-memory attribute:
  // the device's, looked up by its first call of that length.
  static std::atomic<int> per_sm[64][17];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int n = per_sm[dev][warps].load(std::memory_order_acquire);
  if (n == 0) {
    if ((e = cudaFuncSetAttribute(norm_fp8_kernel<kU, kD>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize, kNMaxSmem)) !=
            cudaSuccess ||
        (e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, norm_fp8_kernel<kU, kD>, threads,
                                                           bytes)) != cudaSuccess)
      return e;
    if (n < 1) return cudaErrorInvalidConfiguration;
    per_sm[dev][warps].store(n, std::memory_order_release);
  }
  const int64_t most = static_cast<int64_t>(sms) * n;  // a persistent grid
  const unsigned grid = static_cast<unsigned>(p.rows < most ? p.rows : most);
  return launch_early(norm_fp8_kernel<kU, kD>, grid, threads, bytes, st, 1, p);
}

}  // namespace

}  // namespace lmh

extern "C" int lmhead_rmsnorm_fp8(const uint16_t* x, const uint16_t* residual,
                                  const uint16_t* weight, int64_t rows, int64_t cols, int64_t ld_x,
                                  int64_t ld_residual, float eps, uint16_t* out_residual,
                                  int64_t ld_out_residual, uint8_t* q, float* scale,
                                  struct CUstream_st* stream) {
  using namespace lmh;
  if (rows < 0 || rows > LMH_MAX_DIM || cols < 1 || cols > kNMaxCols)
    return api_set_error(LMH_ERR_INVALID_ARG, "rows out of range, or cols out of [1, 32768]");
  if (!(eps > 0.f && eps <= 3.402823466e38f))
    return api_set_error(LMH_ERR_INVALID_ARG, "eps must be finite and > 0");
  if (ld_x < cols || (residual && ld_residual < cols) || (out_residual && ld_out_residual < cols))
    return api_set_error(LMH_ERR_INVALID_ARG, "a row distance must be at least cols");
  if (out_residual && !residual)
    return api_set_error(LMH_ERR_INVALID_ARG, "out_residual needs a residual");
  if (cols % 16 != 0 || ld_x % 8 != 0 || (residual && ld_residual % 8 != 0) ||
      (out_residual && ld_out_residual % 8 != 0))
    return api_set_error(LMH_ERR_ALIGNMENT,
                         "cols must be a multiple of 16 and the row distances of 8");
  if (rows == 0) return api_set_error(LMH_OK, "");
  if (!x || !weight || !q || !scale)
    return api_set_error(LMH_ERR_INVALID_ARG, "x, weight, q and scale are required");
  if (misaligned(x, 16) || misaligned(residual, 16) || misaligned(weight, 16) ||
      misaligned(out_residual, 16) || misaligned(q, 16) || misaligned(scale, 4))
    return api_set_error(LMH_ERR_ALIGNMENT, "scale needs 4-byte, the rest 16-byte alignment");
  int sms = 0;
  unsigned* status = nullptr;
  const int rc = api_device(&sms, &status);
  if (rc != LMH_OK) return rc;
  NormParams p{};
  p.x = x;
  p.residual = residual;
  p.weight = weight;
  p.rows = rows;
  p.ld_x = ld_x;
  p.ld_res = ld_residual;
  p.ld_out = ld_out_residual;
  p.cols = static_cast<int>(cols);
  p.kb = static_cast<int>((cols + kNBlock - 1) / kNBlock);
  p.eps = eps;
  // a square's underflow is off by 2^-150: next to nothing beside any normal eps
  p.low = eps < 0x1p-126f ? 0x1p-60f : 0.f;
  p.out_residual = out_residual;
  p.q = q;
  p.scale = scale;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  {
    KernelTimer timer(K_NORM_FP8, st);
    // rows ahead as shared memory allows
    if (cols <= 4096)
      e = launch_norm<1, 3>(p, sms, st);
    else if (cols <= 8192)
      e = launch_norm<2, 3>(p, sms, st);
    else if (cols <= 16384)
      e = launch_norm<2, 2>(p, sms, st);
    else
      e = launch_norm<4, 1>(p, sms, st);
    if (e == cudaSuccess) note_launch();
  }
  if (e != cudaSuccess) {
    char msg[256];
    snprintf(msg, sizeof(msg), "norm: %s", cudaGetErrorString(e));
    return api_set_error(LMH_ERR_LAUNCH, msg);
  }
  return api_set_error(LMH_OK, "");
}
