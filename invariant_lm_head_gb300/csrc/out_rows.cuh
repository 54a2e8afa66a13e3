// Finished bf16 logits on their way out of a quantised head's epilogue: a warp's 32
// rows as TMA boxes, or as rows at any address.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>

#include "ptx.cuh"

namespace lmh {

__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint16_t ld_shared_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
// Predicated stores: divergent branches around single stores cost more than they.
__device__ __forceinline__ void st_global_v4_if(uint16_t* at, uint4 v, bool on) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t@p st.global.v4.b32 [%0], {%1, %2, %3, %4};\n\t}" ::
          "l"(at),
      "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(static_cast<int>(on))
      : "memory");
}
__device__ __forceinline__ void st_global_u16_if(uint16_t* at, uint16_t v, bool on) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p st.global.b16 [%0], %1;\n\t}" ::"l"(at),
               "h"(v), "r"(static_cast<int>(on))
               : "memory");
}

// A warp's `rows` (of 32) rows of output, one in each lane as kWords pairs of bf16, to
// rows at any 2-byte address (out + lane * ld), the first n elements of each. A lane
// turns its row, as a ring, by its address's offset in 16 bytes, so that the ring's
// 16-byte chunks are the row's aligned ones; sixteen rows at a time go through 4 KB of
// shared memory, and half a warp writes a row: a chunk a lane, and the first chunk,
// which holds the row's two ends, element by element. T=200 H=3600 V=32003 takes 43.3
// us with it (V=32000, by TMA, 40.3); in boxes of 32 columns, as the 4-byte words that
// they straddle, 53.1: those are 17 writes of parts of a 32-byte sector for 224 bytes.
template <int kWords>
__device__ __forceinline__ void store_rows(uint32_t buf, int lane, uint32_t (&w)[kWords],
                                           uint16_t* out, int64_t ld, int rows, int n) {
  constexpr int kChunks = kWords / 4;
  static_assert(kWords % 4 == 0 && kChunks <= 16, "sixteen rows of 256 bytes");
  {
    const uint32_t off =
        static_cast<uint32_t>(reinterpret_cast<uintptr_t>(out + static_cast<int64_t>(lane) * ld)) & 15u;
    const uint32_t sel = off & 2u ? 0x5432u : 0x7654u;  // by an element
    const uint32_t last = w[kWords - 1];
#pragma unroll
    for (int i = kWords - 1; i > 0; --i) w[i] = __byte_perm(w[i - 1], w[i], sel);
    w[0] = __byte_perm(last, w[0], sel);
#pragma unroll
    for (int by = 1; by <= 2; ++by) {  // by a word, by two
      const bool turn = off & (by == 1 ? 4u : 8u);
      uint32_t end[2] = {w[kWords - by], w[kWords - 1]};
#pragma unroll
      for (int i = kWords - 1; i >= by; --i) w[i] = turn ? w[i - by] : w[i];
#pragma unroll
      for (int i = 0; i < by; ++i) w[i] = turn ? end[i] : w[i];
    }
  }
  const int j = lane & 15;
#pragma unroll 1
  for (int first = 0; first < rows; first += 16) {
    if ((lane & 16) == first) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
        st_shared_v4(buf + j * 256 + ((c ^ (j & 7)) << 4), w[4 * c], w[4 * c + 1], w[4 * c + 2],
                     w[4 * c + 3]);
    }
    __syncwarp();
    uint16_t* o = out + static_cast<int64_t>(first + (lane >> 4)) * ld;
#pragma unroll 4
    for (int i = 0; i < 8; ++i, o += 2 * ld) {
      const int r = 2 * i + (lane >> 4);
      const bool on = first + r < rows;
      const int off = static_cast<int>(reinterpret_cast<uintptr_t>(o) & 15) >> 1;  // elements
      const uint32_t row = buf + r * 256;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (j < kChunks) v = ld_shared_v4(row + ((j ^ (r & 7)) << 4));
      const int e = 8 * j - off;  // the chunk's first element
      st_global_v4_if(o + e, v, on && j < kChunks && e >= 0 && e + 8 <= n);
      // the first chunk, where it is not whole
      const uint16_t x = ld_shared_u16(row + ((r & 7) << 4) + 2 * (j & 7));
      const int ex = j >= off ? j - off : 2 * kWords + j - off;
      st_global_u16_if(o + ex, x, on && j < 8 && (off != 0 || n < 8) && ex < n);
      if (n < 2 * kWords) {  // the vocabulary's end: the chunk that it parts
        const int c = (off + n) >> 3;
        const int el = 8 * c + j - off;
        if (c > 0 && c < kChunks && j < 8)
          st_global_u16_if(o + el, ld_shared_u16(row + ((c ^ (r & 7)) << 4) + 2 * j), on && el < n);
      }
    }
    __syncwarp();
  }
}
// One row's 32 columns as bf16 into a 32 x 32 box with 64-byte swizzle (16-byte
// chunk j of row r at j ^ ((r / 2) % 4)), as the TMA store reads it.
__device__ __forceinline__ void stage_box_row(uint32_t buf, int r, const float* v) {
  const uint32_t row = buf + static_cast<uint32_t>(r) * 64u;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                     row + ((static_cast<uint32_t>(j) ^ ((r >> 1) & 3)) << 4)),
                 "r"(bf16x2_of(v[8 * j], v[8 * j + 1])), "r"(bf16x2_of(v[8 * j + 2], v[8 * j + 3])),
                 "r"(bf16x2_of(v[8 * j + 4], v[8 * j + 5])),
                 "r"(bf16x2_of(v[8 * j + 6], v[8 * j + 7]))
                 : "memory");
}

}  // namespace lmh
