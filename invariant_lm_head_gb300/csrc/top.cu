// What a server reports beside a token (sm_103a): the log-probs of given tokens, the
// entropy, and the likeliest alternatives, from bf16 logits.
//
// For a row x with temperature t (0 counts as 1), z = x / t, m = max z,
//   logprob[i] = z[i] - m - log sum exp(z - m),   entropy = log sum - sum e (z - m) / sum,
// one pass with a running maximum (base 2: y = x * c, c = log2(e) / t rounded once, and
// y - m one FMA). Masked logits (-inf, NaN) weigh nothing, in the entropy either.
//
// The alternatives are the first n in descending order of x, equal ones by index. The
// pass over the row only keeps each thread's largest value: the n-th largest of those is
// reached by n tokens at least, so every alternative reaches it, and only the threads
// whose largest value does (n of them, or a few more) have their share of the row looked
// at again. The tokens found there, n and a few more, are ranked by counting. Where
// more tokens reach it than the list holds (equal logits), the n-th largest value is
// found by bisection over the 16-bit keys, counting over the row.
//
// A row is taken by a cluster of CTAs whose number depends on V alone, each with its
// slice; the first CTA merges their sums in order, and their lists.
//
// Batch invariance: the split and the order of every sum depend on V alone.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdio>

#include <cuda_bf16.h>

#include "internal.h"
#include "lmhead.h"
#include "online_softmax.cuh"
#include "ptx.cuh"

namespace lmh {

namespace {

typedef unsigned long long u64;

constexpr int kPThreads = 256;
constexpr int kPWarps = kPThreads / 32;
constexpr int kPMaxTop = 128;   // most alternatives
constexpr int kPMaxC = 4;       // most CTAs of a row
constexpr int kPList = 1024;    // tokens of a CTA's list
static_assert(kPMaxTop <= kPThreads, "a thread's largest value for each alternative");
constexpr float kPFloor = -200.f;  // 2^-200 is 0: what masked and far values are cut to

struct TopParams {
  const uint16_t* logits;
  int64_t T, V, ld;
  float temperature;
  const float* row_t;
  const int32_t* tokens;
  int n_tokens, n_top;
  float* out_logprob;
  float* out_entropy;
  int32_t* top_token;
  float* top_logprob;
};

// A CTA's sums, and the largest logit of its slice (-inf: all masked).
struct SliceStat {
  float m, s, u, most;
};

struct TopShared {
  u64 list[kPList];
  u64 merged[kPMaxC * kPMaxTop];  // CTA 0: every CTA's best, in order; 0 where it has none
  SliceStat slice[kPMaxC];        // CTA 0
  SliceStat warp[kPWarps];
  uint16_t key[kPThreads];
  uint16_t hit[kPThreads];
  uint32_t count[kPWarps];
  uint32_t bar;                   // the key that alternatives reach
  int n_hit, n_list;
};

// 16 bits in the order of the values: 0 for a masked logit, and equal zeros.
__device__ __forceinline__ uint32_t order_key(uint32_t b) {
  if ((b & 0x7fffu) > 0x7f80u || b == 0xff80u) return 0u;
  if (b == 0x8000u) b = 0u;
  return b & 0x8000u ? 0xffffu - b : b + 0x8000u;
}
__device__ __forceinline__ float value_of_key(uint32_t k) {
  const uint32_t b = k >= 0x8000u ? k - 0x8000u : 0xffffu - k;
  return __uint_as_float(b << 16);
}
// A token in the order of the list: its key, then the lower index.
__device__ __forceinline__ u64 entry_of(uint32_t key, int64_t index) {
  return (static_cast<u64>(key) << 32) | (0xffffffffu - static_cast<uint32_t>(index));
}

constexpr uint32_t kMasked2 = 0xff80ff80u;  // two -inf

// Vector v (elements [8 v, 8 v + 8)) of a row at any address, -inf past its end. A row
// that does not start on 16 bytes is read in the aligned 16 bytes that hold the vector,
// but for its two ends, so that nothing outside the row is.
template <bool kAligned>
__device__ __forceinline__ uint4 load_vector(const uint16_t* row, int64_t V, int64_t v) {
  const uint16_t* at = row + 8 * v;
  if (kAligned && 8 * v + 8 <= V) return *reinterpret_cast<const uint4*>(at);
  if (!kAligned && v > 0 && 8 * v + 16 <= V) {
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at) & 15);
    const uint4* g = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(at) & ~uintptr_t{15});
    const uint4 a = g[0], b = g[1];
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (off & 8u) {
#pragma unroll
      for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (off & 4u) {
#pragma unroll
      for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    if (off & 2u) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  uint32_t w[4] = {kMasked2, kMasked2, kMasked2, kMasked2};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = 8 * v + i < V ? at[i] : 0xff80u;
    w[i / 2] = i & 1 ? (w[i / 2] & 0xffffu) | (b << 16) : (w[i / 2] & 0xffff0000u) | b;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ __nv_bfloat162 bf2(uint32_t w) {
  return *reinterpret_cast<const __nv_bfloat162*>(&w);
}

// Folds 32 values into the state; `most` keeps the largest value.
__device__ __forceinline__ void fold32(OnlineStat& st, float& most, const uint4 (&w)[4], float c) {
  __nv_bfloat162 m2 = bf2(kMasked2);  // a NaN is passed over
#pragma unroll
  for (int k = 0; k < 4; ++k)
    m2 = __hmax2(m2, __hmax2(__hmax2(bf2(w[k].x), bf2(w[k].y)), __hmax2(bf2(w[k].z), bf2(w[k].w))));
  const float gmax = fmaxf(__low2float(m2), __high2float(m2));
  most = fmaxf(most, gmax);
  // never -inf, from which a finite x * c would be infinitely far
  const float mn = fmaxf(fmaxf(st.m, __fmul_rn(gmax, c)), -3.402823466e38f);
  const float d0 = fmaxf(__fsub_rn(st.m, mn), kPFloor);
  const float a = ex2(d0);
  f32x2 s2 = f2_pack(0.f, 0.f), u2 = s2;
  const f32x2 c2 = f2_pack(c, c), nm2 = f2_pack(-mn, -mn);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t ws[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float da, db;
      f2_unpack(f2_fma(bf16x2_f2(ws[q]), c2, nm2), da, db);
      da = fmaxf(da, kPFloor);  // a NaN (a masked value) too
      db = fmaxf(db, kPFloor);
      const f32x2 e2 = f2_pack(ex2(da), ex2(db));
      s2 = f2_add(s2, e2);
      u2 = f2_fma(e2, f2_pack(da, db), u2);
    }
  }
  float s0, s1, u0, u1;
  f2_unpack(s2, s0, s1);
  f2_unpack(u2, u0, u1);
  st.u = __fadd_rn(__fmul_rn(a, __fmaf_rn(st.s, d0, st.u)), __fadd_rn(u0, u1));
  st.s = __fadd_rn(__fmul_rn(st.s, a), __fadd_rn(s0, s1));
  st.m = mn;
}

__device__ __forceinline__ void merge_slice(SliceStat& a, const SliceStat& b) {
  OnlineStat x{a.m, a.s, a.u, 0.f};
  stat_merge(x, OnlineStat{b.m, b.s, b.u, 0.f});
  a = SliceStat{x.m, x.s, x.u, fmaxf(a.most, b.most)};
}

// How many values of the slice have a key of at least k, in every thread.
template <bool kAligned>
__device__ __noinline__ uint32_t count_from(const uint16_t* row, int64_t V, int64_t v0, int64_t v1,
                                            uint32_t k, uint32_t* part) {
  uint32_t n = 0;
  for (int64_t v = v0 + threadIdx.x; v < v1; v += kPThreads) {
    const uint4 x = load_vector<kAligned>(row, V, v);
    const uint32_t ws[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) n += order_key(ws[i / 2] >> (16 * (i & 1)) & 0xffffu) >= k;
  }
  n = __reduce_add_sync(0xffffffffu, n);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = n;
  __syncthreads();
  n = 0;
  for (int w = 0; w < kPWarps; ++w) n += part[w];
  __syncthreads();
  return n;
}

// The slice's first n tokens into sh.list, exactly n: those above the n-th largest key,
// and of those that have it the first by index. At least n tokens are not masked.
template <bool kAligned>
__device__ __noinline__ void list_by_bisection(TopShared& sh, const uint16_t* row, int64_t V,
                                               int64_t v0, int64_t v1, int n) {
  uint32_t lo = 1, hi = 0x10000u;  // count(lo) >= n > count(hi)
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) / 2;
    if (count_from<kAligned>(row, V, v0, v1, mid, sh.count) >= static_cast<uint32_t>(n))
      lo = mid;
    else
      hi = mid;
  }
  const int above = static_cast<int>(count_from<kAligned>(row, V, v0, v1, lo + 1, sh.count));
  if (threadIdx.x == 0) sh.n_list = 0;
  __syncthreads();
  int taken = above;  // list places given to equal ones start here
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int64_t base = v0; base < v1; base += kPThreads) {
    const int64_t v = base + threadIdx.x;
    uint32_t ws[4] = {kMasked2, kMasked2, kMasked2, kMasked2};
    if (v < v1) {
      const uint4 x = load_vector<kAligned>(row, V, v);
      ws[0] = x.x;
      ws[1] = x.y;
      ws[2] = x.z;
      ws[3] = x.w;
    }
    uint32_t equal = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t k = order_key(ws[i / 2] >> (16 * (i & 1)) & 0xffffu);
      equal += k == lo;
      if (k > lo) {
        const int at = atomicAdd(&sh.n_list, 1);
        if (at < above) sh.list[at] = entry_of(k, 8 * v + i);
      }
    }
    // places of the equal ones, in order of index
    uint32_t before = equal;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, before, off);
      if (lane >= off) before += o;
    }
    if (lane == 31) sh.count[warp] = before;
    __syncthreads();
    uint32_t total = 0, ahead = 0;
    for (int w = 0; w < kPWarps; ++w) {
      if (w < warp) ahead += sh.count[w];
      total += sh.count[w];
    }
    uint32_t at = static_cast<uint32_t>(taken) + ahead + before - equal;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t k = order_key(ws[i / 2] >> (16 * (i & 1)) & 0xffffu);
      if (k == lo) {
        if (at < static_cast<uint32_t>(n)) sh.list[at] = entry_of(k, 8 * v + i);
        ++at;
      }
    }
    taken = static_cast<int>(min(static_cast<uint32_t>(n), taken + total));
    __syncthreads();
  }
  if (threadIdx.x == 0) sh.n_list = n;
  __syncthreads();
}

// z - max z where y = x * c is too large to be subtracted from.
__device__ __forceinline__ float far_shift(float x, float most, float t) {
  return x == most ? 0.f : __fdiv_rn(__fsub_rn(x, most), t);
}

// The sums of such a row: logits equal to the largest weigh 1. One CTA, in an order
// fixed by V.
__device__ __noinline__ SliceStat sums_of_extremes(TopShared& sh, const uint16_t* row, int64_t V,
                                                   float t, float most) {
  float s = 0.f, u = 0.f;
  for (int64_t i = threadIdx.x; i < V; i += kPThreads) {
    const float x = __uint_as_float(static_cast<uint32_t>(row[i]) << 16);
    const float d = fmaxf(__fmul_rn(far_shift(x, most, t), kLog2e), kPFloor);
    const float e = ex2(d);
    s += e;
    u += e * d;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, off);
    u += __shfl_xor_sync(0xffffffffu, u, off);
  }
  if ((threadIdx.x & 31) == 0) sh.warp[threadIdx.x >> 5] = SliceStat{0.f, s, u, most};
  __syncthreads();
  SliceStat r{0.f, 0.f, 0.f, most};
  for (int w = 0; w < kPWarps; ++w) {
    r.s += sh.warp[w].s;
    r.u += sh.warp[w].u;
  }
  return r;
}

template <int kC>
__device__ __forceinline__ uint32_t first_cta(const void* here) {
  return kC > 1 ? mapa_shared(smem_u32(here), 0u) : smem_u32(here);
}

template <int kC, bool kAligned>
__global__ void __launch_bounds__(kPThreads, 4) top_logprobs_kernel(const TopParams p) {
  __shared__ __align__(16) TopShared sh;
  const int64_t row = blockIdx.x / kC;
  const int rank = kC > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const uint16_t* x = p.logits + row * p.ld;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // this CTA's vectors: whole runs of 32, but for the row's end
  const int64_t n_vec = (p.V + 7) / 8;
  const int64_t per = ((n_vec + kC - 1) / kC + 31) / 32 * 32;
  const int64_t v0 = min(n_vec, per * rank), v1 = min(n_vec, v0 + per);

  float t = p.row_t ? p.row_t[row] : p.temperature;
  if (t == 0.f) t = 1.f;
  const bool valid_t = t > 0.f && t <= 3.402823466e38f;
  if (!valid_t) t = 1.f;
  const float c = __fdiv_rn(kLog2e, t);
  if (threadIdx.x == 0) sh.n_hit = sh.n_list = 0;

  OnlineStat st = stat_empty();
  float most = -INFINITY;
  for (int64_t v = v0 + threadIdx.x; v < v1; v += 4 * kPThreads) {
    uint4 w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      w[k] = make_uint4(kMasked2, kMasked2, kMasked2, kMasked2);
      if (v + k * kPThreads < v1) w[k] = load_vector<kAligned>(x, p.V, v + k * kPThreads);
    }
    fold32(st, most, w, c);
  }
  sh.key[threadIdx.x] = static_cast<uint16_t>(order_key(__float_as_uint(most) >> 16));
  SliceStat mine{st.m, st.s, st.u, most};
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    SliceStat o;
    o.m = __shfl_down_sync(0xffffffffu, mine.m, off);
    o.s = __shfl_down_sync(0xffffffffu, mine.s, off);
    o.u = __shfl_down_sync(0xffffffffu, mine.u, off);
    o.most = __shfl_down_sync(0xffffffffu, mine.most, off);
    if (lane + off < 32) merge_slice(mine, o);
  }
  if (lane == 0) sh.warp[warp] = mine;
  __syncthreads();

  const int n = p.n_top;
  if (warp == 1 && lane == 0) {
    SliceStat r = sh.warp[0];
    for (int w = 1; w < kPWarps; ++w) merge_slice(r, sh.warp[w]);
    const uint32_t at = first_cta<kC>(&sh.slice[rank]);
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(r.m), "f"(r.s),
                 "f"(r.u), "f"(r.most)
                 : "memory");
  }
  if (warp == 0 && n > 0) {
    // the n-th largest of the threads' keys, by bisection (1 where fewer are not masked)
    uint32_t k[kPThreads / 32];
#pragma unroll
    for (int i = 0; i < kPThreads / 32; ++i) k[i] = sh.key[lane + 32 * i];
    uint32_t bar = 0;
#pragma unroll 1
    for (uint32_t bit = 0x8000u; bit > 0; bit >>= 1) {
      uint32_t reach = 0;
#pragma unroll
      for (int i = 0; i < kPThreads / 32; ++i) reach += k[i] >= (bar | bit);
      if (__reduce_add_sync(0xffffffffu, reach) >= static_cast<uint32_t>(n)) bar |= bit;
    }
    bar = max(bar, 1u);
    int base = 0;
#pragma unroll
    for (int i = 0; i < kPThreads / 32; ++i) {
      const uint32_t on = __ballot_sync(0xffffffffu, k[i] >= bar);
      if (k[i] >= bar)
        sh.hit[base + __popc(on & ((1u << lane) - 1u))] = static_cast<uint16_t>(lane + 32 * i);
      base += __popc(on);
    }
    if (lane == 0) {
      sh.bar = bar;
      sh.n_hit = base;
    }
  }
  __syncthreads();

  if (n > 0) {
    const uint32_t bar = sh.bar;
    const int64_t share = (v1 - v0 + kPThreads - 1) / kPThreads;
    const int64_t looks = share * sh.n_hit;
    for (int64_t i = threadIdx.x; i < looks; i += kPThreads) {
      const int64_t v = v0 + sh.hit[i / share] + (i % share) * kPThreads;
      if (v >= v1) continue;
      const uint4 w = load_vector<kAligned>(x, p.V, v);
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t k = order_key(ws[e / 2] >> (16 * (e & 1)) & 0xffffu);
        if (k >= bar) {
          const int at = atomicAdd(&sh.n_list, 1);
          if (at < kPList) sh.list[at] = entry_of(k, 8 * v + e);
        }
      }
    }
    __syncthreads();
    if (sh.n_list > kPList) list_by_bisection<kAligned>(sh, x, p.V, v0, v1, n);
    const int found = sh.n_list;
    // the first n of them, in order, to the first CTA
    const uint32_t to = first_cta<kC>(&sh.merged[rank * kPMaxTop]);
    for (int i = threadIdx.x; i < found; i += kPThreads) {
      const u64 me = sh.list[i];
      int r = 0;
      for (int j = 0; j < found; ++j) r += sh.list[j] > me;
      if (r < n)
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to + 8u * r), "l"(me) : "memory");
    }
    for (int i = found + threadIdx.x; i < n; i += kPThreads)
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to + 8u * i), "l"(u64{0}) : "memory");
  }
  if (kC > 1) {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    if (rank != 0) return;
  } else {
    __syncthreads();
  }

  SliceStat all = sh.slice[0];
  for (int k = 1; k < kC; ++k) merge_slice(all, sh.slice[k]);
  // The largest y itself is shifted by its product's rounding, up to 2^-4 at 2^20; past
  // that (or where the largest logit is +inf) the row is summed again.
  const bool extreme = all.most > -INFINITY && !(fabsf(__fmul_rn(all.most, c)) <= 0x1p20f);
  if (extreme) all = sums_of_extremes(sh, x, p.V, t, all.most);
  const bool nothing = !(all.most > -INFINITY);
  const float l2s = log2f(all.s);
  const float bad = __int_as_float(0x7fffffff);
  auto logprob = [&](float v) -> float {
    if (!valid_t) return bad;
    if (nothing || !(v > -INFINITY)) return -INFINITY;  // a masked one
    const float d = __fmaf_rn(v, c, -all.m);
    if (extreme || d == -INFINITY)  // in base e what base 2 may not hold
      return __fsub_rn(far_shift(v, all.most, t), __fmul_rn(kLn2, l2s));
    return __fmul_rn(kLn2, __fsub_rn(d, l2s));
  };
  if (threadIdx.x == 0 && p.out_entropy)
    p.out_entropy[row] = !valid_t ? bad
                         : nothing ? 0.f
                                   : __fmul_rn(kLn2, __fsub_rn(l2s, __fdiv_rn(all.u, all.s)));
  for (int i = threadIdx.x; i < p.n_tokens; i += kPThreads) {
    const int32_t id = p.tokens[row * p.n_tokens + i];
    float lp = valid_t ? 0.f : bad;
    if (id >= 0 && id < p.V) lp = logprob(__uint_as_float(static_cast<uint32_t>(x[id]) << 16));
    p.out_logprob[row * p.n_tokens + i] = lp;
  }
  for (int i = threadIdx.x; i < kC * n; i += kPThreads) {
    const u64 me = sh.merged[i / n * kPMaxTop + i % n];
    int r = 0, total = 0;
    for (int k = 0; k < kC; ++k) {
      for (int j = 0; j < n; ++j) {
        const u64 o = sh.merged[k * kPMaxTop + j];
        r += o > me;
        total += o != 0;
      }
    }
    if (me != 0 && r < n && valid_t) {
      p.top_token[row * n + r] = static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(me));
      p.top_logprob[row * n + r] = logprob(value_of_key(static_cast<uint32_t>(me >> 32)));
    }
    if (i < n && (i >= total || !valid_t)) {
      p.top_token[row * n + i] = -1;
      p.top_logprob[row * n + i] = valid_t ? -INFINITY : bad;
    }
  }
}

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

template <int kC, bool kAligned>
cudaError_t launch_top(const TopParams& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.T * kC));
  cfg.blockDim = dim3(kPThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = kC;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, top_logprobs_kernel<kC, kAligned>, p);
}

template <bool kAligned>
cudaError_t launch_by_vocabulary(const TopParams& p, cudaStream_t st) {
  if (p.V > 65536) return launch_top<4, kAligned>(p, st);
  if (p.V > 16384) return launch_top<2, kAligned>(p, st);
  return launch_top<1, kAligned>(p, st);
}

}  // namespace

}  // namespace lmh

extern "C" int lmhead_top_logprobs(const uint16_t* logits, int64_t T, int64_t V, int64_t ld_logits,
                                   float temperature, const float* row_temperature,
                                   const int32_t* tokens, int64_t n_tokens, int64_t n_top,
                                   float* out_logprob, float* out_entropy, int32_t* out_top_token,
                                   float* out_top_logprob, struct CUstream_st* stream) {
  using namespace lmh;
  if (T < 0 || T > LMH_MAX_DIM / 8 || V < 1 || V > LMH_MAX_DIM)
    return api_set_error(LMH_ERR_INVALID_ARG, "T or V out of range");
  if (ld_logits < V)
    return api_set_error(LMH_ERR_INVALID_ARG, "ld_logits must be at least V");
  if (n_tokens < 0 || n_tokens > LMH_MAX_DIM)
    return api_set_error(LMH_ERR_INVALID_ARG, "n_tokens out of range");
  if (n_top < 0 || n_top > kPMaxTop)
    return api_set_error(LMH_ERR_INVALID_ARG, "n_top must be in [0, 128]");
  if (!row_temperature && !(std::isfinite(temperature) && temperature >= 0.f))
    return api_set_error(LMH_ERR_INVALID_ARG, "temperature must be finite and >= 0");
  if (T == 0) return api_set_error(LMH_OK, "");
  if (!logits || (n_tokens > 0 && (!tokens || !out_logprob)) ||
      (n_top > 0 && (!out_top_token || !out_top_logprob)))
    return api_set_error(LMH_ERR_INVALID_ARG,
                         "logits, and what belongs to n_tokens and n_top, are required");
  if (misaligned(logits, 2) || misaligned(row_temperature, 4) || misaligned(tokens, 4) ||
      misaligned(out_logprob, 4) || misaligned(out_entropy, 4) || misaligned(out_top_token, 4) ||
      misaligned(out_top_logprob, 4))
    return api_set_error(LMH_ERR_ALIGNMENT, "logits need 2-byte, the rest 4-byte alignment");
  int sms = 0;
  unsigned* status = nullptr;
  const int rc = api_device(&sms, &status);
  if (rc != LMH_OK) return rc;
  TopParams p{};
  p.logits = logits;
  p.T = T;
  p.V = V;
  p.ld = ld_logits;
  p.temperature = temperature;
  p.row_t = row_temperature;
  p.tokens = tokens;
  p.n_tokens = static_cast<int>(n_tokens);
  p.n_top = static_cast<int>(n_top);
  p.out_logprob = out_logprob;
  p.out_entropy = out_entropy;
  p.top_token = out_top_token;
  p.top_logprob = out_top_logprob;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  {
    KernelTimer timer(K_TOP, st);
    // rows that all start on 16 bytes
    const bool aligned = !misaligned(logits, 16) && (ld_logits % 8 == 0 || T == 1);
    e = aligned ? launch_by_vocabulary<true>(p, st) : launch_by_vocabulary<false>(p, st);
    if (e == cudaSuccess) note_launch();
  }
  if (e != cudaSuccess) {
    char msg[256];
    snprintf(msg, sizeof(msg), "top log-probs: %s", cudaGetErrorString(e));
    return api_set_error(LMH_ERR_LAUNCH, msg);
  }
  return api_set_error(LMH_OK, "");
}
