// What a server reports beside a token (sm_103a): the log-probs of given tokens, the
// entropy, and the likeliest alternatives, from bf16 logits.
//
// For a row x with temperature t (0 counts as 1), z = x / t, m = max z,
//   logprob[i] = z[i] - m - log sum exp(z - m),   entropy = log sum - sum e (z - m) / sum,
// one pass with a running maximum of x: e = 2^((x - max x) * c) with c = log2(e) / t
// rounded once, so that the largest logit's weight is 1 exactly (with the maximum of x * c
// in its place it is off by that product's rounding, and the log-prob of a likely token,
// a number near 0, by several times as much). Masked logits (-inf, NaN) weigh nothing, in
// the entropy either.
//
// The alternatives are the first n in descending order of x, equal ones by index. The
// pass over the row only keeps each thread's largest value: the n-th largest of those is
// reached by n tokens at least, so every alternative reaches it, and only the threads
// whose largest value does (n of them, or a few more) have their share of the row looked
// at again. The tokens found there, n and a few more, are ranked by counting. Where
// more tokens reach it than the list holds (equal logits, a mask of the type's lowest
// value), the n-th largest value is found by bisection over the 16-bit keys, counting over
// the row; first it is tried itself, which it mostly is (1024 rows of 152064 equal logits
// take 116 us, and 2560 without that trial and four vectors at a time). The row is then
// listed from its start until the n are found: a lowest-value mask that leaves fewer than n
// tokens, spread over the row, takes 600 us.
//
// A row is four slices, and every thread of a CTA has its share of each. A cluster of 1
// to 4 CTAs takes the row, as many as a short batch leaves SMs for; a thread's sums are
// merged over the slices as a binary tree, the same one for any number of CTAs, and then
// over the threads.
//
// Batch invariance: the slices and the order of every sum depend on V alone.
//
// What bounds it. Many rows: the issue of instructions (49000 a row of 152064 in warps,
// 64 % of the slots) beside HBM: 64 to 67 us for 1024 rows, 4.6 to 4.9 TB/s, 0.69 to 0.73
// of the copy rate; 1024 rows are 1.7 times what the SMs hold at four CTAs each, and the
// second wave does not fill them. With 90 % of the logits -inf, which sends every group's
// sums to cut_sums, 91 us. Rows off 16 bytes: a ring of twice the size, three CTAs an SM,
// 92 us at V=152061. Middle batches and vocabularies: some 6 us a wave of rows for the
// n-th key, the second look, the ranking and the sums, while nothing is being read (1024
// rows of 8000 15 us, of 32000 23.5; 256 rows of 32000 11.4, of 152064 25.5). Few rows: a chain of short steps, 9.0 us at one row of 152064 on four
// CTAs (9000 cycles to read and fold, 1700 to bisect the keys, 3000 for the second look,
// 1100 for the cluster, 3500 for sums and lists, the kernel behind under way meanwhile).
// Tried and slower at 1024 rows of 152064 (64 us then): 512 threads a CTA (119), 384 (78),
// five vectors a group (74: spills), two CTAs a row (77), three CTAs an SM and three
// groups ahead (70), eight slices (68), each thread's largest value kept for 32 values at
// a time, for a shorter second look (70), the keys bisected two bits at a time (65).
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdio>

#include <cuda_bf16.h>

#include "internal.h"
#include "launch.cuh"
#include "lmhead.h"
#include "online_softmax.cuh"
#include "ptx.cuh"

namespace lmh {

namespace {

typedef unsigned long long u64;

constexpr int kPThreads = 256;
constexpr int kPWarps = kPThreads / 32;
constexpr int kPMaxTop = 128;   // most alternatives
constexpr int kPSlices = 4;     // of a row; the most CTAs that share one
constexpr int kPList = 512;     // tokens of a CTA's list
constexpr int kPGroup = 4;      // vectors that a thread folds at once
constexpr int kPDepth = 2;      // groups on their way to a thread
constexpr int kPMinSlice = kPGroup * kPThreads;  // vectors of a slice, where the row has them
static_assert(kPMaxTop <= kPThreads, "a thread's largest value for each alternative");
constexpr float kPFloor = -200.f;  // 2^-200 is 0: what masked and far values are cut to

struct TopParams {
  const uint16_t* logits;
  int64_t T, V, ld;
  float temperature;
  const float* row_t;
  const int32_t* tokens;
  int n_tokens, n_top;
  int per;  // vectors of a slice: whole runs of 32
  float* out_logprob;
  float* out_entropy;
  int32_t* top_token;
  float* top_logprob;
};

// A slice's largest logit m (-inf: all masked) and its sums s = sum e, u = sum e * (x - m);
// stored whole by 16 bytes.
struct alignas(16) SliceStat {
  float m, s, u;
};
constexpr float kPFar = -1e28f;  // what differences are cut to where their weight is 0 (c >= 1e-25)

template <int kC>
struct TopShared {
  u64 list[kPList];
  u64 merged[kC][kPMaxTop];          // CTA 0: every CTA's best, in order,
  int n_merged[kC];                  // and how many they are
  int n_hit, n_list;
  SliceStat warp[kPWarps];
  float top[kPWarps];                // the warps' largest logits
  uint16_t key[kPSlices / kC][kPThreads];  // a thread's largest value in each slice
  uint16_t hit[kPThreads * kPSlices / kC];
  uint32_t count[kPWarps];
  float temperature;
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

// 8 values at `off` bytes (even, below 16) into two aligned vectors.
__device__ __forceinline__ uint4 shifted(const uint4& a, const uint4& b, uint32_t off) {
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

// Vector v (elements [8 v, 8 v + 8)) of a row at any address, -inf past its end. A row
// that does not start on 16 bytes is read in the aligned 16 bytes that hold the vector,
// but for its two ends, so that nothing outside the row is.
template <bool kAligned>
__device__ __forceinline__ uint4 load_vector(const uint16_t* row, int64_t V, int64_t v) {
  const uint16_t* at = row + 8 * v;
  if (kAligned && 8 * v + 8 <= V) return *reinterpret_cast<const uint4*>(at);
  if (!kAligned && v > 0 && 8 * v + 16 <= V) {
    const uint4* g = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(at) & ~uintptr_t{15});
    return shifted(g[0], g[1], static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at) & 15));
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

// Scales sums to the maximum m (their own or a larger one); those of nothing stay zero.
__device__ __forceinline__ void rescale(SliceStat& a, float m, float c) {
  const float d = fmaxf(__fsub_rn(a.m, m), kPFar);
  const float e = ex2(fmaxf(__fmul_rn(d, c), kPFloor));
  a.u = __fmul_rn(e, __fmaf_rn(a.s, d, a.u));
  a.s = __fmul_rn(a.s, e);
  a.m = m;
}

// a <- a (+) b. An empty side leaves the other's bits.
__device__ __forceinline__ void merge_slice(SliceStat& a, SliceStat b, float c) {
  const float m = fmaxf(a.m, b.m);
  rescale(a, m, c);
  rescale(b, m, c);
  a.s = __fadd_rn(a.s, b.s);
  a.u = __fadd_rn(a.u, b.u);
}

// One pair of values into the packed sums.
template <bool kCut>
__device__ __forceinline__ void add_pair(uint32_t pair, f32x2 nm2, f32x2 c2, f32x2& s2, f32x2& u2) {
  f32x2 d2 = f2_add(bf16x2_f2(pair), nm2);
  float ya, yb;
  f2_unpack(f2_mul(d2, c2), ya, yb);
  if (kCut) {  // a masked value's weight is 0, and its difference finite
    float da, db;
    f2_unpack(d2, da, db);
    d2 = f2_pack(fmaxf(da, kPFar), fmaxf(db, kPFar));  // a NaN too
    ya = fmaxf(ya, kPFloor);
    yb = fmaxf(yb, kPFloor);
  }
  const f32x2 e2 = f2_pack(ex2(ya), ex2(yb));
  s2 = f2_add(s2, e2);
  u2 = f2_fma(e2, d2, u2);
}

__device__ __forceinline__ float2 sum_pairs(f32x2 s2, f32x2 u2) {
  float s0, s1, u0, u1;
  f2_unpack(s2, s0, s1);
  f2_unpack(u2, u0, u1);
  return make_float2(__fadd_rn(s0, s1), __fadd_rn(u0, u1));
}

// A group's sums where some are masked. Out of line: in line its values, kept with those
// of the usual sums, cost registers that every group would spill.
__device__ __noinline__ float2 cut_sums(uint4 a, uint4 b, uint4 g, uint4 h, float m, float c) {
  const f32x2 c2 = f2_pack(c, c), nm2 = f2_pack(-m, -m);
  f32x2 s2 = f2_pack(0.f, 0.f), u2 = s2;
  const uint32_t w[16] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w,
                          g.x, g.y, g.z, g.w, h.x, h.y, h.z, h.w};
#pragma unroll
  for (int i = 0; i < 16; ++i) add_pair<true>(w[i], nm2, c2, s2, u2);
  return sum_pairs(s2, u2);
}

// Folds kV vectors (of w's four, the others masked) into the state. A masked value makes
// the plain sum of e * (x - m) a NaN.
template <int kV>
__device__ __forceinline__ void fold(SliceStat& st, const uint4 (&w)[kPGroup], float c) {
  __nv_bfloat162 hi = bf2(w[0].x);  // passes over a NaN
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    const uint32_t ws[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
    for (int q = 0; q < 4; ++q) hi = __hmax2(hi, bf2(ws[q]));
  }
  // (the larger of two NaN is one: a masked value)
  const float m = fmaxf(st.m, fmaxf(__low2float(hi), __high2float(hi)));
  rescale(st, m, c);
  const f32x2 c2 = f2_pack(c, c), nm2 = f2_pack(-m, -m);
  f32x2 s2 = f2_pack(0.f, 0.f), u2 = s2;
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    add_pair<false>(w[k].x, nm2, c2, s2, u2);
    add_pair<false>(w[k].y, nm2, c2, s2, u2);
    add_pair<false>(w[k].z, nm2, c2, s2, u2);
    add_pair<false>(w[k].w, nm2, c2, s2, u2);
  }
  float2 sums = sum_pairs(s2, u2);
  if (!(fabsf(sums.y) <= 3.402823466e38f)) sums = cut_sums(w[0], w[1], w[2], w[3], m, c);
  st.s = __fadd_rn(st.s, sums.x);
  st.u = __fadd_rn(st.u, sums.y);
}

// A vector's largest key (0: all masked).
__device__ __forceinline__ uint32_t largest_key(const uint4& w) {
  const __nv_bfloat162 m2 = __hmax2(__hmax2(bf2(w.x), bf2(w.y)), __hmax2(bf2(w.z), bf2(w.w)));
  // (the larger of two NaN is one: a masked value)
  return order_key(__float_as_uint(fmaxf(__low2float(m2), __high2float(m2))) >> 16);
}

// How many values of the slice have a key of at least k >= 1, in every thread.
template <bool kAligned>
__device__ __noinline__ uint32_t count_from(const uint16_t* row, int64_t V, int64_t v0, int64_t v1,
                                            uint32_t k, uint32_t* part) {
  uint32_t n = 0;
  for (int64_t v = v0 + threadIdx.x; v < v1; v += 4 * kPThreads) {
    uint4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] = make_uint4(kMasked2, kMasked2, kMasked2, kMasked2);
      if (v + j * kPThreads < v1) x[j] = load_vector<kAligned>(row, V, v + j * kPThreads);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (largest_key(x[j]) < k) continue;
      const uint32_t ws[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) n += order_key(ws[i / 2] >> (16 * (i & 1)) & 0xffffu) >= k;
    }
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
// and of those that have it the first by index. At least n tokens reach `bar`; mostly
// fewer are above it (a mask of the type's lowest value, equal logits), and it is that key.
template <bool kAligned, class Shared>
__device__ __noinline__ void list_by_bisection(Shared& sh, const uint16_t* row, int64_t V,
                                               int64_t v0, int64_t v1, int n, uint32_t bar) {
  uint32_t lo = bar, hi = 0x10000u, many = 0;  // count(lo) >= n > count(hi) = many
  for (uint32_t mid = bar + 1; hi - lo > 1; mid = (lo + hi) / 2) {
    const uint32_t reach = count_from<kAligned>(row, V, v0, v1, mid, sh.count);
    if (reach >= static_cast<uint32_t>(n)) {
      lo = mid;
    } else {
      hi = mid;
      many = reach;
    }
  }
  const int above = static_cast<int>(many);
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
    const bool all = sh.n_list >= above && taken + total >= static_cast<uint32_t>(n);
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
    if (all) break;
  }
  if (threadIdx.x == 0) sh.n_list = n;
  __syncthreads();
}

// z - max z.
__device__ __forceinline__ float shift(float x, float most, float t) {
  const float d = __fsub_rn(x, most);
  if (x == most) return 0.f;
  return d == -INFINITY ? __fsub_rn(__fdiv_rn(x, t), __fdiv_rn(most, t)) : __fdiv_rn(d, t);
}

// The sums (u in units of z) of a row whose differences, or their products with c, leave
// fp32: logits equal to the largest weigh 1. One CTA, in an order fixed by V.
template <class Shared>
__device__ __noinline__ SliceStat sums_of_extremes(Shared& sh, const uint16_t* row, int64_t V,
                                                   float t, float most) {
  float s = 0.f, u = 0.f;
  for (int64_t i = threadIdx.x; i < V; i += kPThreads) {
    const uint32_t b = row[i];
    if (order_key(b) == 0u) continue;
    const float d = shift(__uint_as_float(b << 16), most, t);
    const float e = ex2(fmaxf(__fmul_rn(d, kLog2e), kPFloor));
    s += e;
    u += e > 0.f ? e * d : 0.f;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, off);
    u += __shfl_xor_sync(0xffffffffu, u, off);
  }
  if ((threadIdx.x & 31) == 0) sh.warp[threadIdx.x >> 5] = SliceStat{most, s, u};
  __syncthreads();
  SliceStat r{most, 0.f, 0.f};
  for (int w = 0; w < kPWarps; ++w) {
    r.s += sh.warp[w].s;
    r.u += sh.warp[w].u;
  }
  return r;
}

// Not the .aligned forms: a warp need not be whole where it comes out of a branch.
__device__ __forceinline__ void row_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void row_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

template <int kC>
__device__ __forceinline__ uint32_t first_cta(const void* here) {
  return kC > 1 ? mapa_shared(smem_u32(here), 0u) : smem_u32(here);
}

// How the vectors of a row reach a thread: each copies its own, kPDepth groups of up to
// four ahead, into shared memory that no other thread touches. A row that does not start
// on 16 bytes takes two aligned vectors for each. Vectors outside [lo, hi), whose copies
// would reach outside the row, are read element by element.
template <bool kAligned>
struct Ring {
  static constexpr int kCopies = kAligned ? 1 : 2;
  static constexpr int kBytes = kPDepth * kPGroup * kCopies * kPThreads * 16;
  const uint16_t* row;
  int64_t V;
  uint32_t at;  // this thread's first slot
  int first;    // the CTA's first vector, from which v below counts
  int lo, hi;
  const uint16_t* from;  // this thread's place in the first group, down to 16 bytes
  __device__ __forceinline__ Ring(const uint16_t* row, int64_t V, uint32_t smem, int first)
      : row(row), V(V), at(smem + threadIdx.x * 16), first(first) {
    lo = kAligned ? 0 : 1 - first;
    hi = static_cast<int>(kAligned ? V / 8 : V / 8 - 1) - first;
    from = row + 8 * (static_cast<int64_t>(first) + threadIdx.x);
    if constexpr (!kAligned)
      from = reinterpret_cast<const uint16_t*>(reinterpret_cast<uintptr_t>(from) & ~uintptr_t{15});
  }
  __device__ __forceinline__ uint32_t slot(int depth, int k, int copy) const {
    return at + static_cast<uint32_t>(((depth * kPGroup + k) * kCopies + copy) * kPThreads * 16);
  }
  // The group of vectors v0 + t + 256 k below end.
  __device__ __forceinline__ void fetch(int depth, int v0, int end) const {
    const uint16_t* src = from + 8 * static_cast<int64_t>(v0);
    if (v0 >= lo && v0 + kPGroup * kPThreads <= min(end, hi)) {
#pragma unroll
      for (int k = 0; k < kPGroup; ++k)
#pragma unroll
        for (int c = 0; c < kCopies; ++c)
          copy16_async(slot(depth, k, c), src + 8 * (k * kPThreads + c));
    } else {
#pragma unroll
      for (int k = 0; k < kPGroup; ++k) {
        const int v = v0 + static_cast<int>(threadIdx.x) + k * kPThreads;
        if (v >= end) continue;
        if (v >= lo && v < hi) {
#pragma unroll
          for (int c = 0; c < kCopies; ++c)
            copy16_async(slot(depth, k, c), src + 8 * (k * kPThreads + c));
        } else {
          const uint4 w = load_vector<kAligned>(row, V, static_cast<int64_t>(first) + v);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(slot(depth, k, 0)),
                       "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w)
                       : "memory");
        }
      }
    }
    copies_commit();  // an empty one too: the groups are counted
  }
  __device__ __forceinline__ uint4 take(int depth, int k, int v) const {
    const uint4 a = ld_shared_v4(slot(depth, k, 0));
    if constexpr (kAligned) return a;
    if (v < lo || v >= hi) return a;
    return shifted(a, ld_shared_v4(slot(depth, k, 1)),
                   static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 15));
  }
};

template <int kC, bool kAligned>
__global__ void __launch_bounds__(kPThreads, 4) top_logprobs_kernel(const TopParams p) {
  extern __shared__ __align__(16) uint8_t ring_smem[];
  // CTA 0: the other CTAs' threads' sums, behind the ring
  SliceStat* peer = reinterpret_cast<SliceStat*>(ring_smem + Ring<kAligned>::kBytes);
  __shared__ __align__(16) TopShared<kC> sh;
  constexpr int kMine = kPSlices / kC;  // slices of this CTA
  const int64_t row = blockIdx.x / kC;
  const int rank = kC > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const uint16_t* x = p.logits + row * p.ld;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // This CTA's slices [0, slices) with something in them, of `per` vectors but the last;
  // vectors are counted from the first slice's first.
  constexpr int kStep = kPGroup * kPThreads;
  const int n_vec = static_cast<int>((p.V + 7) / 8), per = p.per;
  const int first = static_cast<int>(min(static_cast<int64_t>(n_vec), static_cast<int64_t>(per) * (rank * kMine)));
  const int n_mine = static_cast<int>(min(static_cast<int64_t>(n_vec - first), static_cast<int64_t>(per) * kMine));
  const int slices = (n_mine + per - 1) / per;

  if (kC > 1) row_arrive();  // this CTA runs: see the wait below
  ahead_done();
  if (threadIdx.x == 0) {
    // one reading of the temperature decides every thread's way
    sh.temperature = p.row_t ? p.row_t[row] : p.temperature;
    sh.n_hit = sh.n_list = 0;
  }

  const Ring<kAligned> ring(x, p.V, smem_u32(ring_smem), first);
  int ahead = 0, ahead_end = min(per, n_mine);  // the next group to fetch, its slice's end
  auto fetch = [&](int depth) {
    ring.fetch(depth, ahead, ahead_end);
    ahead += kStep;
    if (ahead >= ahead_end) {
      ahead = ahead_end;
      ahead_end = min(ahead_end + per, n_mine);
    }
  };
#pragma unroll
  for (int d = 0; d < kPDepth - 1; ++d) fetch(d);
  __syncthreads();
  float t = sh.temperature;
  if (t == 0.f) t = 1.f;
  const bool valid_t = t > 0.f && t <= 3.402823466e38f;
  if (!valid_t) t = 1.f;
  const float c = __fdiv_rn(kLog2e, t);

  // The slices' sums as a binary tree: pairs, then all four. What is missing at the end
  // is empty, and leaves the rest as it is.
  const SliceStat none{-INFINITY, 0.f, 0.f};
  SliceStat one = none, two = none, mine = none;
  uint32_t top_key = 0;  // of this thread's values
  int depth = 0, v0 = 0;
#pragma unroll 1
  for (int i = 0; i < slices; ++i) {
    const int end = min((i + 1) * per, n_mine);
    mine = none;
#pragma unroll 1
    for (; v0 < end; v0 += kStep) {
      fetch(depth == 0 ? kPDepth - 1 : depth - 1);
      copies_wait<kPDepth - 1>();
      const int v = v0 + static_cast<int>(threadIdx.x);
      uint4 w[kPGroup];
      if (v0 + kStep <= end) {
#pragma unroll
        for (int k = 0; k < kPGroup; ++k) w[k] = ring.take(depth, k, v + k * kPThreads);
      } else {
#pragma unroll
        for (int k = 0; k < kPGroup; ++k) {
          w[k] = make_uint4(kMasked2, kMasked2, kMasked2, kMasked2);
          if (v + k * kPThreads < end) w[k] = ring.take(depth, k, v + k * kPThreads);
        }
      }
      if (end - v0 > 3 * kPThreads)
        fold<4>(mine, w, c);
      else if (end - v0 > 2 * kPThreads)
        fold<3>(mine, w, c);
      else if (end - v0 > kPThreads)
        fold<2>(mine, w, c);
      else
        fold<1>(mine, w, c);
      if (++depth == kPDepth) depth = 0;
    }
    v0 = end;
    const uint32_t key = order_key(__float_as_uint(mine.m) >> 16);
    sh.key[i][threadIdx.x] = static_cast<uint16_t>(key);
    top_key = max(top_key, key);
    if (!(i & 1)) {
      one = mine;
    } else {
      merge_slice(one, mine, c);
      if (i == 1)
        two = one;
      else
        merge_slice(two, one, c);
    }
  }
  mine = slices & 1 ? one : none;
  if (slices >= 2) {
    merge_slice(two, mine, c);
    mine = two;
  }
  // The first CTA's shared memory may be written once it runs; a CTA without a slice of
  // its own is here before that.
  if (kC > 1) row_wait();
  if (kC > 1 && rank > 0) {
    const uint32_t at = first_cta<kC>(peer + (rank - 1) * kPThreads + threadIdx.x);
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(mine.m),
                 "f"(mine.s), "f"(mine.u), "f"(0.f)
                 : "memory");
  }
  __syncthreads();

  const int n = p.n_top;
  if (n > 0) {
    // the n-th largest of the threads' keys (1 where fewer are not masked), bit by bit
    uint32_t bar = 0;
#pragma unroll 1
    for (uint32_t bit = 0x8000u; bit > 0; bit >>= 1)
      if (__syncthreads_count(top_key >= (bar | bit)) >= n) bar |= bit;
    bar = max(bar, 1u);
    if (top_key >= bar) {
      for (int i = 0; i < slices; ++i)
        if (sh.key[i][threadIdx.x] >= bar)
          sh.hit[atomicAdd(&sh.n_hit, 1)] = static_cast<uint16_t>(i * kPThreads + threadIdx.x);
    }
    __syncthreads();
    const uint32_t share = static_cast<uint32_t>((per + kPThreads - 1) / kPThreads);
    const uint32_t looks = static_cast<uint32_t>(sh.n_hit) * share;
    for (uint32_t i = threadIdx.x; i < looks; i += kPThreads) {
      if (*static_cast<volatile int*>(&sh.n_list) > kPList) break;  // made another way
      const uint32_t h = i / share, j = i - h * share;
      const int who = sh.hit[h];
      const int from = who / kPThreads * per;
      const int at_v = from + who % kPThreads + static_cast<int>(j) * kPThreads;
      if (at_v >= min(from + per, n_mine)) continue;
      const int64_t v = static_cast<int64_t>(first) + at_v;
      const uint4 w = load_vector<kAligned>(x, p.V, v);
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
      uint32_t reach = 0;  // a bit for each value that does
#pragma unroll
      for (int e = 0; e < 8; ++e)
        reach |= (order_key(ws[e / 2] >> (16 * (e & 1)) & 0xffffu) >= bar ? 1u : 0u) << e;
      if (reach == 0) continue;
      int at = atomicAdd(&sh.n_list, __popc(reach));
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (reach >> e & 1u) {
          if (at < kPList)
            sh.list[at] = entry_of(order_key(ws[e / 2] >> (16 * (e & 1)) & 0xffffu), 8 * v + e);
          ++at;
        }
    }
    __syncthreads();
    if (sh.n_list > kPList)
      list_by_bisection<kAligned>(sh, x, p.V, first, first + n_mine, n, bar);
    const int found = sh.n_list;
    // the first n of them, in order, to the first CTA
    const uint32_t to = first_cta<kC>(&sh.merged[rank][0]);
    for (int i = threadIdx.x; i < found; i += kPThreads) {
      const u64 me = sh.list[i];
      int r = 0;
#pragma unroll 4
      for (int j = 0; j < found; ++j) r += sh.list[j] > me;
      if (r < n)
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to + 8u * r), "l"(me) : "memory");
    }
    if (threadIdx.x == 0)
      st_shared_cluster_u32(first_cta<kC>(&sh.n_merged[rank]), static_cast<uint32_t>(min(found, n)));
  }
  if constexpr (kC > 1) {
    __syncwarp();
    row_arrive();
    row_wait();
    if (rank != 0) return;
    // the rest of the tree: pairs of CTAs, pairs of pairs
    SliceStat part[kC];
    part[0] = mine;
#pragma unroll
    for (int k = 1; k < kC; ++k) part[k] = peer[(k - 1) * kPThreads + threadIdx.x];
#pragma unroll
    for (int by = 1; by < kC; by *= 2)
#pragma unroll
      for (int k = 0; k < kC; k += 2 * by) merge_slice(part[k], part[k + by], c);
    mine = part[0];
  }
  nearly_done();
  // then the threads, all scaled to the row's maximum: within each warp, and the warps in order
  float most = mine.m;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
  if (lane == 0) sh.top[warp] = most;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kPWarps; ++w) most = fmaxf(most, sh.top[w]);
  rescale(mine, most, c);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    mine.s = __fadd_rn(mine.s, __shfl_xor_sync(0xffffffffu, mine.s, off));
    mine.u = __fadd_rn(mine.u, __shfl_xor_sync(0xffffffffu, mine.u, off));
  }
  if (lane == 0) sh.warp[warp] = mine;
  __syncthreads();
  SliceStat all{most, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < kPWarps; ++w) {
    all.s = __fadd_rn(all.s, sh.warp[w].s);
    all.u = __fadd_rn(all.u, sh.warp[w].u);
  }
  all.u = __fdiv_rn(all.u, t);
  // where differences or their products may leave fp32 (or the largest logit is +inf) the
  // row is summed again
  const bool nothing = !(most > -INFINITY);
  if (!nothing && !(most <= 1e36f && c >= 1e-25f && c <= 3.402823466e38f)) {
    __syncthreads();
    all = sums_of_extremes(sh, x, p.V, t, most);
  }
  const float lse = __fmul_rn(kLn2, log2f(all.s));  // of z - max z
  const float bad = __int_as_float(0x7fffffff);
  auto logprob = [&](float v) -> float {
    if (!valid_t) return bad;
    if (nothing || !(v > -INFINITY)) return -INFINITY;  // a masked one
    return __fsub_rn(shift(v, most, t), lse);
  };
  // the last threads take the tokens, the first ones the lists
  const int back = kPThreads - 1 - static_cast<int>(threadIdx.x);
  if (back == 0 && p.out_entropy)
    p.out_entropy[row] = !valid_t ? bad
                         : nothing ? 0.f
                                   : __fsub_rn(lse, __fdiv_rn(all.u, all.s));
  for (int i = back; i < p.n_tokens; i += kPThreads) {
    const int32_t id = p.tokens[row * p.n_tokens + i];
    float lp = valid_t ? 0.f : bad;
    if (id >= 0 && id < p.V) lp = logprob(__uint_as_float(static_cast<uint32_t>(x[id]) << 16));
    p.out_logprob[row * p.n_tokens + i] = lp;
  }
  if (n == 0) return;
  int total = 0;
#pragma unroll
  for (int k = 0; k < kC; ++k) total += sh.n_merged[k];
  if (!valid_t) total = 0;
  for (int i = threadIdx.x; i < n; i += kPThreads) {  // places that no token takes
    if (i >= total) {
      p.top_token[row * n + i] = -1;
      p.top_logprob[row * n + i] = valid_t ? -INFINITY : bad;
    }
  }
  int half = 1;  // steps of a search in a list of up to n
  while (2 * half <= n) half *= 2;
  for (int i = threadIdx.x; i < kC * n; i += kPThreads) {
    const int own = kC == 1 ? 0 : i / n, place = i - own * n;  // a list and the place in it
    if (!valid_t || place >= sh.n_merged[own]) continue;
    const u64 me = sh.merged[own][place];
    int r = place;  // and how many of each other list come before
    if constexpr (kC > 1) {
      int lo[kC], len[kC];
#pragma unroll
      for (int k = 0; k < kC; ++k) {
        lo[k] = 0;
        len[k] = k == own ? 0 : sh.n_merged[k];
      }
#pragma unroll 1
      for (int step = half; step > 0; step >>= 1) {
        u64 other[kC];
#pragma unroll
        for (int k = 0; k < kC; ++k) other[k] = sh.merged[k][min(lo[k] + step, kPMaxTop) - 1];
#pragma unroll
        for (int k = 0; k < kC; ++k)
          if (lo[k] + step <= len[k] && other[k] > me) lo[k] += step;
      }
#pragma unroll
      for (int k = 0; k < kC; ++k) r += lo[k];
    }
    if (r < n) {
      p.top_token[row * n + r] = static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(me));
      p.top_logprob[row * n + r] = logprob(value_of_key(static_cast<uint32_t>(me >> 32)));
    }
  }
}

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

template <int kC, bool kAligned>
cudaError_t launch_top(const TopParams& p, cudaStream_t st) {
  constexpr int kBytes =
      Ring<kAligned>::kBytes + (kC - 1) * kPThreads * static_cast<int>(sizeof(SliceStat));
  // The kernel's shared-memory attribute belongs to the device: set by its first call.
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(top_logprobs_kernel<kC, kAligned>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
    done[dev].store(true, std::memory_order_release);
  }
  return launch_early(top_logprobs_kernel<kC, kAligned>, static_cast<unsigned>(p.T * kC), kPThreads,
                      kBytes, st, kC, p);
}

// CTAs of a row: 4 while the batch then needs no more than two an SM, else 2 likewise,
// else 1; and of them more than half get a part of the row, whose slices are dealt out
// whole, 4 / CTAs to each (so a row of two slices, V up to 16384, takes one). us at 1 / 2 /
// 4 CTAs a row:
//   rows      V=16000             V=32000             V=152064
//     1    6.6   7.0   6.2     7.7   6.8   6.0    16.2  11.6   8.9
//    48    6.7   7.3   7.0     8.2   7.3   7.1    17.5  12.7  11.4
//    76    6.9   7.5   8.0     8.2   7.6   8.3    17.7  14.0  13.9
//   100    7.0   8.6   8.8     8.3   8.7   9.0    18.8  15.5  15.5
//   152    7.1   8.2  12.1     8.5   9.1  12.9    20.6  18.7  22.4
//   256    9.1  11.3  16.0    11.5  11.1  16.7    25.7  24.2  30.8
//   608   10.9  21.7  33.5    14.3  21.3  35.1    40.3  47.9  62.9
// The bounds lose up to 0.8 us to the best of the three, but for 153 to 304 rows of the
// largest vocabulary, where two CTAs would save 0.8 to 2.7.
template <bool kAligned>
cudaError_t launch_by_rows(const TopParams& p, int sms, cudaStream_t st) {
  int most = p.T * 4 <= 2 * sms ? 4 : p.T * 2 <= 2 * sms ? 2 : 1;
  const int64_t used = ((p.V + 7) / 8 + p.per - 1) / p.per;  // slices
  while (most > 1 && (used * most + kPSlices - 1) / kPSlices <= most / 2) most /= 2;
  switch (most) {
    case 4: return launch_top<4, kAligned>(p, st);
    case 2: return launch_top<2, kAligned>(p, st);
    default: return launch_top<1, kAligned>(p, st);
  }
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
  const int64_t per = ((V + 7) / 8 + kPSlices - 1) / kPSlices;
  p.per = static_cast<int>((per > kPMinSlice ? per + 31 : kPMinSlice) / 32 * 32);
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
    e = aligned ? launch_by_rows<true>(p, sms, st) : launch_by_rows<false>(p, sms, st);
    if (e == cudaSuccess) note_launch();
  }
  if (e != cudaSuccess) {
    char msg[256];
    snprintf(msg, sizeof(msg), "top log-probs: %s", cudaGetErrorString(e));
    return api_set_error(LMH_ERR_LAUNCH, msg);
  }
  return api_set_error(LMH_OK, "");
}
