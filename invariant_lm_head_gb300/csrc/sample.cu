// Sampling from bf16 logits (sm_103a): temperature, top-k, top-p and min-p, one
// token per row from a given uniform number.
//
// A row's bf16 logits take few distinct values, and everything the sampler
// decides depends on a token only through its logit and, among equal ones, its
// index. So a row is read once into a histogram of counts over the ordered
// values (shared memory, integer adds), and all later work is on the
// histogram: with m the largest z = x / t (fp32 division), a bin's weight is
// exp(z - m) in fp32 (24 bits: expf's 2 units in the last place, one rounding, and
// what the subtraction lost put back), cut to units of 2^-44, and its mass is
// count * weight. Sums of these integers are exact and have no order, so the
// result is the same whatever adds first; against exact weights a border between
// two tokens is off by their relative error, below 2^-21. Tokens are taken in
// descending logit, ties by index:
//   top-k   the first k;
//   top-p   the shortest prefix of those whose mass reaches p of their mass;
//   min-p   those of weight >= min_p;
//   draw    the first of the kept whose running mass exceeds u * kept mass.
// Each is a prefix of one order, so each is one crossing of the histogram's
// running count or mass. The crossing gives a value and a rank among its equal
// tokens; a second look at the row turns the rank into an index, half a row on
// average (from L2 as long as the rows at work fit it).
//
// Bins. The histogram covers zero and every bf16 of magnitude [2^-32, 2^8),
// one bin per value. A row that holds another value whose weight matters (the
// lowest finite value as a mask does not, next to real logits) is taken in
// seven windows over all bf16 values instead, the row read again for each.
//
// What bounds it. One row of 152064 takes 10.8 us on 8 CTAs: a chain of short steps
// (count 4700 cycles, weigh 5800, cuts and draw 6200, with their cluster barriers),
// where the row's bytes are 0.04 us. 256 rows take 46 us and 1024 rows 152 us, for
// 11 and 46 us of bytes: a row's 4752 warp-wide increments cost 17600 cycles of its
// SM's shared memory, 32 random bins meeting 3.7 deep on a bank (four rows counting
// at once take 83000 cycles, 0.85 of that pipe), and weighing, the shuffles and the
// index search share it. Staggering the four rows of an SM, so that some weigh while
// others count, gains nothing (1024 rows 153-158 us). The two shapes that share an
// SM have 64 registers and spill (-Xptxas -v: <1, 512, 2> 96 bytes stored and 108
// loaded, <1, 256, 4> 112 and 116); the others take 100 and do not.
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

constexpr int kMaxThreads = 512;
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr int kBatch = 5;  // 16-byte loads in flight per thread
constexpr int kMaxC = 8;   // most CTAs of a row (a portable cluster)
// Magnitude bits (sign dropped) of the direct range.
constexpr int kMagLo = (127 - 32) << 7;         // 2^-32
constexpr int kMagHi = ((127 + 8) << 7) - 1;    // largest below 2^8
constexpr int kHalf = kMagHi - kMagLo + 1;      // values of one sign: 5120
constexpr int kBins = 2 * kHalf + 1;            // 10241
constexpr int kBinsPad = 10752;                 // whole rows of 32 bins for 1, 2, 4 or 8 CTAs
static_assert(kBinsPad >= kBins && kBinsPad % (32 * kMaxC) == 0, "bins");
// Every bf16 value in descending order: positive 0 .. 32766, zero 32767,
// negative 32768 .. 65534 (inf and NaN magnitudes included).
constexpr int kFullKeys = 65535;
constexpr int kWindows = (kFullKeys + kBinsPad - 1) / kBinsPad;
constexpr int kDirect = -1;  // the direct range, beside windows 0 .. kWindows - 1
constexpr int kNone = 0x7fffffff;
// A weight below 2^-45 is zero: d < -45 ln 2.
constexpr float kTail = -31.2f;

typedef unsigned long long u64;

// Position of a bf16 bit pattern in the full descending order (both zeros at 32767).
__device__ __forceinline__ int full_key(uint32_t b) {
  const int mag = static_cast<int>(b & 0x7fffu);
  return (b & 0x8000u) ? 32767 + mag : 32767 - mag;
}
__device__ __forceinline__ float key_value(int key) {
  const uint32_t b = key <= 32767 ? static_cast<uint32_t>(32767 - key)
                                  : 0x8000u | static_cast<uint32_t>(key - 32767);
  return __uint_as_float(b << 16);
}
// Never drawn: NaN and -inf.
__device__ __forceinline__ bool is_masked(uint32_t b) {
  return (b & 0x7fffu) > 0x7f80u || b == 0xff80u;
}

struct SampleParams {
  const uint16_t* logits;
  int64_t T, V, ld;
  float temperature, top_p, min_p;
  int top_k;
  const float *row_t, *row_p, *row_m;
  const int32_t* row_k;
  const float* uniform;
  int32_t* token;
  float* logprob;
  int fix;  // weights are in units of 2^-fix
};

// What a row asks for; the temperature is NaN where a setting is out of range.
struct Settings {
  float t, top_p, min_p, u;
  int top_k;
  __device__ __forceinline__ void load(const SampleParams& p, int64_t row) {
    t = p.row_t ? p.row_t[row] : p.temperature;
    top_p = p.row_p ? p.row_p[row] : p.top_p;
    min_p = p.row_m ? p.row_m[row] : p.min_p;
    top_k = p.row_k ? p.row_k[row] : p.top_k;
    u = p.uniform[row];
    if (!(t >= 0.f && t <= 3.402823466e38f && top_p > 0.f && min_p <= 1.f && u >= 0.f && u <= 1.f &&
          top_k >= 0))
      t = __int_as_float(0x7fffffff);
  }
};

struct Totals {
  u64 mass, kept;  // kept: the mass that min-p keeps
  uint32_t count;
};

// The histogram is weighed in rows of 32 bins.
constexpr int kRows = kBinsPad / 32;

struct RowShared {
  Settings set;             // thread 0's reading of them
  u64 row_m[kRows];         // CTA 0: mass and count of every row of bins
  uint32_t row_c[kRows];
  u64 kept[kMaxC];          // CTA 0: every CTA's share of the mass that min-p keeps
  int4 seen[kMaxC];         // every CTA's flags, largest value's position, temperature, min-p
  Totals warp[kMaxWarps];
  u64 found;                // a crossing: the mass up to and with its token,
  int found_bin;            // its bin,
  uint32_t found_rank;      // and the token's rank among the bin's
  int4 order;               // from CTA 0: kLook, the CTA that holds the token, its key, its
                            // rank there; or kBuild and the window to count
  uint32_t hits[2][kMaxWarps];
  int64_t index;
  int flags;                // 1: above the direct range, 2: tiny, 4: below the range
  int top;                  // smallest position of the CTA's own values
};
constexpr int kLook = 0, kBuild = 1;

// ------------------------------------------------------------ the cluster
// Not the .aligned forms: they count a whole warp at once, and a warp that comes
// out of a branch on its lanes (one thread that pushes a total to a peer, say) need
// not be one again.
__device__ __forceinline__ void row_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void row_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
template <int kC>
__device__ __forceinline__ void row_sync() {
  if constexpr (kC > 1) {
    __syncwarp();
    row_arrive();
    row_wait();
  } else {
    __syncthreads();
  }
}
// The address of the same shared variable in CTA c.
template <int kC>
__device__ __forceinline__ uint32_t peer(const void* here, int c) {
  return kC > 1 ? mapa_shared(smem_u32(here), static_cast<uint32_t>(c)) : smem_u32(here);
}
__device__ __forceinline__ uint32_t ld_peer_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_peer_v4(uint32_t addr, int4 v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void st_peer_u64(uint32_t addr, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// ------------------------------------------------------------ two values a word
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// ------------------------------------------------------------ reading a row
// A CTA's part of a row in index order: 2-byte steps up to the row's first
// 16-byte boundary (the first CTA), a run of 16-byte vectors, and the row's last
// elements (the last CTA).
struct Slice {
  const uint16_t* x;   // the row
  const uint4* vec;    // this CTA's vectors
  int n_vec;
  int n_head, n_tail;  // this CTA's elements before and after them (at most 7)
  __device__ __forceinline__ Slice(const uint16_t* row, int64_t V, int rank, int n_ranks) : x(row) {
    const int to16 = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) >> 1;
    const int n = static_cast<int>(V);
    const int head = min(to16, n);
    const int nv = (n - head) >> 3;
    const int per = (nv + n_ranks - 1) / n_ranks;
    const int v0 = min(nv, per * rank);
    n_vec = min(nv, v0 + per) - v0;
    vec = reinterpret_cast<const uint4*>(row + head) + v0;
    n_head = rank == 0 ? head : 0;
    n_tail = rank == n_ranks - 1 ? n - head - 8 * nv : 0;
  }
  __device__ __forceinline__ const uint16_t* tail() const {
    return reinterpret_cast<const uint16_t*>(vec + n_vec);
  }
};

// Counts eight values, two to a word, if all are in the direct range; else does
// nothing and returns false. With t = |x|'s bits - kMagLo the bin is kHalf - 1 - t
// for a positive value and kHalf + 1 + t for a negative one, in byte offsets below
// 2^16: both halves go through every step at once. (A half below the range borrows
// from its neighbour, but is itself far above it then, and the vector is refused.)
__device__ __forceinline__ bool count_vector(const uint4& w, uint32_t* hist) {
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
  uint32_t t[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) t[q] = (ws[q] & 0x7fff7fffu) - kMagLo * 0x10001u;
  constexpr uint32_t kMost = (kHalf - 1) * 0x10001u;
  if (max2(max2(max2(t[0], t[1]), max2(t[2], t[3])), kMost) != kMost) return false;
  const uint32_t h = smem_u32(hist);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t neg;  // each half's sign bit in all of its bits
    asm("prmt.b32 %0, %1, %1, 0xbb99;" : "=r"(neg) : "r"(ws[q]));
    const uint32_t at =
        (((kMost - t[q]) & ~neg) | ((t[q] + (kHalf + 1) * 0x10001u) & neg)) << 2;
    asm volatile("red.shared.add.u32 [%0], 1;" ::"r"(h + (at & 0xffffu)) : "memory");
    asm volatile("red.shared.add.u32 [%0], 1;" ::"r"(h + (at >> 16)) : "memory");
  }
  return true;
}
static_assert(4 * kBins < 65536, "byte offsets of the direct range");
// Counts eight values of which some may be zero, masked or outside the direct
// range; returns the flags of the latter.
__device__ __noinline__ int count_any(uint4 w, uint32_t* hist) {
  constexpr uint32_t kMasked = 0xff80ff80u;
  if (w.x == kMasked && w.y == kMasked && w.z == kMasked && w.w == kMasked) return 0;
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
  int flags = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint32_t b = q & 1 ? ws[q / 2] >> 16 : ws[q / 2] & 0xffffu;
    const int t = static_cast<int>(b & 0x7fffu) - kMagLo;
    if (static_cast<unsigned>(t) < static_cast<unsigned>(kHalf)) {
      atomicAdd(&hist[b & 0x8000u ? kHalf + 1 + t : kHalf - 1 - t], 1u);
    } else if (b != 0xff80u) {
      if (t == -kMagLo)
        atomicAdd(&hist[kHalf], 1u);
      else if (!is_masked(b))
        flags |= t < 0 ? 2 : (b & 0x8000u ? 4 : 1);
    }
  }
  return flags;
}
// The same in a window over all bf16 values that starts at position lo.
__device__ __noinline__ void count_in_window(uint4 w, int lo, uint32_t* hist) {
#pragma unroll 1
  for (int q = 0; q < 8; ++q) {
    const uint32_t b = w.x & 0xffffu;
    w.x = __funnelshift_r(w.x, w.y, 16);
    w.y = __funnelshift_r(w.y, w.z, 16);
    w.z = __funnelshift_r(w.z, w.w, 16);
    w.w >>= 16;
    const int k = full_key(b) - lo;
    if (k >= 0 && k < kBinsPad && !is_masked(b)) atomicAdd(&hist[k], 1u);
  }
}

// Zeroes the histogram and counts the slice's values of window `win` in it.
// Returns what the thread met outside the direct range, and the position of its
// largest value.
template <int kThr>
__device__ __forceinline__ int2 count_slice(const Slice& sl, int win, uint32_t* hist) {
  int flags = 0;
  __nv_bfloat162 most = __halves2bfloat162(__ushort_as_bfloat16(0xff80u), __ushort_as_bfloat16(0xff80u));
  auto one_vector = [&](const uint4& w) {
    if (win != kDirect) {
      count_in_window(w, win * kBinsPad, hist);
      return;
    }
    const __nv_bfloat162* f = reinterpret_cast<const __nv_bfloat162*>(&w);
    most = __hmax2(most, __hmax2(__hmax2(f[0], f[1]), __hmax2(f[2], f[3])));  // NaN is passed over
    if (!count_vector(w, hist)) flags |= count_any(w, hist);
  };
  const uint4* v = sl.vec;
  const int n = sl.n_vec;
  bool zeroed = false;
#pragma unroll 1
  for (int i = threadIdx.x; i < n || !zeroed; i += kBatch * kThr) {
    uint4 w[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (i + k * kThr < n) w[k] = v[i + k * kThr];
    if (!zeroed) {  // while the first loads are under way
      uint4* h = reinterpret_cast<uint4*>(hist);
#pragma unroll 4
      for (int j = threadIdx.x; j < kBinsPad / 4; j += kThr) h[j] = make_uint4(0u, 0u, 0u, 0u);
      __syncthreads();
      zeroed = true;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (i + k * kThr < n) one_vector(w[k]);
  }
  if (threadIdx.x < sl.n_head + sl.n_tail) {
    const int i = threadIdx.x;
    const uint32_t b = i < sl.n_head ? sl.x[i] : sl.tail()[i - sl.n_head];
    one_vector(make_uint4(0xff800000u | b, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u));
  }
  const uint16_t m = __bfloat16_as_ushort(__hmax(__low2bfloat16(most), __high2bfloat16(most)));
  return make_int2(flags, is_masked(m) ? kNone : full_key(m));
}

// ------------------------------------------------------------ one row
template <int kC, int kThr>
struct Row {
  static constexpr int kWarps = kThr / 32;
  static constexpr int kShare = kRows / kC;                    // rows of bins that a CTA sums
  static constexpr int kOwn = (kRows + kThr - 1) / kThr;       // rows of a thread of CTA 0

  uint32_t* hist;
  RowShared* sh;
  int cta;
  float t, z_max, x_max, min_p;
  ScaleDiv div;     // z = x / t
  int fix;
  bool valid;       // the settings are in range
  int window;       // what the histogram holds
  int top;          // the position of the row's largest value, kNone if there is none
  int flags;        // what the row holds outside the direct range
  // CTA 0: what comes before this thread's rows of bins in the built window, and
  // their own totals
  u64 m0, mn;
  uint32_t c0, cn;

  __device__ __forceinline__ int bin_key(int bin) const {
    if (window != kDirect) return window * kBinsPad + bin;
    if (bin < kHalf) return 32767 - (kMagHi - bin);
    return bin == kHalf ? 32767 : 32767 + (bin - kHalf - 1 + kMagLo);
  }
  __device__ __forceinline__ void set_max(int key) {
    x_max = key_value(key);
    z_max = __fdiv_rn(x_max, t);
  }
  // x / t rounded to nearest; in the direct range ScaleDiv's short form holds
  // for every usual temperature (zero divides exactly)
  __device__ __forceinline__ float divide(float v) const {
    if (window != kDirect || div.r == 0.f) return __fdiv_rn(v, t);
    float lo, hi;
    f2_unpack(div.fast_quotient2(f2_pack(v, v)), lo, hi);
    return lo;
  }
  // exp(z - m) of one value in fp32, and as an integer
  __device__ __forceinline__ float weight(float v) const {
    if (v == x_max) return 1.f;
    const float z = divide(v);
    const float d = __fsub_rn(z, z_max);
    if (!(d > -45.f)) return 0.f;
    // what the subtraction rounded off (Knuth's two-sum)
    const float bb = __fsub_rn(d, z);
    const float err = __fsub_rn(__fsub_rn(z, __fsub_rn(d, bb)), __fadd_rn(z_max, bb));
    const float w = expf(d);
    return fmaf(w, err, w);
  }
  __device__ __forceinline__ u64 fixed(float w) const {
    return __float2ull_rn(w * __uint_as_float(static_cast<uint32_t>(127 + fix) << 23));
  }

  // Counts window `win` of the row over the cluster: after the direct range top,
  // flags and the settings that all CTAs use are the whole row's. Another barrier
  // follows (weigh, or the caller's): until then the CTAs read each other's counts.
  __device__ __forceinline__ void count(const Slice& sl, int win) {
    window = win;
    if (threadIdx.x == 0) {
      sh->flags = 0;
      sh->top = kNone;
    }
    const int2 mine = count_slice<kThr>(sl, win, hist);  // its barrier also covers the two above
    const int f = __reduce_or_sync(0xffffffffu, mine.x);
    const int b = __reduce_min_sync(0xffffffffu, mine.y);
    if ((threadIdx.x & 31) == 0) {
      if (f) atomicOr(&sh->flags, f);
      if (b != kNone) atomicMin(&sh->top, b);
    }
    __syncthreads();
    if constexpr (kC == 1) {
      flags = sh->flags;
      top = sh->top;
      t = sh->set.t;
      min_p = sh->set.min_p;
    } else {
      // every CTA of the cluster has started: its memory can be written
      if (win == kDirect) row_wait();
      if (threadIdx.x < kC)
        st_peer_v4(peer<kC>(&sh->seen[cta], threadIdx.x),
                   make_int4(sh->flags, sh->top, __float_as_int(sh->set.t),
                             __float_as_int(sh->set.min_p)));
      row_sync<kC>();
      flags = 0;
      top = kNone;
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        flags |= sh->seen[c].x;
        top = min(top, sh->seen[c].y);
      }
      t = __int_as_float(sh->seen[0].z);
      min_p = __int_as_float(sh->seen[0].w);
    }
    valid = t >= 0.f;  // NaN where a setting is out of range
    if (t == 0.f) t = 1.f;  // greedy: the log-prob is that of temperature 1
  }

  // Sums this CTA's share of the bins over the cluster (in place: no one else
  // reads that share here), weighs them, one lane a bin, and leaves every row's
  // totals in CTA 0, whose threads then hold the prefixes. Returns the window's
  // totals (in CTA 0). x_max must be set.
  __device__ __forceinline__ Totals weigh() {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    u64 q = 0;
#pragma unroll 1
    for (int row = cta * kShare + warp; row < (cta + 1) * kShare; row += kWarps) {
      const int bin = 32 * row + lane;
      uint32_t n = 0;
      if constexpr (kC > 1) {
        uint32_t v[kC];
#pragma unroll
        for (int c = 0; c < kC; ++c) v[c] = ld_peer_u32(peer<kC>(hist + bin, c));
#pragma unroll
        for (int c = 0; c < kC; ++c) n += v[c];
        hist[bin] = n;
      } else {
        n = hist[bin];
      }
      uint32_t c = 0;
      u64 m = 0;
      if (__any_sync(0xffffffffu, n)) {
        if (n) {
          const float w = weight(key_value(bin_key(bin)));
          m = n * fixed(w);
          if (w >= min_p) q += m;
        }
        c = __reduce_add_sync(0xffffffffu, n);
        // a sum of 32 pieces of 22 bits fits 32
        const u64 p0 = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(m) & 0x3fffffu);
        const u64 p1 = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(m >> 22) & 0x3fffffu);
        const u64 p2 = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(m >> 44));
        m = p0 + (p1 << 22) + (p2 << 44);
      }
      if (lane == 0) {
        st_peer_u64(peer<kC>(&sh->row_m[row], 0), m);
        st_shared_cluster_u32(peer<kC>(&sh->row_c[row], 0), c);
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) q += __shfl_xor_sync(0xffffffffu, q, off);
    if constexpr (kC == 1) {
      if (lane == 0) sh->warp[warp].kept = q;
      __syncthreads();
    } else {
      if (lane == 0) sh->warp[warp].kept = q;
      __syncthreads();
      if (threadIdx.x == 0) {
        u64 all = 0;
        for (int w = 0; w < kWarps; ++w) all += sh->warp[w].kept;
        st_peer_u64(peer<kC>(&sh->kept[cta], 0), all);
      }
      row_sync<kC>();
      if (cta != 0) return Totals{0, 0, 0};
    }
    // exclusive prefixes over CTA 0's threads, in order of the rows
    cn = 0;
    mn = 0;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int row = threadIdx.x * kOwn + i;
      if (row < kRows) {
        cn += sh->row_c[row];
        mn += sh->row_m[row];
      }
    }
    uint32_t ic = cn;
    u64 im = mn;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t oc = __shfl_up_sync(0xffffffffu, ic, off);
      const u64 om = __shfl_up_sync(0xffffffffu, im, off);
      if (lane >= off) {
        ic += oc;
        im += om;
      }
    }
    if (lane == 31) {
      sh->warp[warp].mass = im;
      sh->warp[warp].count = ic;
    }
    __syncthreads();
    c0 = ic - cn;
    m0 = im - mn;
    Totals all{0, 0, 0};
#pragma unroll 4
    for (int w = 0; w < kWarps; ++w) {
      const Totals x = sh->warp[w];
      if (w < warp) {
        c0 += x.count;
        m0 += x.mass;
      }
      all.count += x.count;
      all.mass += x.mass;
      if (kC == 1) all.kept += x.kept;
    }
    if constexpr (kC > 1) {
#pragma unroll
      for (int c = 0; c < kC; ++c) all.kept += sh->kept[c];
    }
    return all;
  }

  // CTA 0: the token of rank `at` in the built window (by_mass false), or where
  // its running mass passes `at`; returns the mass up to and with it, and leaves
  // its bin and its rank among the bin's tokens in sh. The thread that owns the
  // crossing's row has its warp look at the bins, one lane each.
  __device__ __forceinline__ u64 cross(bool by_mass, u64 at) {
    const int lane = threadIdx.x & 31;
    const bool mine = by_mass ? m0 <= at && at - m0 < mn : c0 <= at && at - c0 < cn;
    const uint32_t who = __ballot_sync(0xffffffffu, mine);
    __syncthreads();  // the last crossing has been read
    if (who) {
      const int src = __ffs(who) - 1;
      u64 m = __shfl_sync(0xffffffffu, m0, src);
      uint32_t c = __shfl_sync(0xffffffffu, c0, src);
      int row = ((threadIdx.x & ~31) + src) * kOwn;
      if constexpr (kOwn > 1) {  // which of the thread's rows
#pragma unroll
        for (int i = 1; i < kOwn; ++i) {
          const u64 rm = sh->row_m[row];
          const uint32_t rc = sh->row_c[row];
          if (by_mass ? at - m >= rm : at - c >= rc) {
            m += rm;
            c += rc;
            ++row;
          } else {
            break;
          }
        }
      }
      const int bin = 32 * row + lane;
      const uint32_t n = ld_peer_u32(peer<kC>(hist + bin, row / kShare));
      const u64 w = n ? fixed(weight(key_value(bin_key(bin)))) : 0u;
      uint32_t ic = n;
      u64 im = n * w;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t oc = __shfl_up_sync(0xffffffffu, ic, off);
        const u64 om = __shfl_up_sync(0xffffffffu, im, off);
        if (lane >= off) {
          ic += oc;
          im += om;
        }
      }
      m += im - n * w;  // before this bin
      c += ic - n;
      const u64 rest = by_mass ? at - m : at - c;  // huge where the crossing comes before
      if (rest < (by_mass ? n * w : static_cast<u64>(n))) {
        u64 j = rest;  // the rank among the bin's tokens
        if (by_mass) {
          j = static_cast<u64>(__fdividef(static_cast<float>(rest), static_cast<float>(w)));
          while (j * w > rest) --j;
          while ((j + 1) * w <= rest) ++j;
        }
        sh->found = m + (j + 1) * w;
        sh->found_bin = bin;
        sh->found_rank = static_cast<uint32_t>(j);
      }
    }
    __syncthreads();
    return sh->found;
  }

  // CTA 0's first warp: who holds the token that the last crossing found, from
  // the CTAs' own counts of its value (one CTA's was replaced by the sum).
  __device__ __forceinline__ int4 locate() const {
    const int lane = threadIdx.x & 31;
    const int bin = sh->found_bin, summed = bin / 32 / kShare;
    const uint32_t rank = sh->found_rank;
    if constexpr (kC == 1) return make_int4(kLook, 0, bin_key(bin), static_cast<int>(rank));
    uint32_t own = lane < kC ? ld_peer_u32(peer<kC>(hist + bin, min(lane, kC - 1))) : 0u;
    const uint32_t others = __reduce_add_sync(0xffffffffu, lane == summed ? 0u : own);
    if (lane == summed) own -= others;
    uint32_t to = own;
#pragma unroll
    for (int off = 1; off < kC; off <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, to, off);
      if (lane >= off) to += o;
    }
    const uint32_t here = __ballot_sync(0xffffffffu, rank >= to - own && rank < to);
    // No CTA holds it where the row changed between two counts of it: then CTA 0
    // looks for a rank that no row has, finds nothing and writes token -1.
    const int who = here ? __ffs(here) - 1 : 0;
    const uint32_t there = __shfl_sync(0xffffffffu, rank - (to - own), who);
    return make_int4(kLook, who, bin_key(bin), here ? static_cast<int>(there) : kNone);
  }
};

// floor(f * m) for an fp32 f in [0, 1], and whether that is f * m itself.
__device__ __forceinline__ u64 scaled_floor(float f, u64 m, bool& exact) {
  const uint32_t b = __float_as_uint(f) & 0x7fffffffu;  // -0 is 0
  const int e = static_cast<int>(b >> 23);
  const u64 mant = e ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
  const int s = 150 - max(e, 1);  // f = mant * 2^-s, s >= 23
  const u64 hi = __umul64hi(mant, m), lo = mant * m;
  if (s >= 128) {
    exact = (hi | lo) == 0;
    return 0;
  }
  if (s >= 64) {
    const u64 q = s == 64 ? hi : hi >> (s - 64);
    exact = lo == 0 && (s == 64 || (q << (s - 64)) == hi);
    return q;
  }
  exact = (lo << (64 - s)) == 0;
  return (hi << (64 - s)) | (lo >> s);
}

// One bit per matching half of a word: `mask` drops the sign where zero is sought.
__device__ __forceinline__ uint32_t match2(uint32_t w, uint32_t mask, uint32_t want) {
  return min2((w & mask) ^ want, 0x00010001u) ^ 0x00010001u;
}
// Whether a vector holds a match at all, in fewer steps.
__device__ __forceinline__ bool any_match(const uint4& w, uint32_t mask, uint32_t want) {
  const uint32_t m = min2(min2((w.x & mask) ^ want, (w.y & mask) ^ want),
                          min2((w.z & mask) ^ want, (w.w & mask) ^ want));
  return (m & 0xffffu) == 0u || m < 0x10000u;
}
// The matches of a vector: word k's halves at bits k and 16 + k.
__device__ __forceinline__ uint32_t match8(const uint4& w, uint32_t mask, uint32_t want) {
  return match2(w.x, mask, want) | (match2(w.y, mask, want) << 1) |
         (match2(w.z, mask, want) << 2) | (match2(w.w, mask, want) << 3);
}

// Index in the row of the slice's rank-th element (from 0) with this key, -1 if it
// has fewer (a row that changed since it was counted). The slice goes by in
// chunks, each warp holding 128 consecutive vectors of one, until the chunk that
// has the element; half a slice on average. The elements before the vectors go
// with the first chunk's first warp, those after them with the last one's last.
template <int kThr>
__device__ __forceinline__ int64_t index_of(const Slice& sl, RowShared* sh, int key,
                                            uint32_t rank) {
  constexpr int kWarps = kThr / 32, kDepth = 4, kChunk = kThr * kDepth;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t bits = __float_as_uint(key_value(key)) >> 16;
  const uint32_t want = bits | (bits << 16);
  const uint32_t mask = bits ? 0xffffffffu : 0x7fff7fffu;
  // which of n (at most 7) single elements match
  auto ends = [&](const uint16_t* x, int n) {
    return __ballot_sync(0xffffffffu, lane < n && (x[min(lane, 7)] & mask & 0xffffu) == bits);
  };
  auto nth = [](uint32_t m, uint32_t n) {  // position of the n-th set bit
    for (; n > 0; --n) m &= m - 1;
    return __ffs(m) - 1;
  };
  uint32_t left = rank;
  const int base = 32 * kDepth * warp + lane;
  int turn = 0;
#pragma unroll 1
  for (int c0 = 0;; c0 += kChunk, turn ^= 1) {
    const bool last = c0 + kChunk >= sl.n_vec;
    uint4 w[kDepth];
    uint32_t m[kDepth];
    uint32_t n = 0;
#pragma unroll
    for (int k = 0; k < kDepth; ++k)
      if (c0 + base + 32 * k < sl.n_vec) w[k] = sl.vec[c0 + base + 32 * k];
    uint32_t head = 0, tail = 0;
    if (c0 == 0 && warp == 0) head = ends(sl.x, sl.n_head);
    if (last && warp == kWarps - 1) tail = ends(sl.tail(), sl.n_tail);
#pragma unroll
    for (int k = 0; k < kDepth; ++k) {
      m[k] = 0;
      if (c0 + base + 32 * k < sl.n_vec && any_match(w[k], mask, want)) {
        m[k] = match8(w[k], mask, want);
        n += __popc(m[k]);
      }
    }
    n = __reduce_add_sync(0xffffffffu, n) + __popc(head) + __popc(tail);
    if (lane == 0) sh->hits[turn][warp] = n;
    __syncthreads();  // the turn before the last has been read by then
    uint32_t inc = lane < kWarps ? sh->hits[turn][lane] : 0u;
#pragma unroll
    for (int off = 1; off < kWarps; off <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += o;
    }
    const uint32_t all = __shfl_sync(0xffffffffu, inc, kWarps - 1);
    if (left < all) {
      const uint32_t before = __shfl_sync(0xffffffffu, inc, warp) - n;
      if (left >= before && left - before < n) {
        left -= before;
        if (left < __popc(head)) {
          if (lane == 0) sh->index = nth(head, left);
        } else {
          left -= __popc(head);
#pragma unroll
          for (int k = 0; k < kDepth; ++k) {
            uint32_t sum = __popc(m[k]);
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
              const uint32_t o = __shfl_up_sync(0xffffffffu, sum, off);
              if (lane >= off) sum += o;
            }
            const uint32_t low = sum - __popc(m[k]);
            if (low <= left && left < sum) {
              uint32_t in_order = 0;  // bit i: element i of the lane's vector
              for (int i = 0; i < 8; ++i) in_order |= ((m[k] >> (16 * (i & 1) + i / 2)) & 1u) << i;
              const uint16_t* v = reinterpret_cast<const uint16_t*>(sl.vec + c0 + base + 32 * k);
              sh->index = v - sl.x + nth(in_order, left - low);
            }
            left -= __shfl_sync(0xffffffffu, sum, 31);  // wraps past zero once it is found
          }
          if (left < __popc(tail) && lane == 0) sh->index = sl.tail() - sl.x + nth(tail, left);
        }
      }
      __syncthreads();
      return sh->index;
    }
    if (last) return -1;
    left -= all;
  }
}

// One row per cluster of kC CTAs, each counting a contiguous part of it, each
// weighing a share of the bins. CTA 0 takes the cuts and the draw and sends its
// order to all: look for the token (the CTA that holds it), or count a window.
template <int kC, int kThr, int kMin>
__global__ void __launch_bounds__(kThr, kMin) sample_kernel(const SampleParams p) {
  __shared__ __align__(16) uint32_t hist[kBinsPad];
  __shared__ RowShared sh;
  const int cta = kC > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t row = blockIdx.x / kC;
  const Slice sl(p.logits + row * p.ld, p.V, cta, kC);
  Row<kC, kThr> r;
  r.hist = hist;
  r.sh = &sh;
  r.cta = cta;
  r.fix = p.fix;

  if constexpr (kC > 1) row_arrive();  // the first count waits for it
  // Whatever the CTAs and threads have to agree on goes through one copy in shared
  // memory: a caller's other stream that writes a setting or a logit meanwhile gets
  // a senseless token, but all threads meet at the same barriers. A crossing that
  // finds nothing leaves the values below, which are always a bin.
  if (threadIdx.x == 0) {
    sh.set.load(p, row);  // the first count's barrier covers it
    sh.found = 0;
    sh.found_bin = 0;
    sh.found_rank = 0;
  }

  // The row's totals, from the direct range or window by window; then up to
  // three crossings, each in the window that holds it (built again if need be).
  Totals all{0, 0, 0};
  uint32_t wc[kWindows];
  u64 wm[kWindows];
  int n_win = 1, win = kDirect;
  bool totals = true;
  int step = 0;  // 0: top-k, 1: top-p, 2: the draw
  u64 kept = 0;
  int4 order;
#pragma unroll 1
  for (;;) {
    r.count(sl, win);
    const Settings s = sh.set;
    if (win == kDirect) {
      r.div = ScaleDiv::make(r.t);
      if (s.t == 0.f) step = 2;
      const bool none = r.top == kNone;
      if (!none) r.set_max(r.top);
      if (!r.valid || none) {  // nothing to draw, or a setting out of range
        if (cta == 0 && threadIdx.x == 0) {
          p.token[row] = -1;
          if (p.logprob) p.logprob[row] = r.valid ? 0.f : __int_as_float(0x7fffffff);
        }
        return;  // all of the cluster, after a barrier that ended all its reads
      }
      // does a value outside the direct range matter?
      if ((r.flags & 1) || ((r.flags & 2) && !(__fdiv_rn(0x1p-32f, r.t) - r.z_max < kTail)) ||
          ((r.flags & 4) && !(__fdiv_rn(-256.f, r.t) - r.z_max < kTail))) {
        n_win = kWindows;
        win = 0;
        row_sync<kC>();  // every CTA has read what the others have seen
        continue;
      }
    }
    const Totals a = r.weigh();
    if (totals) {
      const int w = max(win, 0);
      wc[w] = a.count;
      wm[w] = a.mass;
      all.count += a.count;
      all.mass += a.mass;
      all.kept += a.kept;
      if (w + 1 < n_win) {
        ++win;
        continue;
      }
      totals = false;
      kept = all.mass;
    }
    if (cta == 0) {
      order = make_int4(kBuild, 0, 0, 0);
#pragma unroll 1
      for (; step < 3; ++step) {
        u64 at, before = 0;
        bool exact;
        int w = 0;
        if (step == 0) {
          if (s.top_k == 0 || static_cast<uint32_t>(s.top_k) >= all.count) continue;
          at = static_cast<u64>(s.top_k) - 1;
          while (w + 1 < n_win && at >= wc[w]) {
            at -= wc[w];
            before += wm[w++];
          }
        } else {
          if (step == 1) {
            if (!(s.top_p < 1.f)) continue;
            at = scaled_floor(s.top_p, kept, exact);
            if (exact && at > 0) --at;  // the token that brings the mass to at + 1 or more
          } else {
            if (all.kept < kept) kept = all.kept;
            at = s.t == 0.f ? 0 : scaled_floor(s.u, kept, exact);
            if (s.t != 0.f && at >= kept) at = kept - 1;
          }
          while (w + 1 < n_win && at >= wm[w]) {
            at -= wm[w];
            before += wm[w++];
          }
        }
        if (n_win > 1 && r.window != w) {
          order.y = w;
          break;
        }
        kept = before + r.cross(step > 0, at);
      }
      if (threadIdx.x < 32) {
        if (step == 3) order = r.locate();
        if (kC > 1) {
          if (threadIdx.x < kC) st_peer_v4(peer<kC>(&sh.order, threadIdx.x), order);
        } else if (threadIdx.x == 0) {
          sh.order = order;
        }
      }
    }
    row_sync<kC>();
    order = sh.order;
    if (order.x == kLook) break;
    win = order.y;
    row_sync<kC>();  // every CTA has the order
  }
  // no CTA reads another's memory from here on
  if (order.y == cta) {
    const int64_t index = index_of<kThr>(sl, &sh, order.z, static_cast<uint32_t>(order.w));
    if (threadIdx.x == 0) p.token[row] = static_cast<int32_t>(index);
  }
  if (p.logprob && cta == 0 && threadIdx.x == kThr - 1) {
    // d - ln(mass * 2^-fix), the logarithm as that of a number in [1, 2) and a
    // multiple of ln 2 whose first part is exact
    const float v = key_value(order.z);
    const float z = __fdiv_rn(v, r.t);
    const float d = v == r.x_max ? 0.f : __fsub_rn(z, r.z_max);
    const float lost =  // what the difference rounded off; 0 where z overflows
        v == r.x_max ? 0.f
                     : __fsub_rn(__fsub_rn(z, __fsub_rn(d, __fsub_rn(d, z))),
                                 __fadd_rn(r.z_max, __fsub_rn(d, z)));
    const int e = 63 - __clzll(static_cast<long long>(all.mass));
    const float f = __ull2float_rn(all.mass) * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    const float k = static_cast<float>(e - p.fix);
    p.logprob[row] = (d - k * 0x1.62ep-1f) + (lost - fmaf(k, 0x1.0bfbe8p-15f, logf(f)));
  }
}

struct LaunchConfig {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  LaunchConfig(int64_t rows, int ctas, int threads, cudaStream_t st) {
    cfg.gridDim = dim3(static_cast<unsigned>(rows * ctas));
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
  }
};

template <int kC, int kThr, int kMin>
cudaError_t launch_sample(const SampleParams& p, cudaStream_t st) {
  LaunchConfig c(p.T, kC, kThr, st);
  return cudaLaunchKernelEx(&c.cfg, sample_kernel<kC, kThr, kMin>, p);
}

// Rows whose clusters of kC CTAs are on the device at once, one CTA to an SM.
template <int kC>
cudaError_t rows_at_once(int sms, int64_t* rows) {
  static std::atomic<int> cached[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int n = dev >= 0 && dev < 64 ? cached[dev].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    LaunchConfig c(sms / kC, kC, 512, nullptr);
    if ((e = cudaOccupancyMaxActiveClusters(&n, sample_kernel<kC, 512, 1>, &c.cfg)) != cudaSuccess)
      return e;
    n = (n < sms / kC ? n : sms / kC) + 1;
    if (dev >= 0 && dev < 64) cached[dev].store(n, std::memory_order_relaxed);
  }
  *rows = n - 1;
  return cudaSuccess;
}

// How a batch is split. A call is a chain of short steps, so a row gets as many
// CTAs as leave one to an SM; past one CTA a row they share SMs, two of 512 threads
// and then four of 256. Measured at V = 32000 / 152064 (us; 8, 4, 2, 1, 1 shared by
// two, 1 of 256 threads shared by four):
//   4 rows    10.8 / 12.0   11.7 / 14.7   13.3 / 19.9   14.2 / 27.8   15.7 / 27.0   21.4 / 33.2
//   32 rows   28.1 / 30.7   12.1 / 15.5   13.7 / 20.5   14.6 / 27.3   15.9 / 28.9   21.7 / 39.3
//   64 rows   45.4 / 50.3   22.8 / 28.6   13.7 / 20.8   14.6 / 27.7   16.1 / 28.8   22.1 / 39.5
//   150 rows  90.9 / 101    51.0 / 64.6   26.6 / 41.2   14.9 / 28.9   16.2 / 29.9   21.9 / 41.8
//   300 rows   177 / 200    93.4 / 122    51.8 / 82.4   28.0 / 59.0   22.7 / 49.6   25.2 / 60.5
//   1024 rows  610 / 673     309 / 393     179 / 272    98.2 / 186    72.6 / 153    62.3 / 156
cudaError_t launch_by_rows(const SampleParams& p, int sms, cudaStream_t st) {
  int64_t n8 = 0, n4 = 0, n2 = 0;
  cudaError_t e;
  if ((e = rows_at_once<8>(sms, &n8)) != cudaSuccess ||
      (e = rows_at_once<4>(sms, &n4)) != cudaSuccess ||
      (e = rows_at_once<2>(sms, &n2)) != cudaSuccess)
    return e;
  if (p.T <= n8) return launch_sample<8, 512, 1>(p, st);
  if (p.T <= n4) return launch_sample<4, 512, 1>(p, st);
  if (p.T <= n2) return launch_sample<2, 512, 1>(p, st);
  if (p.T <= sms) return launch_sample<1, 512, 1>(p, st);
  if (p.T <= 2 * sms) return launch_sample<1, 512, 2>(p, st);
  return launch_sample<1, 256, 4>(p, st);
}

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

}  // namespace

}  // namespace lmh

extern "C" int lmhead_sample(const uint16_t* logits, int64_t T, int64_t V, int64_t ld_logits,
                             float temperature, const float* row_temperature, int32_t top_k,
                             const int32_t* row_top_k, float top_p, const float* row_top_p,
                             float min_p, const float* row_min_p, const float* uniform,
                             int32_t* out_token, float* out_logprob,
                             struct CUstream_st* stream) {
  using namespace lmh;
  if (T < 0 || T > LMH_MAX_DIM / 8 || V < 1 || V > LMH_MAX_DIM)
    return api_set_error(LMH_ERR_INVALID_ARG, "T or V out of range");
  if (ld_logits < V)
    return api_set_error(LMH_ERR_INVALID_ARG, "ld_logits must be at least V");
  if (!row_temperature && !(std::isfinite(temperature) && temperature >= 0.f))
    return api_set_error(LMH_ERR_INVALID_ARG, "temperature must be finite and >= 0");
  if (!row_top_k && top_k < 0)
    return api_set_error(LMH_ERR_INVALID_ARG, "top_k must be >= 0 (0: off)");
  if (!row_top_p && !(top_p > 0.f && top_p <= 1.f))
    return api_set_error(LMH_ERR_INVALID_ARG, "top_p must be in (0, 1]");
  if (!row_min_p && !(min_p >= 0.f && min_p <= 1.f))
    return api_set_error(LMH_ERR_INVALID_ARG, "min_p must be in [0, 1]");
  if (T == 0) return api_set_error(LMH_OK, "");
  if (!logits || !uniform || !out_token)
    return api_set_error(LMH_ERR_INVALID_ARG, "logits, uniform and out_token are required");
  if (misaligned(logits, 2) || misaligned(uniform, 4) || misaligned(out_token, 4) ||
      misaligned(out_logprob, 4) || misaligned(row_temperature, 4) || misaligned(row_top_k, 4) ||
      misaligned(row_top_p, 4) || misaligned(row_min_p, 4))
    return api_set_error(LMH_ERR_ALIGNMENT, "logits need 2-byte, the rest 4-byte alignment");
  int sms = 0;
  unsigned* status = nullptr;
  const int rc = api_device(&sms, &status);
  if (rc != LMH_OK) return rc;
  SampleParams p{};
  p.logits = logits;
  p.T = T;
  p.V = V;
  p.ld = ld_logits;
  p.temperature = temperature;
  p.top_p = top_p;
  p.min_p = min_p;
  p.top_k = top_k;
  p.row_t = row_temperature;
  p.row_p = row_top_p;
  p.row_m = row_min_p;
  p.row_k = row_top_k;
  p.uniform = uniform;
  p.token = out_token;
  p.logprob = out_logprob;
  // V weights of at most 2^fix stay below 2^63
  int bits = 0;
  while ((int64_t{1} << bits) < V) ++bits;
  p.fix = 63 - bits < 44 ? 63 - bits : 44;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  {
    KernelTimer timer(K_SAMPLE, st);
    e = launch_by_rows(p, sms, st);
    if (e == cudaSuccess) note_launch();
  }
  if (e != cudaSuccess) {
    char msg[256];
    snprintf(msg, sizeof(msg), "sampling: %s", cudaGetErrorString(e));
    return api_set_error(LMH_ERR_LAUNCH, msg);
  }
  return api_set_error(LMH_OK, "");
}
