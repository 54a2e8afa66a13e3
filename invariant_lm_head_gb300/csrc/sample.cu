// Sampling from bf16 logits (sm_103a): temperature, top-k, top-p and min-p, one
// token per row from a given uniform number.
//
// A row's bf16 logits take few distinct values, and everything the sampler
// decides depends on a token only through its logit and, among equal ones, its
// index. So a row is read once into a histogram of counts over the ordered
// values (shared memory, integer adds), and all later work is on the
// histogram: with m the largest z = x / t (fp32 division), a bin's weight is
// exp(z - m), held as an integer in units of 2^-44, and its mass is count *
// weight. Sums of integers are exact and have no order, so the result is the
// same whatever adds first. Tokens are taken in descending logit, ties by
// index:
//   top-k   the first k;
//   top-p   the shortest prefix of those whose mass reaches p of their mass;
//   min-p   those of weight >= min_p;
//   draw    the first of the kept whose running mass exceeds u * kept mass.
// Each is a prefix of one order, so each is one crossing of the histogram's
// running count or mass. The crossing gives a value and a rank among its equal
// tokens; a second look at the row (from L2) turns the rank into an index.
//
// Bins. The histogram covers zero and every bf16 of magnitude [2^-32, 2^8),
// one bin per value. A row that holds another value whose weight matters (the
// lowest finite value as a mask does not, next to real logits) is taken in
// seven windows over all bf16 values instead, the row read again for each.
#include <cstdint>
#include <cstdio>
#include <cmath>

#include "internal.h"
#include "lmhead.h"
#include "ptx.cuh"

namespace lmh {

namespace {

constexpr int kSThreads = 512;
constexpr int kSWarps = kSThreads / 32;
constexpr int kBatch = 5;  // 16-byte loads in flight per thread
constexpr int kMaxC = 8;   // most CTAs of a row (a portable cluster)
// Magnitude bits (sign dropped) of the direct range.
constexpr int kMagLo = (127 - 32) << 7;         // 2^-32
constexpr int kMagHi = ((127 + 8) << 7) - 1;    // largest below 2^8
constexpr int kHalf = kMagHi - kMagLo + 1;      // values of one sign: 5120
constexpr int kBins = 2 * kHalf + 1;            // 10241
constexpr int kBinsPad = 10752;                 // whole 16-byte vectors for 1, 2, 4 or 8 CTAs
static_assert(kBinsPad >= kBins && kBinsPad % (4 * kMaxC) == 0, "bins");
// Every bf16 value in descending order: positive 0 .. 32766, zero 32767,
// negative 32768 .. 65534 (inf and NaN magnitudes included).
constexpr int kFullKeys = 65535;
constexpr int kWindows = (kFullKeys + kBinsPad - 1) / kBinsPad;
constexpr int kDirect = -1;  // the direct range, beside windows 0 .. kWindows - 1
constexpr int kNoBin = 0x7fffffff;
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

// What a row asks for; load() is false when a setting is out of range.
struct Settings {
  float t, top_p, min_p, u;
  int top_k;
  __device__ __forceinline__ bool load(const SampleParams& p, int64_t row) {
    t = p.row_t ? p.row_t[row] : p.temperature;
    top_p = p.row_p ? p.row_p[row] : p.top_p;
    min_p = p.row_m ? p.row_m[row] : p.min_p;
    top_k = p.row_k ? p.row_k[row] : p.top_k;
    u = p.uniform[row];
    return t >= 0.f && t <= 3.402823466e38f && top_p > 0.f && min_p <= 1.f && u >= 0.f &&
           u <= 1.f && top_k >= 0;
  }
};

// Where the running count or mass passes a point: the value's key, the token's
// rank among its equals, the mass up to and with it.
struct Crossing {
  u64 upto;
  int key;
  uint32_t rank;
};

struct Totals {
  u64 count, mass, kept;  // kept: the mass that min-p keeps
};

struct RowShared {
  Totals part[kMaxC];       // every CTA's share of the built window
  Crossing found[2];
  u64 warp_c[kSWarps], warp_m[kSWarps], warp_q[kSWarps];
  int64_t index;
  uint32_t hits[kBatch + 1][kSWarps];
  int flags;                // 1: above the direct range, 2: tiny, 4: below the range
  int top;                  // smallest occupied bin of the CTA's own counts
  int cmd_key;              // the token to look for: its key (-1: not in this CTA)
  uint32_t cmd_rank;        // and its rank among the CTA's own tokens of that key
};

// ------------------------------------------------------------ the cluster
template <int kC>
__device__ __forceinline__ void row_sync() {
  if constexpr (kC > 1)
    cluster_sync();
  else
    __syncthreads();
}
// The address of the same shared variable in CTA c.
template <int kC>
__device__ __forceinline__ uint32_t peer(const void* here, int c) {
  return kC > 1 ? mapa_shared(smem_u32(here), static_cast<uint32_t>(c)) : smem_u32(here);
}
__device__ __forceinline__ uint4 ld_peer_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_peer_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_peer_u64(uint32_t addr, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// ------------------------------------------------------------ reading a row
// A CTA's part of a row in index order: 2-byte steps up to the row's first
// 16-byte boundary (the first CTA), a run of 16-byte vectors, and the row's last
// elements (the last CTA).
struct Slice {
  const uint16_t* x;   // the row
  int64_t head;        // elements before the row's first vector
  int64_t v0, v1;      // this CTA's vectors
  int n_head, n_tail;  // this CTA's elements before and after them (at most 7)
  __device__ __forceinline__ Slice(const uint16_t* row, int64_t V, int rank, int n_ranks) : x(row) {
    const int64_t to16 = ((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) >> 1;
    head = to16 < V ? to16 : V;
    const int64_t nv = (V - head) >> 3;
    const int64_t per = (nv + n_ranks - 1) / n_ranks;
    v0 = min(nv, per * rank);
    v1 = min(nv, v0 + per);
    n_head = rank == 0 ? static_cast<int>(head) : 0;
    n_tail = rank == n_ranks - 1 ? static_cast<int>(V - head - 8 * nv) : 0;
  }
  __device__ __forceinline__ const uint4* vec() const {
    return reinterpret_cast<const uint4*>(x + head);
  }
  __device__ __forceinline__ const uint16_t* tail() const { return x + head + 8 * v1; }
};

// What a CTA has seen besides its counts.
struct Seen {
  int flags = 0;
  int top = kNoBin;
};

// Counts one value in the direct range.
__device__ __forceinline__ bool count_in_range(uint32_t b, uint32_t* hist, Seen& seen) {
  const int t = static_cast<int>(b & 0x7fffu) - (kMagLo - 1);
  const bool in = static_cast<unsigned>(t - 1) < static_cast<unsigned>(kHalf);
  const int bin = (b & 0x8000u) ? kHalf + t : kHalf - t;
  if (in) {
    atomicAdd(&hist[bin], 1u);
    seen.top = min(seen.top, bin);
  }
  return in;
}
// The others: zero, masked, or outside the range.
__device__ __forceinline__ void count_rest(uint32_t b, uint32_t* hist, Seen& seen) {
  const uint32_t mag = b & 0x7fffu;
  if (mag == 0u) {
    atomicAdd(&hist[kHalf], 1u);
    seen.top = min(seen.top, kHalf);
  } else if (!is_masked(b)) {
    seen.flags |= mag < kMagLo ? 2 : ((b & 0x8000u) ? 4 : 1);
  }
}
__device__ __forceinline__ void count_in_window(uint32_t b, int lo, uint32_t* hist, Seen& seen) {
  const int k = full_key(b) - lo;
  if (k >= 0 && k < kBinsPad && !is_masked(b)) {
    atomicAdd(&hist[k], 1u);
    seen.top = min(seen.top, k);
  }
}

// Zeroes the histogram and counts the slice's values of window `win` in it.
__device__ __forceinline__ Seen count_slice(const Slice& sl, int win, uint32_t* hist) {
  Seen seen;
  const uint4* v = sl.vec();
  bool zeroed = false;
  for (int64_t i0 = sl.v0 + threadIdx.x; !zeroed || i0 < sl.v1; i0 += kBatch * kSThreads) {
    uint4 w[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (i0 + k * kSThreads < sl.v1) w[k] = v[i0 + k * kSThreads];
    if (!zeroed) {  // while the first loads are under way
      uint4* h = reinterpret_cast<uint4*>(hist);
      for (int i = threadIdx.x; i < kBinsPad / 4; i += kSThreads) h[i] = make_uint4(0u, 0u, 0u, 0u);
      __syncthreads();
      zeroed = true;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (i0 + k * kSThreads >= sl.v1) continue;
      const uint32_t ws[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
      if (win == kDirect) {
        bool all = true;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          all &= count_in_range(ws[q] & 0xffffu, hist, seen);
          all &= count_in_range(ws[q] >> 16, hist, seen);
        }
        if (!all) {
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const uint32_t b = q & 1 ? ws[q / 2] >> 16 : ws[q / 2] & 0xffffu;
            const uint32_t mag = b & 0x7fffu;
            if (mag < kMagLo || mag > kMagHi) count_rest(b, hist, seen);
          }
        }
      } else {
#pragma unroll 1
        for (int q = 0; q < 8; ++q) {
          const uint32_t b = (ws[q / 2] >> (16 * (q & 1))) & 0xffffu;
          count_in_window(b, win * kBinsPad, hist, seen);
        }
      }
    }
  }
  if (threadIdx.x < sl.n_head + sl.n_tail) {
    const int i = threadIdx.x;
    const uint32_t b = i < sl.n_head ? sl.x[i] : sl.tail()[i - sl.n_head];
    if (win != kDirect)
      count_in_window(b, win * kBinsPad, hist, seen);
    else if (!count_in_range(b, hist, seen))
      count_rest(b, hist, seen);
  }
  return seen;
}

// ------------------------------------------------------------ one row
template <int kC>
struct Row {
  static constexpr int kShare = kBinsPad / kC;  // bins that a CTA sums over the cluster
  static constexpr int kVec = (kShare / 4 + kSThreads - 1) / kSThreads;  // 16-byte vectors a thread
  static constexpr int kOwn = 4 * kVec;         // bins of one thread
  static_assert(kOwn <= 32, "one lane per bin in a crossing");

  uint32_t* hist;
  RowShared* sh;
  int cta;
  float t, z_max, x_max, min_p;
  int fix;
  int window;       // what the histogram holds
  int top;          // the window's smallest occupied bin, kNoBin if none
  int flags;        // what the row holds outside the direct range
  int turn;         // which of the two result slots is next
  // this thread's bins in the built window: what comes before them, and their totals
  u64 c0, cn, m0, mn;

  __device__ __forceinline__ int bin_key(int bin) const {
    if (window != kDirect) return window * kBinsPad + bin;
    if (bin < kHalf) return 32767 - (kMagHi - bin);
    return bin == kHalf ? 32767 : 32767 + (bin - kHalf - 1 + kMagLo);
  }
  __device__ __forceinline__ void set_max(int key) {
    x_max = key_value(key);
    z_max = __fdiv_rn(x_max, t);
  }
  // exp(z - m) of one value in fp32, and as an integer
  __device__ __forceinline__ float weight(float v) const {
    if (v == x_max) return 1.f;
    const float z = __fdiv_rn(v, t);
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

  // Counts window `win` of the row over the cluster: afterwards top and flags
  // are the whole row's. Two barriers follow (finish): between them the CTAs read
  // each other's counts.
  __device__ __forceinline__ void count(const Slice& sl, int win) {
    window = win;
    if (threadIdx.x == 0) {
      sh->flags = 0;
      sh->top = kNoBin;
    }
    const Seen seen = count_slice(sl, win, hist);  // its barrier also covers the two above
    const int f = __reduce_or_sync(0xffffffffu, seen.flags);
    const int b = __reduce_min_sync(0xffffffffu, seen.top);
    if ((threadIdx.x & 31) == 0) {
      if (f) atomicOr(&sh->flags, f);
      if (b != kNoBin) atomicMin(&sh->top, b);
    }
    row_sync<kC>();
    flags = 0;
    top = kNoBin;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      flags |= static_cast<int>(ld_peer_u32(peer<kC>(&sh->flags, c)));
      top = min(top, static_cast<int>(ld_peer_u32(peer<kC>(&sh->top, c))));
    }
  }

  // Sums this CTA's share of the bins over the cluster (in place: no one else
  // reads that share here), weighs them, and returns the window's totals. x_max
  // must be set.
  __device__ __forceinline__ Totals finish() {
    uint4* h = reinterpret_cast<uint4*>(hist + cta * kShare) + threadIdx.x * kVec;
    uint4 n[kVec];
    u64 q = 0;
    cn = mn = 0;
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      n[k] = make_uint4(0u, 0u, 0u, 0u);
      if (static_cast<int>(threadIdx.x) * kVec + k < kShare / 4) {
        if constexpr (kC > 1) {
          uint4 v[kC];
#pragma unroll
          for (int c = 0; c < kC; ++c) v[c] = ld_peer_v4(peer<kC>(h + k, c));
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            n[k].x += v[c].x;
            n[k].y += v[c].y;
            n[k].z += v[c].z;
            n[k].w += v[c].w;
          }
          h[k] = n[k];
        } else {
          n[k] = h[k];
        }
      }
    }
    const int bin0 = cta * kShare + threadIdx.x * kOwn;
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      const uint32_t ns[4] = {n[k].x, n[k].y, n[k].z, n[k].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (ns[j]) {
          const float w = weight(key_value(bin_key(bin0 + 4 * k + j)));
          const u64 mass = ns[j] * fixed(w);
          cn += ns[j];
          mn += mass;
          if (w >= min_p) q += mass;
        }
      }
    }
    // exclusive prefixes over the CTA's threads
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    u64 ic = cn, im = mn;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const u64 oc = __shfl_up_sync(0xffffffffu, ic, off), om = __shfl_up_sync(0xffffffffu, im, off);
      if (lane >= off) {
        ic += oc;
        im += om;
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) q += __shfl_xor_sync(0xffffffffu, q, off);
    if (lane == 31) {
      sh->warp_c[warp] = ic;
      sh->warp_m[warp] = im;
      sh->warp_q[warp] = q;
    }
    __syncthreads();
    c0 = ic - cn;
    m0 = im - mn;
    Totals mine{0, 0, 0};
#pragma unroll
    for (int w = 0; w < kSWarps; ++w) {
      if (w < warp) {
        c0 += sh->warp_c[w];
        m0 += sh->warp_m[w];
      }
      mine.count += sh->warp_c[w];
      mine.mass += sh->warp_m[w];
      mine.kept += sh->warp_q[w];
    }
    if (threadIdx.x < kC) {
      const uint32_t to = peer<kC>(&sh->part[cta], threadIdx.x);
      st_peer_u64(to, mine.count);
      st_peer_u64(to + 8, mine.mass);
      st_peer_u64(to + 16, mine.kept);
    }
    row_sync<kC>();
    Totals all{0, 0, 0};
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      if (c < cta) {
        c0 += sh->part[c].count;
        m0 += sh->part[c].mass;
      }
      all.count += sh->part[c].count;
      all.mass += sh->part[c].mass;
      all.kept += sh->part[c].kept;
    }
    return all;
  }

  // The token of rank `at` in the built window (kMass false), or where its
  // running mass passes `at`. The thread that owns the crossing's bins has its
  // warp look at them, one lane each, and tells every CTA. With kLast the CTA that
  // holds the token is told to look for it.
  template <bool kMass, bool kLast>
  __device__ __forceinline__ Crossing cross(u64 at) {
    const int lane = threadIdx.x & 31;
    const bool mine = kMass ? m0 <= at && at - m0 < mn : c0 <= at && at - c0 < cn;
    const uint32_t who = __ballot_sync(0xffffffffu, mine);
    if (who) {
      const int src = __ffs(who) - 1;
      const u64 bm = __shfl_sync(0xffffffffu, m0, src), bc = __shfl_sync(0xffffffffu, c0, src);
      const int bin = cta * kShare + ((threadIdx.x & ~31) + src) * kOwn + lane;
      // a thread's last vectors may lie beyond the share: it counted none of them
      const u64 n = lane < kOwn && bin < (cta + 1) * kShare ? hist[bin] : 0u;
      const u64 w = n ? fixed(weight(key_value(bin_key(bin)))) : 0u;
      u64 c = n, m = n * w;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const u64 oc = __shfl_up_sync(0xffffffffu, c, off);
        const u64 om = __shfl_up_sync(0xffffffffu, m, off);
        if (lane >= off) {
          c += oc;
          m += om;
        }
      }
      c += bc - n;  // before this bin
      m += bm - n * w;
      const bool here = kMass ? m <= at && at - m < n * w : c <= at && at - c < n;
      const int at_lane = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
      // the rank among the bin's tokens; the quotient is below 2^32
      u64 j = at - c;
      if (kMass && here) {
        const u64 rest = at - m;
        j = static_cast<u64>(__fdividef(static_cast<float>(rest), static_cast<float>(w)));
        while (j * w > rest) --j;
        while ((j + 1) * w <= rest) ++j;
      }
      const u64 upto = __shfl_sync(0xffffffffu, m + (j + 1) * w, at_lane);
      uint32_t rank = __shfl_sync(0xffffffffu, static_cast<uint32_t>(j), at_lane);
      const int hit = __shfl_sync(0xffffffffu, bin, at_lane);
      const int key = bin_key(hit);
      if (lane < kC) {
        const uint32_t to = peer<kC>(&sh->found[turn], lane);
        st_peer_u64(to, upto);
        st_peer_u64(to + 8, static_cast<u64>(static_cast<uint32_t>(key)) |
                                (static_cast<u64>(rank) << 32));
      }
      if constexpr (kLast) {
        // each CTA's own count: this CTA's was replaced by the sum
        uint32_t own = lane < kC && lane != cta ? ld_peer_u32(peer<kC>(hist + hit, min(lane, kC - 1))) : 0u;
        const uint32_t others = __reduce_add_sync(0xffffffffu, own);
        if (lane == cta) own = hist[hit] - others;
        uint32_t upto_c = own;
#pragma unroll
        for (int off = 1; off < kC; off <<= 1) {
          const uint32_t o = __shfl_up_sync(0xffffffffu, upto_c, off);
          if (lane >= off) upto_c += o;
        }
        if (lane < kC && rank >= upto_c - own && rank < upto_c) {
          st_shared_cluster_u32(peer<kC>(&sh->cmd_rank, lane), rank - (upto_c - own));
          st_shared_cluster_u32(peer<kC>(&sh->cmd_key, lane), static_cast<uint32_t>(key));
        }
      }
    }
    row_sync<kC>();
    const Crossing r = sh->found[turn];
    turn ^= 1;
    return r;
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

// Index in the row of the slice's rank-th element (from 0) with this key.
// A batch's matches are counted per vector row and warp, in index order.
__device__ __forceinline__ int64_t index_of(const Slice& sl, RowShared* sh, int key,
                                            uint32_t rank) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto match = [&](uint32_t b) { return full_key(b) == key ? 1u : 0u; };
  // the elements before and after the vectors: every warp counts the former
  const uint32_t h = __ballot_sync(0xffffffffu, lane < sl.n_head && match(sl.x[lane]));
  if (rank < __popc(h)) {
    uint32_t m = h;
    for (uint32_t s = rank; s > 0; --s) m &= m - 1;
    return __ffs(m) - 1;
  }
  uint32_t left = rank - __popc(h);
  for (int64_t i0 = sl.v0; i0 < sl.v1; i0 += kBatch * kSThreads) {
    uint4 w[kBatch];
    uint32_t bits[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int64_t i = i0 + k * kSThreads + threadIdx.x;
      if (i < sl.v1) w[k] = sl.vec()[i];
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int64_t i = i0 + k * kSThreads + threadIdx.x;
      bits[k] = 0;
      if (i < sl.v1) {
        const uint32_t ws[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
        for (int q = 0; q < 4; ++q)
          bits[k] |= (match(ws[q] & 0xffffu) << (2 * q)) | (match(ws[q] >> 16) << (2 * q + 1));
      }
      const uint32_t n = __reduce_add_sync(0xffffffffu, __popc(bits[k]));
      if (lane == 0) sh->hits[k][warp] = n;
    }
    __syncthreads();
    uint32_t before = 0, at_k = kBatch, at_w = 0, at_before = 0;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
#pragma unroll
      for (int x = 0; x < kSWarps; ++x) {
        const uint32_t n = sh->hits[k][x];
        if (at_k == kBatch && left < before + n) {
          at_k = k;
          at_w = x;
          at_before = before;
        }
        before += n;
      }
    }
    if (at_k < kBatch) {
      if (warp == static_cast<int>(at_w)) {
        uint32_t mine = 0;
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (k == static_cast<int>(at_k)) mine = bits[k];
        uint32_t inc = __popc(mine);
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const uint32_t o = __shfl_up_sync(0xffffffffu, inc, off);
          if (lane >= off) inc += o;
        }
        const uint32_t want = left - at_before, low = inc - __popc(mine);
        if (low <= want && want < inc) {
          for (uint32_t s = want - low; s > 0; --s) mine &= mine - 1;
          sh->index = sl.head + 8 * (i0 + at_k * kSThreads + threadIdx.x) + __ffs(mine) - 1;
        }
      }
      __syncthreads();
      return sh->index;
    }
    left -= before;
    __syncthreads();  // the counts have been read
  }
  const uint32_t m0 = __ballot_sync(0xffffffffu, lane < sl.n_tail && match(sl.tail()[lane]));
  uint32_t m = m0;
  for (uint32_t s = left; s > 0; --s) m &= m - 1;
  return sl.tail() - sl.x + __ffs(m) - 1;
}

// One row per cluster of kC CTAs, each counting a contiguous part of it, each
// weighing a share of the bins; every step that needs the whole row ends with a
// cluster barrier, after which all CTAs hold the same numbers and go the same way.
template <int kC>
__global__ void __launch_bounds__(kSThreads, 2) sample_kernel(const SampleParams p) {
  __shared__ __align__(16) uint32_t hist[kBinsPad];
  __shared__ RowShared sh;
  const int cta = kC > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t row = blockIdx.x / kC;
  Settings s;
  if (!s.load(p, row)) {
    if (cta == 0 && threadIdx.x == 0) {
      p.token[row] = -1;
      if (p.logprob) p.logprob[row] = __int_as_float(0x7fffffff);
    }
    return;  // the whole cluster leaves
  }
  const bool greedy = s.t == 0.f;
  const Slice sl(p.logits + row * p.ld, p.V, cta, kC);
  Row<kC> r;
  r.hist = hist;
  r.sh = &sh;
  r.cta = cta;
  r.t = greedy ? 1.f : s.t;
  r.min_p = s.min_p;
  r.fix = p.fix;
  r.turn = 0;
  if (threadIdx.x == 0) sh.cmd_key = -1;

  r.count(sl, kDirect);
  if (r.top != kNoBin) r.set_max(r.bin_key(r.top));
  // does a value outside the direct range matter?
  const bool none = r.top == kNoBin;
  const bool windows =
      (r.flags & 1) ||
      ((r.flags & 2) && (none || !(__fdiv_rn(0x1p-32f, r.t) - r.z_max < kTail))) ||
      ((r.flags & 4) && (none || !(__fdiv_rn(-256.f, r.t) - r.z_max < kTail)));
  if (none && !windows) {  // nothing to draw
    if (cta == 0 && threadIdx.x == 0) {
      p.token[row] = -1;
      if (p.logprob) p.logprob[row] = 0.f;
    }
    row_sync<kC>();  // the others have read this CTA's flags
    return;
  }

  Totals all{0, 0, 0};
  u64 wc[kWindows], wm[kWindows];
  const int n_win = windows ? kWindows : 1;
  if (!windows) {
    all = r.finish();
    wc[0] = all.count;
    wm[0] = all.mass;
  } else {
    row_sync<kC>();
    bool any = false;
#pragma unroll 1
    for (int w = 0; w < kWindows; ++w) {
      r.count(sl, w);
      if (!any && r.top != kNoBin) {
        r.set_max(r.bin_key(r.top));
        any = true;
      }
      if (!any) {
        wc[w] = wm[w] = 0;
        row_sync<kC>();
        continue;
      }
      const Totals a = r.finish();
      wc[w] = a.count;
      wm[w] = a.mass;
      all.count += a.count;
      all.mass += a.mass;
      all.kept += a.kept;
    }
  }
  auto enter = [&](int w) {  // make window w the built one
    if (!windows || r.window == w) return;
    r.count(sl, w);
    r.finish();
  };
  // the window where the running mass passes `at`, and the mass before it
  auto find_mass = [&](u64 at, u64& before) {
    int w = 0;
    before = 0;
    while (w + 1 < n_win && at - before >= wm[w]) before += wm[w++];
    return w;
  };

  u64 at = 0;  // the draw: the first token whose running mass exceeds it
  if (!greedy) {
    u64 kept = all.mass, before;
    bool exact;
    if (s.top_k > 0 && static_cast<u64>(s.top_k) < all.count) {
      u64 c = 0, m = 0;
      int w = 0;
      while (static_cast<u64>(s.top_k) - c > wc[w]) {
        c += wc[w];
        m += wm[w++];
      }
      enter(w);
      kept = m + r.template cross<false, false>(s.top_k - c - 1).upto;
    }
    if (s.top_p < 1.f) {
      u64 reach = scaled_floor(s.top_p, kept, exact);
      if (!exact) ++reach;
      reach = reach < 1 ? 1 : reach;
      const int w = find_mass(reach - 1, before);
      enter(w);
      kept = before + r.template cross<true, false>(reach - 1 - before).upto;
    }
    if (all.kept < kept) kept = all.kept;
    at = scaled_floor(s.u, kept, exact);
    if (at >= kept) at = kept - 1;
  }
  u64 before;
  const int w_at = find_mass(at, before);
  enter(w_at);
  const Crossing c = r.template cross<true, true>(at - before);
  // no CTA reads another's memory from here on
  if (sh.cmd_key >= 0) {
    const int64_t index = index_of(sl, &sh, sh.cmd_key, sh.cmd_rank);
    if (threadIdx.x == 0) p.token[row] = static_cast<int32_t>(index);
  }
  if (p.logprob && cta == kC - 1 && threadIdx.x == kSThreads - 1) {
    // d - ln(mass * 2^-fix), the logarithm as that of a number in [1, 2) and a
    // multiple of ln 2 whose first part is exact
    const float v = key_value(c.key);
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

template <int kC>
cudaError_t launch_sample(const SampleParams& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.T * kC));
  cfg.blockDim = dim3(kSThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = kC;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<kC>, p);
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
    const int64_t slots = 2 * static_cast<int64_t>(sms);  // CTAs at work at once
    if (T * 8 <= slots)
      e = launch_sample<8>(p, st);
    else if (T * 4 <= slots)
      e = launch_sample<4>(p, st);
    else if (T * 2 <= slots)
      e = launch_sample<2>(p, st);
    else
      e = launch_sample<1>(p, st);
    if (e == cudaSuccess) note_launch();
  }
  if (e != cudaSuccess) {
    char msg[256];
    snprintf(msg, sizeof(msg), "sampling: %s", cudaGetErrorString(e));
    return api_set_error(LMH_ERR_LAUNCH, msg);
  }
  return api_set_error(LMH_OK, "");
}
