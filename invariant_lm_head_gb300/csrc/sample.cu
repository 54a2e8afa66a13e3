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
// Magnitude bits (sign dropped) of the histogram's range.
constexpr int kMagLo = (127 - 32) << 7;         // 2^-32
constexpr int kMagHi = ((127 + 8) << 7) - 1;    // largest below 2^8
constexpr int kHalf = kMagHi - kMagLo + 1;      // values of one sign: 5120
constexpr int kBins = 2 * kHalf + 1;            // 10241
constexpr int kPer = 21;                        // bins per thread (odd: no bank conflicts)
constexpr int kBinsPad = kPer * kSThreads;      // 10752
static_assert(kBinsPad >= kBins, "every bin needs an owner");
// Every bf16 value in descending order: positive 0 .. 32766, zero 32767,
// negative 32768 .. 65534 (inf and NaN magnitudes included).
constexpr int kFullKeys = 65535;
constexpr int kWindows = (kFullKeys + kBinsPad - 1) / kBinsPad;
// A weight below 2^-45 is zero: d < -45 ln 2.
constexpr float kTail = -31.2f;

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

typedef unsigned long long u64;

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

struct RowShared {
  int flags;       // 1: above the range, 2: tiny, 4: below the range
  int top;         // smallest occupied bin of a window
  uint32_t cnt;    // results of a crossing search
  u64 mass;
  int bin;
  u64 sc[kSWarps], sm[kSWarps], sq[kSWarps];
};

// One row's running state in a CTA.
struct Row {
  const uint16_t* x;
  int64_t V;
  uint32_t* hist;
  RowShared* sh;
  float t, z_max, x_max, min_p;
  int fix;
  int window;       // window held by the histogram: -1 the direct range
  // this thread's exclusive prefix of the built window
  uint32_t c0, cn;
  u64 m0, mn;

  __device__ __forceinline__ int bin_key(int bin) const {
    if (window >= 0) return window * kBinsPad + bin;
    if (bin < kHalf) return 32767 - (kMagHi - bin);
    return bin == kHalf ? 32767 : 32767 + (bin - kHalf - 1 + kMagLo);
  }
  __device__ __forceinline__ int n_bins() const {
    return window < 0 ? kBins : min(kBinsPad, kFullKeys - window * kBinsPad);
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
};

// f(value bits) for every element of the row, whatever its address: 2-byte
// steps up to the first 16-byte boundary, 16-byte loads, 2-byte steps.
template <class F>
__device__ __forceinline__ void for_row(const uint16_t* x, int64_t n, F&& f) {
  const int64_t head =
      min(n, static_cast<int64_t>(((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) >> 1));
  const int64_t nv = (n - head) >> 3;
  for (int64_t i = threadIdx.x; i < head; i += kSThreads) f(static_cast<uint32_t>(x[i]));
  const uint4* v = reinterpret_cast<const uint4*>(x + head);
  for (int64_t i = threadIdx.x; i < nv; i += kSThreads) {
    const uint4 w = v[i];
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f(ws[q] & 0xffffu);
      f(ws[q] >> 16);
    }
  }
  for (int64_t i = head + nv * 8 + threadIdx.x; i < n; i += kSThreads)
    f(static_cast<uint32_t>(x[i]));
}

// Counts the row's values in the direct range; r.sh->flags tells what else it holds.
__device__ void build_direct(Row& r) {
  __syncthreads();
  for (int i = threadIdx.x; i < kBinsPad; i += kSThreads) r.hist[i] = 0u;
  if (threadIdx.x == 0) r.sh->flags = 0;
  __syncthreads();
  int flags = 0;
  uint32_t* hist = r.hist;
  for_row(r.x, r.V, [&](uint32_t b) {
    const int mag = static_cast<int>(b & 0x7fffu);
    const bool neg = b & 0x8000u;
    if (mag >= kMagLo && mag <= kMagHi) {
      atomicAdd(&hist[neg ? kHalf + 1 + (mag - kMagLo) : kMagHi - mag], 1u);
    } else if (mag == 0) {
      atomicAdd(&hist[kHalf], 1u);
    } else if (!is_masked(b)) {
      flags |= mag < kMagLo ? 2 : (neg ? 4 : 1);
    }
  });
  if (flags) atomicOr(&r.sh->flags, flags);
  r.window = -1;
  __syncthreads();
}

__device__ void build_window(Row& r, int w) {
  __syncthreads();
  for (int i = threadIdx.x; i < kBinsPad; i += kSThreads) r.hist[i] = 0u;
  __syncthreads();
  uint32_t* hist = r.hist;
  const int lo = w * kBinsPad;
  for_row(r.x, r.V, [&](uint32_t b) {
    if (is_masked(b)) return;
    const int k = full_key(b) - lo;
    if (k >= 0 && k < kBinsPad) atomicAdd(&hist[k], 1u);
  });
  r.window = w;
  __syncthreads();
}

// The first occupied bin of the built window, or -1.
__device__ int top_bin(Row& r) {
  if (threadIdx.x == 0) r.sh->top = 0x7fffffff;
  __syncthreads();
  for (int i = 0; i < kPer; ++i) {
    const int bin = threadIdx.x * kPer + i;
    if (r.hist[bin]) {
      atomicMin(&r.sh->top, bin);
      break;
    }
  }
  __syncthreads();
  const int top = r.sh->top;
  __syncthreads();
  return top == 0x7fffffff ? -1 : top;
}

// Exclusive prefixes of count and mass over the built window, kept per thread;
// returns the window's totals, and the mass of the bins that min-p keeps.
__device__ void scan_window(Row& r, u64& total_c, u64& total_m, u64& total_q) {
  u64 c = 0, m = 0, q = 0;
  const int nb = r.n_bins();
  for (int i = 0; i < kPer; ++i) {
    const int bin = threadIdx.x * kPer + i;
    const uint32_t n = bin < nb ? r.hist[bin] : 0u;
    if (n) {
      const float w = r.weight(key_value(r.bin_key(bin)));
      const u64 mass = n * r.fixed(w);
      c += n;
      m += mass;
      if (w >= r.min_p) q += mass;
    }
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 ic = c, im = m;
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
    r.sh->sc[warp] = ic;
    r.sh->sm[warp] = im;
    r.sh->sq[warp] = q;
  }
  __syncthreads();
  u64 bc = 0, bm = 0;
  total_c = total_m = total_q = 0;
  for (int w = 0; w < kSWarps; ++w) {
    if (w == warp) {
      bc = total_c;
      bm = total_m;
    }
    total_c += r.sh->sc[w];
    total_m += r.sh->sm[w];
    total_q += r.sh->sq[w];
  }
  r.c0 = static_cast<uint32_t>(bc + ic - c);
  r.cn = static_cast<uint32_t>(c);
  r.m0 = bm + im - m;
  r.mn = m;
  __syncthreads();
}

// Mass of the first `count` tokens of the built window (0 < count <= its total).
__device__ u64 mass_of_count(Row& r, uint32_t count) {
  const uint32_t at = count - 1;
  if (r.c0 <= at && at - r.c0 < r.cn) {
    uint32_t c = r.c0;
    u64 m = r.m0;
    for (int i = 0; i < kPer; ++i) {
      const int bin = threadIdx.x * kPer + i;
      const uint32_t n = r.hist[bin];
      if (!n) continue;
      const u64 w = r.fixed(r.weight(key_value(r.bin_key(bin))));
      if (at - c < n) {
        r.sh->mass = m + (at - c + 1) * w;
        break;
      }
      c += n;
      m += n * w;
    }
  }
  __syncthreads();
  const u64 v = r.sh->mass;
  __syncthreads();
  return v;
}

// The token at running mass `at` of the built window (0 <= at < its total): its
// bin, its rank among the bin's tokens, and the mass up to and with it.
__device__ void at_mass(Row& r, u64 at, int& bin_out, uint32_t& rank, u64& upto) {
  if (r.m0 <= at && at - r.m0 < r.mn) {
    u64 m = r.m0;
    for (int i = 0; i < kPer; ++i) {
      const int bin = threadIdx.x * kPer + i;
      const uint32_t n = r.hist[bin];
      if (!n) continue;
      const u64 w = r.fixed(r.weight(key_value(r.bin_key(bin))));
      if (at - m < n * w) {
        const u64 j = (at - m) / w;
        r.sh->bin = bin;
        r.sh->cnt = static_cast<uint32_t>(j);
        r.sh->mass = m + (j + 1) * w;
        break;
      }
      m += n * w;
    }
  }
  __syncthreads();
  bin_out = r.sh->bin;
  rank = r.sh->cnt;
  upto = r.sh->mass;
  __syncthreads();
}

// Index of the rank-th element (from 0) of the row whose value has this key. Each
// warp owns a contiguous part of the row, in index order.
__device__ int64_t index_of(Row& r, int key, uint32_t rank) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t per = (r.V + kSWarps - 1) / kSWarps;
  const int64_t b = min(r.V, per * warp), e = min(r.V, per * (warp + 1));
  uint32_t n = 0;
  for (int64_t i = b + lane; i < e; i += 32)
    n += full_key(r.x[i]) == key;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) n += __shfl_xor_sync(0xffffffffu, n, off);
  if (lane == 0) r.sh->sc[warp] = n;
  __syncthreads();
  uint32_t before = 0;
  for (int w = 0; w < warp; ++w) before += static_cast<uint32_t>(r.sh->sc[w]);
  if (rank >= before && rank - before < n) {
    uint32_t left = rank - before;
    for (int64_t i = b; i < e; i += 32) {
      const int64_t j = i + lane;
      const bool hit = j < e && full_key(r.x[j]) == key;
      const uint32_t mask = __ballot_sync(0xffffffffu, hit);
      const uint32_t k = __popc(mask);
      if (left < k) {
        if (hit && __popc(mask & ((1u << lane) - 1u)) == left) r.sh->mass = static_cast<u64>(j);
        break;
      }
      left -= k;
    }
  }
  __syncthreads();
  const int64_t v = static_cast<int64_t>(r.sh->mass);
  __syncthreads();
  return v;
}

__global__ void __launch_bounds__(kSThreads) sample_kernel(const SampleParams p) {
  __shared__ uint32_t hist[kBinsPad];
  __shared__ RowShared sh;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    const float t_in = p.row_t ? p.row_t[row] : p.temperature;
    const float top_p = p.row_p ? p.row_p[row] : p.top_p;
    const float min_p = p.row_m ? p.row_m[row] : p.min_p;
    const int top_k = p.row_k ? p.row_k[row] : p.top_k;
    const float u = p.uniform[row];
    if (!(t_in >= 0.f && t_in <= 3.402823466e38f && top_p > 0.f && min_p <= 1.f && u >= 0.f &&
          u <= 1.f && top_k >= 0)) {
      if (threadIdx.x == 0) {
        p.token[row] = -1;
        if (p.logprob) p.logprob[row] = __int_as_float(0x7fffffff);
      }
      continue;
    }
    const bool greedy = t_in == 0.f;
    Row r;
    r.x = p.logits + row * p.ld;
    r.V = p.V;
    r.hist = hist;
    r.sh = &sh;
    r.t = greedy ? 1.f : t_in;
    r.min_p = min_p;
    r.fix = p.fix;

    // the maximum, and whether the direct range holds all that matters
    build_direct(r);
    const int flags = sh.flags;
    int n_win = 1, top_key = -1;
    int top = top_bin(r);
    if (top >= 0) {
      top_key = r.bin_key(top);
      r.x_max = key_value(top_key);
      r.z_max = __fdiv_rn(r.x_max, r.t);
    }
    const bool high = flags & 1;
    const bool tiny = (flags & 2) && (top < 0 || !(__fdiv_rn(0x1p-32f, r.t) - r.z_max < kTail));
    const bool low = (flags & 4) && (top < 0 || !(__fdiv_rn(-256.f, r.t) - r.z_max < kTail));
    if (high || tiny || low) {
      n_win = kWindows;
      top_key = -1;
    }
    // totals, window by window
    u64 wc[kWindows], wm[kWindows], wq[kWindows];
    u64 n_all = 0, m_all = 0, q_all = 0;
#pragma unroll 1
    for (int w = 0; w < n_win; ++w) {
      if (n_win > 1) {
        build_window(r, w);
        if (top_key < 0) {
          top = top_bin(r);
          if (top >= 0) {
            top_key = r.bin_key(top);
            r.x_max = key_value(top_key);
            r.z_max = __fdiv_rn(r.x_max, r.t);
          }
        }
      }
      if (top_key < 0) {
        wc[w] = wm[w] = wq[w] = 0;
        continue;
      }
      scan_window(r, wc[w], wm[w], wq[w]);
      n_all += wc[w];
      m_all += wm[w];
      q_all += wq[w];
    }
    if (top_key < 0) {  // nothing to draw
      if (threadIdx.x == 0) {
        p.token[row] = -1;
        if (p.logprob) p.logprob[row] = 0.f;
      }
      continue;
    }
    auto enter = [&](int w) {  // make window w the built one
      if (n_win == 1 || r.window == w) return;
      build_window(r, w);
      u64 a, b, c;
      scan_window(r, a, b, c);
    };
    // the window where the running mass passes `at`, and the mass before it
    auto find_mass = [&](u64 at, u64& before) {
      int w = 0;
      before = 0;
      while (w + 1 < n_win && at - before >= wm[w]) before += wm[w++];
      return w;
    };

    int key = top_key;
    uint32_t rank = 0;
    if (!greedy) {
      u64 kept = m_all;
      if (top_k > 0 && static_cast<u64>(top_k) < n_all) {
        u64 c = 0, m = 0;
        int w = 0;
        while (static_cast<u64>(top_k) - c > wc[w]) {
          c += wc[w];
          m += wm[w++];
        }
        enter(w);
        kept = m + mass_of_count(r, static_cast<uint32_t>(top_k - c));
      }
      if (top_p < 1.f) {
        u64 reach = static_cast<u64>(ceil(static_cast<double>(top_p) * static_cast<double>(kept)));
        reach = reach < 1 ? 1 : (reach > kept ? kept : reach);
        u64 before, upto;
        const int w = find_mass(reach - 1, before);
        enter(w);
        int bin;
        uint32_t j;
        at_mass(r, reach - 1 - before, bin, j, upto);
        kept = before + upto;
      }
      if (q_all < kept) kept = q_all;
      u64 at = static_cast<u64>(static_cast<double>(u) * static_cast<double>(kept));
      if (at >= kept) at = kept - 1;
      u64 before, upto;
      const int w = find_mass(at, before);
      enter(w);
      int bin;
      at_mass(r, at - before, bin, rank, upto);
      key = r.bin_key(bin);
    }
    const int64_t index = index_of(r, key, rank);
    if (threadIdx.x == 0) {
      p.token[row] = static_cast<int32_t>(index);
      if (p.logprob) {
        const float v = key_value(key);
        const double d = v == r.x_max ? 0.0
                                      : static_cast<double>(__fdiv_rn(v, r.t)) -
                                            static_cast<double>(r.z_max);
        p.logprob[row] =
            static_cast<float>(d - log(ldexp(static_cast<double>(m_all), -p.fix)));
      }
    }
  }
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
  if (T < 0 || T > LMH_MAX_DIM || V < 1 || V > LMH_MAX_DIM)
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
    const int64_t grid = T < 4 * sms ? T : 4 * sms;
    sample_kernel<<<static_cast<unsigned>(grid), kSThreads, 0, st>>>(p);
    e = cudaGetLastError();
    if (e == cudaSuccess) note_launch();
  }
  if (e != cudaSuccess) {
    char msg[256];
    snprintf(msg, sizeof(msg), "sampling: %s", cudaGetErrorString(e));
    return api_set_error(LMH_ERR_LAUNCH, msg);
  }
  return api_set_error(LMH_OK, "");
}
