// sample.cu -- sd_sample: temperature, top-k, top-p, min-p, the draw and the
// truncated row, one thread-block cluster per row.
//
// The row is read once: each CTA of the cluster holds a slice of it in shared
// memory, and every later pass (maximum, counts, sums, the truncated row) runs
// from there.
//
// Weights.  w = 2^-t, t = (m - z) * log2(e) / tau, as an integer multiple of
// 2^-43, so a row of up to 2^20 of them sums exactly in 64 bits and no result
// depends on the order of summation.  They are formed in floats: t is split
// into 4096ths and a rest, 2^-t comes from two 64-entry tables of 2^-x (pairs
// of floats) and a cubic in the rest, about 2^-36 relative.  Rounding weights
// to fewer bits would move cumulative sums past a border (top-p's or the
// draw's) once in 1e4 rows.  That arithmetic, about 27 instructions a token,
// is what bounds rows that need every weight (plain and top-p draws); the
// passes below see to it that other rows need few.
//
// Selection.  A kept set is one (value, index) pair, the cut: the last token of
// the order that is kept.  It is found in one of three ways.
//   A list: every thread knows the maximum of its tokens.  The bin that holds
//   the k-th largest of these maxima is a floor under the k-th largest token,
//   and few tokens beyond k lie above it.  Those go to CTA 0, which ranks them
//   (pairwise up to kFew, sorted up to kItems) and does all the rest there:
//   top-k up to kSmallK.  (Trying it for a top-p alone, where some of the
//   maxima seem to hold its share, gained 5 % at one shape and cost as much at
//   others.)
//   By value: bf16 rows hold few distinct values, so tokens are counted by
//   value (nine octaves of magnitudes of each sign, one atomic addition a
//   token), the order's counts and masses are scanned, and the cut is the n-th
//   token, by index, of one value: 20 us of a row of 129280, against 28 (top-k)
//   and 54 (top-k and top-p) for the next way.
//   By bins: otherwise tokens are counted in 511 bins over the first 20 powers
//   of two of weight (the rest in the last bin).  A target count picks its bin
//   exactly.  For a target mass the bins' nearly exact masses pick a bin, the
//   mass above it is summed exactly, and a neighbour is tried when the target
//   does not lie inside.
//   Only that bin's members (usually a few dozen) are then compared pairwise; a
//   bin of more than kList members is binned again over its own range of
//   values, and equal values are settled by index.
//
// What bounds it.  A row of 129280 bf16 logits is 258 KB on four CTAs, two on an
// SM.  A greedy row takes 9.5 us (load 2.2, maximum 2, draw 1.2, the row out 1
// and the cluster's barriers between them), a top-k of 50 20, a top-p alone 40
// (11 of them the weights of all tokens) and a top-k of 5000 33: chains of short
// phases that two CTAs an SM overlap only in part.  1201 rows of all kinds in
// 366 us are 1.63 TB/s, a quarter of the copy rate.
#include <cooperative_groups.h>

#include <atomic>
#include <cfloat>
#include <cmath>
#include <mutex>

#include "f32x2.cuh"
#include "serving.h"
#include "wait.cuh"

namespace sdk {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 512;         // one per thread
constexpr int kList = 512;         // members compared pairwise, one per thread
constexpr int kItems = 2048;       // tokens sorted by CTA 0 ...
constexpr int kSmallK = 1024;      // ... for a top-k of up to this
constexpr int kFew = 512;          // tokens compared with one another instead
constexpr float kBinned = 20.0f;   // -log2 of the weights that have bins of their own
constexpr float kBinWidth = kBinned / (kBins - 1);
constexpr int kCodes = 9 * 128;    // bf16 magnitudes of a sign that are counted one by one: nine octaves
constexpr int kPer = (2 * kCodes + 1 + kThreads - 1) / kThreads;  // places of their order a thread
constexpr int kOneBits = 43;       // a weight of 1 is 2^43: 2^21 units of 2^-21 and a rest of 2^22 parts
constexpr int kRestBits = 22;
constexpr int kWeightBits = kOneBits + 1;  // beside it, the 20 bits of an index fit a word
constexpr int kLimb = 15;          // masses are added in limbs of 15 bits: a slice has < 2^17 elements
constexpr uint32_t kLimbMask = (1u << kLimb) - 1;
constexpr float kLog2eHi = 1.44269502162933349609375f, kLog2eLo = 1.92596299112661746887e-8f;
constexpr float kLn2 = 0.693147180559945309f;
static_assert(kBins == kThreads && kList == kThreads && kFew == kThreads, "one bin and one member per thread");
static_assert(SD_MAX_V <= 1 << (64 - kWeightBits), "an index beside a weight");

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

template <typename T>
struct Elem;
template <>
struct Elem<uint16_t> {
  static constexpr int N = 8;
  static constexpr uint16_t kNegInf = 0xFF80;
  static constexpr uint32_t kNegInfWord = 0xFF80FF80u;
  __device__ __forceinline__ static void unpack(const uint4& r, float (&f)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ static float value(uint16_t z) { return __uint_as_float(static_cast<uint32_t>(z) << 16); }
  // its largest element; NaN if it has one
  __device__ __forceinline__ static float vmax(const uint4& r) {
    uint32_t a, b;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(r.x), "r"(r.y));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(r.z), "r"(r.w));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
    return max_nan(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u));
  }
  // the vector with every element outside the mask at -inf
  __device__ __forceinline__ static uint4 keep(const uint4& r, uint32_t mask) {
    uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = (mask >> (2 * i)) & 1u ? w[i] & 0xFFFFu : 0xFF80u;
      const uint32_t hi = (mask >> (2 * i + 1)) & 1u ? w[i] & 0xFFFF0000u : 0xFF800000u;
      w[i] = lo | hi;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Elem<uint32_t> {
  static constexpr int N = 4;
  static constexpr uint32_t kNegInf = 0xFF800000u;
  static constexpr uint32_t kNegInfWord = 0xFF800000u;
  __device__ __forceinline__ static float value(uint32_t z) { return __uint_as_float(z); }
  __device__ __forceinline__ static void unpack(const uint4& r, float (&f)[4]) {
    f[0] = __uint_as_float(r.x);
    f[1] = __uint_as_float(r.y);
    f[2] = __uint_as_float(r.z);
    f[3] = __uint_as_float(r.w);
  }
  __device__ __forceinline__ static float vmax(const uint4& r) {
    return max_nan(max_nan(__uint_as_float(r.x), __uint_as_float(r.y)),
                   max_nan(__uint_as_float(r.z), __uint_as_float(r.w)));
  }
  __device__ __forceinline__ static uint4 keep(const uint4& r, uint32_t mask) {
    return make_uint4(mask & 1u ? r.x : kNegInf, mask & 2u ? r.y : kNegInf,
                      mask & 4u ? r.z : kNegInf, mask & 8u ? r.w : kNegInf);
  }
};

// Position of a token in the order, as a key that compares equal for +0 and -0.
__device__ __forceinline__ uint32_t order_key(float z) { return ordered_bits(z + 0.0f); }
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key);
}

// Shared memory of a CTA besides its slice of the row.
struct Shared {
  uint64_t bar;
  float2 t1[kExpTab], t2[kExpTab];
  uint32_t cnt[kBins];
  union {
    struct {            // CTA 0: tokens of a small top-k
      u64 items[kItems];
      u64 few_w[kFew];
    };
    struct {            // a bin at a time
      uint32_t m0[kBins], m1[kBins], m2[kBins];
      uint32_t lkey[kList], lidx[kList];
      u64 lw[kList];
    };
    struct {  // bf16 rows: counts of equal values
      uint32_t code_n[2 * kCodes], code_all[2 * kCodes];  // of this CTA, of the cluster
    };
  };
  uint32_t tiny_of[8];
  u64 tiny_mass_of[8];
  u64 scan_w[kWarps];
  uint32_t scan_c[kWarps];
  // one word per CTA of the cluster, written by its owner in every CTA
  float max_of[8], least_of[8];
  uint32_t bad_of[8], kmin_of[8], kmax_of[8], first_of[8];
  uint32_t ties_of[8][kWarps];
  u64 mass_of[8], all_of[8];
  u64 warp_sum[8][kWarps];
  // results of a step, the same in every CTA of the cluster
  uint32_t pushed;
  uint32_t bin, bin_n, base_c;
  u64 base_m;
  uint32_t cut_key, cut_idx;
};

constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer in the low bits
constexpr float kMagic12 = 1.5f * 2048.0f;    // the same at 2^-12
constexpr float kZero = 60.0f;         // -log2 of a weight that is surely nothing

// What turns a value into its weight w = 2^-t, t = (m - z) (h + l), h + l =
// log2(e) / tau.  Products with h are formed for z - shift, exact for every z
// that matters: shift = 0 while |m| h is moderate, else shift = m (z is then
// within 15 % of m, and the difference exact).
struct Scale {
  float m, h, l;  // the row's maximum; log2(e) / tau, its high part rounded down
  float shift;
  float low;      // z - shift at which t is kZero
  uint32_t km;    // (m - shift) h in 4096ths (with kMagic12's bits) ...
  float rm;       // ... and the rest

  __device__ void set(float max, float tau) {
    m = max;
    h = fminf(__fdiv_rd(kLog2eHi, tau), 3.0e38f);
    l = fminf(__fdiv_rn(__fadd_rn(__fmaf_rn(-h, tau, kLog2eHi), kLog2eLo), tau), 3.0e38f);
    shift = fabsf(m) * h < 400.0f ? 0.0f : m;
    const float v = m - shift;
    low = v - fminf(kZero / h, 3.0e38f);
    split(v, km, rm);
  }
  // v h = k / 4096 + r, |r| <= 2^-13, r within 2^-37
  __device__ __forceinline__ void split(float v, uint32_t& k, float& r) const {
    const float y = __fmaf_rn(v, h, kMagic12);
    k = __float_as_uint(y);
    r = __fmaf_rn(v, l, __fmaf_rn(v, h, -__fsub_rn(y, kMagic12)));
  }
};

// A sum of weights: `a` units of 2^-21 and `b` parts of 2^-43, both modulo 2^32
// with the magic constant's bits counted in n.  |b| <= 0.5625 * 2^22 a weight
// (half a unit and half an ulp of the weight): up to 900 weights a sum.
struct Sum {
  uint32_t a = 0, b = 0, n = 0;
  __device__ __forceinline__ u64 get() const {
    const uint32_t bits = n * __float_as_uint(kMagic);
    return (static_cast<u64>(a - bits) << kRestBits) +
           static_cast<u64>(static_cast<long long>(static_cast<int>(b - bits)));
  }
  // Adds the weights of two values (in: it counts).
  __device__ __forceinline__ void add(const Scale& s, float z0, float z1, bool in0, bool in1, const float2* t1,
                                      const float2* t2) {
    // (at a temperature beyond 1e36 s.low stops short of kZero; -inf still weighs nothing)
    in0 = in0 && z0 > -INFINITY;
    in1 = in1 && z1 > -INFINITY;
    const F2 minus = both(-1.0f), magic = both(kMagic), magic12 = both(kMagic12), h = both(s.h);
    const F2 v = pack(fmaxf(z0 - s.shift, s.low), fmaxf(z1 - s.shift, s.low));
    const F2 y = fma2(v, h, magic12);
    const F2 r = fma2(v, both(s.l), fma2(v, h, fma2(y, minus, magic12)));
    const F2 x = mul2(add2(r, both(-s.rm)), both(kLn2));  // 2^-t = 2^(-k/4096) e^x, |x| < 2^-12
    const F2 c = mul2(x, fma2(x, fma2(x, both(1.0f / 6.0f), both(0.5f)), both(1.0f)));  // e^x - 1
    float y0, y1, c0, c1;
    unpack(y, y0, y1);
    unpack(c, c0, c1);
    const uint32_t k0 = s.km - __float_as_uint(y0), k1 = s.km - __float_as_uint(y1);  // t in 4096ths, nearly
    float wh0, wl0, wh1, wl1;
    product(t1[(k0 >> 6) & 63u], t2[k0 & 63u], c0, wh0, wl0);
    product(t1[(k1 >> 6) & 63u], t2[k1 & 63u], c1, wh1, wl1);
    const F2 wh = pack(wh0, wh1), wl = pack(wl0, wl1);
    const F2 w = add2(wh, wl);  // the pair again, its low part below half an ulp
    const F2 rest_w = fma2(fma2(wh, minus, w), minus, wl);
    const F2 unit = pack(in0 ? unit_of(k0) : 0.0f, in1 ? unit_of(k1) : 0.0f);
    const F2 ya = fma2(w, unit, magic);
    const F2 rest = fma2(rest_w, unit, fma2(w, unit, fma2(ya, minus, magic)));
    const F2 yb = fma2(rest, both(static_cast<float>(1 << kRestBits)), magic);
    float a0, a1, b0, b1;
    unpack(ya, a0, a1);
    unpack(yb, b0, b1);
    a += __float_as_uint(a0) + __float_as_uint(a1);
    b += __float_as_uint(b0) + __float_as_uint(b1);
    n += 2;
  }
  // 2^-k/4096's table product, times 1 + c
  __device__ __forceinline__ static void product(float2 p, float2 q, float c, float& wh, float& wl) {
    wh = __fmul_rn(p.x, q.x);
    wl = __fmaf_rn(p.x, q.x, -wh);
    wl = __fmaf_rn(p.x, q.y, wl);
    wl = __fmaf_rn(p.y, q.x, wl);
    wl = __fmaf_rn(wh, c, wl);
  }
  __device__ __forceinline__ static float unit_of(uint32_t k) {  // 2^-(k / 4096) in units
    return __uint_as_float(((127u + kOneBits - kRestBits) << 23) - ((k >> 12) << 23));
  }
};

// One weight in units of 2^-kOneBits.
__device__ __forceinline__ u64 weight(const Scale& sc, float z, const float2* t1, const float2* t2) {
  Sum s;
  s.add(sc, z, -INFINITY, true, false, t1, t2);
  return s.get();
}

template <typename T>
struct Row {
  static constexpr int N = Elem<T>::N;
  const SampleParams& p;
  Shared& sh;
  const uint4* data;  // this CTA's slice
  int nvec, first;    // vectors of the slice, index of its first element
  int rank, C;
  float top;          // the largest of this thread's tokens (vectors tid, tid + kThreads, ...)
  float least_top;    // the smallest of these, over the cluster's threads that have tokens
  cg::cluster_group cluster;
  Scale sc;
  float bin_scale;
  int code0;  // bf16: smallest magnitude counted by value

  __device__ Shared* of(int r) const { return cluster.map_shared_rank(&sh, r); }

  __device__ __forceinline__ uint32_t bin_of(float z) const {
    const float x = __fsub_rn(sc.m, z) * bin_scale;
    return x < static_cast<float>(kBins - 1) ? static_cast<uint32_t>(x) : kBins - 1;
  }
  __device__ u64 weight_of(float z) const { return weight(sc, z, sh.t1, sh.t2); }

  // fn(value, index) of this thread's tokens.
  template <typename F>
  __device__ __forceinline__ void each(F fn) const {
    for (int v = threadIdx.x; v < nvec; v += kThreads) {
      float f[N];
      Elem<T>::unpack(data[v], f);
#pragma unroll
      for (int e = 0; e < N; ++e) fn(f[e], static_cast<uint32_t>(first + v * N + e));
    }
  }

  __device__ uint32_t block_sum(uint32_t c) {
    c = __reduce_add_sync(kFull, c);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh.scan_c[threadIdx.x >> 5] = c;
    __syncthreads();
    uint32_t s = 0;
    for (int w = 0; w < kWarps; ++w) s += sh.scan_c[w];
    return s;
  }
  __device__ static u64 warp_sum(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
  }
  __device__ u64 block_sum(u64 v) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh.scan_w[threadIdx.x >> 5] = v;
    __syncthreads();
    u64 s = 0;
    for (int w = 0; w < kWarps; ++w) s += sh.scan_w[w];
    return s;
  }

  // Inclusive scan of one count per thread.
  __device__ uint32_t scan_counts(uint32_t c) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t a = __shfl_up_sync(kFull, c, o);
      if (lane >= o) c += a;
    }
    __syncthreads();
    if (lane == 31) sh.scan_c[warp] = c;
    __syncthreads();
    for (int w = 0; w < warp; ++w) c += sh.scan_c[w];
    return c;
  }
  // Inclusive scans of one count and one mass per thread; returns the total mass.
  __device__ u64 scan(uint32_t c, u64 m, uint32_t& ci, u64& mi) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    ci = c;
    mi = m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t a = __shfl_up_sync(kFull, ci, o);
      const u64 b = __shfl_up_sync(kFull, mi, o);
      if (lane >= o) {
        ci += a;
        mi += b;
      }
    }
    __syncthreads();
    if (lane == 31) {
      sh.scan_c[warp] = ci;
      sh.scan_w[warp] = mi;
    }
    __syncthreads();
    u64 total = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) {
        ci += sh.scan_c[w];
        mi += sh.scan_w[w];
      }
      total += sh.scan_w[w];
    }
    return total;
  }

  // ---- a small top-k

  // The tokens at or above a floor under the k-th largest, in CTA 0's items
  // (unordered).  While C * k is small each CTA takes its own floor, without
  // asking the others (they would gather C times the tokens at a larger k, and
  // comparing 400 of them costs 8 us where 55 cost 1).  False: too many tokens.
  __device__ bool gather(int k) {
    const bool alone = C == 1 || C * k <= 64;
    sh.cnt[threadIdx.x] = 0;
    if (threadIdx.x == 0) sh.bin = kBins - 1;  // fewer threads with tokens than k: no floor
    __syncthreads();
    // the maxima in bins from the row's maximum down to the least of them
    const float per = fminf((kBins - 1) / fmaxf(sc.m - least_top, 1e-30f), 3.0e38f);
    if (static_cast<int>(threadIdx.x) < nvec)
      atomicAdd(&sh.cnt[min(static_cast<uint32_t>((sc.m - top) * per), kBins - 1u)], 1u);
    uint32_t c, ci;
    if (alone) {
      __syncthreads();
      c = sh.cnt[threadIdx.x];
    } else {
      cluster.sync();
      c = read_count();
    }
    ci = scan_counts(c);
    if (ci >= static_cast<uint32_t>(k) && ci - c < static_cast<uint32_t>(k)) sh.bin = threadIdx.x;
    __syncthreads();
    const uint32_t g = sh.bin;
    Shared* r0 = of(0);
    // a value that bin g and those before it lie above
    const float low = g == kBins - 1 ? -FLT_MAX : sc.m - (static_cast<float>(g) + 1.01f) / per;
    if (top >= low) {
      const auto hits_of = [&](int v) {  // of a vector, as a mask
        const uint4 x = data[v];
        uint32_t mask = 0;
        if (Elem<T>::vmax(x) >= low) {
          float f[N];
          Elem<T>::unpack(x, f);
#pragma unroll
          for (int e = 0; e < N; ++e) mask |= (f[e] >= low ? 1u : 0u) << e;
        }
        return mask;
      };
      uint32_t hits = 0;
      for (int v = threadIdx.x; v < nvec; v += kThreads) hits += __popc(hits_of(v));
      uint32_t at = atomicAdd(&r0->pushed, hits);
      for (int v = threadIdx.x; v < nvec; v += kThreads)
        for (uint32_t mask = hits_of(v); mask; mask &= mask - 1, ++at) {
          const int e = __ffs(mask) - 1;
          const float z = Elem<T>::value(reinterpret_cast<const T*>(data + v)[e]);
          if (at < kItems) r0->items[at] = static_cast<u64>(~order_key(z)) << 32 | static_cast<uint32_t>(first + v * N + e);
        }
    }
    cluster.sync();
    return r0->pushed <= kItems;
  }

  // CTA 0: items[0..n) ascending, as a bitonic network over all kItems places
  // with four consecutive ones a thread: strides below 4 stay in its registers,
  // those below 128 in its warp, and ten of the 66 steps cross shared memory.
  // With all 66 there, and the draw by a second sort, a list of 1050 took 41 us;
  // it takes 27.
  __device__ void sort_items(int n) {
    static_assert(kItems == 4 * kThreads, "four items a thread");
    const int i0 = 4 * threadIdx.x;
    u64 x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = i0 + e < n ? sh.items[i0 + e] : ~0ull;
    __syncthreads();
#pragma unroll 1
    for (int size = 2; size <= kItems; size <<= 1) {
#pragma unroll 1
      for (int stride = size >> 1; stride >= 4; stride >>= 1) {
        const bool low_first = ((i0 & size) == 0) == ((i0 & stride) == 0);  // this side keeps the smaller
        if (stride >= 128) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sh.items[i0 + e] = x[e];
          __syncthreads();
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const u64 y = stride >= 128 ? sh.items[(i0 ^ stride) + e] : __shfl_xor_sync(kFull, x[e], stride / 4);
          x[e] = (x[e] < y) == low_first ? x[e] : y;
        }
        if (stride >= 128) __syncthreads();
      }
      const auto order = [&](int a, int b, bool up) {
        if ((x[a] > x[b]) == up) {
          const u64 y = x[a];
          x[a] = x[b];
          x[b] = y;
        }
      };
      if (size > 2) {
        const bool up = (i0 & size) == 0;
        order(0, 2, up);
        order(1, 3, up);
        order(0, 1, up);
        order(2, 3, up);
      } else {
        order(0, 1, true);
        order(2, 3, false);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) sh.items[i0 + e] = x[e];
    __syncthreads();
  }

  // CTA 0, n <= kFew items gathered: each is compared with every other by
  // kThreads / n threads, which gives its rank and the mass up to it.  From the
  // floor to the cut that takes 9 us for 60 items and 15 for 250 (sorted: 24 and
  // 25).
  __device__ void few(int n, int k, bool by_p, float tp, float floor_z, float u, int row) {
    int q = 1;  // threads an item
    while (q < 32 && 2 * q * n <= kThreads) q *= 2;
    const int e = threadIdx.x / q, sub = threadIdx.x % q;
    const u64 item = e < n ? sh.items[e] : ~0ull;
    const float z = e < n ? key_value(~static_cast<uint32_t>(item >> 32)) : -INFINITY;
    const bool weighed = by_p || p.tokens != nullptr;
    u64 w = 0;
    if (e < n && weighed) w = weight_of(z);
    if (e < n && sub == 0) sh.few_w[e] = w;
    if (threadIdx.x == 0) {
      sh.bin = min(k, n);  // tokens kept
      sh.bin_n = 0;
    }
    __syncthreads();
    uint32_t rank_e = 0;
    u64 upto = 0;
    if (e < n)
      for (int f = sub; f < n; f += q) {
        const bool in = sh.items[f] <= item;
        rank_e += in;
        if (weighed) upto += in ? sh.few_w[f] : 0;
      }
    for (int o = q >> 1; o > 0; o >>= 1) {
      rank_e += __shfl_xor_sync(kFull, rank_e, o);
      upto += __shfl_xor_sync(kFull, upto, o);
    }
    --rank_e;  // it counted itself
    const bool mine = e < n && sub == 0;
    const uint32_t kept_k = min(k, n);
    if (mine) {
      if (rank_e == kept_k - 1) sh.base_m = upto;
      if (z >= floor_z) atomicMax(&sh.bin_n, rank_e + 1);
    }
    __syncthreads();
    if (by_p && mine) {
      const u64 target = share(tp, sh.base_m);
      if (upto >= target && upto - w < target) atomicMin(&sh.bin, rank_e + 1);
    }
    __syncthreads();
    const uint32_t kept = min(sh.bin, sh.bin_n);
    if (mine && rank_e == kept - 1) {
      set_cut(~static_cast<uint32_t>(item >> 32), static_cast<uint32_t>(item));
      sh.base_m = upto;
    }
    if (!p.tokens) return;
    if (mine && rank_e >= kept) sh.few_w[e] = 0;
    __syncthreads();
    // the draw: mass up to each kept token in vocabulary order
    const uint32_t idx = static_cast<uint32_t>(item);
    u64 before = 0;
    if (e < n && rank_e < kept)
      for (int f = sub; f < n; f += q)
        if (static_cast<uint32_t>(sh.items[f]) < idx) before += sh.few_w[f];
    for (int o = q >> 1; o > 0; o >>= 1) before += __shfl_xor_sync(kFull, before, o);
    const u64 target = drawn(u, sh.base_m);
    if (mine && rank_e < kept && before < target && before + w >= target) p.tokens[row] = static_cast<int>(idx);
  }

  // The first cumulative mass that reaches top_p of a total; the one that
  // passes u of it.
  __device__ static u64 share(float tp, u64 total) {
    const u64 aim = static_cast<u64>(ceil(static_cast<double>(tp) * static_cast<double>(total)));
    return min(max(aim, 1ull), total);
  }
  __device__ static u64 drawn(float u, u64 total) {
    return min(static_cast<u64>(static_cast<double>(u) * static_cast<double>(total)) + 1, total);
  }

  // CTA 0, with more items: sorted.
  __device__ void many(int n, int k, bool by_p, float tp, float floor_z, float u, int row) {
    sort_items(n);
    const int kept_k = min(k, n), j0 = 4 * threadIdx.x;
    const bool weighed = by_p || p.tokens != nullptr;
    if (threadIdx.x == 0) sh.bin = kept_k;  // tokens kept
    float z[4];
    u64 w[4], own = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool in = j0 + e < kept_k;
      z[e] = in ? key_value(~static_cast<uint32_t>(sh.items[j0 + e] >> 32)) : -INFINITY;
      w[e] = in && weighed ? weight_of(z[e]) : 0;
      own += w[e];
    }
    if (by_p) {
      uint32_t ci;
      u64 mi;
      const u64 total = scan(0, own, ci, mi), target = share(tp, total);
      u64 before = mi - own;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (before < target && before + w[e] >= target) sh.bin = j0 + e + 1;
        before += w[e];
      }
    }
    __syncthreads();
    const int kept_p = sh.bin;
    uint32_t count = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) count += j0 + e < kept_p && z[e] >= floor_z;
    const int kept = static_cast<int>(block_sum(count));
    if (threadIdx.x == 0) set_cut(~static_cast<uint32_t>(sh.items[kept - 1] >> 32), static_cast<uint32_t>(sh.items[kept - 1]));
    if (!p.tokens) return;
    // ---- the draw, in vocabulary order: first the block of indices that holds it
    int shift = 0;
    while ((p.V - 1) >> shift >= kFew) ++shift;
    sh.few_w[threadIdx.x] = 0;
    if (threadIdx.x == 0) sh.bin_n = 0;
    __syncthreads();
    uint32_t idx[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      idx[e] = static_cast<uint32_t>(sh.items[j0 + e]);
      if (j0 + e < kept) atomicAdd(&sh.few_w[idx[e] >> shift], w[e]);
    }
    __syncthreads();
    const u64 in_block = sh.few_w[threadIdx.x];
    uint32_t ci;
    u64 mi;
    const u64 target = drawn(u, scan(0, in_block, ci, mi));
    if (mi >= target && mi - in_block < target) {
      sh.bin = threadIdx.x;
      sh.base_m = mi - in_block;
    }
    __syncthreads();  // (the items have been read: their places take the block's members)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (j0 + e < kept && idx[e] >> shift == sh.bin)
        sh.items[atomicAdd(&sh.bin_n, 1u)] = static_cast<u64>(idx[e]) << kWeightBits | w[e];
    __syncthreads();
    const int members = sh.bin_n;
    for (int t = threadIdx.x; t < members; t += kThreads) {
      const u64 member = sh.items[t], weight = member & ((1ull << kWeightBits) - 1);
      u64 upto = sh.base_m;
      for (int f = 0; f < members; ++f) upto += sh.items[f] <= member ? sh.items[f] & ((1ull << kWeightBits) - 1) : 0;
      if (upto >= target && upto - weight < target) p.tokens[row] = static_cast<int>(member >> kWeightBits);
    }
  }

  // ---- counts and masses over the cluster

  // Count of bin threadIdx.x.
  __device__ uint32_t read_count() const {
    uint32_t c = 0;
    for (int r = 0; r < C; ++r) c += of(r)->cnt[threadIdx.x];
    return c;
  }

  // Counts tokens by bin.  With `mass` also each bin's mass, nearly (m0, in 4096ths
  // of the weight at its start).
  __device__ void count_bins(bool mass) {
    sh.cnt[threadIdx.x] = sh.m0[threadIdx.x] = 0;
    __syncthreads();
    uint32_t tail = 0;
    for (int v = threadIdx.x; v < nvec; v += kThreads) {
      float f[N];
      Elem<T>::unpack(data[v], f);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float x = __fsub_rn(sc.m, f[e]) * bin_scale;
        if (x < static_cast<float>(kBins - 1)) {
          const uint32_t b = static_cast<uint32_t>(x);
          atomicAdd(&sh.cnt[b], 1u);
          if (mass) atomicAdd(&sh.m0[b], __float2uint_rn(exp2_ftz(12.0f - (x - static_cast<float>(b)) * kBinWidth)));
        } else {
          ++tail;
        }
      }
    }
    tail = block_sum(tail);
    if (threadIdx.x == 0) sh.cnt[kBins - 1] = tail;
    cluster.sync();
  }

  // Mass of all tokens.
  __device__ u64 all_mass() {
    Sum all;
    for (int v = threadIdx.x; v < nvec; v += kThreads) {
      float f[N];
      Elem<T>::unpack(data[v], f);
      add_all(all, f);
    }
    const u64 mine = block_sum(all.get());
    if (static_cast<int>(threadIdx.x) < C) of(threadIdx.x)->mass_of[rank] = mine;
    cluster.sync();
    u64 total = 0;
    for (int r = 0; r < C; ++r) total += sh.mass_of[r];
    return total;
  }

  __device__ __forceinline__ void add_all(Sum& s, const float (&f)[N]) const {
#pragma unroll
    for (int e = 0; e < N; e += 2) s.add(sc, f[e], f[e + 1], true, true, sh.t1, sh.t2);
  }
  // The tokens of a vector in `mask`, two at a time.
  __device__ __forceinline__ void add_some(Sum& s, const T* vec, uint32_t mask) const {
    while (mask) {
      const int e = __ffs(mask) - 1;
      mask &= mask - 1;
      const int g = mask ? __ffs(mask) - 1 : e;
      s.add(sc, Elem<T>::value(vec[e]), Elem<T>::value(vec[g]), true, mask != 0, sh.t1, sh.t2);
      mask &= mask - 1;
    }
  }

  // Mass of the tokens for which kind(value, index) is 0, and of those for which
  // it is 1.  maybe(x) is false where no value up to x counts.
  template <typename G, typename F>
  __device__ void masses(G maybe, F kind, u64& m0, u64& m1) {
    Sum s0, s1;
    for (int v = threadIdx.x; v < nvec; v += kThreads) {
      const uint4 x = data[v];
      if (!maybe(Elem<T>::vmax(x))) continue;
      float f[N];
      Elem<T>::unpack(x, f);
      uint32_t is0 = 0, is1 = 0;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int k = kind(f[e], static_cast<uint32_t>(first + v * N + e));
        is0 |= (k == 0 ? 1u : 0u) << e;
        is1 |= (k == 1 ? 1u : 0u) << e;
      }
      add_some(s0, reinterpret_cast<const T*>(data + v), is0);
      add_some(s1, reinterpret_cast<const T*>(data + v), is1);
    }
    const u64 a = block_sum(s0.get()), b = block_sum(s1.get());
    if (static_cast<int>(threadIdx.x) < C) {
      of(threadIdx.x)->mass_of[rank] = a;
      of(threadIdx.x)->all_of[rank] = b;
    }
    cluster.sync();
    m0 = m1 = 0;
    for (int r = 0; r < C; ++r) {
      m0 += sh.mass_of[r];
      m1 += sh.all_of[r];
    }
    cluster.sync();  // the words are free again
  }

  // ---- bf16 rows: tokens of equal value are counted together

  // The cut of a top-k or top-p from counts of equal values.  Values are
  // ordered: positive ones from the largest, the tiny ones (one place), negative
  // ones from the smallest magnitude.  First those are counted that should do:
  // for a top-p weights above about 2^-14; for a top-k the tokens above the least
  // of the threads' maxima (tokens in falling order fall on the T threads at
  // random and have met all of them after T ln T or so, so a k of up to 3/4 of
  // that likely lies among them).  Where the crossing lies below, weights down to
  // 2^-24, then all.
  // False: it lies among the tiny values or beyond nine octaves.
  __device__ bool cut_by_value(int k, bool by_p, float tp, u64 total, int threads) {
    // nine octaves of magnitudes from the largest that matters down; zeros, of
    // either sign, are tiny
    const float far = fmaxf(fabsf(sc.m), fabsf(sc.m - fminf(static_cast<float>(kOneBits + 1) / sc.h, 3.0e38f)));
    code0 = max(1, (static_cast<int>(__float_as_uint(far) >> 23) - 8) * 128);
    for (int i = threadIdx.x; i < 2 * kCodes; i += kThreads) sh.code_n[i] = 0;
    __syncthreads();
    Sum tiny;
    uint32_t tiny_n = 0;
    float below = INFINITY;  // values below this are yet to be counted
#pragma unroll 1
    for (int step = k > 0.75f * threads * logf(static_cast<float>(threads)) ? 1 : 0; step < 3; ++step) {
      const float least = step == 2       ? -FLT_MAX
                          : step == 0 && k ? least_top
                                           : sc.m - fminf((step == 0 ? 14.0f : 24.0f) / sc.h, 3.0e38f);
      for (int v = threadIdx.x; v < nvec; v += kThreads) {
        const uint4 x = data[v];
        if (Elem<T>::vmax(x) < least) continue;
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        uint32_t small = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t bits = e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16;
          const float z = __uint_as_float(bits);
          const int d = static_cast<int>(bits >> 16 & 0x7FFFu) - code0;
          const bool in = z >= least && z < below;
          if (in && static_cast<uint32_t>(d) < kCodes) atomicAdd(&sh.code_n[d + (bits >> 31 ? kCodes : 0)], 1u);
          small |= (in && d < 0 ? 1u : 0u) << e;
        }
        for (; small; small &= small - 1, ++tiny_n)
          tiny.add(sc, Elem<T>::value(reinterpret_cast<const T*>(data + v)[__ffs(small) - 1]), -INFINITY, true, false,
                   sh.t1, sh.t2);
      }
      below = least;
      const int got = cut_from_counts(k, by_p, tp, total, tiny, tiny_n);
      if (got >= 0) return got > 0;
      cluster.sync();  // the counts have been read
    }
    return false;
  }

  // 1: the cut is in sh; 0: it lies among the tiny values; -1: below what has
  // been counted.
  __device__ int cut_from_counts(int k, bool by_p, float tp, u64 total, const Sum& tiny, uint32_t tiny_n) {
    if (threadIdx.x == 0) sh.bin = 0xFFFFFFFFu;
    u64 tiny_m = block_sum(tiny.get());
    tiny_n = block_sum(tiny_n);
    if (static_cast<int>(threadIdx.x) < C) {
      Shared* s = of(threadIdx.x);
      s->tiny_mass_of[rank] = tiny_m;
      s->tiny_of[rank] = tiny_n;
    }
    cluster.sync();
    tiny_m = 0;
    tiny_n = 0;
    for (int r = 0; r < C; ++r) {
      tiny_m += sh.tiny_mass_of[r];
      tiny_n += sh.tiny_of[r];
    }
    for (int at = threadIdx.x; at < 2 * kCodes; at += kThreads) {
      uint32_t sum = 0;
      for (int r = 0; r < C; ++r) sum += of(r)->code_n[at];
      sh.code_all[at] = sum;
    }
    __syncthreads();
    // this thread's places of the order: counts, weights of one
    uint32_t n[kPer], count = 0;
    u64 one[kPer], mass = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int o = threadIdx.x * kPer + e;
      n[e] = 0;
      one[e] = 0;
      if (o == kCodes) {
        n[e] = tiny_n;
        count += tiny_n;
        mass += tiny_m;
      } else if (o < 2 * kCodes + 1) {
        const int at = o < kCodes ? kCodes - 1 - o : o - 1;
        n[e] = sh.code_all[at];
        if (n[e]) one[e] = weight_of(key_value(place_key(o)));
        count += n[e];
        mass += n[e] * one[e];
      }
    }
    uint32_t ci;
    u64 mi;
    scan(count, mass, ci, mi);
    uint32_t kth_key = 0, kth_idx = 0;
    u64 total_k = total;
    if (k) {
      uint32_t before = ci - count;
      if (before < static_cast<uint32_t>(k) && ci >= static_cast<uint32_t>(k))
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          if (before < static_cast<uint32_t>(k) && before + n[e] >= static_cast<uint32_t>(k)) found(threadIdx.x * kPer + e, k - before);
          before += n[e];
        }
      __syncthreads();
      if (sh.bin == 0xFFFFFFFFu) return -1;
      if (sh.bin == kCodes) return 0;
      const uint32_t o = sh.bin, need = sh.bin_n;
      // mass up to the k-th: what lies before its place, and its ties up to it
      if (threadIdx.x == o / kPer) {
        u64 m = mi - mass;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          if (threadIdx.x * kPer + e < o) m += threadIdx.x * kPer + e == kCodes ? tiny_m : n[e] * one[e];
          if (threadIdx.x * kPer + e == o) m += need * one[e];
        }
        sh.base_m = m;
      }
      __syncthreads();
      total_k = sh.base_m;
      kth_key = place_key(o);
      kth_idx = need;
      __syncthreads();
    }
    uint32_t key = kth_key, need = kth_idx;
    if (by_p) {
      // the first token whose cumulative mass reaches top_p * total
      const u64 target = share(tp, total_k);
      if (threadIdx.x == 0) sh.bin = 0xFFFFFFFFu;
      __syncthreads();
      u64 before = mi - mass;
      if (before < target && mi >= target)
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          const u64 m = threadIdx.x * kPer + e == kCodes ? tiny_m : n[e] * one[e];
          if (before < target && before + m >= target)
            found(threadIdx.x * kPer + e, one[e] ? static_cast<uint32_t>((target - before + one[e] - 1) / one[e]) : 1);
          before += m;
        }
      __syncthreads();
      if (sh.bin == 0xFFFFFFFFu) return -1;
      if (sh.bin == kCodes) return 0;
      key = place_key(sh.bin);
      need = sh.bin_n;
    }
    resolve_ties(key, need);
    return 1;
  }
  // The crossing lies at place o, at its need-th token.
  __device__ __forceinline__ void found(uint32_t o, uint32_t need) {
    sh.bin = o;
    sh.bin_n = need;
  }
  __device__ __forceinline__ uint32_t place_key(uint32_t o) const {
    const uint32_t code = o < kCodes ? code0 + kCodes - 1 - o : 0x8000u | (code0 + o - 1 - kCodes);
    return order_key(__uint_as_float(code << 16));
  }

  // ---- the cut within a bin

  __device__ __forceinline__ void add_mass(uint32_t b, u64 w) {
    atomicAdd(&sh.m0[b], static_cast<uint32_t>(w) & kLimbMask);
    atomicAdd(&sh.m1[b], static_cast<uint32_t>(w >> kLimb) & kLimbMask);
    atomicAdd(&sh.m2[b], static_cast<uint32_t>(w >> (2 * kLimb)));
  }

  // With the bin of the crossing, its count and what lies before it in sh: the cut.
  __device__ void resolve(bool by_mass, u64 target) {
    const uint32_t b0 = sh.bin;
    uint32_t klo = 0, khi = 0xFFFFFFFFu;
    const auto member = [&](float z, uint32_t key) { return bin_of(z) == b0 && key >= klo && key <= khi; };
    while (sh.bin_n > kList) {
      // range of the members' values
      uint32_t lo = 0xFFFFFFFFu, hi = 0;
      each([&](float z, uint32_t) {
        const uint32_t key = order_key(z);
        if (member(z, key)) {
          lo = min(lo, key);
          hi = max(hi, key);
        }
      });
      lo = __reduce_min_sync(kFull, lo);
      hi = __reduce_max_sync(kFull, hi);
      __syncthreads();
      if (threadIdx.x == 0) {
        sh.lidx[0] = 0xFFFFFFFFu;
        sh.lidx[1] = 0;
      }
      __syncthreads();
      if ((threadIdx.x & 31) == 0) {
        atomicMin(&sh.lidx[0], lo);
        atomicMax(&sh.lidx[1], hi);
      }
      __syncthreads();
      if (static_cast<int>(threadIdx.x) < C) {
        of(threadIdx.x)->kmin_of[rank] = sh.lidx[0];
        of(threadIdx.x)->kmax_of[rank] = sh.lidx[1];
      }
      cluster.sync();
      klo = 0xFFFFFFFFu;
      khi = 0;
      for (int r = 0; r < C; ++r) {
        klo = min(klo, sh.kmin_of[r]);
        khi = max(khi, sh.kmax_of[r]);
      }
      if (klo == khi) {
        const u64 base = by_mass ? sh.base_m : sh.base_c, one = by_mass ? weight_of(key_value(klo)) : 1;
        resolve_ties(klo, one ? (target - base + one - 1) / one : 1);
        return;
      }
      int s = 0;
      while (((khi - klo) >> s) >= kBins) ++s;
      sh.cnt[threadIdx.x] = sh.m0[threadIdx.x] = sh.m1[threadIdx.x] = sh.m2[threadIdx.x] = 0;
      __syncthreads();
      each([&](float z, uint32_t) {
        const uint32_t key = order_key(z);
        if (member(z, key)) {
          const uint32_t b = (khi - key) >> s;
          atomicAdd(&sh.cnt[b], 1u);
          if (by_mass) add_mass(b, weight_of(z));
        }
      });
      cluster.sync();
      uint32_t c = 0, ci;
      u64 a = 0, b = 0, d = 0, mi;
      for (int r = 0; r < C; ++r) {
        const Shared* o = of(r);
        c += o->cnt[threadIdx.x];
        a += o->m0[threadIdx.x];
        b += o->m1[threadIdx.x];
        d += o->m2[threadIdx.x];
      }
      const u64 m = a + (b << kLimb) + (d << (2 * kLimb));
      scan(c, m, ci, mi);
      const uint32_t before_c = sh.base_c;
      const u64 before_m = sh.base_m;
      __syncthreads();
      const u64 incl = by_mass ? before_m + mi : before_c + ci, own = by_mass ? m : c;
      if (incl >= target && incl - own < target) {
        sh.bin = threadIdx.x;
        sh.bin_n = c;
        sh.base_c = before_c + ci - c;
        sh.base_m = before_m + mi - m;
      }
      __syncthreads();
      const uint32_t most = khi - (sh.bin << s);  // largest key of the bin
      klo = max(klo, most - ((1u << s) - 1));
      khi = most;
      cluster.sync();  // the bins are read by every CTA before they are cleared
    }
    // members into the list of CTA 0
    if (threadIdx.x == 0) sh.pushed = 0;
    cluster.sync();
    Shared* r0 = of(0);
    each([&](float z, uint32_t idx) {
      const uint32_t key = order_key(z);
      if (member(z, key)) {
        const uint32_t at = atomicAdd(&r0->pushed, 1u);
        if (at < kList) {
          r0->lkey[at] = key;
          r0->lidx[at] = idx;
          r0->lw[at] = by_mass ? weight_of(z) : 1;
        }
      }
    });
    cluster.sync();
    if (rank == 0) {
      const int n = min(sh.pushed, static_cast<uint32_t>(kList)), e = threadIdx.x;
      if (e < n) {
        const uint32_t key = sh.lkey[e], idx = sh.lidx[e];
        u64 upto = by_mass ? sh.base_m : sh.base_c;
        for (int f = 0; f < n; ++f)
          upto += sh.lkey[f] > key || (sh.lkey[f] == key && sh.lidx[f] <= idx) ? sh.lw[f] : 0;
        if (upto >= target && upto - sh.lw[e] < target) set_cut(key, idx);
      }
    }
    cluster.sync();
  }

  __device__ void set_cut(uint32_t key, uint32_t idx) {
    for (int r = 0; r < C; ++r) {
      of(r)->cut_key = key;
      of(r)->cut_idx = idx;
    }
  }

  // The cut is the need-th token, in vocabulary order, of the value `key`.
  __device__ void resolve_ties(uint32_t key, u64 need) {
    const float value = key_value(key);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (nvec + kWarps - 1) / kWarps, v0 = min(warp * per, nvec), v1 = min(v0 + per, nvec);
    const auto ties = [&](int v) {  // of a vector, as a mask
      float f[N];
      Elem<T>::unpack(data[v], f);
      uint32_t eq = 0;
#pragma unroll
      for (int e = 0; e < N; ++e) eq |= (f[e] == value ? 1u : 0u) << e;
      return eq;
    };
    uint32_t mine = 0;
    for (int v = v0 + lane; v < v1; v += 32) mine += __popc(ties(v));
    mine = __reduce_add_sync(kFull, mine);
    if (lane < C) of(lane)->ties_of[rank][warp] = mine;
    cluster.sync();
    uint32_t before = 0;
    for (int at = lane; at < rank * kWarps + warp; at += 32) before += (&sh.ties_of[0][0])[at];
    before = __reduce_add_sync(kFull, before);
    if (before < need && before + mine >= need) {  // this warp holds it
      uint32_t left = static_cast<uint32_t>(need) - before;
      for (int g = v0; g < v1; g += 32) {
        const uint32_t eq = g + lane < v1 ? ties(g + lane) : 0, c = __popc(eq);
        uint32_t ci = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t a = __shfl_up_sync(kFull, ci, o);
          if (lane >= o) ci += a;
        }
        if (ci >= left && ci - c < left) {
          uint32_t k = left - (ci - c);  // the k-th of this vector
          int e = 0;
          for (;; ++e)
            if ((eq >> e) & 1u)
              if (--k == 0) break;
          set_cut(key, static_cast<uint32_t>(first + (g + lane) * N + e));
        }
        const uint32_t all = __shfl_sync(kFull, ci, 31);
        if (all >= left) break;
        left -= all;
      }
    }
    cluster.sync();
  }

  // ---- any top-k and top-p: the cut into sh
  __device__ void cut_any(int k, bool by_p, float tp, u64 total) {
    count_bins(by_p);
    const uint32_t c = read_count();
    uint32_t ci, near = 0;
    u64 mi;
    for (int r = 0; r < C; ++r) near += of(r)->m0[threadIdx.x];
    const float start = exp2_ftz(static_cast<float>(kOneBits - 12) - static_cast<float>(threadIdx.x) * kBinWidth);
    scan(c, threadIdx.x < kBins - 1 ? static_cast<u64>(static_cast<float>(near) * start) : 0, ci, mi);
    cluster.sync();  // every CTA has read the counts
    if (k) {
      if (ci >= static_cast<uint32_t>(k) && ci - c < static_cast<uint32_t>(k)) {
        sh.bin = threadIdx.x;
        sh.bin_n = c;
        sh.base_c = ci - c;
      }
      __syncthreads();
      resolve(false, k);
      if (by_p) {
        const uint32_t key = sh.cut_key, idx = sh.cut_idx;
        u64 none;
        masses([&](float x) { return x >= key_value(key); },
               [&](float z, uint32_t i) {
                 const uint32_t q = order_key(z);
                 return q > key || (q == key && i <= idx) ? 0 : 2;
               },
               total, none);
      }
    }
    if (!by_p) return;
    // the first token whose cumulative mass reaches top_p * total
    const u64 target = share(tp, total);
    if (threadIdx.x == 0) sh.bin = kBins - 1;
    __syncthreads();
    if (threadIdx.x < kBins - 1 && mi >= target) atomicMin(&sh.bin, threadIdx.x);
    __syncthreads();
    uint32_t g = sh.bin;
    u64 above, within;
    for (;;) {
      masses([&](float x) { return bin_of(x) <= g; },
             [&](float z, uint32_t) {
               const uint32_t b = bin_of(z);
               return b < g ? 0 : b == g ? 1 : 2;
             },
             above, within);
      if (target <= above && g > 0) --g;
      else if (target > above + within && g < kBins - 1) ++g;
      else break;
    }
    __syncthreads();
    if (threadIdx.x == g) {
      sh.bin = g;
      sh.bin_n = c;
      sh.base_m = above;
      sh.base_c = 0;
    }
    __syncthreads();
    resolve(true, target);
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleParams p) {
  extern __shared__ __align__(16) unsigned char raw[];
  __shared__ Shared sh;
  constexpr int N = Elem<T>::N;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int row = static_cast<int>(blockIdx.x) / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (p.cu) {
    const int total = __ldg(p.cu + p.bs);
    if (row >= total || total > p.rows) {
      if (row == 0 && (total < 0 || total > p.rows) && rank == 0 && tid == 0) raise_error(p.err, SD_DEV_ERR_CU_SEQLENS);
      return;
    }
  }
  // ---- the slice into shared memory
  const T* src = static_cast<const T*>(p.logits) + static_cast<long long>(row) * p.V;
  const int first = min(rank * p.slice, p.V), count = min(p.slice, p.V - first);
  const int nvec = (count + N - 1) / N;
  T* mine = reinterpret_cast<T*>(raw);
  if (tid == 0) {
    sh.pushed = 0;
    mbar_init(&sh.bar, 1);
    fence_mbar_init();
  }
  if (tid < kExpTab) {
    sh.t1[tid] = p.t1[tid];
    sh.t2[tid] = p.t2[tid];
  }
  __syncthreads();
  cluster.barrier_arrive();  // (the wait is before the first word to another CTA)
  bool landed = true;
  if (p.bulk) {
    if (tid == 0 && count > 0 && !p.waits.stall) {
      const uint32_t bytes = static_cast<uint32_t>(count) * sizeof(T);
      mbar_arrive_expect_tx(&sh.bar, bytes);
      const uint64_t pol = policy_evict_first();
      constexpr uint32_t kPart = 16384;
      for (uint32_t at = 0; at < bytes; at += kPart)
        bulk_load(raw + at, reinterpret_cast<const unsigned char*>(src + first) + at,
                  min(kPart, bytes - at), &sh.bar, pol);
    }
  } else {
    for (int e = tid; e < nvec * N; e += kThreads)
      mine[e] = e < count ? src[first + e] : Elem<T>::kNegInf;
  }
  // ---- whose row it is, while it travels (uniform over the cluster)
  int i = row;
  bool mine_ok = true;
  if (p.cu) {
    int lo = 0, hi = p.bs;  // last i with cu[i] <= row
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.cu + mid) <= row) lo = mid;
      else hi = mid;
    }
    i = lo;
    const int a = __ldg(p.cu + i), b = __ldg(p.cu + i + 1);
    mine_ok = a >= 0 && a <= row && row < b;
  }
  // ---- parameters, while the row travels
  float tau = __ldg(p.temps + i);
  int k = p.top_k ? __ldg(p.top_k + i) : 0;
  float tp = p.top_p ? __ldg(p.top_p + i) : 1.0f, mp = p.min_p ? __ldg(p.min_p + i) : 0.0f;
  float u = p.uniforms ? __ldg(p.uniforms + row) : 0.0f;
  int err = 0;
  if (!(tau >= 0.0f && isfinite(tau))) {
    err |= SD_DEV_ERR_TEMP;
    tau = 0.0f;
  }
  if (!(tp >= 0.0f)) {
    err |= SD_DEV_ERR_TRUNC;
    tp = 1.0f;
  }
  if (!(mp >= 0.0f)) {
    err |= SD_DEV_ERR_TRUNC;
    mp = 0.0f;
  }
  if (!(u >= 0.0f && u < 1.0f)) {
    err |= SD_DEV_ERR_UNIFORM;
    u = 0.0f;
  }
  if (k <= 0 || k >= p.V) k = 0;
  if (p.bulk && count > 0) landed = wait_phase(&sh.bar, 0, p.waits.limit_us * 1000ull);
  if (!landed) wait_phase(&sh.bar, 0, kDrainNs);
  if (!mine_ok) {  // in every CTA of the cluster alike
    if (rank == 0 && tid == 0) raise_error(p.err, SD_DEV_ERR_CU_SEQLENS);
    cluster.barrier_wait();
    return;
  }
  if (!p.bulk) __syncthreads();

  const uint4* data = reinterpret_cast<const uint4*>(raw);
  // ---- maximum; NaN, +inf
  float top = -INFINITY;
  for (int v = tid; v < nvec; v += kThreads) top = max_nan(top, Elem<T>::vmax(data[v]));
  bool bad = __syncthreads_or(!landed || !(top < INFINITY));
  const float wm = warp_max(top), wl = -warp_max(tid < nvec ? -top : -INFINITY);
  if (lane == 0) sh.scan_w[warp] = static_cast<u64>(__float_as_uint(wl)) << 32 | __float_as_uint(wm);
  __syncthreads();
  cluster.barrier_wait();  // every CTA of the cluster runs
  if (tid < C) {
    float mx = -INFINITY, ml = INFINITY;
    for (int w = 0; w < kWarps; ++w) {
      mx = fmaxf(mx, __uint_as_float(static_cast<uint32_t>(sh.scan_w[w])));
      ml = fminf(ml, __uint_as_float(static_cast<uint32_t>(sh.scan_w[w] >> 32)));
    }
    Shared* s = cluster.map_shared_rank(&sh, tid);
    s->max_of[rank] = mx;
    s->least_of[rank] = ml;
    s->bad_of[rank] = bad;
  }
  cluster.sync();
  float m = -INFINITY, least_top = INFINITY;
  bad = false;
  for (int r = 0; r < C; ++r) {
    m = fmaxf(m, sh.max_of[r]);
    least_top = fminf(least_top, sh.least_of[r]);
    bad |= sh.bad_of[r] != 0;
  }
  if (m == -INFINITY) bad = true;
  if (rank == 0 && tid == 0) {
    if (bad) err |= SD_DEV_ERR_LOGITS;
    if (err) raise_error(p.err, err);
  }
  if (!landed && tid == 0) raise_error(p.err, SD_DEV_ERR_TIMEOUT);

  Row<T> R{p, sh, data, nvec, first, rank, C, top, least_top, cluster, {}, 0.0f, -1};
  // kept: z > cut_z, or z == cut_z and index <= cut_idx; and z >= floor_z (min-p)
  float cut_z = -INFINITY, floor_z = -INFINITY;
  uint32_t cut_idx = 0xFFFFFFFFu;
  const auto kept = [&](float z, uint32_t idx) {
    return (z > cut_z || (z == cut_z && idx <= cut_idx)) && z >= floor_z;
  };
  if (bad) {
    if (rank == 0 && tid == 0 && p.tokens) p.tokens[row] = 0;
  } else if (tau == 0.0f) {
    // ---- greedy: the lowest index of the maximum
    uint32_t at = 0xFFFFFFFFu;
    if (top == m)
      R.each([&](float z, uint32_t idx) {
        if (z == m) at = min(at, idx);
      });
    at = __reduce_min_sync(kFull, at);
    if (lane == 0) sh.scan_c[warp] = at;
    __syncthreads();
    if (tid < C) {
      for (int w = 0; w < kWarps; ++w) at = min(at, sh.scan_c[w]);
      cluster.map_shared_rank(&sh, tid)->first_of[rank] = at;
    }
    cluster.sync();
    at = 0xFFFFFFFFu;
    for (int r = 0; r < C; ++r) at = min(at, sh.first_of[r]);
    if (rank == 0 && tid == 0 && p.tokens) p.tokens[row] = static_cast<int>(at);
    cut_z = m;
    cut_idx = at;
  } else {
    R.sc.set(m, tau);
    R.bin_scale = fminf(R.sc.h / kBinWidth, 3.0e38f);
    // w >= min_p as z >= a float: m + tau * ln(min_p), rounded up
    if (mp > 0.0f)
      floor_z = mp >= 1.0f ? m : __double2float_ru(static_cast<double>(m) + static_cast<double>(tau) * log(static_cast<double>(mp)));
    const bool by_p = tp < 1.0f;
    u64 total = 0;  // what a top-p alone refers to
    if (by_p && !k) total = R.all_mass();
    const int threads_used = min(kThreads, p.slice / N) * C;
    const bool listed = k > 0 && k <= kSmallK && R.gather(k);
    if (listed) {
      if (rank == 0) {
        const int n = static_cast<int>(sh.pushed);
        if (n <= kFew) R.few(n, k, by_p, tp, floor_z, u, row);
        else R.many(n, k, by_p, tp, floor_z, u, row);
      }
      cluster.sync();
    }
    if (!listed && (k || by_p)) {
      cluster.sync();
      bool done = false;
      if constexpr (sizeof(T) == 2) {
        done = R.cut_by_value(k, by_p, tp, total, threads_used);
        if (!done) cluster.sync();
      }
      if (!done) R.cut_any(k, by_p, tp, total);
    }
    if (listed || k || by_p) {
      cut_z = key_value(sh.cut_key);
      cut_idx = sh.cut_idx;
    }
    if (p.tokens && !listed) {
      // ---- the draw: sums of kept weights per warp, in vocabulary order
      const int per = (nvec + kWarps - 1) / kWarps;
      const int v0 = min(warp * per, nvec), v1 = min(v0 + per, nvec);
      const float low = fmaxf(cut_z, floor_z);
      const bool all = low == -INFINITY;
      const auto vec_sum = [&](int v) -> u64 {
        const uint4 x = data[v];
        if (!all && Elem<T>::vmax(x) < low) return 0;
        Sum s;
        float f[N];
        Elem<T>::unpack(x, f);
        if (all) {
          R.add_all(s, f);
        } else {
          uint32_t mask = 0;
#pragma unroll
          for (int e = 0; e < N; ++e)
            mask |= (kept(f[e], static_cast<uint32_t>(first + v * N + e)) ? 1u : 0u) << e;
          R.add_some(s, reinterpret_cast<const T*>(data + v), mask);
        }
        return s.get();
      };
      u64 sum = 0;
      for (int v = v0 + lane; v < v1; v += 32) sum += vec_sum(v);
      sum = Row<T>::warp_sum(sum);
      if (lane < C) cluster.map_shared_rank(&sh, lane)->warp_sum[rank][warp] = sum;
      cluster.sync();
      u64 total = 0, before = 0;
      for (int at = lane; at < C * kWarps; at += 32) {
        const u64 s = (&sh.warp_sum[0][0])[at];
        if (at < rank * kWarps + warp) before += s;
        total += s;
      }
      total = Row<T>::warp_sum(total);
      before = Row<T>::warp_sum(before);
      const u64 target = Row<T>::drawn(u, total);
      if (before < target && before + sum >= target) {
        u64 left = target - before;
        for (int g = v0; g < v1; g += 32) {
          const int v = g + lane;
          const u64 s = v < v1 ? vec_sum(v) : 0;
          u64 si = s;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const u64 a = __shfl_up_sync(kFull, si, o);
            if (lane >= o) si += a;
          }
          if (si >= left && si - s < left) {
            u64 upto = si - s;
            const T* z = reinterpret_cast<const T*>(data + v);
            for (int e = 0; e < N; ++e) {
              const float f = Elem<T>::value(z[e]);
              const uint32_t idx = static_cast<uint32_t>(first + v * N + e);
              if (kept(f, idx)) upto += R.weight_of(f);
              if (upto >= left) {
                p.tokens[row] = static_cast<int>(idx);
                break;
              }
            }
          }
          const u64 all = __shfl_sync(kFull, si, 31);
          if (all >= left) break;
          left -= all;
        }
      }
    }
  }
  // ---- the truncated row
  if (p.kept && landed) {
    T* dst = static_cast<T*>(p.kept) + static_cast<long long>(row) * p.V + first;
    const float low = fmaxf(cut_z, floor_z);
    const bool none = !bad && top < low;  // of this thread's tokens
    for (int v = tid; v < nvec; v += kThreads) {
      uint4 x = make_uint4(Elem<T>::kNegInfWord, Elem<T>::kNegInfWord, Elem<T>::kNegInfWord, Elem<T>::kNegInfWord);
      if (!none) {
        const uint4 y = data[v];
        if (bad || low == -INFINITY) {
          x = y;
        } else if (Elem<T>::vmax(y) >= low) {
          float f[N];
          Elem<T>::unpack(y, f);
          uint32_t mask = 0;
#pragma unroll
          for (int e = 0; e < N; ++e) mask |= (kept(f[e], static_cast<uint32_t>(first + v * N + e)) ? 1u : 0u) << e;
          x = Elem<T>::keep(y, mask);
        }
      }
      if (p.bulk) {
        reinterpret_cast<uint4*>(dst)[v] = x;
      } else {
        const T* y = reinterpret_cast<const T*>(&x);
        for (int e = 0; e < N && v * N + e < count; ++e) dst[v * N + e] = y[e];
      }
    }
  }
  cluster.sync();  // no CTA leaves while another may still read its shared memory
}

// Raises the kernel's dynamic shared-memory limit to the device's, once per
// device: the limit belongs to the kernel, not to a launch, so a call that set
// its own size would refuse another thread's larger one.
template <typename T>
cudaError_t shared_limit(int* limit) {
  constexpr int kMaxDev = 64;
  static std::atomic<int> limit_of[kMaxDev];
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidValue;
  *limit = limit_of[dev].load(std::memory_order_acquire);
  if (*limit != 0) return cudaSuccess;
  std::lock_guard<std::mutex> lock(mu);
  int optin = 0;
  cudaFuncAttributes fa;
  e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, sample_kernel<T>);
  if (e != cudaSuccess) return e;
  const int most = optin - static_cast<int>(fa.sharedSizeBytes);
  e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e != cudaSuccess) return e;
  limit_of[dev].store(most, std::memory_order_release);
  *limit = most;
  return cudaSuccess;
}

constexpr int kFewCtas = 76;  // half the SMs: twice as many CTAs still run side by side

template <typename T>
cudaError_t launch(SampleParams& p, cudaStream_t s) {
  constexpr int N = Elem<T>::N;
  const int vecs = (p.V + N - 1) / N;
  // Slices of up to 66 KB, so that two CTAs share an SM: when a step's 1201
  // truncated rows of 129280 took 380 us, they took 383 with slices of 132 KB and
  // 664 with 34 KB; 256 mixed rows 127, 146 and 168.
  int C = 1;
  while (C < 8 && (vecs + C - 1) / C * 16 > 66 * 1024) C *= 2;
  // few rows: more CTAs a row, while a thread still has a vector (4 rows of 129280
  // with a top-p 52 us, else 66; plain 19, else 23)
  while (C < 8 && p.rows * C <= kFewCtas && vecs >= 2 * C * kThreads) C *= 2;
  const int slice_vecs = (vecs + C - 1) / C;
  p.slice = slice_vecs * N;
  const size_t smem = static_cast<size_t>(slice_vecs) * 16;
  int limit = 0;
  cudaError_t e = shared_limit<T>(&limit);
  if (e != cudaSuccess) return e;
  if (smem > static_cast<size_t>(limit)) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.rows) * C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, p);
}

}  // namespace

cudaError_t launch_sample(SampleParams& p, int elem, cudaStream_t s) {
  const auto pair = [](double x) {
    const float hi = static_cast<float>(x);
    return make_float2(hi, static_cast<float>(x - static_cast<double>(hi)));
  };
  for (int i = 0; i < kExpTab; ++i) {
    p.t1[i] = pair(std::exp2(-i / 64.0));
    p.t2[i] = pair(std::exp2(-i / 4096.0));
  }
  return elem == 2 ? launch<uint16_t>(p, s) : launch<uint32_t>(p, s);
}

}  // namespace sdk
