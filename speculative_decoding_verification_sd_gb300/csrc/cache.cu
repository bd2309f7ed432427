// cache.cu -- sd_cache_append: the step's keys and values into the paged cache.
//
// A copy with an address per row: token kv_lens[i] - n_i + j of request i,
// looked up in the page table.  A CTA takes one or more rows of the step; a
// thread moves eight elements of one head of the keys and of the values (16
// bytes in; 16 or 8 bytes out), so a row of a usual cache is a few whole warps of
// consecutive addresses on both sides.  What bounds a small call is the chain of
// loads before the first store (row range, page, slot), so the row itself is on
// its way before its page is known; a large one into an 8-bit cache fills the
// issue slots, hence packed quotients and no integer division.  4700 rows of 8
// heads of 128 into an 8-bit cache (28 MB in and out) take 9.6 us, 2.9 TB/s of
// the copy's 6.8; a launch with next to nothing to do 2.  Rows, bases or strides
// off 16 bytes go element by element: 2 us more for those rows into an 8-bit cache,
// twice the time into a bf16 one (32 us for 15, with what a launch costs).
#include "cache.cuh"
#include "f32x2.cuh"

namespace sdk {
namespace {

constexpr int kMaxThreads = 256;
constexpr int kVec = 8;  // elements a thread moves

template <bool VEC>
__device__ __forceinline__ uint4 load8(const uint16_t* from) {
  if (VEC) return __ldg(reinterpret_cast<const uint4*>(from));
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = __ldg(from + 2 * e) | static_cast<uint32_t>(__ldg(from + 2 * e + 1)) << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// x / s, eight times.  t = x (1/s), corrected once by its exact remainder, is the
// rounded quotient (Markstein's theorem) while x and s are far from the ends of
// the range; elsewhere the division itself.  For s > 0.
__device__ __forceinline__ void quotients(const uint32_t (&w)[4], float s, float (&q)[kVec]) {
  const float r = __frcp_rn(s);
  const F2 r2 = both(r), minus_s = both(-s);
  uint32_t most = 0;  // of the magnitudes, ordered as their bits
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const F2 x = pack(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u));
    const F2 t = mul2(x, r2);
    unpack(fma2(fma2(t, minus_s, x), r2, t), q[2 * e], q[2 * e + 1]);
    q[2 * e] = copysignf(q[2 * e], __uint_as_float(w[e] << 16));  // (-0 / s is lost in the correction)
    q[2 * e + 1] = copysignf(q[2 * e + 1], __uint_as_float(w[e]));
    most = __vmaxu2(most, w[e] & 0x7FFF7FFFu);
  }
  constexpr uint32_t kFar = 0x5D00;  // 2^59
  if (!(s > 1e-18f && s < 1e18f) || (most & 0xFFFFu) >= kFar || most >> 16 >= kFar)
    for (int e = 0; e < kVec; ++e)
      q[e] = __fdiv_rn(__uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16), s);
}

// n / d of a d whose inverse (inverse_of) came along: one product and a step.
__device__ __forceinline__ int divided(int n, int d, uint32_t inv) {
  const int q = static_cast<int>(__umulhi(static_cast<uint32_t>(n), inv));
  return n - q * d >= d ? q + 1 : q;
}
uint32_t inverse_of(int d) { return d == 1 ? 0xFFFFFFFFu : static_cast<uint32_t>((1ull << 32) / d); }

// Eight elements into the cache.  E4M3: x / scale, rounded twice (the fp32
// quotient, then to nearest even), saturating at +-448.
template <bool E4M3, bool VEC>
__device__ __forceinline__ void store8(void* base, long long at, const uint4& x, float scale) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  if (E4M3) {
    uint8_t* to = static_cast<uint8_t*>(base) + at;
    uint32_t y[4];
    float q[kVec];
    quotients(w, scale, q);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      y[e] = __nv_cvt_float2_to_fp8x2(make_float2(q[2 * e], q[2 * e + 1]), __NV_SATFINITE, __NV_E4M3);
    if (VEC) {
      *reinterpret_cast<uint2*>(to) = make_uint2(y[0] | y[1] << 16, y[2] | y[3] << 16);
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) to[e] = static_cast<uint8_t>(y[e >> 1] >> (8 * (e & 1)));
    }
  } else {
    uint16_t* to = static_cast<uint16_t*>(base) + at;
    if (VEC) {
      *reinterpret_cast<uint4*>(to) = x;
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) to[e] = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
    }
  }
}

template <bool E4M3, bool VEC>
__global__ void __launch_bounds__(kMaxThreads) append_kernel(const AppendParams p, const uint32_t row_inv,
                                                             const uint32_t head_inv, const uint32_t page_inv) {
  const int per_head = p.c.dim / kVec, units = p.c.heads * per_head;
  const int which = static_cast<int>(blockIdx.x * blockDim.y + threadIdx.y);
  const int R = p.k_max + 1, i = divided(which, R, row_inv), j = which - i * R;
  if (i >= p.bs) return;
  const int len = __ldg(p.lens + i);
  const RowRange r = row_range(p.cu, i, p.bs, p.k_max);
  if (j >= r.n) {
    if (r.n < 0 && j == 0 && threadIdx.x == 0) raise_error(p.err, SD_DEV_ERR_CU_SEQLENS);
    return;
  }
  const long long row = (r.first + j) * p.row_stride;
  int unit = threadIdx.x;
  uint4 k = make_uint4(0, 0, 0, 0), v = k;
  int head = 0;
  float ks = 1.0f, vs = 1.0f;
  const auto fetch = [&] {
    if (unit >= units) return;
    k = load8<VEC>(p.k_new + row + unit * kVec);
    v = load8<VEC>(p.v_new + row + unit * kVec);
    head = divided(unit, per_head, head_inv);
    if (E4M3 && p.c.ks) ks = __ldg(p.c.ks + head);
    if (E4M3 && p.c.vs) vs = __ldg(p.c.vs + head);
  };
  fetch();
  const int pos = len < r.n - j ? -1 : len - r.n + j;  // -1: before the first token
  int page = -1;
  const int nth = divided(max(pos, 0), p.c.page_size, page_inv);
  if (pos >= 0 && nth < p.c.max_pages) page = __ldg(p.c.table + static_cast<long long>(i) * p.c.max_pages + nth);
  if (page < 0 || page >= p.c.num_pages) {
    if (threadIdx.x == 0) raise_error(p.err, SD_DEV_ERR_CACHE);
    return;
  }
  const long long slot = slot_offset(p.c, page, pos - nth * p.c.page_size);
  while (unit < units) {
    const long long to = slot + head * p.c.head_stride + (unit - head * per_head) * kVec;
    store8<E4M3, VEC>(p.c.k, to, k, ks);
    store8<E4M3, VEC>(p.c.v, to, v, vs);
    unit += blockDim.x;
    fetch();
  }
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, bool e4m3, bool vec, cudaStream_t s) {
  const int units = p.c.heads * (p.c.dim / kVec);
  const unsigned x = units < kMaxThreads ? (units + 31) / 32 * 32 : kMaxThreads, rows = p.bs * (p.k_max + 1);
  const dim3 threads(x, kMaxThreads / x);  // rows side by side
  const unsigned blocks = (rows + threads.y - 1) / threads.y;
  const auto kernel = e4m3 ? (vec ? append_kernel<true, true> : append_kernel<true, false>)
                           : (vec ? append_kernel<false, true> : append_kernel<false, false>);
  kernel<<<blocks, threads, 0, s>>>(p, inverse_of(p.k_max + 1), inverse_of(p.c.dim / kVec), inverse_of(p.c.page_size));
  return cudaGetLastError();
}

}  // namespace sdk
