// attend_rows.cu -- sd_attend for any cache layout: one CTA per query row and
// query head, its warps taking the tokens in turn.
//
// Each warp keeps a running maximum m, sum l and weighted value sum (online
// softmax, fp32) over its tokens; the lanes split the head dimension, so
// every load is a run of consecutive elements and no alignment is asked for.
// The warps' results are joined at the end in shared memory, in warp order.
//
// It takes what the tensor-core kernel cannot: pages that are no multiple of
// eight tokens, and bases or strides off 16 bytes.  A token is read again by
// every row and head of the step, and what bounds it is the chain of a token's
// loads, product and exponential: one row a request over 64 ragged caches takes
// 1430 us (tensor cores: 106), four tiny ones 35 (11).
#include "cache.cuh"

namespace sdk {
namespace {

constexpr int kWarps = 8;
constexpr int kElems = SD_MAX_HEAD_DIM / 32;  // elements of a row a lane holds

template <bool E4M3>
__device__ __forceinline__ float cache_at(const void* base, long long at) {
  return E4M3 ? e4m3_to_float(__ldg(static_cast<const uint8_t*>(base) + at))
              : bf16_to_float(__ldg(static_cast<const uint16_t*>(base) + at));
}

template <bool E4M3>
__global__ void __launch_bounds__(32 * kWarps) attend_rows_kernel(const AttendParams p) {
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][SD_MAX_HEAD_DIM];
  const int R = p.k_max + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.x / R, j = blockIdx.x - i * R, h = blockIdx.y, kvh = h / p.group;
  const RowRange r = row_range(p.cu, i, p.bs, p.k_max);
  const int given = __ldg(p.lens + i), len = attended_len(p.c, given);
  if (threadIdx.x == 0 && j == 0 && h == 0) {
    if (r.n < 0) raise_error(p.err, SD_DEV_ERR_CU_SEQLENS);
    if (given != len) raise_error(p.err, SD_DEV_ERR_CACHE);
  }
  if (j >= r.n) return;
  const int seen = max(len - r.n + j + 1, 0), D = p.c.dim;
  const long long row = r.first + j;
  float q[kElems], o[kElems], m = -INFINITY, l = 0.0f;
  // logits in units of ln 2: s * log2(e) = q . k * (scale * k_scale * log2 e)
  const float sc = p.scale * (E4M3 && p.c.ks ? __ldg(p.c.ks + kvh) : 1.0f) * kLog2e;
#pragma unroll
  for (int e = 0; e < kElems; ++e) {
    const int d = lane + 32 * e;
    q[e] = d < D ? bf16_to_float(__ldg(p.q + row * p.q_row_stride + static_cast<long long>(h) * D + d)) : 0.0f;
    o[e] = 0.0f;
  }
  const int* pages = p.c.table + static_cast<long long>(i) * p.c.max_pages;
  for (int t = warp; t < seen; t += kWarps) {
    const int page = __ldg(pages + t / p.c.page_size);
    const bool bad = page < 0 || page >= p.c.num_pages;
    if (bad && lane == 0) raise_error(p.err, SD_DEV_ERR_CACHE);
    const long long at = bad ? 0 : slot_offset(p.c, page, t % p.c.page_size) + kvh * p.c.head_stride;
    float s = 0.0f, v[kElems];
#pragma unroll
    for (int e = 0; e < kElems; ++e) {
      const int d = lane + 32 * e;
      const bool in = d < D && !bad;
      s = fmaf(q[e], in ? cache_at<E4M3>(p.c.k, at + d) : 0.0f, s);
      v[e] = in ? cache_at<E4M3>(p.c.v, at + d) : 0.0f;
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(kFull, s, x);
    s *= sc;
    // fmaxf drops a NaN logit from the maximum; the NaN still reaches l and o
    const float m2 = fmaxf(m, s), keep = m2 == -INFINITY ? 1.0f : exp2f(m - m2);
    const float w = s == -INFINITY ? 0.0f : exp2f(s - m2);
    l = fmaf(l, keep, w);
#pragma unroll
    for (int e = 0; e < kElems; ++e) o[e] = fmaf(o[e], keep, w * v[e]);
    m = m2;
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < kElems; ++e) so[warp][lane + 32 * e] = o[e];
  __syncthreads();
  float M = -INFINITY, L = 0.0f;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
  float f[kWarps];
  for (int w = 0; w < kWarps; ++w) {
    f[w] = sm[w] == -INFINITY ? (sl[w] == sl[w] ? 0.0f : sl[w]) : exp2f(sm[w] - M);
    L = fmaf(sl[w], f[w], L);
  }
  const float vscale = E4M3 && p.c.vs ? __ldg(p.c.vs + kvh) : 1.0f;
  for (int d = threadIdx.x; d < D; d += 32 * kWarps) {
    float x = 0.0f;
    for (int w = 0; w < kWarps; ++w) x = fmaf(so[w][d], f[w], x);
    p.out[(row * p.q_heads + h) * D + d] = float_to_bf16(L == 0.0f ? 0.0f : x / L * vscale);
  }
  if (p.lse && threadIdx.x == 0)
    p.lse[row * p.q_heads + h] = L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

}  // namespace

cudaError_t launch_attend_rows(const AttendParams& p, bool e4m3, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.bs) * (p.k_max + 1), p.q_heads);
  if (e4m3) attend_rows_kernel<true><<<grid, 32 * kWarps, 0, s>>>(p);
  else attend_rows_kernel<false><<<grid, 32 * kWarps, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace sdk
