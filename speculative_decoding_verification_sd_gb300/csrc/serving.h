// serving.h -- parameter blocks and launch helpers of the operators around
// the verification step (cache append, paged attention, truncated sampling),
// shared between the host API (serving_api.cu) and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "sd.h"

namespace sdk {

// The caller's cache as the kernels index it (strides in elements).
struct CacheView {
  void* k;
  void* v;
  const int* table;
  const float* ks;
  const float* vs;
  long long page_stride, token_stride, head_stride;
  int num_pages, page_size, max_pages, heads, dim;
};

// How long a wait on the device may last, and the test hook that makes it run out.
constexpr uint32_t kWaitUs = 1000000;  // unless the caller sets one
struct Waits {
  uint32_t limit_us;
  bool stall;
};

struct AppendParams {
  const uint16_t* k_new;
  const uint16_t* v_new;
  long long row_stride;
  CacheView c;
  const int* cu;
  const int* lens;
  int bs, k_max;
  int* err;
};
cudaError_t launch_append(const AppendParams& p, bool e4m3, bool vec, cudaStream_t s);

struct AttendParams {
  const uint16_t* q;
  long long q_row_stride;
  int q_heads, group;
  CacheView c;
  const int* cu;
  const int* lens;
  int bs, k_max;
  float scale;
  uint16_t* out;
  float* lse;
  int* err;
  Waits waits;
};
// The general kernel (any strides, page size and alignment), and the
// tensor-core kernel; *taken = false when the cache's layout has no tensor map.
cudaError_t launch_attend_rows(const AttendParams& p, bool e4m3, cudaStream_t s);
cudaError_t launch_attend_tc(const AttendParams& p, bool e4m3, void* workspace, int ctas, cudaStream_t s,
                             bool* taken);

// Workspace of the tensor-core kernel: arrival counters (zero between calls),
// then maximum and sum, then weighted values, of up to two parts per CTA.
constexpr int kAttendCtas = 160;  // CTAs at most
struct AttendWs {
  size_t ml, o, total;
};
inline int attend_row_cap(int k_max, int group) {
  const long long rows = static_cast<long long>(k_max + 1) * group;
  return rows < 128 ? static_cast<int>(rows) : 128;
}
// Head dimension as the kernel pads its parts.
inline int attend_dim_pad(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }
inline AttendWs attend_ws_layout(int row_cap, int dim_pad) {
  const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  AttendWs w;
  w.ml = up(kAttendCtas * sizeof(int));
  w.o = w.ml + up(2 * kAttendCtas * static_cast<size_t>(row_cap) * 2 * sizeof(float));
  w.total = w.o + 2 * kAttendCtas * static_cast<size_t>(row_cap) * dim_pad * sizeof(float);
  return w;
}

// sd_sample: one cluster of CTAs per row, the row in their shared memory.
constexpr int kExpTab = 64;  // entries of each table of 2^-x
struct SampleParams {
  const void* logits;
  int V, rows;
  const int* cu;  // NULL: parameters are per row
  int bs;
  const float* temps;
  const int* top_k;
  const float* top_p;
  const float* min_p;
  const float* uniforms;
  int* tokens;
  void* kept;
  int* err;
  Waits waits;
  int slice;  // elements of a row per CTA (whole 16-byte vectors)
  bool bulk;  // rows start on 16 bytes and are whole vectors
  float2 t1[kExpTab], t2[kExpTab];  // 2^(-i/64), 2^(-i/4096) as (high, low) pairs
};
cudaError_t launch_sample(SampleParams& p, int elem, cudaStream_t s);

}  // namespace sdk
