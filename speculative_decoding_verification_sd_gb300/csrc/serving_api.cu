// serving_api.cu -- host side of the operators around the verification step:
// argument checks, choice of kernel and launches.  No entry point allocates
// device memory or synchronises the stream.
#include <cmath>

#include "sd_internal.h"
#include "serving.h"

namespace {

using sdk::refuse;

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

sd_status launched(cudaError_t e) {
  return e == cudaSuccess ? SD_OK
                          : refuse(SD_ERR_CUDA, "%s: %s", cudaGetErrorName(e), cudaGetErrorString(e));
}

// The options of the calls that have some.
sd_status read_cfg(const sd_launch_cfg* cfg, sdk::Waits* w) {
  *w = sdk::Waits{sdk::kWaitUs, false};
  if (!cfg) return SD_OK;
  if (cfg->blocks != 0 || cfg->wait_limit_us < 0 || cfg->reserved != 0)
    return refuse(SD_ERR_INVALID_ARG, "sd_launch_cfg: blocks or reserved != 0, or a negative limit");
  if (cfg->flags & ~SD_TEST_STALL) return refuse(SD_ERR_INVALID_ARG, "sd_launch_cfg: unknown flag bits 0x%x", cfg->flags);
  w->stall = (cfg->flags & SD_TEST_STALL) != 0;
  if (cfg->wait_limit_us > 0) w->limit_us = static_cast<uint32_t>(cfg->wait_limit_us);
  return SD_OK;
}

// Checks of a cache and of the step's shape, common to append and attend.
sd_status cache_checks(const sd_kv_cache* c, const int* cu_seqlens, const int* kv_lens, int bs,
                       int k_max, const int* err_flag, sdk::CacheView* view) {
  if (bs < 1 || k_max < 0) return refuse(SD_ERR_INVALID_ARG, "bs=%d, k_max=%d: need bs >= 1, k_max >= 0", bs, k_max);
  if (k_max > SD_MAX_K || bs > SD_MAX_VERIFY_BS)
    return refuse(SD_ERR_UNSUPPORTED, "bs=%d, k_max=%d beyond SD_MAX_VERIFY_BS=%d / SD_MAX_K=%d", bs,
                  k_max, SD_MAX_VERIFY_BS, SD_MAX_K);
  if (!c || !cu_seqlens || !kv_lens || !err_flag)
    return refuse(SD_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!c->k || !c->v || !c->page_table) return refuse(SD_ERR_INVALID_ARG, "a cache pointer is NULL");
  if (c->dt != SD_BF16 && c->dt != SD_E4M3)
    return refuse(SD_ERR_INVALID_ARG, "cache type %d is neither SD_BF16 nor SD_E4M3", c->dt);
  if (c->dt == SD_BF16 && (c->k_scale || c->v_scale))
    return refuse(SD_ERR_INVALID_ARG, "scales are for an SD_E4M3 cache");
  if (c->num_pages < 1 || c->page_size < 1 || c->max_pages < 1 || c->heads < 1)
    return refuse(SD_ERR_INVALID_ARG, "cache sizes: pages %d of %d tokens, %d a request, %d heads",
                  c->num_pages, c->page_size, c->max_pages, c->heads);
  if (c->head_dim < 8 || c->head_dim % 8 != 0 || c->head_dim > SD_MAX_HEAD_DIM)
    return refuse(SD_ERR_UNSUPPORTED, "head_dim=%d: a multiple of 8 up to SD_MAX_HEAD_DIM=%d",
                  c->head_dim, SD_MAX_HEAD_DIM);
  if (c->page_stride < 0 || c->token_stride < 0 || c->head_stride < 0)
    return refuse(SD_ERR_INVALID_ARG, "a cache stride is negative");
  *view = sdk::CacheView{c->k, c->v, c->page_table, c->k_scale, c->v_scale, c->page_stride,
                         c->token_stride, c->head_stride, c->num_pages, c->page_size, c->max_pages,
                         c->heads, c->head_dim};
  return SD_OK;
}

}  // namespace

extern "C" {

sd_status sd_cache_append(const void* k_new, const void* v_new, long long row_stride,
                          const sd_kv_cache* cache, const int* cu_seqlens, const int* kv_lens,
                          int bs, int k_max, int* err_flag, void* stream) {
  sdk::clear_last_error();
  sdk::AppendParams p{};
  const sd_status st = cache_checks(cache, cu_seqlens, kv_lens, bs, k_max, err_flag, &p.c);
  if (st != SD_OK) return st;
  if (!k_new || !v_new) return refuse(SD_ERR_INVALID_ARG, "k_new or v_new is NULL");
  if (row_stride < static_cast<long long>(p.c.heads) * p.c.dim)
    return refuse(SD_ERR_SHAPE, "row_stride=%lld < heads * head_dim", row_stride);
  const bool e4m3 = cache->dt == SD_E4M3;
  const int out = e4m3 ? 8 : 16;  // bytes of eight stored elements
  const bool vec = aligned(k_new, 16) && aligned(v_new, 16) && row_stride % 8 == 0 &&
                   aligned(p.c.k, out) && aligned(p.c.v, out) && p.c.page_stride % 8 == 0 &&
                   p.c.token_stride % 8 == 0 && p.c.head_stride % 8 == 0;
  p.k_new = static_cast<const uint16_t*>(k_new);
  p.v_new = static_cast<const uint16_t*>(v_new);
  p.row_stride = row_stride;
  p.cu = cu_seqlens;
  p.lens = kv_lens;
  p.bs = bs;
  p.k_max = k_max;
  p.err = err_flag;
  return launched(sdk::launch_append(p, e4m3, vec, static_cast<cudaStream_t>(stream)));
}

size_t sd_attend_workspace_bytes(int bs, int k_max, int q_heads, int heads, int head_dim) {
  if (bs < 1 || k_max < 0 || heads < 1 || q_heads < heads || q_heads % heads != 0 || head_dim < 8)
    return 0;
  // an 8-bit cache pads a head dimension up to 64 to 128
  const int pad = sdk::attend_dim_pad(head_dim < 128 ? 128 : head_dim);
  return sdk::attend_ws_layout(sdk::attend_row_cap(k_max, q_heads / heads), pad).total;
}

sd_status sd_attend(const void* q, long long q_row_stride, int q_heads, const sd_kv_cache* cache,
                    const int* cu_seqlens, const int* kv_lens, int bs, int k_max, float scale,
                    void* out, float* lse_out, int* err_flag, void* workspace, size_t ws_bytes,
                    void* stream) {
  return sd_attend_ex(q, q_row_stride, q_heads, cache, cu_seqlens, kv_lens, bs, k_max, scale, out, lse_out, err_flag,
                      workspace, ws_bytes, nullptr, stream);
}

sd_status sd_attend_ex(const void* q, long long q_row_stride, int q_heads, const sd_kv_cache* cache,
                       const int* cu_seqlens, const int* kv_lens, int bs, int k_max, float scale,
                       void* out, float* lse_out, int* err_flag, void* workspace, size_t ws_bytes,
                       const sd_launch_cfg* cfg, void* stream) {
  sdk::clear_last_error();
  sdk::AttendParams p{};
  const sd_status st = cache_checks(cache, cu_seqlens, kv_lens, bs, k_max, err_flag, &p.c);
  if (st != SD_OK) return st;
  if (!q || !out) return refuse(SD_ERR_INVALID_ARG, "q or out is NULL");
  if (q_heads < 1 || q_heads % p.c.heads != 0)
    return refuse(SD_ERR_INVALID_ARG, "q_heads=%d is no multiple of the cache's %d heads", q_heads, p.c.heads);
  if (q_heads / p.c.heads > SD_MAX_HEAD_GROUP)
    return refuse(SD_ERR_UNSUPPORTED, "%d query heads a cache head > SD_MAX_HEAD_GROUP", q_heads / p.c.heads);
  if (!std::isfinite(scale)) return refuse(SD_ERR_INVALID_ARG, "scale is not finite");
  if (q_row_stride < static_cast<long long>(q_heads) * p.c.dim)
    return refuse(SD_ERR_SHAPE, "q_row_stride=%lld < q_heads * head_dim", q_row_stride);
  if (!workspace || !aligned(workspace, 256))
    return refuse(SD_ERR_INVALID_ARG, "workspace NULL or not 256-byte aligned");
  const size_t need = sd_attend_workspace_bytes(bs, k_max, q_heads, p.c.heads, p.c.dim);
  if (ws_bytes < need) return refuse(SD_ERR_SHAPE, "ws_bytes=%zu < %zu", ws_bytes, need);
  p.q = static_cast<const uint16_t*>(q);
  p.q_row_stride = q_row_stride;
  p.q_heads = q_heads;
  p.group = q_heads / p.c.heads;
  p.cu = cu_seqlens;
  p.lens = kv_lens;
  p.bs = bs;
  p.k_max = k_max;
  p.scale = scale;
  const sd_status with = read_cfg(cfg, &p.waits);
  if (with != SD_OK) return with;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse_out;
  p.err = err_flag;
  // The tensor-core kernel wants what TMA wants: bases and strides of whole 16
  // bytes and boxes of whole swizzle atoms (eight tokens of one page).  It is
  // the faster one everywhere (11 us for 35 at the smallest call, 106 for 1430).
  const bool e4m3 = cache->dt == SD_E4M3;
  const int per16 = e4m3 ? 16 : 8;
  const bool tiled = p.c.page_size % 8 == 0 && aligned(p.c.k, 16) && aligned(p.c.v, 16) &&
                     p.c.page_stride % per16 == 0 && p.c.token_stride % per16 == 0 &&
                     p.c.head_stride % per16 == 0 && aligned(q, 16) && q_row_stride % 8 == 0 && aligned(out, 16);
  const cudaStream_t st_cuda = static_cast<cudaStream_t>(stream);
  if (tiled) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return launched(e);
    bool taken = false;
    e = sdk::launch_attend_tc(p, e4m3, workspace, sms < sdk::kAttendCtas ? sms : sdk::kAttendCtas, st_cuda, &taken);
    if (taken || e != cudaSuccess) return launched(e);
  }
  return launched(sdk::launch_attend_rows(p, e4m3, st_cuda));
}

sd_status sd_sample(const void* logits, sd_dtype dt, int V, int rows, const int* cu_seqlens, int bs,
                    const float* temps, const int* top_k, const float* top_p, const float* min_p,
                    const float* uniforms, int* tokens, void* kept_out, int* err_flag,
                    void* stream) {
  return sd_sample_ex(logits, dt, V, rows, cu_seqlens, bs, temps, top_k, top_p, min_p, uniforms, tokens, kept_out,
                      err_flag, nullptr, stream);
}

sd_status sd_sample_ex(const void* logits, sd_dtype dt, int V, int rows, const int* cu_seqlens, int bs,
                       const float* temps, const int* top_k, const float* top_p, const float* min_p,
                       const float* uniforms, int* tokens, void* kept_out, int* err_flag,
                       const sd_launch_cfg* cfg, void* stream) {
  sdk::clear_last_error();
  if (dt != SD_F32 && dt != SD_BF16) return refuse(SD_ERR_INVALID_ARG, "unknown dtype %d", static_cast<int>(dt));
  if (V < 1 || rows < 1) return refuse(SD_ERR_INVALID_ARG, "V=%d, rows=%d: need at least 1", V, rows);
  const int elem = dt == SD_F32 ? 4 : 2;
  if (static_cast<size_t>(V) * elem > static_cast<size_t>(SD_MAX_SAMPLE_ROW_BYTES))
    return refuse(SD_ERR_UNSUPPORTED, "V=%d (%d-byte elements) beyond SD_MAX_SAMPLE_ROW_BYTES", V, elem);
  if (rows > SD_MAX_VERIFY_BS * (SD_MAX_K + 1))
    return refuse(SD_ERR_UNSUPPORTED, "rows=%d > SD_MAX_VERIFY_BS * (SD_MAX_K + 1)", rows);
  if (cu_seqlens && bs < 1) return refuse(SD_ERR_INVALID_ARG, "cu_seqlens with bs=%d", bs);
  if (!logits || !temps || !err_flag) return refuse(SD_ERR_INVALID_ARG, "a required pointer is NULL");
  if ((uniforms == nullptr) != (tokens == nullptr))
    return refuse(SD_ERR_INVALID_ARG, "uniforms and tokens: both or neither");
  if (!tokens && !kept_out) return refuse(SD_ERR_INVALID_ARG, "neither tokens nor kept_out is asked for");
  if (!aligned(logits, elem) || (kept_out && !aligned(kept_out, elem)))
    return refuse(SD_ERR_INVALID_ARG, "logits or kept_out not aligned to its elements");
  sdk::SampleParams p{};
  const sd_status with = read_cfg(cfg, &p.waits);
  if (with != SD_OK) return with;
  p.logits = logits;
  p.V = V;
  p.rows = rows;
  p.cu = cu_seqlens;
  p.bs = bs;
  p.temps = temps;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.uniforms = uniforms;
  p.tokens = tokens;
  p.kept = kept_out;
  p.err = err_flag;
  p.bulk = static_cast<size_t>(V) * elem % 16 == 0 && aligned(logits, 16) &&
           (!kept_out || aligned(kept_out, 16));
  return launched(sdk::launch_sample(p, elem, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
