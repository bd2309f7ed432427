// attend_tc.cu -- sd_attend on the tensor cores: one persistent CTA per SM
// over an equal share of the batch's cache tiles.
//
// Work.  A unit is one tile of TN tokens for one (request, cache head, tile of
// up to 128 query rows); the rows of a step that share a cache head are
// stacked (row m = j * group + head), so a tile of keys and values is read
// once for all of them.  Units are numbered request by request, then head,
// row tile, cache tile, each row tile's run opened by LEAD units without a
// tile, which stand for what a run costs besides its tiles (rows in and out);
// CTA c takes [U c / G, U (c+1) / G).  Lengths stay on
// the device: every CTA sums the batch's units itself.  A run of units of one
// row tile is a segment; a segment cut by a share's border leaves its partial
// sums in the workspace, and the CTA that arrives last joins the parts, in
// order.
//
// A CTA.  Warp 14 brings key and value tiles through a ring of TMA loads, warp
// 12 issues S = Q K^T, warp 13 O += P V, warps 0-7 turn S into P (two per lane,
// each half of the lane's tokens), and warps 8-11 put the next segment's query
// rows into TMEM and take the last segment's O out of it.  Q, S, P and O are all
// in TMEM, so the only operands in shared memory are the tiles themselves
// (reading Q from there too held the 8-bit cache to 79 % of the copy rate); P
// overwrites S.  S is double buffered: the scores of a tile are computed while
// the previous tile's softmax runs.
//
// Rows.  The tensor core computes 128 rows whatever is asked.  Over an 8-bit
// cache, whose softmax costs most, 64 rows or fewer are laid out twice and each
// copy weighs its own half of the tile's tokens (zeros elsewhere): independent
// partial sums, joined at the segment's end, for which all softmax warps work.
// 256 requests of up to 64 rows take 169 us with two copies, 184 with one; 19 of
// 65536 tokens and 4 rows 495 and 547; but 64 ragged single rows 99 and 89.  Over a
// bf16 cache the bytes hide the softmax, and there is one copy.
//
// Softmax.  Running maximum and sum per lane, fp32.  O is rescaled only when
// the maximum has grown by more than 2^SLACK since O's reference; until
// then weights are simply above 1, which the join undoes exactly as it undoes
// the reference.  A weight over a bf16 cache is the sum of two bf16 terms, within
// 2^-16 of it: one term costs as much as the output's own rounding (error against
// 64 bits 0.0023 where two give the output's 0.0017) and saves tensor time that
// the cache's bytes hide (64 ragged single rows 105 us with one, 107 with two; a
// step 110 and 112; two requests of 100000 tokens and more 190 both).
//
// 8-bit caches feed the tensor core as they are.  A query (8 significant
// bits) is the sum of two e4m3 terms after scaling its row by a power of two,
// exact but for elements below 2^-13 of the row's largest (off by up to 2^-17 of
// it); P becomes a half, which is split into three e5m2 terms (e5m2 is the upper
// byte of a half), the last one to nearest: within 2^-9 of a weight at worst and
// 2^-11 at the root mean square, and their exponents reach 2^-27 of the largest
// weight, so a long tail of small weights is not lost.  The products
// of the terms accumulate in the same fp32 accumulators.
//
// What bounds it.  The cache's bytes over a bf16 cache: 19 requests of 65536
// tokens (5.1 GB) take 744 us with up to 64 rows and 761 with 128, 6.7 to 6.9 TB/s,
// the copy rate.  Over an 8-bit cache a tile's 20 tensor instructions take 1280
// cycles, its bytes 1400 at the copy rate, and the chain scores, softmax, weights, O
// shows between them: 5.3 TB/s with 4 rows, 5.1 with 64, 4.2 with 128.  Short segments cost more than
// their tiles: rows in, O out, parts joined, all by warps 8-11 while the next
// segment runs.  What those warps wait for is mostly instructions (the softmax
// warps' code passes through the same caches), so their loops are short, waits
// that do not end at once are out of line, and the softmax is unrolled no further
// than its registers ask for (that took a step over an 8-bit cache from 193 to 153 us).
//
// Every wait is bounded; one that gives up raises SD_DEV_ERR_TIMEOUT and lets the
// CTA run to its end without waiting.
#include <cuda.h>

#include "cache.cuh"
#include "tcgen05.cuh"

namespace sdk {
namespace {

constexpr int kRowWarp = 8, kScoreWarp = 12, kValueWarp = 13, kLoadWarp = 14;  // 0-7: softmax; 8-11: rows in and out
constexpr int kWarps = 15, kThreads = 32 * kWarps;
constexpr int kMaxSlots = 12;
constexpr float kLn2 = 0.693147180559945309f;

template <bool F8, int NBLK>
struct Cfg {
  static constexpr int E = F8 ? 1 : 2;                 // bytes of a cache element
  static constexpr int DP = NBLK * 128 / E;            // head dimension, padded
  static constexpr int TN = DP <= 128 ? 128 : 64;      // tokens of a tile
  static constexpr int SLOT = NBLK * TN * 128;         // bytes of a key or value tile
  static constexpr int QPARTS = F8 ? 2 : 1;            // e4m3 terms of a query
  static constexpr int PPARTS = F8 ? 3 : 2;            // e5m2 or bf16 terms of a weight
  // Words that O passes through on its way out: 128 lanes of 32 columns, each
  // shifted by 16 bytes in the banks; of all 128 columns where the small tiles of
  // an 8-bit cache leave room, so that O is free for the next segment at once
  // (169 us; through 32 columns at a time 173)
  static constexpr int STAGE_WORDS = 128 * (F8 && DP == 128 ? 132 : 36);
  static constexpr int STAGE = STAGE_WORDS * 4;
  static constexpr int QROW = DP * 2 + 16;             // bytes of a fetched query row, shifted in the banks
  static constexpr int QRAW = 128 * QROW;
  static constexpr int TAIL = 10240;                   // Shared, and the base's alignment
  // Tiles' time that a segment costs besides its tiles.  A step over an 8-bit
  // cache: 171 us with 2, 169 with 3, 175 with 4; a ragged one over a bf16 cache
  // 106 with 1, 112 with 2.
  static constexpr int LEAD = SLOT >= 32768 ? 1 : 3;
  static constexpr int FIT = (232448 - STAGE - QRAW - TAIL) / SLOT;
  static constexpr int NS = FIT < kMaxSlots ? FIT : kMaxSlots;
  static constexpr int SMEM = NS * SLOT + STAGE + QRAW + TAIL;
  static constexpr int S_COL = 0, O_COL = 2 * TN, Q_COL = O_COL + DP;  // TMEM columns
  static constexpr int QC = DP / 2;                    // of a query tile
  static constexpr int NQ = Q_COL + 2 * QC <= 512 ? 2 : 1;
  static constexpr float SLACK = F8 ? 4.0f : 8.0f;     // log2: how far the maximum may outgrow O's reference
  static constexpr float LIFT = F8 ? 11.0f : 0.0f;     // log2: weights are stored times 2^LIFT
  static_assert(Q_COL + NQ * QC <= 512 && NS >= 3);
};

struct Wait {
  int stop;  // a wait gave up
  uint32_t limit_us;
};
struct Shared {
  uint64_t kv_full[kMaxSlots], kv_empty[kMaxSlots];
  // per buffer of S: scores there, weights there, weights used (a waiter is
  // never two phases of a buffer ahead of the tensor core)
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t q_full[2], q_empty[2];      // per query buffer
  uint64_t sums_full[2], sums_empty[2];  // per buffer of the softmax's final maxima and sums
  uint64_t o_free, end, end2;
  uint32_t tmem;
  Wait wait;
  int start_i;                    // first request of this CTA's share ...
  long long start_off, u0, u1, total;  // ... and the unit within it; the share; all units
  int last;                       // this CTA joins a segment's parts
  // A byte per softmax warp: it took non-finite values out of the segment's tiles.
  // Four buffers: while segment k's rows go out, O of k + 2 has not been started, so
  // the weights are at most two tiles into it, in k + 3.
  uint64_t odd[4];
  float tile_m[2][2][128];        // maxima of the halves of a lane's tokens, by S's buffer
  float lane_m[2][128], lane_l[2][2][128];  // a segment's maxima and (half) sums, per lane
  float q_scale[2][128];          // 2^-x of a query row's scaling (8-bit caches), per lane
  float row_m[128], row_l[128];   // joined parts, per row
  float row_f[128];               // what a row's sums are multiplied by
  long long warp_units[kWarps];
};
static_assert(sizeof(Shared) + 1024 <= 10240);

struct Params {
  AttendParams a;
  uint32_t group_inv;  // ceil(2^32 / group): m / group for m < 2^16
  int map_head_first;  // order of the tensor maps' middle dimensions
  int box;             // tokens of a TMA box
  int row_cap;         // rows of a part in the workspace
  float* part_o;       // [2 G][row_cap][DP]
  float* part_ml;      // [2 G][row_cap][2]
  int* count;          // [G] arrivals at the segment that starts in a CTA
};

// One request's shape, and one segment of a share.
struct Seg {
  int i, first, n, len, kvh, mt, tiles, t0, t1, rows;
  long long at;  // units of the batch before it
};

// A CTA's share, segment by segment.
template <int TN, int LEAD>
struct Walk {
  const AttendParams& p;
  Seg s;  // the request at hand
  int mts, kvh, mt, v;  // v: next unit of the run, lead included
  long long left;       // units to come
  long long at;         // all units before this run

  // Units of request i (0: no rows, or an invalid range).
  __device__ static long long units(const AttendParams& p, int i, Seg& s, int& mts) {
    const RowRange r = row_range(p.cu, i, p.bs, p.k_max);
    s.i = i;
    s.first = r.first;
    s.n = r.n;
    s.len = attended_len(p.c, __ldg(p.lens + i));
    s.tiles = max(1, (s.len + TN - 1) / TN);
    mts = r.n > 0 ? (r.n * p.group + 127) / 128 : 0;
    return static_cast<long long>(p.c.heads) * mts * (s.tiles + LEAD);
  }
  // u0: all units before the share, `off` of them in request i.
  __device__ Walk(const AttendParams& p, int i, long long off, long long u0, long long count) : p(p), left(count) {
    mts = kvh = mt = v = 0;
    at = u0;
    if (count <= 0) return;
    units(p, i, s, mts);
    const long long run = s.tiles + LEAD, k = off / run;
    kvh = static_cast<int>(k / mts);
    mt = static_cast<int>(k - static_cast<long long>(kvh) * mts);
    v = static_cast<int>(off - k * run);
    at -= v;
  }
  // The next run with a tile in the share.
  __device__ bool next(Seg& out) {
    while (left > 0) {
      if (kvh == p.c.heads) {
        kvh = 0;
        while (units(p, s.i + 1, s, mts) == 0) {
        }
      }
      const int run = s.tiles + LEAD, n = static_cast<int>(min(static_cast<long long>(run - v), left));
      out = s;
      out.kvh = kvh;
      out.mt = mt;
      out.t0 = max(v - LEAD, 0);
      out.t1 = v + n - LEAD;
      out.rows = min(128, s.n * p.group - 128 * mt);
      out.at = at;
      left -= n;
      at += run;
      v = 0;
      if (++mt == mts) {
        mt = 0;
        ++kvh;
      }
      if (out.t1 > out.t0) return true;
    }
    return false;
  }
};

// A place in the ring of tiles (K0 V0 K1 V1 ...) and the parity of its turn.
template <int NS>
struct Ring {
  uint32_t slot = 0, turn = 0;
  __device__ void step() {
    if (++slot == NS) {
      slot = 0;
      turn ^= 1;
    }
  }
  __device__ void skip(uint32_t n) {
    slot += n;
    turn ^= (slot / NS) & 1;
    slot %= NS;
  }
};

__device__ __forceinline__ float4 operator+(const float4& x, const float4& y) {
  return make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
}

// Query row m = j * group + head of a request, split.
__device__ __forceinline__ int row_of(const Params& p, int m) {
  return static_cast<int>(p.a.group == 1 ? m : __umulhi(static_cast<uint32_t>(m), p.group_inv));
}

// Lanes that hold a row.
template <bool F8>
__device__ __forceinline__ int copies(int rows) { return F8 && rows <= 64 ? 2 : 1; }

// A wait that gives up when its time is over or another wait of the CTA gave
// up; after that no wait of the CTA waits.  Out of line: see what bounds the
// kernel.
__device__ __noinline__ void wait_long(uint64_t* bar, uint32_t parity, volatile Wait* wait, int* err) {
  const uint64_t end = clock_ns() + wait->limit_us * 1000ull;
  while (!phase_done(bar, parity)) {
    if (wait->stop) return;
    if (clock_ns() > end) {
      wait->stop = 1;
      raise_error(err, SD_DEV_ERR_TIMEOUT);
      return;
    }
  }
}
__device__ __forceinline__ void wait_or_stop(uint64_t* bar, uint32_t parity, Shared& sh, int* err) {
  if (!phase_done(bar, parity)) wait_long(bar, parity, &sh.wait, err);
}

__device__ __forceinline__ void rows_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// The two softmax warps of one quarter of the lanes.
__device__ __forceinline__ void pair_sync(int quarter) { asm volatile("bar.sync %0, 64;" ::"r"(2 + quarter) : "memory"); }

// ---------------------------------------------------------------------------
// 32 elements of a lane's query row, bf16 in w, into TMEM at `to` (part 0).

template <bool F8, int NBLK>
__device__ __forceinline__ void store_q(const uint32_t (&w)[16], float by, uint32_t to) {
  using C = Cfg<F8, NBLK>;
  if constexpr (!F8) {
    const uint32_t flip = by < 0.0f ? 0x80008000u : 0u;
    uint32_t x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = w[e] ^ flip;
    tmem_store(to, x);
  } else {
    uint32_t x[2][8];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float2 y = make_float2(__uint_as_float(w[e] << 16) * by, __uint_as_float(w[e] & 0xFFFF0000u) * by);
      const __nv_fp8x2_storage_t t = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
      const float2 near = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(t, __NV_E4M3)));
      const uint32_t hi = t, lo = __nv_cvt_float2_to_fp8x2(make_float2(y.x - near.x, y.y - near.y), __NV_SATFINITE, __NV_E4M3);
      if (e & 1) {
        x[0][e >> 1] |= hi << 16;
        x[1][e >> 1] |= lo << 16;
      } else {
        x[0][e >> 1] = hi;
        x[1][e >> 1] = lo;
      }
    }
    tmem_store(to, x[0]);
    tmem_store(to + C::DP / 4, x[1]);
  }
}

// ---------------------------------------------------------------------------
// Softmax of one tile (warps 0-7): NC columns of S from token `first` on, `vis`
// of which this lane's row sees.  The maximum is the pair of warps' common one;
// the sum is this warp's.

// Column of P, relative to S's buffer, of a token (a multiple of 8).  32 tokens
// of P lie within the 32 columns of S that held their scores, so a part of a
// tile can be turned into P while the rest still waits as scores.
template <bool F8>
__device__ __forceinline__ constexpr uint32_t p_column(uint32_t token, uint32_t part) {
  return (token & ~31u) + (F8 ? part * 8 + ((token & 31) >> 2) : part * 16 + ((token & 31) >> 1));
}

// Scores of N tokens.
template <int N>
__device__ __forceinline__ void load_scores(uint32_t (&raw)[N], uint32_t at, int vis) {
  tmem_load(raw, at);
  if (__any_sync(kFull, vis < N)) {
#pragma unroll
    for (int c = 0; c < N; ++c) raw[c] = c < vis ? raw[c] : 0xFF800000u;
  }
}

template <bool F8, int NBLK, int NC>
__device__ __forceinline__ void softmax_tile(uint32_t lane_base, uint32_t s_at, uint32_t first, uint32_t copy, int vis,
                                             float sc, bool fresh, float& ref, float& l, uint32_t buf,
                                             int half, uint64_t* pv_done, uint32_t pv_parity, Shared& sh, int* err) {
  using C = Cfg<F8, NBLK>;
  constexpr int H = NC < 32 ? NC : 32;  // tokens in registers at a time
  const uint32_t at = lane_base + s_at + first;
  const int L = threadIdx.x & 127;
  uint32_t raw[H];
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int h = NC / H - 1; h >= 0; --h) {  // the first ones stay in registers
    load_scores<H>(raw, at + h * H, vis - h * H);
#pragma unroll
    for (int c = 0; c < H; ++c) mx[c & 3] = fmaxf(mx[c & 3], __uint_as_float(raw[c]));
  }
  float m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
  sh.tile_m[buf][half][L] = m;
  pair_sync(L >> 5);
  m = fmaxf(m, sh.tile_m[buf][half ^ 1][L]);
  if (fresh || ref == -INFINITY) ref = m;  // O holds nothing of this lane yet, or zeros
  if (fresh) l = 0.0f;
  const bool grow = m > ref && (m - ref) * sc > C::SLACK;
  if (__any_sync(kFull, grow)) {
    const float to = grow ? m : ref;
    const float f = grow ? exp2_ftz((ref - to) * sc) : 1.0f;
    ref = to;
    l *= f;
    wait_or_stop(pv_done, pv_parity, sh, err);  // the previous tile's O += P V
    __syncwarp();
    tc_fence_after();
    const uint32_t o_at = lane_base + C::O_COL + half * (C::DP / 2);
#pragma unroll 1
    for (uint32_t c = 0; c < C::DP / 2; c += 16) {
      uint32_t o[16];
      tmem_load(o, o_at + c);
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
      tmem_store(o_at + c, o);
    }
  }
  const float shift = ref == -INFINITY ? 0.0f : C::LIFT - ref * sc;
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int W = H / (F8 ? 4 : 2);  // columns of P
  uint32_t w[C::PPARTS][W];
#pragma unroll
  for (int h = 0; h < NC / H; ++h) {
    if (h > 0) load_scores<H>(raw, at + h * H, vis - h * H);
    if constexpr (!F8) {
#pragma unroll
      for (int c = 0; c < W; ++c) {
        const float x = exp2_ftz(fmaf(__uint_as_float(raw[2 * c]), sc, shift));
        const float y = exp2_ftz(fmaf(__uint_as_float(raw[2 * c + 1]), sc, shift));
        sum[(2 * c) & 3] += x;
        sum[(2 * c + 1) & 3] += y;
        // upper half, and the rest; 2^-18 more, so that a weight's rest is positive
        // as the weight is (an infinite value would meet 0 in the second product)
        w[0][c] = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
        const float xr = fmaf(x, 1.0f + 0x1p-18f, -__uint_as_float(w[0][c] << 16));
        const float yr = fmaf(y, 1.0f + 0x1p-18f, -__uint_as_float(w[0][c] & 0xFFFF0000u));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[1][c]) : "f"(yr), "f"(xr));
      }
    } else {
#pragma unroll
      for (int c = 0; c < W; ++c) {
        uint32_t hf[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float x = exp2_ftz(fmaf(__uint_as_float(raw[4 * c + 2 * e]), sc, shift));
          const float y = exp2_ftz(fmaf(__uint_as_float(raw[4 * c + 2 * e + 1]), sc, shift));
          sum[2 * e] += x;
          sum[2 * e + 1] += y;
          asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(hf[e]) : "f"(y), "f"(x));
        }
#pragma unroll
        for (int t = 0; t < C::PPARTS; ++t) {
          // the upper bytes; the last ones to nearest (rounding before the split would
          // add half a step to every weight whose terms hold it in full)
          const uint32_t near = t == C::PPARTS - 1 ? 0x00800080u : 0u;
          w[t][c] = __byte_perm(hf[0] + near, hf[1] + near, 0x7531);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t top = hf[e] & 0xFF00FF00u;
            asm("sub.f16x2 %0, %1, %2;" : "=r"(hf[e]) : "r"(hf[e]), "r"(top));  // exact
          }
        }
      }
    }
#pragma unroll
    for (int t = 0; t < C::PPARTS; ++t)
      tmem_store(lane_base + s_at + p_column<F8>(first + h * H, t), w[t]);
  }
  if constexpr (4 * NC == C::TN) {  // two copies: the other one's tokens weigh nothing in this lane
#pragma unroll
    for (int c = 0; c < W; ++c) w[0][c] = 0;
    const uint32_t other = first + 2 * NC - copy * (4 * NC);
#pragma unroll
    for (int t = 0; t < C::PPARTS; ++t) tmem_store(lane_base + s_at + p_column<F8>(other, t), w[0]);
  }
  l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
  tmem_store_wait();
}

// Which elements of a word of values are not finite, as a mask.
template <bool F8>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  return F8 ? __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu) : __vcmpeq2(w & 0x7F807F80u, 0x7F807F80u);
}

// A tile of values behind its first `by_all` tokens, which every row of the step
// sees: the others meet weights of 0, and 0 * NaN is NaN.  Slots from `used` on
// (beyond the request's length) hold anything and are zeroed; of the step's own
// tokens, the values that are not finite (the rows that see them get them back on
// their way out).  True: there were some in this thread's places.
template <bool F8, int NBLK>
__device__ __noinline__ bool clean_values(unsigned char* v, int by_all, int used, int tid) {
  constexpr int TN = Cfg<F8, NBLK>::TN;
  bool odd = false;
#pragma unroll 1
  for (int c = by_all * 8 + tid; c < TN * 8; c += 256)
#pragma unroll
    for (int b = 0; b < NBLK; ++b) {
      uint4* to = reinterpret_cast<uint4*>(v + b * TN * 128 + c * 16);
      uint4 x = make_uint4(0, 0, 0, 0);
      if (c < used * 8) {
        x = *to;
        const uint4 out = make_uint4(not_finite<F8>(x.x), not_finite<F8>(x.y), not_finite<F8>(x.z), not_finite<F8>(x.w));
        if (!(out.x | out.y | out.z | out.w)) continue;
        odd = true;
        x = make_uint4(x.x & ~out.x, x.y & ~out.y, x.z & ~out.z, x.w & ~out.w);
      }
      *to = x;
    }
  fence_proxy_async();
  return odd;
}

// Adds to a segment's rows, in the output or in their part, the non-finite values of
// the step's own tokens that they see, which clean_values has taken out of the tiles
// (a positive weight times such a value is that value).  Out of line and after the
// rows are out: few calls have such values, and what stands within the rows' way
// out costs every call (a step over an 8-bit cache 164 us, with a call there 176).
template <bool F8, int NBLK>
__device__ __noinline__ void add_not_finite(const Params& p, const Seg s, bool whole, long long part_row, int tid) {
  using C = Cfg<F8, NBLK>;
  const CacheView& c = p.a.c;
  const int one_sees = s.len - s.n + 1, from = max(max(one_sees, 0), s.t0 * C::TN), to = min(s.len, s.t1 * C::TN);
  for (int at = tid; at < s.rows * c.dim; at += 128) {
    const int row = at / c.dim, d = at - row * c.dim, m = 128 * s.mt + row, j = row_of(p, m);
    float x = 0.0f;
    for (int t = from; t < min(to, one_sees + j); ++t) {
      const int nth = t / c.page_size, page = __ldg(c.table + static_cast<long long>(s.i) * c.max_pages + nth);
      if (page < 0 || page >= c.num_pages) continue;  // read as zeros
      const long long el = slot_offset(c, page, t - nth * c.page_size) + s.kvh * c.head_stride + d;
      const float v = F8 ? e4m3_to_float(__ldg(static_cast<const uint8_t*>(c.v) + el))
                         : bf16_to_float(__ldg(static_cast<const uint16_t*>(c.v) + el));
      if (!isfinite(v)) x += v;
    }
    if (isfinite(x)) continue;
    if (whole) {
      const int h = s.kvh * p.a.group + (m - j * p.a.group);
      uint16_t* to_out = p.a.out + ((s.first + j) * static_cast<long long>(p.a.q_heads) + h) * c.dim + d;
      *to_out = float_to_bf16(bf16_to_float(*to_out) + x);
    } else {
      p.part_o[(part_row + row) * C::DP + d] += x;
    }
  }
}

// Row of the workspace where part c of a segment that starts in CTA c0 begins.
__device__ __forceinline__ long long part_slot(int c, int c0, int row_cap) {
  return static_cast<long long>(2 * c + (c == c0 ? 1 : 0)) * row_cap;
}

// Joined rows, K places (four columns of a row) a thread at a time, U parts of each.
template <int DP, int K, int U>
__device__ __forceinline__ void join_places(const Params& p, const Seg& s, int c0, int c1, const Shared& sh, float v_scale,
                                            int tid) {
  const AttendParams& a = p.a;
  const int D = a.c.dim, q4 = D / 4, places = s.rows * q4;
#pragma unroll 1
  for (int at = tid; at < places; at += K * 128) {
    int r[K], d[K];
    float4 o[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int place = min(at + 128 * k, places - 1);
      r[k] = place / q4;
      d[k] = (place - r[k] * q4) * 4;
      o[k] = make_float4(0, 0, 0, 0);
    }
#pragma unroll U
    for (int c = c0; c <= c1; ++c) {
      const long long slot = part_slot(c, c0, p.row_cap);
      float m[K];
      float4 x[K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        m[k] = __ldcg(p.part_ml + (slot + r[k]) * 2);
        x[k] = __ldcg(reinterpret_cast<const float4*>(p.part_o + (slot + r[k]) * DP + d[k]));
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const float f = m[k] == -INFINITY ? 0.0f : exp2f(m[k] - sh.row_m[r[k]]);
        o[k].x = fmaf(x[k].x, f, o[k].x);
        o[k].y = fmaf(x[k].y, f, o[k].y);
        o[k].z = fmaf(x[k].z, f, o[k].z);
        o[k].w = fmaf(x[k].w, f, o[k].w);
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (at + 128 * k >= places) break;
      const float L = sh.row_l[r[k]];
      const int m = 128 * s.mt + r[k], j = row_of(p, m), h = s.kvh * a.group + (m - j * a.group);
      const long long row = (s.first + j) * static_cast<long long>(a.q_heads) + h;
      const float f = L == 0.0f ? 0.0f : v_scale / L;
      uint2 y;
      y.x = float_to_bf16(o[k].x * f) | static_cast<uint32_t>(float_to_bf16(o[k].y * f)) << 16;
      y.y = float_to_bf16(o[k].z * f) | static_cast<uint32_t>(float_to_bf16(o[k].w * f)) << 16;
      *reinterpret_cast<uint2*>(a.out + row * D + d[k]) = y;
      if (d[k] == 0 && a.lse) a.lse[row] = L == 0.0f ? -INFINITY : (sh.row_m[r[k]] + log2f(L)) * kLn2;
    }
  }
}

// Joins the parts of a segment, in order (warps 8-11).
template <int DP>
__device__ void join_parts(const Params& p, const Seg& s, int c0, int c1, Shared& sh, float v_scale, int tid) {
  const AttendParams& a = p.a;
  const int D = a.c.dim;
  const auto slot = [&](int c) { return part_slot(c, c0, p.row_cap); };
  rows_sync();
  if (tid < s.rows) {
    float M = -INFINITY, L = 0.0f;
    for (int c = c0; c <= c1; ++c) M = fmaxf(M, __ldcg(p.part_ml + (slot(c) + tid) * 2));
    for (int c = c0; c <= c1; ++c) {
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + slot(c) + tid);
      L += ml.y * (ml.x == -INFINITY ? 0.0f : exp2f(ml.x - M));
    }
    sh.row_m[tid] = M;
    sh.row_l[tid] = L;
  }
  rows_sync();
  // Loads in flight are what it takes: with many places a thread has four at a
  // time (one at a time, 64 rows of two parts took 13 us), with few it reads the
  // parts of one together.
  if (s.rows * (D / 4) > 128) join_places<DP, 4, 1>(p, s, c0, c1, sh, v_scale, tid);
  else join_places<DP, 1, 4>(p, s, c0, c1, sh, v_scale, tid);
}

// ---------------------------------------------------------------------------

template <bool F8, int NBLK>
__global__ void __launch_bounds__(kThreads, 1)
    attend_tc_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap) {
  using C = Cfg<F8, NBLK>;
  constexpr int TN = C::TN;
  extern __shared__ unsigned char raw_smem[];
  unsigned char* base = raw_smem + ((1024u - (smem_addr(raw_smem) & 1023u)) & 1023u);
  unsigned char* ring = base;
  float* stage = reinterpret_cast<float*>(ring + C::NS * C::SLOT);
  unsigned char* qraw = reinterpret_cast<unsigned char*>(stage) + C::STAGE;
  Shared& sh = *reinterpret_cast<Shared*>(qraw + C::QRAW);
  const AttendParams& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int k = 0; k < C::NS; ++k) {
      mbar_init(&sh.kv_full[k], 1);
      mbar_init(&sh.kv_empty[k], 1);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(&sh.s_full[k], 1);
      mbar_init(&sh.p_full[k], 8);
      mbar_init(&sh.pv_done[k], 1);
      mbar_init(&sh.q_full[k], 4);
      mbar_init(&sh.q_empty[k], F8 ? 9 : 1);  // the segment's last Q K^T; softmax warps that read q_scale
      mbar_init(&sh.sums_full[k], 8);
      mbar_init(&sh.sums_empty[k], 4);
    }
    mbar_init(&sh.o_free, 4);
    mbar_init(&sh.end, 1);
    mbar_init(&sh.end2, 1);
    sh.wait.stop = 0;
    sh.wait.limit_us = a.waits.limit_us;
    fence_mbar_init();
  }
  if (warp == kScoreWarp) tmem_alloc(&sh.tmem, 512);
  // ---- this CTA's share of the units
  {
    const int per = (a.bs + kThreads - 1) / kThreads, i0 = min(tid * per, a.bs), i1 = min(i0 + per, a.bs);
    long long mine = 0;
    Seg s;
    int mts;
    for (int i = i0; i < i1; ++i) {
      mine += Walk<TN, C::LEAD>::units(a, i, s, mts);
      if (blockIdx.x == 0) {
        if (s.n < 0) raise_error(a.err, SD_DEV_ERR_CU_SEQLENS);
        if (s.len != __ldg(a.lens + i)) raise_error(a.err, SD_DEV_ERR_CACHE);
      }
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) sh.warp_units[warp] = incl;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) incl += sh.warp_units[w];
      total += sh.warp_units[w];
    }
    const long long G = min(static_cast<long long>(gridDim.x), total);
    const long long u0 = static_cast<int>(blockIdx.x) < G ? total * blockIdx.x / G : 0;
    const long long u1 = static_cast<int>(blockIdx.x) < G ? total * (blockIdx.x + 1) / G : 0;
    if (tid == 0) {
      sh.u0 = u0;
      sh.u1 = u1;
      sh.total = total;
    }
    if (u1 > u0 && incl > u0 && incl - mine <= u0) {
      long long off = u0 - (incl - mine);
      int i = i0;
      for (long long u; off >= (u = Walk<TN, C::LEAD>::units(a, i, s, mts)); ++i) off -= u;
      sh.start_i = i;
      sh.start_off = off;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  const long long count = sh.u1 - sh.u0;
  const uint32_t tmem = sh.tmem;
  Walk<TN, C::LEAD> walk(a, count > 0 ? sh.start_i : 0, count > 0 ? sh.start_off : 0, sh.u0, count);
  if (warp == kLoadWarp) {
    // ---- key and value tiles
    const uint64_t pol = policy_evict_first();
    const int box = lane / NBLK, blk = lane - box * NBLK;  // this lane's TMA box of a tile
    const bool has = box < TN / p.box;
    Ring<C::NS> at;
    int issued = 0;  // up to NS
    bool turned = false;
    Seg s;
    const auto load = [&](const CUtensorMap* map, const int (&c)[4], bool in, int bytes) {
      if (turned) wait_or_stop(&sh.kv_empty[at.slot], at.turn ^ 1, sh, a.err);
      // (the whole warp or none of it: the lanes meet below)
      if (__any_sync(kFull, *static_cast<volatile int*>(&sh.wait.stop))) return;
      if (lane == 0) mbar_arrive_expect_tx(&sh.kv_full[at.slot], bytes);
      __syncwarp();
      if (in)
        tma_load_4d(ring + at.slot * C::SLOT + blk * (TN * 128) + box * p.box * 128, map, c[0], c[1], c[2], c[3],
                    &sh.kv_full[at.slot], pol);
      at.step();
      if (!turned && ++issued == C::NS) turned = true;
    };
    if (a.waits.stall) walk.left = 0;
    while (walk.next(s)) {
      for (int t = s.t0; t < s.t1; ++t) {
        const int tok = t * TN + box * p.box;
        const bool in = has && tok < s.len;
        int c[4] = {blk * (128 / C::E), 0, 0, 0};
        if (in) {
          const int k = tok / a.c.page_size;
          int page = __ldg(a.c.table + static_cast<long long>(s.i) * a.c.max_pages + k);
          if (page < 0 || page >= a.c.num_pages) {
            raise_error(a.err, SD_DEV_ERR_CACHE);
            page = a.c.num_pages;  // out of the map's range: zeros
          }
          c[p.map_head_first ? 1 : 2] = s.kvh;
          c[p.map_head_first ? 2 : 1] = tok - k * a.c.page_size;
          c[3] = page;
        }
        const int valid = min(max(s.len - t * TN, 0), TN);
        const int bytes = (valid + p.box - 1) / p.box * p.box * 128 * NBLK;
        load(&kmap, c, in, bytes);
        load(&vmap, c, in, bytes);
      }
    }
    // no copy is in flight when the CTA ends (only a stopped CTA waits here)
    for (int k = 0; k < (turned ? C::NS : issued); ++k) {
      const bool this_turn = static_cast<uint32_t>(k) < at.slot;
      wait_phase(&sh.kv_full[k], this_turn ? at.turn : at.turn ^ 1, kDrainNs);
    }
  } else if (warp == kScoreWarp) {
    // ---- S = Q K^T.  The whole warp runs the loop, so that addresses and
    // descriptors stay in uniform registers; one lane issues.  The two products
    // have a warp each: what a tile costs them is mostly waits and issue.
    constexpr uint32_t id = tc_idesc(128, TN, F8 ? kFmtE4M3 : kFmtBf16, F8 ? kFmtE4M3 : kFmtBf16, false);
    const uint32_t tm = __shfl_sync(kFull, tmem, 0);
    const uint64_t k_desc = tc_desc(smem_addr(ring), 16, 1024);
    constexpr int STEPS = NBLK * 4;  // instructions of 32 bytes of the head dimension, 8 columns of Q
    Ring<C::NS> at;
    uint32_t u = 0, segs = 0;
    Seg s;
    while (walk.next(s)) {
      const uint32_t qb = segs % C::NQ;
      wait_or_stop(&sh.q_full[qb], (segs / C::NQ) & 1, sh, a.err);
      for (int t = s.t0; t < s.t1; ++t, ++u) {
        // S's buffer held the weights of unit u - 2
        if (u >= 2) wait_or_stop(&sh.pv_done[u & 1], ((u - 2) >> 1) & 1u, sh, a.err);
        wait_or_stop(&sh.kv_full[at.slot], at.turn, sh, a.err);
        __syncwarp();
        tc_fence_after();
        if (elect_one()) {
          const uint32_t d = tm + C::S_COL + (u & 1u) * TN, q = tm + C::Q_COL + qb * C::QC;
          const uint64_t kt = k_desc + at.slot * (C::SLOT >> 4);
#pragma unroll
          for (int part = 0; part < C::QPARTS; ++part)
#pragma unroll
            for (int st = 0; st < STEPS; ++st)
              tc_mma_ta<F8>(d, q + part * (C::DP / 4) + st * 8, kt + (((st >> 2) * TN * 128 + (st & 3) * 32) >> 4), id,
                            part + st > 0);
          tc_commit(&sh.s_full[u & 1]);
          tc_commit(&sh.kv_empty[at.slot]);
          if (t == s.t1 - 1) tc_commit(&sh.q_empty[qb]);
        }
        __syncwarp();
        at.skip(2);
      }
      ++segs;
    }
    if (elect_one()) tc_commit(&sh.end);
    wait_phase(&sh.end, 0, kDrainNs);
    __syncwarp();
  } else if (warp == kValueWarp) {
    // ---- O += P V
    constexpr uint32_t id = tc_idesc(128, C::DP, F8 ? kFmtE5M2 : kFmtBf16, F8 ? kFmtE4M3 : kFmtBf16, true);
    constexpr int KT = F8 ? 32 : 16;  // tokens of an instruction
    const uint32_t tm = __shfl_sync(kFull, tmem, 0);
    const uint64_t v_desc = tc_desc(smem_addr(ring), TN * 128, 1024);
    Ring<C::NS> at;
    at.skip(1);
    uint32_t u = 0, segs = 0;
    Seg s;
    while (walk.next(s)) {
      for (int t = s.t0; t < s.t1; ++t, ++u) {
        const uint32_t buf = u & 1u;
        const bool first = t == s.t0;
        wait_or_stop(&sh.kv_full[at.slot], at.turn, sh, a.err);
        // a new segment's O starts once the last one's has been read
        if (first && segs > 0) wait_or_stop(&sh.o_free, (segs - 1) & 1, sh, a.err);
        wait_or_stop(&sh.p_full[buf], (u >> 1) & 1u, sh, a.err);
        __syncwarp();
        tc_fence_after();
        if (elect_one()) {
          const uint32_t pa = tm + C::S_COL + buf * TN;
          const uint64_t v = v_desc + at.slot * (C::SLOT >> 4);
#pragma unroll
          for (int part = 0; part < C::PPARTS; ++part)
#pragma unroll
            for (int st = 0; st < TN / KT; ++st)
              tc_mma_ta<F8>(tm + C::O_COL, pa + p_column<F8>(st * KT, part), v + ((st * KT * 128) >> 4), id,
                            !first || part > 0 || st > 0);
          tc_commit(&sh.pv_done[buf]);
          tc_commit(&sh.kv_empty[at.slot]);
        }
        __syncwarp();
        at.skip(2);
      }
      ++segs;
    }
    if (elect_one()) tc_commit(&sh.end2);
    wait_phase(&sh.end2, 0, kDrainNs);
    __syncwarp();
  } else if (warp >= kRowWarp) {
    // ---- query rows in, outputs out
    const int L = (warp & 3) * 32 + lane;  // TMEM lane
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp & 3) << 21);
    uint32_t q_segs = 0, segs = 0, u = 0;
    // A segment's query rows into shared memory (asynchronous) ...
    const auto rows_fetch = [&](const Seg& s) {
      constexpr int CH = C::DP / 8;  // 16-byte chunks of a row: a thread has one of every 128 / CH rows
      const int d = L % CH * 8;
      if (d >= a.c.dim) return;
      const uint16_t* from = a.q + s.first * a.q_row_stride + s.kvh * a.group * a.c.dim + d;
      const long long next_j = a.q_row_stride - a.group * a.c.dim;  // besides the dim that m moves on
#pragma unroll 4
      for (int row = L / CH; row < s.rows; row += 128 / CH) {
        const int m = 128 * s.mt + row;
        cp_async16(qraw + row * C::QROW + 2 * d, from + row_of(p, m) * next_j + m * a.c.dim);
      }
    };
    // ... and from there, each lane its row, into TMEM.
    const auto rows_in = [&](const Seg& s) {
      const int r = L % (128 / copies<F8>(s.rows));
      const auto chunk = [&](int d) {
        return r < s.rows && d < a.c.dim ? *reinterpret_cast<const uint4*>(qraw + r * C::QROW + 2 * d)
                                         : make_uint4(0, 0, 0, 0);
      };
      cp_async_wait_all();
      rows_sync();
      // the softmax multiplies by |scale|
      float by = a.scale < 0.0f ? -1.0f : 1.0f, down = 1.0f;
      if constexpr (F8) {
        // a row's largest value scaled into [128, 256); a row with a non-finite
        // value becomes NaN
        uint32_t most[4] = {0, 0, 0, 0};  // magnitudes are ordered as their bits
#pragma unroll 4
        for (int d = 0; d < C::DP; d += 8) {
          const uint4 y = chunk(d);
          most[0] = __vmaxu2(most[0], y.x & 0x7FFF7FFFu);
          most[1] = __vmaxu2(most[1], y.y & 0x7FFF7FFFu);
          most[2] = __vmaxu2(most[2], y.z & 0x7FFF7FFFu);
          most[3] = __vmaxu2(most[3], y.w & 0x7FFF7FFFu);
        }
        const uint32_t both = __vmaxu2(__vmaxu2(most[0], most[1]), __vmaxu2(most[2], most[3]));
        const uint32_t top = max(both << 16, both & 0xFFFF0000u);
        const uint32_t E = max(top >> 23, 8u);
        const float up = top == 0 ? 1.0f : __uint_as_float((261u - min(E, 254u)) << 23);
        by = E == 255 ? __uint_as_float(0x7FC00000u) : by * up;
        down = 1.0f / up;
      }
      const uint32_t qb = q_segs % C::NQ, turn = q_segs / C::NQ;
      if (turn > 0) wait_or_stop(&sh.q_empty[qb], (turn - 1) & 1, sh, a.err);
      __syncwarp();
      tc_fence_after();
      const uint32_t to = lane_base + C::Q_COL + qb * C::QC;
#pragma unroll 1
      for (int d = 0; d < C::DP; d += 32) {
        uint32_t w[16];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 y = chunk(d + 8 * k);
          w[4 * k] = y.x;
          w[4 * k + 1] = y.y;
          w[4 * k + 2] = y.z;
          w[4 * k + 3] = y.w;
        }
        store_q<F8, NBLK>(w, by, to + d / (F8 ? 4 : 2));
      }
      if (F8) sh.q_scale[qb][L] = down;
      tmem_store_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full[qb]);
      ++q_segs;
      rows_sync();  // the rows have been read
    };
    // Two segments ahead: the rows of the next are laid out, those of the one
    // after it on their way.
    Seg s, s1, s2;
    bool more = false, more1 = walk.next(s1);
    if (more1) rows_fetch(s1);
    for (; more || more1; s = s1, s1 = s2, more = more1, more1 = s2.tiles > 0) {
      s2.tiles = 0;
      if (more1) {
        rows_in(s1);
        if (walk.next(s2)) rows_fetch(s2);
        else s2.tiles = 0;
      }
      if (!more) continue;
      u += s.t1 - s.t0;
      const int rep = copies<F8>(s.rows), R = 128 / rep, r = L % R;
      const float v_scale = F8 && a.c.vs ? __ldg(a.c.vs + s.kvh) : 1.0f;
      const bool whole = s.t0 == 0 && s.t1 == s.tiles;
      // copies of a row: their common maximum, joined sum, and what this one's
      // part of O is multiplied by
      const uint32_t sb = segs & 1;
      wait_or_stop(&sh.sums_full[sb], (segs >> 1) & 1, sh, a.err);
      float M = -INFINITY, sum = 0.0f, ms[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        ms[k] = k < rep ? sh.lane_m[sb][k * R + r] : -INFINITY;
        M = fmaxf(M, ms[k]);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (k < rep)
          sum += (sh.lane_l[sb][0][k * R + r] + sh.lane_l[sb][1][k * R + r]) *
                 (ms[k] == -INFINITY ? 0.0f : exp2_ftz(ms[k] - M));
      const float mine = sh.lane_m[sb][L], f = mine == -INFINITY ? 0.0f : exp2_ftz(mine - M);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.sums_empty[sb]);
      const long long part_row = (2ll * blockIdx.x + (s.t0 == 0 ? 1 : 0)) * p.row_cap;
      const long long out_base = s.first * static_cast<long long>(a.q_heads) + s.kvh * a.group;
      const auto out_row = [&](int row) {  // of the batch's [rows, q_heads]
        const int m = 128 * s.mt + row;
        return out_base + (m + row_of(p, m) * (a.q_heads - a.group));
      };
      if (L < s.rows) {  // the first copies
        if (whole) {
          sh.row_f[L] = sum == 0.0f ? 0.0f : v_scale / sum;
          if (a.lse) a.lse[out_row(L)] = sum == 0.0f ? -INFINITY : (M + log2f(sum)) * kLn2;
        } else {
          *reinterpret_cast<float2*>(p.part_ml + (part_row + L) * 2) = make_float2(M, sum);
        }
      }
      // O through the stage, W columns of every copy of every row at a time
      const int lanes = rep * s.rows;
      const int W = min(C::DP, lanes * 132 <= C::STAGE_WORDS ? 128 : lanes * 68 <= C::STAGE_WORDS ? 64 : 32);
      const int quads = W / 4, shift = W == 128 ? 5 : W == 64 ? 4 : 3;
      const bool mine_valid = r < s.rows;
      float* const my_stage = stage + ((L / R) * s.rows + r) * (W + 4);
      wait_or_stop(&sh.pv_done[(u - 1) & 1], ((u - 1) >> 1) & 1u, sh, a.err);
      __syncwarp();
      tc_fence_after();
      int base = 0;  // first staged column
#pragma unroll 1
      for (int c0 = 0; c0 < C::DP; c0 += 32) {
        uint32_t raw[32];
        tmem_load(raw, lane_base + C::O_COL + c0);
        if (c0 + 32 == C::DP) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.o_free);
        }
        if (mine_valid) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(my_stage + c0 - base + e) =
                make_float4(__uint_as_float(raw[e]) * f, __uint_as_float(raw[e + 1]) * f,
                            __uint_as_float(raw[e + 2]) * f, __uint_as_float(raw[e + 3]) * f);
        }
        if (c0 + 32 - base < W) continue;
        rows_sync();
        // A thread has four columns of every 128 / quads-th row.  Four rows are
        // read before the first is written: a store that might be to shared
        // memory keeps later loads from moving above it, and one at a time they
        // cost as much as the segment's products.
        const int col = (L & (quads - 1)) * 4, d = base + col, step = 128 >> shift;
        const float* from = stage + col;
        const int copy_at = s.rows * (W + 4);
        if (d < a.c.dim) {
#pragma unroll 1
          for (int row0 = L >> shift; row0 < s.rows; row0 += 4 * step) {
            float4 x[4];
            float g[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int row = min(row0 + k * step, s.rows - 1);
              const float* y = from + row * (W + 4);
              x[k] = *reinterpret_cast<const float4*>(y);
              if (rep > 1) x[k] = x[k] + *reinterpret_cast<const float4*>(y + copy_at);
              g[k] = sh.row_f[row];
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int row = row0 + k * step;
              if (row >= s.rows) break;
              if (whole) {
                uint2 o;
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o.x) : "f"(x[k].y * g[k]), "f"(x[k].x * g[k]));
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o.y) : "f"(x[k].w * g[k]), "f"(x[k].z * g[k]));
                *reinterpret_cast<uint2*>(a.out + out_row(row) * a.c.dim + d) = o;
              } else {
                *reinterpret_cast<float4*>(p.part_o + (part_row + row) * C::DP + d) = x[k];
              }
            }
          }
        }
        rows_sync();
        base += W;
      }
      if (sh.odd[segs & 3]) add_not_finite<F8, NBLK>(p, s, whole, part_row, L);
      if (!whole) {
        const long long G = min(static_cast<long long>(gridDim.x), sh.total);
        const auto cta_of = [&](long long x) { return static_cast<int>(((x + 1) * G - 1) / sh.total); };
        const int c0 = cta_of(s.at + C::LEAD), c1 = cta_of(s.at + C::LEAD + s.tiles - 1);
        rows_sync();  // the warps' parts are written: the fence covers all that is before it
        if (L == 0) {
          __threadfence();
          const int n = c1 - c0 + 1, before = atomicAdd(p.count + c0, 1);
          sh.last = before == n - 1;
          if (sh.last) p.count[c0] = 0;
          __threadfence();
        }
        rows_sync();
        if (sh.last) join_parts<C::DP>(p, s, c0, c1, sh, v_scale, L);
        rows_sync();
      }
      ++segs;
    }
  } else {
    // ---- softmax
    const int L = tid & 127, half = warp >> 2;  // TMEM lane, half of its tokens
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp & 3) << 21);
    uint32_t u = 0, segs = 0;
    Ring<C::NS> at;
    Seg s;
    float ref = -INFINITY, l = 0.0f;
    while (walk.next(s)) {
      const int rep = copies<F8>(s.rows), R = 128 / rep, r = L % R, copy = L / R;
      const int m = 128 * s.mt + min(r, s.rows - 1), j = row_of(p, m);
      const int seen = s.len - s.n + j + 1;
      const bool busy = (L & 96) % R < s.rows;  // this warp holds rows
      float sc = fabsf(a.scale) * kLog2e;
      if (F8) {
        const uint32_t qb = segs % C::NQ;
        wait_or_stop(&sh.q_full[qb], (segs / C::NQ) & 1, sh, a.err);
        sc *= sh.q_scale[qb][L];
        if (a.c.ks) sc *= __ldg(a.c.ks + s.kvh);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.q_empty[qb]);
      }
      sc = sc < 1e-37f ? 1e-37f : sc;  // masked scores are -inf, and -inf * 0 is NaN
      bool odd = false;
      for (int t = s.t0; t < s.t1; ++t, ++u) {
        const uint32_t buf = u & 1u;
        const uint32_t s_at = C::S_COL + buf * TN;
        wait_or_stop(&sh.s_full[buf], (u >> 1) & 1u, sh, a.err);
        __syncwarp();
        tc_fence_after();
        uint64_t* pv_done = &sh.pv_done[(u - 1) & 1];  // the previous unit's
        const uint32_t pv_parity = ((u - 1) >> 1) & 1u;
        const bool fresh = t == s.t0;
        if (busy) {
          const int first = copy * (TN / rep) + half * (TN / rep / 2), vis = seen - t * TN - first;
          if (F8 && rep == 2)
            softmax_tile<F8, NBLK, TN / 4>(lane_base, s_at, first, copy, vis, sc, fresh, ref, l, buf, half, pv_done,
                                           pv_parity, sh, a.err);
          else
            softmax_tile<F8, NBLK, TN / 2>(lane_base, s_at, first, copy, vis, sc, fresh, ref, l, buf, half, pv_done,
                                           pv_parity, sh, a.err);
        }
        const int by_all = s.len - s.n + 1 - t * TN;  // tokens of the tile that every row of the step sees
        if (by_all < TN) {
          Ring<C::NS> vt = at;
          vt.skip(2 * (t - s.t0) + 1);
          wait_or_stop(&sh.kv_full[vt.slot], vt.turn, sh, a.err);
          odd |= clean_values<F8, NBLK>(ring + vt.slot * C::SLOT, max(by_all, 0), s.len - t * TN, tid);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[buf]);
      }
      at.skip(2 * (s.t1 - s.t0));
      const uint32_t sb = segs & 1;
      if (segs >= 2) wait_or_stop(&sh.sums_empty[sb], ((segs >> 1) - 1) & 1, sh, a.err);
      if (half == 0) sh.lane_m[sb][L] = ref == -INFINITY ? -INFINITY : ref * sc - C::LIFT;
      sh.lane_l[sb][half][L] = l;
      odd = __any_sync(kFull, odd);
      if (lane == 0) reinterpret_cast<unsigned char*>(&sh.odd[segs & 3])[warp] = odd;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.sums_full[sb]);
      ++segs;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kScoreWarp) tmem_free(tmem, 512);
}

using Encode = decltype(&cuTensorMapEncodeTiled);

Encode encoder() {
  static const Encode fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult st = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &st) != cudaSuccess ||
        st != cudaDriverEntryPointSuccess)
      f = nullptr;
    cudaGetLastError();
    return reinterpret_cast<Encode>(f);
  }();
  return fn;
}

template <bool F8, int NBLK>
cudaError_t launch(Params& p, void* workspace, int ctas, cudaStream_t st, bool* taken) {
  using C = Cfg<F8, NBLK>;
  const CacheView& c = p.a.c;
  const Encode encode = encoder();
  if (!encode) return cudaSuccess;
  p.box = c.page_size & -c.page_size;  // largest power of two that divides the page
  if (p.box > C::TN) p.box = C::TN;
  // the smaller stride first
  p.map_head_first = c.head_stride <= c.token_stride;
  const cuuint64_t tok = c.token_stride * C::E, head = c.head_stride * C::E, page = c.page_stride * C::E;
  const cuuint64_t nt = c.page_size, nh = c.heads;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.dim), p.map_head_first ? nh : nt, p.map_head_first ? nt : nh,
                              static_cast<cuuint64_t>(c.num_pages)};
  const cuuint64_t strides[3] = {p.map_head_first ? head : tok, p.map_head_first ? tok : head, page};
  const cuuint32_t one = 1, rows = static_cast<cuuint32_t>(p.box);
  const cuuint32_t boxes[4] = {128 / C::E, p.map_head_first ? one : rows, p.map_head_first ? rows : one, 1};
  const cuuint32_t steps[4] = {1, 1, 1, 1};
  CUtensorMap maps[2];
  for (int k = 0; k < 2; ++k)
    if (encode(&maps[k], F8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, k ? c.v : c.k, dims,
               strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaSuccess;
  p.row_cap = attend_row_cap(p.a.k_max, p.a.group);
  const AttendWs w = attend_ws_layout(p.row_cap, C::DP);
  p.count = static_cast<int*>(workspace);
  p.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + w.ml);
  p.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + w.o);
  auto* kernel = attend_tc_kernel<F8, NBLK>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  kernel<<<ctas, kThreads, C::SMEM, st>>>(p, maps[0], maps[1]);
  *taken = true;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend_tc(const AttendParams& a, bool e4m3, void* workspace, int ctas, cudaStream_t s,
                             bool* taken) {
  Params p{};
  p.a = a;
  p.group_inv = static_cast<uint32_t>((0x100000000ull + a.group - 1) / a.group);
  *taken = false;
  if (e4m3)
    return a.c.dim <= 128 ? launch<true, 1>(p, workspace, ctas, s, taken)
                          : launch<true, 2>(p, workspace, ctas, s, taken);
  if (a.c.dim <= 64) return launch<false, 1>(p, workspace, ctas, s, taken);
  return a.c.dim <= 128 ? launch<false, 2>(p, workspace, ctas, s, taken)
                        : launch<false, 4>(p, workspace, ctas, s, taken);
}

}  // namespace sdk
