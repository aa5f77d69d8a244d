// Attention over context caches held in four bits, the write of such a cache
// and its read-back (kv4.cuh has the layout).
//
//   y_r = sum_i p_ri V_i,  p_ri = softmax over the visible rows i of scale q_r . K_i
//
// with visible: lo <= i < hi, i <= a + r when causal, i >= a + r + 1 - W with a
// window W (a: the cache row of the sequence's first query). The block pass adds
// the block's own rows, a tile of its own that every query sees.
//
// Two kernels: k_attn4 on the 5th-generation tensor cores, and k_attn4_few on
// mma.sync where the query rows are few. Both keep a running reference m, sum l and
// unnormalised output o per query over a share of the context.
#include <algorithm>
#include <climits>
#include <string>
#include <type_traits>

#include "common.cuh"
#include "dflash.h"
#include "kernels.h"
#include "kv4.cuh"
#include "tc.cuh"

namespace dfl {

// ---------------------------------------------------------------- element types
__device__ __forceinline__ void st_elem(void *p, int64_t i, int dtype, float v) {
  if (dtype == DFLASH_F32) ((float *)p)[i] = v;
  else if (dtype == DFLASH_F16) ((__half *)p)[i] = __float2half_rn(v);
  else ((__nv_bfloat16 *)p)[i] = __float2bfloat16_rn(v);
}

// ---------------------------------------------------------------- write and read
struct Kv4Seqs {
  uint8_t *k[MAX_BATCH], *v[MAX_BATCH];
  int64_t at[MAX_BATCH];
  int64_t head_bytes;  // from one KV head's tiles to the next's
};
struct Kv4Rows {
  const void *p[2];              // K and V rows
  int64_t seq_stride[2], row_stride[2];  // in elements; heads and values of a row are contiguous
  int vec[2];                    // every row on 16 bytes
};

// a / b of whole numbers >= 0; a 32-bit division where both fit (a 64-bit one is some
// hundred instructions).
__device__ __forceinline__ int64_t a4_div(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// Four words of four neighbouring lanes: lane m gets word m of each, in order.
__device__ __forceinline__ void kv4_transpose(uint32_t (&w)[4], int m) {
#pragma unroll
  for (int o = 1; o < 4; o <<= 1)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (!(r & o)) {
        const bool up = m & o;
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[r] : w[r + o], o);
        if (up) w[r] = got;
        else w[r + o] = got;
      }
}

// A thread takes 8 consecutive values of RW = 4 rows, so that its loads are in flight
// together and the codes leave in whole sectors: four neighbours hold the four words
// of a group for each of the 4 rows, turn them around among themselves and store the
// 16 bytes of one row each (64 bytes side by side). What has to move is the rows in and
// 9/16 of a byte a value out: 8 x 4,096 bf16 rows of 8 heads of 128 take 42 us for 172 MB
// (4.1 TB/s), of which the instructions are the larger part. RW = 1 for calls of few
// rows (less than 8 a sequence): a word stored by each thread.
template <int HD, typename T, int RW>
__global__ void __launch_bounds__(256) k_kv4_write(const __grid_constant__ Kv4Rows X, const __grid_constant__ Kv4Seqs S,
                                                   int n, int kv) {
  pdl_wait();
  const int b = blockIdx.y >> 1, kind = blockIdx.y & 1;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int per = kv * (HD / 8);
  const int64_t rb = a4_div(id, per);             // rows RW rb ..
  const int e = (int)(id - rb * per);
  const int h = e / (HD / 8), blk = e % (HD / 8);  // values 8 blk .. of head h
  const int rows = (int)min((int64_t)RW, max((int64_t)0, n - rb * RW));
  const T *src = (const T *)X.p[kind] + b * X.seq_stride[kind] + rb * RW * X.row_stride[kind] + (int64_t)e * 8;
  float x[RW][8];
  if (X.vec[kind]) {
    constexpr int V = sizeof(T) / 2;
    uint4 raw[RW][V];
#pragma unroll
    for (int r = 0; r < RW; ++r)
#pragma unroll
      for (int v = 0; v < V; ++v)
        raw[r][v] = r < rows ? __ldg((const uint4 *)(src + r * X.row_stride[kind]) + v) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      T t[8];
      memcpy(t, raw[r], sizeof(t));
#pragma unroll
      for (int i = 0; i < 8; ++i) x[r][i] = (float)t[i];
    }
  } else {
#pragma unroll
    for (int r = 0; r < RW; ++r)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[r][i] = r < rows ? (float)src[r * X.row_stride[kind] + i] : 0.f;
  }
  bool bad = false;
  uint32_t w[RW], sc[RW];
#pragma unroll
  for (int r = 0; r < RW; ++r) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = kv4_amax(amax, x[r][i]);
    if (!(amax <= KV4_MAX)) {
      amax = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[r][i] = kv4_clean(x[r][i], bad);
        amax = fmaxf(amax, fabsf(x[r][i]));
      }
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const __half sh = kv4_scale(amax);
    sc[r] = __half_as_ushort(sh);
    w[r] = kv4_word<sizeof(T) == 2>(x[r], __half2float(sh));
  }
  const int m = threadIdx.x & 3;
  if constexpr (RW == 4) kv4_transpose(w, m);  // word m of row r is w[r] of neighbour m
  if ((RW == 4 ? m : 0) < rows) {
    const int64_t row = S.at[b] + rb * RW + (RW == 4 ? m : 0);
    uint8_t *tile = (kind ? S.v[b] : S.k[b]) + h * S.head_bytes + (row / KV4_TILE) * kv4_tile_bytes(HD);
    const int i = (int)(row % KV4_TILE), c = blk >> 2;
    if constexpr (RW == 4) {
      *(uint4 *)(tile + kv4_code_off(i, c)) = make_uint4(w[0], w[1], w[2], w[3]);
      const uint32_t s = m == 0 ? sc[0] : m == 1 ? sc[1] : m == 2 ? sc[2] : sc[3];
      *(uint16_t *)(tile + kv4_scale_off(HD, i, c)) = (uint16_t)s;
    } else {
      *(uint32_t *)(tile + kv4_code_off(i, c) + m * 4) = w[0];
      if (m == 0) *(uint16_t *)(tile + kv4_scale_off(HD, i, c)) = (uint16_t)sc[0];
    }
  }
  if (bad) atomicOr(&g_dev_error, DFL_ERR_RANGE);
}

// The exact values of rows at .. at + n - 1, f32 [b][n][kv][HD]. A thread has eight
// values of four rows; a row's 16 code bytes of a group come in one load by one of four
// neighbours, and pairs of neighbours halve their words between them, so that what they
// store is whole sectors: 306 MB in 45 us, HBM's rate (65 us with a row and its eight
// values a thread, each store half of its sectors).
template <int HD>
__global__ void __launch_bounds__(256) k_kv4_read(const __grid_constant__ Kv4Seqs S, int n, int kv,
                                                  float *__restrict__ ok, float *__restrict__ ov) {
  pdl_wait();
  const int b = blockIdx.y >> 1, kind = blockIdx.y & 1, m = threadIdx.x & 3;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int per = kv * (HD / 8);
  const int64_t rb = a4_div(id, per);             // rows 4 rb ..
  const int e = (int)(id - rb * per), h = e / (HD / 8), c = e % (HD / 8) >> 2;
  const int rows = (int)min((int64_t)4, max((int64_t)0, n - rb * 4));
  uint4 mine = make_uint4(0, 0, 0, 0);
  uint32_t sm = 0;
  if (m < rows) {
    const int64_t row = S.at[b] + rb * 4 + m;
    const uint8_t *tile = (kind ? S.v[b] : S.k[b]) + h * S.head_bytes + (row / KV4_TILE) * kv4_tile_bytes(HD);
    const int i = (int)(row % KV4_TILE);
    mine = *(const uint4 *)(tile + kv4_code_off(i, c));
    sm = *(const uint16_t *)(tile + kv4_scale_off(HD, i, c)) * 0x10001u;
  }
  uint32_t w[4] = {mine.x, mine.y, mine.z, mine.w};
  kv4_transpose(w, m);
  float *out = (kind ? ov : ok) + (((int64_t)b * n + rb * 4) * per + (e & ~1)) * 8 + (m & 1) * 4;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    uint32_t s16, m24, a[4];
    kv4_scale_pair(__shfl_sync(0xffffffffu, sm, r, 4), s16, m24);
    // values 0 - 3 of both words in the even neighbour, 4 - 7 in the odd one
    const uint32_t got = __shfl_xor_sync(0xffffffffu, w[r], 1);
    const uint32_t x = m & 1 ? (got >> 8 & 0x00FF00FFu) | (w[r] & 0xFF00FF00u)
                             : (w[r] & 0x00FF00FFu) | (got << 8 & 0xFF00FF00u);
    kv4_dequant8(x, s16, m24, a);
    if (r < rows) {
      const float2 v0 = __half22float2(*(const __half2 *)&a[0]), v1 = __half22float2(*(const __half2 *)&a[1]);
      const float2 v2 = __half22float2(*(const __half2 *)&a[2]), v3 = __half22float2(*(const __half2 *)&a[3]);
      float *o = out + (int64_t)r * per * 8;
      *(float4 *)o = make_float4(v0.x, v0.y, v1.x, v1.y);
      *(float4 *)(o + 8) = make_float4(v2.x, v2.y, v3.x, v3.y);
    }
  }
}

// ---------------------------------------------------------------- sharing out the context
//
// The context rows of all (sequence, KV head) pairs, in rounds of 128 rows, are
// shared out evenly over the CTAs of a launch, whatever the sequences' lengths:
// a CTA takes the next T / G or one more of them, pieces of one or more pairs. A piece
// that is its whole pair in one run gives y; the others leave a partial (unnormalised o,
// reference m, sum l per query) in slot i + (index of the pair), which is different
// for every piece, and a second kernel merges a pair's partials. (With a fixed number
// of splits a pair, 32 blocks over 8,192 rows each took 190 us and not 153: the last
// CTAs of a launch had the GPU to themselves.)
// Weights 2^(x - m) stay at or below 2^TAU, inside f16's range, and a new reference puts
// the row's largest weight so far at 2^BIAS: high, because what a weight's f16 form (or
// its two planes) loses to f16's lowest step is then at most 2^-34 of the largest. (With
// 2^4, weights 20 nats below the largest had lost a sixth of themselves, and those from
// 29 bits below on all.) TAU - BIAS is what scores may grow by before the reference has
// to follow: 5.9 bits cost nothing against 7, 3.9 bits 2 - 15% of a launch.
constexpr float A4_TAU = 15.9f, A4_BIAS = 10.f;
constexpr float A4_NONE = 3.402823466e38f;  // minus the reference of a query that has seen no row

// A matrix instruction cuts off what its f32 sum does not hold, always towards 0, so that
// a sum of n / 16 steps drifts by some 2^-23 of itself a step (3e-4 after 32,768 rows). A
// long piece is therefore taken in runs of at most 256 steps of a sum, whose results are
// joined in ordinary f32 in the piece's slot. (A run's end and the next one's start cost
// k_attn4 about 2.5 us: 32 blocks over 32,768 rows each 529 us, in one run a piece 516.)
constexpr int A4_STEPS = 256;

struct A4Seq {
  const uint8_t *k, *v;    // the caches
  const uint8_t *ok, *ov;  // the block's own rows (one tile a KV head), or null
  int64_t row0;            // first cache row read
  int n;                   // rows read
  int64_t anchor;          // the first query's cache row, relative to row0
};
struct A4Args {
  A4Seq seq[MAX_BATCH];
  int64_t head_bytes;
  const void *q;
  int64_t q_seq, q_row;    // strides of q in elements
  void *y;
  float *lse;
  float *part;
  int dtype;
  int heads, kv, R, window, causal;
  int always_part;         // partials of whole pairs too (the merge packs them)
  float scale;
  int64_t round0[MAX_BATCH + 1];  // the first round of sequence b's pairs
  int64_t run0[MAX_BATCH + 1];    // the first run of sequence b's pairs
  int64_t share;           // rounds of a CTA, at least
  int batch, ctas, more;
  int run;                 // rounds of a run
};

// Rounds of a pair. k_attn4's are the tiles its range touches and the own rows'
// tile; k_attn4_few's are the groups of 16 rows that it touches and the own rows'
// group, eight at a time.
// At least one, so that a query that sees nothing is written too.
__host__ __device__ __forceinline__ int a4_tiles(const A4Seq &s) {
  return (s.n > 0 ? (int)(((int64_t)(s.row0 % KV4_TILE) + s.n + KV4_TILE - 1) / KV4_TILE) : 0) + (s.ok ? 1 : 0);
}
template <bool FEW>
__host__ __device__ __forceinline__ int a4_rounds(const A4Seq &s) {
  if (!FEW) return a4_tiles(s) > 0 ? a4_tiles(s) : 1;
  const int first = (int)(s.row0 % KV4_TILE);
  const int groups = (s.n > 0 ? (int)(((int64_t)first + s.n + 15) / 16) - first / 16 : 0) + (s.ok ? 1 : 0);
  return groups > 8 ? (groups + 7) / 8 : 1;
}
__host__ __device__ __forceinline__ int a4_runs(const A4Args &A, int nr) { return (nr + A.run - 1) / A.run; }
// The first round of CTA i (of them, `more` take one round more than the others);
// the CTA that takes round t.
__device__ __forceinline__ int64_t a4_first(const A4Args &A, int64_t i) { return i * A.share + min(i, (int64_t)A.more); }
__device__ __forceinline__ int64_t a4_cta(const A4Args &A, int64_t t) {
  const int64_t big = A.more * (A.share + 1);
  return t < big ? a4_div(t, A.share + 1) : A.more + a4_div(t - big, A.share);
}

// A CTA's pieces, one after another, run by run.
template <bool FEW>
struct A4Piece {
  int64_t rnd, rend;  // rounds still to take
  int b, h;           // the piece's pair
  int r0, r1, nr;     // the run's rounds [r0, r1) of the pair's nr
  __device__ __forceinline__ void start(const A4Args &A) {
    rnd = a4_first(A, blockIdx.x);
    rend = a4_first(A, (int64_t)blockIdx.x + 1);
    b = 0;
  }
  __device__ __forceinline__ bool next(const A4Args &A) {
    if (rnd >= rend) return false;
    while (rnd >= A.round0[b + 1]) ++b;
    nr = a4_rounds<FEW>(A.seq[b]);
    const int64_t in_seq = rnd - A.round0[b];
    h = (int)a4_div(in_seq, nr);
    r0 = (int)(in_seq - (int64_t)h * nr);
    r1 = (int)min((int64_t)nr, r0 + min(rend - rnd, (int64_t)A4_STEPS));
    rnd += r1 - r0;
    return true;
  }
  // The piece's first round (of which the CTA's first piece may not be the pair's), and
  // how many of its runs are still to come.
  __device__ __forceinline__ int begin(const A4Args &A) const {
    return (int)max((int64_t)0, a4_first(A, blockIdx.x) - (rnd - r1));
  }
  __device__ __forceinline__ int left() const {
    return (int)((min((int64_t)nr - r1, rend - rnd) + A4_STEPS - 1) / A4_STEPS);
  }
  __device__ __forceinline__ int64_t slot(const A4Args &A) const { return (int64_t)blockIdx.x + (int64_t)b * A.kv + h; }
};
// The rows of sequence s's range that every query sees.
__device__ __forceinline__ void a4_clear(const A4Args &A, const A4Seq &s, int &va, int &vb) {
  va = A.window > 0 ? (int)min((int64_t)s.n, max((int64_t)0, s.anchor + A.R - A.window)) : 0;
  vb = A.causal ? (int)max((int64_t)-1, min((int64_t)s.n, s.anchor + 1)) : s.n;
}
// The queries lo <= r <= hi that see row `row` of s's range.
__device__ __forceinline__ void a4_seen(const A4Args &A, const A4Seq &s, int row, int &lo, int &hi) {
  lo = 0;
  hi = A.R - 1;
  if ((unsigned)row >= (unsigned)s.n) hi = -1;
  const int64_t rel = row - s.anchor;
  if (A.window > 0) hi = (int)min((int64_t)hi, max((int64_t)-1, rel - 1 + A.window));
  if (A.causal) lo = (int)min((int64_t)A.R, max((int64_t)0, rel));
}

__device__ __forceinline__ float a4_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two weights as f16: rounded, or (SPL = 2) as hi, the top 11 bits, and lo, the
// rest rounded (together about 22 bits).
template <int SPL>
__device__ __forceinline__ void a4_pack(float p0, float p1, uint32_t &hi, uint32_t &lo) {
  float h0 = p0, h1 = p1;
  if (SPL == 2) {
    h0 = __uint_as_float(__float_as_uint(p0) & 0xFFFFE000u);
    h1 = __uint_as_float(__float_as_uint(p1) & 0xFFFFE000u);
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(p1 - h1), "f"(p0 - h0));
  }
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(h1), "f"(h0));
}
// The power of two f0 * f1 that brings a row's largest magnitude to [2^10, 2^11)
// (1 for a row of zeros or one that is not finite), and the factor from a product
// with the row so scaled to a score in the base-2 domain: above 0, as masks of -inf are
// multiplied by it. (Where it would leave f32's normal range, scores are far below any
// step of a weight: products are below 2^33.)
__device__ __forceinline__ float a4_row_scale(float amax, float scale, float &f0, float &f1) {
  int ex = 0;
  if (amax > 0.f && amax < INFINITY) {
    const int b = __float_as_int(amax);
    ex = 11 - (b >> 23 ? (b >> 23) - 126 : -117 - __clz(b));  // -117 .. 160
  }
  f0 = __int_as_float((127 + ex / 2) << 23);
  f1 = __int_as_float((127 + ex - ex / 2) << 23);
  return fmaxf(scale * 1.4426950408889634f * __int_as_float((127 - ex / 2) << 23) *
                   __int_as_float((127 - (ex - ex / 2)) << 23),
               1.17549435e-38f);
}
// N values of a query row, STEP apart (f32 rows with SPL = 2, f16 or bf16 ones else).
template <int SPL, int N, int STEP>
__device__ __forceinline__ void a4_row(const A4Args &A, int64_t at, float (&x)[N]) {
  if constexpr (SPL == 2) {
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = ((const float *)A.q)[at + STEP * e];
  } else {
    uint16_t w[N];
#pragma unroll
    for (int e = 0; e < N; ++e) w[e] = ((const uint16_t *)A.q)[at + STEP * e];
#pragma unroll
    for (int e = 0; e < N; ++e)
      x[e] = A.dtype == DFLASH_F16 ? __half2float(__ushort_as_half(w[e])) : __uint_as_float((uint32_t)w[e] << 16);
  }
}
// Minus the reference for a query whose largest score is y (base 2). From 2^24 on, where
// a score's rounding passes 1, the reference is a few of its steps lower still: the
// product's rest, which a fused sum with the reference leaves, then never takes the
// largest score's weight away. (At the cap: y is infinite.)
__device__ __forceinline__ float a4_ref(float y) {
  return fabsf(y) >= 16777216.f ? A4_BIAS - y + fminf(fabsf(y) * 0x1p-22f, 1e32f) : A4_BIAS - y;
}
// A score against its new reference, kept inside f16's range as a weight where those
// steps pass it (an ordinary one is never above TAU there).
__device__ __forceinline__ float a4_capped(float x) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(A4_TAU));
  return r;
}
// The larger of two values, NaN when one is.
__device__ __forceinline__ float a4_max(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// ---------------------------------------------------------------- many query rows
//
// One CTA an SM, keys as the MMAs' rows: a chunk is a tile of 128 cache rows.
//   S^T [128 keys][queries] = K Q^T     A = K dequantised into tensor memory,
//                                       B = the queries in shared memory
//   O^T [hd][queries] += V^T P^T        A = V dequantised into shared memory
//                                       (MN-major), B = P in shared memory (MN-major)
// so that all 128 lanes of the softmax hold keys, and up to 64 queries with both
// planes fit one product's N. With f32 rows (SPL = 2) the queries and P enter as
// f16 hi + lo planes side by side in N, their two partial products added in
// registers; f16 and bf16 rows take one plane (P rounded to f16, 2^-12 of each
// weight, below the output's own rounding).
//   warps 0 .. SMW-1   softmax: thread = one key and QPT queries
//   the next 4         K: thread = one key, codes -> f16 -> tensor memory
//   the next 4         V: thread = one key, codes -> f16 -> shared memory
//   the next 4         MMA issue, one thread each: S of even and of odd chunks,
//                      O of even and of odd chunks (two accumulators each, which
//                      halves what their sums lose; one and one issuer at N 128)
// Chunks are counted through the CTA's pieces, so that the next piece's keys and
// scores are under way while the last one's results are written. The softmax warps
// stage a piece's queries. A key's codes come through a ring of stages in shared
// memory that its thread alone fills (asynchronous copies) and reads.
//
// What bounds it: no one part. A chunk takes some 2,200 cycles (with 16 queries a softmax
// thread 3,600), where HBM brings it in 784. The tensor pipe is 19 - 23% active: one
// thread issues an MMA in 50 - 70 cycles (N 32 to 128 alike, on an idle SM), and the last
// one's results are there some 240 cycles later, so that a chunk's eight of S take 810
// cycles and its eight of O 890, beside other chunks'. A softmax turn is mostly its steps
// from one wait, load or vote to the next, and a CTA's first chunk, last results and the
// merge are about 10 us that nothing covers. (Leaving out three quarters of the MMAs, or
// the dequantisation, or the exponentials each shortens a launch by 2 - 10%; two chunks a
// turn, or packed f32 operations, by nothing.) 32 f32 blocks of 16 over up to 8,192 rows
// each (8 KV heads of 128, 2 queries a head): 140 us, the merge included, for 282 MB; one
// block over 32,768 rows (4 queries a head): 43 us.
//
// The softmax runs in base 2 with a lazy reference: P = 2^(x - m) with m moved
// only when a score passes it by more than TAU (then m is the largest score so
// far less BIAS), so that P stays at 2^TAU or below in f16. Scores are per
// key, so finding a new reference reduces over lanes; a chunk in which no score
// passes costs one barrier with a vote. A query that has seen no row yet has
// f32's lowest number as its reference, which any score passes. A score that is not a number
// passes too and makes its query's reference, and so its output, NaN.
template <int HD, int NQ, int SPL>
struct A4 {
  static constexpr int QPT = NQ == 64 ? 16 : 8;      // queries a softmax thread
  static constexpr int SMW = 4 * (NQ / QPT);         // softmax warps
  static constexpr int SMT = 32 * SMW;
  static constexpr int THREADS = 32 * (SMW + 12);
  static constexpr int NS = NQ * SPL;                // columns of S and of O
  static constexpr int NO = NS <= 64 ? 4 : 1;        // output accumulators, taken in turn
  static constexpr int NI = NO == 1 ? 1 : 2;         // threads that issue O's products
  static constexpr int KC = HD / 2;                  // tensor-memory columns of a K slot
  static constexpr int TK = 0, TS = 2 * KC, TO = TS + 2 * NS;
  static_assert(TO + NO * NS <= 512, "tensor memory");
  static constexpr int BLK = KV4_TILE * 128;         // 128 keys x 64 halves
  static constexpr int VST = (HD / 64) * BLK;        // a V stage
  static constexpr int PST = (NS > 64 ? 2 : 1) * BLK;
  static constexpr int QB = NS * 128;                // a 64-wide block of the queries
  static constexpr int QST = (HD / 64) * QB;         // a piece's queries
  // V stages, P stages, the piece's queries, the codes. With HD = 64 the V operand's upper 64
  // rows are whatever follows the stage in shared memory (their outputs are not read)
  static constexpr int OFF_P = 2 * VST, OFF_Q = OFF_P + 2 * PST, OFF_R = OFF_Q + QST;
  static constexpr int RS = NS > 64 ? 3 : 4;         // stages of the codes' ring (K and V)
  static constexpr int OFF_END = OFF_R + 2 * RS * kv4_tile_bytes(HD);
  static constexpr size_t BYTES = 1024 + OFF_END;
};

// Asynchronous copies of 16, 8 or 4 bytes into shared memory.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// N columns of this thread's lane; the caller waits (tc_wait_ld).
template <int N>
__device__ __forceinline__ void tmem_ld_n(uint32_t addr, uint32_t (&r)[N]) {
  if constexpr (N == 16) {
    tmem_ld16(addr, r);
  } else {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr)
                 : "memory");
  }
}
template <int N>
__device__ __forceinline__ void tmem_st_n(uint32_t addr, const uint32_t (&r)[N]) {
  if constexpr (N == 16) {
    tmem_st16(addr, r);
  } else {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
  }
}

// A run of a piece as the warps of k_attn4 read it from shared memory: its first chunk's
// tiles and row of the range, its chunks (the last one the own rows' with `own`).
struct __align__(16) A4Job {
  const uint8_t *k, *v, *ok, *ov;
  int64_t slot;
  int b, h, nch, lo, n, own, whole;
  int prior, left;  // the piece's runs before (are there any) and behind it
};
constexpr int A4_JOBS = 16;  // runs a window holds

// Run `i` (counted from the CTA's first) into *job; false past the last one. A pair's runs
// lie at multiples of A.run rounds from its start; a CTA's first and last may be parts.
template <int HD>
__device__ __forceinline__ bool a4_job(const A4Args &A, int64_t i, A4Job *job) {
  const int64_t r0 = a4_first(A, blockIdx.x), r1 = a4_first(A, (int64_t)blockIdx.x + 1);
  // the run that holds round r0, and the one i further on
  int b = 0;
  while (r0 >= A.round0[b + 1]) ++b;
  int nr = a4_rounds<false>(A.seq[b]);
  const int64_t in_seq = r0 - A.round0[b], h0 = a4_div(in_seq, nr);
  int64_t u = A.run0[b] + h0 * a4_runs(A, nr) + (int)(in_seq - h0 * nr) / A.run + i;
  while (b < A.batch && u >= A.run0[b + 1]) ++b;
  if (b >= A.batch) return false;
  const A4Seq &s = A.seq[b];
  nr = a4_rounds<false>(s);
  u -= A.run0[b];
  const int h = (int)a4_div(u, a4_runs(A, nr)), run = (int)(u - (int64_t)h * a4_runs(A, nr));
  const int64_t t0 = A.round0[b] + (int64_t)h * nr;
  // the piece's rounds, and the run's of them
  const int p0 = (int)max((int64_t)0, r0 - t0), p1 = (int)min((int64_t)nr, r1 - t0);
  const int f = max(p0, run * A.run), e = min(p1, (run + 1) * A.run);
  if (f >= e) return false;
  const int tiles = a4_tiles(s), first = (int)(s.row0 % KV4_TILE);
  job->nch = max(0, min(e, tiles) - f);
  job->own = s.ok != nullptr && e == tiles;
  const int64_t at = h * A.head_bytes + (s.row0 / KV4_TILE + f) * kv4_tile_bytes(HD);
  job->k = s.k + at;
  job->v = s.v + at;
  job->ok = s.ok ? s.ok + (int64_t)h * kv4_tile_bytes(HD) : nullptr;
  job->ov = s.ok ? s.ov + (int64_t)h * kv4_tile_bytes(HD) : nullptr;
  job->b = b;
  job->h = h;
  job->lo = (int)((int64_t)f * KV4_TILE - first);
  job->n = s.n;
  job->whole = f == 0 && e == nr && !A.always_part;
  job->prior = f > p0;
  job->left = (p1 - e + A.run - 1) / A.run;
  job->slot = (int64_t)blockIdx.x + (int64_t)b * A.kv + h;
  return true;
}

// One arrival for the warp's 32 threads, ordered behind what they did. (512 arrivals
// a chunk, one a thread, each took their turn at one address.)
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// A whole warp's wait. The first poll is apart, without the loop that lanes may leave
// one by one: most waits on a chunk's path find their phase complete.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, mbar_try(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait_spin(bar, parity));
}

template <int HD, int NQ, int SPL>
__global__ void __launch_bounds__(A4<HD, NQ, SPL>::THREADS, 1) k_attn4(const __grid_constant__ A4Args A) {
  using C = A4<HD, NQ, SPL>;
  constexpr int QPT = C::QPT, SMW = C::SMW, NS = C::NS, NO = C::NO, NI = C::NI;
  extern __shared__ __align__(1024) uint8_t smraw[];
  uint8_t *sm = smraw + ((1024 - (smem_u32(smraw) & 1023)) & 1023);
  const uint32_t smb = smem_u32(sm);
  __shared__ __align__(8) uint64_t bars[14];
  __shared__ A4Job jobs[A4_JOBS];
  __shared__ int njobs;
  __shared__ uint32_t tslot;
  __shared__ int dead[4];                     // a group of softmax warps gave up a wait
  __shared__ __align__(16) float sl2[NQ];     // a query's score to the base-2 domain
  __shared__ __align__(16) float negm[SMW][QPT];  // -m, each warp's own copy of its queries'
  // a chunk's largest raw scores, by query and quarter of the keys (two sets in turn)
  __shared__ __align__(16) float evmax[2][NQ][4];
  __shared__ __align__(16) float lsum[NQ][4];
  const uint32_t kfull = smem_u32(bars), sfull = kfull + 16, sfree = sfull + 16, pfull = sfree + 16,
                 vfull = pfull + 16, pvdone = vfull + 16, qfull = pvdone + 16, fin = qfull + 8;
  const int rep = A.heads / A.kv, R = A.R, Q = rep * R;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(kfull + 8 * i, 4);
      mbar_init(sfull + 8 * i, 1);
      mbar_init(sfree + 8 * i, SMW);
      mbar_init(pfull + 8 * i, SMW);
      mbar_init(vfull + 8 * i, 4);
      mbar_init(pvdone + 8 * i, 1);
    }
    mbar_init(qfull, SMW);
    mbar_init(fin, 2 + NI);
    mbar_fence_init();
    dead[0] = dead[1] = dead[2] = dead[3] = 0;
  }
  // the first window of pieces (nothing of it comes from an earlier kernel)
  if (warp == 1) {
    const bool have = lane < A4_JOBS && a4_job<HD>(A, lane, jobs + lane);
    const uint32_t m = __ballot_sync(0xffffffffu, have);
    if (lane == 0) njobs = __popc(m);
  }
  pdl_wait();
  if (warp == 0) tmem_alloc(smem_u32(&tslot), 512);
  // The queries of a piece, a softmax warp a row: scaled by a power of two each
  // (small values of a large row keep 22 bits of it), as f16 planes
  auto stage_q = [&](const A4Job &job) {
    uint8_t *qs = sm + C::OFF_Q;
    constexpr int N = NQ / SMW;  // rows a warp: all their loads first
    constexpr int DL = HD / 32;   // consecutive values a lane
    float x[N][DL];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int row = warp + i * SMW, r = row < Q ? row : 0;
      const int64_t at = job.b * A.q_seq + r % R * A.q_row + (job.h * rep + r / R) * HD;
      a4_row<SPL, DL, 1>(A, at + DL * lane, x[i]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int row = warp + i * SMW;
      float amax = 0.f;
#pragma unroll
      for (int e = 0; e < DL; ++e) {
        if (row >= Q) x[i][e] = 0.f;
        amax = fmaxf(amax, fabsf(x[i][e]));
      }
      float f0, f1;
      const float sc = a4_row_scale(warp_max(amax), A.scale, f0, f1);
      if (lane == 0) sl2[row] = sc;
      uint32_t hi[DL / 2], lo[DL / 2];
#pragma unroll
      for (int e = 0; e < DL; e += 2) {
        const float y0 = x[i][e] * f0 * f1, y1 = x[i][e + 1] * f0 * f1;
        const __half2 h = __floats2half2_rn(y0, y1);
        memcpy(&hi[e / 2], &h, 4);
        if (SPL == 2) {
          const float2 f = __half22float2(h);
          const __half2 l = __floats2half2_rn(y0 - f.x, y1 - f.y);
          memcpy(&lo[e / 2], &l, 4);
        }
      }
      const int d = DL * lane, blk = d >> 6, ch = (d & 63) >> 3, in = d & 7;
#pragma unroll
      for (int p = 0; p < SPL; ++p) {
        uint8_t *to = qs + blk * C::QB + sw128_off(p * NQ + row, ch) + in * 2;
        const uint32_t *v = p ? lo : hi;
        if constexpr (DL == 4) *(uint2 *)to = make_uint2(v[0], v[1]);
        else *(uint32_t *)to = v[0];
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  };
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = tslot;

  // The next window of up to A4_JOBS runs (after the first, once every warp is done
  // with the last one): how many there are (fewer in the CTA's last window). Every warp asks for
  // the same windows, in its own loop.
  auto window = [&](int64_t i0, auto makes) {
    if (i0 == 0) return njobs;
    __syncthreads();
    if (decltype(makes)::value && warp == 0) {
      const bool have = lane < A4_JOBS && a4_job<HD>(A, i0 + lane, jobs + lane);
      const uint32_t m = __ballot_sync(0xffffffffu, have);
      if (lane == 0) njobs = __popc(m);
    }
    __syncthreads();
    return njobs;
  };
  // chunks (J) and pieces with chunks (np) are counted through all windows
  int J = 0, np = 0, nj = A4_JOBS;
  bool ok = true;  // no wait of this warp gave up
  if (warp < SMW) {
    // With 28 warps a thread has 72 registers: the softmax warps take 88, the others
    // fewer (4 x 88 + 2 x 56 + 40 = 7 x 72 a thread of the seven warpgroups)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 88;");
    // ------------------------------------------------------------ softmax
    const int key = (warp & 3) * 32 + lane, q0 = (warp >> 2) * QPT;
    const uint32_t lrow = (uint32_t)((warp & 3) * 32) << 16;
    int evs = 0;  // references found so far
    float *nm = negm[warp];
    // four warps, a group, hold all the keys of QPT queries and vote on their references;
    // the groups run through a piece's chunks on their own
    const int group_bar = 2 + (warp >> 2);
    for (int64_t i0 = 0; nj == A4_JOBS; i0 += A4_JOBS) {
    nj = window(i0, std::true_type{});
    for (int ji = 0; ji < nj; ++ji) {
      const A4Job &job = jobs[ji];
      const int nch = job.nch;
      int va, vb;
      a4_clear(A, A.seq[job.b], va, vb);
      float l[QPT];
#pragma unroll
      for (int i = 0; i < QPT; ++i) l[i] = 0.f;
      __syncwarp();  // the warp's lanes have read the references of the piece before
      if (lane < QPT) nm[lane] = A4_NONE;
      if (nch > 0) {
        if (!job.prior) stage_q(job);  // (the scores of the piece before, the last ones' last readers, are done)
        warp_arrive(qfull);
      }
      // the queries' factors are written; the last piece's sums have been read
      asm volatile("bar.sync 1, %0;" ::"n"(C::SMT) : "memory");
      const int own_i = job.own ? nch - 1 : -1, first = job.lo;
      for (int i = 0; i < nch; ++i) {
        const int j = J + i, sb = j & 1, u = j >> 1;
        const bool is_own = i == own_i;
        const int lo = first + i * KV4_TILE;  // the chunk's first row in the range
        const bool edge = is_own || lo < va || vb - lo < KV4_TILE;  // (lo + 128 can pass 2^31)
        ok = ok && mbar_wait_warp(sfull + 8 * sb, u & 1);
        tc_fence_after();
        // scores in the base-2 domain, raw or against the reference
        float t[QPT];
        auto scores = [&](bool raw) {
          uint32_t r0[QPT], r1[SPL == 2 ? QPT : 1];
          tmem_ld_n<QPT>(tb + lrow + C::TS + sb * NS + q0, r0);
          if constexpr (SPL == 2) tmem_ld_n<QPT>(tb + lrow + C::TS + sb * NS + NQ + q0, r1);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < QPT; ++e) {
            t[e] = __uint_as_float(r0[e]);
            if constexpr (SPL == 2) t[e] += __uint_as_float(r1[e]);
          }
#pragma unroll
          for (int e = 0; e < QPT; e += 4) {
            const float4 m = *(const float4 *)(sl2 + q0 + e);
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            if (!raw) s = *(const float4 *)(nm + e);
            t[e] = fmaf(t[e], m.x, s.x);
            t[e + 1] = fmaf(t[e + 1], m.y, s.y);
            t[e + 2] = fmaf(t[e + 2], m.z, s.z);
            t[e + 3] = fmaf(t[e + 3], m.w, s.w);
          }
          if (edge) {
            // queries rlo <= r <= rhi see this thread's key
            int rlo = 0, rhi = key < R ? R - 1 : -1;
            if (!is_own) a4_seen(A, A.seq[job.b], lo + key, rlo, rhi);
            if (rlo > 0 || rhi < R - 1) {
              int r = q0 % R;
#pragma unroll
              for (int e = 0; e < QPT; ++e) {
                if (r < rlo || r > rhi) t[e] = -INFINITY;
                r = r + 1 == R ? 0 : r + 1;
              }
            }
            asm volatile("" : "+f"(t[0]));  // a branch, not selects in every chunk
          }
        };
        float top = -INFINITY;
        if (ok) {
          // (before the first reference the raw scores, so that the first chunk takes them once)
          scores(i == 0);
#pragma unroll
          for (int e = 0; e < QPT; ++e) top = a4_max(top, t[e]);
        } else if (lane == 0) {
          dead[warp >> 2] = 1;
        }
        uint32_t ev;
        asm volatile(
            "{\n .reg .pred a, b;\n setp.ne.u32 a, %1, 0;\n bar.red.or.pred b, %2, 128, a;\n selp.u32 %0, 1, 0, b;\n}\n"
            : "=r"(ev)
            : "r"((uint32_t)(i == 0 || !(top <= A4_TAU) || !ok)), "r"(group_bar)
            : "memory");
        if (ev) {
          // a score passes its reference (or a wait gave up): the chunk's largest
          // raw score of each query, then new references and rescaled l and O
          if (ok) {
            if (i > 0) scores(true);
            // the largest over the warp's 32 keys, the queries halved with every step:
            // lane l ends with query l / (32 / QPT)
            float y[QPT];
#pragma unroll
            for (int e = 0; e < QPT; ++e) y[e] = t[e];
#pragma unroll
            for (int k = 0; k < 5; ++k) {
              const int o = 16 >> k, w = QPT >> (k + 1);
              const bool up = lane & o;
#pragma unroll
              for (int e = 0; e < w; ++e) {
                const float other = __shfl_xor_sync(0xffffffffu, up ? y[e] : y[e + w], o);
                y[e] = a4_max(up ? y[e + w] : y[e], other);
              }
              if (w == 0) y[0] = a4_max(y[0], __shfl_xor_sync(0xffffffffu, y[0], o));
            }
            if (lane % (32 / QPT) == 0) evmax[evs & 1][q0 + lane / (32 / QPT)][warp & 3] = y[0];
          }
          asm volatile("bar.sync %0, 128;" ::"r"(group_bar) : "memory");
          if (*(volatile int *)&dead[warp >> 2]) break;
          const float(*ev4)[4] = evmax[evs & 1] + q0;
          ++evs;
          // a query's new reference: the first rows it sees, or a score past the last one
          auto moved = [&](int e, float old) {
            const float4 v = *(const float4 *)ev4[e];
            const float y = a4_max(a4_max(v.x, v.y), a4_max(v.z, v.w));
            const float nn = a4_ref(y);
            if (old == A4_NONE) return y != -INFINITY ? nn : old;
            return y + old > A4_TAU && nn < old ? nn : old;  // (never back down)
          };
          if (i > 0) {
            // l and O of the chunks before, whose products are done (chunk j - 2's first:
            // a barrier is then at most one phase behind its parity wait)
            if (j >= 2) ok = __all_sync(0xffffffffu, mbar_wait(pvdone + 8 * sb, (u - 1) & 1));
            ok = ok && __all_sync(0xffffffffu, mbar_wait(pvdone + 8 * (sb ^ 1), ((j - 1) >> 1) & 1));
            tc_fence_after();
            float alpha[QPT];
            bool any = false;
#pragma unroll
            for (int e = 0; e < QPT; ++e) {
              const float old = nm[e], nn = moved(e, old);
              alpha[e] = old == A4_NONE || nn == old ? 1.f : a4_ex2(nn - old);
              l[e] *= alpha[e];
              any = any || alpha[e] != 1.f;
            }
            if (any && ok) {  // alike in every lane
#pragma unroll
              for (int o = 0; o < NO; ++o)
                if (o < i) {  // chunk j - 1's accumulator, then those of the chunks before
#pragma unroll
                  for (int p = 0; p < SPL; ++p) {
                    const uint32_t col = tb + lrow + C::TO + ((j - 1 - o) & (NO - 1)) * NS + p * NQ + q0;
                    uint32_t v[QPT];
                    tmem_ld_n<QPT>(col, v);
                    tc_wait_ld();
#pragma unroll
                    for (int e = 0; e < QPT; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha[e]);
                    tmem_st_n<QPT>(col, v);
                  }
                }
              tc_wait_st();
              tc_fence_before();
            }
          }
          // the warp's copy of the references, a lane a query
          float mine = 0.f;
          if (lane < QPT) mine = moved(lane, nm[lane]);
          __syncwarp();
          if (lane < QPT) nm[lane] = mine;
          __syncwarp();
          if (i == 0) {
#pragma unroll
            for (int e = 0; e < QPT; e += 4) {
              const float4 s = *(const float4 *)(nm + e);
              t[e] += s.x;
              t[e + 1] += s.y;
              t[e + 2] += s.z;
              t[e + 3] += s.w;
            }
          } else {
            scores(false);
          }
#pragma unroll
          for (int e = 0; e < QPT; ++e) t[e] = a4_capped(t[e]);
        }
        tc_fence_before();
        warp_arrive(sfree + 8 * sb);
        // (a wait that gives up here ends all the softmax warps at the next vote)
        if (j >= 2) ok = ok && mbar_wait_warp(pvdone + 8 * sb, (u - 1) & 1);
        if (!ok) {
          if (lane == 0) dead[warp >> 2] = 1;
        } else {
          // P = 2^(x - m), rounded to f16 (one plane) or as hi + lo
#pragma unroll
          for (int c = 0; c < QPT / 8; ++c) {
            uint32_t ph[4], pl[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float p0 = a4_ex2(t[8 * c + 2 * e]), p1 = a4_ex2(t[8 * c + 2 * e + 1]);
              l[8 * c + 2 * e] += p0;
              l[8 * c + 2 * e + 1] += p1;
              a4_pack<SPL>(p0, p1, ph[e], pl[e]);
            }
#pragma unroll
            for (int p = 0; p < SPL; ++p) {
              const uint32_t *v = p ? pl : ph;
              const int col = p * NQ + q0 + 8 * c;
              *(uint4 *)(sm + C::OFF_P + sb * C::PST + (col >> 6) * C::BLK + sw128_off(key, (col & 63) >> 3)) =
                  make_uint4(v[0], v[1], v[2], v[3]);
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        warp_arrive(pfull + 8 * sb);
      }
      // the sums over the keys, and O once the piece's products have completed
#pragma unroll
      for (int i = 0; i < QPT; ++i) {
        const float s = warp_sum(l[i]);
        if (lane == 0) lsum[q0 + i][warp & 3] = s;
      }
      asm volatile("bar.sync 1, %0;" ::"n"(C::SMT) : "memory");
      J += nch > 0 ? nch : 0;
      const bool live = !(*(volatile int *)&dead[0] | *(volatile int *)&dead[1] | *(volatile int *)&dead[2] |
                          *(volatile int *)&dead[3]);
      bool have = live && nch > 0;
      if (have && nch > 1) have = __all_sync(0xffffffffu, mbar_wait_spin(pvdone + 8 * (J & 1), ((J - 2) >> 1) & 1));
      if (have) have = __all_sync(0xffffffffu, mbar_wait_spin(pvdone + 8 * ((J - 1) & 1), ((J - 1) >> 1) & 1));
      tc_fence_after();
      float o[QPT];
#pragma unroll
      for (int i = 0; i < QPT; ++i) o[i] = 0.f;
      if (have) {
#pragma unroll
        for (int a = 0; a < NO; ++a)
          if (a < nch) {
#pragma unroll
            for (int p = 0; p < SPL; ++p) {
              uint32_t v[QPT];
              tmem_ld_n<QPT>(tb + lrow + C::TO + ((J - 1 - a) & (NO - 1)) * NS + p * NQ + q0, v);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < QPT; ++i) o[i] += __uint_as_float(v[i]);
            }
          }
      }
      if (nch > 0) {
        ok = have;  // (a wait that gave up: the next piece ends at its first vote)
        ++np;
      }
      const int d = key;  // this thread's dimension of O
      const bool stat = (warp & 3) == 0 && lane < QPT && q0 + lane < Q;  // this lane writes query q0 + lane's statistics
      float *part = A.part + (job.slot * Q + q0) * (HD + 4);
      const int at = HD + job.left % 2 * 2, before = HD + 2 - job.left % 2 * 2;  // this run's and the last one's statistics
      float m = -INFINITY, L = 0.f;
      if (stat && have && nm[lane] != A4_NONE) {
        const float4 s = *(const float4 *)lsum[q0 + lane];
        m = -nm[lane];
        L = s.x + s.y + s.z + s.w;
      }
      // (a query that has seen no row has P and so O of 0)
      if (!job.whole) {
        if (job.prior) {
          // the runs before it, in the slot: a lane a query, then every thread its values of O
          const float mb = lane < QPT && q0 + lane < Q ? part[lane * (HD + 4) + before] : -INFINITY;
          const float mi = lane < QPT && have && nm[lane] != A4_NONE ? -nm[lane] : -INFINITY, M = a4_max(mi, mb);
          const float fi = mi != -INFINITY ? a4_ex2(mi - M) : 0.f;
          const float fb = mb != -INFINITY ? a4_ex2(mb - M) : 0.f;
          if (stat) {
            m = M;
            L = fmaf(part[lane * (HD + 4) + before + 1], fb, L * fi);
          }
#pragma unroll
          for (int i = 0; i < QPT; ++i) {
            const float a = __shfl_sync(0xffffffffu, fi, i), b = __shfl_sync(0xffffffffu, fb, i);
            if (d < HD && q0 + i < Q) o[i] = fmaf(part[i * (HD + 4) + d], b, o[i] * a);
          }
        }
        if (stat) {
          part[lane * (HD + 4) + at] = m;
          part[lane * (HD + 4) + at + 1] = L;
        }
        if (d < HD) {
#pragma unroll
          for (int i = 0; i < QPT; ++i)
            if (q0 + i < Q) part[i * (HD + 4) + d] = o[i];
        }
      } else {
        const int64_t row0 = (int64_t)job.b * R * A.heads + job.h * rep;
        if (stat && A.lse) {
          const int q = q0 + lane;
          A.lse[row0 + (int64_t)(q % R) * A.heads + q / R] = L > 0.f || L != L ? (log2f(L) + m) * 0.6931471805599453f : -INFINITY;
        }
        if (d < HD) {
          int r = q0 % R, hr = q0 / R;
#pragma unroll
          for (int i = 0; i < QPT; ++i) {
            const float4 s = *(const float4 *)lsum[q0 + i];
            // a query that sees no row: 0
            const float inv = have && nm[i] != A4_NONE ? 1.f / (s.x + s.y + s.z + s.w) : 0.f;
            if (q0 + i < Q) st_elem(A.y, (row0 + (int64_t)r * A.heads + hr) * HD + d, A.dtype, o[i] * inv);
            if (++r == R) {
              r = 0;
              ++hr;
            }
          }
        }
      }
      if (!live) break;
    }
    }
  } else if (warp < SMW + 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    // ------------------------------------------------------------ K and V: codes to f16
    const bool isv = warp >= SMW + 4;
    const int key = (warp & 3) * 32 + lane;
    const uint32_t lrow = (uint32_t)((warp & 3) * 32) << 16;
    for (int64_t i0 = 0; nj == A4_JOBS; i0 += A4_JOBS) {
    nj = window(i0, std::false_type{});
    int end = J;
    for (int i = 0; i < nj; ++i) end += jobs[i].nch;
    // this thread's key of the ring's stages: copied, waited for and read by it alone
    uint8_t *ring = sm + C::OFF_R + (isv ? C::RS * kv4_tile_bytes(HD) : 0);
    const uint32_t ring32 = smem_u32(ring);
    int aj = 0, ac = 0, slot = 0;  // the chunk that is asked for next: chunk ac of piece aj
    auto fetch = [&](int to) {
      while (aj < nj && ac == jobs[aj].nch) {
        ++aj;
        ac = 0;
      }
      if (aj < nj) {
        const A4Job &job = jobs[aj];
        const bool is_own = job.own && ac == job.nch - 1;
        const uint8_t *tile = is_own ? (isv ? job.ov : job.ok) : (isv ? job.v : job.k) + (int64_t)ac * kv4_tile_bytes(HD);
        const int row = job.lo + ac * KV4_TILE + key;
        const uint32_t dst = ring32 + to * kv4_tile_bytes(HD);
        if (is_own ? key < R : (unsigned)row < (unsigned)job.n) {
#pragma unroll
          for (int c = 0; c < HD / 32; ++c) cp_async16(dst + kv4_code_off(key, c), tile + kv4_code_off(key, c));
          cp_async_small<HD / 16>(dst + kv4_scale_off(HD, key, 0), tile + kv4_scale_off(HD, key, 0));
        } else {
          // a row that is not read: scale 0, so that its values are 0
          *(uint32_t *)(ring + to * kv4_tile_bytes(HD) + kv4_scale_off(HD, key, 0)) = 0u;
          if (HD == 128) *(uint32_t *)(ring + to * kv4_tile_bytes(HD) + kv4_scale_off(HD, key, 2)) = 0u;
        }
        ++ac;
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < C::RS - 1; ++i) fetch(i);
    for (; J < end; ++J) {
      const int sb = J & 1, u = J >> 1;
      fetch(slot == 0 ? C::RS - 1 : slot - 1);
      cp_async_wait<C::RS - 1>();
      const uint8_t *st = ring + slot * kv4_tile_bytes(HD);
      slot = slot + 1 == C::RS ? 0 : slot + 1;
      // the slot's last reader: S of chunk j - 2 (K), O of chunk j - 2 (V)
      if (J >= 2 && !mbar_wait_warp((isv ? pvdone : sfull) + 8 * sb, (u - 1) & 1)) break;
      tc_fence_after();
      uint32_t sc[HD / 64];
#pragma unroll
      for (int c = 0; c < HD / 64; ++c) sc[c] = *(const uint32_t *)(st + kv4_scale_off(HD, key, 2 * c));
#pragma unroll
      for (int c = 0; c < HD / 32; ++c) {
        const uint4 w4 = *(const uint4 *)(st + kv4_code_off(key, c));
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
        uint32_t s16, m24, a[16];
        kv4_scale_pair(__byte_perm(sc[c >> 1], 0u, (c & 1) ? 0x3232 : 0x1010), s16, m24);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t v[4];
          kv4_dequant8(w[i], s16, m24, v);
#pragma unroll
          for (int e = 0; e < 4; ++e) a[4 * i + e] = v[e];
        }
        if (isv) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *(uint4 *)(sm + sb * C::VST + (c >> 1) * C::BLK + sw128_off(key, (c & 1) * 4 + i)) =
                make_uint4(a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]);
        } else {
          tmem_st16(tb + lrow + C::TK + sb * C::KC + c * 16, a);
        }
      }
      if (isv) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      } else {
        tc_wait_st();
        tc_fence_before();
      }
      warp_arrive((isv ? vfull : kfull) + 8 * sb);
    }
    cp_async_wait<0>();
    }
  } else {
    // ------------------------------------------------------------ MMA issue
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    const int w = warp - (SMW + 8), par = w & 1;
    for (int64_t i0 = 0; nj == A4_JOBS; i0 += A4_JOBS) {
    nj = window(i0, std::false_type{});
    for (int ji = 0; ji < nj && ok && lane == 0; ++ji) {
      const A4Job &job = jobs[ji];
      const int nch = job.nch;
      if (w < 2) {
        constexpr uint32_t idesc = f16_idesc(128, NS);
        const uint32_t qb = smb + C::OFF_Q;
        // the piece's queries (waited for in every piece, so that no phase is skipped)
        if (nch > 0 && !(ok = mbar_wait(qfull, np & 1))) break;
        for (int i = (J ^ par) & 1; i < nch; i += 2) {
          const int u = (J + i) >> 1;
          if (!(ok = mbar_wait(kfull + 8 * par, u & 1))) break;
          if (u >= 1 && !(ok = mbar_wait(sfree + 8 * par, (u - 1) & 1))) break;
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < HD / 16; ++ks)
            mma_ts(tb + C::TS + par * NS, tb + C::TK + par * C::KC + ks * 8,
                   sw128_desc(qb + (ks >> 2) * C::QB + (ks & 3) * 32), idesc, ks > 0);
          mma_commit(sfull + 8 * par);
        }
      } else if (w - 2 < NI) {
        // A (V) and B (P) both MN-major
        constexpr uint32_t idesc = f16_idesc(128, NS) | (1u << 15) | (1u << 16);
        for (int i = NI == 2 ? (J ^ par) & 1 : 0; i < nch; i += NI) {
          const int j = J + i, sb = j & 1, u = j >> 1;
          if (!(ok = mbar_wait(vfull + 8 * sb, u & 1))) break;
          // P written: by then every softmax thread has read the pieces before out of O
          if (!(ok = mbar_wait(pfull + 8 * sb, u & 1))) break;
          tc_fence_after();
          const bool is_own = job.own && i == nch - 1;
          const int lo = job.lo + i * KV4_TILE;
          const int ka = is_own ? 0 : max(0, -lo), kb = is_own ? R : min(KV4_TILE, job.n - lo);
          const uint32_t acc = tb + C::TO + (j & (NO - 1)) * NS;
          const uint32_t vb = smb + sb * C::VST, pb = smb + C::OFF_P + sb * C::PST;
          // only the steps of 16 keys that hold a row
          for (int ks = ka / 16; ks < (kb + 15) / 16; ++ks)
            mma_ss(acc, sw128_mn_desc(vb + ks * 2048, C::BLK), sw128_mn_desc(pb + ks * 2048, C::BLK), idesc,
                   i >= NO || ks > ka / 16);
          mma_commit(pvdone + 8 * sb);
        }
      }
      J += nch;
      np += nch > 0;
    }
    __syncwarp();
    }
  }
  if (lane == 0 && warp >= SMW + 8 && warp - (SMW + 8) < 2 + NI) {
    // every MMA of this thread completed before the tensor memory is freed
    mma_commit(fin);
    mbar_wait(fin, 0);
  }
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tb, 512);
  }
}

// ---------------------------------------------------------------- few query rows
//
// k_attn4 takes some 2,200 cycles for 128 keys, however few the queries, where HBM
// brings them in 784. Up to 32 columns (queries, or twice the queries with hi and lo
// planes) mma.sync m16n8k16 (2 cycles an SM each) is cheaper, and its operands are
// registers: the codes go from global memory through a thread's registers into the
// fragments.
//   S^T (16 keys x 8 queries) = K Q^T, O^T (16 values x 8 queries) += V^T P^T
// with K and V as the A operands. The orders of the contraction (head dimension;
// keys) and of the output's rows are free, so the fragments are laid over the
// cache's bytes: with g = lane / 4, t = lane % 4,
//   K   thread t holds values 32 t .. of keys g / 2 + 4 (g % 2) and that + 8 (16
//       bytes and one scale each); HD = 64: half as many
//   V   thread g holds values 16 g .. of keys t, t + 4, t + 8, t + 12; two keys'
//       words are joined half by half, so that a dequantised pair is one value of
//       two keys
//   P   the score fragment (keys x queries), packed and transposed by movmatrix,
//       is the B operand of the second product
// A warp takes 16 keys at a time, with its own m, l and O (a query's reference
// and sums are in the threads that hold its column) and its own ring of stages in
// shared memory, filled by 16-byte asynchronous copies three groups ahead (with
// the codes one group ahead in registers instead, the warps waited for memory
// 40% of their time). What bounds it is the issue of instructions, 66% of the slots,
// and the pipe that the products share with the dequantisation: 32 tokens over 8,192
// rows each (8 KV heads of 128, 4 queries a head, bf16) take 63 us for 282 MB, 4.5
// TB/s. The groups of 32 values are 272
// (K) and 320 (V) bytes apart in a stage, which keeps the reads free of bank
// conflicts. No warp waits for another until the CTA joins its warps' results.
template <int HD>
struct Few {
  static constexpr int WARPS = 8;                    // a round's groups: one a warp
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int STAGES = 4;
  static constexpr int KG = HD == 128 ? 272 : 288, VG = 320;  // bytes between groups of 32 values
  static constexpr int G = HD / 32;
  static constexpr int OFF_V = G * KG, OFF_KS = OFF_V + G * VG, OFF_VS = OFF_KS + 16 * 2 * G;
  static constexpr int STAGE = (OFF_VS + 16 * 2 * G + 15) / 16 * 16;
  static constexpr int RING = WARPS * STAGES * STAGE;
  static constexpr int osum(int nq) { return WARPS * nq * (HD + 4) * 4; }
  static constexpr int smem(int nq) { return RING > osum(nq) ? RING : osum(nq); }
};
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// 16 s and -24 s of two rows' scales (or of one row's, twice), for kv4_dequant8.
struct FewScale {
  uint32_t s16, m24;
};
__device__ __forceinline__ FewScale few_scale(uint32_t pair) {
  FewScale f;
  kv4_scale_pair(pair, f.s16, f.m24);
  return f;
}
__device__ __forceinline__ void few_dequant8(uint32_t w, const FewScale &f, uint32_t (&a)[4]) {
  kv4_dequant8(w, f.s16, f.m24, a);
}

// CTAs an SM.
constexpr int few_ctas(int nt) { return nt == 1 ? 2 : 1; }
// NT: tiles of 8 queries; SPL: planes of the queries and of P.
template <int HD, int NT, int SPL>
__global__ void __launch_bounds__(Few<HD>::THREADS, few_ctas(NT)) k_attn4_few(const __grid_constant__ A4Args A) {
  constexpr int W = Few<HD>::WARPS, NQ = 8 * NT, MT = HD / 16;
  constexpr int KW = HD / 32, VW = HD / 64;            // words of a key's codes a thread holds
  // the queries' fragments: in registers where they are few, else read from shared
  // memory (in the threads' order, 16 bytes each) with every group of keys
  constexpr bool QREG = NT == 1;
  __shared__ float wm[W][NQ], wl[W][NQ];
  __shared__ __align__(16) float qs[NQ];
  __shared__ __align__(16) uint4 qp[KW][NT][SPL][32];
  extern __shared__ __align__(16) uint8_t few_sm[];    // the warps' rings; then each warp's O, rows padded
  auto osum = [&](int w, int q) { return (float *)few_sm + (w * NQ + q) * (HD + 4); };
  using F = Few<HD>;
  constexpr int S = F::STAGES;
  const int rep = A.heads / A.kv, R = A.R, Q = rep * R;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int krow = (g >> 1) + 4 * (g & 1);             // this thread's keys of a group: krow and krow + 8
  uint8_t *ring = few_sm + warp * (S * F::STAGE);
  const uint32_t ring32 = smem_u32(ring);
  A4Piece<true> P;
  P.start(A);
  bool more = P.next(A);
  pdl_wait();
  for (; more; more = P.next(A)) {
    const int b = P.b, h = P.h;
    const A4Seq &Sq = A.seq[b];
    const int n = Sq.n, first = (int)(Sq.row0 % KV4_TILE);
    // the run's groups of 16 rows, counted from row0's tile on; group ng: the own rows'
    const int ng = n > 0 ? (int)(((int64_t)first + n + 15) / 16) : first / 16;
    const int s0 = first / 16 + 8 * P.r0, send = min(ng + (Sq.ok ? 1 : 0), first / 16 + 8 * P.r1);
    const int s1 = min(ng, send);
    int va, vb;
    a4_clear(A, Sq, va, vb);

    // the queries as f16 planes in shared memory, a warp a query: the row scaled by
    // the power of two that brings its largest value to [2^10, 2^11); thread (g, t)
    // of the fragments takes values HD/4 t .. of query 8 nt + g, 8 at a time
    __syncthreads();  // the piece before has left its queries and the memory of the rings
    for (int q = warp; q < NQ; q += W) {
      const int64_t at = (int64_t)b * A.q_seq + (int64_t)(q % R) * A.q_row + (int64_t)(h * rep + q / R) * HD + lane;
      float x[HD / 32];
      float amax = 0.f;
      if (q < Q) {
        a4_row<SPL, HD / 32, 32>(A, at, x);
      } else {
#pragma unroll
        for (int e = 0; e < HD / 32; ++e) x[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < HD / 32; ++e) amax = fmaxf(amax, fabsf(x[e]));
      float f0, f1;
      const float sc = a4_row_scale(warp_max(amax), A.scale, f0, f1);
      if (lane == 0) qs[q] = sc;
#pragma unroll
      for (int e = 0; e < HD / 32; ++e) {
        const float y = x[e] * f0 * f1;
        const __half hi = __float2half_rn(y);
        const int d = 32 * e + lane, i = d % (HD / 4) / 8, th = q % 8 * 4 + d / (HD / 4);
        ((__half *)&qp[i][q / 8][0][th])[d % 8] = hi;
        if (SPL == 2) ((__half *)&qp[i][q / 8][SPL - 1][th])[d % 8] = __float2half_rn(y - __half2float(hi));
      }
    }
    __syncthreads();
    uint4 qf[QREG ? KW : 1][QREG ? SPL : 1];
    float sl2[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      sl2[nt][0] = qs[8 * nt + 2 * t];
      sl2[nt][1] = qs[8 * nt + 2 * t + 1];
    }
    if constexpr (QREG) {
#pragma unroll
      for (int i = 0; i < KW; ++i)
#pragma unroll
        for (int p = 0; p < SPL; ++p) qf[i][p] = qp[i][0][p][lane];
    }

    // the copies of a lane: pieces lane, lane + 32, .. of a group's codes (16 keys a
    // group of values), and of its scales. A warp's next group is the same rows of
    // the next tile
    const int sw = s0 + warp;
    constexpr int PIECES = HD / 2, SP = HD / 16;         // 16-byte pieces of the codes, and of the scales
    const int64_t base = h * A.head_bytes + (Sq.row0 / KV4_TILE + (sw >> 3)) * kv4_tile_bytes(HD);
    const int row = (sw & 7) * 16, sl = lane < SP ? lane : lane - SP;
    const uint8_t *kp = Sq.k + base + kv4_code_off(row + (lane & 15), lane >> 4);
    const uint8_t *vp = Sq.v + base + kv4_code_off(row + (lane & 15), lane >> 4);
    const uint8_t *cp = (lane < SP ? Sq.k : Sq.v) + base + kv4_scale_off(HD, row, 0) + sl * 16;
    const uint32_t kd = ring32 + (lane >> 4) * F::KG + (lane & 15) * 16;
    const uint32_t vd = ring32 + F::OFF_V + (lane >> 4) * F::VG + (lane & 15) * 16;
    const uint32_t cd = ring32 + (lane < SP ? F::OFF_KS : F::OFF_VS) + sl * 16;
    auto fetch = [&](int slot) {
#pragma unroll
      for (int i = 0; i < PIECES / 32; ++i) {
        cp_async16(kd + slot * F::STAGE + i * 2 * F::KG, kp + kv4_code_off(0, 2 * i));
        cp_async16(vd + slot * F::STAGE + i * 2 * F::VG, vp + kv4_code_off(0, 2 * i));
      }
      if (lane < 2 * SP) cp_async16(cd + slot * F::STAGE, cp);
      kp += kv4_tile_bytes(HD);
      vp += kv4_tile_bytes(HD);
      cp += kv4_tile_bytes(HD);
    };

    float o[MT][NT][4], l[NT][2], negm[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][nt][e] = 0.f;
      l[nt][0] = l[nt][1] = 0.f;
      negm[nt][0] = negm[nt][1] = A4_NONE;               // no row seen yet
    }
    constexpr int KC = HD == 128 ? 1 : 2, VC = HD == 128 ? 2 : 4;  // threads that share a group of 32 values
    const uint32_t kr = ring32 + t / KC * F::KG + krow * 16 + t % KC * 8;
    const uint32_t ksr = ring32 + F::OFF_KS + (krow * F::G + t / KC) * 2;
    const uint32_t vr = ring32 + F::OFF_V + g / VC * F::VG + t * 16 + g % VC * (VW * 4);
    const uint32_t vsr = ring32 + F::OFF_VS + (t * F::G + g / VC) * 2;
    // 16 keys: rows lo .. of a range of nn; edge: some are not rows or not seen by all
    auto step = [&](int lo, int nn, bool edge, bool own, uint32_t off) {
      // this thread's codes and scales; rows outside the range get the scale 0, so that
      // their values are 0 whatever the cache holds there
      uint32_t kw[2][KW], ksc[2], vw[4][VW], vsc[4];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        if constexpr (HD == 128) {
          const uint4 w = lds128(kr + off + 128 * p);
          kw[p][0] = w.x, kw[p][1] = w.y, kw[p][2] = w.z, kw[p][3] = w.w;
        } else {
          const uint2 w = lds64(kr + off + 128 * p);
          kw[p][0] = w.x, kw[p][1] = w.y;
        }
        ksc[p] = lds16(ksr + off + 16 * F::G * p);
      }
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        if constexpr (HD == 128) {
          const uint2 w = lds64(vr + off + 64 * p);
          vw[p][0] = w.x, vw[p][1] = w.y;
        } else {
          vw[p][0] = lds32(vr + off + 64 * p);
        }
        vsc[p] = lds16(vsr + off + 8 * F::G * p);
      }
      if (edge) {
#pragma unroll
        for (int p = 0; p < 2; ++p)
          if ((unsigned)(lo + krow + 8 * p) >= (unsigned)nn) ksc[p] = 0;
#pragma unroll
        for (int p = 0; p < 4; ++p)
          if ((unsigned)(lo + t + 4 * p) >= (unsigned)nn) vsc[p] = 0;
        asm volatile("" : "+r"(ksc[0]));  // a branch, not selects in every group
      }
      // scores of 16 keys
      float c[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) c[nt][0] = c[nt][1] = c[nt][2] = c[nt][3] = 0.f;
      const FewScale f0 = few_scale(ksc[0] * 0x10001u), f1 = few_scale(ksc[1] * 0x10001u);
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        uint32_t x[4], y[4];
        few_dequant8(kw[0][i], f0, x);
        few_dequant8(kw[1][i], f1, y);
        const uint32_t a0[4] = {x[0], y[0], x[1], y[1]}, a1[4] = {x[2], y[2], x[3], y[3]};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int p = 0; p < SPL; ++p) {
            const uint4 w = QREG ? qf[QREG ? i : 0][QREG ? p : 0] : qp[i][nt][p][lane];
            mma16816(c[nt], a0, w.x, w.y);
            mma16816(c[nt], a1, w.z, w.w);
          }
      }
      // keys outside the range or unseen by a query: -inf
      if (edge) {
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          int rlo = 0, rhi = krow + 8 * e2 < R ? R - 1 : -1;
          if (!own) a4_seen(A, Sq, lo + krow + 8 * e2, rlo, rhi);
          if (rlo > 0 || rhi < R - 1) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int r = (8 * nt + 2 * t + e) % R;
                if (r < rlo || r > rhi) c[nt][2 * e2 + e] = -INFINITY;
              }
          }
        }
        asm volatile("" : "+f"(c[0][0]));  // a branch again
      }
      // against the reference (sl2 > 0 keeps -inf)
      float x[NT][4];
      float top = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[nt][e] = fmaf(c[nt][e], sl2[nt][e & 1], negm[nt][e & 1]);
          top = a4_max(top, x[nt][e]);
        }
      if (__any_sync(0xffffffffu, !(top <= A4_TAU))) {
        // new references: a column's largest score over the lanes that share t
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float y = a4_max(c[nt][e], c[nt][2 + e]) * sl2[nt][e];
#pragma unroll
            for (int f = 4; f < 32; f <<= 1) y = a4_max(y, __shfl_xor_sync(0xffffffffu, y, f));
            const float nm = negm[nt][e];
            const float nn = a4_ref(y);
            float al = 1.f;
            if (nm == A4_NONE) {
              if (y != -INFINITY) negm[nt][e] = nn;
            } else if (!(y + nm <= A4_TAU) && !(nn >= nm)) {  // (never back down)
              negm[nt][e] = nn;
              al = a4_ex2(nn - nm);
            }
            l[nt][e] *= al;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              o[i][nt][e] *= al;
              o[i][nt][2 + e] *= al;
            }
#pragma unroll
            for (int k = e; k < 4; k += 2) x[nt][k] = a4_capped(fmaf(c[nt][k], sl2[nt][e], negm[nt][e]));
          }
      }
      uint32_t pf[NT][SPL][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float p0 = a4_ex2(x[nt][2 * e]), p1 = a4_ex2(x[nt][2 * e + 1]);
          l[nt][0] += p0;
          l[nt][1] += p1;
          uint32_t hi, lo2;
          a4_pack<SPL>(p0, p1, hi, lo2);
          pf[nt][0][e] = movmatrix(hi);
          if (SPL == 2) pf[nt][SPL - 1][e] = movmatrix(lo2);
        }
      // O += V P: two keys' words joined, a pair is a value of both
      const FewScale v0 = few_scale(vsc[0] | vsc[1] << 16), v1 = few_scale(vsc[2] | vsc[3] << 16);
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        uint32_t ev[2][4], od[2][4];
        few_dequant8(__byte_perm(vw[0][i], vw[1][i], 0x5410), v0, ev[0]);
        few_dequant8(__byte_perm(vw[0][i], vw[1][i], 0x7632), v0, od[0]);
        few_dequant8(__byte_perm(vw[2][i], vw[3][i], 0x5410), v1, ev[1]);
        few_dequant8(__byte_perm(vw[2][i], vw[3][i], 0x7632), v1, od[1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t a[4] = {ev[0][e], od[0][e], ev[1][e], od[1][e]};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int p = 0; p < SPL; ++p) mma16816(o[4 * i + e][nt], a, pf[nt][p][0], pf[nt][p][1]);
        }
      }
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
      if (sw + i * W < s1) fetch(i);
      cp_async_commit();
    }
    int slot = 0;
    for (int s = sw; s < s1; s += W) {
      cp_async_wait<S - 2>();
      __syncwarp();  // the group has landed for every lane; the one before has been read
      if (s + (S - 1) * W < s1) fetch((slot + S - 1) % S);
      cp_async_commit();
      const int lo = s * 16 - first;
      step(lo, n, lo < va || vb - lo < 16, false, slot * F::STAGE);  // (lo + 16 can pass 2^31)
      slot = (slot + 1) % S;
    }
    cp_async_wait<0>();
    if (send > s1 && warp == ((s1 - s0) & (W - 1))) {
      // the block's own rows: every query sees them
      __syncwarp();
      const int64_t tile = (int64_t)h * kv4_tile_bytes(HD);
      kp = Sq.ok + tile + kv4_code_off(lane & 15, lane >> 4);
      vp = Sq.ov + tile + kv4_code_off(lane & 15, lane >> 4);
      cp = (lane < SP ? Sq.ok : Sq.ov) + tile + kv4_scale_off(HD, 0, 0) + sl * 16;
      fetch(0);
      cp_async_commit();
      cp_async_wait<0>();
      __syncwarp();
      step(0, R, true, true, 0);
    }
    // the warps' results: sums over the keys, then references and O through shared memory
    __syncthreads();  // every warp has left its ring
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[nt][e];
#pragma unroll
        for (int f = 4; f < 32; f <<= 1) x += __shfl_xor_sync(0xffffffffu, x, f);
        const int q = 8 * nt + 2 * t + e;
        if (g == 0) {
          wm[warp][q] = negm[nt][e] == A4_NONE ? -INFINITY : -negm[nt][e];
          wl[warp][q] = x;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)  // tile i's rows: values HD/8 g + 2 i and + 1
          *(float2 *)(osum(warp, q) + HD / 8 * g + 2 * i) = make_float2(o[i][nt][e], o[i][nt][2 + e]);
      }
    if (P.rnd >= P.rend) pdl_trigger();
    __syncthreads();
    constexpr int V4 = HD / 4;
    const bool whole = P.r0 == 0 && P.r1 == P.nr && !A.always_part;
    const int64_t slot0 = P.slot(A);
    for (int id = threadIdx.x; id < Q * V4; id += Few<HD>::THREADS) {
      const int q = id / V4, d = id % V4 * 4;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < W; ++w) M = a4_max(M, wm[w][q]);
      float L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      const bool seen = M != -INFINITY;
      if (seen) {
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float m = wm[w][q], f = m != -INFINITY ? a4_ex2(m - M) : 0.f;
          const float4 x = *(const float4 *)(osum(w, q) + d);
          L = fmaf(wl[w][q], f, L);
          acc.x = fmaf(x.x, f, acc.x);
          acc.y = fmaf(x.y, f, acc.y);
          acc.z = fmaf(x.z, f, acc.z);
          acc.w = fmaf(x.w, f, acc.w);
        }
      }
      if (!whole) {
        float *out = A.part + (slot0 * Q + q) * (HD + 4);
        const int left = P.left();
        if (P.r0 > P.begin(A)) {
          // the runs before, in the slot (their statistics in two places in turn, a piece's
          // last ones where the merge reads them)
          const float Mb = out[HD + 2 - left % 2 * 2], Lb = out[HD + 3 - left % 2 * 2], Mi = M;
          const float4 x = *(const float4 *)(out + d);
          M = a4_max(M, Mb);
          const float fi = seen ? a4_ex2(Mi - M) : 0.f, fb = Mb != -INFINITY ? a4_ex2(Mb - M) : 0.f;
          L = fmaf(Lb, fb, L * fi);
          acc.x = fmaf(x.x, fb, acc.x * fi);
          acc.y = fmaf(x.y, fb, acc.y * fi);
          acc.z = fmaf(x.z, fb, acc.z * fi);
          acc.w = fmaf(x.w, fb, acc.w * fi);
        }
        *(float4 *)(out + d) = acc;
        if (d == 0) {
          out[HD + left % 2 * 2] = M;
          out[HD + 1 + left % 2 * 2] = L;
        }
      } else {
        const int64_t row = ((int64_t)b * R + q % R) * A.heads + h * rep + q / R;
        const float inv = seen ? 1.f / L : 0.f;
        st_elem(A.y, row * HD + d, A.dtype, acc.x * inv);
        st_elem(A.y, row * HD + d + 1, A.dtype, acc.y * inv);
        st_elem(A.y, row * HD + d + 2, A.dtype, acc.z * inv);
        st_elem(A.y, row * HD + d + 3, A.dtype, acc.w * inv);
        if (d == 0 && A.lse) A.lse[row] = seen ? (log2f(L) + M) * 0.6931471805599453f : -INFINITY;
      }
    }
  }
}

// y of a query row from its pair's partials (m in base 2), one warp a row; a row
// that no piece saw anything of is 0 (lse -inf). A pair that one CTA took whole in one run
// is written already. PACK: the row as hi/lo planes into the output projection's
// token tiles; the blocks past `work` clear that GEMM's outputs when it splits.
// NB: twice as many partials are asked for before the first is needed. 8 while the
// launch is one wave (three CTAs an SM then): a divided pair of a single sequence has
// some 20 (one block over 32,768 rows: 39.7 us, with NB 2 43.1). 2 for more rows, whose
// pairs have two or three (32 blocks: 135 us, with NB 8 139).
template <int HD, bool FEW, bool PACK, int NB>
__global__ void __launch_bounds__(128) k_attn4_merge(const __grid_constant__ A4Args A, int work, PackDst P, ZeroSet Z) {
  constexpr int DL = HD / 32;
  pdl_wait();
  if (PACK) pdl_trigger();  // the GEMM this feeds may fetch its weights meanwhile
  if (PACK && (int)blockIdx.x >= work) {
    if (blockIdx.y == 0) zero_set_clear(Z, blockIdx.x - work, gridDim.x - work);
    return;
  }
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int rep = A.heads / A.kv, Q = rep * A.R;
  const int row = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= A.kv * Q) return;
  const int g = row / Q, qi = row - g * Q;
  const int64_t stride = (int64_t)Q * (HD + 4);
  const int nr = a4_rounds<FEW>(A.seq[b]);
  const int64_t t0 = A.round0[b] + (int64_t)g * nr;
  const int64_t i0 = a4_cta(A, t0), i1 = a4_cta(A, t0 + nr - 1);
  if (i0 == i1 && nr <= A.run && !A.always_part) return;
  const int ns = (int)(i1 - i0 + 1);
  const float *base = A.part + ((i0 + (int64_t)b * A.kv + g) * Q + qi) * (HD + 4);
  float v[2][NB][DL];
  auto load = [&](int s0, float(&x)[NB][DL]) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const float *ps = base + (s0 + i) * stride + DL * lane;
      if constexpr (DL == 4) {
        const float4 o = s0 + i < ns ? *(const float4 *)ps : make_float4(0.f, 0.f, 0.f, 0.f);
        x[i][0] = o.x, x[i][1] = o.y, x[i][2] = o.z, x[i][3] = o.w;
      } else {
        const float2 o = s0 + i < ns ? *(const float2 *)ps : make_float2(0.f, 0.f);
        x[i][0] = o.x, x[i][1] = o.y;
      }
    }
  };
  const float m0 = lane < ns ? base[lane * stride + HD] : -INFINITY;
  const float l0 = lane < ns ? base[lane * stride + HD + 1] : 0.f;
  load(0, v[0]);
  load(NB, v[1]);
  float M = m0;
  for (int s = lane + 32; s < ns; s += 32) M = a4_max(M, base[s * stride + HD]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = a4_max(M, __shfl_xor_sync(0xffffffffu, M, o));
  float acc[DL], L = 0.f;
#pragma unroll
  for (int e = 0; e < DL; ++e) acc[e] = 0.f;
  if (M != -INFINITY) {
    float w = 0.f;
    auto add = [&](int s, const float(&x)[NB][DL]) {
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const float ws = __shfl_sync(0xffffffffu, w, (s + i) & 31);
#pragma unroll
        for (int e = 0; e < DL; ++e) acc[e] = fmaf(x[i][e], ws, acc[e]);
      }
    };
    for (int s = 0; s < ns; s += 2 * NB) {
      if ((s & 31) == 0) {  // the weights of the next 32 partials, a lane each
        float m = m0, ls = l0;
        if (s > 0) {
          m = s + lane < ns ? base[(s + lane) * stride + HD] : -INFINITY;
          ls = s + lane < ns ? base[(s + lane) * stride + HD + 1] : 0.f;
        }
        w = m != -INFINITY ? exp2f(m - M) : 0.f;
        L += ls * w;
      }
      add(s, v[0]);
      load(s + 2 * NB, v[0]);
      add(s + NB, v[1]);
      load(s + 3 * NB, v[1]);
    }
    L = warp_sum(L);
  }
  const float inv = M != -INFINITY ? 1.f / L : 0.f;
#pragma unroll
  for (int e = 0; e < DL; ++e) acc[e] *= inv;
  const int trow = b * A.R + qi % A.R, col = (g * rep + qi / A.R) * HD;
  if constexpr (PACK) {
    // 8 consecutive columns a store: lanes 8/DL apart hand theirs to the first
    constexpr int LPC = 8 / DL;
    float x8[8];
#pragma unroll
    for (int j = 0; j < LPC; ++j)
#pragma unroll
      for (int e = 0; e < DL; ++e) x8[j * DL + e] = __shfl_sync(0xffffffffu, acc[e], (lane / LPC) * LPC + j);
    if (lane % LPC == 0) pack_store8(P, trow, col + DL * lane, x8);
  } else {
    const int64_t out = (int64_t)trow * A.heads * HD + col;
#pragma unroll
    for (int e = 0; e < DL; ++e) st_elem(A.y, out + DL * lane + e, A.dtype, acc[e]);
    if (A.lse && lane == 0)
      A.lse[out / HD] = M != -INFINITY ? (log2f(L) + M) * 0.6931471805599453f : -INFINITY;
  }
}

template <int HD, int NQ, int SPL>
static cudaError_t launch_a4(const A4Args &A, cudaStream_t st) {
  using C = A4<HD, NQ, SPL>;
  static PerDevice configured;
  if (cudaError_t e = smem_limit(k_attn4<HD, NQ, SPL>, (int)C::BYTES, configured)) return e;
  return launch_pdl(k_attn4<HD, NQ, SPL>, dim3(A.ctas), dim3(C::THREADS), C::BYTES, st, 1, A);
}
template <int HD>
static cudaError_t launch_a4_hd(const A4Args &A, cudaStream_t st) {
  if (A.dtype != DFLASH_F32) return launch_a4<HD, 64, 1>(A, st);
  if constexpr (HD == 128)
    if (A.heads / A.kv * A.R <= 32) return launch_a4<HD, 32, 2>(A, st);
  return launch_a4<HD, 64, 2>(A, st);
}
template <int HD, int NT, int SPL>
static cudaError_t launch_few(const A4Args &A, cudaStream_t st) {
  const int smem = Few<HD>::smem(8 * NT);
  static PerDevice configured;
  if (cudaError_t e = smem_limit(k_attn4_few<HD, NT, SPL>, smem, configured)) return e;
  return launch_pdl(k_attn4_few<HD, NT, SPL>, dim3(A.ctas), dim3(Few<HD>::THREADS), smem, st, 1, A);
}
template <int HD, int SPL>
static cudaError_t launch_few_hd(const A4Args &A, cudaStream_t st) {
  const int Q = A.heads / A.kv * A.R;
  if (Q <= 8) return launch_few<HD, 1, SPL>(A, st);
  if constexpr (HD == 128 && SPL == 2) {
    return launch_few<HD, 2, SPL>(A, st);
  } else {
    return Q <= 16 ? launch_few<HD, 2, SPL>(A, st) : launch_few<HD, 4, SPL>(A, st);
  }
}
// Whether k_attn4_few takes Q query rows a KV head: up to 16, and up to 32 unless
// they are f32 rows of 128 values. Measured on 16 x 8,192 rows of 8 KV heads (us,
// few against k_attn4): 16 f32 rows of 128 66 : 80, 32 of them 105 : 80; 32 bf16
// rows 72 : 86; 32 f32 rows of 64 63 : 82. (Above 32 its O does not fit a thread.)
static bool takes_few(int Q, int hd, int dtype) { return Q <= 16 || (Q <= 32 && (dtype != DFLASH_F32 || hd == 64)); }

// A CTA takes at least this many rounds, or a whole pair: a merge and a piece's
// start and end cost about as much as these. More CTAs than slots are not started.
constexpr int A4_MIN_ROUNDS = 4;
// Share the rounds out over at most `slots` CTAs; true if no pair is divided.
template <bool FEW>
static bool share_out(A4Args &A, int batch, int hd, int64_t slots) {
  A.batch = batch;
  // a round is a step of each warp of k_attn4_few, and 8 steps of k_attn4, whose chunks take
  // four accumulators in turn where there is room (128 steps of each in 64 chunks)
  A.run = FEW ? A4_STEPS : A.dtype == DFLASH_F32 && (hd == 64 || A.heads / A.kv * A.R > 32) ? A4_STEPS / 8 : A4_STEPS / 4;
  int64_t most = 1;
  for (int i = 0; i < batch; ++i) {
    const int nr = a4_rounds<FEW>(A.seq[i]);
    A.round0[i + 1] = A.round0[i] + (int64_t)nr * A.kv;
    A.run0[i + 1] = A.run0[i] + (int64_t)a4_runs(A, nr) * A.kv;
    most = std::max<int64_t>(most, nr);
  }
  const int64_t T = A.round0[batch], pairs = (int64_t)batch * A.kv;
  bool whole = most <= A4_MIN_ROUNDS;  // every pair by one CTA: no merge
  for (int i = 0; i < batch; ++i) whole = whole && A.round0[i + 1] - A.round0[i] == A.round0[1];
  A.ctas = (int)(whole ? pairs : std::min(slots, std::max<int64_t>(1, T / A4_MIN_ROUNDS)));
  A.share = T / A.ctas;
  A.more = (int)(T % A.ctas);
  return whole;
}
template <bool FEW, bool PACK>
static cudaError_t launch_merge4(const A4Args &A, int hd, int num_sms, int zero_blocks, const PackDst &pack,
                                 const ZeroSet &zero, cudaStream_t st) {
  const int work = (A.heads * A.R + 3) / 4;
  const dim3 grid((unsigned)(work + zero_blocks), A.batch);
  const bool wave = (int64_t)work * A.batch <= 3 * num_sms;
  auto merge = hd == 128 ? (wave ? k_attn4_merge<128, FEW, PACK, 8> : k_attn4_merge<128, FEW, PACK, 2>)
                         : (wave ? k_attn4_merge<64, FEW, PACK, 8> : k_attn4_merge<64, FEW, PACK, 2>);
  return launch_pdl(merge, grid, dim3(128), 0, st, 1, A, work, pack, zero);
}
// The kernel for the rows of A: true in `whole` if it divided no pair (no merge).
static cudaError_t launch_rows(A4Args &A, int batch, int hd, int num_sms, bool &few, bool &whole, cudaStream_t st) {
  num_sms = std::max(1, std::min(num_sms, 512));
  const int Q = A.heads / A.kv * A.R;
  few = takes_few(Q, hd, A.dtype);
  if (few) {
    whole = share_out<true>(A, batch, hd, (int64_t)few_ctas(Q <= 8 ? 1 : Q <= 16 ? 2 : 4) * num_sms);
    if (A.dtype == DFLASH_F32) return hd == 128 ? launch_few_hd<128, 2>(A, st) : launch_few_hd<64, 2>(A, st);
    return hd == 128 ? launch_few_hd<128, 1>(A, st) : launch_few_hd<64, 1>(A, st);
  }
  whole = share_out<false>(A, batch, hd, num_sms);
  return hd == 128 ? launch_a4_hd<128>(A, st) : launch_a4_hd<64>(A, st);
}
// The rows of A, and the merge of divided pairs (and of those of several runs).
static cudaError_t attend(A4Args &A, int batch, int hd, int num_sms, cudaStream_t st) {
  bool few, whole;
  const cudaError_t e = launch_rows(A, batch, hd, num_sms, few, whole, st);
  if (e != cudaSuccess || whole) return e;
  return few ? launch_merge4<true, false>(A, hd, num_sms, 0, PackDst{}, ZeroSet{}, st)
             : launch_merge4<false, false>(A, hd, num_sms, 0, PackDst{}, ZeroSet{}, st);
}

// The block pass's attention.
cudaError_t attention4(const float *q, const uint8_t *own_k, const uint8_t *own_v, const Attn4Seq *seqs, int batch,
                       int heads, int kv, int hd, int R, int window, float scale, float *part, float *y, int num_sms,
                       const PackDst *pack, const ZeroSet *zero, cudaStream_t st) {
  if (batch < 1 || batch > MAX_BATCH || heads / kv * R > 64 || (hd != 64 && hd != 128)) return cudaErrorInvalidValue;
  A4Args A{};
  const int64_t own = (int64_t)kv * kv4_tile_bytes(hd);
  for (int i = 0; i < batch; ++i)
    A.seq[i] = A4Seq{seqs[i].k, seqs[i].v, own_k + i * own, own_v + i * own, seqs[i].row0, seqs[i].n, seqs[i].anchor};
  A.head_bytes = seqs[0].head_bytes;
  A.q = q;
  A.q_row = (int64_t)heads * hd;
  A.q_seq = A.q_row * R;
  A.y = y;
  A.part = part;
  A.dtype = DFLASH_F32;
  A.heads = heads, A.kv = kv, A.R = R, A.window = window;
  A.always_part = pack != nullptr;
  A.scale = scale;
  if (!pack) return attend(A, batch, hd, num_sms, st);
  bool few, whole;
  if (cudaError_t e = launch_rows(A, batch, hd, num_sms, few, whole, st)) return e;
  int64_t most = 0;
  for (int j = 0; j < zero->count; ++j) most = std::max<int64_t>(most, zero->n[j]);
  const int zb = zero->count ? (int)std::min<int64_t>((most + 511) / 512, 256) : 0;
  return few ? launch_merge4<true, true>(A, hd, num_sms, zb, *pack, *zero, st)
             : launch_merge4<false, true>(A, hd, num_sms, zb, *pack, *zero, st);
}

// This file's device error word.
cudaError_t kv4_read_error(unsigned *out, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_dev_error, sizeof(unsigned));
  if (e == cudaSuccess && reset) {
    const unsigned zero = 0;
    e = cudaMemcpyToSymbol(g_dev_error, &zero, sizeof(unsigned));
  }
  return e;
}

namespace {
bool dtype_ok(int d) { return d == DFLASH_F32 || d == DFLASH_F16 || d == DFLASH_BF16; }
int dtype_size(int d) { return d == DFLASH_F32 ? 4 : 2; }
int bad_arg(const char *who, const char *what) { return dflash_fail(DFLASH_E_ARG, std::string(who) + ": " + what); }

// The checks that the three calls share: sizes, and the caches with their rows
// [at, at + n) (n < 0: no rows to check).
int check_caches(const char *who, int batch, int kv, int hd, int64_t rows, void *const *ck, void *const *cv) {
  if (batch < 1 || batch > MAX_BATCH) return bad_arg(who, "batch must be 1..64");
  if (hd != 64 && hd != 128) return bad_arg(who, "head_dim must be 64 or 128");
  if (kv < 1 || kv > 1024) return bad_arg(who, "kv_heads must be 1..1024");
  if (rows < 1 || rows > INT32_MAX) return bad_arg(who, "rows must be 1..2^31-1");
  if (!ck || !cv) return bad_arg(who, "null caches");
  for (int i = 0; i < batch; ++i)
    if (!ck[i] || !cv[i] || ((uintptr_t)ck[i] & 15) || ((uintptr_t)cv[i] & 15))
      return bad_arg(who, "a null or misaligned cache");
  return DFLASH_OK;
}
int64_t head_bytes(int hd, int64_t rows) { return (rows + KV4_TILE - 1) / KV4_TILE * kv4_tile_bytes(hd); }

template <int HD, typename T>
cudaError_t launch_write_t(const Kv4Rows &X, const Kv4Seqs &S, int batch, int n, int kv, cudaStream_t st) {
  // four rows a thread from 8 rows a sequence on
  const int rw = n >= 8 ? 4 : 1;
  const int64_t threads = (int64_t)((n + rw - 1) / rw) * kv * (HD / 8);
  const dim3 grid((unsigned)((threads + 255) / 256), 2 * batch);
  return launch_pdl(rw == 4 ? k_kv4_write<HD, T, 4> : k_kv4_write<HD, T, 1>, grid, dim3(256), 0, st, 1, X, S, n, kv);
}
template <int HD>
cudaError_t launch_write(const Kv4Rows &X, const Kv4Seqs &S, int batch, int n, int kv, int dtype, cudaStream_t st) {
  if (dtype == DFLASH_F32) return launch_write_t<HD, float>(X, S, batch, n, kv, st);
  if (dtype == DFLASH_F16) return launch_write_t<HD, __half>(X, S, batch, n, kv, st);
  return launch_write_t<HD, __nv_bfloat16>(X, S, batch, n, kv, st);
}
}  // namespace

}  // namespace dfl

extern "C" {

size_t dflash_kv4_cache_bytes(int32_t kv_heads, int32_t head_dim, int64_t rows) {
  if (kv_heads < 1 || kv_heads > 1024 || (head_dim != 64 && head_dim != 128) || rows < 1 || rows > INT32_MAX) return 0;
  return (size_t)kv_heads * dfl::head_bytes(head_dim, rows);
}

int dflash_kv4_write(int32_t batch, int32_t kv_heads, int32_t head_dim, int64_t rows, void *const *ctx_k,
                     void *const *ctx_v, const int64_t *at, int32_t n, const void *k, int64_t k_seq_stride,
                     int64_t k_row_stride, const void *v, int64_t v_seq_stride, int64_t v_row_stride, int32_t dtype,
                     void *stream) {
  using namespace dfl;
  const char *who = "kv4_write";
  if (int e = check_caches(who, batch, kv_heads, head_dim, rows, ctx_k, ctx_v)) return e;
  if (!dtype_ok(dtype)) return bad_arg(who, "dtype must be DFLASH_F32, DFLASH_F16 or DFLASH_BF16");
  if (!at || (n > 0 && (!k || !v))) return bad_arg(who, "null pointer");
  const uintptr_t sz = dtype_size(dtype);
  if ((uintptr_t)k % sz || (uintptr_t)v % sz) return bad_arg(who, "misaligned rows");
  if (n < 0) return bad_arg(who, "a negative row count");
  const int64_t width = (int64_t)kv_heads * head_dim;
  if (k_seq_stride < 0 || v_seq_stride < 0 || k_row_stride < width || v_row_stride < width)
    return bad_arg(who, "a row stride below kv_heads * head_dim, or a negative stride");
  for (int i = 0; i < batch; ++i) {
    if (at[i] < 0) return bad_arg(who, "a negative cache row");
    if (at[i] > rows - n) return dflash_fail(DFLASH_E_CAPACITY, "kv4_write: rows past the cache");
  }
  // no cache row is written twice in a call: caches are apart, or one and the same
  const int64_t bytes = (int64_t)kv_heads * head_bytes(head_dim, rows);
  auto apart = [&](const void *a, const void *b) { return (uintptr_t)a + bytes <= (uintptr_t)b || (uintptr_t)b + bytes <= (uintptr_t)a; };
  for (int i = 0; i < batch; ++i)
    for (int j = 0; j < batch; ++j) {
      if (!apart(ctx_k[i], ctx_v[j])) return bad_arg(who, "a K and a V cache in one memory");
      if (j < i && !apart(ctx_k[i], ctx_k[j]) && ctx_k[i] != ctx_k[j]) return bad_arg(who, "two K caches that overlap");
      if (j < i && !apart(ctx_v[i], ctx_v[j]) && ctx_v[i] != ctx_v[j]) return bad_arg(who, "two V caches that overlap");
      if (j < i && (ctx_k[i] == ctx_k[j] || ctx_v[i] == ctx_v[j]) && at[i] < at[j] + n && at[j] < at[i] + n)
        return bad_arg(who, "two sequences write the same rows of one cache");
    }
  if (n == 0) return DFLASH_OK;
  Kv4Rows X{};
  X.p[0] = k, X.p[1] = v;
  X.seq_stride[0] = k_seq_stride, X.seq_stride[1] = v_seq_stride;
  X.row_stride[0] = k_row_stride, X.row_stride[1] = v_row_stride;
  for (int i = 0; i < 2; ++i)
    X.vec[i] = ((uintptr_t)X.p[i] | (uintptr_t)(X.seq_stride[i] * sz) | (uintptr_t)(X.row_stride[i] * sz)) % 16 == 0;
  Kv4Seqs S{};
  for (int i = 0; i < batch; ++i) {
    S.k[i] = (uint8_t *)ctx_k[i];
    S.v[i] = (uint8_t *)ctx_v[i];
    S.at[i] = at[i];
  }
  S.head_bytes = head_bytes(head_dim, rows);
  const cudaError_t e = head_dim == 128 ? launch_write<128>(X, S, batch, n, kv_heads, dtype, (cudaStream_t)stream)
                                        : launch_write<64>(X, S, batch, n, kv_heads, dtype, (cudaStream_t)stream);
  if (e != cudaSuccess) return dflash_fail(DFLASH_E_CUDA, std::string("kv4_write: ") + cudaGetErrorString(e));
  return DFLASH_OK;
}

int dflash_kv4_read(int32_t batch, int32_t kv_heads, int32_t head_dim, int64_t rows, void *const *ctx_k,
                    void *const *ctx_v, const int64_t *at, int32_t n, float *k, float *v, void *stream) {
  using namespace dfl;
  const char *who = "kv4_read";
  if (int e = check_caches(who, batch, kv_heads, head_dim, rows, ctx_k, ctx_v)) return e;
  if (!at || (n > 0 && (!k || !v))) return bad_arg(who, "null pointer");
  if (((uintptr_t)k & 15) || ((uintptr_t)v & 15)) return bad_arg(who, "misaligned output");
  if (n < 0) return bad_arg(who, "a negative row count");
  for (int i = 0; i < batch; ++i) {
    if (at[i] < 0) return bad_arg(who, "a negative cache row");
    if (at[i] > rows - n) return dflash_fail(DFLASH_E_CAPACITY, "kv4_read: rows past the cache");
  }
  if (n == 0) return DFLASH_OK;
  Kv4Seqs S{};
  for (int i = 0; i < batch; ++i) {
    S.k[i] = (uint8_t *)ctx_k[i];
    S.v[i] = (uint8_t *)ctx_v[i];
    S.at[i] = at[i];
  }
  S.head_bytes = head_bytes(head_dim, rows);
  const int64_t threads = ((int64_t)n + 3) / 4 * kv_heads * (head_dim / 8);
  const dim3 grid((unsigned)((threads + 255) / 256), 2 * batch);
  const cudaError_t e = head_dim == 128
                            ? launch_pdl(k_kv4_read<128>, grid, dim3(256), 0, (cudaStream_t)stream, 1, S, n, kv_heads, k, v)
                            : launch_pdl(k_kv4_read<64>, grid, dim3(256), 0, (cudaStream_t)stream, 1, S, n, kv_heads, k, v);
  if (e != cudaSuccess) return dflash_fail(DFLASH_E_CUDA, std::string("kv4_read: ") + cudaGetErrorString(e));
  return DFLASH_OK;
}

size_t dflash_kv4_attention_workspace_bytes(int32_t batch, int32_t q_rows, int32_t heads, int32_t kv_heads,
                                            int32_t head_dim) {
  if (batch < 1 || batch > dfl::MAX_BATCH || q_rows < 1 || kv_heads < 1 || kv_heads > 1024 || heads < 1 ||
      heads % kv_heads || (head_dim != 64 && head_dim != 128) || (int64_t)heads / kv_heads * q_rows > 64)
    return 0;
  // a partial per piece: at most CTAs (1,024, share_out) plus pairs of them
  return ((size_t)1024 + 2 * (size_t)batch * kv_heads) * (heads / kv_heads * q_rows) * (head_dim + 4) * sizeof(float);
}

int dflash_kv4_attention(int32_t batch, int32_t q_rows, int32_t heads, int32_t kv_heads, int32_t head_dim,
                         int64_t rows, void *const *ctx_k, void *const *ctx_v, const int64_t *lo, const int64_t *hi,
                         const int64_t *anchor, int32_t window, int32_t causal, float scale, const void *q,
                         int64_t q_seq_stride, int64_t q_row_stride, int32_t dtype, void *y, float *lse,
                         void *workspace, size_t workspace_bytes, void *stream) {
  using namespace dfl;
  const char *who = "kv4_attention";
  if (int e = check_caches(who, batch, kv_heads, head_dim, rows, ctx_k, ctx_v)) return e;
  if (!dtype_ok(dtype)) return bad_arg(who, "dtype must be DFLASH_F32, DFLASH_F16 or DFLASH_BF16");
  if (!lo || !hi || !anchor || !q || !y) return bad_arg(who, "null pointer");
  const size_t need = dflash_kv4_attention_workspace_bytes(batch, q_rows, heads, kv_heads, head_dim);
  if (need == 0)
    return bad_arg(who, "heads must be a multiple of kv_heads and heads / kv_heads * q_rows 1..64");
  const uintptr_t sz = dtype_size(dtype);
  if ((uintptr_t)q % sz || (uintptr_t)y % sz || ((uintptr_t)lse & 3)) return bad_arg(who, "misaligned q, y or lse");
  if (q_seq_stride < 0 || q_row_stride < (int64_t)heads * head_dim)
    return bad_arg(who, "a q row stride below heads * head_dim, or a negative stride");
  if (window < 0) return bad_arg(who, "a negative window");
  if (!(scale > 0.f) || !(scale < INFINITY)) return bad_arg(who, "scale must be positive and finite");
  for (int i = 0; i < batch; ++i) {
    if (lo[i] < 0 || hi[i] < lo[i]) return bad_arg(who, "a range with lo < 0 or hi < lo");
    if (anchor[i] < 0 || anchor[i] > INT32_MAX) return bad_arg(who, "anchor must be 0..2^31-1");
    if (hi[i] > rows) return dflash_fail(DFLASH_E_CAPACITY, "kv4_attention: rows past the cache");
  }
  if (!workspace || ((uintptr_t)workspace & 15)) return bad_arg(who, "null or misaligned workspace");
  if (workspace_bytes < need)
    return dflash_fail(DFLASH_E_CAPACITY, "kv4_attention: workspace smaller than dflash_kv4_attention_workspace_bytes");
  A4Args A{};
  for (int i = 0; i < batch; ++i) {
    // the rows that some query sees: from the first query's window on, to the last query's own row
    const int64_t to = causal ? std::min(hi[i], anchor[i] + q_rows) : hi[i];
    const int64_t from = window ? std::max(lo[i], anchor[i] + 1 - window) : lo[i];
    A.seq[i] = A4Seq{(const uint8_t *)ctx_k[i], (const uint8_t *)ctx_v[i], nullptr, nullptr, from,
                     (int)std::max<int64_t>(to - from, 0), anchor[i] - from};
  }
  A.head_bytes = head_bytes(head_dim, rows);
  A.q = q;
  A.q_seq = q_seq_stride, A.q_row = q_row_stride;
  A.y = y, A.lse = lse;
  A.dtype = dtype;
  A.heads = heads, A.kv = kv_heads, A.R = q_rows, A.window = window, A.causal = causal != 0;
  A.scale = scale;
  A.part = (float *)workspace;
  const cudaError_t e = attend(A, batch, head_dim, device_sms(), (cudaStream_t)stream);
  if (e != cudaSuccess) return dflash_fail(DFLASH_E_CUDA, std::string("kv4_attention: ") + cudaGetErrorString(e));
  return DFLASH_OK;
}

}  // extern "C"
