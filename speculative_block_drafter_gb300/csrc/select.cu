// The selector (cortiq-engine src/cortiq_engine/dflash.rs, `Drafter::select_with`
// and `top_k`): per draft row, the `top` largest logits (larger first, the lower
// index first among equals), then the candidates re-scored in order against the
// token chosen before: score = logit + (P[prev] * hp) . C[cand], the first
// strictly greater score winning, the chain starting at the anchor token.
//
// Stage 1 (chunks x rows CTAs): the largest key (value, then lower index) of
// each chunk of 2048 logits.
// Stage 2 (chunks x rows CTAs): tau = the top-th largest of the row's chunk
// maxima. The top chunk maxima are `top` distinct logits of the row, so the
// row's top-th largest key is at least tau, and every key >= tau is a
// candidate: the chunks append theirs to the row's list (typically a few
// dozen entries). The chunks that hold one are dealt out to the row's warps by
// quarters (with a chunk a warp, where they came, stage 2 took 37 us and not 20
// on 480 rows of 151,936).
// Stage 3 (one CTA per row): the list ranked among itself gives the row's top
// `top` in order (a list past its capacity, from many equal logits, falls back
// to `top` exact passes over the row); the CTA also ranks the previous row's
// list and computes every score the chain can ask of the row (row j's
// predecessors are the anchor for j = 0, else row j-1's candidates).
// Stage 4 (one CTA per sequence): the chain itself, over the tables copied
// into shared memory.
#include <mutex>
#include <string>

#include "common.cuh"
#include "dflash.h"
#include "fixed.cuh"
#include "kernels.h"

namespace dfl {

constexpr int SEL_THREADS = 256;
constexpr int SEL_CHUNK = SELECT_CHUNK;            // logits per chunk of stage 1
static_assert(SEL_CHUNK % 1024 == 0, "a warp takes a quarter chunk in vectors of 8");
constexpr int ROW_THREADS = 512;
constexpr int CAND_CAP = 1024;                     // candidates (and chunk maxima) a row CTA holds
constexpr int MAX_CHUNKS = CAND_CAP;               // width <= 2 M
constexpr int TOP_MAX = 32;
constexpr int RANK_MAX = 256;
constexpr int CHAIN_THREADS = 512;
constexpr int KMAX = 15;

static inline int sel_chunks(int width) { return (width + SEL_CHUNK - 1) / SEL_CHUNK; }

// Scratch of one call, per row: the chunk maxima (u64), the candidate count and
// list (u64, CAND_CAP), the row's top (u32) and its score table (f32 [top][top]).
static size_t row_scratch(int width, int top) {
  return (size_t)sel_chunks(width) * 8 + 8 + (size_t)CAND_CAP * 8 + (size_t)top * 4 + (size_t)top * top * 4;
}
size_t select_scratch_bytes(int max_rows, int width, int top) { return (size_t)max_rows * row_scratch(width, top) + 256; }


// Eight logits of a row from `idx` on, as two vectors where the row's start allows it
// (0 for those past the row: the caller looks at the index before it makes a key).
__device__ __forceinline__ void load_logits8(const float *__restrict__ lr, int idx, int width, float (&x)[8]) {
  if (idx + 8 <= width && ((uintptr_t)(lr + idx) & 15) == 0) {
    const float4 a = __ldg((const float4 *)(lr + idx)), b = __ldg((const float4 *)(lr + idx) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = idx + i < width ? __ldg(lr + idx + i) : 0.f;
  }
}
// The largest key of a chunk, by one warp. The comparison is of the values' ordered
// bits; the index joins the thread's best only at the end (its own are ascending,
// so the first of equal values is kept).
__device__ __forceinline__ unsigned long long chunk_best(const float *__restrict__ lr, int chunk, int width) {
  const int lane = threadIdx.x & 31;
  uint32_t bv = 0u, bi = 0u;
  bool any = false;
#pragma unroll
  for (int i = 0; i < SEL_CHUNK / 256; ++i) {
    const int idx = chunk * SEL_CHUNK + i * 256 + lane * 8;
    float x[8];
    load_logits8(lr, idx, width, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t v = f32_ordered(x[e]);
      if (idx + e < width && (v > bv || !any)) {
        bv = v;
        bi = (uint32_t)(idx + e);
        any = true;
      }
    }
  }
  return warp_max_u64(any ? ((unsigned long long)bv << 32) | (unsigned long long)(0xFFFFFFFFu - bi) : 0ull);
}

// Stage 1: a warp a chunk of a row.
__global__ void __launch_bounds__(SEL_THREADS) k_chunk_max(const float *__restrict__ logits, int width, int nchunks,
                                                           unsigned long long *__restrict__ cmax,
                                                           int *__restrict__ cnt) {
  pdl_wait();
  const int row = blockIdx.y, chunk = blockIdx.x * (SEL_THREADS / 32) + (threadIdx.x >> 5);
  if (chunk < nchunks) {
    const unsigned long long best = chunk_best(logits + (int64_t)row * width, chunk, width);
    if ((threadIdx.x & 31) == 0) cmax[(int64_t)row * nchunks + chunk] = best;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) cnt[row] = 0;
}

// Stage 2: some CTAs a row; tau = the row's top-th
// largest chunk maximum (the top chunk maxima are `top` distinct logits of the
// row, so the row's top-th key is at least tau); the chunks' keys >= tau join
// the row's candidate list.
__global__ void __launch_bounds__(SEL_THREADS) k_chunk_filter(const float *__restrict__ logits, int width, int top,
                                                              int nchunks,
                                                              const unsigned long long *__restrict__ cmax,
                                                              int *__restrict__ cnt,
                                                              unsigned long long *__restrict__ cands) {
  pdl_wait();
  __shared__ unsigned long long cm[MAX_CHUNKS];
  __shared__ unsigned long long tau;
  __shared__ uint16_t hit[MAX_CHUNKS];
  __shared__ int nhit;
  const int row = blockIdx.y;
  for (int i = threadIdx.x; i < nchunks; i += SEL_THREADS) cm[i] = cmax[(int64_t)row * nchunks + i];
  if (threadIdx.x == 0) tau = 0ull;  // fewer chunks than `top`: every logit is a candidate
  __syncthreads();
  if (nchunks >= top)
    for (int i = threadIdx.x; i < nchunks; i += SEL_THREADS) {
      const unsigned long long k = cm[i];
      int above = 0;
      for (int m = 0; m < nchunks; ++m) above += cm[m] > k;
      if (above == top - 1) tau = k;  // keys are unique: exactly one thread
    }
  __syncthreads();
  const unsigned long long t = tau;
  const float *lr = logits + (int64_t)row * width;
  unsigned long long *out = cands + (int64_t)row * CAND_CAP;
  // the chunks that reach tau, in order (the row's CTAs make the same list); its
  // quarters are dealt out to the row's warps
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp == 0) {
    int n = 0;
    for (int i = 0; i < nchunks; i += 32) {
      const bool in = i + lane < nchunks && cm[i + lane] >= t;
      const unsigned m = __ballot_sync(0xffffffffu, in);
      if (in) hit[n + __popc(m & ((1u << lane) - 1))] = (uint16_t)(i + lane);
      n += __popc(m);
    }
    if (lane == 0) nhit = n;
  }
  __syncthreads();
  constexpr int PARTS = 4, PART = SEL_CHUNK / PARTS, NV = PART / 256;
  const uint32_t tv = (uint32_t)(t >> 32);
  for (int i = blockIdx.x + warp * gridDim.x; i < nhit * PARTS; i += gridDim.x * (SEL_THREADS / 32)) {
    const int first = hit[i / PARTS] * SEL_CHUNK + i % PARTS * PART + lane * 8;
    float x[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) load_logits8(lr, first + v * 256, width, x[v]);
    unsigned m = 0u;  // the thread's keys that reach tau
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int idx = first + v * 256 + e;
        if (f32_ordered(x[v][e]) >= tv && idx < width && cand_key(x[v][e], (uint32_t)idx) >= t) m |= 1u << (v * 8 + e);
      }
    if (m) {
      int at = atomicAdd(cnt + row, __popc(m));
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (m >> (v * 8 + e) & 1) {
            if (at < CAND_CAP) out[at] = cand_key(x[v][e], (uint32_t)(first + v * 256 + e));
            ++at;
          }
    }
  }
}

// The largest key below `below` in the row (block-wide), for the exact fallback.
__device__ unsigned long long row_max_below(const float *__restrict__ lr, int width, unsigned long long below,
                                            unsigned long long *red) {
  unsigned long long best = 0ull;
  for (int idx = threadIdx.x; idx < width; idx += ROW_THREADS) {
    const unsigned long long k = cand_key(lr[idx], (uint32_t)idx);
    if (k < below) best = umax64(best, k);
  }
  best = warp_max_u64(best);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = best;
  __syncthreads();
  unsigned long long v = 0ull;
  for (int w = 0; w < ROW_THREADS / 32; ++w) v = umax64(v, red[w]);
  return v;
}

// The row's top `top` keys' indices, in order, into out (shared memory): its
// candidate list ranked among itself, or, when the list overflowed (many equal
// logits), `top` exact passes over the row.
__device__ void row_top(const float *__restrict__ lr, int width, int top, int n,
                        const unsigned long long *__restrict__ list, unsigned long long *keys, unsigned long long *red,
                        uint32_t *out) {
  __syncthreads();
  if (n <= CAND_CAP) {
    for (int i = threadIdx.x; i < n; i += ROW_THREADS) keys[i] = list[i];
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += ROW_THREADS) {
      const unsigned long long k = keys[i];
      int above = 0;
      for (int m = 0; m < n; ++m) above += keys[m] > k;
      if (above < top) out[above] = cand_index(k);
    }
  } else {
    unsigned long long below = ~0ull;
    for (int r = 0; r < top; ++r) {
      below = row_max_below(lr, width, below, red);
      if (threadIdx.x == 0) out[r] = cand_index(below);
    }
  }
  __syncthreads();
}

// Stage 3: one CTA per row j of a sequence: its candidates, its possible
// predecessors (the anchor, or row j-1's candidates, ranked again here) and the
// score table score[p][c] = logit[cand_c] + sum_i (P[prev_p][i] * hp[i]) * C[cand_c][i].
__global__ void __launch_bounds__(ROW_THREADS) k_row_select(
    const float *__restrict__ logits, const float *__restrict__ hp, const uint32_t *__restrict__ anchor_tok,
    const uint16_t *__restrict__ pred, const uint16_t *__restrict__ succ, int k, int width, int rank, int top,
    int vocab, const int *__restrict__ cnt, const unsigned long long *__restrict__ cands, uint32_t *__restrict__ ctok,
    float *__restrict__ score) {
  pdl_wait();
  __shared__ unsigned long long keys[CAND_CAP];
  __shared__ unsigned long long red[ROW_THREADS / 32];
  __shared__ uint32_t cur[TOP_MAX], prv[TOP_MAX];
  __shared__ __align__(16) uint16_t Ps[TOP_MAX * RANK_MAX];
  __shared__ __align__(16) uint16_t Cs[TOP_MAX * RANK_MAX];
  __shared__ float hs[RANK_MAX];
  __shared__ float clog[TOP_MAX];
  const int row = blockIdx.x, b = row / k, j = row % k;
  const uint32_t anchor = anchor_tok[b];
  if (anchor >= (uint32_t)vocab) return;  // the chain reports it
  row_top(logits + (int64_t)row * width, width, top, cnt[row], cands + (int64_t)row * CAND_CAP, keys, red, cur);
  if (j > 0)
    row_top(logits + (int64_t)(row - 1) * width, width, top, cnt[row - 1], cands + (int64_t)(row - 1) * CAND_CAP,
            keys, red, prv);
  else if (threadIdx.x == 0)
    prv[0] = anchor;
  __syncthreads();
  const int np = j > 0 ? top : 1;
  const int r2 = rank / 2;
  for (int i = threadIdx.x; i < top * r2; i += ROW_THREADS) {
    const int c = i / r2, e = i % r2;
    ((uint32_t *)Cs)[c * r2 + e] = __ldg((const uint32_t *)(succ + (int64_t)cur[c] * rank) + e);
    if (c < np) ((uint32_t *)Ps)[c * r2 + e] = __ldg((const uint32_t *)(pred + (int64_t)prv[c] * rank) + e);
  }
  for (int i = threadIdx.x; i < rank; i += ROW_THREADS) hs[i] = hp[(int64_t)row * rank + i];
  for (int c = threadIdx.x; c < top; c += ROW_THREADS) {
    clog[c] = logits[(int64_t)row * width + cur[c]];
    ctok[(int64_t)row * top + c] = cur[c];
  }
  __syncthreads();
  for (int it = threadIdx.x; it < np * top; it += ROW_THREADS) {
    const int p = it / top, c = it % top;
    const __half2 *pr = (const __half2 *)(Ps + p * rank);
    const __half2 *cr = (const __half2 *)(Cs + c * rank);
    float acc = 0.f;
    for (int e = 0; e < r2; ++e) {
      const float2 pv = __half22float2(pr[e]);
      const float2 cv = __half22float2(cr[e]);
      acc = fmaf(pv.x * hs[2 * e], cv.x, acc);
      acc = fmaf(pv.y * hs[2 * e + 1], cv.y, acc);
    }
    score[((int64_t)row * top + p) * top + c] = clog[c] + acc;
  }
}

// Stage 4: one CTA per sequence runs the chain over the rows' tables: the first
// strictly greater score in candidate order wins and is the next predecessor.
__global__ void __launch_bounds__(CHAIN_THREADS) k_chain(const uint32_t *__restrict__ anchor_tok, int k, int top,
                                                         int vocab, const uint32_t *__restrict__ ctok,
                                                         const float *__restrict__ score, uint32_t *__restrict__ chosen,
                                                         uint32_t *__restrict__ plain) {
  pdl_wait();
  extern __shared__ __align__(16) uint8_t chain_sm[];
  float *sc = (float *)chain_sm;                    // [k][top][top]
  uint32_t *cand = (uint32_t *)(sc + k * top * top);  // [k][top]
  const int b = blockIdx.x;
  if (anchor_tok[b] >= (uint32_t)vocab) {
    for (int j = threadIdx.x; j < k; j += CHAIN_THREADS) chosen[b * k + j] = plain[b * k + j] = 0xFFFFFFFFu;
    return;
  }
  const float *sg = score + (int64_t)b * k * top * top;
  for (int i = threadIdx.x; i < k * top * top; i += CHAIN_THREADS) {
    const int j = i / (top * top);
    const int p = (i / top) % top;
    if (j > 0 || p == 0) sc[i] = sg[i];  // row 0 has one predecessor, the anchor
  }
  for (int i = threadIdx.x; i < k * top; i += CHAIN_THREADS) cand[i] = ctok[(int64_t)b * k * top + i];
  __syncthreads();
  if (threadIdx.x == 0) {
    int slot = 0;  // the predecessor's place among the previous row's candidates
    for (int j = 0; j < k; ++j) {
      const float *r = sc + (j * top + slot) * top;
      float bs = -INFINITY;
      int bc = 0;
      for (int c = 0; c < top; ++c)
        if (r[c] > bs) {
          bs = r[c];
          bc = c;
        }
      chosen[b * k + j] = cand[j * top + bc];
      plain[b * k + j] = cand[j * top];
      slot = bc;
    }
  }
}

void select_stage1(void *scratch, int rows, int width, unsigned long long **cmax, int **cnt, int *nchunks) {
  *nchunks = sel_chunks(width);
  *cmax = (unsigned long long *)scratch;
  unsigned long long *cands = *cmax + (size_t)rows * *nchunks;
  *cnt = (int *)(cands + (size_t)rows * CAND_CAP);
}

// Stages 1 and 2: each row's candidate list and its length.
static cudaError_t row_candidates(const float *logits, int rows, int width, int top, unsigned long long *cmax,
                                  unsigned long long *cands, int *cnt, int num_sms, cudaStream_t st,
                                  bool stage1_done) {
  const int nchunks = sel_chunks(width);
  // Stage 1: 8 chunks a CTA, however many CTAs that makes (480 rows: 10 us less than
  // one wave of CTAs with 24 to 32 chunks). Stage 2, whose CTAs all find tau: about 4 an SM
  // (480 rows: 82 us for the whole selector; with 1 to 3 an SM, and with 8, 84).
  const int most = (nchunks + SEL_THREADS / 32 - 1) / (SEL_THREADS / 32);
  const dim3 g1(most, rows), g2(std::min(most, (4 * num_sms + rows - 1) / rows), rows);
  cudaError_t e = cudaSuccess;
  if (!stage1_done) {
    e = launch_pdl(k_chunk_max, g1, dim3(SEL_THREADS), 0, st, 1, logits, width, nchunks, cmax, cnt);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(k_chunk_filter, g2, dim3(SEL_THREADS), 0, st, 1, logits, width, top, nchunks, cmax, cnt,
                    cands);
}

cudaError_t select_tokens(const float *logits, const float *hp, const uint32_t *anchor_tok, const uint16_t *pred,
                          const uint16_t *succ, int batch, int k, int width, int rank, int top, int vocab, void *scratch,
                          uint32_t *chosen, uint32_t *plain, int num_sms, cudaStream_t st, bool stage1_done) {
  if (top > TOP_MAX || rank > RANK_MAX || top < 1 || k > KMAX || rank % 2) return cudaErrorInvalidValue;
  const int nchunks = sel_chunks(width);
  if (nchunks > MAX_CHUNKS) return cudaErrorInvalidValue;
  const int rows = batch * k;
  unsigned long long *cmax = (unsigned long long *)scratch;
  unsigned long long *cands = cmax + (size_t)rows * nchunks;
  int *cnt = (int *)(cands + (size_t)rows * CAND_CAP);
  uint32_t *ctok = (uint32_t *)(cnt + ((rows + 1) & ~1));
  float *score = (float *)(ctok + (size_t)rows * top);
  static PerDevice configured;
  const size_t smem = (size_t)k * top * top * 4 + (size_t)k * top * 4;
  const size_t most = (size_t)KMAX * TOP_MAX * TOP_MAX * 4 + (size_t)KMAX * TOP_MAX * 4;
  if (cudaError_t e = smem_limit(k_chain, (int)most, configured)) return e;
  cudaError_t e = row_candidates(logits, rows, width, top, cmax, cands, cnt, num_sms, st, stage1_done);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k_row_select, dim3(rows), dim3(ROW_THREADS), 0, st, 1, logits, hp, anchor_tok, pred, succ, k, width,
                 rank, top, vocab, cnt, cands, ctok, score);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_chain, dim3(batch), dim3(CHAIN_THREADS), smem, st, 1, anchor_tok, k, top, vocab, ctok, score,
                    chosen, plain);
}

// ---------------------------------------------------------------------------
// The sampled chain: the token of each row drawn from softmax(score / T) over
// the row's candidates with a given uniform number, the proposal that
// dflash_verify weighs against the target. Stages 1 and 2 as above; then
//   stage 3 (one CTA per row): the candidates and, for every predecessor the
//   chain can ask of the row, its candidates' probabilities and the one drawn.
//   A warp takes a predecessor, a lane a candidate (up to 16 candidates: half a
//   lane's products each); cumulative weights are whole numbers (fixed.cuh).
//   stage 4 (one CTA per sequence): the chain, a table look-up a row.
// 480 rows of 151,936 (top 16, rank 64): 83 us, of which stage 1 some 48 (HBM: 292 MB),
// stage 2 and 3 15 - 20 each; 15 rows: 17 us, four launches of some 4 us of latency.
// The scores are sums of exact products kept as two floats (a sum of n terms is then
// off by n^2 2^-48 of their sizes at worst: 2^-36 for 64, where 2^-43 is usual): a
// choice turns on a border between two cumulative weights, and an f32 score would move
// it by 2^-20.
struct SampleScratch {
  unsigned long long *cmax, *cands;
  float *q;       // [rows][top predecessors][top candidates]
  int *cnt, *nxt;  // nxt: [rows][top predecessors], the candidate drawn
  uint32_t *ctok;
  size_t bytes;
};
static SampleScratch sample_scratch(void *base, int64_t rows, int width, int top) {
  SampleScratch s;
  s.cmax = (unsigned long long *)base;
  s.cands = s.cmax + rows * sel_chunks(width);
  s.q = (float *)(s.cands + rows * CAND_CAP);
  s.cnt = (int *)(s.q + rows * top * top);
  s.nxt = s.cnt + rows;
  s.ctok = (uint32_t *)(s.nxt + rows * top);
  s.bytes = (size_t)((char *)(s.ctok + rows * top) - (char *)base);
  return s;
}

__device__ __forceinline__ void two_add(float &h, float &l, float x) {
  const float s = h + x, b = s - h;
  l += (h - (s - b)) + (x - b);
  h = s;
}

__global__ void __launch_bounds__(ROW_THREADS) k_row_sample(
    const float *__restrict__ logits, const float *__restrict__ hp, const uint32_t *__restrict__ anchor_tok,
    const uint16_t *__restrict__ pred, const uint16_t *__restrict__ succ, const float *__restrict__ temperature,
    const float *__restrict__ uniforms, int k, int width, int rank, int top, int vocab, SampleScratch S) {
  __shared__ unsigned long long keys[2][CAND_CAP];
  __shared__ unsigned long long red[ROW_THREADS / 32];
  __shared__ unsigned long long tab[64];
  __shared__ uint32_t ids[2][TOP_MAX];  // the row's candidates; the row's before it (row 0: the anchor)
  __shared__ __align__(16) uint16_t Ps[TOP_MAX * RANK_MAX];
  extern __shared__ __align__(16) uint8_t rs_sm[];  // the successors' rows, padded by one word
  __shared__ float hs[RANK_MAX];
  uint32_t *Cs = (uint32_t *)rs_sm;
  if (threadIdx.x < 64) tab[threadIdx.x] = kFxTable[threadIdx.x];
  pdl_wait();
  const int row = blockIdx.x, b = row / k, j = row % k;
  const uint32_t anchor = anchor_tok[b];
  if (anchor >= (uint32_t)vocab) return;  // the chain reports it
  // ranked by half the threads each; a list that overflowed, by all of them
  const int n0 = S.cnt[row], n1 = j > 0 ? S.cnt[row - 1] : 0;
  {
    const int half = threadIdx.x / (ROW_THREADS / 2), t = threadIdx.x % (ROW_THREADS / 2);
    const int n = half ? n1 : n0;
    const unsigned long long *list = S.cands + (int64_t)(row - half) * CAND_CAP;
    if (n <= CAND_CAP)
      for (int i = t; i < n; i += ROW_THREADS / 2) keys[half][i] = list[i];
    if (j == 0 && threadIdx.x == 0) ids[1][0] = anchor;
    __syncthreads();
    if (n <= CAND_CAP)
      for (int i = t; i < n; i += ROW_THREADS / 2) {
        const unsigned long long key = keys[half][i];
        int above = 0;
        for (int m = 0; m < n; ++m) above += keys[half][m] > key;
        if (above < top) ids[half][above] = cand_index(key);
      }
  }
  const float *lr = logits + (int64_t)row * width;
  if (n0 > CAND_CAP) row_top(lr, width, top, n0, nullptr, nullptr, red, ids[0]);
  if (n1 > CAND_CAP) row_top(lr - width, width, top, n1, nullptr, nullptr, red, ids[1]);
  __syncthreads();
  const uint32_t *cur = ids[0], *prv = ids[1];
  const int np = j > 0 ? top : 1, r2 = rank / 2, ldc = r2 + 1;
  for (int i = threadIdx.x; i < top * r2; i += ROW_THREADS) {
    const int c = i / r2, e = i % r2;
    Cs[c * ldc + e] = __ldg((const uint32_t *)(succ + (int64_t)cur[c] * rank) + e);
    if (c < np) ((uint32_t *)Ps)[c * r2 + e] = __ldg((const uint32_t *)(pred + (int64_t)prv[c] * rank) + e);
  }
  for (int i = threadIdx.x; i < rank; i += ROW_THREADS) hs[i] = hp[(int64_t)row * rank + i];
  for (int c = threadIdx.x; c < top; c += ROW_THREADS) S.ctok[(int64_t)row * top + c] = cur[c];
  __syncthreads();
  const float T = temperature ? temperature[b] : 1.f, u = uniforms[row];
  const FxScale fs = fx_scale(T > 0.f ? T : 1.f);
  const int lane = threadIdx.x & 31;
  const int parts = top <= 16 ? 2 : 1, c = parts == 2 ? lane & 15 : lane, part = parts == 2 ? lane >> 4 : 0;
  for (int p = threadIdx.x >> 5; p < np; p += ROW_THREADS / 32) {
    float h = part ? 0.f : -INFINITY, l = 0.f;
    if (c < top) {
      if (part == 0) h = lr[cur[c]];
      const __half2 *pr = (const __half2 *)(Ps + p * rank), *cr = (const __half2 *)(Cs + c * ldc);
      const int e1 = (part + 1) * r2 / parts;
#pragma unroll 4
      for (int e = part * r2 / parts; e < e1; ++e) {
        const float2 pv = __half22float2(pr[e]), cv = __half22float2(cr[e]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float x = i ? pv.y : pv.x, z = i ? cv.y : cv.x, s = hs[2 * e + i];
          const float a = x * s, al = fmaf(x, s, -a);  // x s = a + al
          const float y = __fmul_rn(a, z);         // (fused into the sum below, its rounding would count twice)
          two_add(h, l, y);
          l += fmaf(a, z, -y) + al * z;
        }
      }
    }
    if (parts == 2) {
      const float oh = __shfl_xor_sync(0xffffffffu, h, 16), ol = __shfl_xor_sync(0xffffffffu, l, 16);
      two_add(h, l, oh);
      l += ol;
      if (part) h = -INFINITY;
    }
    // the first largest score (as two floats, in order), and the weights against it
    if (h > -INFINITY && h < INFINITY) {
      const float r = h + l;
      l -= r - h;
      h = r;
    } else {
      l = 0.f;  // infinite, or not a number: never the largest
    }
    float mh = h, ml = l;
    int at = h > -INFINITY ? lane : 32;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float vh = __shfl_xor_sync(0xffffffffu, mh, o), vl = __shfl_xor_sync(0xffffffffu, ml, o);
      const int i = __shfl_xor_sync(0xffffffffu, at, o);
      if (i < 32 && (at == 32 || vh > mh || (vh == mh && (vl > ml || (vl == ml && i < at))))) {
        mh = vh;
        ml = vl;
        at = i;
      }
    }
    unsigned long long w = 0ull;
    if (at == 32) {
      w = lane == 0 ? 1ull : 0ull;  // no score is a number above -inf: the first candidate
    } else if (!(T > 0.f)) {
      w = lane == at ? 1ull : 0ull;
    } else if (mh == INFINITY) {
      w = h == INFINITY ? 1ull : 0ull;
    } else if (h > -INFINITY) {     // (lanes past the candidates hold -inf)
      float d = h - mh;
      const float b = d - h;
      float e = (h - (d - b)) + (-mh - b) + (l - ml);
      const float r = d + e;        // (where h and mh are near, the low parts are the larger)
      e -= r - d;
      d = r;
      w = fx_weight_diff(d, e, fs, tab);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long v = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += v;
    }
    const unsigned long long total = __shfl_sync(0xffffffffu, w, top - 1);
    unsigned long long own = __shfl_up_sync(0xffffffffu, w, 1);
    own = lane ? w - own : w;
    const unsigned over = __ballot_sync(0xffffffffu, lane < top && w > fx_target(u, total));
    if (lane < top) S.q[((int64_t)row * top + p) * top + lane] = fx_ratio(own, total);
    if (lane == 0) S.nxt[(int64_t)row * top + p] = __ffs(over) - 1;
  }
}

__global__ void __launch_bounds__(CHAIN_THREADS) k_chain_sample(const uint32_t *__restrict__ anchor_tok, int k, int top,
                                                                int vocab, SampleScratch S,
                                                                uint32_t *__restrict__ chosen,
                                                                uint32_t *__restrict__ cand, float *__restrict__ q) {
  __shared__ int nxt[KMAX * TOP_MAX], slots[KMAX + 1];
  pdl_wait();
  const int b = blockIdx.x;
  if (anchor_tok[b] >= (uint32_t)vocab) {
    for (int i = threadIdx.x; i < k; i += CHAIN_THREADS) chosen[b * k + i] = 0xFFFFFFFFu;
    for (int i = threadIdx.x; i < k * top; i += CHAIN_THREADS) {
      cand[(int64_t)b * k * top + i] = 0xFFFFFFFFu;
      q[(int64_t)b * k * top + i] = 0.f;
    }
    return;
  }
  // (row 0 has one predecessor, the anchor)
  for (int i = threadIdx.x; i < k * top; i += CHAIN_THREADS)
    if (i == 0 || i >= top) nxt[i] = S.nxt[(int64_t)b * k * top + i];
  __syncthreads();
  if (threadIdx.x == 0) {
    int slot = 0;
    for (int j = 0; j < k; ++j) {
      slots[j] = slot;
      slot = nxt[j * top + slot];
    }
    slots[k] = slot;
  }
  __syncthreads();
  // the candidates and their probabilities after the chosen predecessors
  for (int i = threadIdx.x; i < k * top; i += CHAIN_THREADS) {
    const int j = i / top, c = i % top;
    const int64_t r = (int64_t)b * k + j;
    const uint32_t id = S.ctok[r * top + c];
    cand[r * top + c] = id;
    q[r * top + c] = S.q[(r * top + slots[j]) * top + c];
    if (c == slots[j + 1]) chosen[r] = id;
  }
}

}  // namespace dfl

// ---------------------------------------------------------------------------
// The selector for callers that cannot allocate device memory.
//
// Some callers have no way to hand the library scratch memory: code that runs
// under another framework's memory pool (which owns the device heap and does
// not let a plug-in call cudaMalloc), decode loops that must not take
// cudaMalloc's implicit device-wide synchronisation in the middle of a token,
// and foreign-function callers with no device allocator of their own. For
// them the selector's candidate scratch lives in a fixed array below, part of
// the library image: every GPU that loads the library holds it until the
// process exits.

namespace dfl {
namespace {

constexpr size_t kStaticSelectScratch = 8u << 20;  // bytes: 9,888 a row at a 151,936 vocabulary and top 16
static __device__ __align__(256) unsigned char g_select_scratch[kStaticSelectScratch];

// Host code cannot use g_select_scratch as a device address (in host code the
// name is a host-side stand-in), so each device's address is looked up once.
std::mutex g_scratch_mu;
void *g_scratch_addr[64] = {};

cudaError_t static_scratch(void **out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_addr[dev]) {
    void *p = nullptr;
    e = cudaGetSymbolAddress(&p, g_select_scratch);
    if (e != cudaSuccess) return e;
    g_scratch_addr[dev] = p;
  }
  *out = g_scratch_addr[dev];
  return cudaSuccess;
}

}  // namespace

}  // namespace dfl

extern "C" int dflash_select_static(const float *logits, const float *hp, const uint32_t *anchor_tok,
                                    const uint16_t *pred_book, const uint16_t *succ_book, int32_t batch, int32_t k,
                                    int32_t width, int32_t vocab, int32_t rank, int32_t top, uint32_t *chosen,
                                    uint32_t *plain, void *stream) {
  using namespace dfl;
  if (!logits || !hp || !anchor_tok || !pred_book || !succ_book || !chosen || !plain)
    return dflash_fail(DFLASH_E_ARG, "select_static: null pointer");
  if (batch < 1 || k < 1 || k > KMAX || top < 1 || top > TOP_MAX || width < top || width > vocab ||
      rank < 16 || rank > RANK_MAX || rank % 16)
    return dflash_fail(DFLASH_E_ARG, "select_static: batch >= 1, 1 <= k <= 15, 1 <= top <= 32, "
                                     "top <= width <= vocab, rank a multiple of 16 in 16..256");
  if (sel_chunks(width) > MAX_CHUNKS) return dflash_fail(DFLASH_E_ARG, "select_static: width beyond 2 M");
  const size_t need = select_scratch_bytes(batch * k, width, top);
  if (need > kStaticSelectScratch)
    return dflash_fail(DFLASH_E_CAPACITY, "select_static: the call's candidates and score tables exceed the fixed "
                                          "8 MiB scratch; use dflash_select");
  void *scratch = nullptr;
  cudaError_t e = static_scratch(&scratch);
  if (e != cudaSuccess)
    return dflash_fail(DFLASH_E_CUDA, std::string("select_static: cudaGetSymbolAddress: ") + cudaGetErrorString(e));
  int sms = 148, dev = 0;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  e = select_tokens(logits, hp, anchor_tok, pred_book, succ_book, batch, k, width, rank, top, vocab, scratch,
                    chosen, plain, sms, (cudaStream_t)stream);
  if (e != cudaSuccess) return dflash_fail(DFLASH_E_CUDA, std::string("select_static: ") + cudaGetErrorString(e));
  return DFLASH_OK;
}

extern "C" size_t dflash_select_sample_workspace_bytes(int32_t batch, int32_t k, int32_t width, int32_t top) {
  using namespace dfl;
  if (batch < 1 || k < 1 || k > KMAX || (int64_t)batch * k > 65535 || top < 1 || top > TOP_MAX || width < top ||
      sel_chunks(width) > MAX_CHUNKS)
    return 0;
  return sample_scratch(nullptr, (int64_t)batch * k, width, top).bytes;
}

extern "C" int dflash_select_sample(const float *logits, const float *hp, const uint32_t *anchor_tok,
                                    const uint16_t *pred_book, const uint16_t *succ_book, int32_t batch, int32_t k,
                                    int32_t width, int32_t vocab, int32_t rank, int32_t top, const float *temperature,
                                    const float *uniforms, uint32_t *chosen, uint32_t *cand, float *cand_q,
                                    void *workspace, size_t workspace_bytes, void *stream) {
  using namespace dfl;
  if (!logits || !hp || !anchor_tok || !pred_book || !succ_book || !uniforms || !chosen || !cand || !cand_q)
    return dflash_fail(DFLASH_E_ARG, "select_sample: null pointer");
  const size_t need = dflash_select_sample_workspace_bytes(batch, k, width, top);
  if (need == 0 || width > vocab || rank < 16 || rank > RANK_MAX || rank % 16)
    return dflash_fail(DFLASH_E_ARG, "select_sample: batch >= 1, 1 <= k <= 15, batch * k <= 65,535, 1 <= top <= 32, "
                                     "top <= width <= vocab and 2 M, rank a multiple of 16 in 16..256");
  for (const void *p : {(const void *)logits, (const void *)hp, (const void *)anchor_tok, (const void *)pred_book,
                        (const void *)succ_book, (const void *)temperature, (const void *)uniforms,
                        (const void *)chosen, (const void *)cand, (const void *)cand_q})
    if ((uintptr_t)p & 3) return dflash_fail(DFLASH_E_ARG, "select_sample: misaligned pointer");
  if (!workspace || ((uintptr_t)workspace & 15))
    return dflash_fail(DFLASH_E_ARG, "select_sample: null or misaligned workspace");
  if (workspace_bytes < need)
    return dflash_fail(DFLASH_E_CAPACITY, "select_sample: workspace smaller than dflash_select_sample_workspace_bytes");
  const int rows = batch * k;
  const SampleScratch S = sample_scratch(workspace, rows, width, top);
  cudaStream_t st = (cudaStream_t)stream;
  static PerDevice row_done;
  cudaError_t e = smem_limit(k_row_sample, TOP_MAX * (RANK_MAX / 2 + 1) * 4, row_done);
  if (e == cudaSuccess) e = row_candidates(logits, rows, width, top, S.cmax, S.cands, S.cnt, device_sms(), st, false);
  if (e == cudaSuccess)
    e = launch_pdl(k_row_sample, dim3(rows), dim3(ROW_THREADS), (size_t)top * (rank / 2 + 1) * 4, st, 1, logits, hp,
                   anchor_tok, pred_book, succ_book, temperature, uniforms, k, width, rank, top, vocab, S);
  if (e == cudaSuccess)
    e = launch_pdl(k_chain_sample, dim3(batch), dim3(CHAIN_THREADS), 0, st, 1, anchor_tok, k, top, vocab, S, chosen, cand,
                   cand_q);
  if (e != cudaSuccess) return dflash_fail(DFLASH_E_CUDA, std::string("select_sample: ") + cudaGetErrorString(e));
  return DFLASH_OK;
}
