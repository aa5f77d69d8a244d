// Verification of drafted tokens against the target's probabilities (the accept
// and residual rules of speculative sampling: Leviathan, Kalman and Matias,
// "Fast inference from transformers via speculative decoding"; Chen et al.,
// "Accelerating large language model decoding with speculative sampling").
//
//   p_j = softmax(l_j / T);  x_j is kept while u_j q_j(x_j) < p_j(x_j);
//   the token after the kept ones is drawn from max(p - q, 0) of the first row
//   that was not kept, or from p of the row after the last draft.
//
// Two launches. k_verify_stats reads every logit once: per part of a row its largest
// value and the sum of its exponentials (109 MB of bf16 in 27 us, 4.1 TB/s: a CTA's
// loads, reductions and end follow one another, six CTAs an SM). k_verify_sample has
// CTAs per (chunks of the vocabulary, sequence): each merges its sequence's parts (a
// warp a row) and decides how far the draft is kept, then its warps sum whole-number
// weights (fixed.cuh) of 128 tokens each of the one row a token is drawn from; the
// sequence's last CTA takes out the proposal's part, finds the 128 tokens that the
// uniform number falls into and then the token. The weights are integers, so the draw
// does not depend on the order of any sum. It is a chain of small steps: 2 us until
// the draft is decided, 1 - 10 us for the weights (some 80 instructions each), and some
// 5 us from the last CTA's ticket to the token. One sequence of 16 f32 rows of 151,936:
// 14 us for both launches; 32 of up to 16 bf16 rows: 53, and 55 with no greedy sequence.
#include <algorithm>
#include <climits>
#include <string>
#include <type_traits>

#include <cuda_bf16.h>

#include "common.cuh"
#include "dflash.h"
#include "fixed.cuh"
#include "kernels.h"

namespace dfl {

constexpr int VF_THREADS = 256;
constexpr int VF_PART = 8192;    // logits a CTA of the first launch
constexpr int VS_THREADS = 512;  // of the second: a warp a row of up to 16
constexpr int VF_CHUNK = 2048;   // logits a CTA of the second
constexpr int VF_RUN = VF_CHUNK / (VS_THREADS / 32);  // of a warp: a run, whose weights are summed
constexpr int VF_TOP = 32;
constexpr int VF_ROWS = 256;     // rows of a sequence (k + 1)
constexpr uint32_t VF_NONE = 0xFFFFFFFFu;
constexpr int VF_OPEN = -1;

struct VfArgs {
  const void *logits;
  int64_t ld;
  int batch, k, vocab, top, nparts, nruns;
  int per_cta;                   // chunks a CTA of k_verify_sample
  const uint32_t *drafted;
  const int32_t *n_drafted;
  const uint32_t *cand;
  const float *cand_q;
  const float *temperature;
  const float *u;
  int32_t *accepted;
  uint32_t *tokens;
  float4 *part;                  // [rows][nparts]: largest value, sum, its index (bits)
  unsigned long long *csum;      // [batch][nruns]
  unsigned *ticket;              // [batch]
};

__device__ __forceinline__ int vf_drafted(const VfArgs &A, int b) {
  return A.n_drafted ? max(0, min(A.k, A.n_drafted[b])) : A.k;
}
__device__ __forceinline__ float vf_temperature(const VfArgs &A, int b) { return A.temperature ? A.temperature[b] : 1.f; }

// NaN logits are never chosen: they count as -inf.
template <typename T>
__device__ __forceinline__ float vf_value(T x) {
  const float f = (float)x;
  return f == f ? f : -INFINITY;
}

__device__ __forceinline__ float vf_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Value i of a 16-byte vector of logits.
template <typename T>
__device__ __forceinline__ float vf_elem(const uint4 &w, int i) {
  if constexpr (sizeof(T) == 4) {
    return __uint_as_float(i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w);
  } else {
    const uint32_t h = i / 2 == 0 ? w.x : i / 2 == 1 ? w.y : i / 2 == 2 ? w.z : w.w;
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      return __uint_as_float(i & 1 ? h & 0xFFFF0000u : h << 16);
    } else {
      return __half2float(__ushort_as_half((unsigned short)(i & 1 ? h >> 16 : h & 0xFFFFu)));
    }
  }
}

// The larger values of two pairs, the number where one is not one.
template <typename T>
__device__ __forceinline__ uint32_t vf_max2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (std::is_same<T, __nv_bfloat16>::value) asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A thread's logits stay in registers, as they came, between the maximum and the
// exponentials. Rows may start anywhere: the vectors are those of the aligned
// address below a row's start, and the first and last vectors are read by single
// values, -inf outside the row.
template <typename T>
__global__ void __launch_bounds__(VF_THREADS, 6) k_verify_stats(const __grid_constant__ VfArgs A) {
  constexpr int VL = 16 / (int)sizeof(T), NV = VF_PART / (VF_THREADS * VL);
  __shared__ float redm[VF_THREADS / 32], reds[VF_THREADS / 32];
  __shared__ int redi[VF_THREADS / 32];
  const int row = blockIdx.y, b = row / (A.k + 1), j = row - b * (A.k + 1);
  const T *lr = (const T *)A.logits + (int64_t)row * A.ld;
  const int shift = (int)(((uintptr_t)lr & 15) / sizeof(T));  // values between the aligned address and the row
  pdl_wait();
  if (blockIdx.x == 0 && j == 0 && threadIdx.x == 0) A.ticket[b] = 0u;
  if (j > vf_drafted(A, b)) return;  // past the sequence's draft
  const float T0 = vf_temperature(A, b);
  uint4 x[NV];
  const int e0 = blockIdx.x * VF_PART + threadIdx.x * VL - shift;  // the thread's first value
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = e0 + v * VF_THREADS * VL;
    if (e >= 0 && e + VL <= A.vocab) {
      x[v] = __ldg((const uint4 *)(lr + e));
    } else {
      T t[VL];
#pragma unroll
      for (int i = 0; i < VL; ++i) t[i] = e + i >= 0 && e + i < A.vocab ? lr[e + i] : (T)(-INFINITY);
      memcpy(&x[v], t, 16);
    }
  }
  float m = -INFINITY;  // (NaN is left out of it)
  if constexpr (sizeof(T) == 2) {  // two values an instruction, before any is converted
    uint32_t p = vf_max2<T>(x[0].x, x[0].y);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (v > 0) p = vf_max2<T>(p, vf_max2<T>(x[v].x, x[v].y));
      p = vf_max2<T>(p, vf_max2<T>(x[v].z, x[v].w));
    }
    const uint4 two = make_uint4(p, 0u, 0u, 0u);
    m = fmaxf(m, fmaxf(vf_elem<T>(two, 0), vf_elem<T>(two, 1)));
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < VL; ++i) m = fmaxf(m, vf_elem<T>(x[v], i));
  }
  m = warp_max(m);
  float s = 0.f;
  int at = INT_MAX;
  const float c = fminf(1.4426950408889634f / T0, 1e30f);
  if (T0 > 0.f) {
    const bool plain = m > -INFINITY && m < INFINITY && c > 0.f;
    if (plain) {
      float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < VL; ++i) s4[i & 3] += vf_ex2((vf_elem<T>(x[v], i) - m) * c);
      s = (s4[0] + s4[1]) + (s4[2] + s4[3]);
    }
    if (!plain || !(s == s)) {  // infinite values, an infinite temperature, or NaN among them
      s = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < VL; ++i) {
          const float f = vf_elem<T>(x[v], i);
          if (f > -INFINITY) s += m == INFINITY ? (f == INFINITY ? 1.f : 0.f) : vf_ex2((f - m) * c);
        }
    }
  } else if (m > -INFINITY) {  // greedy: the lowest index of the largest value
#pragma unroll
    for (int v = NV - 1; v >= 0; --v)
#pragma unroll
      for (int i = VL - 1; i >= 0; --i)
        if (vf_elem<T>(x[v], i) == m) at = e0 + v * VF_THREADS * VL + i;
  }
  s = warp_sum(s);
  at = __reduce_min_sync(0xffffffffu, at);
  if ((threadIdx.x & 31) == 0) {
    redm[threadIdx.x >> 5] = m;
    reds[threadIdx.x >> 5] = s;
    redi[threadIdx.x >> 5] = at;
  }
  __syncthreads();
  if (threadIdx.x < 32) {  // (a warp's sum is against its own largest value)
    const int w = threadIdx.x;
    const float mw = w < VF_THREADS / 32 ? redm[w] : -INFINITY, sw = w < VF_THREADS / 32 ? reds[w] : 0.f;
    m = warp_max(mw);
    s = warp_sum(mw == m ? sw : mw > -INFINITY && m < INFINITY ? sw * vf_ex2((mw - m) * c) : 0.f);
    at = __reduce_min_sync(0xffffffffu, w < VF_THREADS / 32 && mw == m ? redi[w] : INT_MAX);
    if (w == 0) A.part[(int64_t)row * A.nparts + blockIdx.x] = make_float4(m, s, __int_as_float(at), 0.f);
  }
}

// Inclusive sum over the CTA's threads; `total` in every thread.
__device__ __forceinline__ unsigned long long vf_scan(unsigned long long v, unsigned long long *red,
                                                      unsigned long long &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long w = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += w;
  }
  __syncthreads();
  if (lane == 31) red[warp] = v;
  __syncthreads();
  unsigned long long before = 0ull;
  total = 0ull;
#pragma unroll
  for (int w = 0; w < VS_THREADS / 32; ++w) {
    if (w < warp) before += red[w];
    total += red[w];
  }
  return v + before;
}

__device__ __forceinline__ unsigned long long vf_warp_sum(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// u q Z 2^40 < w: 1 or 0, or -1 where Z, a sum of f32 exponentials, does not tell. Z is
// within 2^-16 of the sum of the row's whole-number weights: exponents are off by 2^-22 of
// up to 21 that matter, their powers by 2^-22 in each of three steps, the sums by 32
// roundings, and the weights by 1.5 of 2^40 for each of up to 2^21.
__device__ __forceinline__ int vf_below(float u, float q, float Z, unsigned long long w) {
  const float p = u * q, pe = fmaf(u, q, -p);
  const float z = p * Z, ze = fmaf(p, Z, -z) + pe * Z;
  const float wh = __ull2float_rn(w), wl = __ll2float_rn((long long)(w - __float2ull_rn(wh)));
  const float sc = (float)(1ull << FX_BITS);
  const float d = (z * sc - wh) + (ze * sc - wl);
  return w > 0ull && fabsf(d) <= z * sc * 0x1p-16f ? -1 : d < 0.f;
}
// u q Z < w of whole numbers w <= Z, exactly.
__device__ bool vf_less(float u, float q, unsigned long long Z, unsigned long long w) {
  if (!(u * q < 2.f)) return false;  // (nor where it is not a number)
  if (!(u > 0.f && q > 0.f)) return w > 0ull;
  const int bu = __float_as_int(u), bq = __float_as_int(q), eu = bu >> 23, eq = bq >> 23;
  const unsigned long long m = (unsigned long long)(eu ? (bu & 0x7fffff) | 0x800000 : bu) *
                               (unsigned long long)(eq ? (bq & 0x7fffff) | 0x800000 : bq);
  const int sh = 300 - (eu ? eu : 1) - (eq ? eq : 1);  // u q = m 2^-sh, m < 2^48
  if (w == 0ull || sh < 0) return false;
  if (64 - __clzll((long long)w) + sh > 127) return true;  // m Z < 2^110
  return (unsigned __int128)m * Z < (unsigned __int128)w << sh;
}

template <typename T>
__global__ void __launch_bounds__(VS_THREADS, 2) k_verify_sample(const __grid_constant__ VfArgs A) {
  constexpr int W = VS_THREADS / 32, PER = VF_RUN / 32;
  __shared__ unsigned long long tab[64], red[W], sub[VS_THREADS], taken, base, target;
  __shared__ float rowm[VF_ROWS];
  __shared__ int rowi[VF_ROWS];    // greedy: the largest value's index; else VF_OPEN where not decided
  __shared__ float rowq[VF_ROWS];
  __shared__ int kept, last, pick, owner, open;
  if (threadIdx.x < 64) tab[threadIdx.x] = kFxTable[threadIdx.x];
  if (threadIdx.x == 64) {
    kept = A.k;
    open = INT_MAX;
  }
  sub[threadIdx.x] = 0ull;
  __syncthreads();
  const int b = blockIdx.y, chunk = blockIdx.x, t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int K1 = A.k + 1;
  pdl_wait();
  const int n = vf_drafted(A, b);
  const float T0 = vf_temperature(A, b);
  const float u_last = A.u[(int64_t)b * K1 + A.k];
  const bool greedy = !(T0 > 0.f);
  const FxScale sc = fx_scale(greedy ? 1.f : T0);
  // a warp a row: its largest value and sum; whether its draft is kept. (What a row needs
  // is asked for before n and T are known, but for the logits, which n bounds.)
  for (int r = warp; r <= A.k; r += W) {
    const float4 *part = A.part + ((int64_t)b * K1 + r) * A.nparts;
    const float4 p0 = lane < A.nparts ? part[lane] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
    uint32_t x = VF_NONE, cx = VF_NONE;
    float cq = 0.f, u = 0.f;
    if (r < A.k) {
      x = A.drafted[(int64_t)b * A.k + r];
      u = A.u[(int64_t)b * K1 + r];
      if (lane < A.top) {
        cx = A.cand[((int64_t)b * A.k + r) * A.top + lane];
        cq = A.cand_q[((int64_t)b * A.k + r) * A.top + lane];
      }
    }
    const float l = r < n && x < (uint32_t)A.vocab ? vf_value(((const T *)A.logits)[((int64_t)b * K1 + r) * A.ld + x]) : -INFINITY;
    if (r > n) break;
    const float q = A.top > 0 ? warp_sum(cx == x && lane < A.top ? fmaxf(cq, 0.f) : 0.f) : 1.f;
    float M = p0.x;
    int at = __float_as_int(p0.z);
    for (int i = lane + 32; i < A.nparts; i += 32) {
      const float4 p = part[i];
      if (p.x > M) {
        M = p.x;
        at = __float_as_int(p.z);
      }
    }
    const float Mr = warp_max(M);
    at = __reduce_min_sync(0xffffffffu, M == Mr ? at : INT_MAX);
    M = Mr;
    float Z = 0.f;
    if (!greedy && M > -INFINITY) {
      auto add = [&](const float4 &p) {
        if (p.x == M) Z += p.y;
        else if (p.x > -INFINITY && M < INFINITY) Z = fmaf(p.y, exp2f((p.x - M) * sc.hi), Z);
      };
      add(p0);
      for (int i = lane + 32; i < A.nparts; i += 32) add(part[i]);
      Z = warp_sum(Z);
    }
    if (lane == 0) {
      rowm[r] = M;
      rowi[r] = at;
      if (r < n) {
        const int keep =
            greedy ? M > -INFINITY && x == (uint32_t)at : vf_below(u, q, Z, fx_weight(l, M, sc, tab));
        if (keep < 0) {
          rowi[r] = VF_OPEN;
          rowq[r] = q;
          atomicMin(&open, r);
        }
        if (keep == 0) atomicMin(&kept, r);
      }
    }
  }
  if (greedy && chunk > 0) return;
  __syncthreads();
  // rows too near their border for Z (one in 30,000 and fewer) are summed in whole numbers,
  // by all threads, in the rows' order
  for (int r = open; r < min(kept, n); ++r) {
    if (greedy || rowi[r] != VF_OPEN) continue;
    const T *lo = (const T *)A.logits + ((int64_t)b * K1 + r) * A.ld;
    const float m = rowm[r];
    unsigned long long s = 0ull;
    for (int e = t; e < A.vocab; e += VS_THREADS) s += fx_weight(vf_value(lo[e]), m, sc, tab);
    s = vf_warp_sum(s);
    if (lane == 0) red[warp] = s;
    __syncthreads();
    if (t == 0) {
      s = 0ull;
      for (int w = 0; w < W; ++w) s += red[w];
      const float l = vf_value(lo[A.drafted[(int64_t)b * A.k + r]]);  // (a token of the vocabulary: its weight is not 0)
      if (!vf_less(A.u[(int64_t)b * K1 + r], rowq[r], s, fx_weight(l, m, sc, tab))) kept = r;
    }
    __syncthreads();
  }
  const int a = min(kept, n);      // drafts kept; the token is drawn from row a
  const float M = rowm[a];
  const T *lr = (const T *)A.logits + ((int64_t)b * K1 + a) * A.ld;
  // what the sequence's last CTA will need: the proposal for row a (q = 1 of the draft
  // itself, or the candidates), its tokens' logits, in warp 0; the drafts
  const int ncand = greedy || a >= n ? 0 : A.top > 0 ? A.top : 1;
  uint32_t cx = VF_NONE;
  float cq = 0.f, cl = -INFINITY;
  if (t < ncand) {
    const int64_t o = ((int64_t)b * A.k + a) * A.top + t;
    cx = A.top > 0 ? A.cand[o] : A.drafted[(int64_t)b * A.k + a];
    cq = A.top > 0 ? fmaxf(A.cand_q[o], 0.f) : 1.f;
    if (cx < (uint32_t)A.vocab) cl = vf_value(lr[cx]);
  }
  const uint32_t draft = t < a ? A.drafted[(int64_t)b * A.k + t] : VF_NONE;
  uint32_t token = VF_NONE;        // no token has a probability
  if (greedy) {
    if (M > -INFINITY) token = (uint32_t)rowi[a];
  } else {
    // this CTA's chunks' weights, a run a warp; the next chunk's logits are on their way
    // meanwhile
    unsigned long long *cs = A.csum + (int64_t)b * A.nruns;
    const int c1 = min((chunk + 1) * A.per_cta, (A.nruns + W - 1) / W);
    T x[2][PER];
    auto load = [&](int c, T(&v)[PER]) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = c * VF_CHUNK + warp * VF_RUN + i * 32 + lane;
        v[i] = c < c1 && e < A.vocab ? lr[e] : (T)(-INFINITY);
      }
    };
    auto sum = [&](int c, const T(&v)[PER]) {
      unsigned long long s = 0ull;
#pragma unroll
      for (int i = 0; i < PER; ++i) s += fx_weight(vf_value(v[i]), M, sc, tab);
      s = vf_warp_sum(s);
      if (lane == 0 && c * W + warp < A.nruns) cs[c * W + warp] = s;
    };
    int c = chunk * A.per_cta;
    load(c, x[0]);
    for (; c < c1; c += 2) {
      load(c + 1, x[1]);
      sum(c, x[0]);
      load(c + 2, x[0]);
      if (c + 1 < c1) sum(c + 1, x[1]);
    }
    if (lane == 0) __threadfence();
    __syncthreads();
    if (t == 0) {
      last = atomicAdd(A.ticket + b, 1u) == gridDim.x - 1;
      pick = 0;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    // the sequence's last CTA: the sum of the row (a thread's runs are consecutive),
    // then the proposal's part of it
    const volatile unsigned long long *vs = cs;
    const int per = (A.nruns + VS_THREADS - 1) / VS_THREADS;  // at most 32
    unsigned long long own = 0ull;
#pragma unroll 4
    for (int i = 0; i < per; ++i) {
      const int r = t * per + i;
      if (r < A.nruns) own += vs[r];
    }
    unsigned long long cut = 0ull;   // warp 0: what a lane's candidate takes from p
    if (warp == 0 && ncand > 0) {
      // equal candidates' probabilities are added up, and count at the first of them
      const unsigned same = __match_any_sync(0xffffffffu, cx);
      if (__any_sync(0xffffffffu, lane < ncand && same != (1u << lane))) {
        const float q = cq;
        cq = 0.f;
        for (int i = 0; i < ncand; ++i) {
          const float qi = __shfl_sync(0xffffffffu, q, i);
          if (same >> i & 1) cq += qi;
        }
      }
      if (cx < (uint32_t)A.vocab && (same & ((1u << lane) - 1)) == 0u) cut = fx_weight(cl, M, sc, tab);
      else cx = VF_NONE;
    }
    unsigned long long Z, run = vf_scan(own, red, Z);
    if (ncand > 0) {
      if (warp == 0) {
        const unsigned long long qz = fx_mul(cq, Z);
        cut = cut < qz ? cut : qz;
        if (cx != VF_NONE) atomicAdd(&sub[cx / VF_RUN / per], cut);
        const unsigned long long all = vf_warp_sum(cut);
        if (all == Z) {
          cut = 0ull;                // nothing is left of p: drawn from p itself
          cx = VF_NONE;
        }
        if (lane == 0) taken = all;
      }
      __syncthreads();
      if (taken != Z) {
        own -= sub[t];
        run = vf_scan(own, red, Z);
      }
    }
    if (Z > 0ull) {
      // the run in which the cumulative sum passes the target: its thread, then the
      // run among the thread's, then the token in the run
      const unsigned long long goal = fx_target(u_last, Z);
      if (run - own <= goal && goal < run) {
        owner = t;
        base = run - own;
      }
      if (t < VF_RUN) sub[t] = 0ull;
      __syncthreads();
      if (warp == 0) {
        const int r = owner * per + lane;
        unsigned long long v = lane < per && r < A.nruns ? vs[r] : 0ull;
        for (int i = 0; i < ncand; ++i) {
          const uint32_t ci = __shfl_sync(0xffffffffu, cx, i);
          const unsigned long long w = __shfl_sync(0xffffffffu, cut, i);
          if (ci != VF_NONE && ci / VF_RUN == (uint32_t)r) v -= w;
        }
        unsigned long long end = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned long long w = __shfl_up_sync(0xffffffffu, end, o);
          if (lane >= o) end += w;
        }
        end += base;
        const unsigned hit = __ballot_sync(0xffffffffu, end - v <= goal && goal < end);
        const int at = __ffs(hit) - 1;
        const int p = owner * per + at;
        if (lane == at) target = goal - (end - v);
        if (lane == 0) pick = p;
        if (cx != VF_NONE && cx / VF_RUN == (uint32_t)p) sub[cx % VF_RUN] = cut;
      }
      __syncthreads();
      const int p0 = pick * VF_RUN;
      unsigned long long mine = 0ull, all;
      if (t < VF_RUN && p0 + t < A.vocab) mine = fx_weight(vf_value(lr[p0 + t]), M, sc, tab) - sub[t];
      const unsigned long long end = vf_scan(mine, red, all);
      if (end - mine <= target && target < end) pick = p0 + t;
      __syncthreads();
      token = (uint32_t)pick;
    }
  }
  if (t <= A.k)
    A.tokens[(int64_t)b * K1 + t] = t == a ? token : draft;
  if (t == 0) A.accepted[b] = a;
}

static size_t vf_bytes(int64_t batch, int64_t k, int64_t vocab, int &nparts, int &nruns) {
  nparts = (int)((vocab + 7 + VF_PART - 1) / VF_PART);  // up to 7 values before a row's aligned address
  nruns = (int)((vocab + VF_RUN - 1) / VF_RUN);
  return (size_t)(batch * (k + 1) * nparts * 16 + batch * nruns * 8 + (batch * 4 + 15) / 16 * 16);
}

template <typename T>
static cudaError_t launch_verify(const VfArgs &A, cudaStream_t st) {
  cudaError_t e = launch_pdl(k_verify_stats<T>, dim3(A.nparts, A.batch * (A.k + 1)), dim3(VF_THREADS), 0, st, 1, A);
  if (e != cudaSuccess) return e;
  const int chunks = (A.vocab + VF_CHUNK - 1) / VF_CHUNK;
  return launch_pdl(k_verify_sample<T>, dim3((chunks + A.per_cta - 1) / A.per_cta, A.batch), dim3(VS_THREADS), 0, st, 1,
                    A);
}

}  // namespace dfl

extern "C" size_t dflash_verify_workspace_bytes(int32_t batch, int32_t k, int32_t vocab) {
  if (batch < 1 || k < 0 || k >= dfl::VF_ROWS || vocab < 1 || vocab > (1 << 21) || (int64_t)batch * (k + 1) > 65535)
    return 0;
  int a, b;
  return dfl::vf_bytes(batch, k, vocab, a, b);
}

extern "C" int dflash_verify(int32_t batch, int32_t k, int32_t vocab, const void *logits, int32_t dtype, int64_t ld,
                             const uint32_t *drafted, const int32_t *n_drafted, const uint32_t *cand,
                             const float *cand_q, int32_t top, const float *temperature, const float *uniforms,
                             int32_t *accepted, uint32_t *tokens, void *workspace, size_t workspace_bytes,
                             void *stream) {
  using namespace dfl;
  const size_t need = dflash_verify_workspace_bytes(batch, k, vocab);
  if (need == 0)
    return dflash_fail(DFLASH_E_ARG, "verify: batch >= 1, 0 <= k <= 255, vocab 1..2,097,152, batch * (k + 1) <= 65,535");
  if (dtype != DFLASH_F32 && dtype != DFLASH_F16 && dtype != DFLASH_BF16)
    return dflash_fail(DFLASH_E_ARG, "verify: dtype must be DFLASH_F32, DFLASH_F16 or DFLASH_BF16");
  if (!logits || (k > 0 && !drafted) || !uniforms || !accepted || !tokens)
    return dflash_fail(DFLASH_E_ARG, "verify: null pointer");
  if ((uintptr_t)logits % (dtype == DFLASH_F32 ? 4 : 2)) return dflash_fail(DFLASH_E_ARG, "verify: misaligned logits");
  if (ld < vocab) return dflash_fail(DFLASH_E_ARG, "verify: a row stride below vocab");
  if (top < 0 || top > VF_TOP) return dflash_fail(DFLASH_E_ARG, "verify: top must be 0..32");
  if (top > 0 && k > 0 && (!cand || !cand_q)) return dflash_fail(DFLASH_E_ARG, "verify: null candidates");
  for (const void *p : {(const void *)drafted, (const void *)n_drafted, (const void *)cand, (const void *)cand_q,
                        (const void *)temperature, (const void *)uniforms, (const void *)accepted, (const void *)tokens})
    if ((uintptr_t)p & 3) return dflash_fail(DFLASH_E_ARG, "verify: misaligned pointer");
  if (!workspace || ((uintptr_t)workspace & 15)) return dflash_fail(DFLASH_E_ARG, "verify: null or misaligned workspace");
  if (workspace_bytes < need)
    return dflash_fail(DFLASH_E_CAPACITY, "verify: workspace smaller than dflash_verify_workspace_bytes");
  VfArgs A{};
  vf_bytes(batch, k, vocab, A.nparts, A.nruns);
  A.logits = logits, A.ld = ld;
  A.batch = batch, A.k = k, A.vocab = vocab, A.top = top;
  A.drafted = drafted, A.n_drafted = n_drafted, A.cand = cand, A.cand_q = cand_q;
  A.temperature = temperature, A.u = uniforms;
  A.accepted = accepted, A.tokens = tokens;
  A.part = (float4 *)workspace;
  A.csum = (unsigned long long *)(A.part + (size_t)batch * (k + 1) * A.nparts);
  A.ticket = (unsigned *)(A.csum + (size_t)batch * A.nruns);
  // every CTA decides for its sequence: two CTAs an SM, then more chunks each
  const int64_t chunks = (int64_t)batch * ((vocab + VF_CHUNK - 1) / VF_CHUNK);
  A.per_cta = (int)std::max<int64_t>(1, (chunks + 2 * device_sms() - 1) / (2 * device_sms()));
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = dtype == DFLASH_F32   ? launch_verify<float>(A, st)
                        : dtype == DFLASH_F16 ? launch_verify<__half>(A, st)
                                              : launch_verify<__nv_bfloat16>(A, st);
  if (e != cudaSuccess) return dflash_fail(DFLASH_E_CUDA, std::string("verify: ") + cudaGetErrorString(e));
  return DFLASH_OK;
}
