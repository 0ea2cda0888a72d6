// Row-wise operators of a decode step: the residual's addition with the norm, and the log probabilities of tokens.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <type_traits>

#include <cuda_fp8.h>

#include "async.cuh"

namespace pic {

namespace {

// ------------------------------------------------------------------ h += delta; y = RMSNorm(h) gain
//
// One CTA per row, the row in registers between its sum of squares and its output: every byte is read and written once.
// Thread i holds the float4s i, i + blockDim, ...: a warp's float4 is 128 columns, one group of 8-bit values, whose
// greatest is five shuffles away. Bound by HBM when rows are many (8192 rows of 4096: 69 us to fp16, 6.8 TB/s, as a copy; 70 to e4m3,
// 92 %: a reciprocal and five shuffles a group), by a launch and one round through memory when they are few (one row: 2.1 us).
constexpr int kXGroup = 128;
constexpr float kF16Top = 65504.f, kE4m3Top = 448.f;

struct AddNormArgs {
  int d4;                          // float4s of a row
  float* h;
  const float* delta;
  const float* gain;
  int64_t h_stride, delta_stride;
  float inv_d, eps;
  void* y;
  float* scales;
  int groups;
  unsigned* flag;
};

__device__ __forceinline__ bool beyond(float4 v, float top) {   // or NaN
  return !(fabsf(v.x) <= top) | !(fabsf(v.y) <= top) | !(fabsf(v.z) <= top) | !(fabsf(v.w) <= top);
}

// The sum over the CTA; the same bits in every thread. `part`: a float a warp.
__device__ __forceinline__ float cta_sum(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int w = 0; w < (int)blockDim.x >> 5; ++w) v += part[w];
  return v;
}
__device__ __forceinline__ float squares(float4 v) { return v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w; }
__device__ __forceinline__ float4 times(float4 v, float f) { return make_float4(v.x * f, v.y * f, v.z * f, v.w * f); }

// float4 i of row t's output is x r gain (the whole warp: a group's scale is its lanes'; `in`: i is within the row). True where the type
// does not hold it.
template <int OUT>
__device__ __forceinline__ bool put(const AddNormArgs& a, int t, int i, bool in, float4 x, float r) {
  const float4 g = in && a.gain ? reinterpret_cast<const float4*>(a.gain)[i] : make_float4(1.f, 1.f, 1.f, 1.f);
  const float4 y = make_float4(x.x * r * g.x, x.y * r * g.y, x.z * r * g.z, x.w * r * g.w);
  bool bad = false;
  if constexpr (OUT == PIC_E4M3) {
    float top = fmaxf(fmaxf(fabsf(y.x), fabsf(y.y)), fmaxf(fabsf(y.z), fabsf(y.w)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    bad = beyond(y, FLT_MAX);
    const float s = top / kE4m3Top;
    float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
    if (s >= 0x1p-120f) {                    // (the reciprocal is finite)
      q = times(y, 1.f / s);
    } else if (s > 0.f) {
      q = make_float4(y.x / s, y.y / s, y.z / s, y.w / s);
    }
    if (in) {
      const __nv_fp8x4_e4m3 c(q);          // saturates at 448
      reinterpret_cast<__nv_fp8x4_e4m3*>(a.y)[(size_t)t * a.d4 + i] = c;
      if ((threadIdx.x & 31) == 0) a.scales[(size_t)t * a.groups + i / 32] = s;
    }
  } else if constexpr (OUT == PIC_F16) {
    bad = beyond(y, kF16Top);
    const __half2 lo = __floats2half2_rn(y.x, y.y), hi = __floats2half2_rn(y.z, y.w);
    if (in)
      reinterpret_cast<uint2*>(a.y)[(size_t)t * a.d4 + i] =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  } else {
    if (in) reinterpret_cast<float4*>(a.y)[(size_t)t * a.d4 + i] = y;
  }
  return bad;
}

// A row whose squares fp32 does not hold: |h| from 2^56 on (or not finite), or below 2^-40 with no larger eps; m: the mean that came of
// it. With squares of h 2^-96 or h 2^95 the sum lies between 2^-108 and 2^124, and r h = (r 2^-64) (h 2^-32) or r (h 2^95) keeps the bits
// that its type has. The row is read again, so that other rows keep no registers for it.
template <int OUT>
__device__ __forceinline__ bool far_row(const AddNormArgs& a, int t, const float4* h, float m, float* part) {
  const bool large = !(m < 0x1p-96f);
  const float f = large ? 0x1p-96f : 0x1p95f;
  const int nt = blockDim.x;
  float ss = 0.f;
  for (int i = threadIdx.x; i < a.d4; i += nt) ss += squares(times(h[i], f));
  __syncthreads();                           // `part` has been read
  const float r = rsqrtf(cta_sum(ss, part) * a.inv_d + a.eps * f * f) * (large ? 0x1p-64f : 1.f);
  bool bad = false;
  for (int i0 = 0; i0 < a.d4; i0 += nt) {
    const int i = i0 + threadIdx.x;
    const bool in = i < a.d4;
    bad |= put<OUT>(a, t, i, in, in ? times(h[i], large ? 0x1p-32f : f) : make_float4(0.f, 0.f, 0.f, 0.f), r);
  }
  return bad;
}

// The same as a call, where its registers would be too many in the kernel itself (4096 rows of 8192 to fp16: 73 us for 83); a call costs short
// rows more (one row of 4096: 2.1 us for 2.2).
template <int OUT>
__device__ __noinline__ bool far_row_apart(const AddNormArgs& a, int t, const float4* h, float m, float* part) {
  return far_row<OUT>(a, t, h, m, part);
}

template <int OUT, int VPT>
__global__ void __launch_bounds__(1024) add_norm_kernel(const __grid_constant__ AddNormArgs a) {
  __shared__ float part[32];
  const int t = blockIdx.x, nt = blockDim.x;
  float4* h = reinterpret_cast<float4*>(a.h + t * a.h_stride);
  const float4* delta = reinterpret_cast<const float4*>(a.delta + t * a.delta_stride);
  float4 x[VPT];
  float ss = 0.f;
  pdl_enter();
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int i = threadIdx.x + v * nt;
    x[v] = i < a.d4 ? h[i] : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  if (a.delta) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int i = threadIdx.x + v * nt;
      if (i < a.d4) {
        const float4 u = delta[i];
        x[v] = make_float4(x[v].x + u.x, x[v].y + u.y, x[v].z + u.z, x[v].w + u.w);
        h[i] = x[v];
      }
    }
  }
#pragma unroll
  for (int v = 0; v < VPT; ++v) ss += squares(x[v]);
  const float m = cta_sum(ss, part) * a.inv_d + a.eps;
  bool bad = false;
  if (m >= 0x1p-96f && m <= FLT_MAX) {
    const float r = rsqrtf(m);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int i = threadIdx.x + v * nt;
      bad |= put<OUT>(a, t, i, i < a.d4, x[v], r);
    }
  } else {
    bad = VPT <= 2 ? far_row<OUT>(a, t, h, m, part) : far_row_apart<OUT>(a, t, h, m, part);
  }
  batch_flag(a.flag, bad ? kBatchRange : 0);
}

template <int OUT>
cudaError_t launch_add_norm(const AddNormArgs& a, int T, int sms, cudaStream_t st) {
  // Few rows: as many threads as there are float4s (one row of 4096: 2.1 us). Many: 512 at most, two to eight float4s a thread (8192 rows
  // of 4096 to e4m3: 70 us; 83 with 1024 threads, 81 with 256, 92 with 128).
  const int most = T <= 2 * sms ? 1024 : 512;
  int per = 1;
  while (per < 8 && (a.d4 + per - 1) / per > most) per *= 2;
  const int nt = ((a.d4 + per - 1) / per + 31) / 32 * 32;
  if (per == 1) return launch_dependent(add_norm_kernel<OUT, 1>, dim3(T), dim3(nt), 0, st, a);
  if (per == 2) return launch_dependent(add_norm_kernel<OUT, 2>, dim3(T), dim3(nt), 0, st, a);
  if (per == 4) return launch_dependent(add_norm_kernel<OUT, 4>, dim3(T), dim3(nt), 0, st, a);
  return launch_dependent(add_norm_kernel<OUT, 8>, dim3(T), dim3(nt), 0, st, a);
}

// ------------------------------------------------------------------ log probabilities
//
// One pass over the row: the CTAs of a cluster take a share of it each, which comes in chunks by bulk copies (the last warp), while
// the other warps read the chunk before. What a warp knows:
//   m = max;  n = how many are m;  rest = sum over the others of e^(x - m);  e = sum of e^(x - m) (x - m),
// so that log sum e^(x - m) = log n + log1p(rest / n) keeps its digits when one token has nearly all of the probability. m is the
// warp's, the others are each lane's; a chunk without a new maximum takes the short loop.
// Alternatives: the `top`-th greatest of 64 maxima, each of what a few threads have seen, is a bound that at least `top` logits reach, and
// a lane whose chunk reaches it puts what does on the CTA's list. The warps meet to set it at the first chunk, and at the next ones while it
// is -inf (ids masked in a run; the next chunk's logits would all reach it). Then one warp sets the bound anew (chunks 2, 4, 8 .. from there)
// from the maxima as it finds them: an old bound is as right, it lets more through. At the end the list is ordered by counting, for each,
// the greater ones. Where more reach the bound than the list holds (a run masked by a number, ties by the hundred, rising rows), the share is
// read again with the last bound; where that is still too many (a few threads' columns hold all that is great), its greatest are
// found one after the other. (1024 rows of 128256 with 32: 120 us; the first 8192 masked by -inf 118, by the lowest number 261; the
// share searched for one after the other in such rows 5610.)
// The CTAs of a cluster put their numbers and lists into the first one's shared memory, which joins them.
// Bound by HBM for fp32 logits (512 rows of 128256: 48 us, 5.5 TB/s, 81 % of a copy, without alternatives; 1024 rows with 5: 100 us), by
// instructions for 16-bit ones (1024 rows of bf16: 69 us, 56 %: conversion, exponential and two sums for every 2 bytes), and by its start,
// the list and the joins for few rows (one of 128256 with 20 alternatives: 11 us).
constexpr int kLpWarps = 8, kLpThreads = kLpWarps * 32, kLpChunk = 32768, kLpStages = 3, kMaxTop = 32, kLpList = 1024, kLpCluster = 8;
constexpr int kLpCtas = 2;                         // an SM
constexpr int kLpGroup = kLpThreads / 64;          // threads that share a maximum

struct LogprobArgs {
  int V, top;
  const void* logits;
  int64_t stride;
  const int* tokens;
  float* logprob;
  float* entropy;
  int* top_ids;
  float* top_logprobs;
  unsigned* flag;
};

template <typename T>
__device__ __forceinline__ float as_float(T x) {
  if constexpr (std::is_same<T, float>::value) return x;
  else if constexpr (std::is_same<T, __half>::value) return __half2float(x);
  else return __bfloat162float(x);
}
// The values of 16 bytes
template <typename T>
__device__ __forceinline__ void unpack(uint4 u, float* x) {
  const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same<T, float>::value) {
      x[i] = __uint_as_float(w[i]);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {   // NaN if one of them is
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// two fp32 operations at once
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(r))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(r))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(r))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Order of the alternatives as that of an unsigned: falling logits (-0 with 0), then rising ids. 0: none.
using Key = unsigned long long;
__device__ __forceinline__ Key order_key(float x, int id) {
  const unsigned u = __float_as_uint(x + 0.f);
  return (Key)(u >> 31 ? ~u : u | 0x80000000u) << 32 | (0xffffffffu - (unsigned)id);
}
__device__ __forceinline__ float key_logit(Key k) {
  const unsigned u = (unsigned)(k >> 32);
  return __uint_as_float(u >> 31 ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ int key_id(Key k) { return (int)(0xffffffffu - (unsigned)k); }

// What is known of a part of the row.
struct LpPart {
  float m, n, rest, e;       // -inf, 0, 0, 0 without a token
};
__device__ __forceinline__ LpPart join(const LpPart& a, const LpPart& b) {
  const LpPart &hi = a.m >= b.m ? a : b, &lo = a.m >= b.m ? b : a;
  LpPart r = hi;
  if (lo.m == hi.m) {
    r.n += lo.n;
    r.rest += lo.rest;
    r.e += lo.e;
  } else if (lo.n + lo.rest > 0.f) {
    const float d = lo.m - hi.m, f = ex2(d * kLog2e), l = lo.n + lo.rest;
    r.rest += f * l;
    r.e += f * (lo.e + l * fmaxf(d, -1000.f));     // (f is 0 there)
  }
  return r;
}
__device__ __forceinline__ LpPart join_lanes(LpPart p, int width) {
  for (int o = width / 2; o > 0; o >>= 1) {
    LpPart q;
    q.m = __shfl_xor_sync(0xffffffffu, p.m, o);
    q.n = __shfl_xor_sync(0xffffffffu, p.n, o);
    q.rest = __shfl_xor_sync(0xffffffffu, p.rest, o);
    q.e = __shfl_xor_sync(0xffffffffu, p.e, o);
    p = join(p, q);
  }
  return p;
}

struct LpShared {
  Key list[kLpList];                 // candidates
  Key joined[kLpCluster * kMaxTop];  // the cluster's lists
  Key top[kMaxTop];                  // the greatest, in order; 0 behind them
  Key warp_key[kLpWarps];
  LpPart part[kLpWarps];
  LpPart all[kLpCluster];            // of the CTAs
  int bad[kLpCluster];
  uint64_t full[kLpStages], empty[kLpStages];
  float group[64];                   // maxima of a few threads
  float bound;
  int count;
  unsigned abort;
};
__device__ __forceinline__ void lp_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kLpThreads) : "memory"); }   // of the warps that read

// the same, and whether one of their threads says so
__device__ __forceinline__ bool lp_sync_or(bool x) {
  uint32_t any;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
               : "=r"(any)
               : "r"((uint32_t)x), "n"(kLpThreads)
               : "memory");
  return any != 0;
}

// The `top` greatest keys of list[0 .. n) in order into s.top (they are distinct, but for 0: none).
__device__ __noinline__ void lp_order(LpShared& s, const Key* list, int n, int top) {
  if ((int)threadIdx.x < top) s.top[threadIdx.x] = 0;
  lp_sync();
  for (int i0 = 0; i0 < n; i0 += kLpThreads / 4) {   // four threads a key
    const int i = i0 + threadIdx.x / 4;
    const Key k = i < n ? list[i] : 0;
    int before = 0;
    for (int j = threadIdx.x % 4; j < n; j += 4) before += list[j] > k;
    before += __shfl_xor_sync(0xffffffffu, before, 1);
    before += __shfl_xor_sync(0xffffffffu, before, 2);
    if (k != 0 && threadIdx.x % 4 == 0 && before < top) s.top[before] = k;
  }
  lp_sync();
}

// A candidate (their order in the list does not matter). What the list does not hold is counted.
__device__ __forceinline__ void lp_push(LpShared& s, float x, int id) {
  const int at = atomicAdd(&s.count, 1);
  if (at < kLpList) s.list[at] = order_key(x, id);
}

// The `top`-th greatest of the maxima, by one warp: each lane counts, for two of them, the greater ones.
__device__ __forceinline__ void lp_bound(LpShared& s, int top) {
  const int lane = threadIdx.x & 31;
  const volatile float* group = s.group;           // (others write while this reads: any mixture will do)
  const float a = group[lane], b = group[lane + 32];
  int na = 0, nb = 0;
#pragma unroll 8
  for (int j = 0; j < 32; ++j) {
    const float x = __shfl_sync(0xffffffffu, a, j), y = __shfl_sync(0xffffffffu, b, j);
    na += (x > a || (x == a && j < lane)) + (y > a);
    nb += (x >= b) + (y > b || (y == b && j < lane));
  }
  if (na == top - 1) s.bound = a;
  if (nb == top - 1) s.bound = b;
}

// The candidates among the n vectors from `from` on, whose first element is token id0, once more, by the bound that is known in the end: the
// logits above it, and each warp's first `top` of those that equal it (it goes through them in the order of their ids).
template <typename T>
__device__ __forceinline__ void lp_again(LpShared& s, int top, const uint4* from, int n, int id0) {
  constexpr int E = 16 / sizeof(T), U = 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  lp_sync();                                       // (the count has been read)
  if (warp == 0) lp_bound(s, top);
  if (threadIdx.x == 0) s.count = 0;
  lp_sync();
  const float bound = s.bound;
  int tied = 0;
  for (int i0 = warp * 32; i0 < n; i0 += U * kLpThreads) {
    uint4 vec[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kLpThreads + lane;
      vec[u] = from[min(i, n - 1)];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kLpThreads + lane;
      float x[E];
      unpack<T>(vec[u], x);
      unsigned above = 0, ties = 0;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        above |= (unsigned)(x[e] > bound) << e;
        ties |= (unsigned)(x[e] == bound) << e;
      }
      if (i >= n) above = ties = 0;
      for (; above; above &= above - 1) {
        const int e = __ffs(above) - 1;
        lp_push(s, as_float(reinterpret_cast<const T*>(from + i)[e]), id0 + i * E + e);
      }
      if (tied < top && bound > -INFINITY && __any_sync(0xffffffffu, ties)) {
        const int own = __popc(ties);
        int upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int before = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += before;
        }
        for (int nth = tied + upto - own; ties && nth < top; ties &= ties - 1, ++nth) lp_push(s, bound, id0 + i * E + __ffs(ties) - 1);
        tied += __shfl_sync(0xffffffffu, upto, 31);
      }
    }
  }
}

// The `top` greatest of row[i0 .. i1) into s.top, one after the other.
template <typename T>
__device__ __forceinline__ void lp_one_by_one(LpShared& s, int top, const T* row, int64_t i0, int64_t i1) {
  Key before = ~0ull;
  for (int j = 0; j < top; ++j) {
    Key best = 0;
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kLpThreads) {
      const float x = as_float(row[i]);
      if (x > -INFINITY) {
        const Key k = order_key(x, (int)i);
        if (k < before && k > best) best = k;
      }
    }
    for (int o = 16; o > 0; o >>= 1) {
      const Key k = __shfl_xor_sync(0xffffffffu, best, o);
      best = k > best ? k : best;
    }
    lp_sync();
    if (threadIdx.x % 32 == 0) s.warp_key[threadIdx.x / 32] = best;
    lp_sync();
    for (int w = 0; w < kLpWarps; ++w) best = s.warp_key[w] > best ? s.warp_key[w] : best;
    if (threadIdx.x == 0) s.top[j] = best;         // 0 when there are no more
    before = best;
  }
  lp_sync();
}

// The same where the list could not hold all candidates. The CTA's share: logits i0 .. id0, n vectors from id0 on, and `tail` more.
template <typename T>
__device__ __noinline__ void lp_crowded(LpShared& s, int top, const T* row, int i0, int id0, int n, int tail) {
  constexpr int E = 16 / sizeof(T);
  lp_again<T>(s, top, reinterpret_cast<const uint4*>(row + id0), n, id0);
  const int behind = id0 + n * E, e = threadIdx.x, i = e < E ? (e < id0 - i0 ? i0 + e : -1) : e < 2 * E && e - E < tail ? behind + e - E : -1;
  if (i >= 0) {
    const float x = as_float(row[i]);
    if (x > -INFINITY) lp_push(s, x, i);
  }
  lp_sync();
  if (s.count <= kLpList) lp_order(s, s.list, s.count, top);
  else lp_one_by_one(s, top, row, i0, behind + tail);
}

template <typename T>
__device__ __forceinline__ T* remote(T* p, unsigned rank) {   // of another CTA of the cluster
  T* r;
  asm("mapa.u64 %0, %1, %2;" : "=l"(r) : "l"(p), "r"(rank));
  return r;
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads + 32, kLpCtas) logprob_kernel(LogprobArgs a) {
  constexpr int E = 16 / sizeof(T), kVecs = kLpChunk / 16, NV = kVecs / kLpThreads, kEach = NV * E;   // elements of a vector; vectors of a chunk; a thread's
  static_assert(kEach <= 64, "a bit for each");
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ LpShared s;
  unsigned ctas, rank;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ctas));
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int t = blockIdx.x / ctas, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* row = (const T*)a.logits + t * a.stride;
  pdl_wait();
  const int token = a.tokens ? __ldg(a.tokens + t) : 0;
  if (token < 0 || token >= a.V) {                 // the whole cluster
    if (tid == 0 && rank == 0 && token != -1) batch_flag(a.flag, kBatchBadToken);
    return;
  }
  if (ctas > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;");   // (waited for before another CTA's memory is written)
  // the row: up to E - 1 logits before the first 16-byte border, whole vectors, up to E - 1 behind them
  const int head = min(a.V, (int)((16 - ((uintptr_t)row & 15)) % 16 / sizeof(T)));
  const int vectors = (a.V - head) / E, tail = a.V - head - vectors * E;
  const int chunks = (vectors + kVecs - 1) / kVecs;
  const int c0 = (int)((int64_t)chunks * rank / ctas), c1 = (int)((int64_t)chunks * (rank + 1) / ctas);
  if (tid == 0) {
    s.count = 0;
    s.bad[0] = 0;
    s.abort = 0;
    s.bound = -INFINITY;
    for (int i = 0; i < kLpStages; ++i) {
      mbar_init(smem_u32(s.full + i), 1);
      mbar_init(smem_u32(s.empty + i), kLpWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  __syncthreads();
  bool bad = false;
  if (warp == kLpWarps) {
    if (lane == 0) {
      uint64_t policy;
      asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
      int issued = 0;
      for (int c = c0; c < c1; ++c, ++issued) {
        const int st = issued % kLpStages;
        if (!mbar_wait(smem_u32(s.empty + st), (issued / kLpStages & 1) ^ 1, &s.abort, a.flag)) break;
        const uint32_t bytes = 16u * min(kVecs, vectors - c * kVecs), fb = smem_u32(s.full + st);
        mbar_expect_tx(fb, bytes);
        bulk_load(smem_u32(ring) + st * kLpChunk, (const uint8_t*)(row + head) + (int64_t)c * kLpChunk, bytes, fb, policy);
      }
      for (int j = max(0, issued - kLpStages); j < issued; ++j)   // copies under way land before the CTA ends
        mbar_settle(smem_u32(s.full + j % kLpStages), (uint32_t)((j / kLpStages) & 1), a.flag);
    }
  } else {
    LpPart mine{-INFINITY, 0.f, 0.f, 0.f};         // m the warp's
    float seen = -INFINITY;                        // this thread's maximum
    bool landed = true;                            // (after a wait that was given up chunks count as empty: the barriers below still meet)
    int settled = 0;                               // chunks since there is a bound
    // a new maximum of the warp
    auto raise = [&](float top1) {
      if (!__any_sync(0xffffffffu, top1 > mine.m)) return;
      float m = top1;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const LpPart none{m, 0.f, 0.f, 0.f};
      mine = join(none, mine);
    };
    if (warp == 0 && (rank == 0 || rank == ctas - 1)) {   // the row's ends
      const int i = lane < E ? (rank == 0 && lane < head ? lane : -1) : rank == ctas - 1 && lane - E < tail ? a.V - tail + lane - E : -1;
      float x = i >= 0 ? as_float(row[i]) : -INFINITY;
      if (x != x || x == INFINITY) bad = true;
      if (x != x) x = -INFINITY;
      raise(x == INFINITY ? -INFINITY : x);
      if (x > -INFINITY && mine.m > -INFINITY) {
        const float d = fmaxf(x - mine.m, -1000.f), p = ex2(d * kLog2e);
        if (x == mine.m) mine.n = 1.f;
        else mine.rest = p;
        mine.e = p * d;
      }
      if (a.top > 0 && x > -INFINITY) lp_push(s, x, i);
    }
    int st = 0;
    uint32_t ph = 0;
    for (int c = c0; c < c1; ++c) {
      landed = landed && warp_wait(smem_u32(s.full + st), ph, &s.abort, a.flag);
      const int n_vec = min(kVecs, vectors - c * kVecs);
      const uint8_t* part = ring + st * kLpChunk + tid * 16;   // this thread's vectors are kLpThreads apart
      const int own = landed && tid < n_vec ? (n_vec - tid - 1) / kLpThreads + 1 : 0;
      float x[kEach], top1 = -INFINITY;
      if (own == NV) {
#pragma unroll
        for (int v = 0; v < NV; ++v) unpack<T>(*reinterpret_cast<const uint4*>(part + v * (kLpThreads * 16)), x + v * E);
      } else {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int e = 0; e < E; ++e) x[v * E + e] = -INFINITY;
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if (v < own) unpack<T>(*reinterpret_cast<const uint4*>(part + v * (kLpThreads * 16)), x + v * E);
      }
#pragma unroll
      for (int v = 0; v < kEach; v += 4) top1 = max_nan(top1, max_nan(x[v], x[v + 1], x[v + 2]), x[v + 3]);
      auto again = [&](int j) { return as_float(reinterpret_cast<const T*>(part + j / E * (kLpThreads * 16))[j % E]); };   // x[j]
      if (top1 != top1 || top1 == INFINITY) {      // the row's numbers are NaN; its order goes on
        bad = true;
        top1 = -INFINITY;
#pragma unroll 1
        for (int j = 0; j < own * E; ++j) top1 = fmaxf(top1, again(j));
      }
      raise(top1 == INFINITY ? -INFINITY : top1);
      if (mine.m > -INFINITY) {
        // in the log2 domain, two at a time; of a chunk that holds m (few do) the logits that are m count apart
        const bool holds = __any_sync(0xffffffffu, top1 == mine.m);
        const float2 from = make_float2(-mine.m, -mine.m), unit = make_float2(kLog2e, kLog2e);
        float2 rest = make_float2(0.f, 0.f), e = rest;
        unsigned n = 0;
#pragma unroll
        for (int j = 0; j < kEach; j += 2) {
          float2 d = mul2(add2(make_float2(x[j], x[j + 1]), from), unit);
          d = make_float2(fmaxf(d.x, -1500.f), fmaxf(d.y, -1500.f));   // (-inf: p is 0)
          float2 p = make_float2(ex2(d.x), ex2(d.y));
          if (holds) {
            n += (x[j] == mine.m) + (x[j + 1] == mine.m);
            p = make_float2(x[j] == mine.m ? 0.f : p.x, x[j + 1] == mine.m ? 0.f : p.y);
          }
          rest = add2(rest, p);
          e = fma2(p, d, e);
        }
        mine.n += (float)n;
        mine.rest += rest.x + rest.y;
        mine.e += (e.x + e.y) * kLn2;
      }
      if (a.top > 0) {
        seen = fmaxf(seen, top1);
        float g = seen;
#pragma unroll
        for (int o = 1; o < kLpGroup; o <<= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
        if (lane % kLpGroup == 0) const_cast<volatile float*>(s.group)[tid / kLpGroup] = g;
        if (settled == 0) {                        // (the same in every warp)
          if (lp_sync_or(top1 > -INFINITY)) {
            if (warp == 0) lp_bound(s, a.top);
            lp_sync();
            settled = *const_cast<volatile float*>(&s.bound) > -INFINITY;
          }
        } else {
          if ((settled & (settled + 1)) == 0 && __popc(settled) % kLpWarps == warp) {   // chunks 2, 4, 8 ..
            __syncwarp();
            lp_bound(s, a.top);
          }
          ++settled;
        }
        const float bound = *const_cast<volatile float*>(&s.bound);
        if (top1 >= bound && top1 > -INFINITY) {   // few lanes, of one or two logits mostly
          unsigned long long reach = 0;
#pragma unroll
          for (int j = 0; j < kEach; ++j) reach |= (unsigned long long)(x[j] >= bound) << j;
          if (*const_cast<volatile int*>(&s.count) > kLpList) reach = 0;   // they will be found once more anyway
          for (; reach; reach &= reach - 1) {
            const int j = __ffsll(reach) - 1;
            const float y = again(j);
            if (j < own * E && y > -INFINITY) lp_push(s, y, head + (c * kVecs + j / E * kLpThreads + tid) * E + j % E);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(s.empty + st));
      if (++st == kLpStages) st = 0, ph ^= 1;
    }
    // the CTA's numbers and list
    const LpPart part = join_lanes(mine, 32);
    if (lane == 0) s.part[warp] = part;
    lp_sync();
    if (a.top > 0) {
      if (s.count <= kLpList) lp_order(s, s.list, s.count, a.top);
      else lp_crowded(s, a.top, row, rank == 0 ? 0 : head + c0 * (kVecs * E), head + c0 * (kVecs * E), min(vectors, c1 * kVecs) - c0 * kVecs, rank == ctas - 1 ? tail : 0);
    }
  }
  bad = __syncthreads_or(bad);
  if (ctas > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // every CTA has begun
  if (tid == 0) {
    LpPart part = s.part[0];
#pragma unroll
    for (int w = 1; w < kLpWarps; ++w) part = join(part, s.part[w]);
    remote(s.all, 0)[rank] = part;
    remote(s.bad, 0)[rank] = bad;
  }
  if (tid < a.top) remote(s.joined, 0)[rank * a.top + tid] = s.top[tid];
  if (ctas > 1) cluster_sync();
  else __syncthreads();
  if (rank != 0 || warp >= kLpWarps) return;
  // every thread: the row's numbers
  LpPart all = s.all[0];
  bad = s.bad[0] != 0;
  for (unsigned c = 1; c < ctas; ++c) {
    all = join(all, s.all[c]);
    bad |= s.bad[c] != 0;
  }
  const float lose = all.n > 0.f ? logf(all.n) + log1pf(all.rest / all.n) : 0.f;   // log sum e^(x - m)
  const float from = all.n > 0.f ? all.m : 0.f;
  if (tid == 0) {
    if (a.tokens) a.logprob[t] = bad ? NAN : as_float(row[token]) - from - lose;
    if (a.entropy) a.entropy[t] = bad ? NAN : all.n > 0.f ? lose - all.e / (all.n + all.rest) : 0.f;
  }
  if (a.top == 0) return;
  if (ctas > 1) lp_order(s, s.joined, (int)ctas * a.top, a.top);
  if (warp > 0) return;
  const Key k = lane < a.top ? s.top[lane] : 0;
  const int have = __popc(__ballot_sync(0xffffffffu, k != 0));
  int id = key_id(k);
  float lp = key_logit(k) - from - lose;
  if (have < a.top) {                              // tokens without probability, in the order of their ids
    int found = have;
    for (int i0 = 0; i0 < a.V && found < a.top; i0 += 32) {
      const float x = lane < a.V - i0 ? as_float(row[i0 + lane]) : 0.f;
      const unsigned some = __ballot_sync(0xffffffffu, !(x > -INFINITY));
      const int nth = lane - found;                // this lane's place wants the nth of them
      if (nth >= 0 && nth < __popc(some)) {
        unsigned left = some;
        for (int q = 0; q < nth; ++q) left &= left - 1;
        id = i0 + __ffs(left) - 1;
        lp = -INFINITY;
      }
      found += __popc(some);
    }
  }
  if (lane < a.top) {
    a.top_ids[(size_t)t * a.top + lane] = id;
    a.top_logprobs[(size_t)t * a.top + lane] = bad ? NAN : lp;
  }
}

template <typename T>
pic_status launch_logprob(const LogprobArgs& a, int rows, int slots, int dev, cudaStream_t st) {
  // CTAs of a row: the fewest turns of all CTAs over their chunks, each with its start and end (as long as three chunks)
  const int64_t chunks = std::max<int64_t>(1, ((int64_t)a.V * sizeof(T) + kLpChunk - 1) / kLpChunk);
  int ctas = 1;
  int64_t least = INT64_MAX;
  for (int c = 1; c <= std::min<int64_t>(chunks, kLpCluster); ++c) {
    const int64_t cost = ((int64_t)rows * c + slots - 1) / slots * ((chunks + c - 1) / c + 3);
    if (cost < least) least = cost, ctas = c;
  }
  static SharedMemory<logprob_kernel<T>> memory;
  PIC_CUDA(memory.allow(dev, kLpStages * kLpChunk));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)rows * ctas);
  cfg.blockDim = dim3(kLpThreads + 32);
  cfg.dynamicSmemBytes = kLpStages * kLpChunk;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  PIC_CUDA(cudaLaunchKernelEx(&cfg, logprob_kernel<T>, a));
  return PIC_OK;
}

bool misaligned(const void* p, unsigned to) { return ((uintptr_t)p & (to - 1)) != 0; }

}  // namespace

}  // namespace pic

using namespace pic;

extern "C" {

pic_status pic_op_add_rms_norm(int32_t out_dtype, int32_t T, int32_t d, float* h, int64_t h_stride, const float* delta,
                               int64_t delta_stride, const float* gain, float eps, void* y, float* scales,
                               pic_stream_t stream) {
  const bool e4m3 = out_dtype == PIC_E4M3;
  constexpr int64_t kMaxStride = (int64_t)1 << 38;
  if (T < 1 || d < 4 || d % 4 || !h || !y || !(eps >= 0.f) || (!e4m3 && out_dtype != PIC_F32 && out_dtype != PIC_F16) ||
      e4m3 != (scales != nullptr) || h_stride < d || h_stride % 4 || h_stride >= kMaxStride ||
      (delta && (delta_stride < d || delta_stride % 4 || delta_stride >= kMaxStride)))
    return fail(PIC_ERR_INVALID_ARG, "invalid norm arguments (d and strides multiples of 4, scales with 8-bit output)");
  if (d > 32768) return fail(PIC_ERR_UNSUPPORTED, "norm rows of more than 32768 values");
  if (misaligned(h, 16) || misaligned(delta, 16) || misaligned(gain, 16) || misaligned(y, 16) || misaligned(scales, 16))
    return fail(PIC_ERR_INVALID_ARG, "h, delta, gain, y and scales must be 16-byte aligned");
  const int groups = (d + kXGroup - 1) / kXGroup;
  const size_t h_bytes = 4 * ((size_t)(T - 1) * h_stride + d), y_bytes = (size_t)T * d * (e4m3 ? 1 : out_dtype == PIC_F16 ? 2 : 4);
  const size_t d_bytes = delta ? 4 * ((size_t)(T - 1) * delta_stride + d) : 0, s_bytes = scales ? (size_t)T * groups * 4 : 0;
  if (overlap(h, h_bytes, y, y_bytes) || (delta && (overlap(h, h_bytes, delta, d_bytes) || overlap(y, y_bytes, delta, d_bytes))) ||
      (gain && (overlap(gain, (size_t)d * 4, y, y_bytes) || overlap(gain, (size_t)d * 4, h, delta ? h_bytes : 0))) ||
      (scales && (overlap(scales, s_bytes, h, h_bytes) || overlap(scales, s_bytes, y, y_bytes) ||
                  (delta && overlap(scales, s_bytes, delta, d_bytes)) || (gain && overlap(scales, s_bytes, gain, (size_t)d * 4)))))
    return fail(PIC_ERR_INVALID_ARG, "h, delta, gain, y and scales must not overlap");
  AddNormArgs a{d / 4, h, delta, gain, h_stride, delta_stride, 1.f / d, eps, y, scales, groups, nullptr};
  pic_status e = batch_flag_address(&a.flag);
  if (e != PIC_OK) return e;
  int dev = 0;
  PIC_CUDA(cudaGetDevice(&dev));
  const int sms = device_sms(dev);
  cudaStream_t st = (cudaStream_t)stream;
  PIC_CUDA(e4m3                   ? launch_add_norm<PIC_E4M3>(a, T, sms, st)
           : out_dtype == PIC_F16 ? launch_add_norm<PIC_F16>(a, T, sms, st)
                                  : launch_add_norm<PIC_F32>(a, T, sms, st));
  return PIC_OK;
}

pic_status pic_op_token_logprobs(int32_t dtype, int32_t T, int32_t vocab, const void* logits, int64_t logits_stride,
                                 const int32_t* tokens, int32_t top, float* logprob, float* entropy, int32_t* top_ids,
                                 float* top_logprobs, pic_stream_t stream) {
  if (T < 1 || vocab < 1 || !logits || logits_stride < vocab || logits_stride >= (int64_t)1 << 38 || top < 0 ||
      top > kMaxTop || top > vocab || (tokens != nullptr) != (logprob != nullptr) || (top > 0) != (top_ids != nullptr) ||
      (top > 0) != (top_logprobs != nullptr) || (dtype != PIC_F32 && dtype != PIC_BF16 && dtype != PIC_F16))
    return fail(PIC_ERR_INVALID_ARG, "invalid token log probability arguments (top 0 to 32, at most the vocabulary; tokens with "
                                     "logprob, top_ids and top_logprobs with top)");
  const unsigned size = dtype == PIC_F32 ? 4 : 2;
  if (misaligned(logits, size) || misaligned(tokens, 4) || misaligned(logprob, 4) || misaligned(entropy, 4) ||
      misaligned(top_ids, 4) || misaligned(top_logprobs, 4))
    return fail(PIC_ERR_INVALID_ARG, "logits and outputs must be aligned to their types");
  const size_t in_bytes = ((size_t)(T - 1) * logits_stride + vocab) * size, row = (size_t)T * 4, tops = (size_t)T * top * 4;
  const void* outs[4] = {logprob, entropy, top_ids, top_logprobs};
  const size_t bytes[4] = {row, row, tops, tops};
  for (int i = 0; i < 4; ++i) {
    if (!outs[i]) continue;
    bool met = overlap(outs[i], bytes[i], logits, in_bytes) || (tokens && overlap(outs[i], bytes[i], tokens, row));
    for (int j = 0; j < i; ++j) met |= outs[j] && overlap(outs[i], bytes[i], outs[j], bytes[j]);
    if (met) return fail(PIC_ERR_INVALID_ARG, "outputs must not overlap logits, tokens or one another");
  }
  if (!logprob && !entropy && !top) return fail(PIC_ERR_INVALID_ARG, "token log probabilities: no output is asked for");
  if (T > INT_MAX / kLpCluster) return fail(PIC_ERR_CAPACITY, "token log probabilities: too many rows");
  LogprobArgs a{vocab, top, logits, logits_stride, tokens, logprob, entropy, top_ids, top_logprobs, nullptr};
  pic_status e = batch_flag_address(&a.flag);
  if (e != PIC_OK) return e;
  int dev = 0;
  PIC_CUDA(cudaGetDevice(&dev));
  const int sms = device_sms(dev);
  cudaStream_t st = (cudaStream_t)stream;
  return dtype == PIC_F32   ? launch_logprob<float>(a, T, kLpCtas * sms, dev, st)
         : dtype == PIC_F16 ? launch_logprob<__half>(a, T, kLpCtas * sms, dev, st)
                            : launch_logprob<__nv_bfloat16>(a, T, kLpCtas * sms, dev, st);
}

}  // extern "C"
