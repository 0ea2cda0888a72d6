// Row-wise operators of a decode step: the residual's addition with the norm, and the log probabilities of tokens.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <type_traits>

#include <cuda_fp8.h>

#include "batch_internal.cuh"

namespace pic {

namespace {

// ------------------------------------------------------------------ h += delta; y = RMSNorm(h) gain
//
// One CTA per row, the row in registers between its sum of squares and its output: every byte is read and written once.
// Thread i holds the float4s i, i + blockDim, ...: a warp's float4 is 128 columns, one group of 8-bit values, whose
// greatest is five shuffles away.
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

template <int OUT, int VPT>
__global__ void __launch_bounds__(1024) add_norm_kernel(AddNormArgs a) {
  __shared__ float part[32];
  const int t = blockIdx.x, nt = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float4* h = reinterpret_cast<float4*>(a.h + t * a.h_stride);
  const float4* delta = reinterpret_cast<const float4*>(a.delta + t * a.delta_stride);
  float4 x[VPT];
  float ss = 0.f;
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
  for (int v = 0; v < VPT; ++v) ss += x[v].x * x[v].x + x[v].y * x[v].y + x[v].z * x[v].z + x[v].w * x[v].w;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (lane == 0) part[warp] = ss;
  __syncthreads();
  ss = 0.f;
  for (int w = 0; w < nt >> 5; ++w) ss += part[w];
  const float r = rsqrtf(ss * a.inv_d + a.eps);
  bool bad = false;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int i = threadIdx.x + v * nt;
    const bool in = i < a.d4;
    const float4 g = in && a.gain ? reinterpret_cast<const float4*>(a.gain)[i] : make_float4(1.f, 1.f, 1.f, 1.f);
    const float4 y = make_float4(x[v].x * r * g.x, x[v].y * r * g.y, x[v].z * r * g.z, x[v].w * r * g.w);
    if constexpr (OUT == PIC_E4M3) {
      float top = fmaxf(fmaxf(fabsf(y.x), fabsf(y.y)), fmaxf(fabsf(y.z), fabsf(y.w)));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      bad |= beyond(y, FLT_MAX);
      const float s = top / kE4m3Top;
      float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s > 0.f) q = make_float4(y.x / s, y.y / s, y.z / s, y.w / s);
      if (in) {
        const __nv_fp8x4_e4m3 c(q);          // saturates at 448
        reinterpret_cast<__nv_fp8x4_e4m3*>(a.y)[(size_t)t * a.d4 + i] = c;
        if (lane == 0) a.scales[(size_t)t * a.groups + i / 32] = s;
      }
    } else if constexpr (OUT == PIC_F16) {
      bad |= beyond(y, kF16Top);
      const __half2 lo = __floats2half2_rn(y.x, y.y), hi = __floats2half2_rn(y.z, y.w);
      if (in)
        reinterpret_cast<uint2*>(a.y)[(size_t)t * a.d4 + i] =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    } else {
      if (in) reinterpret_cast<float4*>(a.y)[(size_t)t * a.d4 + i] = y;
    }
  }
  batch_flag(a.flag, bad ? kBatchRange : 0);
}

template <int OUT>
void launch_add_norm(const AddNormArgs& a, int T, cudaStream_t st) {
  const int per = a.d4 <= 1024 ? 1 : a.d4 <= 4096 ? 4 : 8;
  const int nt = ((a.d4 + per - 1) / per + 31) / 32 * 32;
  if (per == 1) add_norm_kernel<OUT, 1><<<T, nt, 0, st>>>(a);
  else if (per == 4) add_norm_kernel<OUT, 4><<<T, nt, 0, st>>>(a);
  else add_norm_kernel<OUT, 8><<<T, nt, 0, st>>>(a);
}

// ------------------------------------------------------------------ log probabilities

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

constexpr int kLogprobThreads = 256, kMaxTop = 32;

template <typename T>
__device__ __forceinline__ float as_float(T x) {
  if constexpr (std::is_same<T, float>::value) return x;
  else if constexpr (std::is_same<T, __half>::value) return __half2float(x);
  else return __bfloat162float(x);
}
// Order of the alternatives as that of an unsigned: falling logits (NaN with -inf, -0 with 0), then rising ids.
__device__ __forceinline__ unsigned long long order_key(float x, int id) {
  x = x != x ? -INFINITY : x + 0.f;
  const unsigned u = __float_as_uint(x);
  return (unsigned long long)(u >> 31 ? ~u : u | 0x80000000u) << 32 | (0xffffffffu - (unsigned)id);
}

template <typename T, typename F>
__device__ T block_reduce(T x, T* sh, F f) {
  for (int o = 16; o > 0; o >>= 1) x = f(x, __shfl_xor_sync(0xffffffffu, x, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
  __syncthreads();
  x = sh[0];
  for (int w = 1; w < kLogprobThreads / 32; ++w) x = f(x, sh[w]);
  return x;
}

template <typename T>
__global__ void __launch_bounds__(kLogprobThreads) logprob_kernel(LogprobArgs a) {
  __shared__ double shd[8];
  __shared__ unsigned long long shk[8];
  const int t = blockIdx.x;
  const T* x = (const T*)a.logits + t * a.stride;
  const int token = a.tokens ? a.tokens[t] : 0;
  if (a.tokens && (token < 0 || token >= a.V)) {
    if (threadIdx.x == 0 && token != -1) batch_flag(a.flag, kBatchBadToken);
    return;
  }
  double m = -INFINITY, bad = 0;
  for (int i = threadIdx.x; i < a.V; i += kLogprobThreads) {
    const float v = as_float(x[i]);
    if (v != v || v == INFINITY) bad = 1;
    else m = fmax(m, (double)v);
  }
  auto most = [](double p, double q) { return p > q ? p : q; };
  auto sum = [](double p, double q) { return p + q; };
  m = block_reduce(m, shd, most);
  bad = block_reduce(bad, shd, most);
  double l = 0, e = 0;
  if (m > -INFINITY)
    for (int i = threadIdx.x; i < a.V; i += kLogprobThreads) {
      const double y = (double)as_float(x[i]) - m;
      const double p = exp(y);
      l += p;
      e += p > 0 ? p * y : 0;
    }
  l = block_reduce(l, shd, sum);
  e = block_reduce(e, shd, sum);
  const double none = bad ? NAN : 0.0, lse = m > -INFINITY ? m + log(l) : 0.0;
  if (threadIdx.x == 0) {
    if (a.tokens) a.logprob[t] = (float)((double)as_float(x[token]) - lse + none);
    if (a.entropy) a.entropy[t] = (float)((m > -INFINITY ? log(l) - e / l : 0.0) + none);
  }
  unsigned long long before = ~0ull;
  for (int j = 0; j < a.top; ++j) {
    unsigned long long best = 0;
    for (int i = threadIdx.x; i < a.V; i += kLogprobThreads) {
      const unsigned long long k = order_key(as_float(x[i]), i);
      if (k < before && k > best) best = k;
    }
    before = block_reduce(best, shk, [](unsigned long long p, unsigned long long q) { return p > q ? p : q; });
    if (threadIdx.x == 0) {
      const int id = (int)(0xffffffffu - (unsigned)before);
      a.top_ids[(size_t)t * a.top + j] = id;
      a.top_logprobs[(size_t)t * a.top + j] = (float)((double)as_float(x[id]) - lse + none);
    }
  }
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
  cudaStream_t st = (cudaStream_t)stream;
  if (e4m3) launch_add_norm<PIC_E4M3>(a, T, st);
  else if (out_dtype == PIC_F16) launch_add_norm<PIC_F16>(a, T, st);
  else launch_add_norm<PIC_F32>(a, T, st);
  PIC_CUDA(cudaGetLastError());
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
  LogprobArgs a{vocab, top, logits, logits_stride, tokens, logprob, entropy, top_ids, top_logprobs, nullptr};
  pic_status e = batch_flag_address(&a.flag);
  if (e != PIC_OK) return e;
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == PIC_F32) logprob_kernel<float><<<T, kLogprobThreads, 0, st>>>(a);
  else if (dtype == PIC_F16) logprob_kernel<__half><<<T, kLogprobThreads, 0, st>>>(a);
  else logprob_kernel<__nv_bfloat16><<<T, kLogprobThreads, 0, st>>>(a);
  PIC_CUDA(cudaGetLastError());
  return PIC_OK;
}

}  // extern "C"
