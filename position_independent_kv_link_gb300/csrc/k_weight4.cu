// 4-bit weights with group scales: packing, unpacking, and the product of few rows with them.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <type_traits>

#include <cuda_fp8.h>

#include "batch_internal.cuh"
#include "weight4.cuh"

namespace pic {

namespace {

// ------------------------------------------------------------------ packing
//
// One CTA packs a tile; a thread holds 32 columns of a row (16 bytes of codes), the four threads of a row's 128 columns lie
// side by side, so that the extremes of a group of 64 or 128 are shuffles away.
constexpr int kPackThreads = 256;

template <typename T>
__device__ __forceinline__ void load32(const T* p, float* x) {   // 32 values, 16-byte aligned
  constexpr int E = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < 32; i += E) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p + i));
    const T* v = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int j = 0; j < E; ++j) {
      if constexpr (std::is_same<T, float>::value) x[i + j] = v[j];
      else if constexpr (std::is_same<T, __half>::value) x[i + j] = __half2float(v[j]);
      else x[i + j] = __bfloat162float(v[j]);
    }
  }
}

// The integer nearest to x / s (ties to even), decided exactly: the quotient in fp32 gives an integer k that may be off by
// one next to a border; x - k s is exact in fp32 (s has 11 bits, and x lies within 16 s), as is s / 2.
__device__ __forceinline__ float nearest_quotient(float x, float s) {
  float k = rintf(x / s);
  const float d = fmaf(-k, s, x), half = 0.5f * s;
  const bool odd = fmodf(k, 2.f) != 0.f;
  if (d > half || (d == half && odd)) k += 1.f;
  else if (d < -half || (d == -half && odd)) k -= 1.f;
  return k;
}

template <typename T>
__global__ void __launch_bounds__(kPackThreads) pack4_kernel(const T* __restrict__ W, uint8_t* __restrict__ out, W4Shape p,
                                                             unsigned* flag) {
  const int nt = blockIdx.x / p.k_tiles, kt = blockIdx.x % p.k_tiles;
  uint8_t* tile = out + (size_t)blockIdx.x * p.tile_bytes;
  const int per = kW4Cols / p.group;                   // groups of a tile's row
  const int lanes = p.group / 32;                      // threads that share a group
  for (int i = threadIdx.x; i < kW4Rows * 4; i += kPackThreads) {
    const int r = i / 4, j = i % 4;
    const int n = nt * kW4Rows + r, k = kt * kW4Cols + 32 * j;
    float x[32];
    const bool in = n < p.N && k < p.K;
    if (in) {
      load32(W + (size_t)n * p.K + k, x);
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] = 0.f;
    }
    float lo = 0.f, hi = 0.f;
    bool fine = true;
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      lo = fminf(lo, x[e]);
      hi = fmaxf(hi, x[e]);
      fine = fine && fabsf(x[e]) <= FLT_MAX;
    }
    for (int o = 1; o < lanes; o <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      fine = __shfl_xor_sync(0xffffffffu, fine, o) && fine;
    }
    __half hs = __float2half_rn((float)(((double)hi - (double)lo) / 15.0));
    if (__hisinf(hs)) fine = false;
    if (!fine) {
      batch_flag(flag, kBatchRange);
      hs = __float2half_rn(0.f);
    }
    const float s = __half2float(hs);
    const float z = s > 0.f ? fminf(nearest_quotient(-lo, s), 15.f) : 0.f;
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      w[q] = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float c = s > 0.f ? fminf(fmaxf(nearest_quotient(x[8 * q + e], s) + z, 0.f), 15.f) : 0.f;
        w[q] |= (uint32_t)c << w4_shift(e);
      }
    }
    *reinterpret_cast<uint4*>(tile + j * (kW4Rows * 16) + r * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    if (j % lanes == 0) {
      const int g = j / lanes;
      reinterpret_cast<__half*>(tile + kW4Codes)[g * kW4Rows + r] = hs;
      tile[kW4Codes + per * kW4Rows * 2 + g * kW4Rows + r] = (uint8_t)z;
    }
  }
}

__global__ void __launch_bounds__(kPackThreads) pack_codes4_kernel(const uint8_t* __restrict__ codes,
                                                                   const __half* __restrict__ scales,
                                                                   const uint8_t* __restrict__ zeros, uint8_t* __restrict__ out,
                                                                   W4Shape p, unsigned* flag) {
  const int nt = blockIdx.x / p.k_tiles, kt = blockIdx.x % p.k_tiles;
  uint8_t* tile = out + (size_t)blockIdx.x * p.tile_bytes;
  const int per = kW4Cols / p.group, lanes = p.group / 32;
  for (int i = threadIdx.x; i < kW4Rows * 4; i += kPackThreads) {
    const int r = i / 4, j = i % 4;
    const int n = nt * kW4Rows + r, k = kt * kW4Cols + 32 * j;
    const bool in = n < p.N && k < p.K;
    uint32_t c[8] = {};
    if (in) {
      const uint4* src = reinterpret_cast<const uint4*>(codes + (size_t)n * p.K + k);
      const uint4 a = __ldg(src), b = __ldg(src + 1);
      c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w, c[4] = b.x, c[5] = b.y, c[6] = b.z, c[7] = b.w;
    }
    uint32_t over = 0, w[4];
#pragma unroll
    for (int q = 0; q < 8; ++q) over |= c[q] & 0xf0f0f0f0u;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      w[q] = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) w[q] |= (c[2 * q + e / 4] >> (8 * (e % 4)) & 15u) << w4_shift(e);
    }
    *reinterpret_cast<uint4*>(tile + j * (kW4Rows * 16) + r * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    if (j % lanes == 0) {
      const int g = j / lanes;
      const size_t at = (size_t)n * p.groups + (kt * kW4Cols + g * p.group) / p.group;
      const uint8_t z = !in ? 0 : zeros ? zeros[at] : 8;
      over |= z & 0xf0u;
      reinterpret_cast<__half*>(tile + kW4Codes)[g * kW4Rows + r] = in ? scales[at] : __float2half_rn(0.f);
      tile[kW4Codes + per * kW4Rows * 2 + g * kW4Rows + r] = z & 15;
    }
    if (over) batch_flag(flag, kBatchBadCode);
  }
}

// A thread writes the 8 values of a word, 16 threads a row's part of the tile.
__global__ void __launch_bounds__(kPackThreads) unpack4_kernel(const uint8_t* __restrict__ w4, float* __restrict__ W, W4Shape p) {
  const int nt = blockIdx.x / p.k_tiles, kt = blockIdx.x % p.k_tiles;
  const uint8_t* tile = w4 + (size_t)blockIdx.x * p.tile_bytes;
  const int per = kW4Cols / p.group;
  for (int i = threadIdx.x; i < kW4Rows * 16; i += kPackThreads) {
    const int r = i / 16, q = i % 16, n = nt * kW4Rows + r, k = kt * kW4Cols + 8 * q;
    if (n >= p.N || k >= p.K) continue;
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(tile + q / 4 * (kW4Rows * 16) + r * 16 + q % 4 * 4));
    const int g = 8 * q / p.group;
    const float s = __half2float(reinterpret_cast<const __half*>(tile + kW4Codes)[g * kW4Rows + r]);
    const int z = tile[kW4Codes + per * kW4Rows * 2 + g * kW4Rows + r];
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = s * (float)((int)(w >> w4_shift(e) & 15u) - z);
    float4* dst = reinterpret_cast<float4*>(W + (size_t)n * p.K + k);
    dst[0] = make_float4(y[0], y[1], y[2], y[3]);
    dst[1] = make_float4(y[4], y[5], y[6], y[7]);
  }
}

// ------------------------------------------------------------------ product

struct Gemm4Args {
  W4Shape w;
  const uint8_t* w4;
  const void* x;
  int64_t x_stride;
  const float* x_scales;
  float* y;
  int T;
};

constexpr int kSimpleRows = 8;   // of X per CTA

// One thread per weight row, kSimpleRows rows of X in shared memory.
template <bool E4M3>
__global__ void __launch_bounds__(kW4Rows) gemm4_kernel(Gemm4Args a) {
  __shared__ float xs[kSimpleRows][kW4Cols];
  const int nt = blockIdx.x, t0 = blockIdx.y * kSimpleRows, r = threadIdx.x, n = nt * kW4Rows + r;
  const int per = kW4Cols / a.w.group, x_groups = a.w.k_tiles;
  float acc[kSimpleRows] = {};
  for (int kt = 0; kt < a.w.k_tiles; ++kt) {
    const uint8_t* tile = a.w4 + ((size_t)nt * a.w.k_tiles + kt) * a.w.tile_bytes;
    for (int i = threadIdx.x; i < kSimpleRows * kW4Cols; i += kW4Rows) {
      const int t = t0 + i / kW4Cols, k = kt * kW4Cols + i % kW4Cols;
      float v = 0.f;
      if (t < a.T && k < a.w.K) {
        if (E4M3)
          v = __half2float(__half(__nv_cvt_fp8_to_halfraw(((const uint8_t*)a.x)[t * a.x_stride + k], __NV_E4M3)));
        else
          v = __half2float(((const __half*)a.x)[t * a.x_stride + k]);
      }
      xs[i / kW4Cols][i % kW4Cols] = v;
    }
    __syncthreads();
    for (int g = 0; g < per; ++g) {
      const float s = __half2float(reinterpret_cast<const __half*>(tile + kW4Codes)[g * kW4Rows + r]);
      const int z = tile[kW4Codes + per * kW4Rows * 2 + g * kW4Rows + r];
      float sum[kSimpleRows] = {};
      for (int q = g * a.w.group / 8; q < (g + 1) * a.w.group / 8; ++q) {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(tile + q / 4 * (kW4Rows * 16) + r * 16 + q % 4 * 4));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float c = (float)((int)(w >> w4_shift(e) & 15u) - z);
#pragma unroll
          for (int t = 0; t < kSimpleRows; ++t) sum[t] = fmaf(c, xs[t][8 * q + e], sum[t]);
        }
      }
#pragma unroll
      for (int t = 0; t < kSimpleRows; ++t) {
        const float sx = E4M3 && t0 + t < a.T ? a.x_scales[(size_t)(t0 + t) * x_groups + kt] : 1.f;
        acc[t] = fmaf(E4M3 ? sum[t] * sx : sum[t], s, acc[t]);
      }
    }
    __syncthreads();
  }
  if (n >= a.w.N) return;
#pragma unroll
  for (int t = 0; t < kSimpleRows; ++t)
    if (t0 + t < a.T) a.y[(size_t)(t0 + t) * a.w.N + n] = acc[t];
}

bool misaligned(const void* p, unsigned to) { return ((uintptr_t)p & (to - 1)) != 0; }

}  // namespace

}  // namespace pic

using namespace pic;

extern "C" {

size_t pic_op_weight4_bytes(int32_t N, int32_t K, int32_t group) {
  if (!w4_ok(N, K, group)) return 0;
  const W4Shape s = w4_shape(N, K, group);
  return (size_t)s.n_tiles * s.k_tiles * s.tile_bytes;
}

pic_status pic_op_pack_weight4(int32_t dtype, const void* W, void* out, int32_t N, int32_t K, int32_t group,
                               pic_stream_t stream) {
  if (!W || !out || !w4_ok(N, K, group) || (dtype != PIC_F32 && dtype != PIC_BF16 && dtype != PIC_F16))
    return fail(PIC_ERR_INVALID_ARG, "invalid 4-bit pack arguments (K a multiple of 32, group 32, 64 or 128)");
  if (misaligned(W, 16) || misaligned(out, 128))
    return fail(PIC_ERR_INVALID_ARG, "4-bit pack: W must be 16-byte, the packed weights 128-byte aligned");
  const W4Shape s = w4_shape(N, K, group);
  if (overlap(W, (size_t)N * K * (dtype == PIC_F32 ? 4 : 2), out, (size_t)s.n_tiles * s.k_tiles * s.tile_bytes))
    return fail(PIC_ERR_INVALID_ARG, "4-bit pack: the packed weights must not overlap W");
  unsigned* flag = nullptr;
  pic_status e = batch_flag_address(&flag);
  if (e != PIC_OK) return e;
  const int grid = s.n_tiles * s.k_tiles;
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == PIC_F32) pack4_kernel<<<grid, kPackThreads, 0, st>>>((const float*)W, (uint8_t*)out, s, flag);
  else if (dtype == PIC_F16) pack4_kernel<<<grid, kPackThreads, 0, st>>>((const __half*)W, (uint8_t*)out, s, flag);
  else pack4_kernel<<<grid, kPackThreads, 0, st>>>((const __nv_bfloat16*)W, (uint8_t*)out, s, flag);
  PIC_CUDA(cudaGetLastError());
  return PIC_OK;
}

pic_status pic_op_pack_codes4(const uint8_t* codes, const void* scales, const uint8_t* zeros, void* out, int32_t N,
                              int32_t K, int32_t group, pic_stream_t stream) {
  if (!codes || !scales || !out || !w4_ok(N, K, group))
    return fail(PIC_ERR_INVALID_ARG, "invalid 4-bit pack arguments (K a multiple of 32, group 32, 64 or 128)");
  if (misaligned(codes, 16) || misaligned(scales, 2) || misaligned(out, 128))
    return fail(PIC_ERR_INVALID_ARG, "4-bit pack: codes must be 16-byte, the packed weights 128-byte aligned");
  const W4Shape s = w4_shape(N, K, group);
  const size_t bytes = (size_t)s.n_tiles * s.k_tiles * s.tile_bytes;
  if (overlap(codes, (size_t)N * K, out, bytes) || overlap(scales, (size_t)N * s.groups * 2, out, bytes) ||
      (zeros && overlap(zeros, (size_t)N * s.groups, out, bytes)))
    return fail(PIC_ERR_INVALID_ARG, "4-bit pack: the packed weights must not overlap the codes, scales or zeros");
  unsigned* flag = nullptr;
  pic_status e = batch_flag_address(&flag);
  if (e != PIC_OK) return e;
  pack_codes4_kernel<<<s.n_tiles * s.k_tiles, kPackThreads, 0, (cudaStream_t)stream>>>(codes, (const __half*)scales, zeros,
                                                                                       (uint8_t*)out, s, flag);
  PIC_CUDA(cudaGetLastError());
  return PIC_OK;
}

pic_status pic_op_unpack_weight4(const void* W4, float* W, int32_t N, int32_t K, int32_t group, pic_stream_t stream) {
  if (!W4 || !W || !w4_ok(N, K, group))
    return fail(PIC_ERR_INVALID_ARG, "invalid 4-bit unpack arguments (K a multiple of 32, group 32, 64 or 128)");
  if (misaligned(W4, 128) || misaligned(W, 32))
    return fail(PIC_ERR_INVALID_ARG, "4-bit unpack: the packed weights must be 128-byte, W 32-byte aligned");
  const W4Shape s = w4_shape(N, K, group);
  if (overlap(W4, (size_t)s.n_tiles * s.k_tiles * s.tile_bytes, W, (size_t)N * K * 4))
    return fail(PIC_ERR_INVALID_ARG, "4-bit unpack: W must not overlap the packed weights");
  unpack4_kernel<<<s.n_tiles * s.k_tiles, kPackThreads, 0, (cudaStream_t)stream>>>((const uint8_t*)W4, W, s);
  PIC_CUDA(cudaGetLastError());
  return PIC_OK;
}

pic_status pic_op_gemm_w4(int32_t x_dtype, const void* W4, const void* X, int64_t x_stride, const float* x_scales,
                          float* Y, int32_t N, int32_t K, int32_t T, int32_t group, pic_stream_t stream) {
  const bool e4m3 = x_dtype == PIC_E4M3;
  if (!W4 || !X || !Y || T < 1 || !w4_ok(N, K, group) || (!e4m3 && x_dtype != PIC_F16) || e4m3 != (x_scales != nullptr) ||
      x_stride < K || x_stride >= (int64_t)1 << 38 || x_stride % (e4m3 ? 16 : 8))
    return fail(PIC_ERR_INVALID_ARG, "invalid 4-bit gemm arguments (K a multiple of 32, group 32, 64 or 128, rows of X a "
                                     "multiple of 16 bytes apart, x_scales with 8-bit rows)");
  if (T > 65535 * 64) return fail(PIC_ERR_CAPACITY, "4-bit gemm: more than 4194240 rows");
  if (misaligned(W4, 128) || misaligned(X, 16) || misaligned(Y, 16) || misaligned(x_scales, 4))
    return fail(PIC_ERR_INVALID_ARG, "4-bit gemm: X and Y must be 16-byte, the packed weights 128-byte aligned");
  const W4Shape s = w4_shape(N, K, group);
  const size_t y_bytes = (size_t)T * N * 4;
  if (overlap(Y, y_bytes, X, ((size_t)(T - 1) * x_stride + K) * (e4m3 ? 1 : 2)) ||
      overlap(Y, y_bytes, W4, (size_t)s.n_tiles * s.k_tiles * s.tile_bytes) ||
      (x_scales && overlap(Y, y_bytes, x_scales, (size_t)T * s.k_tiles * 4)))
    return fail(PIC_ERR_INVALID_ARG, "4-bit gemm: Y must not overlap the packed weights, X or its scales");
  const Gemm4Args a{s, (const uint8_t*)W4, X, x_stride, x_scales, Y, T};
  for (int t0 = 0; t0 < T; t0 += 65535 * kSimpleRows) {
    Gemm4Args b = a;
    b.x = (const uint8_t*)X + (size_t)t0 * x_stride * (e4m3 ? 1 : 2);
    b.x_scales = x_scales ? x_scales + (size_t)t0 * s.k_tiles : nullptr;
    b.y = Y + (size_t)t0 * N;
    b.T = std::min(T - t0, 65535 * kSimpleRows);
    const dim3 grid(s.n_tiles, (b.T + kSimpleRows - 1) / kSimpleRows);
    if (e4m3) gemm4_kernel<true><<<grid, kW4Rows, 0, (cudaStream_t)stream>>>(b);
    else gemm4_kernel<false><<<grid, kW4Rows, 0, (cudaStream_t)stream>>>(b);
    PIC_CUDA(cudaGetLastError());
  }
  return PIC_OK;
}

}  // extern "C"
