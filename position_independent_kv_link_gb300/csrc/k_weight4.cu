// 4-bit weights with group scales: packing, unpacking, and the product of few rows with them.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <climits>
#include <mutex>
#include <type_traits>

#include <cuda_fp8.h>

#include "async.cuh"
#include "weight4.cuh"

namespace pic {

namespace {

// ------------------------------------------------------------------ packing
//
// One CTA packs a tile; a thread holds 32 columns of a row (16 bytes of codes), the four threads of a row's 128 columns lie
// side by side, so that the extremes of a group of 64 or 128 are shuffles away. Bound by instructions for 16-bit weights (28672 x 4096
// bf16 in groups of 64: 76 us, 3.9 TB/s, issue slots 67 % busy; fp16 in groups of 128: 69 us), by HBM for fp32 (89 us, 6.0 TB/s).
// Unpacking writes 8 bytes for every one that it reads: 84 us, 6.3 TB/s, 93 % of a copy (98 us in pieces of 16 bytes a lane instead of 32).
constexpr int kPackThreads = 256;

template <bool WIDE, typename T>
__device__ __forceinline__ void load32(const T* p, float* x) {   // 32 values, 16-byte aligned (32 when WIDE)
  constexpr int E = 32 / sizeof(T);
#pragma unroll
  for (int i = 0; i < 32; i += E) {
    uint32_t u[8];
    if constexpr (WIDE) {
      asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                   : "l"(p + i));
    } else {
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(p + i)), b = __ldg(reinterpret_cast<const uint4*>(p + i) + 1);
      u[0] = a.x, u[1] = a.y, u[2] = a.z, u[3] = a.w, u[4] = b.x, u[5] = b.y, u[6] = b.z, u[7] = b.w;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (std::is_same<T, float>::value) {
        x[i + j] = __uint_as_float(u[j]);
      } else if constexpr (std::is_same<T, __half>::value) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[j]));
        x[i + 2 * j] = f.x, x[i + 2 * j + 1] = f.y;
      } else {
        x[i + 2 * j] = __uint_as_float(u[j] << 16);
        x[i + 2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
      }
    }
  }
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(r))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;"
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
__device__ __forceinline__ float max_nan(float a, float b) {   // NaN when one is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

constexpr float kMagic = 12582912.f;                   // 1.5 2^23: integers are the spacing there

// The integer nearest to x / s (ties to even), decided exactly: x (1 / s) in fp32 gives an integer k that may be off by one next
// to a border; x - k s is exact in fp32 (s has 11 bits, and x lies within some 23 s), as is s / 2. rs: 1 / s.
__device__ __forceinline__ int nearest_quotient(float x, float s, float rs) {
  const float t = fmaf(x, rs, kMagic), d = fmaf(kMagic - t, s, x), half = 0.5f * s;
  const int k = __float_as_int(t) - __float_as_int(kMagic);
  return k + (d > half || (d == half && (k & 1))) - (d < -half || (d == -half && (k & 1)));
}

// fp16 of fp32 of (hi - lo) / 15 in 64 bits. In fp32 the quotient is within 2^-22 of itself, so its fp16 is known unless a border lies
// within 2^-20: only then 64 bits decide (this GPU has few units for them: in every group, 28672 x 4096 took 117 us for 103).
__device__ __forceinline__ __half group_scale(float lo, float hi) {
  const float q = (hi - lo) * (1.f / 15.f);
  const __half a = __float2half_rn(q * (1.f - 1.f / 1048576)), b = __float2half_rn(q * (1.f + 1.f / 1048576));
  if (__half_as_ushort(a) == __half_as_ushort(b)) return a;
  return __float2half_rn((float)(((double)hi - (double)lo) / 15.0));
}

// The codes of 32 weights, eight a word. The integer next to x rs + z is nearest_quotient(x) + z, but where x / s is within 2^-18 of a border;
// then |x - k s| is within 2^-17 of s / 2, and the word is done again one by one, exactly (bf16 weights stand on borders often: in 4 of
// 10 warps' 1024). So are those of scales so far below fp16's normal range that a zero beyond 15 was cut (`cut`): only there can
// a code be below 0.
__device__ __forceinline__ void codes32(const float* x, float s, float rs, int z, bool cut, uint32_t* w) {
  const float m = kMagic + z, near = 0.5f * s * (1.f - 1.f / 65536);
  const float2 rs2 = make_float2(rs, rs), m2 = make_float2(m, m), less = make_float2(-m, -m), ns = make_float2(-s, -s);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float far = 0.f;
    uint32_t u = 0;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float2 v = make_float2(x[8 * q + e], x[8 * q + e + 1]);
      const float2 t = fma2(v, rs2, m2), d = fma2(add2(t, less), ns, v);
      far = max3_abs(far, d.x, d.y);
      uint32_t two = __byte_perm(__float_as_uint(t.x), __float_as_uint(t.y), 0x5410);   // (kMagic's lower half is 0)
      asm("min.u16x2 %0, %0, %1;" : "+r"(two) : "r"(0x000f000fu));
      static_assert(w4_shift(1) - w4_shift(0) == 16 && w4_shift(7) - w4_shift(6) == 16, "two columns side by side stand 16 bits apart");
      u += two << w4_shift(e);
    }
    if (far >= near || cut) {
      u = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) u |= (uint32_t)min(max(nearest_quotient(x[8 * q + e], s, rs) + z, 0), 15) << w4_shift(e);
    }
    w[q] = u;
  }
}

// The four threads of a row hold its runs' words of each piece; they trade them for a piece each, and write 64 bytes together.
__device__ __forceinline__ void put_pieces(uint8_t* tile, int r, int j, uint32_t* w) {
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    const bool up = j & o;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int lo = o == 1 ? 2 * i : i, hi = lo + o;
      const uint32_t t = __shfl_xor_sync(0xffffffffu, up ? w[lo] : w[hi], o);
      if (up) w[lo] = t;
      else w[hi] = t;
    }
  }
  *reinterpret_cast<uint4*>(tile + w4_piece(r, j)) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool WIDE, typename T>
__global__ void __launch_bounds__(kPackThreads) pack4_kernel(const T* __restrict__ W, uint8_t* __restrict__ out, W4Shape p,
                                                             unsigned* flag) {
  const int nt = blockIdx.x / p.k_tiles, kt = blockIdx.x % p.k_tiles;
  uint8_t* tile = out + (size_t)blockIdx.x * p.tile_bytes;
  const int per = kW4Cols / p.group;                   // groups of a tile's row
  const int lanes = p.group / 32;                      // threads that share a group
#pragma unroll 1
  for (int i = threadIdx.x; i < kW4Rows * 4; i += kPackThreads) {
    const int r = i / 4, j = i % 4;
    const int n = nt * kW4Rows + r, k = kt * kW4Cols + 32 * j;
    float x[32];
    if (n < p.N && k < p.K) {
      load32<WIDE>(W + (size_t)n * p.K + k, x);
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] = 0.f;
    }
    float lo = 0.f, hi = 0.f;                          // (NaN when a weight is)
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      lo = min3(lo, x[e], x[e + 1]);
      hi = max3_nan(hi, x[e], x[e + 1]);
    }
    for (int o = 1; o < lanes; o <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    bool fine = hi == hi;
    __half hs = group_scale(lo, hi);
    if (__hisinf(hs)) fine = false;                    // infinite weights too
    if (!fine) {
      batch_flag(flag, kBatchRange);
      hs = __float2half_rn(0.f);
    }
    const float s = __half2float(hs), rs = s > 0.f ? 1.f / s : 0.f;
    const int z0 = s > 0.f ? nearest_quotient(-lo, s, rs) : 0, z = min(z0, 15);
    uint32_t w[4] = {};
    if (s > 0.f) codes32(x, s, rs, z, z0 > 15, w);
    put_pieces(tile, r, j, w);
    if (j % lanes == 0) {
      const int g = j / lanes;
      reinterpret_cast<__half*>(tile + kW4Codes)[g * kW4Rows + w4_place(r)] = hs;
      tile[kW4Codes + per * kW4Rows * 2 + g * kW4Rows + w4_place(r)] = (uint8_t)z;
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
    uint32_t over = 0, w[4] = {};
#pragma unroll
    for (int q = 0; q < 8; ++q) over |= c[q] & 0xf0f0f0f0u;
#pragma unroll
    for (int e = 0; e < 32; ++e) w[e / 8] |= (c[e / 4] >> (8 * (e % 4)) & 15u) << w4_shift(e % 8);
    put_pieces(tile, r, j, w);
    if (j % lanes == 0) {
      const int g = j / lanes;
      const size_t at = (size_t)n * p.groups + (kt * kW4Cols + g * p.group) / p.group;
      const uint8_t z = !in ? 0 : zeros ? zeros[at] : 8;
      over |= z & 0xf0u;
      reinterpret_cast<__half*>(tile + kW4Codes)[g * kW4Rows + w4_place(r)] = in ? scales[at] : __float2half_rn(0.f);
      tile[kW4Codes + per * kW4Rows * 2 + g * kW4Rows + w4_place(r)] = z & 15;
    }
    if (over) batch_flag(flag, kBatchBadCode);
  }
}

// A lane holds a word of codes and writes its 8 values, a warp two rows' parts of the tile.
__global__ void __launch_bounds__(kPackThreads) unpack4_kernel(const uint8_t* __restrict__ w4, float* __restrict__ W, W4Shape p) {
  const int nt = blockIdx.x / p.k_tiles, kt = blockIdx.x % p.k_tiles;
  const uint8_t* tile = w4 + (size_t)blockIdx.x * p.tile_bytes;
  const int per = kW4Cols / p.group, c = 8 * (threadIdx.x % 16), g = c / p.group, k = kt * kW4Cols + c;
  const __half* scales = reinterpret_cast<const __half*>(tile + kW4Codes) + g * kW4Rows;
  const uint8_t* zeros = tile + kW4Codes + per * kW4Rows * 2 + g * kW4Rows;
  float* to = W + (size_t)nt * kW4Rows * p.K + k;
  const int rows = min(kW4Rows, p.N - nt * kW4Rows);
  if (k >= p.K) return;
#pragma unroll 8
  for (int r = threadIdx.x / 16; r < rows; r += kPackThreads / 16) {
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(tile + w4_piece(r, c % 32 / 8) + c / 32 * 4));
    const float s = __half2float(__ldg(scales + w4_place(r)));
    const int z = __ldg(zeros + w4_place(r));
    auto value = [&](int e) { return s * (float)((int)(w >> w4_shift(e) & 15u) - z); };
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + (size_t)r * p.K), "f"(value(0)),
                 "f"(value(1)), "f"(value(2)), "f"(value(3)), "f"(value(4)), "f"(value(5)), "f"(value(6)), "f"(value(7))
                 : "memory");
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
  int lg;                    // log2 of a group's 32-column steps
  unsigned* flag;
};

// Sums of (code - zero) x, exact products of integers below 16 with fp16 (or e4m3) numbers in fp32, times the group's scale in fp32. The
// weights' 4 bits are the bytes that count: HBM would allow 0.19 us for a 128 x 128 block an SM. Turning codes into operands (9
// instructions for 8 codes), the sums and the handshakes cost more: 0.26 us with one row, 0.33 with 16, 0.39 and 0.48 with 64 in fp16 and
// e4m3 (LM head of 128256 x 4096: 55 us, 69, 83, 101; floors 41, 42, 45, 45). 4096 x 14336: 1 row 12 us, 16 rows 14, 64 rows 20; floor
// 4.5 to 5.
//
// A band is 128 rows of W (256 in the tcgen05 kernel) against one tile of rows of X; its columns come in blocks of 128. With many
// bands the CTAs take whole ones in turn, and their copies run on over the ends of bands. With few, and for what is left after the last
// full turn, the CTAs of a cluster share one band's blocks and add their sums through each other's shared memory, in the order of
// their ranks. So there is no scratch, and the same call gives the same bits again.

struct Gemm4Plan {
  int stages, x_bytes;       // of X in a stage
  int across, bands;         // bands of one tile of X, of all
  int whole;                 // the first ones, which CTAs take whole
};

// Shared memory by its own addresses (through pointers that were rounded up the loads become generic ones)
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ float lds_half(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
  return __half2float(__ushort_as_half(v));
}
__device__ __forceinline__ float4 lds_f32x4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ void sts_f32(uint32_t at, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory"); }
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// The scales of `rows` rows of 8-bit X for one block (0 behind the last row) by the lanes of a warp; each lane's arrive follows its copies.
__device__ __forceinline__ void x_scales_to(uint32_t dst, const float* src, int rows, int k_tiles, int nt, int lane, uint32_t bar) {
  for (int t = lane; t < nt; t += 32)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + 4 * t), "l"(src + (size_t)(t < rows ? t : 0) * k_tiles),
                 "r"(t < rows ? 4 : 0)
                 : "memory");
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// Low word of the descriptor of K-major rows of 128 bytes, 128-byte swizzle, 8-row groups 1024 bytes apart; the high word is fixed
constexpr uint32_t kDescHi = (1024 >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr) { return (addr & 0x3FFFFu) >> 4; }
// D (fp32) in tensor memory += A (tensor memory, 128 lanes) . B^T (shared memory, N rows); fp16, or e4m3
template <bool E4M3>
__device__ __forceinline__ void umma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (E4M3)
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.b32 p, %5, 0;\n mov.b64 y, {%2, %4};\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], y, %3, p;\n}\n" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(kDescHi),
        "r"(acc));
  else
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.b32 p, %5, 0;\n mov.b64 y, {%2, %4};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}\n" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(kDescHi),
        "r"(acc));
}
// one lane of a whole warp, always the same
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void umma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float2* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(v[0].x), "=f"(v[0].y), "=f"(v[1].x), "=f"(v[1].y), "=f"(v[2].x), "=f"(v[2].y), "=f"(v[3].x), "=f"(v[3].y),
        "=f"(v[4].x), "=f"(v[4].y), "=f"(v[5].x), "=f"(v[5].y), "=f"(v[6].x), "=f"(v[6].y), "=f"(v[7].x), "=f"(v[7].y)
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld16(float2* v) {   // the registers are operands, so that no use moves ahead
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0].x), "+f"(v[0].y), "+f"(v[1].x), "+f"(v[1].y), "+f"(v[2].x), "+f"(v[2].y), "+f"(v[3].x),
                 "+f"(v[3].y), "+f"(v[4].x), "+f"(v[4].y), "+f"(v[5].x), "+f"(v[5].y), "+f"(v[6].x), "+f"(v[6].y),
                 "+f"(v[7].x), "+f"(v[7].y)
               :
               : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float2* v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(v[0].x), "=f"(v[0].y), "=f"(v[1].x), "=f"(v[1].y), "=f"(v[2].x), "=f"(v[2].y), "=f"(v[3].x), "=f"(v[3].y)
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld8(float2* v) {   // the registers are operands, so that no use moves ahead
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0].x), "+f"(v[0].y), "+f"(v[1].x), "+f"(v[1].y), "+f"(v[2].x), "+f"(v[2].y), "+f"(v[3].x), "+f"(v[3].y)
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
// Y[t][n] = the sum over the cluster's CTAs, in the order of their ranks, of the fp32 value at `at` + t pitch, for t = first, first +
// step, .. < end. A value of another CTA takes most of a microsecond, so many are asked for at a time: of R rows and C CTAs.
template <int R, int C>
__device__ __forceinline__ void cluster_rows(uint32_t at, uint32_t pitch, uint32_t ctas, int first, int end, int step, float* y,
                                             int N) {
  for (int t = first; t < end; t += R * step) {
    float sum[R] = {};
#pragma unroll C
    for (uint32_t c = 0; c < ctas; ++c) {
      uint32_t there;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(c));
      float v[R];
#pragma unroll
      for (int i = 0; i < R; ++i)
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[i]) : "r"(there + min(t + i * step, end - 1) * pitch) : "memory");
#pragma unroll
      for (int i = 0; i < R; ++i) sum[i] += v[i];
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (t + i * step < end) y[(size_t)(t + i * step) * N] = sum[i];
  }
}
__device__ __forceinline__ void cluster_sums(uint32_t at, uint32_t pitch, uint32_t ctas, int first, int end, int step, float* y,
                                             int N) {
  if (end - first <= step) cluster_rows<1, 8>(at, pitch, ctas, first, end, step, y, N);
  else cluster_rows<4, 2>(at, pitch, ctas, first, end, step, y, N);
}
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {   // (a & b) | c
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// The 8 integers code - zero of a word in fp16, exact: z0 = 1024 + zero, z1 = -(64 + zero), twice each
__device__ __forceinline__ void codes_f16(uint32_t x, uint32_t z0, uint32_t z1, uint32_t* v) {
  const uint32_t y = x >> 8;
  v[0] = hsub2(and_or(x, 0x000f000fu, 0x64006400u), z0);                   // 1024 + c - (1024 + zero)
  v[1] = hfma2(and_or(x, 0x00f000f0u, 0x64006400u), 0x2c002c00u, z1);      // (1024 + 16 c) / 16 - (64 + zero)
  v[2] = hsub2(and_or(y, 0x000f000fu, 0x64006400u), z0);
  v[3] = hfma2(and_or(y, 0x00f000f0u, 0x64006400u), 0x2c002c00u, z1);
}

constexpr int kMaxStages = 12, kFewRows = 16, kTcBlocks = 1536;

// A CTA's blocks, in the order in which all of its warps take them: whole bands in turn, then its cluster's share of one.
struct Gemm4Walk {
  int split, rank;           // CTAs of the cluster
  int n_band, t_tile, kb;    // the block: band down W, tile of X, block of the band
  int band, k1, k_tiles, bands, whole, across, step;

  __device__ __forceinline__ Gemm4Walk(const Gemm4Args& a, const Gemm4Plan& p) {
    uint32_t x, y;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(x));
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(y));
    split = (int)x;
    rank = (int)y;
    across = p.across;
    k_tiles = a.w.k_tiles;
    bands = p.bands;
    whole = p.whole;
    step = gridDim.x;
    enter(blockIdx.x);
  }
  __device__ __forceinline__ int shared_band() const { return whole + (int)blockIdx.x / split; }   // (bands and up: none)
  __device__ __forceinline__ void enter(int b) {
    band = b;
    kb = 0;
    k1 = k_tiles;
    if (band >= whole) {
      band = split > 1 ? shared_band() : bands;
      kb = (int)((int64_t)k_tiles * rank / split);
      k1 = (int)((int64_t)k_tiles * (rank + 1) / split);
    }
    n_band = band % across;
    t_tile = band / across;
  }
  __device__ __forceinline__ bool more() const { return band < bands; }
  __device__ __forceinline__ bool next() {         // true behind the last block of a whole band
    if (++kb < k1) return false;
    const bool was_whole = band < whole;
    if (was_whole) enter(band + step);
    else band = bands;
    return was_whole;
  }
};

// More than kFewRows rows of X: tcgen05. A band is two tiles of 128 rows, which share the block of X.
//
//   warps 0-7   thread r of a tile's four warps: the 64 bytes of codes of row r become the integers code - zero in fp16, exact, in
//               tensor memory as the A operand (the row's lane)
//   warps 8-15  thread r of a tile's four warps: the sums of row r with the rows of X are read back for each group of columns, multiplied
//               by the row's scale and added in fp32 registers. So a scale is a factor of one thread, products and sums within a group are exact integers times X,
//               and no rounding enters but those of the fp32 sums.
//   one warp: one thread asks for the packed tiles (bulk copies of 8.4 to 9.5 KB) and the block of X (TMA) of each stage
//   the last two, one a tile: issue the products, D[row][t] for each group of columns, into one of two accumulators
//
// What a warp does besides its arithmetic decides the time (waits, arrivals, the loop): with one issuing warp and 16 that add the issue slots
// were 73 % busy (64 fp16 rows of 128256 x 4096: 114 us); with an issuing warp a tile, 8 that add and no wait that another implies it is
// 83. 8-bit X needs a factor for each row and block: 32 rows of X a warp and 16 warps (101 us), as 64 spill (181).
//
// 8-bit X: the integer c = 0..15 is the e4m3 number c 2^-9 (subnormal up to 7, then the first binade with the same spacing), so the
// codes need only be spread to bytes. The zero goes in by a second product with a row of -zero 2^-9, 8 columns of tensor
// memory for a whole group; both are exact.
//
// Barriers: FULL, EMPTY of a stage: the copies have landed (AFULL and DFULL tell the same to those that wait for them); the warps have
// read it, and the products, which the warps that add have waited for. For each tile by itself, so that the two warps of an SM's
// quarter that write operands do not wait at the same time: AFULL, AEMPTY of an operand buffer: the four warps have written it; the
// products of the block have ended. DFULL, DEMPTY of an accumulator: the products of a group have ended; the warps that add have read
// it. Each is waited for by every thread that could fall a phase behind.
constexpr int kTcTiles = 2;
template <bool E4M3, int NT>
struct TcShape {
  static constexpr int kCols = E4M3 ? 32 : NT;         // rows of X that a warp adds
  static constexpr int kAdd = 8 * (NT / kCols), kLoad = 8 + kAdd;   // warps that add; the one that loads, those behind it that issue
  static constexpr int kThreads = (kLoad + 1 + kTcTiles) * 32;
};
constexpr int kTcA = 64, kTcTile = 256, kTcCols = 512;   // columns of tensor memory: an A buffer (two a tile), a tile, all

template <bool E4M3, int NT>
__global__ void __launch_bounds__(TcShape<E4M3, NT>::kThreads, 1)
    gemm4_tc_kernel(const __grid_constant__ CUtensorMap map_x, const Gemm4Args a, const Gemm4Plan p) {
  constexpr int kAdd = TcShape<E4M3, NT>::kAdd, kLoad = TcShape<E4M3, NT>::kLoad, kCols = TcShape<E4M3, NT>::kCols,
                kChunk = E4M3 ? 8 : 16;
  static_assert(2 * kTcA + 2 * NT <= kTcTile && kTcTiles * kTcTile == kTcCols, "tensor memory");
  extern __shared__ uint8_t smem_raw[];
  const uint32_t xs = (smem_u32(smem_raw) + 1023) & ~1023u, ws = xs + p.stages * p.x_bytes;   // [stages] X; [stages][kTcTiles] tiles; [stages][NT] scales of X
  const uint32_t ss = ws + p.stages * kTcTiles * a.w.tile_bytes;
  __shared__ uint64_t s_full[kMaxStages], s_empty[kMaxStages], s_afull[kTcTiles][2], s_aempty[kTcTiles][2], s_dfull[kTcTiles][2],
      s_dempty[kTcTiles][2], s_done;
  __shared__ uint32_t s_tmem;
  __shared__ unsigned s_abort;
  volatile unsigned* abort = &s_abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Gemm4Walk w(a, p);
  const int per = 4 >> a.lg, last = (1 << a.lg) - 1;   // groups of a block; 32-column steps of one, less one

  if (threadIdx.x == 0) {
    s_abort = 0;
    prefetch_map(&map_x);
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(smem_u32(s_full + i), E4M3 ? 33 : 1);
      mbar_init(smem_u32(s_empty + i), kLoad);
    }
    for (int g = 0; g < kTcTiles; ++g)
      for (int i = 0; i < 2; ++i) {
        mbar_init(smem_u32(s_afull[g] + i), 4);
        mbar_init(smem_u32(s_aempty[g] + i), 1);
        mbar_init(smem_u32(s_dfull[g] + i), 1);
        mbar_init(smem_u32(s_dempty[g] + i), kAdd / kTcTiles);
      }
    mbar_init(smem_u32(&s_done), kTcTiles);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == kLoad) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(kTcCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    fence_before();
  }
  pdl_wait();
  __syncthreads();
  fence_after();
  const uint32_t tmem = s_tmem;
  int st = 0;
  uint32_t ph = 0;                                 // of the stage
  auto next_stage = [&] {
    if (++st == p.stages) st = 0, ph ^= 1;
  };

  if (warp == kLoad) {
    // Whole warps loop and one lane issues: in a branch of one lane a product took 140 cycles to issue, a stage's copies 1100.
    uint64_t pol_w, pol_x;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol_w));
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(pol_x));
    int issued = 0;
    for (; w.more(); w.next()) {
      if (!warp_wait(smem_u32(s_empty + st), ph ^ 1, abort, a.flag)) break;
      const int n0 = w.n_band * kTcTiles, tiles = min(kTcTiles, a.w.n_tiles - n0);
      const uint32_t fb = smem_u32(s_full + st), x = xs + st * p.x_bytes;
      if (elect()) {
        mbar_expect_tx(fb, p.x_bytes + tiles * a.w.tile_bytes);
        for (int g = 0; g < tiles; ++g)
          bulk_load(ws + (st * kTcTiles + g) * a.w.tile_bytes,
                    a.w4 + ((size_t)(n0 + g) * a.w.k_tiles + w.kb) * a.w.tile_bytes, a.w.tile_bytes, fb, pol_w);
        tma_2d(x, &map_x, w.kb * kW4Cols, w.t_tile * NT, fb, pol_x);
        if (!E4M3) tma_2d(x + NT * 128, &map_x, w.kb * kW4Cols + 64, w.t_tile * NT, fb, pol_x);
      }
      __syncwarp();
      if constexpr (E4M3) {
        const int t0 = w.t_tile * NT;
        x_scales_to(ss + st * NT * 4, a.x_scales + (size_t)t0 * a.w.k_tiles + w.kb, a.T - t0, a.w.k_tiles, NT, lane, fb);
      }
      ++issued;
      next_stage();
    }
    for (int j = max(0, issued - p.stages); j < issued; ++j)   // copies under way land before the CTA ends
      mbar_settle(smem_u32(s_full + j % p.stages), (uint32_t)((j / p.stages) & 1), a.flag);
  } else if (warp > kLoad) {
    constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(NT >> 3) << 17) | ((uint32_t)(kW4Rows >> 4) << 24);
    const int g = warp - kLoad - 1;                // tile
    uint32_t i = 0, q = 0;                         // blocks, groups so far
    bool going = true;
    for (; w.more() && going; w.next(), ++i) {
      const uint32_t X = desc_lo(xs + st * p.x_bytes), A = tmem + g * kTcTile + (i & 1) * kTcA;
      if (!warp_wait(smem_u32(s_afull[g] + (i & 1)), (i >> 1) & 1, abort, a.flag)) break;
      auto issue = [&](auto steps) {               // 32-column steps of a group
        constexpr int S = decltype(steps)::value;
#pragma unroll
        for (int k = 0; k < 4 / S; ++k, ++q) {
          going = going && warp_wait(smem_u32(s_dempty[g] + (q & 1)), ((q >> 1) & 1) ^ 1, abort, a.flag);
          if (!going) return;
          fence_after();
          const uint32_t D = tmem + g * kTcTile + 2 * kTcA + (q & 1) * NT;
          if (elect()) {
#pragma unroll
            for (int j = k * S; j < (k + 1) * S; ++j) {
              if constexpr (E4M3) {
                umma<true>(D, A + j * 8, X + j * 2, idesc, j > k * S);
                umma<true>(D, A + 32 + k * 8, X + j * 2, idesc, 1);
              } else {
                const uint32_t at = X + ((j >> 1) * (NT * 128) + (j & 1) * 64) / 16;
                umma<false>(D, A + j * 16, at, idesc, j > k * S);
                umma<false>(D, A + j * 16 + 8, at + 2, idesc, 1);
              }
            }
            umma_commit(smem_u32(s_dfull[g] + (q & 1)));
            if (k == 4 / S - 1) umma_commit(smem_u32(s_aempty[g] + (i & 1)));
          }
          __syncwarp();
        }
      };
      if (a.lg == 2) issue(std::integral_constant<int, 4>());
      else if (a.lg == 1) issue(std::integral_constant<int, 2>());
      else issue(std::integral_constant<int, 1>());
      next_stage();
    }
    if (elect()) umma_commit(smem_u32(&s_done));     // products under way end before tensor memory is given back
    __syncwarp();
    mbar_settle(smem_u32(&s_done), 0, a.flag);
  } else if (warp < 8) {
    const int g = warp >> 2, r = threadIdx.x & 127;   // tile; row of the tile = lane of tensor memory
    const uint32_t T = tmem + ((uint32_t)((warp & 3) * 32) << 16) + g * kTcTile;
    // (the second tile behind the last band's end: what lies in shared memory, its sums are not kept)
    const uint32_t tile = ws + g * a.w.tile_bytes, zeros = kW4Codes + per * (kW4Rows * 2) + w4_place(r);
    for (uint32_t i = 0; w.more(); w.next(), ++i) {
      if (!warp_wait(smem_u32(s_full + st), ph, abort, a.flag)) break;
      const uint32_t at = tile + st * kTcTiles * a.w.tile_bytes;
      const uint32_t A = T + (i & 1) * kTcA;
      uint4 u[4];                                  // pieces of the row
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = lds128(at + w4_piece(r, e));
      if (!warp_wait(smem_u32(s_aempty[g] + (i & 1)), ((i >> 1) & 1) ^ 1, abort, a.flag)) break;
      fence_after();
      uint32_t z0 = 0, z1 = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool begins = (j & last) == 0;
        if (begins) {
          z0 = lds8(at + zeros + (j >> a.lg) * kW4Rows);
          if constexpr (E4M3) {
            z1 = 0x80808080u | 0x01010101u * z0;                          // -zero 2^-9
          } else {
            z0 = 0x64006400u + 0x00010001u * z0;                          // 1024 + zero
            z1 = hsub2(0x63806380u, z0);                                  // 960 - (1024 + zero)
          }
        }
        uint32_t v[16];
#pragma unroll
        for (int e = 0; e < 4; ++e) {              // pieces: columns 8 e .. 8 e + 7
          const uint32_t x = j == 0 ? u[e].x : j == 1 ? u[e].y : j == 2 ? u[e].z : u[e].w;
          if constexpr (E4M3) {
            const uint32_t lo = x & 0x0f0f0f0fu, hi = (x >> 4) & 0x0f0f0f0fu;
            v[2 * e] = __byte_perm(lo, hi, 0x6420);
            v[2 * e + 1] = __byte_perm(lo, hi, 0x7531);
          } else {
            codes_f16(x, z0, z1, v + 4 * e);
          }
        }
        if constexpr (E4M3) {
          tmem_st8(A + j * 8, v);
          if (begins) {
            const uint32_t same[8] = {z1, z1, z1, z1, z1, z1, z1, z1};
            tmem_st8(A + 32 + (j >> a.lg) * 8, same);
          }
        } else {
          tmem_st16(A + j * 16, v);
        }
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(s_afull[g] + (i & 1)));
        mbar_arrive(smem_u32(s_empty + st));
      }
      next_stage();
    }
  }

  float2 acc[kCols / 2];                           // rows first .. of the tile of X, two by two
  const bool adds = warp >= 8 && warp < kLoad;
  const int first = (warp - 8) / 8 * kCols;
  if (adds) {
#pragma unroll
    for (int t = 0; t < kCols / 2; ++t) acc[t] = make_float2(0.f, 0.f);
    const int g = (warp - 8) >> 2 & 1, r = threadIdx.x & 127;
    const uint32_t D = tmem + ((uint32_t)((warp & 3) * 32) << 16) + g * kTcTile + 2 * kTcA + first;
    uint32_t q = 0;                                // groups so far
    bool going = true;
    while (w.more() && going) {
      const int t0 = w.t_tile * NT + first;
      const uint32_t scales = ws + (st * kTcTiles + g) * a.w.tile_bytes + kW4Codes + 2 * w4_place(r);
#pragma unroll 1
      for (int k = 0; k < per; ++k, ++q) {
        if (!warp_wait(smem_u32(s_dfull[g] + (q & 1)), (q >> 1) & 1, abort, a.flag)) {
          going = false;
          break;
        }
        const float s1 = (E4M3 ? 512.f : 1.f) * lds_half(scales + 2 * k * kW4Rows);
        const float2 s = make_float2(s1, s1);
        fence_after();
#pragma unroll
        for (int c = 0; c < kCols; c += kChunk) {
          float2 v[kChunk / 2], f[kChunk / 2];
          if constexpr (E4M3) {
            tmem_ld8(D + (q & 1) * NT + c, v);
#pragma unroll
            for (int t = 0; t < kChunk / 2; t += 2) {
              const float4 x = lds_f32x4(ss + (st * NT + first + c + 2 * t) * 4);
              f[t] = mul2(s, make_float2(x.x, x.y));
              f[t + 1] = mul2(s, make_float2(x.z, x.w));
            }
            tmem_wait_ld8(v);
          } else {
            tmem_ld16(D + (q & 1) * NT + c, v);
            tmem_wait_ld16(v);
          }
#pragma unroll
          for (int t = 0; t < kChunk / 2; ++t) acc[c / 2 + t] = fma2(v[t], E4M3 ? f[t] : s, acc[c / 2 + t]);
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(s_dempty[g] + (q & 1)));
      }
      if (lane == 0) mbar_arrive(smem_u32(s_empty + st));
      next_stage();
      const int n = (w.n_band * kTcTiles + g) * kW4Rows + r;
      if (w.next()) {                              // a band of this CTA's own
        float* to = a.y + (size_t)t0 * a.w.N + n;
#pragma unroll
        for (int t = 0; t < kCols; ++t, to += a.w.N) {
          if (n < a.w.N && t0 + t < a.T) *to = t % 2 ? acc[t / 2].y : acc[t / 2].x;
          if (t % 2) acc[t / 2] = make_float2(0.f, 0.f);
        }
      }
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  pdl_leave();
  if (warp == kLoad) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTcCols));
  const int band = w.shared_band();
  if (w.split == 1 || band >= w.bands) return;     // (for all CTAs of the cluster)
  const int col = threadIdx.x & 255;
  const uint32_t sums = xs + 4 * col;              // [NT][256] fp32; every stage has been read
  if (adds) {
#pragma unroll
    for (int t = 0; t < kCols; ++t) sts_f32(sums + (first + t) * 1024, t % 2 ? acc[t / 2].y : acc[t / 2].x);
  }
  cluster_sync();
  const int t0 = band / p.across * NT, n = band % p.across * 256 + col;
  if (adds && n < a.w.N) {                         // rows of X: this CTA's share, in kAdd / 8 turns
    const int rows = min(NT, a.T - t0), end = rows * (w.rank + 1) / w.split;
    cluster_sums(sums, 1024, w.split, rows * w.rank / w.split + (warp - 8) / 8, end, kAdd / 8, a.y + (size_t)t0 * a.w.N + n, a.w.N);
  }
  cluster_sync();
}

// Few rows of X: mma.sync m16n8k16, whose operands are registers, so that no warp waits for another. A band is 128 rows, 32 for each of
// the four warps; warp 4 asks for the copies. The codes become the integers code - zero in fp16, 8-bit X becomes fp16, both
// exact. A lane's weights of two products are one word of codes for each row, its part of X the columns 8 q .. 8 q + 7 of a 32-column
// run, which stand where the products want 2 q, 2 q + 1, 8 + 2 q, 9 + 2 q (the sum over columns does not mind).
// Where a cluster shares a band, each CTA puts its sums of a row of X into the shared memory of the CTA that the row belongs to, while others
// may still work (16 rows of 4096 x 4096: 7.0 us; 8.8 when it read them there after a barrier, and left after another).
// No unit is full (one row of 28672 x 4096: issue slots 51 % busy, the ALU 44, the pipe of fp16 operations 36, tensor 20, HBM 47): of 3.4
// warps an SM quarter 0.9 are ready, and start and end take 4 of 17 us. 16 rows of W a warp and twice as many warps are slower all
// the same (one row of 128256 x 4096: 65 us for 55; 16 rows of 28672 x 4096: 22 for 20), as the loop's own instructions then serve
// half as many codes.
constexpr int kRowsThreads = 160;

// Row of an 8-row tile of X that lane group g reads, and the column of a product that is its: rows that one access of
// a warp touches together lie in different banks of the swizzled tile.
template <bool E4M3>
__host__ __device__ constexpr int x_row(int g) { return E4M3 ? (g & 3) * 2 + (g >> 2) : (g >> 1) + (g & 1) * 4; }

__device__ __forceinline__ void mma_f16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t e4m3_f16(uint32_t two) {   // the lower two bytes
  uint32_t r;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}\n" : "=r"(r) : "r"(two));
  return r;
}

template <bool E4M3, int NT>
struct RowsShape {
  static constexpr int kCtas = NT == 8 ? 4 : NT == 16 ? 3 : 2;   // an SM, by registers
};

template <bool E4M3, int NT>
__global__ void __launch_bounds__(kRowsThreads, RowsShape<E4M3, NT>::kCtas)
    gemm4_rows_kernel(const __grid_constant__ CUtensorMap map_x, const Gemm4Args a, const Gemm4Plan p) {
  constexpr int U = NT / 8;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t xs = (smem_u32(smem_raw) + 1023) & ~1023u, ws = xs + p.stages * p.x_bytes;   // [stages] X; [stages] tiles; [stages][NT] scales of X
  const uint32_t ss = ws + p.stages * a.w.tile_bytes, rs = ss + (E4M3 ? p.stages * NT * 4 : 0);   // rs: sums from the cluster
  __shared__ uint64_t s_full[kMaxStages], s_empty[kMaxStages];
  __shared__ unsigned s_abort;
  volatile unsigned* abort = &s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3, row0 = warp * 32 + g;
  Gemm4Walk w(a, p);
  const int per = 4 >> a.lg, last = (1 << a.lg) - 1;   // groups of a block; 32-column steps of one, less one
  if (threadIdx.x == 0) {
    s_abort = 0;
    prefetch_map(&map_x);
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(smem_u32(s_full + i), E4M3 ? 33 : 1);
      mbar_init(smem_u32(s_empty + i), 4);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  pdl_wait();
  __syncthreads();

  if (w.split > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;");
  float acc[2][U][4] = {};                         // rows g and g + 8 of two 16-row tiles, columns tok[2 u], tok[2 u + 1]
  auto tok = [&](int i) { return i / 2 * 8 + x_row<E4M3>(2 * q + i % 2); };   // rows of X that are this lane's columns
  if (warp == 4) {
    uint64_t pol_w, pol_x;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol_w));
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(pol_x));
    int st = 0, issued = 0;
    uint32_t ph = 1;
    for (; w.more(); w.next()) {
      if (!warp_wait(smem_u32(s_empty + st), ph, abort, a.flag)) break;
      const uint32_t fb = smem_u32(s_full + st), x = xs + st * p.x_bytes;
      if (elect()) {
        mbar_expect_tx(fb, p.x_bytes + a.w.tile_bytes);
        bulk_load(ws + st * a.w.tile_bytes, a.w4 + ((size_t)w.n_band * a.w.k_tiles + w.kb) * a.w.tile_bytes,
                  a.w.tile_bytes, fb, pol_w);
        tma_2d(x, &map_x, w.kb * kW4Cols, w.t_tile * NT, fb, pol_x);
        if (!E4M3) tma_2d(x + NT * 128, &map_x, w.kb * kW4Cols + 64, w.t_tile * NT, fb, pol_x);
      }
      __syncwarp();
      if constexpr (E4M3) {
        const int t0 = w.t_tile * NT;
        x_scales_to(ss + st * NT * 4, a.x_scales + (size_t)t0 * a.w.k_tiles + w.kb, a.T - t0, a.w.k_tiles, NT, lane, fb);
      }
      ++issued;
      if (++st == p.stages) st = 0, ph ^= 1;
    }
    for (int j = max(0, issued - p.stages); j < issued; ++j)   // copies under way land before the CTA ends
      mbar_settle(smem_u32(s_full + j % p.stages), (uint32_t)((j / p.stages) & 1), a.flag);
  } else {
    const uint32_t piece = w4_piece(row0, q);      // (rows 8 apart: 512 bytes)
    uint32_t x_at[E4M3 ? 4 : 2];                   // columns 8 q .. of a run of X's row
#pragma unroll
    for (int j = 0; j < (E4M3 ? 4 : 2); ++j)
      x_at[j] = x_row<E4M3>(g) * 128 + (E4M3 ? ((2 * j + (q >> 1)) ^ x_row<E4M3>(g)) * 16 + (q & 1) * 8 : ((4 * j + q) ^ x_row<E4M3>(g)) * 16);
    int st = 0;
    uint32_t ph = 0;
    while (w.more()) {
      const int t0 = w.t_tile * NT;
      if (!warp_wait(smem_u32(s_full + st), ph, abort, a.flag)) break;
      const uint32_t xt = xs + st * p.x_bytes, tile = ws + st * a.w.tile_bytes;
      float sx[E4M3 ? 2 * U : 1];
      if constexpr (E4M3) {
#pragma unroll
        for (int i = 0; i < 2 * U; ++i) sx[i] = __uint_as_float(lds32(ss + (st * NT + tok(i)) * 4));
      }
      const uint32_t scales = tile + kW4Codes + 2 * (warp * 32 + g * 4), zeros = tile + kW4Codes + per * (kW4Rows * 2) + warp * 32 + g * 4;
      uint4 c[4];                                  // rows g, g + 8, g + 16, g + 24 of the warp's
#pragma unroll
      for (int m = 0; m < 4; ++m) c[m] = lds128(tile + piece + 512 * m);
      float d[2][U][4], sc[4];
      uint32_t z0[4], z1[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if ((j & last) == 0) {
          const int at = (j >> a.lg) * kW4Rows;
          const uint2 v = lds64(scales + 2 * at);
          const uint32_t z = lds32(zeros + at);
          const float2 s01 = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
          const float2 s23 = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
          sc[0] = s01.x, sc[1] = s01.y, sc[2] = s23.x, sc[3] = s23.y;
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            z0[m] = 0x64006400u + (z >> (8 * m) & 255u) * 0x00010001u;     // 1024 + zero
            z1[m] = hsub2(0x63806380u, z0[m]);                              // 960 - (1024 + zero)
          }
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int u = 0; u < U; ++u) d[m][u][0] = d[m][u][1] = d[m][u][2] = d[m][u][3] = 0.f;
        }
        uint32_t f[4][4];
#pragma unroll
        for (int m = 0; m < 4; ++m) codes_f16(j == 0 ? c[m].x : j == 1 ? c[m].y : j == 2 ? c[m].z : c[m].w, z0[m], z1[m], f[m]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          uint32_t b[4];
          if constexpr (E4M3) {
            const uint2 v = lds64(xt + u * 1024 + x_at[j]);
            b[0] = e4m3_f16(v.x), b[1] = e4m3_f16(v.x >> 16), b[2] = e4m3_f16(v.y), b[3] = e4m3_f16(v.y >> 16);
          } else {
            const uint4 v = lds128(xt + (j >> 1) * (NT * 128) + u * 1024 + x_at[j & 1]);
            b[0] = v.x, b[1] = v.y, b[2] = v.z, b[3] = v.w;
          }
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            mma_f16(d[m][u], f[2 * m][0], f[2 * m + 1][0], f[2 * m][1], f[2 * m + 1][1], b[0], b[1]);
            mma_f16(d[m][u], f[2 * m][2], f[2 * m + 1][2], f[2 * m][3], f[2 * m + 1][3], b[2], b[3]);
          }
        }
        if ((j & last) == last) {
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                acc[m][u][e] = fmaf(d[m][u][e], E4M3 ? sc[2 * m + (e >> 1)] * sx[2 * u + (e & 1)] : sc[2 * m + (e >> 1)], acc[m][u][e]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(s_empty + st));
      if (++st == p.stages) st = 0, ph ^= 1;
      const int n0 = w.n_band * kW4Rows + row0;
      if (w.next()) {                              // a band of this CTA's own
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int t = t0 + tok(2 * u + (e & 1)), n = n0 + m * 16 + (e >> 1) * 8;
              if (t < a.T && n < a.w.N) a.y[(size_t)t * a.w.N + n] = acc[m][u][e];
              acc[m][u][e] = 0.f;
            }
      }
    }
  }
  if (w.split == 1) return;
  const int band = w.shared_band();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // all CTAs' shared memory is there
  if (band >= w.bands) return;                     // (for all CTAs of the cluster)
  // Each row of X belongs to one CTA, which gets the others' sums for it, [CTA][its rows][128], put side by side here first
  const int t0 = band / p.across * NT, rows = min(NT, a.T - t0), most = (rows + w.split - 1) / w.split;
  constexpr int kPitch = 136;                      // rows of X 4 apart meet no bank twice
  __syncthreads();                                 // every stage has been read
  if (warp < 4) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) sts_f32(xs + 4 * (tok(2 * u + (e & 1)) * kPitch + row0 + m * 16 + (e >> 1) * 8), acc[m][u][e]);
    __syncwarp();
    for (int i = lane; i < rows * 8; i += 32) {    // four of the warp's 32 weight rows
      const int t = i / 8, at = warp * 32 + i % 8 * 4;
      const int owner = (w.split * (t + 1) + rows - 1) / rows - 1, slot = w.rank * most + t - rows * owner / w.split;
      const float4 v = lds_f32x4(xs + 4 * (t * kPitch + at));
      uint32_t there;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(rs + (slot * kW4Rows + at) * 4), "r"(owner));
      asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(there), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
    }
  }
  cluster_sync();
  const int n = band % p.across * kW4Rows + threadIdx.x;
  if (warp < 4 && n < a.w.N) {
    const int first = rows * w.rank / w.split, own = rows * (w.rank + 1) / w.split - first;
    float* to = a.y + (size_t)(t0 + first) * a.w.N + n;
    auto sums = [&](auto wide, auto ctas) {        // so many rows, and CTAs, at a time
      constexpr int R = decltype(wide)::value, C = decltype(ctas)::value;
      for (int t = 0; t < own; t += R) {
        float sum[R] = {};
#pragma unroll C
        for (int c = 0; c < w.split; ++c)
#pragma unroll
          for (int i = 0; i < R; ++i)
            sum[i] += __uint_as_float(lds32(rs + ((c * most + min(t + i, own - 1)) * kW4Rows + threadIdx.x) * 4));
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (t + i < own) to[(size_t)(t + i) * a.w.N] = sum[i];
      }
    };
    if (own == 1) sums(std::integral_constant<int, 1>(), std::integral_constant<int, 8>());
    else sums(std::integral_constant<int, 4>(), std::integral_constant<int, 2>());
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_tiled() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    cudaDriverEntryPointQueryResult q;
    void* f = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// CTAs of a cluster that share a band, or 1. What is compared: 0.19 us a block for an SM (HBM's part of it), 0.3 for a CTA by itself (kernel
// of few rows), 0.1 a CTA for the joining; so a band is shared while that spreads the blocks better, or lets more CTAs work at once, and
// all clusters find room together: 23 clusters of 6 CTAs that fill an SM each do, a 24th waits for a whole turn (6144 x 4096, 64 rows:
// half as long again).
template <typename Room>
int gemm4_split(int bands, int blocks, int slots, int sms, Room room) {
  int best = 1;
  double least = 1e30;
  for (int c = 1; c <= std::min(8, blocks); ++c) {
    const int64_t ctas = (int64_t)bands * c;
    if (c > 1 && (ctas > slots || bands > room(c))) continue;
    const int own = (blocks + c - 1) / c;
    const double cost = std::max((double)((ctas + sms - 1) / sms) * own * 0.19, own * 0.3) + 0.1 * c;
    if (cost < least) least = cost, best = c;
  }
  return best;
}

template <auto kernel>
pic_status launch_gemm4(const Gemm4Args& a, bool e4m3, int rows, int tiles, int threads, int per_sm, int ring, int dev,
                        cudaStream_t st) {
  const int sms = device_sms(dev);
  Gemm4Plan p;
  p.x_bytes = rows * kW4Cols * (e4m3 ? 1 : 2);
  const int stage = p.x_bytes + tiles * a.w.tile_bytes + (e4m3 ? 4 * rows : 0);
  p.across = (a.w.n_tiles + tiles - 1) / tiles;
  p.bands = p.across * ((a.T + rows - 1) / rows);
  const auto enc = encode_tiled();
  CUtensorMap map;
  const cuuint64_t dims[2] = {(cuuint64_t)a.w.K, (cuuint64_t)a.T};
  const cuuint64_t strides[1] = {(cuuint64_t)a.x_stride * (e4m3 ? 1 : 2)};
  const cuuint32_t box[2] = {e4m3 ? 128u : 64u, (cuuint32_t)rows}, step[2] = {1, 1};
  if (!enc || enc(&map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(a.x), dims,
                  strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return fail(PIC_ERR_CUDA, "4-bit gemm: cuTensorMapEncodeTiled failed");
  static SharedMemory<kernel> memory;
  PIC_CUDA(memory.allow(dev, 1024 + ring));
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = 1024 + ring;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  const int slots = per_sm * sms, rest = p.bands % slots;
  int split = 1;
  p.whole = p.bands;
  if (p.bands < slots) {
    static ClusterRoom<kernel> fits;
    split = gemm4_split(p.bands, a.w.k_tiles, slots, sms, [&](int c) { return fits.clusters(dev, c, cfg, at, sms); });
  } else if (rest > 0 && rest <= slots / 2 && slots % 2 == 0 && a.w.k_tiles > 1) {
    split = 2;
  }
  if (split > 1) p.whole -= rest;
  const int t_most = std::min(rows, a.T), recv = split > 1 && tiles == 1 ? split * ((t_most + split - 1) / split) * kW4Rows * 4 : 0;
  p.stages = std::min(kMaxStages, (ring - recv) / stage);
  cfg.dynamicSmemBytes = 1024 + (size_t)p.stages * stage + recv;
  cfg.gridDim = dim3(p.bands >= slots ? (unsigned)slots : (unsigned)(p.bands * split));
  at[0].val.clusterDim.x = split;
  PIC_CUDA(cudaLaunchKernelEx(&cfg, kernel, map, a, p));
  return PIC_OK;
}

template <bool E4M3, int NT>
pic_status launch_gemm4_rows(const Gemm4Args& a, int dev, cudaStream_t st) {
  constexpr int kCtas = RowsShape<E4M3, NT>::kCtas;
  return launch_gemm4<gemm4_rows_kernel<E4M3, NT>>(a, E4M3, NT, 1, kRowsThreads, kCtas,
                                                   (kCtas == 4 ? 54 : kCtas == 3 ? 73 : 111) * 1024, dev, st);
}

template <bool E4M3, int NT>
pic_status launch_gemm4_tc(const Gemm4Args& a, int dev, cudaStream_t st) {
  return launch_gemm4<gemm4_tc_kernel<E4M3, NT>>(a, E4M3, NT, kTcTiles, TcShape<E4M3, NT>::kThreads, 1, 222 * 1024, dev, st);
}

template <bool E4M3>
pic_status launch_gemm4(const Gemm4Args& a, int dev, cudaStream_t st) {
  // tcgen05 (us; in brackets mma.sync), 17 and 64 rows in fp16, then e4m3: 8192 x 4096 (2048 blocks) 10.9 (12.6), 12.8 (19.8); 11.1 (13.8),
  // 14.1 (22.6). 6144 x 4096 (1536) 10.1 (11.2), 12.6 (15.2); 10.2 (12.4), 13.8 (17.1). 4096 x 4096 (1024) 9.3 (8.3), 11.3 (12.4); 9.5
  // (9.0), 13.2 (13.8). 4096 x 2048 (512), where its wide bands leave SMs idle, 7.5 (6.3), 9.3 (8.2); 7.7 (6.8), 10.7 (9.1). LM head of
  // 128256 x 4096: 32 rows 76 (110), but 16 rows 75 (70). Few tall bands lose little by it: 128 x 199936 120 (134), 131 (134); 118 (153), 165 (153).
  if (a.T > kFewRows && (int64_t)a.w.n_tiles * a.w.k_tiles * ((a.T + 31) / 32) >= kTcBlocks)
    return a.T <= 32 ? launch_gemm4_tc<E4M3, 32>(a, dev, st) : launch_gemm4_tc<E4M3, 64>(a, dev, st);
  return a.T <= 8 ? launch_gemm4_rows<E4M3, 8>(a, dev, st) : a.T <= 16 ? launch_gemm4_rows<E4M3, 16>(a, dev, st) : launch_gemm4_rows<E4M3, 32>(a, dev, st);
}

template <typename T>
void launch_pack4(const T* W, void* out, const W4Shape& s, unsigned* flag, cudaStream_t st) {
  const int grid = s.n_tiles * s.k_tiles;
  // loads of 32 bytes a lane where W's alignment allows (28672 x 4096: fp32 89 us for 109, 16-bit weights the same)
  if ((uintptr_t)W % 32 == 0) pack4_kernel<true><<<grid, kPackThreads, 0, st>>>(W, (uint8_t*)out, s, flag);
  else pack4_kernel<false><<<grid, kPackThreads, 0, st>>>(W, (uint8_t*)out, s, flag);
}

constexpr int kMaxRows = 1 << 20;   // of X

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
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == PIC_F32) launch_pack4((const float*)W, out, s, flag, st);
  else if (dtype == PIC_F16) launch_pack4((const __half*)W, out, s, flag, st);
  else launch_pack4((const __nv_bfloat16*)W, out, s, flag, st);
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
  if (T > kMaxRows) return fail(PIC_ERR_CAPACITY, "4-bit gemm: more than 2^20 rows");
  if (misaligned(W4, 128) || misaligned(X, 16) || misaligned(Y, 16) || misaligned(x_scales, 4))
    return fail(PIC_ERR_INVALID_ARG, "4-bit gemm: X and Y must be 16-byte, the packed weights 128-byte aligned");
  const W4Shape s = w4_shape(N, K, group);
  if ((int64_t)s.n_tiles * ((T + 31) / 32) > INT_MAX / 8) return fail(PIC_ERR_CAPACITY, "4-bit gemm: too many rows of both");
  const size_t y_bytes = (size_t)T * N * 4;
  if (overlap(Y, y_bytes, X, ((size_t)(T - 1) * x_stride + K) * (e4m3 ? 1 : 2)) ||
      overlap(Y, y_bytes, W4, (size_t)s.n_tiles * s.k_tiles * s.tile_bytes) ||
      (x_scales && overlap(Y, y_bytes, x_scales, (size_t)T * s.k_tiles * 4)))
    return fail(PIC_ERR_INVALID_ARG, "4-bit gemm: Y must not overlap the packed weights, X or its scales");
  int dev = 0;
  PIC_CUDA(cudaGetDevice(&dev));
  Gemm4Args a{s, (const uint8_t*)W4, X, x_stride, x_scales, Y, T, group == 32 ? 0 : group == 64 ? 1 : 2, nullptr};
  pic_status e = batch_flag_address(&a.flag);
  if (e != PIC_OK) return e;
  return e4m3 ? launch_gemm4<true>(a, dev, (cudaStream_t)stream) : launch_gemm4<false>(a, dev, (cudaStream_t)stream);
}

}  // extern "C"
