// Batched paged attention over device-resident page tables: a sliding window with a few first
// tokens that stay visible, and a batch behind one shared prefix.
//
//   out[t][h] = sum_u p_u V[u][g] / sum_u p_u,   p_u = exp(q[t][h] . RoPE(K[u][g], pos(u)) / sqrt(D))
//
// over the keys u that row t sees; g = h / (H / G). The plan (batch_plan.h) cuts the work evenly
// over the CTAs; items cut at a share's edge, and the two segments of a prefix batch, are joined by
// the merge kernel from their normalized sums, maxima and denominators (log-sum-exp), in a fixed
// order.
//
// This file: the kernel of fp32 pools (fp32 arithmetic), the merge kernel and the C entry points; bf16 pools
// go to the tensor-core kernel.
#include <mutex>

#include "batch_internal.cuh"

namespace pic {

namespace {

__device__ unsigned g_batch_flag = 0;   // kBatch* bits since the last pic_sync

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThreads = 256;
constexpr int kRows = 16;             // rows (token x head) of an item
constexpr int kPages = 4;             // pages of a key tile
constexpr int kKeys = kPages * kPage;

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void put4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
template <int D> struct SimtSmem {
  float q[kRows][D];
  float k[kKeys][D + 4];              // + 4: rows of neighbouring keys start in different banks
  float v[kKeys][D];
  float p[kRows][kKeys];
  int pos[kKeys];                     // key positions (INT_MAX: no key)
  PageMeta page[kPages];
  PlanShared plan;
};

// 16 threads per row: each has 4 of the tile's 64 scores and D / 16 of the row's output columns.
// fp32 throughout: 2 D FMA per (row, key) pair bound it where rows are many, the pool's bytes
// where they are few (two to four CTAs per SM hide the loads' latency).
template <int D>
__global__ void __launch_bounds__(kThreads) batch_simt_kernel(const __grid_constant__ BatchArgs a) {
  using T = float;
  using A = float;
  extern __shared__ __align__(16) uint8_t raw[];
  SimtSmem<D>& s = *reinterpret_cast<SimtSmem<D>*>(raw);
  const BatchView& v = a.v;
  asm volatile("griddepcontrol.launch_dependents;");
  const BatchShare sh = plan_batch<kThreads>(a, s.plan);
  const int tid = threadIdx.x, row = tid >> 4, lane = tid & 15;
  constexpr int NO = D / 64;          // float4 groups of output columns per thread
  const float scale = kLog2e * rsqrtf((float)D);
  unsigned bad = 0;
  for (int bi = sh.first; bi <= sh.last; ++bi) {
    const BatchBlock b = a.blocks[bi];
    const int nt = block_tiles(v, b), c = tile_cost(v, b);
    const unsigned ilen = item_len(v, b);
    const int tok = row * v.rep_inv >> 16, hh = row - tok * v.rep;
    const bool mine = tok < b.nrows && row < v.rb * v.rep;
    const int qp = b.req < 0 ? INT_MAX - 1 : b.pos0 + tok;
    for (int g = 0; g < v.G; ++g) {
      const unsigned start = b.cum + g * ilen;
      const int j0 = tile_lower(v, start, nt, c, sh.x0), j1 = tile_lower(v, start, nt, c, sh.x1);
      if (j0 >= j1) continue;
      const size_t head = mine ? (size_t)(b.row0 + tok) * a.H + g * v.rep + hh : 0;
      const A* q = static_cast<const A*>(a.q) + head * D;
      for (int i = 0; i < NO; ++i) {
        float4 x = mine ? load4(q + 4 * lane + 64 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
        x.x *= scale, x.y *= scale, x.z *= scale, x.w *= scale;
        *reinterpret_cast<float4*>(&s.q[row][4 * lane + 64 * i]) = x;
      }
      float m = -INFINITY, l = 0.f;
      float4 o[NO] = {};
      for (int j = j0; j < j1; ++j) {
        __syncthreads();              // the tile before is used up
        if (tid < kPages) {
          const int i = j * kPages + tid;
          s.page[tid] = i < b.nv ? page_meta(v, b, page_raw(v, b, i), bad) : PageMeta{0, 0, 0};
        }
        __syncthreads();
        // K rotated by its position, V; rows that hold no key are zero
        const T* kl = static_cast<const T*>(a.k_layer);
        const T* vl = static_cast<const T*>(a.v_layer);
        for (int u = tid; u < kKeys * (D / 8); u += kThreads) {
          const int key = u / (D / 8), i = u % (D / 8) * 4, r = key % kPage;
          const PageMeta pm = s.page[key / kPage];
          float4 y1 = make_float4(0.f, 0.f, 0.f, 0.f), y2 = y1, z1 = y1, z2 = y1;
          if (pm.rows >> r & 1u) {
            const size_t at = (((size_t)pm.blk * v.G + g) * kPage + r) * D;
            const float4 x1 = load4(kl + at + i), x2 = load4(kl + at + D / 2 + i);
            z1 = load4(vl + at + i);
            z2 = load4(vl + at + D / 2 + i);
            const float4* f = reinterpret_cast<const float4*>(a.rope_cs + (size_t)(pm.pos + r) * (D / 2) + i);
            const float4 f0 = f[0], f1 = f[1];
            y1 = make_float4(x1.x * f0.x - x2.x * f0.y, x1.y * f0.z - x2.y * f0.w, x1.z * f1.x - x2.z * f1.y,
                             x1.w * f1.z - x2.w * f1.w);
            y2 = make_float4(x2.x * f0.x + x1.x * f0.y, x2.y * f0.z + x1.y * f0.w, x2.z * f1.x + x1.z * f1.y,
                             x2.w * f1.z + x1.w * f1.w);
          }
          *reinterpret_cast<float4*>(&s.k[key][i]) = y1;
          *reinterpret_cast<float4*>(&s.k[key][D / 2 + i]) = y2;
          *reinterpret_cast<float4*>(&s.v[key][i]) = z1;
          *reinterpret_cast<float4*>(&s.v[key][D / 2 + i]) = z2;
        }
        if (tid < kKeys) {
          const PageMeta pm = s.page[tid / kPage];
          s.pos[tid] = pm.rows >> tid % kPage & 1u ? pm.pos + tid % kPage : INT_MAX;
        }
        __syncthreads();
        float x[4] = {};
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
          const float4 qv = *reinterpret_cast<const float4*>(&s.q[row][d]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 kv = *reinterpret_cast<const float4*>(&s.k[lane + 16 * e][d]);
            x[e] += qv.x * kv.x + qv.y * kv.y + qv.z * kv.z + qv.w * kv.w;
          }
        }
        float mx = m;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int u = s.pos[lane + 16 * e];
          const bool seen = b.req < 0 ? u != INT_MAX : sees(v, qp, u);
          if (!seen) x[e] = -INFINITY;
          mx = fmaxf(mx, x[e]);
        }
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d, 16));
        const float ref = mx == -INFINITY ? 0.f : mx;   // nothing seen so far: every p is 0
        const float keep = exp2f(m - ref);
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = exp2f(x[e] - ref);
          s.p[row][lane + 16 * e] = p;
          sum += p;
        }
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d, 16);
        l = l * keep + sum;
        m = mx;
#pragma unroll
        for (int i = 0; i < NO; ++i) o[i].x *= keep, o[i].y *= keep, o[i].z *= keep, o[i].w *= keep;
        __syncwarp();                 // a row's p is written and read by one half-warp
#pragma unroll 8
        for (int key = 0; key < kKeys; ++key) {
          const float p = s.p[row][key];
#pragma unroll
          for (int i = 0; i < NO; ++i) {
            const float4 y = *reinterpret_cast<const float4*>(&s.v[key][4 * lane + 64 * i]);
            o[i].x += p * y.x, o[i].y += p * y.y, o[i].z += p * y.z, o[i].w += p * y.w;
          }
        }
      }
      const bool whole = j0 == 0 && j1 == nt;
      if (mine) {
        const float inv = l == 0.f ? 0.f : 1.f / l;   // NaN stays NaN
        float* po;
        float2* pml;
        if (whole && v.pre_len == 0) {
          A* dst = static_cast<A*>(a.out) + head * D;
          for (int i = 0; i < NO; ++i)
            put4(dst + 4 * lane + 64 * i, make_float4(o[i].x * inv, o[i].y * inv, o[i].z * inv, o[i].w * inv));
        } else {
          if (whole) {
            const size_t at = (b.req < 0 ? 0 : (size_t)v.T * a.H) + head;
            po = a.seg_o + at * D;
            pml = a.seg_ml + at;
          } else {
            const size_t at = (size_t)part_slot(blockIdx.x, start, sh.x0) * a.part_rows + row;
            po = a.part_o + at * D;
            pml = a.part_ml + at;
          }
          for (int i = 0; i < NO; ++i)
            put4(po + 4 * lane + 64 * i, make_float4(o[i].x * inv, o[i].y * inv, o[i].z * inv, o[i].w * inv));
          if (lane == 0) *pml = make_float2(m, l);
        }
      }
    }
  }
  batch_flag(a.flag, bad);
}

// Joins what the attention kernels left in parts: GL lanes per (row, head), D / GL columns per
// lane; result = sum_i w_i O_i / sum_i w_i with w_i = l_i 2^(m_i - max). Rows that see no key
// (sum 0) give zeros. A lane finds one part each (of the row's item of the prefix, then of its own);
// their rows are read several at a time. A batch with a prefix merges every row, of few parts: 8 lanes a row, grid
// (own row blocks, G, rows of a block / 32); one without only the items that a share's edge cuts, of up to dozens
// of parts: 32 lanes, grid (shares, 1, rows / 8). Latency bounds both, five loads that depend on one another a row.
template <int N, typename A>
__device__ __forceinline__ void store_columns(A* dst, const float* o, float f) {
  alignas(16) A x[N];
#pragma unroll
  for (int e = 0; e < N; ++e) x[e] = from_f<A>(o[e] * f);
  constexpr int B = N * sizeof(A);
  if constexpr (B % 16 == 0) {
#pragma unroll
    for (int i = 0; i < B / 16; ++i) reinterpret_cast<uint4*>(dst)[i] = reinterpret_cast<const uint4*>(x)[i];
  } else if constexpr (B == 8) {
    *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(x);
  } else {
    static_assert(B == 4, "");
    *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(x);
  }
}
template <typename A, int D, int GL>
__global__ void __launch_bounds__(256) batch_merge_kernel(const __grid_constant__ MergeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int C = D / GL, V = C < 4 ? C : 4, RPW = 32 / GL;   // columns of a lane, of a load; rows of a warp
  constexpr unsigned kAll = 0xffffffffu;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x % GL, group = (threadIdx.x & 31) / GL;
  int g = blockIdx.y, first = blockIdx.x;
  struct Parts {          // the parts of one item
    unsigned start, U, len;
    int nt, c, c0, n;
  };
  auto parts = [&](const MergeSegment& s, const BatchHead& hd, const BatchBlock& b) {
    Parts p;
    p.U = hd.U, p.len = hd.len;
    p.nt = block_tiles(s.v, b), p.c = tile_cost(s.v, b);
    p.start = b.cum + g * item_len(s.v, b);
    p.c0 = 0, p.n = 1;
    if (p.len) {
      p.c0 = owner(p.len, p.start);
      p.n = owner(p.len, tile_place(s.v, p.start, p.c, p.nt - 1)) - p.c0 + 1;
    }
    return p;
  };
  const BatchHead hd = *a.s[1].head, hp = *a.s[0].head;
  int last = hd.n_blocks - hd.n_prefix - 1;
  if (!a.prefix) {
    const BatchCut cut = a.s[1].cuts[blockIdx.x];
    if (cut.block < 0) return;
    first = last = cut.block;
    g = cut.g;
  }
#pragma unroll 1
  for (int bi = hd.n_prefix + first; bi <= hd.n_prefix + last; bi += gridDim.x) {
    const BatchBlock own = a.s[1].blocks[bi];
    const Parts po = parts(a.s[1], hd, own);
    if (po.n == 1 && !a.prefix) continue;   // the edge fell between the item's tiles and its end: out is written
    const int rows = own.nrows * a.rep;
#pragma unroll 1
    for (int r0 = (blockIdx.z * 8 + warp) * RPW; r0 < rows; r0 += 8 * RPW * gridDim.z) {
      const bool live = r0 + group < rows;
      const int rr = live ? r0 + group : r0, tok = rr * a.rep_inv >> 16, hh = rr - tok * a.rep, t = own.row0 + tok;
      const size_t head = (size_t)t * a.H + g * a.rep + hh;
      const int pb = a.prefix ? (unsigned)t / (unsigned)a.s[0].v.rb : 0;
      Parts pp{};
      if (a.prefix) pp = parts(a.s[0], hp, a.s[0].blocks[pb]);
      float M = -INFINITY, L = 0.f, o[C] = {};
#pragma unroll 1
      for (int i0 = 0; __any_sync(kAll, i0 < pp.n + po.n); i0 += GL) {
        const int i = i0 + lane, seg = i >= pp.n, p = seg ? i - pp.n : i;
        const Parts& q = seg ? po : pp;
        const MergeSegment& s = a.s[seg];
        bool on = i < pp.n + po.n;
        size_t at = (size_t)seg * a.T * a.H + head;   // a whole item's result
        const bool whole = q.n == 1;
        if (on && !whole) {
          const unsigned x0 = share(q.U, q.len, q.c0 + p), x1 = share(q.U, q.len, q.c0 + p + 1);
          on = tile_lower(s.v, q.start, q.nt, q.c, x0) < tile_lower(s.v, q.start, q.nt, q.c, x1);
          const int lrow = seg ? rr : (t - pb * a.s[0].v.rb) * a.rep + hh;
          at = (size_t)part_slot(q.c0 + p, q.start, x0) * s.part_rows + lrow;
        }
        const float2 x = on ? (whole ? a.seg_ml : s.part_ml)[at] : make_float2(-INFINITY, 0.f);
        const float* src = (whole ? a.seg_o : s.part_o) + at * D;
        float mx = x.x;
#pragma unroll
        for (int d = GL / 2; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, d));
        mx = fmaxf(mx, M);
        const float ref = mx == -INFINITY ? 0.f : mx, keep = exp2f(M - ref), w = x.y * exp2f(x.x - ref);
        float sum = w;
#pragma unroll
        for (int d = GL / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
        M = mx;
        L = L * keep + sum;
#pragma unroll
        for (int e = 0; e < C; ++e) o[e] *= keep;
        // the group's lanes whose part counts
        unsigned left = __ballot_sync(kAll, on && x.y != 0.f) >> (GL * group) & (GL < 32 ? (1u << GL) - 1u : kAll);
        auto add = [&](auto batch) {   // so many rows on their way at once
          constexpr int N = decltype(batch)::value;
          float y[N][C], ww[N];
          const bool any = left != 0;
          int k = 0;
#pragma unroll
          for (int u = 0; u < N; ++u) {
            k = left ? __ffs(left) - 1 : k;    // behind the last row: that row again, with weight 0
            const float wk = __shfl_sync(kAll, w, k, GL);
            const float* row = reinterpret_cast<const float*>(__shfl_sync(kAll, (unsigned long long)src, k, GL)) + lane * C;
            ww[u] = left ? wk : 0.f;
#pragma unroll
            for (int e = 0; e < C; e += V) {
              if constexpr (V == 4) {
                *reinterpret_cast<float4*>(y[u] + e) = any ? *reinterpret_cast<const float4*>(row + e) : make_float4(0.f, 0.f, 0.f, 0.f);
              } else {
                *reinterpret_cast<float2*>(y[u] + e) = any ? *reinterpret_cast<const float2*>(row + e) : make_float2(0.f, 0.f);
              }
            }
            left &= left - 1;
          }
#pragma unroll
          for (int u = 0; u < N; ++u)
#pragma unroll
            for (int e = 0; e < C; ++e) o[e] += ww[u] * y[u][e];
        };
#pragma unroll 1
        while (__any_sync(kAll, left != 0)) {
          if constexpr (GL == 32) {
            if (__popc(left) > 4) add(std::integral_constant<int, 20>());
            else add(std::integral_constant<int, 4>());
          } else {
            add(std::integral_constant<int, 2>());
          }
        }
      }
      if (live) store_columns<C>(static_cast<A*>(a.out) + head * D + lane * C, o, L == 0.f ? 0.f : 1.f / L);
    }
  }
}

template <int D>
cudaError_t launch_simt(const BatchArgs& a, cudaStream_t st) {
  const int smem = (int)sizeof(SimtSmem<D>);
  cudaError_t e = cudaFuncSetAttribute(batch_simt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  batch_simt_kernel<D><<<a.grid, kThreads, smem, st>>>(a);
  return cudaGetLastError();
}

int device_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 152;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 152;
  return n;
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

void launch_batch_merge(const MergeArgs& m, int dtype, int D, cudaStream_t st) {
  // as many warps as a block has rows when the requests have equally many
  const BatchView& v = m.s[1].v;
  const int own = v.T / v.rb + v.n_reqs, rows = pmin(v.rb, pdiv(v.T, v.n_reqs)) * v.rep;
  // 8 lanes a row from where 32 would need more warps than are resident at once (4 CTAs of 8 an SM): rows are then
  // of few parts, as there are many items. 32 requests of 32 rows behind 4096: 117 us, with 32 lanes 120; 64 and 4
  // single rows with 8 lanes: 90 us for 87, 75 for 61.
  const bool many = m.prefix && (long long)v.T * m.H > 32ll * m.grid;
  const int z = pdiv(rows, many ? 32 : 8);
  const dim3 grid = m.prefix ? dim3(own, v.G, z) : dim3(m.grid, 1, z);
  auto go = [&](auto* k8, auto* k32) { launch_dependent(many ? k8 : k32, grid, dim3(256), 0, st, m); };
  if (dtype == PIC_BF16) {
    if (D == 128) go(batch_merge_kernel<__half, 128, 8>, batch_merge_kernel<__half, 128, 32>);
    else go(batch_merge_kernel<__half, 64, 8>, batch_merge_kernel<__half, 64, 32>);
  } else {
    if (D == 128) go(batch_merge_kernel<float, 128, 8>, batch_merge_kernel<float, 128, 32>);
    else go(batch_merge_kernel<float, 64, 8>, batch_merge_kernel<float, 64, 32>);
  }
}

// A call as one or two plans: both segments of a batch in one, or, when the prefix or the own pages
// take K rotated ahead, one each.
struct BatchCall {
  BatchArgs a[2] = {};
  int n = 1;
  bool wide[2] = {false, false};
};

// When K is rotated ahead, once per page, and items have two MMA tiles: when a KV head's keys meet
// enough rows that the MMAs bound the time -- in-kernel rotation, done for every 128 rows anew,
// would then take longer than they do. Below that HBM bounds, and the rotated K (two fp16 parts) with V
// takes five times K's bytes to write and read. These (for the whole tables: the host does not know the lengths) must
// stay within 1 GB.
// Measured on 8 KV heads of 4 query heads, D = 128, ahead and in the kernel, requests of 4096 keys: 512 rows (16 requests
// of 128) 322 and 266 us; 1024 rows (8 of 256) 273 and 257 us, with a window of 1024 120 and 100 us, (256 single rows behind
// a prefix of 16384) 195 and 191 us; 2048 rows (4 of 512) 225 and 248 us, with the window, where fewer of them meet a key,
// 108 and 98 us, (512 single rows behind the prefix) 314 and 359 us; 16384 rows (2 of 4096), window 1024, 200 and 259 us.
constexpr size_t kMaxRotated = (size_t)1 << 30;
double most_slots(int G, int D) { return (double)kMaxRotated / ((double)G * kPage * D * 2 * 3); }
bool wide_pays(long long rows, double slots, int G, int D) { return rows >= 2048 && slots <= most_slots(G, D); }
constexpr int kRowsWithPrefix = 64;

void set_shape(BatchCall& c, int dtype, int T, int n_reqs, int H, int G, int D, int table_stride, int prefix_len,
               int prefix_pages) {
  BatchArgs& a = c.a[0];
  a.v.T = T;
  a.v.n_reqs = n_reqs;
  a.v.G = G;
  a.v.rep = H / G;
  a.v.rep_inv = (65535 + a.v.rep) / a.v.rep;
  a.v.stride = table_stride;
  a.v.pre_len = prefix_len;
  a.v.pre_pages = prefix_pages;
  a.H = H;
  a.D = D;
  if (dtype == PIC_F32) {
    batch_simt_view(a.v);
    a.grid = batch_simt_grid(D);
    return;
  }
  a.grid = device_sms();
  const double own_slots = (double)n_reqs * table_stride;
  const long long own_rows = (long long)pdiv(T, n_reqs) * a.v.rep;
  bool own = wide_pays(own_rows, own_slots, G, D);
  const bool pre = prefix_len > 0 && wide_pays((long long)T * a.v.rep, prefix_pages, G, D);
  // Behind a prefix for the wide kernel the own pages go with it, in one plan, from half an MMA tile of rows a
  // request on and when their tables are at most twice as long as the prefix: one launch less, and 128 rows a tile
  // where they are not many more than one. Together and apart: 32 requests of 32 rows behind 4096, 32 keys of their own:
  // 137 and 147 us; 16 of 32 rows: 85 and 97; 64 of 16 rows, 64 keys: equal, 1024 keys: 260 and 210; 8 of 64 rows behind
  // 8192, 2000 keys: 176 and 179.
  const bool both = pre && own_rows >= kRowsWithPrefix && own_slots <= 2.0 * prefix_pages && own_slots + prefix_pages <= most_slots(G, D);
  if (prefix_len > 0 && (own || pre) && !both) {
    c.n = 2;
    c.a[1] = a;
    c.a[0].v.only = 1;
    c.a[1].v.only = 2;
    c.wide[0] = pre;
    c.wide[1] = own;
    c.a[0].krot_slots = pre ? prefix_pages : 0;
    c.a[1].krot_slots = own ? n_reqs * table_stride : 0;
  } else {
    own = own || both;
    c.wide[0] = own;
    a.krot_own = both ? prefix_pages : 0;
    a.krot_slots = own ? a.krot_own + n_reqs * table_stride : 0;
  }
  for (int i = 0; i < c.n; ++i) {
    BatchView& v = c.a[i].v;
    // Narrow when the requests have no more rows on average than one narrow item (the prefix' rows one at most).
    // Narrow and not: 32 decoding requests 113 and 134 us, 64 of 4 rows and 1000 keys (4 query heads a KV head)
    // 77 and 78, one of 1024 keys 18.2 and 17.7.
    const int most = kRows / v.rep;   // tokens of a narrow item
    const bool narrow = !c.wide[i] && (v.only == 1 || T <= (long long)n_reqs * most) && (v.only == 2 || prefix_len == 0 || T <= most);
    batch_tc_view(v, c.wide[i], narrow);
  }
}

// Whether 31 bits hold the plans' cost axes, if need be with a unit for each tile, and 32 the merge's rows.
bool fits_plan(BatchCall& c) {
  bool fits = 2.0 * c.a[0].v.T * c.a[0].H < 4294967295.0;
  for (int i = 0; i < c.n; ++i) {
    BatchView& v = c.a[i].v;
    const double n_own = v.only == 1 ? 0.0 : v.T / v.rb + (double)v.n_reqs;
    const double n_pre = v.pre_len > 0 && v.only != 2 ? v.T / v.rb + 1.0 : 0.0;
    if (axis_bound(v, n_own, n_pre) >= 2147483647.0) v.cost_item = v.cost_full = v.cost_half = 1;
    fits = fits && axis_bound(v, n_own, n_pre) < 2147483647.0;
  }
  return fits;
}

// Scratch layout of a call (bytes); `base` null: the size alone.
size_t layout(BatchCall& c, char* base) {
  size_t o = 0;
  auto take = [&](size_t n) {
    char* p = base ? base + o : nullptr;
    o += align256(n);
    return p;
  };
  for (int i = 0; i < c.n; ++i) {
    BatchArgs& a = c.a[i];
    const BatchView& v = a.v;
    const bool own = v.only != 1, pre = v.pre_len > 0 && v.only != 2;
    a.n_blocks_max = (own ? v.T / v.rb + v.n_reqs : 0) + (pre ? v.T / v.rb + 1 : 0);
    a.part_rows = (int)(((long long)v.T * v.rep < v.mrows) ? (long long)v.T * v.rep : v.mrows);
    a.head = (BatchHead*)take(sizeof(BatchHead));
    a.base = (int*)take(((size_t)v.n_reqs + 1) * 4);
    a.blocks = (BatchBlock*)take((size_t)a.n_blocks_max * sizeof(BatchBlock));
    a.cuts = (BatchCut*)take((size_t)a.grid * sizeof(BatchCut));
    const size_t rows = 2 * (size_t)a.grid * a.part_rows;
    a.part_ml = (float2*)take(rows * sizeof(float2));
    a.part_o = (float*)take(rows * a.D * 4);
    a.krot = a.krot_slots ? (__half*)take(3 * (size_t)a.krot_slots * v.G * kPage * a.D * 2) : nullptr;
  }
  if (c.a[0].v.pre_len > 0) {
    const size_t rows = 2 * (size_t)c.a[0].v.T * c.a[0].H;
    c.a[0].seg_ml = c.a[1].seg_ml = (float2*)take(rows * sizeof(float2));
    c.a[0].seg_o = c.a[1].seg_o = (float*)take(rows * c.a[0].D * 4);
  }
  return o;
}

bool shape_ok(int dtype, int T, int n_reqs, int H, int G, int D) {
  return (dtype == PIC_F32 || dtype == PIC_BF16) && T >= 1 && n_reqs >= 1 && G >= 1 && H >= 1 && H % G == 0 &&
         (D == 64 || D == 128);
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// c.a[0] holds the caller's pointers and numbers.
pic_status run(BatchCall& c, int dtype, int T, int n_reqs, int H, int G, int D, void* scratch, size_t scratch_bytes,
               cudaStream_t st) {
  const BatchView v0 = c.a[0].v;
  set_shape(c, dtype, T, n_reqs, H, G, D, v0.stride, v0.pre_len, v0.pre_pages);
  if (!fits_plan(c))
    return fail(PIC_ERR_CAPACITY, "batch too large: rows x heads, or row blocks x KV heads x pages of a table row");
  if (scratch_bytes < layout(c, nullptr)) return fail(PIC_ERR_INVALID_ARG, "attention scratch too small");
  unsigned* flag = nullptr;
  pic_status e = batch_flag_address(&flag);
  if (e != PIC_OK) return e;
  layout(c, (char*)scratch);
  MergeArgs m{};
  for (int i = 0; i < c.n; ++i) {
    BatchArgs& a = c.a[i];
    a.flag = flag;
    if (dtype == PIC_BF16) {
      if (c.wide[i] && (e = launch_batch_rotate(a, st)) != PIC_OK) return e;
      if ((e = launch_batch_tc(a, c.wide[i], st)) != PIC_OK) return e;
    } else {
      launch_batch_simt(a, st);
      PIC_CUDA(cudaGetLastError());
    }
  }
  for (int i = 0; i < 2; ++i) {
    const BatchArgs& a = c.a[c.n == 2 ? i : 0];
    m.s[i] = MergeSegment{a.v, a.head, a.blocks, a.cuts, a.part_ml, a.part_o, a.part_rows};
    m.grid = a.grid;
  }
  m.T = T, m.H = H, m.G = G, m.rep = H / G;
  m.rep_inv = c.a[0].v.rep_inv;
  m.prefix = v0.pre_len > 0;
  m.seg_ml = c.a[0].seg_ml, m.seg_o = c.a[0].seg_o;
  m.out = c.a[0].out;
  launch_batch_merge(m, dtype, D, st);
  PIC_CUDA(cudaGetLastError());
  return PIC_OK;
}

// What both calls check: the shapes, pointers and their alignment.
pic_status check_common(int32_t dtype, int32_t T, int32_t n_reqs, int32_t H, int32_t G, int32_t D, const void* q,
                        const int32_t* row_start, const int32_t* kv_len, const int32_t* block_table,
                        int32_t table_stride, const int32_t* page_pos, const int32_t* n_pages, const void* k_layer,
                        const void* v_layer, int32_t pool_blocks, const void* rope_cs, int32_t rope_positions,
                        void* out, void* scratch) {
  if (!shape_ok(dtype, T, n_reqs, H, G, D)) return fail(PIC_ERR_INVALID_ARG, "invalid attention shape");
  if (H / G > kRows) return fail(PIC_ERR_UNSUPPORTED, "more than 16 query heads per KV head");
  if (!q || !row_start || !kv_len || !block_table || table_stride < 1 || !k_layer || !v_layer || pool_blocks < 1 ||
      !rope_cs || rope_positions < kPage || !out || !scratch)
    return fail(PIC_ERR_INVALID_ARG, "invalid attention arguments");
  if ((page_pos == nullptr) != (n_pages == nullptr))
    return fail(PIC_ERR_INVALID_ARG, "page_pos and n_pages come together");
  if (!aligned16(q) || !aligned16(k_layer) || !aligned16(v_layer) || !aligned16(rope_cs) || ((uintptr_t)out & 31) ||
      ((uintptr_t)scratch & 255))
    return fail(PIC_ERR_INVALID_ARG,
                "q, pools and RoPE table must be 16-byte, out 32-byte, scratch 256-byte aligned");
  const size_t size = (size_t)T * H * D * (dtype == PIC_BF16 ? 2 : 4);
  if (overlap(q, size, out, size)) return fail(PIC_ERR_INVALID_ARG, "out must not overlap q");
  return PIC_OK;
}

BatchCall common_args(const void* q, const int32_t* row_start, const int32_t* kv_len, const int32_t* block_table,
                      int32_t table_stride, const int32_t* page_pos, const int32_t* n_pages, const void* k_layer,
                      const void* v_layer, int32_t pool_blocks, const void* rope_cs, int32_t rope_positions,
                      void* out) {
  BatchCall c;
  BatchArgs& a = c.a[0];
  a.v.row_start = row_start;
  a.v.kv_len = kv_len;
  a.v.block_table = block_table;
  a.v.stride = table_stride;
  a.v.page_pos = page_pos;
  a.v.n_pages = n_pages;
  a.v.window = INT_MAX;
  a.v.pool_blocks = pool_blocks;
  a.v.rope_positions = rope_positions;
  a.q = q;
  a.k_layer = k_layer;
  a.v_layer = v_layer;
  a.rope_cs = (const float2*)rope_cs;
  a.out = out;
  return c;
}

}  // namespace

void batch_simt_view(BatchView& v) {
  v.mrows = kRows;
  v.rb = kRows / v.rep;
  v.kpages = kPages;
  v.cost_item = 1;
  v.cost_full = v.cost_half = 2;
}

int batch_simt_grid(int D) {
  return device_sms() * (D == 128 ? 2 : 4);   // resident CTAs by shared memory (84 and 45 KB)
}

void launch_batch_simt(const BatchArgs& a, cudaStream_t st) {
  a.D == 128 ? launch_simt<128>(a, st) : launch_simt<64>(a, st);
}

namespace {
constexpr int kDevices = 64;
std::mutex g_flag_mu;
unsigned* g_flag_addr[kDevices] = {};   // null: no batched call on that device yet
}  // namespace

// The flag word's device address, looked up once per device.
pic_status batch_flag_address(unsigned** out) {
  int dev = 0;
  PIC_CUDA(cudaGetDevice(&dev));
  if (dev < 0 || dev >= kDevices) return fail(PIC_ERR_UNSUPPORTED, "device index beyond the supported range");
  std::lock_guard<std::mutex> lock(g_flag_mu);
  if (!g_flag_addr[dev]) {
    void* p = nullptr;
    PIC_CUDA(cudaGetSymbolAddress(&p, g_batch_flag));
    g_flag_addr[dev] = (unsigned*)p;
  }
  *out = g_flag_addr[dev];
  return PIC_OK;
}

pic_status batch_check_flags() {
  // without a batched call nothing has been flagged, and pic_sync is spared a copy (28 us instead of 37)
  int dev = 0;
  PIC_CUDA(cudaGetDevice(&dev));
  if (dev < 0 || dev >= kDevices) return PIC_OK;
  {
    std::lock_guard<std::mutex> lock(g_flag_mu);
    if (!g_flag_addr[dev]) return PIC_OK;
  }
  unsigned f = 0;
  const unsigned zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&f, g_batch_flag, sizeof(f));
  if (e != cudaSuccess) return fail(PIC_ERR_CUDA, std::string("batch flag: ") + cudaGetErrorString(e));
  if (!f) return PIC_OK;
  cudaMemcpyToSymbol(g_batch_flag, &zero, sizeof(zero));
  if (f & kBatchTimeout) return fail(PIC_ERR_DEVICE_TIMEOUT, "the batched attention kernel gave up a bounded wait");
  // in the order in which the host calls check: what is inconsistent, what does not fit, what is not free
  if (f & (kBatchBadLengths | kBatchBadBlock | kBatchBadPosition)) {
    std::string what = "device metadata:";
    if (f & kBatchBadLengths) what += " lengths that do not fit together (the request was skipped)";
    if (f & kBatchBadBlock) what += " a block outside the pool (taken as empty)";
    if (f & kBatchBadPosition) what += " a position outside the RoPE table (skipped)";
    return fail(PIC_ERR_INVALID_ARG, what);
  }
  if (f & kBatchCapacity)
    return fail(PIC_ERR_CAPACITY, "block tables: a request's pages exceed its table row, or the rows max_rows; nothing changed");
  return fail(PIC_ERR_OUT_OF_BLOCKS, "block tables: not enough free blocks; nothing changed");
}

}  // namespace pic

using namespace pic;

extern "C" {

size_t pic_op_attention_batch_scratch_bytes(int32_t dtype, int32_t T, int32_t n_reqs, int32_t n_heads,
                                            int32_t n_kv_heads, int32_t head_dim, int32_t table_stride,
                                            int32_t prefix_len, int32_t prefix_pages) {
  if (!shape_ok(dtype, T, n_reqs, n_heads, n_kv_heads, head_dim) || n_heads / n_kv_heads > kRows || table_stride < 1 ||
      prefix_len < 0 || prefix_pages < 0)
    return 0;
  BatchCall c;
  set_shape(c, dtype, T, n_reqs, n_heads, n_kv_heads, head_dim, table_stride, prefix_len, prefix_pages);
  return fits_plan(c) ? layout(c, nullptr) : 0;
}

pic_status pic_op_attention_window(int32_t dtype, int32_t T, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                                   const void* q, const int32_t* row_start, int32_t n_reqs, const int32_t* kv_len,
                                   const int32_t* block_table, int32_t table_stride, const int32_t* page_pos,
                                   const int32_t* n_pages, int32_t window, int32_t sinks, const void* k_layer,
                                   const void* v_layer, int32_t pool_blocks, const void* rope_cs,
                                   int32_t rope_positions, void* out, void* scratch, size_t scratch_bytes,
                                   pic_stream_t stream) {
  pic_status e = check_common(dtype, T, n_reqs, n_heads, n_kv_heads, head_dim, q, row_start, kv_len, block_table,
                              table_stride, page_pos, n_pages, k_layer, v_layer, pool_blocks, rope_cs, rope_positions,
                              out, scratch);
  if (e != PIC_OK) return e;
  if (window < 0 || sinks < 0) return fail(PIC_ERR_INVALID_ARG, "window and sinks must not be negative");
  BatchCall c = common_args(q, row_start, kv_len, block_table, table_stride, page_pos, n_pages, k_layer, v_layer,
                            pool_blocks, rope_cs, rope_positions, out);
  c.a[0].v.window = window > 0 ? window : INT_MAX;
  c.a[0].v.sinks = sinks;
  return run(c, dtype, T, n_reqs, n_heads, n_kv_heads, head_dim, scratch, scratch_bytes, (cudaStream_t)stream);
}

pic_status pic_op_attention_prefix(int32_t dtype, int32_t T, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                                   const void* q, const int32_t* row_start, const int32_t* prefix_blocks,
                                   const int32_t* prefix_pos, int32_t prefix_pages, int32_t prefix_len, int32_t n_reqs,
                                   const int32_t* kv_len, const int32_t* block_table, int32_t table_stride,
                                   const int32_t* page_pos, const int32_t* n_pages, const void* k_layer,
                                   const void* v_layer, int32_t pool_blocks, const void* rope_cs,
                                   int32_t rope_positions, void* out, void* scratch, size_t scratch_bytes,
                                   pic_stream_t stream) {
  pic_status e = check_common(dtype, T, n_reqs, n_heads, n_kv_heads, head_dim, q, row_start, kv_len, block_table,
                              table_stride, page_pos, n_pages, k_layer, v_layer, pool_blocks, rope_cs, rope_positions,
                              out, scratch);
  if (e != PIC_OK) return e;
  if (prefix_len < 0 || prefix_len > rope_positions || (prefix_len > 0 && !prefix_blocks) ||
      prefix_pages < pdiv(prefix_len, kPage) || (prefix_pages > prefix_len) ||
      (!prefix_pos && prefix_pages != pdiv(prefix_len, kPage)))
    return fail(PIC_ERR_INVALID_ARG, "invalid prefix: its pages must hold prefix_len positions of the RoPE table");
  BatchCall c = common_args(q, row_start, kv_len, block_table, table_stride, page_pos, n_pages, k_layer, v_layer,
                            pool_blocks, rope_cs, rope_positions, out);
  BatchArgs& a = c.a[0];
  a.v.pre_blocks = prefix_blocks;
  a.v.pre_pos = prefix_pos;
  a.v.pre_pages = prefix_pages;
  a.v.pre_len = prefix_len;
  return run(c, dtype, T, n_reqs, n_heads, n_kv_heads, head_dim, scratch, scratch_bytes, (cudaStream_t)stream);
}

}  // extern "C"
