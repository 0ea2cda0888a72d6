// Shared device side of the batched paged-attention kernels: the plan (batch_plan.h) computed by
// every CTA for itself, and the arguments of the attention and merge kernels.
#pragma once
#include "batch_plan.h"
#include "pic_internal.h"

namespace pic {

struct BatchCut {         // the item that CTA c's share begins inside of, for the first CTA it continues in; block -1: none
  int block, g;
};
struct BatchHead {        // written by CTA 0
  unsigned U, len;        // length of the cost axis, of a share (0: no item is cut)
  int n_prefix, n_blocks; // prefix row blocks; all row blocks
};

struct BatchArgs {
  BatchView v;
  int H, D;
  int n_blocks_max;       // capacity of blocks[]
  int grid;               // CTAs of the attention kernel (shares of the plan)
  int part_rows;          // rows of one partial slot
  const void* q;          // [T][H][D] rotated; fp16 for bf16 pools, fp32 for fp32 pools
  const void* k_layer;    // [pool_blocks][G][16][D], K unrotated
  const void* v_layer;
  const float2* rope_cs;  // [rope_positions][D / 2]
  __half* krot;           // scratch, K rotated ahead: [prefix page] (unless of the own pages alone), [request][page], x [G][16][D]; or null
  int krot_slots;         // pages of krot
  int krot_own;           // prefix pages of a plan of both
  void* out;              // [T][H][D], q's type
  unsigned* flag;         // the device's word of kBatch* bits
  // scratch
  BatchHead* head;
  int* base;              // [n_reqs + 1] row blocks of the requests before
  BatchBlock* blocks;     // [n_blocks_max]
  BatchCut* cuts;         // [grid]
  float2* part_ml;        // [2 grid][part_rows] (maximum, sum) in the log2 domain
  float* part_o;          // [2 grid][part_rows][D] normalized
  // prefix batches: whole items' results, [2][T][H] (segment 0: the prefix, 1: own pages)
  float2* seg_ml;
  float* seg_o;           // [2][T][H][D]
};

// Whether [a, a + na) and [b, b + nb) share a byte.
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y ? y - x < na : x - y < nb;
}

__device__ __forceinline__ void batch_flag(unsigned* flag, unsigned bad) {
  if (bad) atomicOr(flag, bad);
}

// Exclusive sum of x over the NT threads; `total` gets the whole sum. sh: NT / 32 + 1 values.
template <int NT, typename T>
__device__ __noinline__ T block_scan(T x, T* sh, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) sh[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const T w = lane < NT / 32 ? sh[lane] : 0;
    T wi = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, wi, o);
      if (lane >= o) wi += y;
    }
    if (lane < NT / 32) sh[lane] = wi - w;
    if (lane == 31) sh[NT / 32] = wi;
  }
  __syncthreads();
  total = sh[NT / 32];
  const T r = sh[warp] + inc - x;
  __syncthreads();
  return r;
}

struct BatchShare {   // one CTA's part of the plan
  unsigned x0, x1;
  int first, last;       // the blocks that meet it
};
struct PlanShared {
  unsigned scan[33];
  BatchBlock block;      // a copy of the first one
  int ends[2];
  unsigned edge[2];
};

// The kernels' code is kept small: what runs once or seldom is not inlined (an instruction cache
// that turns over between tiles cost more than all the arithmetic).
static __device__ __noinline__ int plan_rows(const BatchView& v, int r, int& row0, unsigned& bad) {
  return request_rows(v, r, row0, bad);
}
// Row block b: of the n_pre prefix blocks, else of a request (one: request b - n_pre has one block).
static __device__ __noinline__ void plan_block(const BatchArgs& a, int b, int n_pre, int live, bool one, BatchBlock& out, unsigned& bad) {
  const BatchView& v = a.v;
  if (b < n_pre) {
    out = prefix_block(v, live, b);
    return;
  }
  int r = b - n_pre, k = 0;
  if (!one) {
    int lo = 0, hi = v.n_reqs - 1;   // the last request with base <= r
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.base[mid] <= r) lo = mid;
      else hi = mid - 1;
    }
    k = r - a.base[lo];
    r = lo;
  }
  int row0;
  unsigned ignored = 0;
  const int m = plan_rows(v, r, row0, ignored);
  out = own_block(v, r, row0, m, k, &bad);
}

// The CTA's share of the plan. Every thread of the CTA (NT of them) calls it; the blocks that meet
// the share are in a.blocks afterwards, the first also in sh.block. CTAs whose shares meet the same
// block write the same values there, and each reads only after its own writes.
template <int NT>
__device__ __forceinline__ BatchShare plan_batch(const BatchArgs& a, PlanShared& sh) {
  const BatchView& v = a.v;
  const int tid = threadIdx.x, n = v.only == 1 ? 0 : v.n_reqs;
  unsigned bad = 0;
  const int live = pmax(0, pmin(v.row_start[v.n_reqs], v.T));
  const int n_pre = v.pre_len > 0 && v.only != 2 ? pdiv(live, v.rb) : 0;
  if (tid == 0) sh.ends[0] = 0, sh.ends[1] = -1;
  // row blocks of the requests
  const int per_r = pdiv(n, NT), r0 = pmin(tid * per_r, n), r1 = pmin(r0 + per_r, n);
  unsigned cnt = 0;
  bool one = true;
#pragma unroll 1
  for (int r = r0; r < r1; ++r) {
    int row0;
    const int k = pdiv(plan_rows(v, r, row0, bad), v.rb);
    one = one && k == 1;
    cnt += k;
  }
  int n_own = n;
  one = __syncthreads_and(one);
  if (!one) {   // some request has no block or several: base[r] blocks come before request r's
    unsigned total, at = block_scan<NT>(cnt, sh.scan, total);
#pragma unroll 1
    for (int r = r0; r < r1; ++r) {
      int row0;
      unsigned ignored = 0;
      a.base[r] = (int)at;
      if (r + 1 < r1) at += pdiv(plan_rows(v, r, row0, ignored), v.rb);
    }
    n_own = (int)total;
    if (n_own > a.n_blocks_max - n_pre) {   // overlapping row ranges
      n_own = pmax(0, a.n_blocks_max - n_pre);
      bad |= kBatchBadLengths;
    }
    __syncthreads();
  }
  const int nb = n_pre + n_own;
  const int per_b = pdiv(nb, NT), b0 = pmin(tid * per_b, nb), b1 = pmin(b0 + per_b, nb);
  unsigned len = 0, most = 0, U;
  BatchBlock kept{};
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    plan_block(a, b, n_pre, live, one, kept, bad);
    len += block_len(v, kept);
    if (block_len(v, kept) > 0 && item_len(v, kept) > most) most = item_len(v, kept);
  }
  BatchShare s;
  unsigned cum = block_scan<NT>(len, sh.scan, U);
  const unsigned part = share_len(U, a.grid);
  s.x0 = share(U, part, blockIdx.x);
  s.x1 = share(U, part, blockIdx.x + 1);
  const bool whole = __syncthreads_and(whole_pays(most, part));
  if (whole) {   // the edges move to the next item's start
    if (tid < 2) sh.edge[tid] = U;
    __syncthreads();
    unsigned c = cum;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      if (per_b > 1) plan_block(a, b, n_pre, live, one, kept, bad);
      kept.cum = c;
      c += block_len(v, kept);
      if (kept.cum <= s.x0 && s.x0 < c) sh.edge[0] = item_edge(v, kept, s.x0);
      if (kept.cum <= s.x1 && s.x1 < c) sh.edge[1] = item_edge(v, kept, s.x1);
    }
    __syncthreads();
    s.x0 = sh.edge[0], s.x1 = sh.edge[1];
  }
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    if (per_b > 1) plan_block(a, b, n_pre, live, one, kept, bad);
    kept.cum = cum;
    cum += block_len(v, kept);
    if (kept.cum < s.x1 && cum > s.x0) {
      a.blocks[b] = kept;
      if (kept.cum <= s.x0) {
        sh.ends[0] = b;
        sh.block = kept;
      }
      if (cum >= s.x1) sh.ends[1] = b;
    }
  }
  // the item the share begins inside of, when the CTA before began it: the merge finds the cut items here
  __syncthreads();
  if (tid == 0) {
    BatchCut cut{-1, 0};
    const BatchBlock& b = sh.block;
    if (!whole && s.x0 < s.x1 && s.x0 > 0) {
      const unsigned ilen = item_len(v, b), g = (s.x0 - b.cum) / ilen, start = b.cum + g * ilen;
      if (start < s.x0 && owner(part, start) == (int)blockIdx.x - 1) cut = BatchCut{sh.ends[0], (int)g};
    }
    a.cuts[blockIdx.x] = cut;
  }
  if (blockIdx.x == 0) {
    batch_flag(a.flag, bad);
    if (tid == 0) *a.head = BatchHead{U, whole ? 0 : part, n_pre, nb};
  }
  __syncthreads();
  s.first = sh.ends[0];
  s.last = sh.ends[1];
  return s;
}

// Where an item's result goes when its tiles [j0, j1) of nt are done by CTA c: whole items of a
// batch without prefix straight to out, whole items of a prefix batch to their segment, parts to
// a slot.
__device__ __forceinline__ int part_slot(int c, unsigned start, unsigned x0) { return start < x0 ? 2 * c : 2 * c + 1; }

// The merge kernel's view of one segment's plan (0: the shared prefix, 1: the requests' own pages).
struct MergeSegment {
  BatchView v;
  const BatchHead* head;
  const BatchBlock* blocks;
  const BatchCut* cuts;
  const float2* part_ml;
  const float* part_o;
  int part_rows;
};
struct MergeArgs {
  MergeSegment s[2];
  int T, H, G, rep, grid;
  unsigned rep_inv;
  bool prefix;
  const float2* seg_ml;
  const float* seg_o;
  void* out;
};

void launch_batch_simt(const BatchArgs& a, cudaStream_t st);
int batch_simt_grid(int D);
void batch_simt_view(BatchView& v);
// wide: two MMA tiles and K rotated ahead
void batch_tc_view(BatchView& v, bool wide, bool narrow);
// K of the plan's pages, rotated, into a.krot.
pic_status launch_batch_rotate(const BatchArgs& a, cudaStream_t st);
pic_status launch_batch_tc(const BatchArgs& a, bool wide, cudaStream_t st);

}  // namespace pic
