// Block tables and slot maps of a batch's next step, built on the GPU from its lengths: the integer
// bookkeeping that decode and link do on the host, for programs whose lengths live on the device
// (captured decode loops). And the C entries of the row-wise batch calls.
#include <cooperative_groups.h>

#include "batch_internal.cuh"

namespace cg = cooperative_groups;

namespace pic {

namespace {

constexpr int kThreads = 512;
constexpr int kCluster = 8;
constexpr int kMaxReqs = 12288;       // two ints of shared memory per request

struct TablesArgs {
  int n, stride, n_free, max_rows, first;
  const int *kv_len, *new_len;
  int* block_table;                   // [n][stride], extended in place
  int* page_pos;                      // [n][stride] or null
  const int* n_pages;                 // with page_pos
  const int* free_blocks;
  const int* free_used;               // or null
  int *kv_out, *np_out, *row_start, *row_pos, *row_slot, *counts;
  unsigned* flag;
};

struct Req {
  int kv, m, np, last, room, more;   // rows before, new rows; pages; position of the last page; first free position; new pages
  bool ok;
};
__device__ __forceinline__ Req request(const TablesArgs& a, int r, unsigned& bad) {
  Req q;
  q.kv = a.kv_len[r];
  q.m = a.new_len[r];
  q.ok = q.kv >= 0 && q.m >= 0 && q.kv <= INT_MAX - a.first - kPage && q.m <= INT_MAX - a.first - kPage - q.kv;
  if (!q.ok) q.kv = q.m = 0;
  q.np = a.page_pos ? a.n_pages[r] : pdiv(q.kv, kPage);
  q.last = (q.np - 1) * kPage;
  if (q.np < 0 || q.np > a.stride) {
    bad |= q.np < 0 ? kBatchBadLengths : kBatchCapacity;
    q.np = 0;
  } else if (a.page_pos) {
    q.last = q.np > 0 ? a.page_pos[(size_t)r * a.stride + q.np - 1] - a.first : -kPage;
    q.ok = q.ok && (q.np > 0 ? q.last >= 0 && q.last < q.kv && q.kv - q.last <= kPage : q.kv == 0);
  }
  if (!q.ok) bad |= kBatchBadLengths;
  q.room = q.np > 0 ? q.last + kPage : 0;
  const int over = q.kv + q.m - q.room;
  q.more = over > 0 ? pdiv(over, kPage) : 0;
  if (q.ok && q.np + q.more > a.stride) bad |= kBatchCapacity;
  return q;
}

// The last r with base[r] <= x (base ascending, base[0] = 0; among equal ones the last, which is
// the one that has rows or pages).
__device__ __forceinline__ int find(const int* base, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (base[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// One cluster. Every CTA scans all the lengths (so none waits for another's sums), then the rows
// and the new pages are dealt over the cluster's threads, each finding its request by bisection in
// shared memory; the lengths themselves are overwritten (the outputs may be the inputs) only after
// a cluster barrier, when no CTA reads them any more. A call moves a few KB: latency bounds it.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) tables_kernel(const __grid_constant__ TablesArgs a) {
  extern __shared__ int sm[];
  int* s_row = sm;                    // [n] rows of the requests before
  int* s_blk = sm + a.n;              // [n] new pages of the requests before
  __shared__ long long s_scan[kThreads / 32 + 1];
  __shared__ unsigned s_bad;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, rank = cluster.block_rank();
  if (tid == 0) s_bad = 0;
  __syncthreads();
  const int per = pdiv(a.n, kThreads), r0 = pmin(tid * per, a.n), r1 = pmin(r0 + per, a.n);
  unsigned bad = 0;
  long long rows = 0, more = 0, all_rows, all_more;
  for (int r = r0; r < r1; ++r) {
    const Req q = request(a, r, bad);
    rows += q.m;
    more += q.more;
  }
  const int used = a.free_used ? *a.free_used : 0;
  long long at_row = block_scan<kThreads>(rows, s_scan, all_rows);
  long long at_blk = block_scan<kThreads>(more, s_scan, all_more);
  if (all_rows > a.max_rows) bad |= kBatchCapacity;
  if (used < 0 || all_more > (long long)a.n_free - used) bad |= kBatchOutOfBlocks;
  if (bad) atomicOr(&s_bad, bad);
  for (int r = r0; r < r1; ++r) {
    unsigned ignored = 0;
    const Req q = request(a, r, ignored);
    s_row[r] = (int)at_row;
    s_blk[r] = (int)at_blk;
    at_row += q.m;
    at_blk += q.more;
  }
  __syncthreads();
  bad = s_bad;                        // the same in every CTA: all or nothing
  const int n_rows = bad ? 0 : (int)all_rows, n_more = bad ? 0 : (int)all_more;
  const int t0 = rank * kThreads + tid, step = kCluster * kThreads;
  for (int t = t0; t < a.max_rows; t += step) {
    int pos = 0, slot = -1;
    if (t < n_rows) {
      const int r = find(s_row, a.n, t);
      unsigned ignored = 0;
      const Req q = request(a, r, ignored);
      pos = q.kv + t - s_row[r];
      const int over = pos - q.room;
      const int blk = over >= 0 ? a.free_blocks[used + s_blk[r] + over / kPage]
                                : a.block_table[(size_t)r * a.stride + q.np - 1];
      const bool good = blk >= 0 && blk < INT_MAX / kPage;
      slot = good ? blk * kPage + (over >= 0 ? over % kPage : pos - q.last) : -1;
      if (!good) batch_flag(a.flag, kBatchBadBlock);
      pos += a.first;
    }
    a.row_pos[t] = pos;
    a.row_slot[t] = slot;
  }
  for (int i = t0; i < n_more; i += step) {
    const int r = find(s_blk, a.n, i), k = i - s_blk[r];
    unsigned ignored = 0;
    const Req q = request(a, r, ignored);
    const size_t at = (size_t)r * a.stride + q.np + k;
    a.block_table[at] = a.free_blocks[used + i];
    if (a.page_pos) a.page_pos[at] = a.first + q.room + kPage * k;
  }
  // the lengths of this thread's requests, read before the barrier
  constexpr int kKeep = kMaxReqs / (kThreads * kCluster);
  int kv[kKeep], np[kKeep];
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    const int r = t0 + i * step;
    if (r < a.n) {
      unsigned ignored = 0;
      const Req q = request(a, r, ignored);
      kv[i] = bad ? a.kv_len[r] : q.kv + q.m;
      np[i] = bad ? (a.page_pos ? a.n_pages[r] : q.np) : q.np + q.more;
    }
  }
  cluster.sync();
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    const int r = t0 + i * step;
    if (r < a.n) {
      a.kv_out[r] = kv[i];
      a.np_out[r] = np[i];
      a.row_start[r] = bad ? 0 : s_row[r];
    }
  }
  if (t0 == 0) {
    a.row_start[a.n] = n_rows;
    a.counts[0] = n_rows;
    a.counts[1] = used + n_more;
    a.counts[2] = (int)bad;
    batch_flag(a.flag, bad);
  }
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

}  // namespace

}  // namespace pic

using namespace pic;

extern "C" {

pic_status pic_op_block_tables(int32_t n_reqs, const int32_t* kv_len, const int32_t* new_len, int32_t* block_table,
                               int32_t table_stride, int32_t* page_pos, const int32_t* n_pages,
                               const int32_t* free_blocks, int32_t n_free, const int32_t* free_used, int32_t first,
                               int32_t max_rows, int32_t* kv_len_out, int32_t* n_pages_out, int32_t* row_start,
                               int32_t* row_pos, int32_t* row_slot, int32_t* counts, pic_stream_t stream) {
  if (n_reqs < 1 || !kv_len || !new_len || !block_table || table_stride < 1 || n_free < 0 ||
      (n_free > 0 && !free_blocks) || first < 0 || max_rows < 1 || !kv_len_out || !n_pages_out || !row_start ||
      !row_pos || !row_slot || !counts)
    return fail(PIC_ERR_INVALID_ARG, "invalid block table arguments");
  if ((page_pos == nullptr) != (n_pages == nullptr))
    return fail(PIC_ERR_INVALID_ARG, "page_pos and n_pages come together");
  if (n_reqs > kMaxReqs) return fail(PIC_ERR_CAPACITY, "more than 12288 requests in one block table call");
  TablesArgs a{n_reqs, table_stride, n_free, max_rows, first, kv_len, new_len, block_table, page_pos, n_pages,
               free_blocks, free_used, kv_len_out, n_pages_out, row_start, row_pos, row_slot, counts, nullptr};
  pic_status e = batch_flag_address(&a.flag);
  if (e != PIC_OK) return e;
  const int smem = n_reqs * 8;
  if (smem > 40 * 1024)
    PIC_CUDA(cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxReqs * 8));
  tables_kernel<<<kCluster, kThreads, smem, (cudaStream_t)stream>>>(a);
  PIC_CUDA(cudaGetLastError());
  return PIC_OK;
}

pic_status pic_op_qk_norm_rope(int32_t dtype, int32_t T, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                               const float* qkv, int64_t qkv_stride, const float* q_gain, const float* k_gain,
                               float eps, const int32_t* row_pos, const int32_t* row_slot, const void* rope_cs,
                               int32_t rope_positions, void* q_out, void* k_layer, void* v_layer, int32_t pool_blocks,
                               pic_stream_t stream) {
  if (T < 1 || n_heads < 1 || n_kv_heads < 1 || (head_dim != 64 && head_dim != 128) ||
      (dtype != PIC_F32 && dtype != PIC_BF16) || !qkv || !row_pos || !row_slot || !rope_cs || rope_positions < 1 ||
      !q_out || !k_layer || !v_layer || pool_blocks < 1 || pool_blocks > INT_MAX / kPage || !(eps >= 0.f) ||
      n_heads > INT_MAX / 512 || n_kv_heads > INT_MAX / 512 ||
      qkv_stride < (int64_t)(n_heads + 2 * n_kv_heads) * head_dim || qkv_stride % 4)
    return fail(PIC_ERR_INVALID_ARG, "invalid q/k norm arguments");
  if (!aligned16(qkv) || !aligned16(rope_cs) || !aligned16(q_out) || !aligned16(k_layer) || !aligned16(v_layer) ||
      !aligned16(q_gain) || !aligned16(k_gain))
    return fail(PIC_ERR_INVALID_ARG, "qkv, gains, RoPE table, q_out and pools must be 16-byte aligned");
  unsigned* flag = nullptr;
  pic_status e = batch_flag_address(&flag);
  if (e != PIC_OK) return e;
  launch_qk_norm_rope(dtype, T, n_heads, n_kv_heads, head_dim, qkv, (size_t)qkv_stride, q_gain, k_gain, eps, row_pos,
                      row_slot, (const float2*)rope_cs, rope_positions, q_out, k_layer, v_layer, pool_blocks, flag,
                      (cudaStream_t)stream);
  PIC_CUDA(cudaGetLastError());
  return PIC_OK;
}

}  // extern "C"
