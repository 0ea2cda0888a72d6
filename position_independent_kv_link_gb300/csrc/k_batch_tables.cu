// Block tables and slot maps of a batch's next step, built on the GPU from its lengths: the integer
// bookkeeping that decode and link do on the host, for programs whose lengths live on the device
// (captured decode loops). And the C entries of the row-wise batch calls.
#include <cooperative_groups.h>

#include "batch_internal.cuh"

namespace cg = cooperative_groups;

namespace pic {

namespace {

constexpr int kThreads = 512;
constexpr int kClusterCtas = 8;
constexpr int kMaxReqs = 12288;       // four ints of shared memory per request
constexpr int kMaxStride = 1 << 26;    // pages of a request, packed with 5 bits of its last page's rows
constexpr int kRowsInCluster = 24576;   // in one launch and in two: 8192 rows of 1024 requests 5.8 and 8.8 us, 32768 rows 11.8 and 10.1
constexpr int kMaxReqsAlone = 1024, kRowsAlone = 1024;   // one CTA does all

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

__device__ __forceinline__ void put_row(const TablesArgs& a, int t, int pos, int blk, int row) {
  const bool good = blk >= 0 && blk < INT_MAX / kPage;
  if (!good) batch_flag(a.flag, kBatchBadBlock);
  a.row_pos[t] = pos + a.first;
  a.row_slot[t] = good ? blk * kPage + row : -1;
}

// One CTA (few requests and rows) or one cluster. Every CTA scans all the lengths (so none waits for
// another's sums) and keeps what it read in shared memory; then the new pages, and the rows when there
// are few, are dealt over the threads, each finding its request by bisection there. The lengths
// themselves are overwritten (the outputs may be the inputs) only after a barrier, when no CTA reads
// them any more. A call moves a few KB: the latency of its loads bounds it.
template <int kCluster, bool kRowsHere>
__device__ __forceinline__ void tables(const TablesArgs& a) {
  extern __shared__ int sm[];
  int* s_row = sm;                    // [n] new rows, then those of the requests before
  int* s_blk = sm + a.n;              // [n] new pages, then those of the requests before
  int* s_kv = sm + 2 * a.n;           // [n]
  int* s_np = sm + 3 * a.n;           // [n] pages * 32 + rows of the last page
  __shared__ long long s_scan[kThreads / 32 + 1];
  __shared__ unsigned s_bad;
  const int tid = threadIdx.x, rank = kCluster > 1 ? cg::this_cluster().block_rank() : 0;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  unsigned bad = 0;
#pragma unroll 4
  for (int r = tid; r < a.n; r += kThreads) {
    const Req q = request(a, r, bad);
    s_row[r] = q.m;
    s_blk[r] = q.more;
    s_kv[r] = q.kv;
    s_np[r] = q.np * 32 + (q.ok ? q.kv - q.last : 0);
  }
  const int used = a.free_used ? *a.free_used : 0;
  __syncthreads();
  const int per = pdiv(a.n, kThreads), r0 = pmin(tid * per, a.n), r1 = pmin(r0 + per, a.n);
  long long rows = 0, more = 0, all_rows, all_more;
  for (int r = r0; r < r1; ++r) {
    rows += s_row[r];
    more += s_blk[r];
  }
  long long at_row = block_scan<kThreads>(rows, s_scan, all_rows);
  long long at_blk = block_scan<kThreads>(more, s_scan, all_more);
  if (all_rows > a.max_rows) bad |= kBatchCapacity;
  if (used < 0 || all_more > (long long)a.n_free - used) bad |= kBatchOutOfBlocks;
  if (bad) atomicOr(&s_bad, bad);
  for (int r = r0; r < r1; ++r) {
    const int m = s_row[r], b = s_blk[r];
    s_row[r] = (int)at_row;
    s_blk[r] = (int)at_blk;
    at_row += m;
    at_blk += b;
  }
  __syncthreads();
  bad = s_bad;                        // the same in every CTA: all or nothing
  const int n_rows = bad ? 0 : (int)all_rows, n_more = bad ? 0 : (int)all_more;
  const int t0 = rank * kThreads + tid, step = kCluster * kThreads;
  if constexpr (kRowsHere) {
    for (int t = t0; t < a.max_rows; t += step) {
      if (t < n_rows) {
        const int r = find(s_row, a.n, t), np = s_np[r] >> 5, kv = s_kv[r], last = kv - (s_np[r] & 31);
        const int pos = kv + t - s_row[r];
        const int over = pos - last - kPage;
        const int blk = over >= 0 ? a.free_blocks[used + s_blk[r] + over / kPage]
                                  : a.block_table[(size_t)r * a.stride + np - 1];
        put_row(a, t, pos, blk, over >= 0 ? over % kPage : pos - last);
      } else {
        a.row_pos[t] = 0;
        a.row_slot[t] = -1;
      }
    }
  }
  for (int i = t0; i < n_more; i += step) {
    const int r = find(s_blk, a.n, i), k = i - s_blk[r];
    const size_t at = (size_t)r * a.stride + (s_np[r] >> 5) + k;
    a.block_table[at] = a.free_blocks[used + i];
    if (a.page_pos) a.page_pos[at] = a.first + s_kv[r] - (s_np[r] & 31) + kPage * (k + 1);
  }
  // the lengths of this thread's requests, read before the barrier
  constexpr int kKeep = (kCluster > 1 ? kMaxReqs : kMaxReqsAlone) / (kThreads * kCluster);
  int kv[kKeep], np[kKeep];
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    const int r = t0 + i * step;
    if (r < a.n) {
      const bool end = r == a.n - 1;
      kv[i] = bad ? a.kv_len[r] : s_kv[r] + (end ? n_rows : s_row[r + 1]) - s_row[r];
      np[i] = bad ? (a.page_pos ? a.n_pages[r] : s_np[r] >> 5)
                  : (s_np[r] >> 5) + (end ? n_more : s_blk[r + 1]) - s_blk[r];
    }
  }
  if constexpr (kCluster > 1) cg::this_cluster().sync();
  else __syncthreads();
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

template <bool kRowsHere>
__global__ void __cluster_dims__(kClusterCtas, 1, 1) __launch_bounds__(kThreads) tables_cluster_kernel(const __grid_constant__ TablesArgs a) {
  tables<kClusterCtas, kRowsHere>(a);
}
__global__ void __launch_bounds__(kThreads) tables_kernel(const __grid_constant__ TablesArgs a) { tables<1, true>(a); }

// The rows of many-row calls, after tables_cluster_kernel<false> and from what it wrote: pages from the old
// last one on lie 16 positions apart, so a row's page is counted back from the request's last.
// A CTA takes 1024 rows and finds the requests of its first and last one by two parallel counts
// over row_start; its threads bisect between the two.
constexpr int kRowThreadsT = 256, kRowsPerCta = 1024;
__device__ __forceinline__ int count_le(const int* base, int lo, int n, int stride, int x) {
  // over i = lo, lo + stride, ... < n (at most kRowThreadsT of them): how many base[i] <= x
  const int i = lo + threadIdx.x * stride;
  return __syncthreads_count(i < n && base[i] <= x);
}
__global__ void __launch_bounds__(kRowThreadsT) table_rows_kernel(const __grid_constant__ TablesArgs a) {
  pdl_enter();
  const int t0 = blockIdx.x * kRowsPerCta, n_rows = a.counts[0];
  int lo = 0, hi = 0;
  if (t0 < n_rows) {
    const int jump = pdiv(a.n, kRowThreadsT);    // 48 at most
    const int t1 = pmin(t0 + kRowsPerCta, n_rows) - 1;
    // base[0] = 0 <= x: the counts are at least 1
    lo = (count_le(a.row_start, 0, a.n, jump, t0) - 1) * jump;
    lo += count_le(a.row_start, lo, pmin(lo + jump, a.n), 1, t0) - 1;
    hi = (count_le(a.row_start, 0, a.n, jump, t1) - 1) * jump;
    hi += count_le(a.row_start, hi, pmin(hi + jump, a.n), 1, t1) - 1;
  }
#pragma unroll
  for (int j = 0; j < kRowsPerCta / kRowThreadsT; ++j) {
    const int t = t0 + j * kRowThreadsT + threadIdx.x;
    if (t < n_rows) {
      const int r = lo + find(a.row_start + lo, hi - lo + 1, t);
      const int kv = a.kv_out[r], np = a.np_out[r], pos = kv - (a.row_start[r + 1] - t);
      const size_t row = (size_t)r * a.stride;
      const int last = a.page_pos ? a.page_pos[row + np - 1] - a.first : (np - 1) * kPage;
      const int back = pos < last ? pdiv(last - pos, kPage) : 0;
      put_row(a, t, pos, a.block_table[row + np - 1 - back], pos - (last - back * kPage));
    } else if (t < a.max_rows) {
      a.row_pos[t] = 0;
      a.row_slot[t] = -1;
    }
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
  if (table_stride >= kMaxStride) return fail(PIC_ERR_CAPACITY, "more than 2^26 - 1 pages in a request's table row");
  TablesArgs a{n_reqs, table_stride, n_free, max_rows, first, kv_len, new_len, block_table, page_pos, n_pages,
               free_blocks, free_used, kv_len_out, n_pages_out, row_start, row_pos, row_slot, counts, nullptr};
  pic_status e = batch_flag_address(&a.flag);
  if (e != PIC_OK) return e;
  // One CTA when its threads have two requests and rows each at most: launching a cluster costs the host more.
  // 256 requests of one row: 4.9 us on the GPU and 34 us to call, with the cluster 5.2 and 39.
  if (n_reqs <= kMaxReqsAlone && max_rows <= kRowsAlone) {
    tables_kernel<<<1, kThreads, n_reqs * 16, (cudaStream_t)stream>>>(a);
    PIC_CUDA(cudaGetLastError());
    return PIC_OK;
  }
  const bool rows_here = max_rows <= kRowsInCluster;
  const auto kernel = rows_here ? tables_cluster_kernel<true> : tables_cluster_kernel<false>;
  const int smem = n_reqs * 16;
  if (smem > 40 * 1024)
    PIC_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxReqs * 16));
  kernel<<<kClusterCtas, kThreads, smem, (cudaStream_t)stream>>>(a);
  if (!rows_here)
    launch_dependent(table_rows_kernel, dim3(pdiv(max_rows, kRowsPerCta)), dim3(kRowThreadsT), 0, (cudaStream_t)stream, a);
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
  if (overlap(qkv, 4 * ((size_t)(T - 1) * qkv_stride + (size_t)(n_heads + 2 * n_kv_heads) * head_dim), q_out,
              (size_t)T * n_heads * head_dim * (dtype == PIC_BF16 ? 2 : 4)))
    return fail(PIC_ERR_INVALID_ARG, "q_out must not overlap qkv");
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
