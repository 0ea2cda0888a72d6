// Work plan of the batched paged-attention kernels, computed on the GPU from device-resident
// lengths (so that a captured graph serves other lengths when it is replayed). Scalar functions
// only, usable from host code too (tests/test_batch_plan_host.py runs them on the CPU).
//
// Rows are grouped in row blocks: up to rb consecutive rows of one request (its own pages), or,
// for a shared prefix, up to rb consecutive rows of the whole batch. An item is (row block, KV
// head): the block's rows x the rep query heads of that KV head against the block's pages, in key
// tiles of kpages pages. Items lie end to end on a cost axis, blocks in order (prefix blocks
// first), the KV heads of a block in order, each item cost_item + tiles x tile_cost long. The axis
// is cut into equal shares, one per CTA: CTA c takes the key tiles whose start lies in [X_c, X_c+1).
// With only short items (whole_pays) the shares' edges move to the next item's start instead.
// An item cut by a share boundary leaves partial results: CTA c's slot 2c holds its part of an
// item begun by an earlier CTA, slot 2c + 1 its part of an item it begins and does not finish
// (at most one of each per CTA, so the slots never collide).
#pragma once
#include <limits.h>
#include <stdint.h>

#ifdef __CUDACC__
#define PIC_HD __host__ __device__ __forceinline__
#else
#define PIC_HD inline
#endif

namespace pic {

constexpr int kPage = 16;   // tokens per page

struct BatchView {
  int n_reqs, T, G, rep;
  const int* row_start;     // [n_reqs + 1]
  const int* kv_len;        // [n_reqs]: keys in the request's own pages, its rows' own included
  const int* block_table;   // [n_reqs][stride]
  int stride;
  const int* page_pos;      // [n_reqs][stride] position of each page's first row, or null: first + 16 p
  const int* n_pages;       // [n_reqs], with page_pos
  const int* pre_blocks;    // [pre_pages]
  const int* pre_pos;       // [pre_pages], or null: 16 p
  int pre_len, pre_pages;   // shared prefix: positions [0, pre_len); 0: none
  int window, sinks;        // key u seen from p when u <= p and (u > p - window or u < sinks)
  int pool_blocks, rope_positions;
  int mrows, rb, kpages;    // rows (token x head) of an item, tokens of a row block (mrows / rep), pages of a tile
  int half_rows;            // tokens up to which an item costs cost_half a tile
  int only;                 // 1: a plan of the prefix blocks alone, 2: of the own ones, 0: of both
  int whole_tiles;          // the pages of the sinks fill whole tiles (a tile's pages are then neighbours)
  unsigned rep_inv;         // ceil(2^16 / rep): m / rep = m * rep_inv >> 16 for m < 256
  int cost_item;            // cost of an item's start and drain,
  int cost_full, cost_half; // of a key tile, and of one whose item has at most half_rows tokens
};

// what a kernel met and skipped; pic_sync reports it
enum : unsigned {
  kBatchBadLengths = 1,    // row_start, kv_len, n_pages or the last page's position inconsistent: the request is
                           // skipped; a page's position and the next one's: it is taken as empty
  kBatchBadBlock = 2,      // a block id outside the pool: its page is taken as empty
  kBatchBadPosition = 4,   // a position outside the RoPE table: its page or row is skipped
  kBatchOutOfBlocks = 8,   // block_tables: not enough free blocks
  kBatchCapacity = 16,     // block_tables: a table row or the row arrays are too short
  kBatchTimeout = 32,      // a bounded wait was given up
  kBatchRange = 64,        // a value beyond the type it was bound for
  kBatchBadToken = 128,    // token_logprobs: a token outside the vocabulary: its row is skipped
  kBatchBadCode = 256      // pack_codes4: a code or zero above 15
};

struct BatchBlock {        // one row block, 48 bytes
  unsigned cum;            // its first item's place on the cost axis
  int req;                 // request, or -1: prefix block
  int row0, nrows;         // rows of q / out
  int pos0;                // position of row 0 (own blocks)
  int sp, wp, nv, np;      // page list: [0, sp) and [wp, wp + nv - sp) of the request's np pages
  int end;                 // position after the request's last key
  int pad[2];              // 48 bytes
};

PIC_HD int pdiv(int a, int b) { return (a + b - 1) / b; }
PIC_HD int pmin(int a, int b) { return a < b ? a : b; }
PIC_HD int pmax(int a, int b) { return a > b ? a : b; }

// First position of a request's own pages.
PIC_HD int own_first(const BatchView& v) { return v.pre_len; }

// Number of pages of request r (checked by request_rows).
PIC_HD int own_pages(const BatchView& v, int r) { return v.page_pos ? v.n_pages[r] : pdiv(v.kv_len[r], kPage); }

// Rows of request r and their first row; 0 (and a flag) when its lengths do not fit together. No row lies behind
// row_start[n_reqs], up to which the prefix' blocks are planned.
PIC_HD int request_rows(const BatchView& v, int r, int& row0, unsigned& bad) {
  const int a = v.row_start[r], b = v.row_start[r + 1], kv = v.kv_len[r], first = own_first(v);
  row0 = a;
  if (a < 0 || b < a || b > pmin(v.T, v.row_start[v.n_reqs]) || kv < 0 || b - a > kv || kv > v.rope_positions - first) {
    bad |= kBatchBadLengths;
    return 0;
  }
  if (b == a) return 0;
  const int np = own_pages(v, r);
  bool ok = np >= 1 && np <= v.stride;
  if (ok && v.page_pos) {
    const int last = v.page_pos[(size_t)r * v.stride + np - 1];
    ok = last >= first && last < first + kv && first + kv - last <= kPage;
  }
  if (!ok) {
    bad |= kBatchBadLengths;
    return 0;
  }
  return b - a;
}

// Page of request r holding position x (first <= x < first + kv), of its np pages.
PIC_HD int page_of(const BatchView& v, int r, int np, int x) {
  const int first = own_first(v);
  if (!v.page_pos) return (x - first) / kPage;
  const int* pos = v.page_pos + (size_t)r * v.stride;
  // a page holds at most 16 and at least 1 position
  int lo = pmin((x - first) / kPage, np - 1), hi = pmin(x - first, np - 1);
  while (lo < hi) {
    const int mid = lo + (hi - lo + 1) / 2;
    if (pos[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Row block k of request r (rows [k rb, ...) of its m rows, the first at row0): everything but cum. At least one page,
// whatever order page_pos has (bad: a flag when its order shows).
PIC_HD BatchBlock own_block(const BatchView& v, int r, int row0, int m, int k, unsigned* bad = nullptr) {
  BatchBlock b{};
  const int a = k * v.rb;
  b.req = r;
  b.row0 = row0 + a;
  b.nrows = pmin(v.rb, m - a);
  b.end = own_first(v) + v.kv_len[r];
  b.pos0 = b.end - m + a;
  b.np = own_pages(v, r);
  const int last = b.pos0 + b.nrows - 1;
  int pe = a + b.nrows == m ? b.np : page_of(v, r, b.np, last) + 1;
  // keys below b.pos0 - window + 1 are seen by no row of the block, but for the first `sinks`
  const int lo = b.pos0 - v.window + 1;
  b.wp = lo > own_first(v) ? page_of(v, r, b.np, lo) : 0;
  if (pe <= b.wp) {
    pe = b.wp + 1;
    if (bad) *bad |= kBatchBadLengths;
  }
  b.sp = v.sinks > 0 ? pmin(b.wp, page_of(v, r, b.np, pmin(v.sinks - 1, last)) + 1) : 0;
  if (v.whole_tiles) b.sp = pmin(b.wp, pdiv(b.sp, v.kpages) * v.kpages);
  b.nv = b.sp + pe - b.wp;
  return b;
}
// A request's rows as one block, its page list all its pages.
PIC_HD BatchBlock request_block(const BatchView& v, int r, int row0, int m) {
  BatchBlock b{};
  b.req = r;
  b.row0 = row0;
  b.nrows = m;
  b.np = b.nv = own_pages(v, r);
  b.end = own_first(v) + v.kv_len[r];
  b.pos0 = b.end - m;
  return b;
}
// Row block k of the shared prefix over the batch's first `live` rows.
PIC_HD BatchBlock prefix_block(const BatchView& v, int live, int k) {
  BatchBlock b{};
  b.req = -1;
  b.row0 = k * v.rb;
  b.nrows = pmin(v.rb, live - b.row0);
  b.np = v.pre_pages;
  b.nv = v.pre_pages;
  return b;
}

PIC_HD int block_tiles(const BatchView& v, const BatchBlock& b) { return pdiv(b.nv, v.kpages); }
PIC_HD int tile_cost(const BatchView& v, const BatchBlock& b) {
  return b.nrows <= v.half_rows ? v.cost_half : v.cost_full;
}
// Lengths on the cost axis: 32 bits hold the whole axis (axis_bound below 2^31 is checked on the host).
PIC_HD unsigned item_len(const BatchView& v, const BatchBlock& b) {
  return v.cost_item + (unsigned)block_tiles(v, b) * tile_cost(v, b);
}
PIC_HD unsigned block_len(const BatchView& v, const BatchBlock& b) {
  return b.nrows > 0 && b.nv > 0 ? item_len(v, b) * v.G : 0;
}
// No plan over tables of this width is longer: every row block as long as its table allows.
inline double axis_bound(const BatchView& v, double n_own, double n_prefix) {
  const double item = v.cost_item + (v.stride / v.kpages + 2.0) * v.cost_full;
  const double pre = v.cost_item + (v.pre_pages / v.kpages + 2.0) * v.cost_full;
  return (n_own * item + n_prefix * pre) * v.G;
}
// When the longest item is at most 1 / kWholeItems of a share, none is cut: the longest share is then at most
// that much over the others' length, where cutting costs the parts' way through memory and the merge.
// (Two prompts of 4096 rows: 181 us with items cut, 161 without.)
constexpr int kWholeItems = 4;
PIC_HD bool whole_pays(unsigned longest_item, unsigned share) { return longest_item <= share / kWholeItems; }
// The right edge of a share at x, inside block b: the item's start at or after x.
PIC_HD unsigned item_edge(const BatchView& v, const BatchBlock& b, unsigned x) {
  const unsigned ilen = item_len(v, b);
  return b.cum + (x - b.cum + ilen - 1) / ilen * ilen;
}
// Shares of an axis of length U: the length of each (the last ones may be shorter or empty), the left
// end of CTA c's, the CTA a place x belongs to.
PIC_HD unsigned share_len(unsigned U, int grid) { return U > (unsigned)grid ? (U + grid - 1) / grid : 1; }
PIC_HD unsigned share(unsigned U, unsigned len, int c) { return (unsigned)c * len < U ? c * len : U; }
PIC_HD int owner(unsigned len, unsigned x) { return (int)(x / len); }
// First tile of an item starting at `start` whose place is >= x (place of tile 0: start; of tile j:
// start + cost_item + j c), at most nt.
PIC_HD int tile_lower(const BatchView& v, unsigned start, int nt, int c, unsigned x) {
  if (x <= start) return 0;
  const unsigned d = x - start;
  const unsigned j = d <= (unsigned)v.cost_item ? 0 : (d - v.cost_item + c - 1) / c;
  return (int)(j < 1 ? 1 : j > (unsigned)nt ? nt : j);
}
PIC_HD unsigned tile_place(const BatchView& v, unsigned start, int c, int j) {
  return j == 0 ? start : start + v.cost_item + (unsigned)j * c;
}

struct PageMeta {
  int blk, pos;        // block, position of row 0
  unsigned rows;       // bit r: row r holds a key that some row of the block sees (0: the page is skipped)
};
struct PageRaw {
  int blk, pos, end;   // block, position of row 0, position after the last row
};
// Place in the tables of page `i` of block b's page list (0 <= i < b.nv), and what they have there.
PIC_HD int page_index(const BatchBlock& b, int i) { return i < b.sp ? i : b.wp + i - b.sp; }
PIC_HD PageRaw page_raw(const BatchView& v, const BatchBlock& b, int i) {
  PageRaw m;
  const int p = page_index(b, i);
  const bool pre = b.req < 0;
  const size_t at = pre ? 0 : (size_t)b.req * v.stride;
  const int* const pos = pre ? v.pre_pos : v.page_pos;
  m.blk = (pre ? v.pre_blocks : v.block_table)[at + p];
  m.pos = pos ? pos[at + p] : (pre ? 0 : own_first(v)) + kPage * p;
  m.end = pos && p + 1 < (pre ? v.pre_pages : b.np) ? pos[at + p + 1] : pre ? v.pre_len : b.end;
  if (!pos) m.end = pmin(m.end, m.pos + kPage);
  return m;
}
// What of it block b uses, checked.
PIC_HD PageMeta page_meta(const BatchView& v, const BatchBlock& b, const PageRaw& raw, unsigned& bad) {
  PageMeta m{raw.blk, raw.pos, 0};
  const int end = raw.end;
  int len = m.pos >= 0 && end > m.pos ? pmin(kPage, end - m.pos) : 0;
  if (m.pos < 0 || m.pos > v.rope_positions - len) {
    bad |= kBatchBadPosition;
    m.pos = 0;
    len = 0;
  } else if (end <= m.pos || end - m.pos > kPage) {   // no page holds none or more than kPage
    bad |= kBatchBadLengths;
    len = 0;
  }
  if (m.blk < 0 || m.blk >= v.pool_blocks) {
    if (len > 0) bad |= kBatchBadBlock;
    m.blk = 0;
    len = 0;
  }
  if (b.req >= 0 && len > 0) {
    len = pmax(0, pmin(len, b.pos0 + b.nrows - m.pos));      // keys after the block's last row
    m.rows = (1u << len) - 1u;
    // keys between the sinks and the first row's window
    const int lo = b.pos0 - v.window + 1;
    const int r0 = pmax(0, pmin(len, v.sinks - m.pos)), r1 = pmax(r0, lo > m.pos ? pmin(len, lo - m.pos) : 0);
    m.rows &= ~(((1u << r1) - 1u) ^ ((1u << r0) - 1u));
  } else {
    m.rows = (1u << len) - 1u;
  }
  return m;
}
// Whether the row at position qp sees the key at position u (of its own pages).
PIC_HD bool sees(const BatchView& v, int qp, int u) { return u <= qp && (u > qp - v.window || u < v.sinks); }

}  // namespace pic
