// Host walk of the batched attention plan (csrc/batch_plan.h) for the CPU tests: the same scalar
// functions the kernels call, with the block sums done serially.
#include <vector>

#include "batch_plan.h"

using namespace pic;

extern "C" {

// ints: T, G, rep, stride, pre_len, pre_pages, window, sinks, pool_blocks, rope_positions, mrows, kpages,
//       cost_item, cost_full, cost_half, grid, n_reqs
// items out: [max][12] = cta, req, row0, nrows, pos0, g, j0, j1, tiles, slot (-1: whole), block, sp
// pages out: [max][5] = block, index, blk, pos, mask of rows
// counts: items, pages, blocks, flags, owners that disagree with the shares
int batch_plan_host(const int* p, const int* row_start, const int* kv_len, const int* table, const int* page_pos,
                    const int* n_pages, const int* pre_blocks, const int* pre_pos, int* items, int max_items,
                    int* pages, int max_pages, int* counts) {
  BatchView v{};
  v.T = p[0], v.G = p[1], v.rep = p[2], v.stride = p[3], v.pre_len = p[4], v.pre_pages = p[5];
  v.window = p[6], v.sinks = p[7], v.pool_blocks = p[8], v.rope_positions = p[9];
  v.mrows = p[10], v.rb = p[10] / p[2], v.kpages = p[11], v.cost_item = p[12], v.cost_full = p[13], v.cost_half = p[14];
  v.half_rows = v.rb / 2;
  const int grid = p[15];
  v.n_reqs = p[16];
  v.row_start = row_start, v.kv_len = kv_len, v.block_table = table, v.page_pos = page_pos, v.n_pages = n_pages;
  v.pre_blocks = pre_blocks, v.pre_pos = pre_pos;
  unsigned bad = 0;
  std::vector<BatchBlock> blocks;
  const int live = pmax(0, pmin(row_start[v.n_reqs], v.T));
  if (v.pre_len > 0)
    for (int k = 0; k < pdiv(live, v.rb); ++k) blocks.push_back(prefix_block(v, live, k));
  for (int r = 0; r < v.n_reqs; ++r) {
    int row0;
    const int m = request_rows(v, r, row0, bad);
    for (int k = 0; k < pdiv(m, v.rb); ++k) blocks.push_back(own_block(v, r, row0, m, k));
  }
  unsigned U = 0;
  int np = 0, ni = 0, wrong = 0;
  for (size_t i = 0; i < blocks.size(); ++i) {
    BatchBlock& b = blocks[i];
    b.cum = U;
    U += block_len(v, b);
    for (int j = 0; j < b.nv; ++j) {
      const PageMeta m = page_meta(v, b, page_raw(v, b, j), bad);
      if (np >= max_pages) return 1;
      int* o = pages + 5 * np++;
      o[0] = (int)i, o[1] = j, o[2] = m.blk, o[3] = m.pos, o[4] = (int)m.rows;
    }
  }
  if (U > axis_bound(v, v.T / v.rb + v.n_reqs, v.pre_len > 0 ? v.T / v.rb + 1 : 0)) return 3;
  const unsigned len = share_len(U, grid);
  unsigned longest = 0;
  for (const BatchBlock& b : blocks)
    if (block_len(v, b) > 0 && item_len(v, b) > longest) longest = item_len(v, b);
  const bool whole_items = whole_pays(longest, len);
  if (share(U, len, grid) != U) return 2;   // the shares do not reach the end
  for (int c = 0; c < grid && U > 0; ++c) {
    unsigned x0 = share(U, len, c), x1 = share(U, len, c + 1);
    if (whole_items)
      for (unsigned* x : {&x0, &x1})
        for (const BatchBlock& b : blocks)
          if (b.cum <= *x && *x < b.cum + block_len(v, b)) {
            *x = item_edge(v, b, *x);
            break;
          }
    for (size_t i = 0; i < blocks.size(); ++i) {
      const BatchBlock& b = blocks[i];
      const int nt = block_tiles(v, b), tc = tile_cost(v, b);
      for (int g = 0; g < v.G; ++g) {
        const unsigned start = b.cum + g * item_len(v, b);
        const int j0 = tile_lower(v, start, nt, tc, x0), j1 = tile_lower(v, start, nt, tc, x1);
        if (j0 >= j1) continue;
        for (int j = j0; j < j1; ++j)
          if (!whole_items && owner(len, tile_place(v, start, tc, j)) != c) ++wrong;
        if (whole_items && (j0 != 0 || j1 != nt)) ++wrong;
        if (ni >= max_items) return 1;
        int* o = items + 12 * ni++;
        const bool whole = j0 == 0 && j1 == nt;
        o[0] = c, o[1] = b.req, o[2] = b.row0, o[3] = b.nrows, o[4] = b.pos0, o[5] = g, o[6] = j0, o[7] = j1;
        o[8] = nt, o[9] = whole ? -1 : (start < x0 ? 2 * c : 2 * c + 1), o[10] = (int)i, o[11] = b.sp;
      }
    }
  }
  counts[0] = ni, counts[1] = np, counts[2] = (int)blocks.size(), counts[3] = (int)bad, counts[4] = wrong;
  return 0;
}
}
