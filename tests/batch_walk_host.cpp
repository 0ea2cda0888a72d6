// The batched attention's plan walked on the host as the kernels walk it (csrc/batch_plan.h): row blocks, shares, the
// blocks that meet a share, the items of a CTA one after the other; and what the merge of a prefix batch looks up.
#include <vector>

#include "batch_plan.h"

using namespace pic;

extern "C" {

// ints: T, G, rep, stride, pre_len, pre_pages, window, sinks, pool_blocks, rope_positions, mrows, kpages,
//       cost_item, cost_full, cost_half, grid, n_reqs
// blocks out: [max][5] = req, row0, nrows, tiles of an item, pages listed
// done out: [max][G] tiles that the CTAs walked; beyond[max][G] tiles that do not exist among them
// counts: blocks, prefix blocks, flags, rows of own blocks whose prefix block does not exist
int batch_walk_host(const int* p, const int* row_start, const int* kv_len, const int* table, const int* page_pos,
                    const int* n_pages, const int* pre_blocks, const int* pre_pos, int* out, int* done, int* beyond,
                    int max_blocks, int* counts) {
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
  const int n_pre = v.pre_len > 0 ? pdiv(live, v.rb) : 0;
  for (int k = 0; k < n_pre; ++k) blocks.push_back(prefix_block(v, live, k));
  for (int r = 0; r < v.n_reqs; ++r) {
    int row0;
    const int m = request_rows(v, r, row0, bad);
    for (int k = 0; k < pdiv(m, v.rb); ++k) blocks.push_back(own_block(v, r, row0, m, k, &bad));
  }
  const int nb = (int)blocks.size();
  if (nb > max_blocks) return 1;
  unsigned U = 0, longest = 0;
  int lost = 0;
  for (int i = 0; i < nb; ++i) {
    BatchBlock& b = blocks[i];
    b.cum = U;
    U += block_len(v, b);
    if (block_len(v, b) > 0 && item_len(v, b) > longest) longest = item_len(v, b);
    int* o = out + 5 * i;
    o[0] = b.req, o[1] = b.row0, o[2] = b.nrows, o[3] = block_tiles(v, b), o[4] = b.nv;
    if (v.pre_len > 0 && b.req >= 0)
      for (int t = b.row0; t < b.row0 + b.nrows; ++t) lost += t / v.rb >= n_pre;
    unsigned ignored = 0;
    for (int j = 0; j < b.nv; ++j) page_meta(v, b, page_raw(v, b, j), ignored);
    bad |= ignored;
  }
  const unsigned len = share_len(U, grid);
  const bool whole = whole_pays(longest, len);
  for (int cta = 0; cta < grid; ++cta) {
    unsigned x0 = share(U, len, cta), x1 = share(U, len, cta + 1);
    if (whole)
      for (unsigned* x : {&x0, &x1})
        for (const BatchBlock& b : blocks)
          if (b.cum <= *x && *x < b.cum + block_len(v, b)) {
            *x = item_edge(v, b, *x);
            break;
          }
    int first = 0, last = -1;
    for (int i = 0; i < nb; ++i) {
      const unsigned from = blocks[i].cum, to = from + block_len(v, blocks[i]);
      if (from < x1 && to > x0) {
        if (from <= x0) first = i;
        if (to >= x1) last = i;
      }
    }
    // the items: the first that has tiles here, then the next ones
    int bi = first, g = 0, nt = 0, c = 0;
    unsigned start = 0, ilen = 0;
    auto load = [&] {
      nt = block_tiles(v, blocks[bi]);
      c = tile_cost(v, blocks[bi]);
      ilen = item_len(v, blocks[bi]);
    };
    auto take = [&] {
      const int j0 = start < x0 ? tile_lower(v, start, nt, c, x0) : 0;
      const int j1 = start + ilen > x1 ? tile_lower(v, start, nt, c, x1) : nt;
      for (int j = j0; j < j1; ++j) ++(j < nt ? done : beyond)[bi * v.G + g];
    };
    if (bi > last) continue;
    load();
    const unsigned skip = x0 > blocks[bi].cum ? (x0 - blocks[bi].cum) / ilen : 0;
    g = (int)skip;
    start = blocks[bi].cum + skip * ilen;
    take();
    for (;;) {
      if (++g == v.G) {
        if (++bi > last) break;
        load();
        g = 0;
        start = blocks[bi].cum;
      } else {
        start += ilen;
      }
      if (start >= x1) break;
      take();
    }
  }
  counts[0] = nb, counts[1] = n_pre, counts[2] = (int)bad, counts[3] = lost;
  return 0;
}
}
