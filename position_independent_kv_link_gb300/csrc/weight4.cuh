// The packed layout of 4-bit weights (include/pic.h, pic_op_weight4_bytes) as the kernels see it.
#pragma once
#include <cstdint>

namespace pic {

constexpr int kW4Rows = 128, kW4Cols = 128;          // of a tile
constexpr int kW4Codes = kW4Rows * kW4Cols / 2;      // bytes of a tile's codes; scales and zeros follow

struct W4Shape {
  int N, K, group;
  int n_tiles, k_tiles, groups;   // tiles down and across; groups of a row
  int tile_bytes;
};

inline W4Shape w4_shape(int N, int K, int group) {
  W4Shape s;
  s.N = N;
  s.K = K;
  s.group = group;
  s.n_tiles = (N + kW4Rows - 1) / kW4Rows;
  s.k_tiles = (K + kW4Cols - 1) / kW4Cols;
  s.groups = (K + group - 1) / group;
  s.tile_bytes = kW4Codes + kW4Cols / group * kW4Rows * 3;
  return s;
}
inline bool w4_ok(int N, int K, int group) {
  return N >= 1 && K >= 32 && K % 32 == 0 && N <= INT32_MAX - kW4Rows && K <= INT32_MAX - kW4Cols &&
         (group == 32 || group == 64 || group == 128) &&
         (int64_t)((N + kW4Rows - 1) / kW4Rows) * ((K + kW4Cols - 1) / kW4Cols) <= INT32_MAX;
}

// Where a tile keeps what (include/pic.h). The 16-byte piece q of row r holds one 32-bit word for each of the tile's four
// 32-column runs: the run's columns 8 q .. 8 q + 7. Column e of the 8 is in bits 4 i .. 4 i + 3, i = e / 2 + 4 (e % 2), so that
// (w >> 4 i) & 0x000f000f are columns 2 i and 2 i + 1 in the halves of a register. A row's scale and zero stand beside those of
// the rows 8 apart.
// A thread that reads its row's pieces meets no other in a bank, nor do four threads that read one row's pieces.
__host__ __device__ constexpr int w4_piece(int r, int q) { return r * 64 + (q ^ (r >> 1 & 3)) * 16; }
__host__ __device__ constexpr int w4_shift(int e) { return 4 * (e / 2 + 4 * (e % 2)); }
__host__ __device__ constexpr int w4_place(int r) { return (r & ~31) + (r & 7) * 4 + (r >> 3 & 3); }

}  // namespace pic
