// The packed layout of 4-bit weights (csrc/weight4.cuh) for the CPU tests.
#define __host__
#define __device__
#include "weight4.cuh"

extern "C" {
int piece(int r, int q) { return pic::w4_piece(r, q); }
int place(int r) { return pic::w4_place(r); }
int shift(int e) { return pic::w4_shift(e); }
int tile_bytes(int n, int k, int group) { return pic::w4_shape(n, k, group).tile_bytes; }
}
