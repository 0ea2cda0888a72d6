// tcgen05 kernel of the batched paged attention: bf16 pools, head_dim 64 or 128, up to 16 query
// heads per KV head, one persistent CTA per SM over its share of the plan (batch_plan.h).
//
// An item is a row block x a KV head: MT tiles of up to 128 MMA rows (half_rows tokens x the rep heads of the
// group, a multiple of 8 tokens), or, narrow, up to 16 rows. Its pages come in windows of 32 (one record each)
// and key tiles of 64 keys, which pass through rings of stages in shared memory:
//
//   meta warp   walks the share: reads the page tables a window ahead and writes the windows' records (item,
//               rows, pages with the rows that hold keys).
//   load        (the meta warp, or, MT = 2, a warp of its own) asks for the items' rows of q (TMA boxes of 8
//               tokens x rep heads, when the item before has had its last S product) and for V: one box a page (a
//               page is one K = 16 step of the PV product, so pages need not be neighbours), or, MT = 2, two
//               boxes of four pages of its copy.
//   K warp      asks for K, one TMA box a page wherever its block lies, with the RoPE table row of the page's
//               position. On its own: with the records' work in the same warp K came late (the decode batch
//               below took 18 % longer).
//   rotation    (MT = 1) turns raw K into the fp16 operand: thread = two rows of a page x 8 pairs of dims; the
//               key in row r of a page at position P is turned by the angle of r (registers) and then by row
//               P of the table (shared memory, one row a page), pairs of fp32 at a time, so that a key needs no
//               table row of its own.
//   V mending   rows that hold no key any row of the block sees are zeroed in V (P is 0 there, V must be
//               finite), by the PV warp or (MT = 2) a warp of its own. K needs none: their S is masked.
//   S warps     (one per MMA tile) issue S_t = Q_t K^T of a key tile as soon as the softmax has the S before
//               it in registers.
//   PV warps    (one per MMA tile) issue O_t += P_t V (P from TMEM). A warp for each product of each tile: one
//               thread for both products of a tile, S(j + 2) right behind PV(j) in its in-order queue, took half as
//               long again. The warp loops as a whole and an elected lane issues: operands stay in uniform
//               registers (4 to 10 % of a call).
//   softmax     warpgroup t = MMA tile t, thread = row: mask, running maximum (O in TMEM is rescaled
//               only when it grows by more than 2^8), P = 2^(S - ref) into one of two P buffers, the sum of the
//               unrounded fp32 weights, and the item's result: out, or for parts of items and for prefix
//               batches the normalized fp32 row with its maximum and sum for the merge.
//   narrow      (single decoded tokens) the four softmax warps have the same rows, at MMA rows 16 w of tiles of 64
//               (q is loaded four times; with tiles of 128 rows the tensor pipe took 7 % longer calls), and one page of each key tile each, with zero P for the others: one warp's 64
//               columns a tile would take longer than anything else. Their four O's, with maxima and sums of
//               their own, are joined through shared memory at the item's end. A kernel of its own: both
//               softmaxes in one cost either 5 % (instruction cache).
//
// Roundings. The result is fp16; what comes before it is held to fewer than half that rounding. Rotated K is two
// fp16 numbers (22 bits), S the sum of both products: with one (11 bits, error of a score about 3e-4 at scores of
// order 1) the result's error was twice that of its rounding alone. P is two bf16 numbers (16 bits; V is stored bf16,
// and both operands of a product have one type) in two PV products. Error against 64 bits relative to the result's
// norm: 2.1e-4, that of rounding it. One fp16 K and one bf16 P: 1.7e-3, and 16 to 20 % faster; P as one fp16
// number with V as fp16, in the two-tile form, 2.7e-4 to 2.9e-4, and 15 to 19 % faster.
//
// The roles' loops are kept small, and few on each scheduler: with three times the code every role ran
// at 8 cycles an instruction (ncu: no_instruction the largest stall).
//
// MT = 1: few rows, K is rotated on its way. MT = 2: many rows; K has been rotated ahead, once per page, into a
// scratch (batch_rotate_kernel). Rotating it here instead, for every 256 rows anew, kept the schedulers busier
// than the MMAs.
//
// Measured, 8 KV heads of 4 query heads, D = 128, whole call: 32 decoding requests of 3000 to 32000 keys, window
// 4096 (0.53 GB of K and V): 115 us, 4.7 TB/s, about 850 ns a key tile of 64; neither HBM, tensor pipe nor issue slots are
// full: the roles' waits for one another bound it. (With tiles of 128 rows, 124 us: without K's second product 115, without
// the rotation's arithmetic 119, without P's second product 121.) Two prompts of 4096, window 1024 (121 GFLOP by the
// formula): 203 us, 0.60 PFLOP/s of the formula's; 268 GFLOP with both operands' second parts and the masked edges of the
// tiles are 144 us at 1865 TFLOP/s; rotation ahead and item ends 32, tensor pipe 65 % busy.
//
// Every wait is bounded: on expiry the CTA raises the timeout flag, stops issuing, waits (bounded)
// for what is in flight, frees its TMEM and returns.
#include <atomic>
#include <mutex>

#include <cudaTypedefs.h>

#include "batch_internal.cuh"

namespace pic {

namespace {

constexpr float kRescale = 8.f;           // rescale O when the row maximum grows by more than 2^8
constexpr unsigned long long kWaitLimit = 4000000000ull;   // cycles, about 2 s

constexpr int KT = 64, KP = KT / kPage;   // keys, pages of a tile
constexpr int WIN = 32, WT = WIN / KP;    // pages, tiles of a window
constexpr int NWIN = 6;                   // window records

template <int D_, int MT_, bool NARROW_ = false>
struct Cfg {
  static constexpr int D = D_, MT = MT_;
  static constexpr bool NARROW = NARROW_;
  static constexpr int NQ = 1;                        // Q buffers per MMA tile
  static constexpr int NBP = 2;                       // P buffers per MMA tile
  // P over its S, two of each per MMA tile (MT = 2 has no room for more; one S and one P beside it take 2 % longer); else
  // one S beside two P's
  static constexpr bool OVER = MT == 2;
  static constexpr int NX = MT == 2 ? 0 : D == 128 ? 3 : 6;   // raw K stages (with table rows)
  static constexpr int NK = MT == 2 ? (D == 128 ? 3 : 6) : (D == 128 ? 2 : 3);   // K operand stages
  static constexpr int NV = MT == 2 ? (D == 128 ? 3 : 6) : (D == 128 ? 4 : 8);   // V stages
  static constexpr int NR = MT == 2 ? 0 : 8;          // rotation warps
  static constexpr int M = NARROW ? 64 : 128;         // MMA rows: of 64, rows 16 w + i are TMEM lanes 32 w + i
  static constexpr int Q_TILE = M * D * 2, Q_HALF = M * 128, K_BYTES = KT * D * 2, PAGE_BYTES = kPage * D * 2, CS_ROW = D * 4;
  static constexpr int K_STAGE = 2 * K_BYTES;         // fp16 and what it leaves out
  // V of a tile: [page][64-dim half][16 keys][128 B] (pool pages), MT 2: [half][64 keys][128 B] (scratch pages)
  static constexpr int V_PAGE = MT == 2 ? 2048 : PAGE_BYTES, V_HALF = MT == 2 ? KT * 128 : 2048;
  // Roles of the warps behind the 4 MT softmax warps. Warp w runs on scheduler w % 4, whose small
  // instruction cache is shared by its warps. Rotation: warps 4..11.
  static constexpr int THREADS = 512;
  static constexpr int W_S = MT == 2 ? 8 : 15, W_PV = MT == 2 ? 10 : 13;   // the first of MT
  static constexpr int W_META = MT == 2 ? 12 : 14, W_K = MT == 2 ? 13 : 12, W_MEND = MT == 2 ? 14 : -1;
  static constexpr int W_LOAD = MT == 2 ? 15 : W_META;   // q and V
  // shared memory (bytes from a 1024-aligned base)
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + MT * NQ * Q_TILE;      // [NK][2] [64-dim half][key][128 B]
  static constexpr int OFF_V = OFF_K + NK * K_STAGE;          // [NV]
  static constexpr int OFF_X = OFF_V + NV * K_BYTES;          // [NX] raw K [page][64-dim half][16 keys][128 B]
  static constexpr int OFF_CS = OFF_X + NX * K_BYTES;         // [NX][KP] table rows, [4][CH][16 B] each
  static constexpr int OFF_REC = OFF_CS + NX * KP * CS_ROW;   // WinRec [NWIN]
  static constexpr int OFF_PAGE = OFF_REC + NWIN * 48;        // int4 [NWIN][WIN] page of the pool, position, rows, page of the rotated K
  static constexpr int OFF_LIM = OFF_PAGE + NWIN * WIN * 16;  // int2 [NWIN][WT] last key, first one behind the sinks
  static constexpr int OFF_END = OFF_LIM + NWIN * WT * 8;     // int [NX] no tile any more
  static constexpr int OFF_JOIN = OFF_END + (NX * 4 + 15) / 16 * 16;         // float2 [4][16], float [4][3][16][8] (narrow): the rows' parts
  static constexpr int OFF_BAR = OFF_JOIN + (NARROW ? 512 + 12 * 16 * 8 * 4 : 0);
  // barriers
  static constexpr int B_META = 0, B_RFREE = B_META + NWIN, B_XFULL = B_RFREE + NWIN, B_XEMPTY = B_XFULL + NX,
                       B_READY = B_XEMPTY + NX, B_KEMPTY = B_READY + NK, B_VFULL = B_KEMPTY + NK,
                       B_VEMPTY = B_VFULL + NV, B_VREADY = B_VEMPTY + NV, B_SFULL = B_VREADY + (MT == 2 ? NV : 0),
                       B_SFREE = B_SFULL + MT * (OVER ? 2 : 1), B_PREADY = B_SFREE + MT, B_PVDONE = B_PREADY + MT * NBP,
                       B_QFULL = B_PVDONE + MT * NBP, B_QEMPTY = B_QFULL + MT * NQ,
                       B_DONE = B_QEMPTY + MT * NQ, B_JOIN = B_DONE + 2 * MT, N_BARS = B_JOIN + 1;
  static constexpr int SMEM = OFF_BAR + N_BARS * 8;
  static_assert(SMEM + 1024 <= 226 * 1024, "shared memory budget (the plan's few static words besides)");
  // TMEM columns: O_t at D t; S_t at TM_S + 128 t, P buffer b of tile t (two bf16 parts) at TM_P + 128 t + KT b; OVER:
  // S and P buffer b there
  static constexpr uint32_t TM_S = MT * D, TM_P = OVER ? TM_S : TM_S + KT;
  static constexpr uint32_t TMEM_COLS = 512;
};

constexpr int kFirst = 1, kLast = 2, kTwo = 4, kEnd = 8, kWhole = 16;
struct WinRec {           // 48 bytes
  int flags;              // first / last window of the item's part, the item has rows for MMA tile 1, no more
                          // windows, the part is the whole item
  int tiles, req, row0, nrows, pos0, g;
  int slot;               // partial slot (parts)
  int pad[4];
};

// Every waiter of a barrier sees each of its phases before the next can complete (a parity wait
// cannot tell phase n from n + 2). META, RFREE: a record is rewritten only when every warp that
// reads records has arrived at RFREE for the window before in its slot. XFULL, XEMPTY: between the
// K warp and the rotation, all of whose warps arrive. READY (of K), KEMPTY: the rotation, or the K
// warp's TMA, of tile j + NK follows the S products of tile j. VFULL, VEMPTY: V of tile j + NV follows
// PV of j, which waits for VREADY (or VFULL); VREADY: VFULL seen and mended. SFULL, SFREE (MT = 1): between the
// S warp and warpgroup t, all of whose warps arrive. PREADY, PVDONE: between warpgroup t and the PV
// warp; P(j + 2) into a buffer (MT = 2: S(j + 2), then P over it) follows the end of PV(j). QFULL, QEMPTY: between the load and the S warp.
// JOIN: the four softmax warps of a narrow item, which all wait.
// No wait is for what waits in turn. Record i needs the readers' passage of window i - NWIN, and by then (MT 1)
// the meta warp has asked for q and V up to window i - 4; K, S, P and PV of windows up to there need only
// records before i. V and q of a tile wait for products of earlier tiles only.

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
// SM clock cycles (reading the global timer instead takes long enough to delay every wait)
__device__ __forceinline__ unsigned long long cycles() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%clock64;" : "=l"(t));
  return t;
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}
// false (and the timeout flag) after kWaitLimit, or when the CTA has given up (`abort`: its word in
// shared memory, 0: wait on). Not inlined: there are some thirty waits.
__device__ __noinline__ bool mbar_wait_on(uint32_t bar, uint32_t parity, uint32_t abort, unsigned* flag) {
  const unsigned long long t0 = cycles();
  for (;;) {
    if (mbar_try(bar, parity)) return true;
    uint32_t gone = 0;
    if (abort) asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(gone) : "r"(abort) : "memory");
    if (gone) return false;
    if (cycles() - t0 > kWaitLimit) {
      atomicOr(flag, kBatchTimeout);
      if (abort) asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(abort), "r"(1u) : "memory");
      return false;
    }
  }
}
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, uint32_t abort, unsigned* flag) {
  return mbar_test(bar, parity) || mbar_try(bar, parity) || mbar_wait_on(bar, parity, abort, flag);
}
// 4-D box at (0, c1, c2, c3)
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int c1, int c2, int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}
// 5-D box at (0, 0, c2, c3, c4)
__device__ __forceinline__ void tma_5d(uint32_t dst, const CUtensorMap* map, int c2, int c3, int c4, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %3, %4, "
      "%5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
      : "memory");
}
// 16-byte chunk c (0..7) of row r of a [rows][128 B] tile, 128-byte swizzle (the TMA and UMMA layout)
__device__ __forceinline__ uint32_t sw128(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }
// Matrix descriptors, 128-byte swizzle, 8-row groups 1024 B apart: the low word is the address and, for
// the MN-major V ([16 keys][64 dims] a half), the distance of the halves; the high word is fixed.
constexpr uint32_t kDescHi = (1024 >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo = 0) {
  return (addr & 0x3FFFFu) >> 4 | (lbo >> 4) << 16;
}
// kind::f16, fp32 accumulator, M x N: fp16 K-major operands; bf16 A (TMEM) with MN-major B
__device__ __forceinline__ constexpr uint32_t idesc_s(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ constexpr uint32_t idesc_pv(int M, int N) {
  return idesc_s(M, N) | 1u << 7 | 1u << 10 | (1u << 16);
}
template <bool ACC>
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %5, 0;\n mov.b64 x, {%1, %4};\n mov.b64 y, {%2, %4};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(kDescHi), "n"((int)ACC));
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.b32 p, %5, 0;\n mov.b64 y, {%2, %4};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(kDescHi), "r"(acc));
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
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* v) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 32 bytes, a whole sector: the rows of a warp's store lie a row apart
__device__ __forceinline__ void stg256(void* p, const uint32_t* u) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]),
               "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
               : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  tmem_ld16(taddr, v);
  tmem_ld16(taddr + 16, v + 16);
}
// two fp32 operations at once
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ float2 unpack_f16x2(uint32_t x) {
  float2 f;
  asm("{\n .reg .f16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}" : "=f"(f.x), "=f"(f.y) : "r"(x));
  return f;
}
// x = hi + lo: 16 of 24 bits as bf16, 22 as fp16 (as many as lie above 2^-25)
__device__ __forceinline__ void split_bf16x2(float2 x, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(x.x, x.y);
  const float2 d = add2(x, make_float2(-__uint_as_float(hi << 16), -__uint_as_float(hi & 0xffff0000u)));
  lo = pack_bf16x2(d.x, d.y);
}
__device__ __forceinline__ void split_f16x2(float2 x, uint32_t& hi, uint32_t& lo) {
  hi = pack_f16x2(x.x, x.y);
  const float2 h = unpack_f16x2(hi), d = add2(x, make_float2(-h.x, -h.y));
  lo = pack_f16x2(d.x, d.y);
}

struct TcArgs {
  CUtensorMap kmap, vmap, qmap, cmap;
  BatchArgs b;
};

// The items of a CTA's share in order; only the first can start and only the last can end inside
// an item.
struct Walk {
  BatchBlock b;
  int bi, last, g, nt, c, j0, j1;
  unsigned start, ilen, x0, x1;
  __device__ __forceinline__ void range(const BatchView& v) {
    j0 = 0, j1 = nt;
    if (start < x0) j0 = lower(v, x0);
    if (start + ilen > x1) j1 = lower(v, x1);
  }
  __device__ __noinline__ int lower(const BatchView& v, unsigned x) const { return tile_lower(v, start, nt, c, x); }
  __device__ __forceinline__ void load(const BatchArgs& a, const BatchBlock& from) {
    b = from;
    nt = block_tiles(a.v, b);
    c = tile_cost(a.v, b);
    ilen = item_len(a.v, b);
  }
  // the first item with tiles of this CTA; false: none
  __device__ __forceinline__ bool begin(const BatchArgs& a, const BatchShare& s, const BatchBlock& block) {
    x0 = s.x0, x1 = s.x1, bi = s.first, last = s.last;
    if (bi > last) return false;
    load(a, block);
    const unsigned skip = x0 > b.cum ? (x0 - b.cum) / ilen : 0;
    g = (int)skip;
    start = b.cum + skip * ilen;
    range(a.v);
    return j0 < j1 || next(a);
  }
  __device__ __forceinline__ bool next(const BatchArgs& a) {
    for (;;) {
      if (++g == a.v.G) {
        if (++bi > last) return false;
        load(a, a.blocks[bi]);
        g = 0;
        start = b.cum;
      } else {
        start += ilen;
      }
      if (start >= x1) return false;
      range(a.v);
      if (j0 < j1) return true;
    }
  }
};

// Bit i: the row at qp (own keys at or below lo as sinks only) sees key i of the page.
__device__ __forceinline__ unsigned seen_bits(int4 p, int qp, int lo, int sinks) {
  const int pos = p.y, up = min(max(qp - pos + 1, 0), 16), from = min(max(lo - pos + 1, 0), 16), sk = min(max(sinks - pos, 0), 16);
  const unsigned upto = (1u << up) - 1u, old = (1u << from) - 1u, first = (1u << sk) - 1u;
  return (unsigned)p.z & upto & (~old | first);
}

template <typename C>
__global__ void __launch_bounds__(C::THREADS, 1) batch_tc_kernel(const __grid_constant__ TcArgs ta) {
  constexpr bool narrow = C::NARROW;
  constexpr int D = C::D, MT = C::MT, NQ = C::NQ, NK = C::NK, NV = C::NV, NBP = C::NBP;
  constexpr bool OVER = C::OVER;
  const BatchArgs& a = ta.b;
  const BatchView& v = a.v;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  WinRec* sRec = reinterpret_cast<WinRec*>(sm + C::OFF_REC);
  int4* sPage = reinterpret_cast<int4*>(sm + C::OFF_PAGE);
  int2* sLim = reinterpret_cast<int2*>(sm + C::OFF_LIM);
  int* sEnd = reinterpret_cast<int*>(sm + C::OFF_END);
  const uint32_t base = smem_u32(sm);
  auto bar = [&](int i) { return base + C::OFF_BAR + 8 * i; };
  __shared__ PlanShared s_plan;
  __shared__ uint32_t s_tmem, s_abort;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t abort = smem_u32(&s_abort);
  auto give_up = [&] { asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(abort), "r"(1u) : "memory"); };
  auto wait = [&](int i, uint32_t parity) { return mbar_wait(bar(i), parity, abort, a.flag); };
  auto wait_meta = [&](uint32_t w) { return wait(C::B_META + w % NWIN, (w / NWIN) & 1); };
  auto done_with = [&](uint32_t w) {   // this warp (all its lanes) reads window w's record no more
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C::B_RFREE + w % NWIN));
  };

  // A warp zeroes the rows of V tile i of a window that hold no key any row of the block sees (lane: rows of its page)
  auto mend = [&](int st, int i, unsigned rows) {
    unsigned todo = __ballot_sync(0xffffffffu, lane / KP == i && rows != 0xffffu);   // pages, by lane
    if (!todo) return;
    uint8_t* vs = sm + C::OFF_V + st * C::K_BYTES + lane * 16;
#pragma unroll 1
    for (; todo; todo &= todo - 1) {
      const int l = __ffs(todo) - 1;
      const unsigned gone = ~__shfl_sync(0xffffffffu, rows, l) >> lane / 8;   // bit 4 k: row lane / 8 + 4 k, a lane a 16-byte chunk
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (gone >> 4 * k & 1u) *reinterpret_cast<uint4*>(vs + l % KP * C::V_PAGE + h * C::V_HALF + k * 512) = make_uint4(0, 0, 0, 0);
    }
    fence_async_smem();
    __syncwarp();
  };

  if (tid == 32 * C::W_PV) {   // not a warp that small plans keep busy
    s_abort = 0;
    auto init = [&](int i, int n, int count) {
#pragma unroll 1
      for (int k = 0; k < n; ++k) mbar_init(bar(i + k), count);
    };
    init(C::B_META, NWIN, 1);
    init(C::B_RFREE, NWIN, 4 * MT + 2 * MT + (MT == 2 ? 3 : 1));
    init(C::B_XFULL, C::NX, 1);
    init(C::B_XEMPTY, C::NX, C::NR);
    init(C::B_READY, NK, MT == 2 ? 1 : C::NR);
    if (MT == 2) init(C::B_VREADY, NV, 1);
    init(C::B_KEMPTY, NK, MT);
    init(C::B_VFULL, NV, 1);
    init(C::B_VEMPTY, NV, MT);
    init(C::B_SFULL, C::B_SFREE - C::B_SFULL, 1);
    init(C::B_SFREE, MT, 4);
    init(C::B_PREADY, MT * NBP, 4);
    init(C::B_PVDONE, MT * NBP, 1);
    init(C::B_QFULL, 2 * MT * NQ + 2 * MT, 1);   // QFULL, QEMPTY, DONE
    init(C::B_JOIN, 1, 4);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == C::W_S) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                 "r"(C::TMEM_COLS));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("griddepcontrol.launch_dependents;");
  fence_before();
  const BatchShare share_ = plan_batch<C::THREADS>(a, s_plan);   // ends with a __syncthreads
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);

  if (warp < 4 * MT) {
    // =============================== softmax: MMA tile t, row m of the item
    const int t = warp >> 2, wq = warp & 3;
    const int i0 = narrow ? lane : 32 * wq + lane, tok0 = i0 * v.rep_inv >> 16;
    const int tok = tok0 < v.half_rows ? t * v.half_rows + tok0 : INT_MAX, hh = i0 - tok0 * v.rep;   // INT_MAX: unused row
    uint32_t joins = 0;
    auto join = [&]() {        // the four warps meet
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::B_JOIN));
      return __all_sync(0xffffffffu, wait(C::B_JOIN, joins++ & 1)) != 0;
    };
    const uint32_t trow = tmem + ((uint32_t)(32 * wq) << 16);
    const uint32_t t_o = trow + D * t;
    const float sl = 1.4426950408889634f * rsqrtf((float)D);
    uint32_t ct = 0;           // key tiles of this MMA tile
    bool ok = true, mine = false, idle = false;
    int qp = 0, lo = 0;
    float mref = 0.f, l = 0.f;
    // O, which holds the item's earlier tiles (a finite earlier maximum), after their PVs
    auto rescale = [&](float scale, uint32_t ct) {
      if (!__all_sync(0xffffffffu, wait(C::B_PVDONE + t * NBP + (ct - 1) % NBP, ((ct - 1) / NBP) & 1))) return false;
      fence_after();
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        float o[16];
        uint32_t u[16];
        tmem_ld16(t_o + c, o);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(o[e] * scale);
        tmem_st16(t_o + c, u);
      }
      return true;
    };
#pragma unroll 1
    for (uint32_t win = 0; ok; ++win) {
      ok = __all_sync(0xffffffffu, wait_meta(win));
      if (!ok) break;
      const WinRec& rec = sRec[win % NWIN];
      const int flags = rec.flags, row0 = rec.row0, nrows = rec.nrows, g = rec.g, slot = rec.slot, req = rec.req;
      if (flags & kEnd) break;
      const int n = t == 1 && !(flags & kTwo) ? 0 : rec.tiles;
      if (flags & kFirst) {
        mine = tok < rec.nrows;
        idle = !narrow && !__any_sync(0xffffffffu, mine);
        qp = req < 0 ? INT_MAX - 1 : rec.pos0 + (mine ? tok : 0);
        lo = req < 0 ? -1 : qp - v.window;   // own keys at or below lo are seen as sinks only
        mref = -INFINITY;
        l = 0.f;
      }
#pragma unroll 1
      for (int j = 0; j < n; ++j, ++ct) {
        const int b = ct % NBP;
        const uint32_t t_p = trow + C::TM_P + 128 * t + KT * b, t_sb = OVER ? t_p : trow + C::TM_S + 128 * t;
        const int2 lim = sLim[win % NWIN * WT + j];
        const bool masked = __any_sync(0xffffffffu, lim.x > qp || lim.y <= lo);
        ok = __all_sync(0xffffffffu, OVER ? wait(C::B_SFULL + 2 * t + b, (ct / 2) & 1) : wait(C::B_SFULL + t, ct & 1));
        if (!ok) break;
        if constexpr (narrow) {
          fence_after();
          float s[16];
          tmem_ld16(t_sb + 16 * wq, s);
          tmem_wait_ld();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::B_SFREE + t));
          if (masked) {
            const unsigned seen = seen_bits(sPage[win % NWIN * WIN + j * KP + wq], qp, lo, v.sinks);
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = seen >> i & 1u ? s[i] : -INFINITY;
          }
          float m2[2] = {s[0], s[1]};
#pragma unroll
          for (int i = 2; i < 16; ++i) m2[i & 1] = fmaxf(m2[i & 1], s[i]);
          const float mx = fmaxf(m2[0], m2[1]) * sl;
          const bool grow = mx > mref + kRescale;
          const float mnew = grow ? mx : mref;
          const float scale = (grow && mref != -INFINITY) ? ex2(mref - mnew) : 1.f;
          mref = mnew;
          const float mz = mref == -INFINITY ? 0.f : -mref;
          float2 sum = make_float2(l * scale, 0.f);
          uint32_t pv[8], pl[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float2 p = fma2(make_float2(s[2 * e], s[2 * e + 1]), make_float2(sl, sl), make_float2(mz, mz));
            p.x = ex2(p.x);
            p.y = ex2(p.y);
            sum = add2(sum, p);
            split_bf16x2(p, pv[e], pl[e]);
          }
          l = sum.x + sum.y;
          ok = __all_sync(0xffffffffu, wait(C::B_PVDONE + t * NBP + b, (ct / NBP + 1) & 1));
          if (!ok) break;
          fence_after();
          const uint32_t none[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
          for (int k = 0; k < KP; ++k) {
            if (k == wq) tmem_st8(t_p + 8 * k, pv), tmem_st8(t_p + KT / 2 + 8 * k, pl);
            else tmem_st8(t_p + 8 * k, none), tmem_st8(t_p + KT / 2 + 8 * k, none);
          }
          if (__any_sync(0xffffffffu, mine && scale != 1.f)) {
            ok = rescale(scale, ct);
            if (!ok) break;
          }
          tmem_wait_st();
          fence_before();
        } else if (!idle) {
          fence_after();
          float s[KT];
#pragma unroll
          for (int c = 0; c < KT; c += 16) tmem_ld16(t_sb + c, s + c);
          tmem_wait_ld();
          fence_before();
          if constexpr (!OVER) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_SFREE + t));   // the next S may come
          }
          if (masked) {
            const int4* pages = sPage + win % NWIN * WIN + j * KP;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const unsigned seen = seen_bits(pages[2 * c], qp, lo, v.sinks) | seen_bits(pages[2 * c + 1], qp, lo, v.sinks) << 16;
#pragma unroll
              for (int i = 0; i < 32; ++i) s[32 * c + i] = seen >> i & 1u ? s[32 * c + i] : -INFINITY;
            }
          }
          float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int i = 4; i < KT; ++i) m4[i & 3] = fmaxf(m4[i & 3], s[i]);
          const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * sl;
          const bool grow = mx > mref + kRescale;
          const float mnew = grow ? mx : mref;
          const float scale = (grow && mref != -INFINITY) ? ex2(mref - mnew) : 1.f;
          mref = mnew;
          const float mz = mref == -INFINITY ? 0.f : -mref;   // nothing seen so far: every s is -inf, p = 0
          float2 sum[2] = {make_float2(l * scale, 0.f), make_float2(0.f, 0.f)};
          if constexpr (!OVER) {
            // the P buffer's PV two tiles before is done (the first round's waits return at once)
            ok = __all_sync(0xffffffffu, wait(C::B_PVDONE + t * NBP + b, (ct / NBP + 1) & 1));
            if (!ok) break;
            fence_after();
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t pv[16], pl[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float2 p = fma2(make_float2(s[32 * c + 2 * e], s[32 * c + 2 * e + 1]), make_float2(sl, sl), make_float2(mz, mz));
              p.x = ex2(p.x);
              p.y = ex2(p.y);
              sum[e & 1] = add2(sum[e & 1], p);
              split_bf16x2(p, pv[e], pl[e]);
            }
            tmem_st16(t_p + 16 * c, pv);
            tmem_st16(t_p + KT / 2 + 16 * c, pl);
          }
          l = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          if (__any_sync(0xffffffffu, mine && scale != 1.f)) {
            ok = rescale(scale, ct);
            if (!ok) break;
          }
          tmem_wait_st();
          fence_before();
        }
        __syncwarp();
        if (lane == 0) {
          if (!OVER && idle) mbar_arrive(bar(C::B_SFREE + t));
          mbar_arrive(bar(C::B_PREADY + t * NBP + b));
        }
      }
      if (!ok) break;
      done_with(win);
      if (!(flags & kLast) || n == 0) continue;
      // the item's result
      ok = __all_sync(0xffffffffu, wait(C::B_PVDONE + t * NBP + (ct - 1) % NBP, ((ct - 1) / NBP) & 1));
      if (!ok) break;
      if (idle) continue;
      fence_after();
      const bool whole = flags & kWhole;
      const size_t head = mine ? (size_t)(row0 + tok) * a.H + g * v.rep + hh : 0;
      __half* dst = nullptr;
      float* po = nullptr;
      float2* pml = nullptr;
      if (mine) {
        if (whole && v.pre_len == 0) {
          dst = static_cast<__half*>(a.out) + head * D;
        } else {
          const size_t at = whole ? (req < 0 ? 0 : (size_t)v.T * a.H) + head : (size_t)slot * a.part_rows + tok * v.rep + hh;
          po = (whole ? a.seg_o : a.part_o) + at * D;
          pml = (whole ? a.seg_ml : a.part_ml) + at;
        }
      }
      if constexpr (narrow) {
        // The row's four parts, sum and maximum each of its own: warp w sums 8 of every 32 columns, the others'
        // through shared memory, [chunk of 32 columns][to][from][row][8]; with few rows several chunks at once.
        const int nr = nrows * v.rep, chunks = min(D / 32, 16 / nr);
        // The last product has had P from all four warps: they are done with the parts of the item before.
        float2* ml = reinterpret_cast<float2*>(sm + C::OFF_JOIN) + lane % 16;
        if (lane < 16) ml[16 * wq] = make_float2(mref, l);
        float* part = reinterpret_cast<float*>(sm + C::OFF_JOIN + 512) + lane * 8;
        float own = 0.f, other[3] = {};   // weights, over the sum: no key seen gives zeros, NaN stays NaN
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32 * chunks) {
          if (c0) ok = join();
          if (!ok) break;
          const int n32 = min(chunks, (D - c0) / 32);
#pragma unroll 1
          for (int r = 0; r < n32; ++r) {
            float o[24];
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 3; ++k) tmem_ld8(t_o + c0 + 32 * r + 8 * ((wq + k + 1) & 3), o + 8 * k);
            tmem_wait_ld();
            if (mine) {
#pragma unroll
              for (int k = 0; k < 3; ++k) {
                float4* to = reinterpret_cast<float4*>(part + ((r * 4 + ((wq + k + 1) & 3)) * 3 + k) * nr * 8);
                to[0] = make_float4(o[8 * k], o[8 * k + 1], o[8 * k + 2], o[8 * k + 3]);
                to[1] = make_float4(o[8 * k + 4], o[8 * k + 5], o[8 * k + 6], o[8 * k + 7]);
              }
            }
          }
          ok = join();
          if (!ok) break;
          if (c0 == 0) {
            float2 x[3];
            float mx = mref;
#pragma unroll
            for (int k = 0; k < 3; ++k) {
              x[k] = ml[16 * ((wq - k - 1) & 3)];
              mx = fmaxf(mx, x[k].x);
            }
            const float ref = mx == -INFINITY ? 0.f : mx;
            own = ex2(mref - ref);
            // in the warps' order, so that all four have the same sum
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 y = ml[16 * k];
              sum += y.y * ex2(y.x - ref);
            }
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            own *= inv;
#pragma unroll
            for (int k = 0; k < 3; ++k) other[k] = ex2(x[k].x - ref) * inv;
            if (pml && wq == 0) *pml = make_float2(mx, sum);
          }
#pragma unroll 1
          for (int r = 0; r < n32; ++r) {
            const int col = c0 + 32 * r + 8 * wq;
            float y[8];
            __syncwarp();
            tmem_ld8(t_o + col, y);
            tmem_wait_ld();
            if (!mine) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] *= own;
#pragma unroll
            for (int k = 0; k < 3; ++k) {
              const float4* from = reinterpret_cast<const float4*>(part + ((r * 4 + wq) * 3 + k) * nr * 8);
              const float4 x0 = from[0], x1 = from[1];
              const float w = other[k];
              y[0] += w * x0.x, y[1] += w * x0.y, y[2] += w * x0.z, y[3] += w * x0.w;
              y[4] += w * x1.x, y[5] += w * x1.y, y[6] += w * x1.z, y[7] += w * x1.w;
            }
            if (dst)
              *reinterpret_cast<uint4*>(dst + col) =
                  make_uint4(pack_f16x2(y[0], y[1]), pack_f16x2(y[2], y[3]), pack_f16x2(y[4], y[5]), pack_f16x2(y[6], y[7]));
            else
              stg256(po + col, reinterpret_cast<const uint32_t*>(y));
          }
        }
        if (!ok) break;
        __syncwarp();
      } else {
        if (pml) *pml = make_float2(mref, l);
        const float inv = l == 0.f ? 0.f : 1.f / l;   // no key seen: zeros; NaN stays NaN
        const bool none = __any_sync(0xffffffffu, mine && l == 0.f);
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          float o[32];
          tmem_ld32(t_o + c0, o);
          tmem_wait_ld();
          if (none) {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = l == 0.f ? 0.f : o[e];
          }
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 y = mul2(make_float2(o[e], o[e + 1]), make_float2(inv, inv));
            o[e] = y.x, o[e + 1] = y.y;
          }
          if (dst) {
#pragma unroll
            for (int c = 0; c < 32; c += 16) {
              uint32_t u[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) u[e] = pack_f16x2(o[c + 2 * e], o[c + 2 * e + 1]);
              stg256(dst + c0 + c, u);
            }
          } else if (po) {
#pragma unroll
            for (int c = 0; c < 32; c += 8) stg256(po + c0 + c, reinterpret_cast<const uint32_t*>(o + c));
          }
        }
      }
      fence_before();   // the next item's first PV overwrites O only after this warp's next P
    }
    if (!ok) give_up();
  } else if ((warp >= C::W_S && warp < C::W_S + MT) || (warp >= C::W_PV && warp < C::W_PV + MT)) {
    // =============================== products: S or PV of MMA tile t
    // The whole warp runs the loop, an elected lane (always the same) issues: operands then stay in
    // uniform registers.
    const bool s_warp = warp >= C::W_S && warp < C::W_S + MT;
    const int t = s_warp ? warp - C::W_S : warp - C::W_PV;
    const bool one = elect();
    constexpr uint32_t id_s = idesc_s(C::M, KT), id_pv = idesc_pv(C::M, D);
    const int full = s_warp ? C::B_READY : MT == 2 ? C::B_VREADY : C::B_VFULL, empty = s_warp ? C::B_KEMPTY : C::B_VEMPTY;
    uint32_t gt = 0, ct = 0, qi = 0;   // tiles of the CTA, of the MMA tile; items of it
    bool ok = true;
    auto wait_all = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, wait(i, parity)) != 0; };
#pragma unroll 1
    for (uint32_t win = 0; ok; ++win) {
      ok = wait_all(C::B_META + win % NWIN, (win / NWIN) & 1);
      if (!ok) break;
      const int flags = __shfl_sync(0xffffffffu, sRec[win % NWIN].flags, 0), n = __shfl_sync(0xffffffffu, sRec[win % NWIN].tiles, 0);
      if (flags & kEnd) break;
      unsigned rows = 0;
      if (MT == 1 && !s_warp) rows = (unsigned)sPage[win % NWIN * WIN + lane].z;
      done_with(win);
      const bool mine = t == 0 || (flags & kTwo);
      const uint32_t qb = qi % NQ, qd = desc_lo(base + C::OFF_Q + (t * NQ + qb) * C::Q_TILE);
      if (s_warp && mine && (flags & kFirst)) ok = wait_all(C::B_QFULL + t * NQ + qb, (qi / NQ) & 1);
#pragma unroll 1
      for (int j = 0; j < n && ok; ++j, ++gt) {
        const int st = s_warp ? gt % NK : gt % NV;
        ok = wait_all(full + st, (s_warp ? gt / NK : gt / NV) & 1);
        if (!mine) {                  // its share of the stage is released
          if (ok && one) mbar_arrive(bar(empty + st));
          continue;
        }
        if (MT == 1 && !s_warp && ok) mend(st, j, rows);
        const int b = ct % NBP;
        // S: the softmax has read the buffer, or (OVER) PV the P that was written over it (the first waits return at
        // once); PV: its P is written
        ok = ok && (!s_warp ? wait_all(C::B_PREADY + t * NBP + b, (ct / NBP) & 1)
                    : OVER  ? wait_all(C::B_PVDONE + t * NBP + b, (ct / NBP + 1) & 1)
                            : wait_all(C::B_SFREE + t, (ct + 1) & 1));
        if (!ok) break;
        fence_after();
        const uint32_t buf = tmem + 128 * t + (s_warp && !OVER ? C::TM_S : C::TM_P + KT * b);
        if (one) {
          if (s_warp) {
            const uint32_t kd = desc_lo(base + C::OFF_K + st * C::K_STAGE);
            umma_ss<false>(buf, qd, kd, id_s);
#pragma unroll
            for (int k = 1; k < D / 8; ++k) { // 16 dims: 32 bytes; 64 dims: a half; then the same for K's second part
              const int e = k % (D / 16);
              umma_ss<true>(buf, qd + (e >> 2) * (C::Q_HALF / 16) + 2 * (e & 3), kd + (k >> 2) * (KT * 128 / 16) + 2 * (k & 3), id_s);
            }
          } else {
            const bool first = j == 0 && (flags & kFirst);
            const uint32_t vd = desc_lo(base + C::OFF_V + st * C::K_BYTES, C::V_HALF);
#pragma unroll
            for (int k = 0; k < KP; ++k)      // 16 keys: a page
              umma_ts(tmem + D * t, buf + 8 * k, vd + k * (C::V_PAGE / 16), id_pv, !first || k != 0);
#pragma unroll
            for (int k = 0; k < KP; ++k)      // P's second part
              umma_ts(tmem + D * t, buf + KT / 2 + 8 * k, vd + k * (C::V_PAGE / 16), id_pv, 1);
          }
          umma_commit(bar(!s_warp ? C::B_PVDONE + t * NBP + b : C::B_SFULL + (OVER ? 2 * t + b : t)));
          umma_commit(bar(empty + st));
        }
        __syncwarp();
        ++ct;
      }
      if (s_warp && ok && mine && (flags & kLast)) {
        if (one) umma_commit(bar(C::B_QEMPTY + t * NQ + qb));
        __syncwarp();
        ++qi;
      }
    }
    if (!ok) give_up();
    if (one) {
      const int d = C::B_DONE + (s_warp ? 0 : MT) + t;
      umma_commit(bar(d));              // fires once every MMA of this thread has retired
      mbar_wait_on(bar(d), 0, 0, a.flag);
    }
  } else if (warp == C::W_META || warp == C::W_LOAD) {
    // =============================== window records; q of the items into the A operands, V
    if (MT == 2 && warp == C::W_LOAD) asm volatile("griddepcontrol.wait;" ::: "memory");   // V
    // Lane i holds page i of a window. `next`: the tables' entries of the window after the last one
    // written (the same item's or the next one's), on their way.
    Walk w;
    const bool meta = warp == C::W_META, load = warp == C::W_LOAD;
    bool more = meta && w.begin(a, share_, s_plan.block), ok = true;
    unsigned bad = 0;
    int j = more ? w.j0 : 0;             // next tile to be described
    PageRaw next{0, 0, 0};
    bool fetched = false;                // (one place for the loads: in line, so that nothing waits for them there)
    uint32_t n_win = 0, qi[MT] = {}, gt = 0;   // windows written; items and tiles asked for
    const int tpt = v.half_rows;
    bool ended = !meta;
#pragma unroll 1
    for (uint32_t win = 0; ok; ++win) {  // V of window win, by the same warp when the two after it are described
#pragma unroll 1
      while (!ended && n_win < win + (win == 0 ? 2 : 3)) {
        if (fetched) {
          const int ws = n_win % NWIN;
          ok = n_win < NWIN || __all_sync(0xffffffffu, wait(C::B_RFREE + ws, (n_win / NWIN - 1) & 1));
          if (!ok) break;
          if (!more) {
            if (lane == 0) {
              sRec[ws].flags = kEnd;
              mbar_arrive(bar(C::B_META + ws));
            }
            ended = true;
            break;
          }
          const int i = j * KP + lane, n = min(w.j1 - j, WT);
          PageMeta pm{0, 0, 0};
          if (lane < n * KP && i < w.b.nv) pm = page_meta(v, w.b, next, bad);
          int top = pm.rows == 0xffffu ? pm.pos + 15 : INT_MAX;
          const int sk = min(max(v.sinks - pm.pos, 0), 16);
          const unsigned behind = pm.rows >> sk << sk;
          int low = behind ? pm.pos + __ffs(behind) - 1 : INT_MAX;
#pragma unroll
          for (int d = 1; d < KP; d <<= 1) {
            top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
            low = min(low, __shfl_xor_sync(0xffffffffu, low, d));
          }
          int krot = 0;                    // the page's place in the rotated K
          if (MT == 2) krot = page_index(w.b, i) + (w.b.req < 0 ? 0 : a.krot_own + w.b.req * v.stride);
          sPage[ws * WIN + lane] = make_int4(pm.blk * v.G + w.g, pm.pos, (int)pm.rows, krot);
          if (lane % KP == 0) sLim[ws * WT + lane / KP] = make_int2(top, low);
          if (lane == 0) {
            WinRec& r = sRec[ws];
            r.flags = (j == w.j0 ? kFirst : 0) | (j + n == w.j1 ? kLast : 0) | (w.b.nrows > v.half_rows ? kTwo : 0) |
                      (w.j0 == 0 && w.j1 == w.nt ? kWhole : 0);
            r.tiles = n, r.req = w.b.req, r.row0 = w.b.row0, r.nrows = w.b.nrows, r.pos0 = w.b.pos0, r.g = w.g;
            r.slot = part_slot(blockIdx.x, w.start, w.x0);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::B_META + ws));
          ++n_win;
          j += n;
          if (j == w.j1) {
            more = w.next(a);
            j = w.j0;
          }
        }
        fetched = true;
        const int i = j * KP + lane;
        next = more && i < w.b.nv ? page_raw(v, w.b, i) : PageRaw{0, 0, 0};
      }
      if (!ok) break;
      if (!load) {
        if (ended) break;
        continue;
      }
      if (!meta) ok = __all_sync(0xffffffffu, wait_meta(win));
      if (!ok) break;
      __syncwarp();
      const WinRec& rec = sRec[win % NWIN];
      const int flags = rec.flags;
      if (flags & kEnd) break;
      const int row0 = rec.row0, g = rec.g, rows = rec.nrows, n = rec.tiles;
      const int4 pg = sPage[win % NWIN * WIN + lane];
      if (!meta) done_with(win);
      if (flags & kFirst) {
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          if (rows <= tpt * t || !ok) continue;
          const uint32_t q = qi[t], qb = q % NQ;
          if (q >= NQ) {
            if (lane == 0) ok = wait(C::B_QEMPTY + t * NQ + qb, (q / NQ - 1) & 1);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
          }
          ++qi[t];
          // tokens behind the item's are read with the last box, rows of the operand behind it stay as
          // they are (their results are not used)
          const uint32_t dst = base + C::OFF_Q + (t * NQ + qb) * C::Q_TILE, full = bar(C::B_QFULL + t * NQ + qb);
          if constexpr (narrow) {         // rows 32 w: the same for each softmax warp w
            if (lane == 0) mbar_expect_tx(full, 4 * (D / 64) * v.mrows * 128);
            __syncwarp();
            if (lane < 4 * (D / 64))
              tma_4d(dst + lane / 4 * C::Q_HALF + lane % 4 * 2048, &ta.qmap, g * v.rep, lane / 4, row0, full);
            continue;
          }
          const int boxes = pdiv(min(rows - t * tpt, tpt), 8);
          if (lane == 0) mbar_expect_tx(full, boxes * (D / 64) * 8 * v.rep * 128);
          __syncwarp();
          for (int i = lane; i < boxes * (D / 64); i += 32) {
            const int h = i % (D / 64), k = i / (D / 64);
            tma_4d(dst + h * C::Q_HALF + k * 8 * v.rep * 128, &ta.qmap, g * v.rep, h, row0 + t * tpt + 8 * k, full);
          }
        }
      }
#pragma unroll 1
      for (int i = 0; i < n && ok; ++i) {
        const int st = gt % NV;
        if (lane == 0) ok = gt < NV || wait(C::B_VEMPTY + st, (gt / NV - 1) & 1);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if constexpr (MT == 2) {
          const int slot = 2 * a.krot_slots + __shfl_sync(0xffffffffu, pg.w, i * KP);
          if (lane == 0) mbar_expect_tx(bar(C::B_VFULL + st), C::K_BYTES);
          __syncwarp();
          if (lane < D / 64)
            tma_5d(base + C::OFF_V + st * C::K_BYTES + lane * (KT * 128), &ta.kmap, lane, g, slot, bar(C::B_VFULL + st));
        } else {
          const bool live = lane / KP == i && pg.z != 0;
          const unsigned who = __ballot_sync(0xffffffffu, live);
          if (lane == 0) mbar_expect_tx(bar(C::B_VFULL + st), (uint32_t)__popc(who) * C::PAGE_BYTES);
          __syncwarp();
          if (live) tma_4d(base + C::OFF_V + st * C::K_BYTES + lane % KP * C::PAGE_BYTES, &ta.vmap, 0, 0, pg.x, bar(C::B_VFULL + st));
        }
        ++gt;
      }
    }
    if (!ok) give_up();
    batch_flag(a.flag, bad);
    // at the end every box asked for has landed
    if (lane == 0) {
#pragma unroll 1
      for (uint32_t s = 0; s < NV; ++s) {
        const uint32_t n = (gt + NV - 1 - s) / NV;
        if (n) mbar_wait_on(bar(C::B_VFULL + s), (n - 1) & 1, 0, a.flag);
      }
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (uint32_t b = 0; b < NQ; ++b) {
          const uint32_t n = (qi[t] + NQ - 1 - b) / NQ;
          if (n) mbar_wait_on(bar(C::B_QFULL + t * NQ + b), (n - 1) & 1, 0, a.flag);
        }
    }
  } else if (warp == C::W_K) {
    // =============================== K, raw with table rows (MT 1) or rotated ahead (MT 2)
    if (MT == 2) asm volatile("griddepcontrol.wait;" ::: "memory");   // the rotated K
    uint32_t gt = 0;                     // tiles asked for
    constexpr int NS = MT == 2 ? NK : C::NX;   // stages K goes to
    bool ok = true;
#pragma unroll 1
    for (uint32_t win = 0; ok; ++win) {
      ok = __all_sync(0xffffffffu, wait_meta(win));
      if (!ok) break;
      const bool end = sRec[win % NWIN].flags & kEnd;
      if (MT == 2 && end) break;
      const int n = end ? 1 : sRec[win % NWIN].tiles, g = sRec[win % NWIN].g;   // MT 1: the rotation sees the end as a tile
      const int4 pg = sPage[win % NWIN * WIN + lane];
      done_with(win);
#pragma unroll 1
      for (int i = 0; i < n; ++i, ++gt) {
        const int st = gt % NS;
        ok = gt < NS || __all_sync(0xffffffffu, wait((MT == 2 ? C::B_KEMPTY : C::B_XEMPTY) + st, (gt / NS - 1) & 1));
        if (!ok) break;
        if constexpr (MT == 2) {
          const int slot = __shfl_sync(0xffffffffu, pg.w, i * KP);
          if (lane == 0) mbar_expect_tx(bar(C::B_READY + st), C::K_STAGE);
          __syncwarp();
          if (lane < D / 32)
            tma_5d(base + C::OFF_K + st * C::K_STAGE + lane * (KT * 128), &ta.kmap, lane % (D / 64), g,
                   slot + (lane < D / 64 ? 0 : a.krot_slots), bar(C::B_READY + st));
        } else {
          const bool live = !end && lane / KP == i && pg.z != 0;
          const unsigned who = __ballot_sync(0xffffffffu, live);
          if (lane == 0) {
            sEnd[st] = end;
            mbar_expect_tx(bar(C::B_XFULL + st), (uint32_t)__popc(who) * (C::PAGE_BYTES + C::CS_ROW));
          }
          __syncwarp();
          if (live) {
            tma_4d(base + C::OFF_X + st * C::K_BYTES + lane % KP * C::PAGE_BYTES, &ta.kmap, 0, 0, pg.x, bar(C::B_XFULL + st));
            tma_4d(base + C::OFF_CS + (st * KP + lane % KP) * C::CS_ROW, &ta.cmap, 0, 0, pg.y, bar(C::B_XFULL + st));
          }
        }
      }
      if (end) break;
    }
    if (!ok) give_up();
    // every copy has landed before the shared memory is given up (at once on the normal path)
    if (lane == 0) {
#pragma unroll 1
      for (uint32_t s = 0; s < NS; ++s) {
        const uint32_t n = (gt + NS - 1 - s) / NS;
        if (n) mbar_wait_on(bar((MT == 2 ? C::B_READY : C::B_XFULL) + s), (n - 1) & 1, 0, a.flag);
      }
    }
  } else if (warp == C::W_MEND) {
    // =============================== rows of V without a key to zero
    uint32_t gt = 0;
    bool ok = true;
#pragma unroll 1
    for (uint32_t win = 0; ok; ++win) {
      ok = __all_sync(0xffffffffu, wait_meta(win));
      if (!ok || (sRec[win % NWIN].flags & kEnd)) break;
      const int n = sRec[win % NWIN].tiles;
      const unsigned rows = (unsigned)sPage[win % NWIN * WIN + lane].z;
      done_with(win);
#pragma unroll 1
      for (int i = 0; i < n; ++i, ++gt) {
        const int st = gt % NV;
        ok = __all_sync(0xffffffffu, wait(C::B_VFULL + st, (gt / NV) & 1));
        if (!ok) break;
        mend(st, i, rows);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::B_VREADY + st));
      }
    }
    if (!ok) give_up();
  } else if constexpr (MT == 1) {
    // =============================== raw K to the K operand
    constexpr int NX = C::NX;
    constexpr int CH = D / 16, NP = KT * CH / (C::NR * 32), RS = kPage / NP;   // threads of a row; rows of a thread, their distance
    static_assert(RS == 8 || RS == 16, "rows of a thread lie whole swizzle atoms apart");
    const int rt = tid - 128, c = rt % CH, r = rt / CH % RS, p = rt / (RS * CH);
    // of r theta for the thread's 8 frequencies, pairs of frequencies: cos, sin; as the quotient of the table's rows r
    // and 0, so that what every row holds besides (a factor, an angle) enters once, with the page's row. (An exact
    // division's code makes 64 requests behind a prefix take 96 us for 91: instruction cache.)
    float2 oc[NP][4], os[NP][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float4 z = reinterpret_cast<const float4*>(a.rope_cs + 8 * c)[e];
      const float d0 = __fdividef(1.f, z.x * z.x + z.y * z.y), d1 = __fdividef(1.f, z.z * z.z + z.w * z.w);
#pragma unroll
      for (int u = 0; u < NP; ++u) {
        const float4 f = reinterpret_cast<const float4*>(a.rope_cs + (size_t)(r + RS * u) * (D / 2) + 8 * c)[e];
        oc[u][e] = make_float2((f.x * z.x + f.y * z.y) * d0, (f.z * z.z + f.w * z.w) * d1);
        os[u][e] = make_float2((f.y * z.x - f.x * z.y) * d0, (f.w * z.z - f.z * z.w) * d1);
      }
    }
    // the thread's two 16-byte chunks (dims 8c.. and their partners) of its first row: in a raw K or V
    // stage, and in a K stage
    const int x1 = p * C::PAGE_BYTES + sw128(r, c), x2 = D == 128 ? x1 + 2048 : p * C::PAGE_BYTES + sw128(r, c + CH);
    const int k1 = p * 2048 + sw128(r, c), k2 = D == 128 ? KT * 128 + k1 : p * 2048 + sw128(r, c + CH);
    bool ok = true;
    uint32_t sx = 0, px = 0, sk = 0, pk = 1;   // stages and their parities
#pragma unroll 1
    for (;;) {
      ok = __all_sync(0xffffffffu, wait(C::B_XFULL + sx, px));
      if (!ok) break;
      if (sEnd[sx]) break;
      const uint8_t* xs = sm + C::OFF_X + sx * C::K_BYTES;
      const float4* cs = reinterpret_cast<const float4*>(sm + C::OFF_CS + (sx * KP + p) * C::CS_ROW) + c;
      uint4 w1[NP], w2[NP], z1[NP], z2[NP];
      float4 f[4];       // (cos, sin) of P theta
#pragma unroll
      for (int u = 0; u < NP; ++u) {
        w1[u] = *reinterpret_cast<const uint4*>(xs + x1 + u * RS * 128);
        w2[u] = *reinterpret_cast<const uint4*>(xs + x2 + u * RS * 128);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = cs[e * CH];
#pragma unroll
      for (int u = 0; u < NP; ++u) {
        uint32_t* a1 = reinterpret_cast<uint32_t*>(&w1[u]);
        uint32_t* a2 = reinterpret_cast<uint32_t*>(&w2[u]);
        uint32_t* b1 = reinterpret_cast<uint32_t*>(&z1[u]);
        uint32_t* b2 = reinterpret_cast<uint32_t*>(&z2[u]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 k = make_float2(__uint_as_float(a1[e] << 16), __uint_as_float(a1[e] & 0xffff0000u));
          const float2 z = make_float2(__uint_as_float(a2[e] << 16), __uint_as_float(a2[e] & 0xffff0000u));
          const float2 y = fma2(make_float2(-z.x, -z.y), os[u][e], mul2(k, oc[u][e])), x = fma2(k, os[u][e], mul2(z, oc[u][e]));
          split_f16x2(make_float2(y.x * f[e].x - x.x * f[e].y, y.y * f[e].z - x.y * f[e].w), a1[e], b1[e]);
          split_f16x2(make_float2(x.x * f[e].x + y.x * f[e].y, x.y * f[e].z + y.y * f[e].w), a2[e], b2[e]);
        }
      }
      ok = __all_sync(0xffffffffu, wait(C::B_KEMPTY + sk, pk));   // the first round's waits return at once
      if (!ok) break;
      uint8_t* ks = sm + C::OFF_K + sk * C::K_STAGE;
#pragma unroll
      for (int u = 0; u < NP; ++u) {
        *reinterpret_cast<uint4*>(ks + k1 + u * RS * 128) = w1[u];
        *reinterpret_cast<uint4*>(ks + k2 + u * RS * 128) = w2[u];
        *reinterpret_cast<uint4*>(ks + C::K_BYTES + k1 + u * RS * 128) = z1[u];
        *reinterpret_cast<uint4*>(ks + C::K_BYTES + k2 + u * RS * 128) = z2[u];
      }
      fence_async_smem();   // the MMAs read these rows through the async proxy, TMA rewrites the raw ones
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(C::B_READY + sk));
        mbar_arrive(bar(C::B_XEMPTY + sx));
      }
      if (++sx == NX) sx = 0, px ^= 1;
      if (++sk == NK) sk = 0, pk ^= 1;
    }
    if (!ok) give_up();
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (warp == C::W_S)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS));
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
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

// A pool layer [blocks][G][16][D] of bf16 as (64 dims, 16 rows, D / 64 halves, G x blocks pages); a
// box is one page, landing as [half][row][128 B].
bool page_map(CUtensorMap* m, const void* base, int blocks, int G, int D) {
  auto enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[4] = {64, (cuuint64_t)kPage, (cuuint64_t)(D / 64), (cuuint64_t)G * blocks};
  const cuuint64_t strides[3] = {(cuuint64_t)D * 2, 128, (cuuint64_t)kPage * D * 2};
  const cuuint32_t estr[4] = {1, 1, 1, 1}, box[4] = {64, kPage, (cuuint32_t)(D / 64), 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// q [T][H][D] of fp16 as (64 dims, H heads, D / 64 halves, T rows); a box is one half of the rep heads
// of a KV head of `rows` rows, landing as [row][head][128 B].
bool q_map(CUtensorMap* m, const BatchArgs& a, int rows) {
  auto enc = encode_fn();
  const cuuint64_t dims[4] = {64, (cuuint64_t)a.H, (cuuint64_t)(a.D / 64), (cuuint64_t)a.v.T};
  const cuuint64_t strides[3] = {(cuuint64_t)a.D * 2, 128, (cuuint64_t)a.H * a.D * 2};
  const cuuint32_t estr[4] = {1, 1, 1, 1}, box[4] = {64, (cuuint32_t)a.v.rep, 1, (cuuint32_t)rows};
  return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(a.q), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The RoPE table [positions][D / 2] of (cos, sin) as (4 floats, D / 16 threads' chunks, 4 chunks of a
// thread, positions): a box is one row with its 16-byte chunks ordered [chunk of a thread][thread], so
// that the rotation's threads read neighbouring ones (no bank conflicts).
bool cs_map(CUtensorMap* m, const BatchArgs& a) {
  auto enc = encode_fn();
  const cuuint64_t dims[4] = {4, (cuuint64_t)(a.D / 16), 4, (cuuint64_t)a.v.rope_positions};
  const cuuint64_t strides[3] = {64, 16, (cuuint64_t)a.D * 4};
  const cuuint32_t estr[4] = {1, 1, 1, 1}, box[4] = {4, (cuuint32_t)(a.D / 16), 4, 1};
  return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, (void*)a.rope_cs, dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// K rotated ahead, [slots][G][16][D] of fp16, as (64 dims, 16 rows, D / 64 halves, G, slots); a box is
// one half of four neighbouring pages, landing as [key][128 B].
bool krot_map(CUtensorMap* m, const BatchArgs& a) {
  auto enc = encode_fn();
  const cuuint64_t dims[5] = {64, (cuuint64_t)kPage, (cuuint64_t)(a.D / 64), (cuuint64_t)a.v.G, 3 * (cuuint64_t)a.krot_slots};
  const cuuint64_t strides[4] = {(cuuint64_t)a.D * 2, 128, (cuuint64_t)kPage * a.D * 2, (cuuint64_t)a.v.G * kPage * a.D * 2};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1}, box[5] = {64, kPage, 1, 1, KP};
  return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, a.krot, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename C>
pic_status launch(const TcArgs& ta, cudaStream_t st) {
  static std::atomic<bool> set[64];
  int dev = 0;
  PIC_CUDA(cudaGetDevice(&dev));
  const int smem = C::SMEM + 1024;
  if (dev < 0 || dev >= 64 || !set[dev]) {
    PIC_CUDA(cudaFuncSetAttribute(batch_tc_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  if (C::MT == 2) {   // its plan under the tail of the rotation
    PIC_CUDA(launch_dependent(batch_tc_kernel<C>, dim3(ta.b.grid), dim3(C::THREADS), smem, st, ta));
  } else {
    batch_tc_kernel<C><<<ta.b.grid, C::THREADS, smem, st>>>(ta);
    PIC_CUDA(cudaGetLastError());
  }
  return PIC_OK;
}

// K of every page that some row of the batch sees (or of the prefix), rotated to its keys' positions, as fp16,
// then what that leaves out, then V as it is (a tile's four pages are neighbours then), each [slot][G][16][D]. One CTA
// a page: a thread has one row and 8 pairs of dims, and takes their table entries once for all KV heads.
// HBM-bound: K and V read once, three such arrays written.
template <int D>
__global__ void __launch_bounds__(256) batch_rotate_kernel(const __grid_constant__ BatchArgs a) {
  asm volatile("griddepcontrol.launch_dependents;");
  const BatchView& v = a.v;
  constexpr int CH = D / 16, HP = 256 / (16 * CH);   // KV heads at once
  const int n_pre = v.only == 1 ? v.pre_pages : a.krot_own, i = (int)blockIdx.x - n_pre;
  const int r = i < 0 ? -1 : i / v.stride, p = i < 0 ? (int)blockIdx.x : i - r * v.stride, c = threadIdx.x % CH, row = threadIdx.x / CH % kPage, g0 = threadIdx.x / (16 * CH);
  unsigned bad = 0;
  BatchBlock b;
  if (r < 0) {
    b = prefix_block(v, 1, 0);
  } else {
    int row0;
    const int m = request_rows(v, r, row0, bad);
    if (m == 0) return;                              // the plan flags what is wrong with it
    b = request_block(v, r, row0, m);
    if (p >= b.np) return;
  }
  bad = 0;
  const PageMeta pm = page_meta(v, b, page_raw(v, b, p), bad);
  if (threadIdx.x == 0) batch_flag(a.flag, bad);
  if (!(pm.rows >> row & 1u)) return;
  const float4* cs = reinterpret_cast<const float4*>(a.rope_cs + (size_t)(pm.pos + row) * (D / 2) + 8 * c);
  float4 f[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = cs[e];
  const size_t from = (size_t)pm.blk * v.G * kPage * D + row * D + 8 * c, part = (size_t)a.krot_slots * v.G * kPage * D / 8;   // uint4 of an array
  const __nv_bfloat16 *src = static_cast<const __nv_bfloat16*>(a.k_layer) + from, *vsrc = static_cast<const __nv_bfloat16*>(a.v_layer) + from;
  __half* dst = a.krot + (size_t)blockIdx.x * v.G * kPage * D + row * D + 8 * c;
#pragma unroll 2
  for (int g = g0 + HP * blockIdx.y; g < v.G; g += HP * gridDim.y) {
    const uint4 u1 = *reinterpret_cast<const uint4*>(src + (size_t)g * kPage * D);
    const uint4 u2 = *reinterpret_cast<const uint4*>(src + (size_t)g * kPage * D + D / 2);
    const uint32_t a1[4] = {u1.x, u1.y, u1.z, u1.w}, a2[4] = {u2.x, u2.y, u2.z, u2.w};
    uint32_t o1[4], o2[4], p1[4], p2[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float q0 = __uint_as_float(a1[e] << 16), q1 = __uint_as_float(a1[e] & 0xffff0000u);
      const float z0 = __uint_as_float(a2[e] << 16), z1 = __uint_as_float(a2[e] & 0xffff0000u);
      split_f16x2(make_float2(q0 * f[e].x - z0 * f[e].y, q1 * f[e].z - z1 * f[e].w), o1[e], p1[e]);
      split_f16x2(make_float2(z0 * f[e].x + q0 * f[e].y, z1 * f[e].z + q1 * f[e].w), o2[e], p2[e]);
    }
    uint4* d1 = reinterpret_cast<uint4*>(dst + (size_t)g * kPage * D);
    uint4* d2 = reinterpret_cast<uint4*>(dst + (size_t)g * kPage * D + D / 2);
    d1[0] = make_uint4(o1[0], o1[1], o1[2], o1[3]);
    d2[0] = make_uint4(o2[0], o2[1], o2[2], o2[3]);
    d1[part] = make_uint4(p1[0], p1[1], p1[2], p1[3]);
    d2[part] = make_uint4(p2[0], p2[1], p2[2], p2[3]);
    d1[2 * part] = *reinterpret_cast<const uint4*>(vsrc + (size_t)g * kPage * D);
    d2[2 * part] = *reinterpret_cast<const uint4*>(vsrc + (size_t)g * kPage * D + D / 2);
  }
}

}  // namespace

void batch_tc_view(BatchView& v, bool wide, bool narrow) {
  v.half_rows = narrow ? 16 / v.rep : 128 / v.rep & ~7;   // a box of q is 8 tokens, or all of a narrow item
  v.rb = wide ? 2 * v.half_rows : v.half_rows;
  v.mrows = v.rb * v.rep;
  v.kpages = KP;
  v.whole_tiles = wide;
  // in eighths of a key tile; from per-CTA times, an item's start and drain take as long as 2 to 4.5 key tiles.
  // (28, 18, 20 instead: one request's window 21.7 us for 19.2, two prompts 175 us for 166.)
  v.cost_item = wide ? 24 : narrow ? 32 : 17;
  v.cost_full = 8;
  v.cost_half = wide ? 6 : 8;
}

pic_status launch_batch_rotate(const BatchArgs& a, cudaStream_t st) {
  // few pages: the KV heads on CTAs of their own too (a CTA takes two heads of 128 or four of 64 at once)
  const int at_once = a.D == 128 ? 2 : 4;
  const dim3 grid(a.krot_slots, a.krot_slots < 4096 ? pdiv(a.v.G, at_once) : 1);
  if (a.D == 128) batch_rotate_kernel<128><<<grid, 256, 0, st>>>(a);
  else batch_rotate_kernel<64><<<grid, 256, 0, st>>>(a);
  PIC_CUDA(cudaGetLastError());
  return PIC_OK;
}

pic_status launch_batch_tc(const BatchArgs& a, bool wide, cudaStream_t st) {
  TcArgs ta;
  ta.b = a;
  const bool narrow = a.v.mrows <= 16;
  if (!page_map(&ta.vmap, a.v_layer, a.v.pool_blocks, a.v.G, a.D) || !q_map(&ta.qmap, a, narrow ? a.v.half_rows : 8) ||
      !(wide ? krot_map(&ta.kmap, a) : page_map(&ta.kmap, a.k_layer, a.v.pool_blocks, a.v.G, a.D) && cs_map(&ta.cmap, a)))
    return fail(PIC_ERR_CUDA, "cuTensorMapEncodeTiled failed for the pools, q, the RoPE table or the rotated K");
  if (narrow) return a.D == 128 ? launch<Cfg<128, 1, true>>(ta, st) : launch<Cfg<64, 1, true>>(ta, st);
  if (a.D == 128) return wide ? launch<Cfg<128, 2>>(ta, st) : launch<Cfg<128, 1>>(ta, st);
  return wide ? launch<Cfg<64, 2>>(ta, st) : launch<Cfg<64, 1>>(ta, st);
}

}  // namespace pic
