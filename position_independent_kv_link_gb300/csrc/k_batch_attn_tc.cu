// tcgen05 kernel of the batched paged attention: bf16 pools, head_dim 64 or 128, up to 16 query
// heads per KV head, one persistent CTA per SM over its share of the plan (batch_plan.h).
//
// An item is a row block x a KV head: MT tiles of 128 MMA rows, row m = token * rep + head of the
// group. Key tiles of KT keys pass through a ring of stages (K and V released apart: K when its
// S products have retired, V when its PV products have):
//
//   load warp   per key tile one TMA box per page and 64-dim half of K and of V (16 rows x 128 B,
//               128-byte swizzled: the MMA operand layout, wherever the page's block lies), one
//               bulk copy of the RoPE table row of each page's position, the keys' positions for
//               the mask. Page tables are read a tile ahead.
//   rotation    4 warps turn K in place in the stage: thread = row of a page x 8 pairs of dims; the
//               angle of row r of a page at position P is composed from the table rows of P (with
//               the stage) and of r (in registers), so that a key needs no table row of its own.
//               bf16 -> fp16, one rounding (the MMA takes Q and K as fp16: 3 bits more than bf16 in
//               S). Rows that hold no key any row of the block sees are zeroed in K and V.
//   MMA warps   one issuing thread per MMA tile: O_t += P_t V of key tile j as soon as P_t(j) is
//               written, S_t of tile j + NBS (Q_t K^T, fp16) into the S buffer that PV has just
//               read (one thread's MMAs run in order), also across items.
//   Q warp      copies the items' rows of q into the swizzled A operand (double-buffered for one MMA
//               tile, else when the item's last S product has retired).
//   softmax     warpgroup t = MMA tile t, thread = row: mask, running maximum (O in TMEM is rescaled
//               only when it grows by more than 2^8), P = 2^(S - ref) as bf16 over the S columns
//               (V is stored bf16 and both operands have one type; the sum is of the unrounded
//               fp32 weights), and the item's result: out, or for parts of items and for prefix
//               batches the normalized fp32 row with its maximum and sum for the merge.
//
// MT = 1, KT = 64, two S buffers, many small stages: few rows, HBM-bound -- what counts is bytes in
// flight. MT = 2, KT = 128, one S buffer per tile: many rows, MMA-bound -- a K tile is rotated once
// for 256 rows, and an S product of 128 keys reads its operands from shared memory as fast as it
// multiplies (64 cycles each), which one of 64 keys does not; the two tiles alternate on the tensor
// pipe, one's softmax under the other's products.
//
// Every wait is bounded: on expiry the CTA raises the timeout flag, stops issuing, waits (bounded)
// for what is in flight, frees its TMEM and returns.
#include <mutex>

#include <cudaTypedefs.h>

#include "batch_internal.cuh"

namespace pic {

namespace {

constexpr float kRescale = 8.f;           // rescale O when the row maximum grows by more than 2^8
constexpr unsigned long long kWaitLimitNs = 2000000000ull;

template <int D_, int MT_>
struct Cfg {
  static constexpr int D = D_, MT = MT_;
  static constexpr int KT = MT == 2 ? 128 : 64;       // keys per tile
  static constexpr int KP = KT / kPage;               // pages per tile
  static constexpr int NBS = MT == 2 ? 1 : 2;         // S buffers per MMA tile
  static constexpr int NQ = MT == 2 ? 1 : 2;          // Q buffers per MMA tile
  static constexpr int NH = D / 64;                   // 64-dim halves
  static constexpr int NST = D == 128 ? (MT == 2 ? 2 : 4) : (MT == 2 ? 4 : 8);
  static constexpr int Q_TILE = 128 * D * 2, K_BYTES = KT * D * 2, CS_ROW = D * 4, CS_BYTES = KP * CS_ROW;
  static constexpr int W_MMA = 4 * MT, W_LOAD = W_MMA + MT, W_Q = W_LOAD + 1, W_ROT = 4 * MT + 4;
  static constexpr int THREADS = (W_ROT + 4) * 32;
  static constexpr int NPOS = 2 * NST;                // slots of key positions (see the load warp)
  // shared memory (bytes from a 1024-aligned base)
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + MT * NQ * Q_TILE;
  static constexpr int OFF_V = OFF_K + NST * K_BYTES;
  static constexpr int OFF_CS = OFF_V + NST * K_BYTES;
  static constexpr int OFF_POS = OFF_CS + NST * CS_BYTES;     // int [NPOS][KT] key positions (INT_MAX: no key)
  static constexpr int OFF_LIM = OFF_POS + NPOS * KT * 4;     // int2 [NPOS] last key, first key behind the sinks
  static constexpr int OFF_MASK = OFF_LIM + NPOS * 8;         // uint [NST][KP] rows of each page that hold a key
  static constexpr int OFF_BAR = (OFF_MASK + NST * KP * 4 + 7) / 8 * 8;
  // barriers
  static constexpr int B_KFULL = 0, B_VFULL = B_KFULL + NST, B_READY = B_VFULL + NST, B_KEMPTY = B_READY + NST,
                       B_VEMPTY = B_KEMPTY + NST, B_SFULL = B_VEMPTY + NST, B_PREADY = B_SFULL + MT * NBS,
                       B_PVDONE = B_PREADY + MT * NBS, B_QFULL = B_PVDONE + MT * NBS, B_QEMPTY = B_QFULL + MT * NQ,
                       B_DONE = B_QEMPTY + MT * NQ, N_BARS = B_DONE + MT;
  static constexpr int SMEM = OFF_BAR + N_BARS * 8;
  static_assert(SMEM + 1024 <= 226 * 1024, "shared memory budget (the plan's few static words besides)");
  // TMEM columns: O_t at D t, S buffer b of tile t at TM_S + 128 t + KT b
  static constexpr uint32_t TM_S = MT * D;
  static constexpr uint32_t TMEM_COLS = MT == 2 ? 512 : 256;
};
// Every waiter of a barrier sees each of its phases before the next can complete (a parity wait
// cannot tell phase n from n + 2): KFULL (rotation warps): a stage is refilled after KEMPTY, i.e.
// after the S products that followed READY. VFULL (MMA warps; rotation warps of a tile with empty
// rows): after VEMPTY, to which every MMA warp arrives once per tile, after its wait for VFULL.
// READY (MMA warps): needs KFULL. SFULL, PREADY, PVDONE as a ring between MMA thread t and
// warpgroup t: S(j + NBS) follows PV(j), which waits for all four warps' P(j). QFULL, QEMPTY:
// between the Q warp and MMA thread t.

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ unsigned long long gtimer() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
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
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// false (and the timeout flag) after kWaitLimitNs, or when the CTA has given up
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* abort, unsigned* flag) {
  if (mbar_try(bar, parity)) return true;
  const unsigned long long t0 = gtimer();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try(bar, parity)) return true;
    if ((i & 63u) == 0) {
      if (*abort) return false;
      if (gtimer() - t0 > kWaitLimitNs) {
        atomicOr(flag, kBatchTimeout);
        *abort = 1;
        return false;
      }
    }
  }
}
__device__ __forceinline__ void bulk_g2s(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap* map, int half, int g, int blk, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %2, %4, "
      "%5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(half), "r"(g), "r"(blk), "r"(bar)
      : "memory");
}
// 16-byte chunk c (0..7) of row r of a [rows][128 B] tile, 128-byte swizzle (the TMA and UMMA layout)
__device__ __forceinline__ uint32_t sw128(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }
// K-major operand: 8-row atoms 1024 B apart
__device__ __forceinline__ uint64_t desc_kmajor(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// MN-major operand [k rows][n], 64 n per 128-byte row: blocks of 64 n `lbo` bytes apart, groups of 8 k rows 1024 B
__device__ __forceinline__ uint64_t desc_mnmajor(uint32_t addr, uint32_t lbo) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// kind::f16, fp32 accumulator, M x N: fp16 K-major operands; bf16 A (TMEM) with MN-major B
__device__ __forceinline__ constexpr uint32_t idesc_s(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ constexpr uint32_t idesc_pv(int M, int N) {
  return idesc_s(M, N) | (1u << 7) | (1u << 10) | (1u << 16);
}
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc));
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
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
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
template <int R> __device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R> __device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

struct TcArgs {
  CUtensorMap kmap, vmap;
  BatchArgs b;
};

// The items of a CTA's share in order; only the first can start and only the last can end inside
// an item.
struct Walk {
  BatchBlock b;
  int bi, last, g, nt, c, j0, j1;
  long long start, ilen, x0, x1;
  __device__ __forceinline__ void range(const BatchView& v) {
    j0 = start < x0 ? tile_lower(v, start, nt, c, x0) : 0;
    j1 = start + ilen > x1 ? tile_lower(v, start, nt, c, x1) : nt;
  }
  __device__ __forceinline__ void load(const BatchArgs& a) {
    b = a.blocks[bi];
    nt = block_tiles(a.v, b);
    c = tile_cost(a.v, b);
    ilen = item_len(a.v, b);
  }
  // the first item with tiles of this CTA; false: none
  __device__ __forceinline__ bool begin(const BatchArgs& a, const BatchShare& s) {
    x0 = s.x0, x1 = s.x1, bi = s.first, last = s.last;
    if (bi > last) return false;
    load(a);
    const long long skip = x0 > b.cum ? (x0 - b.cum) / ilen : 0;
    g = (int)skip;
    start = b.cum + skip * ilen;
    range(a.v);
    return j0 < j1 || next(a);
  }
  __device__ __forceinline__ bool next(const BatchArgs& a) {
    for (;;) {
      if (++g == a.v.G) {
        if (++bi > last) return false;
        load(a);
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

template <typename C>
__global__ void __launch_bounds__(C::THREADS, 1) batch_tc_kernel(const __grid_constant__ TcArgs ta) {
  constexpr int D = C::D, MT = C::MT, KT = C::KT, KP = C::KP, NBS = C::NBS, NQ = C::NQ, NH = C::NH, NST = C::NST;
  const BatchArgs& a = ta.b;
  const BatchView& v = a.v;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  int* sPos = reinterpret_cast<int*>(sm + C::OFF_POS);
  int2* sLim = reinterpret_cast<int2*>(sm + C::OFF_LIM);
  unsigned* sMask = reinterpret_cast<unsigned*>(sm + C::OFF_MASK);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
  auto bar = [&](int i) { return smem_u32(bars + i); };
  __shared__ long long s_scan[C::THREADS / 32 + 1];
  __shared__ int s_ends[2];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto wait = [&](int i, uint32_t parity) { return mbar_wait(bar(i), parity, &s_abort, a.flag); };

  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < NST; ++i) {
      mbar_init(bar(C::B_KFULL + i), 1);
      mbar_init(bar(C::B_VFULL + i), 1);
      mbar_init(bar(C::B_READY + i), 4);
      mbar_init(bar(C::B_KEMPTY + i), MT);
      mbar_init(bar(C::B_VEMPTY + i), MT);
    }
    for (int i = 0; i < MT * NBS; ++i) {
      mbar_init(bar(C::B_SFULL + i), 1);
      mbar_init(bar(C::B_PREADY + i), 4);
      mbar_init(bar(C::B_PVDONE + i), 1);
    }
    for (int i = 0; i < MT * NQ; ++i) {
      mbar_init(bar(C::B_QFULL + i), 1);
      mbar_init(bar(C::B_QEMPTY + i), 1);
    }
    for (int t = 0; t < MT; ++t) mbar_init(bar(C::B_DONE + t), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == C::W_MMA) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                 "r"(C::TMEM_COLS));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("griddepcontrol.launch_dependents;");
  fence_before();
  const BatchShare share_ = plan_batch<C::THREADS>(a, s_scan, s_ends);   // ends with a __syncthreads
  fence_after();
  const uint32_t tmem = s_tmem;
  Walk w;

  if (warp < 4 * MT) {
    // =============================== softmax: MMA tile t, row m of the item
    if constexpr (MT == 2) regs_inc<176>();
    const int t = warp >> 2, m = 128 * t + 32 * (warp & 3) + lane;
    const int tok = m / v.rep, hh = m % v.rep;
    const uint32_t trow = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t t_o = trow + D * t, t_sb = trow + C::TM_S + 128 * t;
    const float sl = 1.4426950408889634f * rsqrtf((float)D);
    uint32_t gt = 0, ct = 0;   // key tiles of the CTA, of this MMA tile
    bool ok = true;
    for (bool more = w.begin(a, share_); more && ok; more = w.next(a)) {
      const int n = w.j1 - w.j0;
      if (w.b.nrows * v.rep <= 128 * t) {   // the item has no rows for this MMA tile
        gt += n;
        continue;
      }
      const bool mine = tok < w.b.nrows && m < v.rb * v.rep;
      const bool idle = !__any_sync(0xffffffffu, mine);
      const int qp = w.b.req < 0 ? INT_MAX - 1 : w.b.pos0 + (mine ? tok : 0);
      const int lo = w.b.req < 0 ? -1 : qp - v.window;   // own keys at or below lo are seen as sinks only
      float mref = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j, ++gt, ++ct) {
        const int b = ct % NBS, slot = gt % C::NPOS;
        const uint32_t t_s = t_sb + KT * b;
        ok = __all_sync(0xffffffffu, wait(C::B_SFULL + t * NBS + b, (ct / NBS) & 1));
        if (!ok) break;
        fence_after();
        if (!idle) {
          const int2 lim = sLim[slot];
          float s[KT];
#pragma unroll
          for (int c = 0; c < KT; c += 16) tmem_ld16(t_s + c, s + c);
          tmem_wait_ld();
          if (__any_sync(0xffffffffu, lim.x > qp || lim.y <= lo)) {
            const int4* kp = reinterpret_cast<const int4*>(sPos + slot * KT);
#pragma unroll
            for (int i = 0; i < KT / 4; ++i) {
              const int4 k4 = kp[i];
              auto out = [&](int u) { return u > qp || (u <= lo && u >= v.sinks); };
              if (out(k4.x)) s[4 * i] = -INFINITY;
              if (out(k4.y)) s[4 * i + 1] = -INFINITY;
              if (out(k4.z)) s[4 * i + 2] = -INFINITY;
              if (out(k4.w)) s[4 * i + 3] = -INFINITY;
            }
          }
          float m4[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) m4[u] = s[u];
#pragma unroll
          for (int i = 4; i < KT; ++i) m4[i & 3] = fmaxf(m4[i & 3], s[i]);
          const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * sl;
          const bool grow = mx > mref + kRescale;
          const float mnew = grow ? mx : mref;
          const float scale = (grow && mref != -INFINITY) ? ex2(mref - mnew) : 1.f;
          l *= scale;
          mref = mnew;
          const float mz = mref == -INFINITY ? 0.f : mref;   // nothing seen so far: every s is -inf, p = 0
          float r4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int h = 0; h < KT / 32; ++h) {
            uint32_t pv[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float p0 = ex2(fmaf(s[32 * h + 2 * e], sl, -mz)), p1 = ex2(fmaf(s[32 * h + 2 * e + 1], sl, -mz));
              r4[e & 3] += p0 + p1;
              pv[e] = pack_bf16x2(p0, p1);
            }
            tmem_st16(t_s + KT / 2 + 16 * h, pv);
          }
          l += (r4[0] + r4[1]) + (r4[2] + r4[3]);
          if (__any_sync(0xffffffffu, scale != 1.f)) {
            // O holds the item's earlier tiles (a finite earlier maximum): their PVs first
            ok = __all_sync(0xffffffffu, wait(C::B_PVDONE + t * NBS + (ct - 1) % NBS, ((ct - 1) / NBS) & 1));
            if (!ok) break;
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
          }
          tmem_wait_st();
          fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::B_PREADY + t * NBS + b));
      }
      if (!ok) break;
      ok = __all_sync(0xffffffffu, wait(C::B_PVDONE + t * NBS + (ct - 1) % NBS, ((ct - 1) / NBS) & 1));
      if (!ok) break;
      if (idle) continue;
      fence_after();
      const float inv = l == 0.f ? 0.f : 1.f / l;   // no key seen: zeros; NaN stays NaN
      const bool whole = w.j0 == 0 && w.j1 == w.nt;
      const size_t head = mine ? (size_t)(w.b.row0 + tok) * a.H + w.g * v.rep + hh : 0;
      __half* dst = nullptr;
      float* po = nullptr;
      if (whole && v.pre_len == 0) {
        dst = static_cast<__half*>(a.out) + head * D;
      } else if (mine) {
        const size_t at = whole ? (w.b.req < 0 ? 0 : (size_t)v.T * a.H) + head
                                : (size_t)part_slot(blockIdx.x, w.start, w.x0) * a.part_rows + m;
        po = (whole ? a.seg_o : a.part_o) + at * D;
        (whole ? a.seg_ml : a.part_ml)[at] = make_float2(mref, l);
      }
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        float o[32];
        tmem_ld16(t_o + c0, o);
        tmem_ld16(t_o + c0 + 16, o + 16);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = l == 0.f ? 0.f : o[e] * inv;
        if (!mine) continue;
        if (dst) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint4*>(dst + c0 + 8 * c) =
                make_uint4(pack_f16x2(o[8 * c], o[8 * c + 1]), pack_f16x2(o[8 * c + 2], o[8 * c + 3]),
                           pack_f16x2(o[8 * c + 4], o[8 * c + 5]), pack_f16x2(o[8 * c + 6], o[8 * c + 7]));
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c)
            *reinterpret_cast<float4*>(po + c0 + 4 * c) = make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
        }
      }
      fence_before();   // the next item's first PV overwrites O only after this warp's next P
    }
    if (!ok) s_abort = 1;
  } else if (warp < C::W_ROT) {
    if constexpr (MT == 2) regs_dec<80>();
    if (warp < C::W_LOAD) {
      // =============================== MMA tile t: one thread issues its products
      const int t = warp - C::W_MMA;
      if (lane == 0) {
        constexpr uint32_t id_s = idesc_s(128, KT), id_pv = idesc_pv(128, D);
        // two walks over the same tiles: S products up to NBS tiles ahead of the PV products
        Walk ws;
        bool mp = w.begin(a, share_), ms = ws.begin(a, share_);
        uint32_t gs = 0, gp = 0, cs = 0, cp = 0, qs = 0;   // tiles of the CTA, of this MMA tile; items of it
        int js = ws.j0, jp = w.j0;
        bool ok = true;
        uint32_t idle = 0;
        unsigned long long t_idle = 0;
        while (mp && ok) {
          bool prog = false;
          if (w.b.nrows * v.rep <= 128 * t) {
            // no rows in this item: its share of each stage is released once the tile is there
            for (; jp < w.j1 && ok; ++jp, ++gp) {
              const int st = gp % NST;
              ok = wait(C::B_READY + st, (gp / NST) & 1) && wait(C::B_VFULL + st, (gp / NST) & 1);
              if (ok) {
                mbar_arrive(bar(C::B_KEMPTY + st));
                mbar_arrive(bar(C::B_VEMPTY + st));
              }
            }
            mp = w.next(a);
            jp = w.j0;
            continue;
          }
          if (cp < cs) {   // PV of the next tile
            const int b = cp % NBS, st = gp % NST;
            if (mbar_test(bar(C::B_PREADY + t * NBS + b), (cp / NBS) & 1) &&
                mbar_test(bar(C::B_VFULL + st), (gp / NST) & 1)) {
              fence_after();
              const uint32_t vb = smem_u32(sm + C::OFF_V + st * C::K_BYTES);
              const uint32_t pa = tmem + C::TM_S + 128 * t + KT * b + KT / 2;
#pragma unroll
              for (int k = 0; k < KT / 16; ++k)
                umma_ts(tmem + D * t, pa + 8 * k, desc_mnmajor(vb + k * 2048, KT * 128), id_pv, jp != w.j0 || k != 0);
              umma_commit(bar(C::B_PVDONE + t * NBS + b));
              umma_commit(bar(C::B_VEMPTY + st));
              ++cp, ++gp;
              if (++jp == w.j1) {
                mp = w.next(a);
                jp = w.j0;
              }
              prog = true;
            }
          }
          if (ms && cs < cp + NBS) {   // S of the tile after
            if (ws.b.nrows * v.rep <= 128 * t) {   // released in the PV walk above
              gs += ws.j1 - ws.j0;
              ms = ws.next(a);
              js = ws.j0;
              prog = true;
            } else {
              const int b = cs % NBS, st = gs % NST, qb = qs % NQ;
              if (mbar_test(bar(C::B_READY + st), (gs / NST) & 1) &&
                  (js > ws.j0 || mbar_test(bar(C::B_QFULL + t * NQ + qb), (qs / NQ) & 1))) {
                fence_after();
                const uint32_t qa = smem_u32(sm + C::OFF_Q + (t * NQ + qb) * C::Q_TILE);
                const uint32_t kb = smem_u32(sm + C::OFF_K + st * C::K_BYTES);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                  const uint32_t off = (k & 3) * 32;
                  umma_ss(tmem + C::TM_S + 128 * t + KT * b, desc_kmajor(qa + (k >> 2) * 16384 + off),
                          desc_kmajor(kb + (k >> 2) * (KT * 128) + off), id_s, k != 0);
                }
                umma_commit(bar(C::B_SFULL + t * NBS + b));
                umma_commit(bar(C::B_KEMPTY + st));
                ++cs, ++gs;
                if (++js == ws.j1) {
                  umma_commit(bar(C::B_QEMPTY + t * NQ + qb));
                  ++qs;
                  ms = ws.next(a);
                  js = ws.j0;
                }
                prog = true;
              }
            }
          }
          if (prog) {
            idle = 0;
          } else if (idle++ == 0) {
            t_idle = gtimer();
          } else if ((idle & 255) == 0 && (s_abort || gtimer() - t_idle > kWaitLimitNs)) {
            if (!s_abort) atomicOr(a.flag, kBatchTimeout);
            ok = false;
          }
        }
        if (!ok) s_abort = 1;
        umma_commit(bar(C::B_DONE + t));   // fires once every MMA of this thread has retired
        volatile int never = 0;
        mbar_wait(bar(C::B_DONE + t), 0, &never, a.flag);
      }
    } else if (warp == C::W_LOAD) {
      // =============================== loads
      // A stage's K is free when its S products have retired, but its keys' positions are read by
      // the softmax after that: they have a ring of their own, twice as long (S(j + NST) is only
      // issued after P(j + NST - NBS), so the softmax of tile j is over when slot j is reused).
      bool more = w.begin(a, share_), ok = true;
      uint32_t gt = 0, gk = 0;   // tiles whose V, whose K is asked for
      unsigned bad = 0;
      PageMeta nx{0, 0, 0};
      auto fetch = [&](int j) {   // lane p: page p of tile j of the item w
        const int i = j * KP + lane;
        nx = lane < KP && i < w.b.nv ? page_meta(v, w.b, i, bad) : PageMeta{0, 0, 0};
      };
      int j = more ? w.j0 : 0;
      if (more) fetch(j);
      while (more && ok) {
        const PageMeta pm = nx;
        const int st = gt % NST, slot = gt % C::NPOS, g = w.g;
        const uint32_t kr = gt / NST;
        if (++j == w.j1) {
          more = w.next(a);
          j = w.j0;
        }
        if (more) fetch(j);
        if (lane == 0) ok = kr == 0 || wait(C::B_KEMPTY + st, (kr - 1) & 1);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        // key positions, two or four keys per lane; the last key (INT_MAX when a row holds none)
        // and the first one behind the sinks
        int last = -1, first = INT_MAX;
#pragma unroll
        for (int e = 0; e < KT / 32; ++e) {
          const int key = 32 * e + lane, q = key / kPage, r = key % kPage;
          const int pos = __shfl_sync(0xffffffffu, pm.pos, q);
          const unsigned rows = __shfl_sync(0xffffffffu, pm.rows, q);
          const int u = rows >> r & 1u ? pos + r : INT_MAX;
          sPos[slot * KT + key] = u;
          last = max(last, u);
          if (u >= v.sinks) first = min(first, u);
        }
        last = __reduce_max_sync(0xffffffffu, last);
        first = __reduce_min_sync(0xffffffffu, first);
        if (lane == 0) sLim[slot] = make_int2(last, first);
        if (lane < KP) sMask[st * KP + lane] = pm.rows;
        const int n_full = __popc(__ballot_sync(0xffffffffu, pm.rows != 0));
        __syncwarp();
        const uint32_t kf = bar(C::B_KFULL + st), vf = bar(C::B_VFULL + st);
        if (lane == 0) mbar_expect_tx(kf, (uint32_t)n_full * (kPage * D * 2 + C::CS_ROW));
        __syncwarp();
        const int pg = lane / NH, half = lane % NH;   // one box per lane
        const int blk = __shfl_sync(0xffffffffu, pm.blk, pg % KP);
        const unsigned rows = __shfl_sync(0xffffffffu, pm.rows, pg % KP);
        const uint32_t box = half * (KT * 128) + pg * 2048;
        const bool boxed = pg < KP && rows != 0;
        if (boxed) tma_page(smem_u32(sm + C::OFF_K + st * C::K_BYTES) + box, &ta.kmap, half, g, blk, kf);
        if (lane < KP && pm.rows != 0)
          bulk_g2s(smem_u32(sm + C::OFF_CS + st * C::CS_BYTES + lane * C::CS_ROW), a.rope_cs + (size_t)pm.pos * (D / 2),
                   C::CS_ROW, kf);
        ++gk;
        if (lane == 0) ok = kr == 0 || wait(C::B_VEMPTY + st, (kr - 1) & 1);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(vf, (uint32_t)n_full * (kPage * D * 2));
        __syncwarp();
        if (boxed) tma_page(smem_u32(sm + C::OFF_V + st * C::K_BYTES) + box, &ta.vmap, half, g, blk, vf);
        ++gt;
      }
      batch_flag(a.flag, bad);
      // every copy has landed before the shared memory is given up (at once on the normal path)
      if (lane == 0) {
        volatile int never = 0;
        for (uint32_t s = 0; s < NST; ++s) {
          const uint32_t nk = (gk + NST - 1 - s) / NST, nv = (gt + NST - 1 - s) / NST;
          if (nk) mbar_wait(bar(C::B_KFULL + s), (nk - 1) & 1, &never, a.flag);
          if (nv) mbar_wait(bar(C::B_VFULL + s), (nv - 1) & 1, &never, a.flag);
        }
      }
    } else if (warp == C::W_Q) {
      // =============================== q of the items into the A operands
      uint32_t qi[MT] = {};
      bool ok = true;
      for (bool more = w.begin(a, share_); more && ok; more = w.next(a)) {
        const int rows = w.b.nrows * v.rep;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          if (rows <= 128 * t || !ok) continue;
          const uint32_t q = qi[t]++, qb = q % NQ;
          if (q >= NQ) {
            if (lane == 0) ok = wait(C::B_QEMPTY + t * NQ + qb, (q / NQ - 1) & 1);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
          }
          const uint32_t dst = smem_u32(sm + C::OFF_Q + (t * NQ + qb) * C::Q_TILE);
          const int n = min(128, rows - 128 * t) * (D / 8);   // 16-byte chunks; rows behind the item's stay as they are
          for (int i = lane; i < n; i += 32) {
            const int mr = i / (D / 8), ch = i % (D / 8), mm = 128 * t + mr;
            const __half* src = static_cast<const __half*>(a.q) +
                                ((size_t)(w.b.row0 + mm / v.rep) * a.H + w.g * v.rep + mm % v.rep) * D + 8 * ch;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + (ch >> 3) * 16384 + sw128(mr, ch & 7)),
                         "l"(src)
                         : "memory");
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::B_QFULL + t * NQ + qb));
        }
      }
    }
  } else {
    // =============================== rotation of K in the stages
    if constexpr (MT == 2) regs_dec<80>();
    constexpr int CH = D / 16;                 // 16-byte chunks of the first half of a row's dims
    constexpr int PP = 128 / (16 * CH);        // pages at once: 1 (D 128), 2 (D 64)
    const int rt = tid - C::W_ROT * 32, c = rt % CH, r = rt / CH % kPage, p0 = rt / (16 * CH);
    // (cos, sin) of r theta for the thread's 8 frequencies
    float4 off[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) off[e] = reinterpret_cast<const float4*>(a.rope_cs + (size_t)r * (D / 2) + 8 * c)[e];
    uint32_t gt = 0;
    bool ok = true;
    for (bool more = w.begin(a, share_); more && ok; more = w.next(a)) {
      for (int j = w.j0; j < w.j1; ++j, ++gt) {
        const int st = gt % NST;
        const uint32_t ph = (gt / NST) & 1;
        ok = wait(C::B_KFULL + st, ph);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint8_t* ks = sm + C::OFF_K + st * C::K_BYTES;
        const float4* cs = reinterpret_cast<const float4*>(sm + C::OFF_CS + st * C::CS_BYTES);
        bool holes = false;
#pragma unroll 2
        for (int p = p0; p < KP; p += PP) {
          const unsigned rows = sMask[st * KP + p];
          holes |= rows != 0xffffu;
          uint4* k1 = reinterpret_cast<uint4*>(ks + sw128(p * kPage + r, c));
          uint4* k2 = reinterpret_cast<uint4*>(D == 128 ? ks + KT * 128 + sw128(p * kPage + r, c)
                                                        : ks + sw128(p * kPage + r, c + CH));
          uint4 y1 = make_uint4(0, 0, 0, 0), y2 = y1;
          if (rows >> r & 1u) {
            const uint4 u1 = *k1, u2 = *k2;
            const uint32_t w1[4] = {u1.x, u1.y, u1.z, u1.w}, w2[4] = {u2.x, u2.y, u2.z, u2.w};
            uint32_t o1[4], o2[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 f = cs[p * (D / 4) + 4 * c + e];   // (cos, sin) of P theta, two frequencies
              const float c0 = f.x * off[e].x - f.y * off[e].y, s0 = f.y * off[e].x + f.x * off[e].y;
              const float c1 = f.z * off[e].z - f.w * off[e].w, s1 = f.w * off[e].z + f.z * off[e].w;
              const float a0 = __uint_as_float(w1[e] << 16), a1 = __uint_as_float(w1[e] & 0xffff0000u);
              const float b0 = __uint_as_float(w2[e] << 16), b1 = __uint_as_float(w2[e] & 0xffff0000u);
              o1[e] = pack_f16x2(a0 * c0 - b0 * s0, a1 * c1 - b1 * s1);
              o2[e] = pack_f16x2(b0 * c0 + a0 * s0, b1 * c1 + a1 * s1);
            }
            y1 = make_uint4(o1[0], o1[1], o1[2], o1[3]);
            y2 = make_uint4(o2[0], o2[1], o2[2], o2[3]);
          }
          *k1 = y1;
          *k2 = y2;
        }
        if (__any_sync(0xffffffffu, holes)) {   // rows of V without a key: P is 0 there, V must be finite
          ok = wait(C::B_VFULL + st, ph);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          uint8_t* vs = sm + C::OFF_V + st * C::K_BYTES;
          for (int p = p0; p < KP; p += PP)
            if (!(sMask[st * KP + p] >> r & 1u)) {
              *reinterpret_cast<uint4*>(vs + sw128(p * kPage + r, c)) = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(D == 128 ? vs + KT * 128 + sw128(p * kPage + r, c)
                                                 : vs + sw128(p * kPage + r, c + CH)) = make_uint4(0, 0, 0, 0);
            }
        }
        fence_async_smem();   // the MMAs read these rows through the async proxy
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::B_READY + st));
      }
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (warp == C::W_MMA)
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

// A pool layer [blocks][G][16][D] of bf16 as (64 dims, D / 64 halves, 16 rows, G, blocks); a box is
// one half of one page.
bool page_map(CUtensorMap* m, const void* base, int blocks, int G, int D) {
  auto enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[5] = {64, (cuuint64_t)(D / 64), (cuuint64_t)kPage, (cuuint64_t)G, (cuuint64_t)blocks};
  const cuuint64_t strides[4] = {128, (cuuint64_t)D * 2, (cuuint64_t)kPage * D * 2, (cuuint64_t)G * kPage * D * 2};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1}, box[5] = {64, 1, kPage, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename C>
pic_status launch(const TcArgs& ta, cudaStream_t st) {
  static bool set[64] = {};
  int dev = 0;
  PIC_CUDA(cudaGetDevice(&dev));
  const int smem = C::SMEM + 1024;
  if (dev < 0 || dev >= 64 || !set[dev]) {
    PIC_CUDA(cudaFuncSetAttribute(batch_tc_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  batch_tc_kernel<C><<<ta.b.grid, C::THREADS, smem, st>>>(ta);
  PIC_CUDA(cudaGetLastError());
  return PIC_OK;
}

}  // namespace

// Rows of an item: 128 (one MMA tile) or 256. Two tiles share every K and V tile they load and
// rotate, which pays when blocks fill them; with fewer rows one tile and smaller stages keep more
// bytes in flight.
void batch_tc_view(BatchView& v, int D) {
  const long long rows = (v.pre_len > 0 ? (long long)v.T : pdiv(v.T, v.n_reqs)) * v.rep;
  const bool two = rows > 128;
  v.mrows = two ? 256 : 128;
  v.rb = v.mrows / v.rep;
  v.kpages = two ? Cfg<128, 2>::KP : Cfg<128, 1>::KP;
  v.cost_item = 4;
  v.cost_full = 8;
  v.cost_half = two ? 5 : 8;
  (void)D;
}

pic_status launch_batch_tc(const BatchArgs& a, cudaStream_t st) {
  TcArgs ta;
  ta.b = a;
  if (!page_map(&ta.kmap, a.k_layer, a.v.pool_blocks, a.v.G, a.D) ||
      !page_map(&ta.vmap, a.v_layer, a.v.pool_blocks, a.v.G, a.D))
    return fail(PIC_ERR_CUDA, "cuTensorMapEncodeTiled failed for the pools");
  if (a.D == 128) return a.v.mrows == 256 ? launch<Cfg<128, 2>>(ta, st) : launch<Cfg<128, 1>>(ta, st);
  return a.v.mrows == 256 ? launch<Cfg<64, 2>>(ta, st) : launch<Cfg<64, 1>>(ta, st);
}

}  // namespace pic
