// Tree attention on the 5th-generation tensor
// cores (tcgen05, accumulators in tensor memory), K and V fetched by TMA.
//
// The same operation and the same equal shares of one list of tiles as in
// avsg_tree_attn.cuh; here a unit is up to 256 query rows of a request and
// kv-head and a tile is 128 keys.
//
// One CTA per SM, twelve warps:
//   warps 0-3, 4-7  softmax of stream 0 and 1: a thread owns one row, so the
//                   row's maximum and sum need no exchange; it reads its scores
//                   from tensor memory, writes P over them and scales the
//                   output there when the maximum has grown by more than 2^8
//                   (until then weights up to 2^8 stand in for it: the same
//                   quotient, no pass over the output);
//   warps 8, 10     K and V tiles by TMA, one box per page, a lane each, into a
//                   ring of 160 KB that runs on into the next unit;
//   warps 9, 11     issue the products of stream 0 and 1: S = Q K^T (both in
//                   shared memory), O += P V (P in tensor memory).  An issuing
//                   warp is held up by the products before, so that one warp's
//                   waits for P would leave the tensor cores idle: with one warp
//                   for both streams a tile of 256 rows took 4000 cycles.
// In tiles that some rows see only in part, the softmax warps also make V's
// rows behind the last key and its values that are not finite 0 before the
// product (0 times them would be NaN in rows that do not see them);
// add_bad_values gives the latter back to the rows that do.
// A stream works on halves of a tile (64 keys) with two places for scores, so
// that the scores of its next half are there when it has finished one: its
// softmax follows its softmax, and the products of both streams run beside.
// More than 128 rows: stream x holds rows 128x .. and both use every tile (K
// and V are read once for 256 rows).  Up to 128 rows: the streams take the
// even and the odd tiles, with an output each, joined at the end of the unit.
// Heads of 256: two outputs would leave no tensor memory for scores, so there
// is stream 0 alone, of 128 rows, with tiles of 64 keys (a tile is its half):
// the products of one half hide the softmax of the next.  Stream 1's softmax
// warps write half of the output, its issuing warp passes every tile on.  Q lies
// in tensor memory, where stream 1's scores would be: a product of 64 keys then
// takes 32 cycles (4096 after 4096: 636 us, 710 with both operands in shared
// memory).  The ring has 128 KB there; with 192 or 224 HBM gives less (16 x 8
// units of 32768 tokens: 626 and 632 us, 605 so).
//
// Tiles are taken from the last key backwards: where scores carry a distance
// bias, the largest come first and the output is hardly ever scaled.
//
// Tensor memory (512 columns): S/P of stream x at 128 x + 64 (half & 1), O at
// 256 + 128 x.
//
// What bounds it.  Up to 128 rows: HBM (16 x 8 units of 32768 tokens, 16-token
// pages, heads of 128: 318 us, 6.75 of 6.78 TB/s).  256 rows: the tensor cores
// (64 drafts of 4 heads over the same: 412 to 420 us, 1.3 PFLOP/s; a causal
// 4096-token chunk after 4096: 332 us, 1.24 PFLOP/s of the pairs that are seen:
// about 0.7 of what the products' own cycles, 440 + 256 a half, allow).  A product of 128 rows
// and 64 keys reads both operands from shared memory and takes 55 cycles, not
// 32: the price of two places for scores.  One place of 128 keys (64 cycles a
// product) made the streams wait for one another (533 us), and so did weights
// in shared memory, which free the place early but cost a proxy fence a half
// (554 us).  Heads of 256: 600 us for 16 x 8 units of 32768 tokens (7.2 TB/s), 636 us for
// 4096 after 4096 (1.30 PFLOP/s of the pairs that are seen; four softmax warps carry all of it,
// stream 1's wait for the output).  Short units pay 6 to 10 us each for their beginning and
// end, a third of it hidden by the loads that run ahead (256 x 8 units of 1000 tokens, 64
// rows: 234 us, 256 rows: 383 us).
// P is rounded to the cache's type, half a step, like the result: the error against 64 bits is 1.4
// times that of fp32 weights in bf16, 1.2 in fp16 (the remainder as a second product would cost the
// time of the first again, a third of the tensor cores' time).  Sums, maxima and outputs are fp32.
// Every wait is bounded; a wait that gives up latches AVSG_ERR_TIMEOUT, and
// the waits after it return at once.  A warp whose wait failed issues no copy
// after it and passes no buffer on, so that none is filled while its barrier
// still expects a copy; the products after it are of no use to anyone (and
// harmless: all operands lie where they always do).  Copies and products that
// were issued are awaited all the same before the CTA ends or frees its tensor
// memory.
#pragma once

#include <cuda.h>
#include <stdlib.h>

#include "avsg_tree_attn.cuh"

namespace avsg {
namespace tree {
namespace {

constexpr int UM = 128;                    // rows per stream
constexpr int kUmmaThreads = 384;
constexpr int UH = 64;                     // keys per half tile
constexpr float kLazy = 8.f;               // growth of the maximum (log2) that O is scaled for
constexpr long long kWaitClocks = 4000000000LL;  // about two seconds

struct UmmaArgs {
  TreeArgs t;
  int box_rows;                            // tokens per TMA box: min(page, tile)
  int q_vec;                               // rows of q are 16-byte aligned
#ifdef AVSG_DEBUG_BOUNDS
  long long wait_clocks;                   // what a wait may take
#endif
};

template <int D>
struct Mem {
  static constexpr bool SOLO = D > 128;    // one stream
  static constexpr int UT = SOLO ? UH : 2 * UH;  // keys per tile
  static constexpr int ROWS = SOLO ? UM : 2 * UM;  // rows of a unit
  static constexpr int Q = SOLO ? 0 : UM * D * 2;  // bytes of one stream's rows
  static constexpr int TILE = UT * D * 2;
  static constexpr int BUFS = D == 64 ? 10 : D == 128 ? 5 : 4;  // 160 KB, 128 KB for D of 256
  // Heads of 256: m and l of the rows (see s_m), then q on its way to tensor memory in padded rows.
  static constexpr int STAGE = 2 * UM * 4, STAGE_ROW = D * 2 + 16;
  static constexpr int RING = SOLO ? (STAGE + UM * STAGE_ROW + 1023) / 1024 * 1024 : 2 * Q;
  static constexpr int BARS = RING + BUFS * TILE;
  static constexpr int SMEM = BARS + 8 * (2 * BUFS + 16);
};

__device__ __forceinline__ void bar_init(uint32_t b, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(b), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(b) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t b, int bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(b), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(b), "r"(parity)
      : "memory");
  return ok != 0;
}
// The same without the wait that the hardware may put into a try.
__device__ __forceinline__ bool bar_test(uint32_t b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(b), "r"(parity)
      : "memory");
  return ok != 0;
}
// One arrival for a warp (32 of them to one barrier cost 300 cycles).
__device__ __forceinline__ void warp_arrive(uint32_t b, int lane) {
  __syncwarp();
  if (lane == 0) bar_arrive(b);
}
// Waits for the phase of the given parity.  False: it did not come in time, or another wait has given
// up and this one would have had to wait.  In the bounds-checked build a call may set the limit, and
// a try does not wait in the hardware, so that a test can let waits run out.
struct Waits {
  long long clocks;
  volatile int* gave_up;
  DevErr* err;
};
__device__ __forceinline__ bool bar_wait(uint32_t b, uint32_t parity, const Waits& w) {
#ifdef AVSG_DEBUG_BOUNDS
  auto come = [&] { return bar_test(b, parity); };
#else
  auto come = [&] { return bar_try(b, parity); };
#endif
  if (come()) return true;
  const long long t0 = clock64();
  while (!come()) {
    if (*w.gave_up) return false;
    if (clock64() - t0 > w.clocks) {
      *w.gave_up = 1;
      raise_error(w.err, AVSG_ERR_TIMEOUT, -1, -1);
      return false;
    }
  }
  return true;
}
// Waits for copies or products that were issued: their end comes whatever became of other waits.
__device__ __forceinline__ void bar_drain(uint32_t b, uint32_t parity) {
  if (bar_try(b, parity)) return;
  const long long t0 = clock64();
  while (!bar_try(b, parity) && clock64() - t0 <= kWaitClocks) {}
}
// One lane of a converged warp, always the same one.  (Code under it keeps the operands of
// the tensor and copy instructions in uniform registers; under `lane == 0` each of them cost
// 90 to 180 cycles to issue.)
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(ok));
  return ok != 0;
}
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int group, int page) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%3, %3, %3, %4, %5}], [%2];" ::
          "r"(dst), "l"(map), "r"(bar), "r"(0), "r"(group), "r"(page)
      : "memory");
}
// The same as the L2's first candidate for eviction.
__device__ __forceinline__ void tma_box_once(uint32_t dst, const CUtensorMap* map, uint32_t bar, int group, int page,
                                             uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
      "[%1, {%3, %3, %3, %4, %5}], [%2], %6;" ::
          "r"(dst), "l"(map), "r"(bar), "r"(0), "r"(group), "r"(page), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
               : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, int add) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
      "r"(add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, int add) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
      "r"(add)
      : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void async_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// (The loaded registers pass through the wait: their uses cannot move above it.)
__device__ __forceinline__ void tm_wait_ld(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               ::"memory");
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 consecutive columns of this thread's lane.
__device__ __forceinline__ void tm_ld32(uint32_t at, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}
__device__ __forceinline__ void tm_st32(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
      "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]),
      "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(at)
      : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(at)
      : "memory");
}

__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float at_most_60(float x) { return x > 60.f ? 60.f : x; }  // (NaN stays)
// Two fp32 values at once.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t x;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(lo), "f"(hi));
  return x;
}
__device__ __forceinline__ void unpair(uint64_t x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Shared-memory operand of 128-byte swizzled rows: atoms of 8 rows by 64
// columns (1024 bytes), the COLS atoms of 8 whole rows beside each other, so
// groups of 8 rows lie 1024 * COLS bytes apart and blocks of 64 columns 1024.
// A box of one page thus lands in one piece: its TMA dimensions are 64
// columns, 8 rows, COLS blocks, row groups and the page.
// The low word holds the address, the rest is the same for all operands.
__device__ __forceinline__ uint32_t operand_low(uint32_t at) { return (at >> 4) | ((1024 >> 4) << 16); }
template <int COLS>
__device__ __forceinline__ uint64_t operand(uint32_t low) {
  constexpr uint32_t high = (1024 * COLS >> 4) | (1u << 14) | (2u << 29);
  uint64_t x;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "r"(low), "n"(high));
  return x;
}
// A value that all lanes hold, known to the compiler to be one (it then stays in a uniform
// register, where the tensor instructions want their operands: without it every operand is moved
// there lane by lane, 57 cycles an instruction).
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_or_sync(0xffffffffu, x); }

template <typename T>
__device__ constexpr uint32_t instruction(int n, bool b_along_k) {
  const uint32_t type = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
  return (1u << 4) | (type << 7) | (type << 10) | (b_along_k ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(UM >> 4) << 24);
}

// Place of tile t's V among the segment's loads (see the load order below).
__device__ __forceinline__ int v_place(bool two, int t, int count) {
  return two ? 2 * t + 1 : count == 1 ? 1 : 2 + t + min(t, count - 2);
}

// One capped score, in units of log 2.
__device__ __forceinline__ float capped(const TreeArgs& a, float x) {
  const float t = x * a.cap_in * kCapUnit, u = t * t;
  if (fabsf(t) <= kCapNear) return t * a.cap_out * fmaf(fmaf(fmaf(kCap3, u, kCap2), u, kCap1), u, 1.f);
  return a.cap_out * (1.f - __fdividef(2.f, ex2(x * a.cap_in) + 1.f));
}

// Adds what the products left out: values of V that are not finite, in tiles
// that some rows see only in part, times this row's weights (rows that do not
// see them are thus not reached).  `row` is the row's written output, `ref`
// the maximum (log2) its weights are relative to, `inv` their factor.
template <typename T, typename TO, int D>
__device__ __noinline__ void add_bad_values(const TreeArgs& a, const Piece& s, const unsigned char* q, int tok,
                                            int q_pos, unsigned long long bits, float slope, float ref,
                                            float inv, TO* row) {
  constexpr int UT = Mem<D>::UT;
  for (int t = 0; t < s.count; ++t) {
    if (!s.edge<Mem<D>::UT>(t, a.window)) continue;
    const int end = min(s.j0 + (t + 1) * UT, s.limit);
    for (int j = a.window > 0 ? s.j0 + t * UT : max(s.j0 + t * UT, s.all_see); j < end; ++j) {
      const int page = a.tables[(size_t)s.r * a.max_pages + (j >> a.shift)];
      if (page < 0 || page >= a.num_pages) continue;
      const long long at = ((((long long)page * a.H + s.h) << a.shift) + (j & ((1 << a.shift) - 1))) * D;
      const uint32_t* v = reinterpret_cast<const uint32_t*>(a.v) + at / 2;
      const uint32_t* k = reinterpret_cast<const uint32_t*>(a.k) + at / 2;
      bool bad = false;
      for (int d = 0; d < D / 2; ++d) bad |= not_finite<T>(v[d]);
      if (!bad) continue;
      const int jd = j - s.len;
      bool see = true;
      int k_pos = j;
      if (jd >= 0) {
        if (s.chain) {
          see = jd <= tok;
        } else {
          see = jd < 64 && ((bits >> jd) & 1);
          const unsigned long long w = a.mask[s.f + jd];
          if (w) k_pos = s.len + __popcll(w) - 1;
        }
      }
      if (!see || (a.window > 0 && q_pos - k_pos >= a.window)) continue;
      float x = 0.f;
      for (int d = 0; d < D / 2; ++d) {
        const float2 y = unpack<T>(reinterpret_cast<const uint32_t*>(q)[d]), z = unpack<T>(k[d]);
        x += y.x * z.x + y.y * z.y;
      }
      if (a.cap_in != 0.f) x = capped(a, x);
      else x *= a.score_log2;
      // (a weight that rounds to 0 gives NaN, as it does in the products of tiles seen whole)
      const float p = unpack<T>(pack<T>(ex2(x - slope * (float)(q_pos - k_pos) - ref), 0.f)).x;
      for (int d = 0; d < D; ++d) {
        const uint32_t pair = v[d / 2];
        if (!not_finite<T>(d & 1 ? pair & 0xffff0000u : pair & 0xffffu)) continue;
        const float2 y = unpack<T>(pair);
        const float add = p * inv * (d & 1 ? y.y : y.x);
        if constexpr (sizeof(TO) == 4) row[d] += add;
        else row[d] = static_cast<TO>(static_cast<float>(row[d]) + add);
      }
    }
  }
}

// EXTRA: with a score cap or a distance bias.  SHARED: one part of an attention over common prefixes.
template <typename T, int D, bool EXTRA, bool SHARED>
__global__ void __launch_bounds__(kUmmaThreads, 1)
    tree_umma_kernel(UmmaArgs ua, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map) {
  using M = Mem<D>;
  constexpr int kRing = M::BUFS, UT = M::UT;
  constexpr bool SOLO = M::SOLO;
  constexpr bool HALF = std::is_same<T, __half>::value;
  constexpr float SHIFT = HALF ? kHalfShift : 0.f;
  constexpr int COLS = D / 64;             // blocks of 64 columns
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ long long s_warp[kUmmaThreads / 32];
  __shared__ Begin<UT, SHARED> s_begin;
  __shared__ int s_give_up, s_bad[2];
  __shared__ uint32_t s_tmem;
  __shared__ unsigned char s_depth[2][kMaxDrafts];
  // The softmax warps' walk: its state would cost registers that the scores need.
  __shared__ Walk<UT, SHARED> s_walk;
  __shared__ Piece s_piece[2];
  __shared__ int s_more[2];
  const TreeArgs& a = ua.t;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = blockIdx.x;
  const uint32_t smem = smem_u32(smem_raw);
  float* s_m = reinterpret_cast<float*>(smem_raw + M::Q);  // (where up to 128 rows leave stream 1's q free)
  float* s_l = s_m + (SOLO ? UM : 2 * UM);
  const uint32_t bars = smem + M::BARS;
  auto full = [&](int b) { return bars + 8 * b; };
  auto empty = [&](int b) { return bars + 8 * (kRing + b); };
  auto s_full = [&](int x, int b) { return bars + 8 * (2 * kRing + 2 * x + b); };
  auto p_full = [&](int x, int b) { return bars + 8 * (2 * kRing + 4 + 2 * x + b); };
  auto o_done = [&](int x) { return bars + 8 * (2 * kRing + 8 + x); };
  auto o_last = [&](int x) { return bars + 8 * (2 * kRing + 10 + x); };
  auto q_full = [&](int x) { return bars + 8 * (2 * kRing + 12 + x); };  // 129 to 256 rows
  const uint32_t q_one = bars + 8 * (2 * kRing + 14);                     // up to 128
  const uint32_t drained = bars + 8 * (2 * kRing + 15);  // every product has ended

  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (int b = 0; b < kRing; ++b) {
      bar_init(full(b), 1);
      bar_init(empty(b), 2);
    }
    for (int x = 0; x < 2; ++x) {
      for (int b = 0; b < 2; ++b) {
        bar_init(s_full(x, b), 1);
        bar_init(p_full(x, b), UM / 32);
      }
      bar_init(o_done(x), 1);
      bar_init(o_last(x), 1);
      bar_init(q_full(x), UM / 32);
    }
    bar_init(q_one, UM / 32);
    bar_init(drained, 2);
    s_give_up = s_bad[0] = s_bad[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (!SHARED || a.part == 0) griddep_wait();  // (part 1 waits for part 0 at its end)
  if (SHARED) griddep_launch();
  Walk<UT, SHARED> walk;
  const bool idle = !walk.begin(a, s_warp, &s_begin);
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  if (idle) {
    if (SHARED) griddep_wait();
    else if (tid == 0) a.head[cta] = make_int4(0, 0, 0, 0);
    if (warp == 9)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    return;
  }
  if (!SHARED) griddep_launch();
#ifdef AVSG_DEBUG_BOUNDS
  const Waits waits{ua.wait_clocks, &s_give_up, a.err};
#else
  const Waits waits{kWaitClocks, &s_give_up, a.err};
#endif
  if (tid == 0) {
    if (smem & 1023) raise_error(a.err, AVSG_ERR_INTERNAL, -1, -1);  // (atoms are 1024-byte aligned)
    s_walk = walk;
    s_more[0] = s_walk.next(a, s_piece[0]);
  }
  __syncthreads();

  if (warp < 8) {
    // ---- softmax: one row per thread
    const int x = warp >> 2, row = tid & (UM - 1);
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes, in bits 16 and up
    const uint32_t to = tmem + lanes + 256 + 128 * x;
    int4 head = make_int4(0, 0, 0, 0);
    int hh = 0, seg = 0, idx = 0;  // hh: halves of this stream since the start
    // V of tile t, made safe to multiply: see above.  Rows that every query sees are left alone
    // (what they hold reaches every query anyway), which without a window are all but the new
    // tokens'.  Both streams may do the same tile: they write the same values.  The load before
    // it in its buffer came before this tile's K, which has been seen, so the parity tells.
    auto clean_v = [&](const Piece& s, bool two, int t) {
      const int n = idx + v_place(two, t, s.count), b = n % kRing;
      const int j = s.j0 + (s.count - 1 - t) * UT, rows = min(UT, s.limit - j);
      const int from = a.window > 0 ? 0 : max(0, s.all_see - j);
      bar_wait(full(b), (n / kRing) & 1, waits);
      unsigned char* v = smem_raw + M::RING + b * M::TILE;
      bool bad = false;
      for (int y = from * (D / 8) + row; y < UT * (D / 8); y += UM) {
        const int vr = y / (D / 8), ch = y % (D / 8);  // row, 16-byte chunk of it (of any order)
        uint4* at = reinterpret_cast<uint4*>(v + (vr / 8) * (1024 * COLS) + (ch / 8) * 1024 + (vr & 7) * 128 +
                                             (ch & 7) * 16);
        if (vr >= rows) {
          *at = make_uint4(0u, 0u, 0u, 0u);
          continue;
        }
        uint4 c = *at;
        uint32_t e[4] = {c.x, c.y, c.z, c.w};
        bool here = false;
#pragma unroll
        for (int z = 0; z < 4; ++z)
          if (not_finite<T>(e[z])) {
            if (not_finite<T>(e[z] & 0xffffu)) e[z] &= 0xffff0000u;
            if (not_finite<T>(e[z] & 0xffff0000u)) e[z] &= 0xffffu;
            here = true;
          }
        if (here) {
          *at = make_uint4(e[0], e[1], e[2], e[3]);
          bad = true;
        }
      }
      if (bad) s_bad[seg & 1] = 1;
      async_fence();
    };
    for (; s_more[seg & 1]; ++seg) {
      const Piece& s = s_piece[seg & 1];
      const bool two = !SOLO && s.ntok * a.G > UM;
      const int rl = two ? x * UM + row : row;
      const bool mine = rl < s.ntok * a.G;
      const int lt = rl / a.G, gg = rl - lt * a.G;
      // q into shared memory, a row by D / 8 lanes; rows past the unit's are zeros
      const bool warp_live = rl - lane < s.ntok * a.G;
      bool q_loading = false;
      // (part 0) a member's token, looked up once by the lane whose row it is in
      int token = 0;
      if (SHARED && a.part == 0 && mine) token = token_of<SHARED>(a, s, s.tok0 + lt);
      if (two || x == 0) {
        if (warp_live) {
          // (Each lane finds its own row, the warp then loads row by row: the arithmetic of an address is
          // a chain that few warps have nothing to put beside.)
          constexpr int LPR = D / 8, RPI = 32 / LPR;
          const int ch = lane % LPR, sub = lane / LPR;
          const long long own =
              ((long long)(SHARED && a.part == 0 ? token : s.f + s.tok0 + lt) * a.q_stride + (s.h * a.G + gg) * D) * 2;
          const uint32_t to = SOLO ? smem + M::STAGE + ((warp & 3) * 32 + sub) * M::STAGE_ROW + ch * 16
                                   : smem + x * M::Q + (ch / 8) * 1024 + (warp & 3) * (4 * 1024 * COLS);
          const uint32_t shown = __ballot_sync(0xffffffffu, mine);
#pragma unroll
          for (int k = 0; k < 32; k += RPI) {
            const bool ok = shown >> (k + sub) & 1;
            const long long from = __shfl_sync(0xffffffffu, own, k + sub);
            const unsigned char* src = a.q + (ok ? from + ch * 16 : 0);
            const int r8 = (k & 7) | sub;              // the row in its group of 8
            const uint32_t dst = SOLO ? to + k * M::STAGE_ROW
                                      : to + (k / 8) * (1024 * COLS) + r8 * 128 + (((ch & 7) ^ r8) << 4);
            if (ua.q_vec) {
              cp_async16(dst, src, ok ? 16 : 0);
            } else {
#pragma unroll
              for (int z = 0; z < 4; ++z) cp_async4(dst + 4 * z, src + 4 * z, ok ? 4 : 0);
            }
          }
          cp_commit();
          q_loading = true;
        }
      }
      const int tok = mine ? s.tok0 + lt : -1;
      int q_pos = s.len + max(tok, 0);
      unsigned long long bits = 0;
      if (SHARED && a.part == 0) {
        if (mine && (a.slopes || a.window > 0)) q_pos = member_position(a, s, tok, token);
      } else if (!s.chain && mine) {
        bits = a.mask[s.f + tok];
        if (bits) q_pos = s.len + __popcll(bits) - 1;
        if (s.n < 64) bits &= (1ull << s.n) - 1;
      }
      const float slope = a.slopes && mine ? a.slopes[s.h * a.G + gg] * 1.4426950408889634f : 0.f;
      if (!s.chain && (a.slopes || a.window > 0)) {
        // depths of the request's drafts, a copy per stream
        if (row < s.n) {
          const unsigned long long w = a.mask[s.f + row];
          s_depth[x][row] = w ? __popcll(w) - 1 : row;
        }
        __syncwarp();
        asm volatile("bar.sync %0, 128;" ::"r"(3 + x) : "memory");
        if (a.window > 0)
          for (int d = 0; d < s.n; ++d)
            if (q_pos - (s.len + s_depth[x][d]) >= a.window) bits &= ~(1ull << d);
      }
      if (q_loading) {
        cp_wait<0>();
        if constexpr (SOLO) {              // on to tensor memory, a row by the thread that owns it
          __syncwarp();
#pragma unroll 1
          for (int c = 0; c < D / 64; ++c) {
            uint32_t r[32];
#pragma unroll
            for (int y = 0; y < 8; ++y) {
              const uint4 z =
                  *reinterpret_cast<const uint4*>(smem_raw + M::STAGE + row * M::STAGE_ROW + c * 128 + y * 16);
              r[4 * y] = z.x;
              r[4 * y + 1] = z.y;
              r[4 * y + 2] = z.z;
              r[4 * y + 3] = z.w;
            }
            tm_st32(tmem + lanes + 128 + c * 32, r);
          }
          tm_wait_st();
          tc_fence_before();
        } else {
          async_fence();
        }
      }
      if (two || x == 0) warp_arrive(two ? q_full(x) : q_one, lane);

      if (tid == 0) {                      // the next piece, while the first scores are on their way
        s_bad[(seg + 1) & 1] = 0;
        s_more[(seg + 1) & 1] = s_walk.next(a, s_piece[(seg + 1) & 1]);
      }
      float m = -INFINITY, l = 0.f;
      const int halves = SOLO ? (x == 0 ? s.count : 0) : 2 * (two ? s.count : (s.count - x + 1) >> 1);
      // tiles e0 .. e1 - 1 of the piece are seen whole by every row (Piece::edge)
      const int e1 = min(s.count, max(0, s.all_see - s.j0) / UT);
      const int e0 = a.window > 0 ? max(0, (s.far_pos - a.window - s.j0 + UT) / UT) : 0;
      auto wait_scores = [&](int n) {
        bar_wait(s_full(x, n & 1), (n >> 1) & 1, waits);
        __syncwarp();                      // (tensor-memory accesses are the whole warp's)
        tc_fence_after();
      };
      const int last = s.count - 1;
      const uint32_t ts0 = tmem + lanes + 128 * x;
      uint32_t w[2][32];
      if (halves > 0 && warp_live) {
        wait_scores(hh);
        tm_ld32(ts0 + 64 * (hh & 1), w[0]);
        tm_ld32(ts0 + 64 * (hh & 1) + 32, w[1]);
      }
      for (int i = 0; i < halves; ++i, ++hh) {
        const int t = SOLO ? i : two ? i >> 1 : (i & ~1) + x, half = SOLO ? 0 : hh & 1;  // tile, its half
        const int kt = last - t;           // place among the piece's keys
        const bool edge = kt < e0 || kt >= e1;
        const uint32_t ts = ts0 + 64 * (hh & 1);
        if (!warp_live) {                  // only padding: nobody reads what these rows give
          wait_scores(hh);
          if (__builtin_expect(edge && half == 0, 0)) clean_v(s, two, t);
          tc_fence_before();
          warp_arrive(p_full(x, hh & 1), lane);
          continue;
        }
        // gives the keys that the row does not see this value
        auto hide = [&](uint32_t with) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            // committed tokens (a chain: up to this one) below, the window's begin above
            const int j = s.j0 + kt * UT + half * UH + c * 32;
            const int below = s.len + (s.chain ? tok + 1 : 0) - j;
            uint32_t see = below >= 32 ? 0xffffffffu : below <= 0 ? 0u : (1u << below) - 1;
            if (a.window > 0) {
              const int from = q_pos - a.window + 1 - j;
              see &= from <= 0 ? 0xffffffffu : from >= 32 ? 0u : 0xffffffffu << from;
            }
            const int d = j - s.len;       // draft of the chunk's first key
            if (!s.chain && d > -32 && d < 64)
              see |= d >= 0 ? (uint32_t)(bits >> d) : (uint32_t)(bits << -d);
#pragma unroll
            for (int y = 0; y < 32; ++y)
              if (!((see >> y) & 1)) w[c][y] = with;
          }
        };
        // The weights are taken relative to the maximum so far while this half's is found: neither
        // waits for the other.  Where it turns out to have grown too far, once per piece and
        // seldom after, the scores are read again.
        float sum;
        for (bool again = true; again;) {
          tm_wait_ld(w[0]);
          tm_wait_ld(w[1]);
          float scale = a.score_log2;
          float away = 0.f;                // a row's part of the distance bias, the same for all keys
          if constexpr (EXTRA) {
            // capped, in units of log 2
            scale = 1.f;
            float far = 0.f;
            if (a.cap_in != 0.f) {
              // What a row does not see must not choose how its scores are capped, nor reach, as
              // a NaN, the score that it shares a reciprocal with.
              if (__builtin_expect(edge, 0)) hide(0u);
#pragma unroll
              for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int y = 0; y < 32; y += 2)
                  far = max3(far, fabsf(__uint_as_float(w[c][y])), fabsf(__uint_as_float(w[c][y + 1])));
            }
            // The polynomial for a row whose scores of this half are all near 0, the quotient for the
            // others (see cap_polynomial_reach).  Where all rows are near, the special functions are
            // left to the weights (16 x 8 units of 16384 tokens, 256 rows, D 128: 358 to 372 us;
            // the quotient alone 440, both in one warp 560; without a cap 227).
            const float k = a.cap_in * kCapUnit, co = a.cap_out;
            const uint64_t k2 = pair(k, k), one = pair(co, co), c1 = pair(kCap1 * co, kCap1 * co),
                           c2 = pair(kCap2 * co, kCap2 * co), c3 = pair(kCap3 * co, kCap3 * co);
            auto near = [&](uint64_t t) {
              const uint64_t u = mul2(t, t);
              return mul2(t, fma2(fma2(fma2(c3, u, c2), u, c1), u, one));
            };
            // cap tanh(x / cap) = cap (1 - 2 / (exp(2 x / cap) + 1)); two scores share a reciprocal.
            // Beyond 2^60 the quotient is below the last bit anyway.
            auto quotient = [&](float s0, float s1, float& x0, float& x1) {
              const float e0 = ex2(at_most_60(s0 * a.cap_in)) + 1.f;
              const float e1 = ex2(at_most_60(s1 * a.cap_in)) + 1.f;
              const float r = reciprocal(e0 * e1) * (-2.f * co);
              x0 = fmaf(r, e1, co);
              x1 = fmaf(r, e0, co);
            };
            if (a.cap_in != 0.f && __all_sync(0xffffffffu, far * k <= kCapNear)) {
#pragma unroll
              for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int y = 0; y < 32; y += 2) {
                  float x0, x1;
                  unpair(near(mul2(pair(__uint_as_float(w[c][y]), __uint_as_float(w[c][y + 1])), k2)), x0, x1);
                  w[c][y] = __float_as_uint(x0);
                  w[c][y + 1] = __float_as_uint(x1);
                }
            } else if (a.cap_in != 0.f && __all_sync(0xffffffffu, !mine || cap_polynomial_reach(far * k, co) < 0.f)) {
              // (padding rows, whose scores are 0, have no say)
#pragma unroll
              for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int y = 0; y < 32; y += 2) {
                  float x0, x1;
                  quotient(__uint_as_float(w[c][y]), __uint_as_float(w[c][y + 1]), x0, x1);
                  w[c][y] = __float_as_uint(x0);
                  w[c][y + 1] = __float_as_uint(x1);
                }
            } else if (a.cap_in != 0.f) {
              const float reach = cap_polynomial_reach(far * k, co);
#pragma unroll
              for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int y = 0; y < 32; y += 2) {
                  const float s0 = __uint_as_float(w[c][y]), s1 = __uint_as_float(w[c][y + 1]);
                  const uint64_t t = mul2(pair(s0, s1), k2);
                  float t0, t1, n0, n1, x0, x1;
                  unpair(t, t0, t1);
                  unpair(near(t), n0, n1);
                  quotient(s0, s1, x0, x1);
                  w[c][y] = __float_as_uint(fabsf(t0) <= reach ? n0 : x0);
                  w[c][y + 1] = __float_as_uint(fabsf(t1) <= reach ? n1 : x1);
                }
            } else {
#pragma unroll
              for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int y = 0; y < 32; ++y) w[c][y] = __float_as_uint(__uint_as_float(w[c][y]) * a.score_log2);
            }
            if (a.slopes) {
              // slope (pos_q - pos_k), less what is the same for the half's keys
              const int j = s.j0 + kt * UT + half * UH;
              away = slope * (float)(q_pos - j);
              if (s.chain || j + UH <= s.len) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                  for (int y = 0; y < 32; ++y)
                    w[c][y] = __float_as_uint(fmaf(slope, (float)(c * 32 + y), __uint_as_float(w[c][y])));
              } else {
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                  for (int y = 0; y < 32; ++y) {
                    const int d = j + c * 32 + y - s.len;
                    const float at = d >= 0 ? (float)(s.len + s_depth[x][d & 63] - j) : (float)(c * 32 + y);
                    w[c][y] = __float_as_uint(fmaf(slope, at, __uint_as_float(w[c][y])));
                  }
              }
            }
          }
          if (__builtin_expect(edge, 0)) hide(0xff800000u);
          float tops[4];
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const uint32_t* e = w[z >> 1] + 16 * (z & 1);
            tops[z] = __uint_as_float(e[0]);
#pragma unroll
            for (int y = 1; y < 15; y += 2)
              tops[z] = max3(tops[z], __uint_as_float(e[y]), __uint_as_float(e[y + 1]));
            tops[z] = fmaxf(tops[z], __uint_as_float(e[15]));
          }
          const float use = m == -INFINITY ? 0.f : m;
          const uint64_t scale2 = pair(scale, scale), minus2 = pair(SHIFT - use - away, SHIFT - use - away);
          uint64_t sums[2] = {0, 0};
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int y = 0; y < 16; ++y) {
              float p0, p1;
              unpair(fma2(pair(__uint_as_float(w[c][2 * y]), __uint_as_float(w[c][2 * y + 1])), scale2, minus2),
                     p0, p1);
              p0 = ex2(p0);
              p1 = ex2(p1);
              sums[y & 1] = add2(sums[y & 1], pair(p0, p1));
              w[c][y] = pack<T>(p0, p1);
            }
          float sum1;
          unpair(add2(sums[0], sums[1]), sum, sum1);
          sum += sum1;
          const float top = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]) * scale - away;
          const bool grow = top > m + kLazy || (m == -INFINITY && top > m);
          __syncwarp();
          again = __any_sync(0xffffffffu, grow);
          if (__builtin_expect(again, 0)) {
            const float f = grow ? ex2(m - top) : 1.f;
            l *= f;
            m = grow ? top : m;
            if (i > 0) {
              // the product before this one has to be done (the one before it is: these scores
              // came after it)
              bar_wait(o_done(x), (hh - 1) & 1, waits);
              __syncwarp();
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                tm_ld32(to + c * 32, w[0]);
                tm_wait_ld(w[0]);
#pragma unroll
                for (int y = 0; y < 32; ++y) w[0][y] = __float_as_uint(__uint_as_float(w[0][y]) * f);
                tm_st32(to + c * 32, w[0]);
              }
              tm_wait_st();
            }
            tm_ld32(ts, w[0]);
            tm_ld32(ts + 32, w[1]);
          }
        }
        tm_st16(ts, w[0]);                 // over scores that have been read
        tm_st16(ts + 16, w[1]);
        l += sum;
        if (__builtin_expect(edge && half == 0, 0)) clean_v(s, two, t);
        __syncwarp();
        // the next half's scores come while P is stored, where they are there already
        const bool more = i + 1 < halves;
        const bool early =
            more && __all_sync(0xffffffffu, bar_test(s_full(x, ~hh & 1), ((hh + 1) >> 1) & 1));
        if (early) {
          tc_fence_after();
          tm_ld32(ts0 + 64 * (~hh & 1), w[0]);
          tm_ld32(ts0 + 64 * (~hh & 1) + 32, w[1]);
        }
        tm_wait_st();
        tc_fence_before();
        warp_arrive(p_full(x, hh & 1), lane);
        if (more && !early) {
          wait_scores(hh + 1);
          tm_ld32(ts0 + 64 * (~hh & 1), w[0]);
          tm_ld32(ts0 + 64 * (~hh & 1) + 32, w[1]);
        }
      }

      // ---- the end of the piece
      // Up to 128 rows the two streams' outputs are joined here (stream 1 has none in a piece of
      // one tile), half of the columns by either stream's warps.
      const bool join = !SOLO && !two && s.count > 1;
      bar_wait(o_last(x), seg & 1, waits);
      if (!two && (!SOLO || x == 0)) {
        s_m[UM * x + row] = m;
        s_l[UM * x + row] = l;
      }
      __syncwarp();
      tc_fence_after();
      asm volatile("bar.sync 1, 256;" ::: "memory");
      tc_fence_after();
      const bool bad = s_bad[seg & 1] != 0;
      float m1 = -INFINITY, l1 = 0.f;
      if (!two) {
        m = s_m[row];
        l = s_l[row];
        if (join) {
          m1 = s_m[UM + row];
          l1 = s_l[UM + row];
        }
      }
      const float top = fmaxf(m, m1), use = top == -INFINITY ? 0.f : top;
      const float f0 = ex2(m - use), f1 = ex2(m1 - use);
      const float sum = l * f0 + l1 * f1;
      // (SHARED: only requests without a prefix write their output here)
      const bool direct = SHARED && s.whole && a.part == 1 && a.shared[s.r] == 0;
      auto whole = [&] { return SHARED ? direct : s.whole; };
      if (SHARED && a.part == 1) token = s.f + max(tok, 0);
      const float inv = whole() ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
      const long long at = (long long)(SHARED ? token : s.f + max(tok, 0)) * a.H * a.G + s.h * a.G + gg;
      const long long slot = SHARED && s.whole ? at : ((long long)(2 * cta + (s.begins ? 1 : 0)) * M::ROWS + rl);
      auto partial = [&] { return SHARED && s.whole ? a.rows : a.partial; };
      if (SHARED && !two && !SOLO && !direct) asm volatile("bar.sync 2, 256;" ::: "memory");  // (see below)
      if (warp_live) {
        const uint32_t from = two ? to : tmem + lanes + 256;
        const float g0 = f0 * inv, g1 = f1 * inv;  // (inv is 1 where the output is not divided yet)
        uint32_t w0[32], w1[32];
        // (SHARED, where most units leave partials: document of 32768 tokens before 64 requests, 7.0 us from
        // the last product to the CTA's end otherwise, 5.0 so; single units of the tree attention lose 1 to 2%.)
        // Partials pass through shared memory, so that a store writes whole lines and not 16 bytes of 32
        // rows: this warp's part of q's place, which the products are done with (4 KB of 32 rows by 32
        // columns, 16-byte chunks swapped by the row).  Up to 128 rows, m and l lie there too: read by now.
        const uint32_t shown = SHARED ? __ballot_sync(0xffffffffu, mine) : 0;
        float* const first_row = a.partial + (slot - lane + (lane >> 3)) * D;
        unsigned char* const st = smem_raw + (SOLO ? M::STAGE + warp * 4096 : x * M::Q + (warp & 3) * (32 * D * 2));
#pragma unroll 1
        for (int c = two ? 0 : x * (D / 64); c < (two ? D / 32 : (x + 1) * (D / 64)); ++c) {
          tm_ld32(from + c * 32, w0);
          if (join) tm_ld32(from + 128 + c * 32, w1);
          tm_wait_ld(w0);
          tm_wait_ld(w1);
          // (the output of a stream that saw nothing is 0; one that is not finite stays so)
#pragma unroll
          for (int y = 0; y < 32; ++y) {
            float o = __uint_as_float(w0[y]) * g0;
            if (join) o += __uint_as_float(w1[y]) * g1;
            w0[y] = __float_as_uint(o);
          }
          auto o = [&](int y) { return __uint_as_float(w0[y]); };
          if (SHARED && !direct) {
#pragma unroll
            for (int y = 0; y < 8; ++y)
              *reinterpret_cast<float4*>(st + lane * 128 + ((y ^ (lane & 7)) << 4)) =
                  make_float4(o(4 * y), o(4 * y + 1), o(4 * y + 2), o(4 * y + 3));
            __syncwarp();
#pragma unroll
            for (int y = 0; y < 8; ++y) {
              const int r = 4 * y + (lane >> 3);
              // a unit's rows lie one after the other, a token's where the token does
              float* to_row = s.whole ? a.rows + __shfl_sync(0xffffffffu, slot, r) * D
                                      : first_row + (4 * y) * D;
              if (shown >> r & 1)
                *reinterpret_cast<float4*>(to_row + c * 32 + (lane & 7) * 4) =
                    *reinterpret_cast<const float4*>(st + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
            }
          } else if (!mine) {
          } else if (SHARED || s.whole) {
            uint4* dst = reinterpret_cast<uint4*>(a.out + (at * D + c * 32) * 2);
#pragma unroll
            for (int y = 0; y < 4; ++y)
              dst[y] = make_uint4(pack<T>(o(8 * y), o(8 * y + 1)), pack<T>(o(8 * y + 2), o(8 * y + 3)),
                                  pack<T>(o(8 * y + 4), o(8 * y + 5)), pack<T>(o(8 * y + 6), o(8 * y + 7)));
          } else {
            float4* dst = reinterpret_cast<float4*>(a.partial + slot * D + c * 32);
#pragma unroll
            for (int y = 0; y < 8; ++y) dst[y] = make_float4(o(4 * y), o(4 * y + 1), o(4 * y + 2), o(4 * y + 3));
          }
          __syncwarp();
        }
        if (mine && (two || x == 0)) {
          if (!whole())
            *reinterpret_cast<float2*>((SHARED && s.whole ? a.rows_ml : a.ml) + slot * 2) = make_float2(top, sum);
          else if (a.lse)
            a.lse[at] = sum == 0.f ? -INFINITY : (top - SHIFT) * 0.6931471805599453f + logf(sum);
        }
      }
      if (__builtin_expect(bad, 0)) {
        __syncwarp();
        asm volatile("bar.sync 6, 256;" ::: "memory");  // the rows are written
        if (mine && (two || x == 0)) {
          const unsigned char* q =
              a.q + ((long long)(SHARED ? token : s.f + tok) * a.q_stride + (long long)(s.h * a.G + gg) * D) * 2;
          if (whole())
            add_bad_values<T, T, D>(a, s, q, tok, q_pos, bits, slope, use - SHIFT, inv,
                                    reinterpret_cast<T*>(a.out) + at * D);
          else
            add_bad_values<T, float, D>(a, s, q, tok, q_pos, bits, slope, use - SHIFT, 1.f, partial() + slot * D);
        }
      }
      idx += 2 * s.count;
      if (SHARED && s.begins) note_unit(a, s, cta, tid, 2 * UM);
      if (!s.whole && s.begins) head = make_int4(s.last - cta + 1, s.f + s.tok0, s.h, s.ntok * a.G);
      tc_fence_before();
      __syncwarp();
      asm volatile("bar.sync 5, 256;" ::: "memory");  // both outputs are read
    }
    if (!SHARED && tid == 0) a.head[cta] = head;
  } else if (warp == 8 || warp == 10) {
    // ---- loads.  Order of a segment: two streams over all tiles: K0 V0 K1 V1 ...; one tile each
    // in turn: K0 K1 V0 K2 V1 K3 ... -- the order in which the products use them.  Warp 8 fills
    // the buffers of even number, warp 10 the others: a warp has then seen every phase of its
    // buffers' barriers, which their parity alone does not tell apart.  Page ids are looked up
    // one load ahead.
    Piece s;
    const int part = warp == 8 ? 0 : 1;
    const int boxes = UT / ua.box_rows;
    int idx = 0, buf = 0, x = 0;           // the next load: its number, its buffer, its place
    bool more = walk.next(a, s);
    auto step = [&]() {
      ++idx;
      if (++buf == kRing) buf = 0;
      if (++x == 2 * s.count) {
        x = 0;
        more = walk.next(a, s);
      }
    };
    while (more && (buf & 1) != part) step();
    // This warp's next load, this lane's box.  Its page is checked when it is used: right behind the
    // lookup, the check would hold the load before it up.
    int page = -1, group = 0, is_v = 0, to = 0, use = 0, of = 0, key = -1;
    int end = 0;                           // the loads before this one were issued
    auto look_up = [&]() {
      const bool two = !SOLO && s.ntok * a.G > UM;
      int t;
      if (two) {
        t = x >> 1;
        is_v = x & 1;
      } else if (x < 2) {                  // K0, then K1 (or V0 of a single tile)
        is_v = x == 1 && s.count == 1;
        t = is_v ? 0 : x;
      } else {                             // pairs V_t K_{t + 2}, then the last two V
        const int z = x - 2, pairs = 2 * (s.count - 2);
        is_v = z >= pairs || !(z & 1);
        t = z >= pairs ? s.count - 2 + z - pairs : (z >> 1) + ((z & 1) ? 2 : 0);
      }
      const int j = s.j0 + (s.count - 1 - t) * UT + lane * ua.box_rows;
      page = key = -1;
      if (lane < boxes && j < s.limit) {
        page = __ldg(a.tables + (size_t)s.r * a.max_pages + (j >> a.shift));
        group = ((s.h << a.shift) + (j & ((1 << a.shift) - 1))) >> 3;
        of = s.r;
        key = j;
      }
      to = buf;
      use = idx / kRing;
      do step();
      while (more && (buf & 1) != part);
    };
    bool have = more;
    if (have) look_up();
    uint64_t policy = 0;
    if constexpr (SHARED) asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    while (have) {
      int now = page;
      const int now_group = group, now_v = is_v, b = to, phase = use, now_of = of, now_key = key;
      have = more;
      if (more) look_up();
      if (now < 0 || now >= a.num_pages) {
        if (now_key >= 0) raise_error(a.err, AVSG_ERR_BAD_SELECTION, now_of, now_key);
        now = -1;
      }
      const int n = __popc(__ballot_sync(0xffffffffu, now >= 0));
      if (!__all_sync(0xffffffffu, bar_wait(empty(b), (phase & 1) ^ 1, waits))) break;
      end = phase * kRing + b + 1;
      if (lane == 0) bar_expect(full(b), n * ua.box_rows * D * 2);
      __syncwarp();
      if constexpr (SHARED) {
        if (now >= 0)
          tma_box_once(smem + M::RING + b * M::TILE + lane * ua.box_rows * D * 2, now_v ? &v_map : &k_map, full(b),
                       now_group, now, policy);
      } else if (now >= 0) {
        tma_box(smem + M::RING + b * M::TILE + lane * ua.box_rows * D * 2, now_v ? &v_map : &k_map, full(b),
                now_group, now);
      }
    }
    // every copy of this warp has landed before the CTA may end
    for (int b = part; b < kRing && b < end; b += 2) bar_drain(full(b), ((end - 1 - b) / kRing) & 1);
  } else {
      // ---- products.  Up to 128 rows, both warps follow every load, in order: a tile that is the
      // other stream's is passed on, so that a buffer is filled again only when both have seen it
      // (a barrier's parity does not tell a phase from the one two before it).
      Piece s;
      const int me = warp == 9 ? 0 : 1;
      int idx = 0, qs = 0, q1 = 0;
      int ps = 0;                          // halves of this stream since the start
      const uint32_t id_s = instruction<T>(UH, false), id_o = instruction<T>(D, true);
      constexpr uint32_t HALF_TILE = UH / 8 * 1024 * COLS;
      // A wait of this lane has given up: it passes no buffer on.  (Each lane by itself, without a
      // vote: those that pass on are always the same.  A branch around the waits would cost a prompt
      // chunk of heads of 256 5%, products that heed it capped calls 1.5%.)
      bool stop = false;
      auto wait = [&](uint32_t bar, int phase) {
        stop |= !bar_wait(bar, phase & 1, waits);
      };
      auto wait_load = [&](int place) -> uint32_t {
        const int i = idx + place, b = i % kRing;
        wait(full(b), i / kRing);
        return smem + M::RING + b * M::TILE;
      };
      // Scores of half hh (of the stream's halves since the start) from rows q and the keys at k.
      auto scores = [&](int x, int q, uint32_t k, int hh) {
        __syncwarp();
        const uint32_t qa = uniform(operand_low(smem + q * M::Q)), to = uniform(tmem + 128 * x + 64 * (hh & 1));
        const uint32_t to_q = uniform(tmem + 128);   // (heads of 256)
        const uint32_t ka = uniform(operand_low(k + (SOLO ? 0 : (hh & 1) * HALF_TILE))), bar = uniform(s_full(x, hh & 1));
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = ((ks / 4) * 1024 + (ks % 4) * 32) >> 4;
            if constexpr (SOLO) mma_ts(to, to_q + ks * 8, operand<COLS>(ka + off), id_s, ks > 0);
            else mma_ss(to, operand<COLS>(qa + off), operand<COLS>(ka + off), id_s, ks > 0);
          }
          mma_commit(bar);
        }
      };
      // P V of half hh of stream x; v: its tile.
      auto output = [&](int x, uint32_t v, int hh, bool first) {
        wait(p_full(x, hh & 1), hh >> 1);
        tc_fence_after();
        __syncwarp();
        const uint32_t va = uniform(operand_low(v + (SOLO ? 0 : (hh & 1) * HALF_TILE))), bar = uniform(o_done(x));
        const uint32_t from = uniform(tmem + 128 * x + 64 * (hh & 1)), to = uniform(tmem + 256 + 128 * x);
        const uint32_t add = uniform(first ? 0 : 1);
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < UH / 16; ++ks)
            mma_ts(to, from + ks * 8, operand<COLS>(va + ks * (2048 * COLS >> 4)), id_o, ks > 0 ? 1 : add);
          mma_commit(bar);
        }
      };
      auto finish = [&](int x) {
        if (elect_one() && !stop) mma_commit(o_last(x));
      };
      auto pass_on = [&](int place) {
        __syncwarp();
        if (lane == 0 && !stop) bar_arrive(empty((idx + place) % kRing));
      };
      auto release = [&](int place) {
        const uint32_t bar = uniform(empty((idx + place) % kRing));
        if (elect_one() && !stop) mma_commit(bar);
      };
      while (walk.next(a, s)) {
        const bool two = !SOLO && s.ntok * a.G > UM;
        const int x = me;
        if (SOLO) {
          wait(q_one, q1);  // (both warps: the end of the unit before)
          ++q1;
          tc_fence_after();
        }
        if (SOLO && me == 1) {
          for (int i = 0; i < 2 * s.count; ++i) {
            wait_load(i);
            pass_on(i);
          }
        } else if (SOLO) {
          for (int t = 0; t < 2 && t < s.count; ++t) {
            scores(0, 0, wait_load(t), ps + t);
            release(t);
          }
          for (int t = 0; t < s.count; ++t) {
            const int place = v_place(false, t, s.count);
            output(0, wait_load(place), ps + t, t == 0);
            release(place);
            if (t + 2 < s.count) {
              scores(0, 0, wait_load(place + 1), ps + t + 2);
              release(place + 1);
            }
          }
        } else if (two) {
          const int hh = ps;
          wait(q_full(x), qs);
          ++qs;
          tc_fence_after();
          uint32_t k = wait_load(0);
          scores(x, x, k, 0);
          scores(x, x, k, 1);
          release(0);
          for (int t = 0; t < s.count; ++t) {
            const uint32_t v = wait_load(2 * t + 1);
            const bool more = t + 1 < s.count;
            output(x, v, hh + 2 * t, t == 0);
            if (more) {
              k = wait_load(2 * t + 2);
              scores(x, x, k, 0);
            }
            output(x, v, hh + 2 * t + 1, false);
            release(2 * t + 1);
            if (more) {
              scores(x, x, k, 1);
              release(2 * t + 2);
            }
          }
        } else {
          wait(q_one, q1);
          ++q1;
          tc_fence_after();
          for (int t = 0; t < 2 && t < s.count; ++t) {
            const uint32_t k = wait_load(t);
            if (t != me) {
              pass_on(t);
              continue;
            }
            scores(x, 0, k, 0);
            scores(x, 0, k, 1);
            release(t);
          }
          for (int t = 0; t < s.count; ++t) {
            const int place = v_place(false, t, s.count), hh = ps + (t & ~1);
            const bool more = t + 2 < s.count;
            const uint32_t v = wait_load(place);
            if ((t & 1) != me) {
              pass_on(place);
              if (more) {
                wait_load(place + 1);
                pass_on(place + 1);
              }
              continue;
            }
            output(x, v, hh, t < 2);
            const uint32_t k = more ? wait_load(place + 1) : 0;
            if (more) scores(x, 0, k, 0);
            output(x, v, hh + 1, false);
            release(place);
            if (more) {
              scores(x, 0, k, 1);
              release(place + 1);
            }
          }
        }
        // (also where stream 1 has no tile: its softmax warps wait for this warp to have come by)
        finish(x);
        ps += SOLO ? s.count : 2 * (two ? s.count : (s.count + 1 - me) >> 1);
        idx += 2 * s.count;
        __syncwarp();
      }
      // every product of both warps has ended before tensor memory is given back
      if (elect_one()) mma_commit(drained);
      __syncwarp();
      bar_drain(drained, 0);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  if (SHARED) griddep_wait();
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
            cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

// Pages as [num_pages][H * page / 8 groups][D / 64 blocks][8 rows][64 columns]
// (strides of the plain layout), in boxes of min(page, tile) whole rows.
bool encode_pages(CUtensorMap* map, const unsigned char* pages, const TreeArgs& a, int dtype, int D, int box) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return false;
  const cuuint64_t row = (cuuint64_t)D * 2, rows = (cuuint64_t)a.H << a.shift;
  const cuuint64_t dims[5] = {64, 8, (cuuint64_t)D / 64, rows / 8, (cuuint64_t)a.num_pages};
  const cuuint64_t strides[4] = {row, 128, 8 * row, rows * row};
  const cuuint32_t size[5] = {64, 8, (cuuint32_t)D / 64, (cuuint32_t)box / 8, 1}, step[5] = {1, 1, 1, 1, 1};
  return encode(map, dtype == AVSG_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5,
                const_cast<unsigned char*>(pages), dims, strides, size, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

#ifdef AVSG_DEBUG_BOUNDS
// AVSG_TREE_WAIT_CLOCKS in the environment: a shorter limit for the waits.
long long wait_clocks() {
  const char* v = getenv("AVSG_TREE_WAIT_CLOCKS");
  const long long x = v && *v ? atoll(v) : kWaitClocks;
  return x < 0 || x > kWaitClocks ? kWaitClocks : x;
}
#endif

template <typename T, int D, bool EXTRA, bool SHARED>
cudaError_t launch_umma_one(const TreeArgs& a, int dtype, int dev, cudaStream_t st) {
  static SmemLimit limit;
  auto kernel = tree_umma_kernel<T, D, EXTRA, SHARED>;
  cudaError_t e = limit.raise(reinterpret_cast<const void*>(kernel), Mem<D>::SMEM, dev);
  if (e != cudaSuccess) return e;
  UmmaArgs u{};
  u.t = a;
  u.box_rows = (1 << a.shift) < Mem<D>::UT ? 1 << a.shift : Mem<D>::UT;
#ifdef AVSG_DEBUG_BOUNDS
  u.wait_clocks = wait_clocks();
#endif
  u.q_vec = reinterpret_cast<uintptr_t>(a.q) % 16 == 0 && a.q_stride % 8 == 0;
  CUtensorMap k_map, v_map;
  if (!encode_pages(&k_map, a.k, a, dtype, D, u.box_rows) || !encode_pages(&v_map, a.v, a, dtype, D, u.box_rows))
    return cudaErrorInvalidValue;
  e = launch_pdl(kernel, dim3(a.ctas), dim3(kUmmaThreads), Mem<D>::SMEM, st, u, k_map, v_map);
  return e != cudaSuccess || SHARED ? e : launch_merge<T, D>(a, Mem<D>::ROWS, st);
}

template <typename T, int D, bool SHARED>
cudaError_t launch_umma(const TreeArgs& a, int dtype, int dev, cudaStream_t st) {
  return a.cap_in != 0.f || a.slopes ? launch_umma_one<T, D, true, SHARED>(a, dtype, dev, st)
                                     : launch_umma_one<T, D, false, SHARED>(a, dtype, dev, st);
}
template <bool SHARED>
cudaError_t launch_umma_any(const TreeArgs& a, int dtype, int D, int dev, cudaStream_t st) {
  if (dtype == AVSG_BF16)
    return D == 64    ? launch_umma<__nv_bfloat16, 64, SHARED>(a, dtype, dev, st)
           : D == 128 ? launch_umma<__nv_bfloat16, 128, SHARED>(a, dtype, dev, st)
                      : launch_umma<__nv_bfloat16, 256, SHARED>(a, dtype, dev, st);
  return D == 64    ? launch_umma<__half, 64, SHARED>(a, dtype, dev, st)
         : D == 128 ? launch_umma<__half, 128, SHARED>(a, dtype, dev, st)
                    : launch_umma<__half, 256, SHARED>(a, dtype, dev, st);
}

}  // namespace
}  // namespace tree
}  // namespace avsg
