// Tree attention for heads of 64 or 128 values on the 5th-generation tensor
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
//   warp 8          K and V tiles by TMA, one box per page and 64 columns, a
//                   lane each, into a ring of five 32 KB buffers that runs on
//                   into the next unit;
//   warp 9          issues the products: S = Q K^T (both in shared memory),
//                   O += P V (P in tensor memory);
//   warps 10, 11    in tiles that some rows see only in part: V's rows behind
//                   the last key and values that are not finite become 0.
// Two streams keep the tensor cores busy while the other's softmax runs.
// More than 128 rows: stream x holds rows 128x .. and both use every tile (K
// and V are read once for 256 rows).  Up to 128 rows: the streams take the
// even and the odd tiles, with an output each, joined at the end of the unit.
//
// Tensor memory (512 columns): S/P of stream x at 128 x, O at 256 + 128 x.
// Every wait is bounded; a wait that gives up latches AVSG_ERR_TIMEOUT, and
// the waits after it return at once.
#include <cuda.h>

#include "avsg_tree_attn.cuh"

namespace avsg {
namespace tree {
namespace {

constexpr int UT = 128;                    // keys per tile
constexpr int UM = 128;                    // rows per stream
constexpr int kUmmaThreads = 384;
constexpr int kRing = 5;
constexpr float kLazy = 8.f;               // growth of the maximum (log2) that O is scaled for
constexpr long long kWaitClocks = 4000000000LL;

struct UmmaArgs {
  TreeArgs t;
  int box_rows;                            // tokens per TMA box: min(page, 128)
  int q_vec;                               // rows of q are 16-byte aligned
};

template <int D>
struct Mem {
  static constexpr int Q = UM * D * 2;     // bytes of one stream's rows
  static constexpr int TILE = UT * D * 2;
  static constexpr int RING = 2 * Q;
  static constexpr int BARS = RING + kRing * TILE;
  static constexpr int SMEM = BARS + 256 + 1024;  // + alignment of the base to 1024
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
// Waits for the phase of the given parity, a few seconds at most.
__device__ __forceinline__ void bar_wait(uint32_t b, uint32_t parity, volatile int* gave_up, DevErr* err) {
  if (bar_try(b, parity)) return;
  const long long t0 = clock64();
  while (!bar_try(b, parity)) {
    if (*gave_up) return;
    if (clock64() - t0 > kWaitClocks) {
      *gave_up = 1;
      raise_error(err, AVSG_ERR_TIMEOUT, -1, -1);
      return;
    }
  }
}
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::
          "r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
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

// Shared-memory operand of 128-byte swizzled rows (8 rows of 128 bytes make an
// atom of 1024 bytes).  Rows along M or N: groups of 8 rows lie 1024 bytes
// apart.  Rows along K (V): blocks of 64 columns lie `block` bytes apart.
__device__ __forceinline__ uint64_t operand(uint32_t at, uint32_t block) {
  return (uint64_t)((at & 0x3FFFF) >> 4) | ((uint64_t)(block >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
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

// Adds what the products left out: values of V that are not finite, in tiles
// that some rows see only in part, times this row's weights (rows that do not
// see them are thus not reached).  `row` is the row's written output, `ref`
// the maximum (log2) its weights are relative to, `inv` their factor.
template <typename T, typename TO, int D>
__device__ __noinline__ void add_bad_values(const TreeArgs& a, const Piece& s, const unsigned char* q, int tok,
                                            int q_pos, unsigned long long bits, float slope, float ref,
                                            float inv, TO* row) {
  for (int t = 0; t < s.count; ++t) {
    if (!s.edge<UT>(t, a.window)) continue;
    const int end = min(s.j0 + (t + 1) * UT, s.limit);
    for (int j = s.j0 + t * UT; j < end; ++j) {
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
      if (a.cap_in != 0.f) x = a.cap_out * (1.f - __fdividef(2.f, ex2(x * a.cap_in) + 1.f));
      else x *= a.score_log2;
      const float p = unpack<T>(pack<T>(ex2(x - slope * (float)(q_pos - k_pos) - ref), 0.f)).x;
      if (p == 0.f) continue;
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

template <typename T, int D>
__global__ void __launch_bounds__(kUmmaThreads, 1)
    tree_umma_kernel(UmmaArgs ua, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map) {
  using M = Mem<D>;
  constexpr bool HALF = std::is_same<T, __half>::value;
  constexpr float SHIFT = HALF ? kHalfShift : 0.f;
  constexpr int COLS = D / 64;             // blocks of 64 columns
  extern __shared__ unsigned char smem_raw[];
  __shared__ long long s_warp[kUmmaThreads / 32];
  __shared__ long long s_base;
  __shared__ int s_r, s_give_up, s_bad[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_depth[2][kMaxDrafts];
  __shared__ float s_m[UM], s_l[UM];
  const TreeArgs& a = ua.t;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = blockIdx.x;
  const uint32_t smem = (smem_u32(smem_raw) + 1023) & ~1023u;
  const uint32_t bars = smem + M::BARS;
  auto full = [&](int b) { return bars + 8 * b; };
  auto empty = [&](int b) { return bars + 8 * (kRing + b); };
  auto s_full = [&](int x) { return bars + 8 * (2 * kRing + x); };
  auto p_full = [&](int x) { return bars + 8 * (2 * kRing + 2 + x); };
  auto o_full = [&](int x) { return bars + 8 * (2 * kRing + 4 + x); };
  const uint32_t q_full = bars + 8 * (2 * kRing + 6), v_in = bars + 8 * (2 * kRing + 7),
                 v_ok = bars + 8 * (2 * kRing + 8);

  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (int b = 0; b < kRing; ++b) {
      bar_init(full(b), 1);
      bar_init(empty(b), 1);
    }
    for (int x = 0; x < 2; ++x) {
      bar_init(s_full(x), 1);
      bar_init(p_full(x), UM);
      bar_init(o_full(x), 1);
    }
    bar_init(q_full, 2 * UM);
    bar_init(v_in, 1);
    bar_init(v_ok, 64);
    s_give_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  griddep_wait();
  Walk<UT> walk;
  const bool idle = __syncthreads_or(load_err(a.err) != 0) || !walk.begin(a, s_warp, &s_base, &s_r);
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  if (idle) {
    if (tid == 0) a.head[cta] = make_int4(0, 0, 0, 0);
    if (warp == 9)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    return;
  }
  volatile int* give_up = &s_give_up;
  Piece s;

  if (warp == 8) {
    // ---- loads.  Order of a segment: two streams over all tiles: K0 V0 K1 V1 ...; one tile
    // each in turn: K0 K1 V0 K2 V1 K3 ... -- the order in which the products use them.
    int idx = 0;
    const int boxes = UT / ua.box_rows;
    const int bi = lane / COLS, col = lane % COLS;
    while (walk.next(a, s)) {
      const bool two = s.ntok * a.G > UM;
      const int32_t* table = a.tables + (size_t)s.r * a.max_pages;
      for (int x = 0; x < 2 * s.count; ++x, ++idx) {
        int t;
        bool is_v;
        if (two) {
          t = x >> 1;
          is_v = x & 1;
        } else if (x < 2) {                // K0, then K1 (or V0 of a single tile)
          is_v = x == 1 && s.count == 1;
          t = is_v ? 0 : x;
        } else {                           // pairs V_t K_{t + 2}, then the last V
          const int y = x - 2, pairs = 2 * (s.count - 2);
          is_v = y >= pairs || !(y & 1);
          t = y >= pairs ? s.count - 2 + y - pairs : (y >> 1) + ((y & 1) ? 2 : 0);
        }
        const int j = s.j0 + t * UT + bi * ua.box_rows;
        int page = -1;
        if (bi < boxes && j < s.limit) {
          page = __ldg(table + (j >> a.shift));
          if (page < 0 || page >= a.num_pages) {
            raise_error(a.err, AVSG_ERR_BAD_SELECTION, s.r, j);
            page = -1;
          }
        }
        const int b = idx % kRing;
        const int n = __popc(__ballot_sync(0xffffffffu, page >= 0));
        bar_wait(empty(b), ((idx / kRing) & 1) ^ 1, give_up, a.err);
        if (lane == 0) bar_expect(full(b), n * ua.box_rows * 128);
        __syncwarp();
        if (page >= 0)
          tma_box(smem + M::RING + b * M::TILE + col * (UT * 128) + bi * ua.box_rows * 128,
                  is_v ? &v_map : &k_map, full(b), col * 64, (s.h << a.shift) + (j & ((1 << a.shift) - 1)),
                  page);
      }
    }
    // every copy has landed before the CTA may end
    for (int b = 0; b < kRing && b < idx; ++b) {
      const int last = (idx - 1 - b) / kRing;  // use number of buffer b's last load
      bar_wait(full(b), last & 1, give_up, a.err);
    }
  } else if (warp == 9) {
    // ---- products
    int idx = 0, seg = 0, pv[2] = {0, 0}, edges = 0;
    const uint32_t id_s = instruction<T>(UT, false), id_o = instruction<T>(D, true);
    auto wait_load = [&](int place) -> uint32_t {
      const int i = idx + place, b = i % kRing;
      bar_wait(full(b), (i / kRing) & 1, give_up, a.err);
      return smem + M::RING + b * M::TILE;
    };
    auto scores = [&](int x, int q, uint32_t k) {
      if (lane == 0) {
        const uint32_t qa = smem + q * M::Q;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = (ks / 4) * (UT * 128) + (ks % 4) * 32;
          mma_ss(tmem + 128 * x, operand(qa + off, 16), operand(k + off, 16), id_s, ks > 0);
        }
        mma_commit(s_full(x));
      }
    };
    auto output = [&](int x, uint32_t v, bool first) {
      if (lane == 0) {
#pragma unroll
        for (int ks = 0; ks < UT / 16; ++ks)
          mma_ts(tmem + 256 + 128 * x, tmem + 128 * x + ks * 8, operand(v + ks * 2048, UT * 128), id_o,
                 !first || ks > 0);
      }
    };
    auto release = [&](int place) {
      if (lane == 0) mma_commit(empty((idx + place) % kRing));
    };
    auto finish = [&](int x) {
      if (lane == 0) mma_commit(o_full(x));
    };
    auto wait_p = [&](int x) {
      bar_wait(p_full(x), pv[x] & 1, give_up, a.err);
      ++pv[x];
      tc_fence_after();
    };
    auto wait_v = [&](bool two, int t) -> uint32_t {
      const uint32_t v = wait_load(v_place(two, t, s.count));
      if (s.edge<UT>(t, a.window)) {
        if (lane == 0) bar_arrive(v_in);
        bar_wait(v_ok, edges & 1, give_up, a.err);
        ++edges;
      }
      tc_fence_after();
      return v;
    };
    while (walk.next(a, s)) {
      const bool two = s.ntok * a.G > UM;
      bar_wait(q_full, seg & 1, give_up, a.err);
      ++seg;
      tc_fence_after();
      if (two) {
        uint32_t k = wait_load(0);
        scores(0, 0, k);
        scores(1, 1, k);
        release(0);
        for (int t = 0; t < s.count; ++t) {
          const uint32_t v = wait_v(true, t);
          const bool more = t + 1 < s.count;
          wait_p(0);
          output(0, v, t == 0);
          if (more) {
            k = wait_load(2 * t + 2);
            scores(0, 0, k);
          } else {
            finish(0);
          }
          wait_p(1);
          output(1, v, t == 0);
          release(2 * t + 1);
          if (more) {
            scores(1, 1, k);
            release(2 * t + 2);
          } else {
            finish(1);
          }
        }
      } else {
        for (int t = 0; t < 2 && t < s.count; ++t) {
          scores(t, 0, wait_load(t));
          release(t);
        }
        for (int t = 0; t < s.count; ++t) {
          const int x = t & 1;
          const uint32_t v = wait_v(false, t);
          wait_p(x);
          output(x, v, t < 2);
          const int place = v_place(false, t, s.count);
          release(place);
          if (t + 2 < s.count) {
            scores(x, 0, wait_load(place + 1));
            release(place + 1);
          } else {
            finish(x);
          }
        }
      }
      idx += 2 * s.count;
      __syncwarp();
    }
  } else if (warp >= 10) {
    // ---- V of tiles that some rows see in part
    // (warp 9 says when such a tile has come: these warps do not follow every load, and a
    // barrier's parity alone does not tell a phase from the one two before it)
    int idx = 0, seg = 0, edges = 0;
    const int me = tid - 320;              // 0 .. 63
    while (walk.next(a, s)) {
      const bool two = s.ntok * a.G > UM;
      if (me == 0) s_bad[seg & 1] = 0;
      __syncwarp();
      asm volatile("bar.sync 2, 64;" ::: "memory");
      for (int t = 0; t < s.count; ++t) {
        if (!s.edge<UT>(t, a.window)) continue;
        const int b = (idx + v_place(two, t, s.count)) % kRing;
        bar_wait(v_in, edges & 1, give_up, a.err);
        ++edges;
        unsigned char* v = smem_raw + (smem - smem_u32(smem_raw)) + M::RING + b * M::TILE;
        const int rows = min(UT, s.limit - s.j0 - t * UT);
        bool bad = false;
        for (int x = me; x < M::TILE / 16; x += 64) {
          const int row = (x / 8) % UT;    // 8 chunks a row, 64 columns a block
          uint4* p = reinterpret_cast<uint4*>(v + x * 16);
          if (row >= rows) {
            *p = make_uint4(0u, 0u, 0u, 0u);
            continue;
          }
          uint4 w = *p;
          uint32_t* e = reinterpret_cast<uint32_t*>(&w);
          bool here = false;
#pragma unroll
          for (int y = 0; y < 4; ++y)
            if (not_finite<T>(e[y])) {
              if (not_finite<T>(e[y] & 0xffffu)) e[y] &= 0xffff0000u;
              if (not_finite<T>(e[y] & 0xffff0000u)) e[y] &= 0xffffu;
              here = true;
            }
          if (here) {
            *p = w;
            bad = true;
          }
        }
        if (bad) s_bad[seg & 1] = 1;
        async_fence();
        bar_arrive(v_ok);
      }
      idx += 2 * s.count;
      __syncwarp();
      asm volatile("bar.sync 1, 320;" ::: "memory");  // with the softmax warps: s_bad stands
      ++seg;
    }
  } else {
    // ---- softmax: one row per thread
    const int x = warp >> 2, row = tid & (UM - 1);
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes, in bits 16 and up
    const uint32_t ts = tmem + lanes + 128 * x, to = tmem + lanes + 256 + 128 * x;
    int4 head = make_int4(0, 0, 0, 0);
    int tiles_done = 0, outs1 = 0, seg = 0;
    while (walk.next(a, s)) {
      const bool two = s.ntok * a.G > UM;
      const int rl = two ? x * UM + row : row;
      const bool mine = rl < s.ntok * a.G;
      const int lt = rl / a.G, gg = rl - lt * a.G;
      const int tok = mine ? s.tok0 + lt : -1;
      int q_pos = s.len + max(tok, 0);
      unsigned long long bits = 0;
      if (!s.chain && mine) {
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
      // this row of q
      if (two || x == 0) {
        unsigned char* q = smem_raw + (smem - smem_u32(smem_raw)) + x * M::Q + row * 128;
        const unsigned char* src =
            a.q + ((long long)(s.f + max(tok, 0)) * a.q_stride + (long long)(s.h * a.G + gg) * D) * 2;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          uint4 w = make_uint4(0u, 0u, 0u, 0u);
          if (mine) {
            if (ua.q_vec) {
              w = *reinterpret_cast<const uint4*>(src + c * 16);
            } else {
              const uint32_t* p = reinterpret_cast<const uint32_t*>(src + c * 16);
              w = make_uint4(p[0], p[1], p[2], p[3]);
            }
          }
          *reinterpret_cast<uint4*>(q + (c / 8) * (UT * 128) + (((c & 7) ^ (row & 7)) << 4)) = w;
        }
      }
      async_fence();
      bar_arrive(q_full);

      float m = -INFINITY, l = 0.f;
      const int my_tiles = two ? s.count : (s.count - x + 1) >> 1;
      for (int i = 0; i < my_tiles; ++i, ++tiles_done) {
        const int t = two ? i : 2 * i + x;
        const int j0 = s.j0 + t * UT;
        const bool edge = s.edge<UT>(t, a.window);
        const bool plain = !edge && a.cap_in == 0.f && !a.slopes;
        bar_wait(s_full(x), tiles_done & 1, give_up, a.err);
        __syncwarp();                      // (tensor-memory accesses are the whole warp's)
        tc_fence_after();
        float top = -INFINITY;
        uint32_t w[32];
        if (plain) {
#pragma unroll
          for (int c = 0; c < UT / 32; ++c) {
            tm_ld32(ts + c * 32, w);
            tm_wait_ld(w);
#pragma unroll
            for (int y = 0; y < 32; ++y) top = fmaxf(top, __uint_as_float(w[y]));
          }
          top *= a.score_log2;
        } else {
          // scores in units of log 2, capped, biased, -inf where not visible; back to their place
#pragma unroll 1
          for (int c = 0; c < UT / 32; ++c) {
            tm_ld32(ts + c * 32, w);
            tm_wait_ld(w);
            const int j = j0 + c * 32;
            uint32_t see = 0xffffffffu;
            if (edge) {
              // committed tokens (a chain: up to this one) below, the window's begin above
              const int below = s.len + (s.chain ? tok + 1 : 0) - j;
              see = below >= 32 ? 0xffffffffu : below <= 0 ? 0u : (1u << below) - 1;
              if (a.window > 0) {
                const int from = q_pos - a.window + 1 - j;
                see &= from <= 0 ? 0xffffffffu : from >= 32 ? 0u : 0xffffffffu << from;
              }
              const int d = j - s.len;     // draft of the chunk's first key
              if (!s.chain && d > -32 && d < 64)
                see |= d >= 0 ? (uint32_t)(bits >> d) : (uint32_t)(bits << -d);
            }
            float far = slope * (float)(q_pos - j);
            const bool drafts = a.slopes && !s.chain && j + 32 > s.len;
#pragma unroll
            for (int y = 0; y < 32; ++y) {
              float v = __uint_as_float(w[y]);
              if (a.cap_in != 0.f) v = a.cap_out * (1.f - __fdividef(2.f, ex2(v * a.cap_in) + 1.f));
              else v *= a.score_log2;
              if (a.slopes) {
                float bias = far - slope * (float)y;
                if (drafts && j + y >= s.len)
                  bias = slope * (float)(q_pos - s.len - s_depth[x][(j + y - s.len) & 63]);
                v -= bias;
              }
              v = (see >> y) & 1 ? v : -INFINITY;
              top = fmaxf(top, v);
              w[y] = __float_as_uint(v);
            }
            __syncwarp();
            tm_st32(ts + c * 32, w);
          }
          tm_wait_st();
        }
        // the maximum that the weights are relative to
        const bool grow = top > m + kLazy || (m == -INFINITY && top > m);
        const float now = grow ? top : m;
        const float use = now == -INFINITY ? 0.f : now;
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow ? ex2(m - use) : 1.f;
          l *= f;
          m = now;
          if (i > 0) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              tm_ld32(to + c * 32, w);
              tm_wait_ld(w);
#pragma unroll
              for (int y = 0; y < 32; ++y) w[y] = __float_as_uint(__uint_as_float(w[y]) * f);
              tm_st32(to + c * 32, w);
            }
          }
        }
        const float scale = plain ? a.score_log2 : 1.f, minus = SHIFT - use;
        float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
        for (int c = 0; c < UT / 32; ++c) {
          uint32_t p[16];
          tm_ld32(ts + c * 32, w);
          tm_wait_ld(w);
#pragma unroll
          for (int y = 0; y < 16; ++y) {
            const float p0 = ex2(fmaf(__uint_as_float(w[2 * y]), scale, minus));
            const float p1 = ex2(fmaf(__uint_as_float(w[2 * y + 1]), scale, minus));
            sum0 += p0;
            sum1 += p1;
            p[y] = pack<T>(p0, p1);
          }
          tm_st16(ts + c * 16, p);         // over scores that have been read
        }
        l += sum0 + sum1;
        tm_wait_st();
        tc_fence_before();
        bar_arrive(p_full(x));
      }

      // ---- the end of the piece
      // (stream 1 has no tile, and no output, in a piece of one tile with up to 128 rows)
      const bool both = two || s.count > 1;
      const bool other = !two && both && x == 0;  // stream 0 joins stream 1's output to its own
      if (x == 0) bar_wait(o_full(0), seg & 1, give_up, a.err);
      if (both && (x == 1 || other)) bar_wait(o_full(1), outs1 & 1, give_up, a.err);
      if (both) ++outs1;
      if (!two && x == 1) {
        s_m[row] = m;
        s_l[row] = l;
      }
      __syncwarp();
      tc_fence_after();
      asm volatile("bar.sync 1, 320;" ::: "memory");
      const bool bad = s_bad[seg & 1] != 0;
      if (two || x == 0) {
        const float m1 = other ? s_m[row] : -INFINITY, l1 = other ? s_l[row] : 0.f;
        const float top = fmaxf(m, m1), use = top == -INFINITY ? 0.f : top;
        const float f0 = ex2(m - use), f1 = ex2(m1 - use);
        const float sum = l * f0 + l1 * f1;
        const float inv = s.whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
        const long long at = (long long)(s.f + max(tok, 0)) * a.H * a.G + s.h * a.G + gg;
        const long long slot = ((long long)(2 * cta + (s.begins ? 1 : 0)) * (2 * UM) + rl);
        uint32_t w[32], w1[32];
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          tm_ld32(to + c * 32, w);
          tm_wait_ld(w);
          if (other) {
            tm_ld32(to + 128 + c * 32, w1);
            tm_wait_ld(w1);
          }
          float o[32];
#pragma unroll
          for (int y = 0; y < 32; ++y) {
            o[y] = f0 == 0.f ? 0.f : __uint_as_float(w[y]) * f0;
            if (other && f1 != 0.f) o[y] += __uint_as_float(w1[y]) * f1;
          }
          if (!mine) {
          } else if (s.whole) {
            uint4* dst = reinterpret_cast<uint4*>(a.out + (at * D + c * 32) * 2);
#pragma unroll
            for (int y = 0; y < 4; ++y)
              dst[y] = make_uint4(pack<T>(o[8 * y] * inv, o[8 * y + 1] * inv),
                                  pack<T>(o[8 * y + 2] * inv, o[8 * y + 3] * inv),
                                  pack<T>(o[8 * y + 4] * inv, o[8 * y + 5] * inv),
                                  pack<T>(o[8 * y + 6] * inv, o[8 * y + 7] * inv));
          } else {
            float4* dst = reinterpret_cast<float4*>(a.part + slot * D + c * 32);
#pragma unroll
            for (int y = 0; y < 8; ++y)
              dst[y] = make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
          }
          __syncwarp();
        }
        if (mine) {
          if (bad) {
            const unsigned char* q =
                a.q + ((long long)(s.f + tok) * a.q_stride + (long long)(s.h * a.G + gg) * D) * 2;
            if (s.whole)
              add_bad_values<T, T, D>(a, s, q, tok, q_pos, bits, slope, use - SHIFT, inv,
                                      reinterpret_cast<T*>(a.out) + at * D);
            else
              add_bad_values<T, float, D>(a, s, q, tok, q_pos, bits, slope, use - SHIFT, 1.f,
                                          a.part + slot * D);
          }
          if (!s.whole)
            *reinterpret_cast<float2*>(a.ml + slot * 2) = make_float2(top, sum);
          else if (a.lse)
            a.lse[at] = sum == 0.f ? -INFINITY : (top - SHIFT) * 0.6931471805599453f + logf(sum);
        }
      }
      if (!s.whole && s.begins) head = make_int4(s.last - cta + 1, s.f + s.tok0, s.h, s.ntok * a.G);
      tc_fence_before();
      __syncwarp();
      asm volatile("bar.sync 5, 256;" ::: "memory");  // both outputs are read
      ++seg;
    }
    if (tid == 0) a.head[cta] = head;
  }
  griddep_launch();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
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

// Pages as [num_pages][H * page][D], in boxes of 64 columns and min(page, 128) tokens.
bool encode_pages(CUtensorMap* map, const unsigned char* pages, const TreeArgs& a, int dtype, int D, int box) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.H << a.shift, (cuuint64_t)a.num_pages};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, ((cuuint64_t)a.H << a.shift) * D * 2};
  const cuuint32_t size[3] = {64, (cuuint32_t)box, 1}, step[3] = {1, 1, 1};
  return encode(map, dtype == AVSG_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                const_cast<unsigned char*>(pages), dims, strides, size, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D>
cudaError_t launch_umma(const TreeArgs& a, int dtype, int dev, cudaStream_t st) {
  static SmemLimit limit;
  auto kernel = tree_umma_kernel<T, D>;
  cudaError_t e = limit.raise(reinterpret_cast<const void*>(kernel), Mem<D>::SMEM, dev);
  if (e != cudaSuccess) return e;
  UmmaArgs u{};
  u.t = a;
  u.box_rows = (1 << a.shift) < UT ? 1 << a.shift : UT;
  u.q_vec = reinterpret_cast<uintptr_t>(a.q) % 16 == 0 && a.q_stride % 8 == 0;
  CUtensorMap k_map, v_map;
  if (!encode_pages(&k_map, a.k, a, dtype, D, u.box_rows) || !encode_pages(&v_map, a.v, a, dtype, D, u.box_rows))
    return cudaErrorInvalidValue;
  e = launch_pdl(kernel, dim3(a.ctas), dim3(kUmmaThreads), Mem<D>::SMEM, st, u, k_map, v_map);
  return e != cudaSuccess ? e : launch_merge<T, D>(a, 2 * UM, st);
}

}  // namespace
}  // namespace tree

cudaError_t launch_tree_umma(const TreeArgs& a, int dtype, int D, int dev, cudaStream_t st) {
  if (dtype == AVSG_BF16)
    return D == 64 ? tree::launch_umma<__nv_bfloat16, 64>(a, dtype, dev, st)
                   : tree::launch_umma<__nv_bfloat16, 128>(a, dtype, dev, st);
  return D == 64 ? tree::launch_umma<__half, 64>(a, dtype, dev, st)
                 : tree::launch_umma<__half, 128>(a, dtype, dev, st);
}
}  // namespace avsg
