// Tree attention over a paged cache: the kernel for few rows per kv-head and
// what it shares with its host side.
//
//   s = scale q.k;  s = cap tanh(s / cap);  s -= slope_h (pos_q - pos_k)
//   out = sum_visible softmax(s) v,  lse = log sum_visible exp(s)
//
// New token i of a request sees the request's committed tokens and, of its
// new ones, those whose bit its mask word has (no masks, or more than 64 new
// tokens: the tokens up to itself), all of them less than `window` positions
// away where a window is given.
//
// What bounds it: the bytes of K and V, read once per (request, kv-head) for
// all of its n * G query rows.  So
// * the rows of a request and kv-head form the M of the tensor-core products
//   (an m-tile holds whole tokens: up to MT / G of them);
// * the tiles of 64 keys of all (request, kv-head, m-tile) units are one list,
//   and every CTA takes an equal contiguous share of it whatever the lengths
//   are (they are known on the device only): one long request among short
//   ones, or a single one, still uses every SM.  A unit that crosses CTAs
//   leaves partials (at most two per CTA: the unit that ends in its share and
//   the one that begins in it), which tree_merge_kernel joins;
// * K and V tiles stream through shared memory by 16-byte cp.async, their
//   page ids looked up one tile ahead; rows past the end are zero-filled;
// * scores, the running maximum and sum, and the output stay in registers
//   (fp32); P is rounded to the cache's type for the second product, half a
//   step and the only rounding before the last one (avsg_tree_umma.cuh).
// Measured (GB300, 6.78 TB/s copy): 64 requests x 8 kv-heads of 1000 tokens,
// one token each, 4 query heads of 128: 57 us, 4.6 TB/s; 8 x 8 of 4000: 34 us;
// one request of 4096 tokens and one head: 11 us with its merge, of which
// the bytes need 0.3 (two dependent chains of loads, lengths - tables - rows
// and head - partials, and two launches).  Heads of 256 (8 x 8 of 16000, pages
// of 4): 271 us at one token (3.9 TB/s), 314 us at 64 rows.  With more rows
// mma.sync's rate bounds it (16 x 8 units of 8192 tokens, 256 rows, heads of
// 128, pages of 1 or 4: 580 us, 134 on tcgen05 with pages of 16).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <limits.h>
#include <math.h>

#include "avsg_paged.cuh"

namespace avsg {

struct TreeArgs {
  const unsigned char* k;        // the layer's pages
  const unsigned char* v;
  const int32_t* tables;
  const int32_t* len;
  const int32_t* first;
  const unsigned long long* mask;
  const float* slopes;
  const unsigned char* q;
  unsigned char* out;
  float* lse;
  int4* head;                    // [ctas] {pieces, first token, kv-head, rows} of the unit that
                                 // begins in the CTA's share and ends in another (pieces 0: none)
  float* ml;                     // [2 * ctas][MT][2] running maximum (log2) and sum of a partial
  float* partial;                // [2 * ctas][MT][D] its output, not divided by the sum
  DevErr* err;
  long long q_stride;            // values between tokens of q
  int R, H, G, T;
  int shift, max_pages, num_pages, max_new;
  int tpm;                       // tokens per m-tile
  int window;
  int ctas, min_tiles;
  // What the beginning and the end of a unit cost a CTA (its q rows, the first scores, the
  // output), in tiles: the shares count it, or a CTA with many short units would finish late.
  int begin;
  float score_log2;              // scale * log2(e)
  float cap_in, cap_out;         // 2 log2(e) scale / cap, cap * log2(e); cap_in 0: no cap
  // Attention over common prefixes (avsg_prefix_api.cu).  part 0: the keys of a group's prefix,
  // for the new tokens of all its members; 1: every request's own keys.  No part writes the
  // output of a request that has a prefix.
  int part;
  // How the SMs are divided between the parts, by what their lists cost (in hundredths of an SM's
  // microsecond; nothing but the time depends on it).
  struct Cost {
    int keys, tpm;               // keys of a tile, tokens per m-tile
    int begin;                   // of a unit's beginning and end
    int tile, small;             // of a tile, with more than half an m-tile's rows and with fewer
    int per_sm;                  // CTAs
  } cost[2];
  // Places of a tile in the list, of m-tiles with up to small_rows rows and with more.
  int w_small, w_full, small_rows;
  int sms;
  int lead;                      // part 0's begin and end beyond part 1's, in hundredths of a microsecond
  int places;                    // entries of token and request
  const int32_t* shared;         // [R] tokens of the prefix
  const int32_t* group_first;    // [R + 1] a leader's first place
  const int32_t* token;          // [places] the token in a place, and its request
  const int32_t* request;
  int4* unit;                    // [T][H] {CTA of the unit's begin, pieces, number in the unit, tokens of the
                                 // prefix}; pieces 0: a row of `rows`, -1: the output is written; of part 0
                                 // {and the group's leader from bit 16 on, .., .., place of the unit's first}
  float* rows;                   // [T][H][G][D] outputs of units that lie in one share
  float* rows_ml;                // [T][H][G][2]
};

// Splits of the row count per m-tile, and launchers of one head width each.
cudaError_t launch_tree_d64(const TreeArgs& a, int dtype, int wm, int dev, cudaStream_t st);
cudaError_t launch_tree_d128(const TreeArgs& a, int dtype, int wm, int dev, cudaStream_t st);
cudaError_t launch_tree_d256(const TreeArgs& a, int dtype, int wm, int dev, cudaStream_t st);
// Pages of at least 8 tokens, 256 rows per m-tile, 128 for D of 256 (avsg_tree_umma.cuh).
cudaError_t launch_tree_umma(const TreeArgs& a, int dtype, int D, int dev, cudaStream_t st);
// One part of an attention over common prefixes, without the joining of its pieces.
cudaError_t launch_prefix_part(const TreeArgs& a, int dtype, int D, int wm, int dev, cudaStream_t st);
cudaError_t launch_prefix_umma(const TreeArgs& a, int dtype, int D, int dev, cudaStream_t st);

namespace tree {

constexpr int KT = 64;           // keys per tile
// fp16 weights are held times 2^6: the smallest normal one is then 2^-20 of
// the largest, not 2^-14; with the 2^8 that a weight may reach relative to a
// maximum not yet followed (avsg_tree_umma.cuh) it is far from the type's end.
constexpr float kHalfShift = 6.f;

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
// 16 bytes, or zeros when bytes is 0 (the source is then not read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
template <typename T>
__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <typename T>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&x);
  } else {
    const __half2 x = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&x);
  }
}
template <typename T>
__device__ __forceinline__ float2 unpack(uint32_t x) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
}
// Whether one of the two values is an infinity or a NaN.
template <typename T>
__device__ __forceinline__ bool not_finite(uint32_t x) {
  constexpr uint32_t e = std::is_same<T, __nv_bfloat16>::value ? 0x7f80u : 0x7c00u;
  return (x & e) == e || ((x >> 16) & e) == e;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// sum of floor((a i + b) / m) over i < n (the Euclid-like recursion on lattice points)
__device__ __forceinline__ long long floor_sum(long long n, long long m, long long a, long long b) {
  long long sum = 0;
  while (n > 0) {
    sum += n * (n - 1) / 2 * (a / m) + n * (b / m);
    a %= m;
    b %= m;
    const long long top = a * n + b;
    if (top < m) break;
    n = top / m;
    b = top % m;
    const long long x = m;
    m = a;
    a = x;
  }
  return sum;
}

// cap tanh(t) for t = x / cap within a half: t (1 + c1 t^2 + c2 t^4 + c3 t^6), fitted to the least
// largest error (2e-7; near 0 the relative error vanishes, so that a cap far above the scores
// leaves them as they are).  Elsewhere cap (1 - 2 / (exp(2 t) + 1)), whose error is a rounding of the
// cap.
constexpr float kCapNear = 0.5f, kCap1 = -0.33326461f, kCap2 = 0.13185862f, kCap3 = -0.04422929f;
constexpr float kCapUnit = 0.34657359028f;  // t = x cap_in log(2) / 2
// The largest |t| of a row's scores that takes the polynomial; far: the largest |t| that the row sees
// among the keys at hand.  All of them or none: a row then depends on nothing but what it sees, and
// where a warp's rows agree one of the two is all that is computed.  A cap so large that its rounding
// (cap 2^-22, in units of log 2) would show beside that of a 16-bit weight (2^-9) decides score by score.
constexpr float kCapLarge = 512.f;
__device__ __forceinline__ float cap_polynomial_reach(float far, float cap_out) {
  return far <= kCapNear || cap_out > kCapLarge ? kCapNear : -1.f;
}

// One request as the kernels see it (or one group, whose keys are its
// prefix).  A request with a bad length is latched and has no work.  Its rows
// are cut into mts units of tpm tokens per kv-head.
template <bool SHARED>
struct Fresh {};
template <>
struct Fresh<true> {
  int fresh;                               // new tokens that are keys
  int w, w_last;                           // places of a tile, of the last m-tile's
};
template <int KT, bool SHARED>
struct Req : Fresh<SHARED> {
  int len, n, f, lo, mts, begin;
  bool chain;

  __device__ int new_keys() const {
    if constexpr (SHARED) return this->fresh;
    else return n;
  }

  // Places of unit mt in the list: `begin` for its beginning, then its
  // tiles, counted from key lo, up to the last key that a row may see.
  __device__ int tiles(int mt, int tpm) const {
    return (len - lo + (chain ? min(n, (mt + 1) * tpm) : new_keys()) + KT - 1) / KT;
  }
  __device__ int weight(int mt) const {
    if constexpr (SHARED) return mt == mts - 1 ? this->w_last : this->w;
    else return 1;
  }
  __device__ int places(int mt, int tpm) const { return begin + tiles(mt, tpm) * weight(mt); }
  // Places of the units before mt.
  __device__ long long before(int mt, int tpm) const {
    if (mt == 0) return 0;
    if constexpr (SHARED) {
      if (!chain) return (long long)mt * (begin + tiles(0, tpm) * this->w);
    }
    if (!chain) return (long long)mt * places(0, tpm);
    return (long long)mt * begin + floor_sum(mt, KT, tpm, (long long)(len - lo) + tpm + KT - 1);
  }
  __device__ long long per_head(int tpm) const {
    return n ? before(mts - 1, tpm) + places(mts - 1, tpm) : 0;
  }
};
template <int KT, bool SHARED>
__device__ __forceinline__ Req<KT, SHARED> load_req(const TreeArgs& a, int r) {
  Req<KT, SHARED> q;
  if constexpr (SHARED) {
    const int len = a.len[r], common = a.shared[r], page_mask = (1 << a.shift) - 1;
    if (a.part == 0) {
      q.f = a.group_first[r];
      const int end = a.group_first[r + 1];
      q.len = common;
      q.n = end - q.f;
      q.fresh = 0;
      q.begin = a.begin;
      q.chain = false;
      if (q.f < 0 || end < q.f || end > a.places || common < 0 || common > len || (common & page_mask) != 0 ||
          (common >> a.shift) > a.max_pages) {
        raise_error(a.err, AVSG_ERR_BAD_SELECTION, r, -1);
        q.n = 0;
      }
      if (common == 0) q.n = 0;
      // no member is shorter than its prefix: what lies before that one's window nobody sees
      q.lo = a.window > 0 ? max(0, min(common - a.window + 1, common - 1)) & ~(KT - 1) : 0;
      q.mts = (q.n + a.tpm - 1) / a.tpm;
      q.w = a.w_full;
      q.w_last = (q.n - (q.mts - 1) * a.tpm) * a.G <= a.small_rows ? a.w_small : a.w_full;
      return q;
    }
  }
  q.f = a.first[r];
  const int end = a.first[r + 1];
  q.len = a.len[r];
  q.n = end - q.f;
  q.begin = a.begin;
  int code = 0;
  if (q.f < 0 || end < q.f || end > a.T || q.len < 0) code = AVSG_ERR_BAD_SELECTION;
  else if (q.n > a.max_new ||
           (((long long)q.len + q.n + (1 << a.shift) - 1) >> a.shift) > a.max_pages)
    code = AVSG_ERR_CAPACITY;
  if (code) {
    raise_error(a.err, code, r, -1);
    q.n = q.len = 0;
  }
  q.chain = !a.mask || q.n > kMaxDrafts;
  q.lo = a.window > 0 && q.len >= a.window ? (q.len - a.window + 1) & ~(KT - 1) : 0;
  if constexpr (SHARED) {                  // from the prefix on, in tiles counted from there
    const int common = a.shared[r];
    if (common < 0 || common > q.len || (common & ((1 << a.shift) - 1)) != 0) {
      if (q.n) raise_error(a.err, AVSG_ERR_BAD_SELECTION, r, -1);
      q.n = q.len = q.lo = 0;
    } else {
      q.lo = common + (a.window > 0 ? max(0, q.len - a.window + 1 - common) & ~(KT - 1) : 0);
    }
    q.fresh = q.n;
    q.w = q.w_last = 1;                    // (a chain's sums know one weight)
  }
  q.mts = (q.n + a.tpm - 1) / a.tpm;
  return q;
}

// A CTA's piece of a unit.
struct Piece {
  int r, h, f, len, n;                     // request
  int tok0, ntok;                          // the unit's tokens
  int j0, count;                           // first key of the first tile; tiles
  // Keys that some row may see, keys that every row sees (the window aside),
  // the largest position a row can have.
  int limit, all_see, far_pos;
  int last;                                // CTA of the unit's last tile
  bool chain, whole, begins;               // begins: the unit's first tile is in this piece

  // Whether some row sees only part of tile t.
  template <int KT>
  __device__ bool edge(int t, int window) const {
    const int j = j0 + t * KT;
    return j + KT > all_see || (window > 0 && far_pos - j >= window);
  }
};

// What part `part` of an attention over prefixes costs in all of request (or group) r's units of one kv-head.
// (This and the next one run on the host too, for arrays there: so they are tested.)
__host__ __device__ __forceinline__ float part_cost(const TreeArgs& a, int part, int r) {
  const TreeArgs::Cost& c = a.cost[part];
  const int common = max(a.shared[r], 0);
  int n, keys;
  if (part == 0) {
    n = common > 0 ? max(a.group_first[r + 1] - a.group_first[r], 0) : 0;
    keys = min(a.window > 0 ? min(common, a.window) : common, INT_MAX - 1024);
  } else {
    n = max(a.first[r + 1] - a.first[r], 0);
    keys = max(a.len[r] - common, 0);
    if (a.window > 0) keys = min(keys, a.window);
    keys = min(keys, INT_MAX - 1024) + min(n, kMaxDrafts);
  }
  const int full = n / c.tpm, rest = n - full * c.tpm;
  const float tiles = (float)((keys + c.keys - 1) / c.keys);
  return (float)c.begin * (float)(full + (rest > 0)) +
         tiles * ((float)full * (float)c.tile + (float)(rest == 0 ? 0 : 2 * rest > c.tpm ? c.tile : c.small));
}

// SMs of part 0: the fewest with which it ends no later than part 1 on the others, `lead` before it.
__host__ __device__ __forceinline__ int first_sms(const TreeArgs& a, float c0, float c1) {
  if (c0 == 0.f) return 0;
  if (c1 == 0.f) return a.sms;
  // the positive root k of  c0 / k + lead = c1 / (sms - k)  (short calls need no room for the lead)
  const float n = (float)a.sms, lead = fminf((float)a.lead, 0.5f * (c0 + c1) / n), b = c0 + c1 - lead * n;
  const float up = 2.f * c0 * n, down = b + sqrtf(b * b + 4.f * lead * c0 * n);
#ifdef __CUDA_ARCH__
  const float k = __fdividef(up, down);
#else
  const float k = up / down;
#endif
  return min(max((int)ceilf(k), 1), a.sms - 1);
}

// Where a CTA's share begins, found by one of its threads.
template <int KT, bool SHARED>
struct Begin {
  Req<KT, SHARED> q;
  int r;
  long long before;                        // list position of the request's first place
};

// The CTA's share of the list: every thread walks it alike.
template <int KT, bool SHARED>
struct Walk {
  Req<KT, SHARED> q;
  long long at, end, W;                    // list positions, length of the list
  int C;                                   // CTAs with a share
  int r, h, mt, ta;                        // ta: the next place of the unit

  // Finds the share (all threads of the block; barriers inside).  False: no work, or an
  // error latched before (its word and the lengths are read side by side).
  __device__ bool begin(const TreeArgs& a, long long* s_warp, Begin<KT, SHARED>* s_begin) {
    const bool latched = load_err(a.err) != 0;
    const int per = (a.R + blockDim.x - 1) / blockDim.x;
    const int r0 = min(a.R, (int)threadIdx.x * per), r1 = min(a.R, r0 + per);
    float2 c = make_float2(0.f, 0.f);
    if constexpr (SHARED)
      for (int i = r0; i < r1; ++i) {      // (first, so that all their loads are on the way together)
        c.x += part_cost(a, 0, i);
        c.y += part_cost(a, 1, i);
      }
    long long mine = 0;
    for (int i = r0; i < r1; ++i) mine += load_req<KT, SHARED>(a, i).per_head(a.tpm) * a.H;
    int ctas = a.ctas;
    if constexpr (SHARED) {
      // The parts run side by side, each on its share of the SMs: the CTAs behind it have no work.
#pragma unroll
      for (int d = 16; d; d >>= 1) {
        c.x += __shfl_xor_sync(0xffffffffu, c.x, d);
        c.y += __shfl_xor_sync(0xffffffffu, c.y, d);
      }
      float2* s_cost = reinterpret_cast<float2*>(s_warp);
      if ((threadIdx.x & 31) == 0) s_cost[threadIdx.x >> 5] = c;
      __syncthreads();
      c = make_float2(0.f, 0.f);
      for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
        c.x += s_cost[w].x;
        c.y += s_cost[w].y;
      }
      __syncthreads();
      int first = first_sms(a, c.x * a.H, c.y * a.H);
      // Part 0 as a whole number of CTAs per kv-head, where that costs little: one group's units are alike,
      // and a CTA with a piece of two pays for two beginnings and ends (63 us instead of 56).
      const int near = max(1, (first + a.H / 2) / a.H) * a.H;
      if (c.x > 0.f && c.y > 0.f && near < a.sms && abs(near - first) <= first / 12) first = near;
      ctas = max(1, a.part == 0 ? first * a.cost[0].per_sm : (a.sms - first) * a.cost[1].per_sm);
    }
    long long before = block_exclusive(mine, s_warp, &W);
    const long long fit = W / a.min_tiles;
    C = fit < 1 ? 1 : fit < ctas ? (int)fit : ctas;
    const int cta = blockIdx.x;
    if (__syncthreads_or(latched) || W == 0 || cta >= C) return false;  // (alike in the whole block)
    at = cta * W / C;
    end = (cta + 1) * W / C;
    if (before <= at && at < before + mine)
      for (int i = r0; i < r1; ++i) {
        const Req<KT, SHARED> req = load_req<KT, SHARED>(a, i);
        const long long w = req.per_head(a.tpm) * a.H;
        if (at < before + w) {
          s_begin->q = req;
          s_begin->r = i;
          s_begin->before = before;
          break;
        }
        before += w;
      }
    __syncthreads();
    r = s_begin->r;
    q = s_begin->q;
    const long long head = q.per_head(a.tpm), off = at - s_begin->before;
    h = (int)(off / head);
    const long long rest = off - h * head;
    int lo = 0, hi = q.mts;                // before(lo) <= rest < before(hi)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (q.before(mid, a.tpm) <= rest) lo = mid;
      else hi = mid;
    }
    mt = lo;
    ta = (int)(rest - q.before(lo, a.tpm));
    return true;
  }

  // The next piece with work; false at the end of the share.
  __device__ bool next(const TreeArgs& a, Piece& p) {
    while (at < end) {
      const int all = q.places(mt, a.tpm);
      const int t0 = ta, t1 = (int)min((long long)all, ta + (end - at));
      const int weight = q.weight(mt);
      const long long unit_end = at - ta + all;
      const int lo = q.lo;                 // (q may move on below)
      p.r = r;
      p.h = h;
      p.f = q.f;
      p.len = q.len;
      p.n = q.n;
      p.chain = q.chain;
      p.tok0 = mt * a.tpm;
      p.ntok = min(a.tpm, q.n - p.tok0);
      p.limit = q.len + (q.chain ? p.tok0 + p.ntok : q.n);
      p.all_see = q.len + (q.chain ? p.tok0 + 1 : 0);
      // (a position is the number of a word's bits, those past the request's tokens too)
      p.far_pos = q.len + (q.chain ? p.tok0 + p.ntok : kMaxDrafts) - 1;
      if constexpr (SHARED) {
        if (a.part == 0) {                 // no new token is a key; rows lie anywhere behind
          p.n = 0;
          p.limit = q.len;
          p.far_pos = INT_MAX - 1024;  // (room for sums)
        }
      }
      // tiles that lie before the window of every row have no work
      int skip = a.begin;
      if (a.window > 0 && q.chain)
        skip += max(0, (q.len + p.tok0 - a.window + 1 - q.lo) / KT);
      at += t1 - t0;
      ta = t1;
      if (t1 == all) {
        ta = 0;
        if (++mt == q.mts) {
          mt = 0;
          if (++h == a.H) {
            h = 0;
            if (at < end) {
              do q = load_req<KT, SHARED>(a, ++r); // (one with work follows: at < end <= W)
              while (q.n == 0 && r + 1 < a.R);
            }
          }
        }
      }
      if constexpr (SHARED) {
        // a tile is the CTA's in whose share its first place lies (a share has at least a tile's places)
        auto up = [&](int places) { return max(0, places - a.begin + weight - 1) / weight; };
        const int first = up(t0), from = max(first, skip - a.begin), to = up(t1);
        if (from >= to) continue;
        p.j0 = lo + from * KT;
        p.count = to - from;
        p.begins = first <= skip - a.begin;
        p.whole = p.begins && to == up(all);
        p.last = (int)(((unit_end - weight + 1) * C - 1) / W);
        return true;
      }
      const int from = max(t0, skip);
      if (from >= t1) continue;
      p.j0 = lo + (from - a.begin) * KT;
      p.count = t1 - from;
      p.begins = t0 <= skip;
      p.whole = p.begins && t1 == all;
      p.last = (int)((unit_end * C - 1) / W);
      return true;
    }
    return false;
  }
};

// The token in a row of a piece.
template <bool SHARED>
__device__ __forceinline__ int token_of(const TreeArgs& a, const Piece& p, int tok) {
  if constexpr (SHARED) {
    if (a.part == 0) {
      const int t = a.token[p.f + tok];
      if (t >= 0 && t < a.T) return t;
      raise_error(a.err, AVSG_ERR_BAD_SELECTION, p.r, p.f + tok);
      return 0;
    }
  }
  return p.f + tok;
}
// The position of that token where it is another request's (part 0), wanted for biases and windows.
__device__ __forceinline__ int member_position(const TreeArgs& a, const Piece& p, int tok, int t) {
  const int r = a.request[p.f + tok];
  if (r < 0 || r >= a.R) {
    raise_error(a.err, AVSG_ERR_BAD_SELECTION, p.r, p.f + tok);
    return 0;
  }
  const int f = a.first[r];
  const unsigned long long w = a.mask && a.first[r + 1] - f <= kMaxDrafts ? a.mask[t] : 0;
  return a.len[r] + (w ? __popcll(w) - 1 : t - f);
}
// (SHARED) Notes where the partial outputs of a unit's tokens lie; tid of `threads` threads.  (All but a
// token's number is the unit's: with its place in the loop a step of draft trees took 332 us instead of 302.)
__device__ __forceinline__ void note_unit(const TreeArgs& a, const Piece& p, int cta, int tid, int threads) {
  static_assert(kMaxPagedRequests <= 1 << 15, "a leader and a CTA share a word");
  const int prefix = a.part == 1 ? a.shared[p.r] : 0;
  const int pieces = !p.whole ? p.last - cta + 1 : a.part == 1 && !prefix ? -1 : 0;
  const int from = a.part == 0 ? p.r << 16 | cta : cta, more = a.part == 0 ? p.f + p.tok0 : prefix;
  for (int x = tid; x < p.ntok; x += threads)
    a.unit[(long long)token_of<true>(a, p, p.tok0 + x) * a.H + p.h] = make_int4(from, pieces, x, more);
}

template <typename T_, int D_, int WM_, bool SHARED_>
struct Shape {
  using T = T_;
  static constexpr bool SHARED = SHARED_;
  // Heads of 256 values leave room for one CTA per SM: eight warps, where each can have 16 keys.
  static constexpr int D = D_, WM = WM_, WARPS = D_ == 256 && WM_ > 1 ? 8 : 4, WK = WARPS / WM_, MT = 16 * WM_;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int NK = KT / WK;                 // keys of a tile per warp
  static constexpr int STAGES = D == 64 ? 4 : 3;
  static constexpr int CTAS_PER_SM = D == 256 ? 1 : 2;
  static constexpr bool Q_SMEM = D == 256;           // its fragments do not fit the registers
  static constexpr int TILE = KT * D * 2;            // bytes of a K or V tile
  static constexpr int RING = STAGES * KT * 8;       // row offsets of the staged tiles
  static constexpr int OP = D + 8;                   // floats per output row in shared memory
  static constexpr int SMEM = STAGES * 2 * TILE + RING + (Q_SMEM ? MT * D * 2 : 0);
  static_assert(WK * MT * OP * 4 <= STAGES * 2 * TILE, "the outputs overlay the stages");
  static_assert(MT * KT * 2 <= TILE, "P overlays a K tile");
};

template <class SH>
__global__ void __launch_bounds__(SH::THREADS, SH::CTAS_PER_SM) tree_attn_kernel(TreeArgs a) {
  using T = typename SH::T;
  constexpr int kThreads = SH::THREADS;
  constexpr int D = SH::D, WM = SH::WM, WK = SH::WK, MT = SH::MT, NK = SH::NK, S = SH::STAGES;
  constexpr int CPR = D / 8;                         // 16-byte chunks per row
  constexpr bool HALF = std::is_same<T, __half>::value, SHARED = SH::SHARED;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long s_warp[kThreads / 32];
  __shared__ Begin<KT, SHARED> s_begin;
  __shared__ float s_m[WK][MT], s_l[WK][MT];
  __shared__ int s_depth[kMaxDrafts];
  long long* s_row = reinterpret_cast<long long*>(smem + S * 2 * SH::TILE);
  unsigned char* s_q = smem + S * 2 * SH::TILE + SH::RING;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wm = warp % WM, wk = warp / WM;
  const int g = lane >> 2, c = lane & 3;
  const int cta = blockIdx.x;
  int4 head = make_int4(0, 0, 0, 0);

  // (part 1 of an attention over prefixes may run beside part 0, which it waits for at its end)
  if (!SHARED || a.part == 0) griddep_wait();
  if (SHARED) griddep_launch();
  Walk<KT, SHARED> walk;
  if (!walk.begin(a, s_warp, &s_begin)) {
    if (SHARED) griddep_wait();
    else if (tid == 0) a.head[cta] = head;
    return;
  }

  if (!SHARED) griddep_launch();                     // (the merge waits for the whole grid anyway)
  Piece pc;
  while (walk.next(a, pc)) {
    const int rows = pc.ntok * a.G, count = pc.count, h = pc.h;
    const int32_t* table = a.tables + (size_t)pc.r * a.max_pages;
    // Row of key (tid % KT) of the i-th tile, in two steps: its page, and a tile later, when the page has
    // come, the row (a check right behind the load holds the tile up for as long as the load takes).
    constexpr int32_t kNoPage = INT_MIN;
    auto find_page = [&](int i) -> int32_t {
      const int j = pc.j0 + i * KT + (tid & (KT - 1));
      return i < count && j < pc.limit ? __ldg(table + (j >> a.shift)) : kNoPage;
    };
    auto row_of = [&](int i, int32_t page) -> long long {
      const int j = pc.j0 + i * KT + (tid & (KT - 1));
      if (page < 0 || page >= a.num_pages) {
        if (i < count && j < pc.limit) raise_error(a.err, AVSG_ERR_BAD_SELECTION, pc.r, j);
        return -1;
      }
      return (((long long)page * a.H + h) << a.shift) + (j & ((1 << a.shift) - 1));
    };
    auto issue = [&](int st) {
      const uint32_t kst = smem_u32(smem + st * 2 * SH::TILE);
#pragma unroll
      for (int it = 0; it < KT * CPR / kThreads; ++it) {
        const int x = it * kThreads + tid, row = x / CPR, ch = x % CPR;
        const long long src = s_row[st * KT + row];
        const uint32_t dst = kst + row * (D * 2) + ((ch ^ (row & 7)) << 4);
        const long long off = src < 0 ? 0 : src * (D * 2) + ch * 16;
        const int bytes = src < 0 ? 0 : 16;
        cp_async16(dst, a.k + off, bytes);
        cp_async16(dst + SH::TILE, a.v + off, bytes);
      }
    };

    __syncthreads();                                 // the stages are free (earlier segment)
    if (tid < KT) {
      int32_t page[S - 1];
#pragma unroll
      for (int i = 0; i < S - 1; ++i) page[i] = find_page(i);
#pragma unroll
      for (int i = 0; i < S - 1; ++i) s_row[i * KT + tid] = row_of(i, page[i]);
    }
    if (!pc.chain && tid >= KT && tid - KT < pc.n) {
      const unsigned long long w = a.mask[pc.f + tid - KT];
      s_depth[tid - KT] = w ? __popcll(w) - 1 : tid - KT;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
      if (i < count) issue(i);
      cp_commit();
    }
    int32_t next_page = tid < KT ? find_page(S - 1) : kNoPage;

    // The two rows of this thread.
    int tok[2], q_pos[2];
    unsigned long long bits[2] = {0, 0};
    float slope[2] = {0.f, 0.f};
    const unsigned char* q_row[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int rl = wm * 16 + g + 8 * x;
      const int lt = rl / a.G, gg = rl - lt * a.G;
      const bool ok = rl < rows;
      tok[x] = ok ? pc.tok0 + lt : -1;                  // -1: a padding row, sees no new token
      q_pos[x] = pc.len + max(tok[x], 0);
      int token = pc.f + tok[x];
      if (SHARED && a.part == 0) {
        if (ok) token = token_of<SHARED>(a, pc, tok[x]);
        if (ok && (a.slopes || a.window > 0)) q_pos[x] = member_position(a, pc, tok[x], token);
      } else if (!pc.chain && ok) {
        bits[x] = a.mask[pc.f + tok[x]];
        if (bits[x]) q_pos[x] = pc.len + __popcll(bits[x]) - 1;
      }
      if (a.slopes && ok) slope[x] = a.slopes[h * a.G + gg] * 1.4426950408889634f;
      q_row[x] = ok ? a.q + ((long long)token * a.q_stride + (long long)(h * a.G + gg) * D) * 2
                    : nullptr;
    }
    uint32_t qf[SH::Q_SMEM ? 1 : D / 16][4];
    if constexpr (!SH::Q_SMEM) {
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          qf[ks][x] = q_row[x & 1] ? *reinterpret_cast<const uint32_t*>(
                                         q_row[x & 1] + (ks * 16 + 2 * c + 8 * (x >> 1)) * 2)
                                   : 0u;
    } else {
      // fragments of this warp's 16 rows, [k-step][lane][4], written and read by the same thread
      if (wk == 0) {
#pragma unroll 4
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t f[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            f[x] = q_row[x & 1] ? *reinterpret_cast<const uint32_t*>(
                                      q_row[x & 1] + (ks * 16 + 2 * c + 8 * (x >> 1)) * 2)
                                : 0u;
          *reinterpret_cast<uint4*>(s_q + ((wm * (D / 16) + ks) * 32 + lane) * 16) =
              make_uint4(f[0], f[1], f[2], f[3]);
        }
      }
    }

    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float acc[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int x = 0; x < 4; ++x) acc[i][x] = 0.f;

    for (int i = 0; i < count; ++i) {
      const int st = i % S;
      if (tid < KT) s_row[((i + S - 1) % S) * KT + tid] = row_of(i + S - 1, next_page);
      cp_wait<S - 2>();
      __syncthreads();                               // tile i is here; stage (i - 1) % S is free
      if (i + S - 1 < count) issue((i + S - 1) % S);
      cp_commit();
      if (tid < KT) next_page = find_page(i + S);

      unsigned char* kst = smem + st * 2 * SH::TILE;
      const uint32_t ka = smem_u32(kst), va = ka + SH::TILE;
      float s[NK / 8][4];
#pragma unroll
      for (int x = 0; x < NK / 8; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) s[x][y] = 0.f;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t qa[4];
        if constexpr (SH::Q_SMEM) {
          const uint4 f = *reinterpret_cast<const uint4*>(s_q + ((wm * (D / 16) + ks) * 32 + lane) * 16);
          qa[0] = f.x; qa[1] = f.y; qa[2] = f.z; qa[3] = f.w;
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x) qa[x] = qf[ks][x];
        }
#pragma unroll
        for (int nt = 0; nt < NK / 16; ++nt) {
          const int row = wk * NK + nt * 16 + (lane & 7) + ((lane >> 4) << 3);
          const int ch = ks * 2 + ((lane >> 3) & 1);
          uint32_t b[4];
          ldsm4(ka + row * (D * 2) + ((ch ^ (row & 7)) << 4), b);
          mma<T>(s[2 * nt], qa, b[0], b[1]);
          mma<T>(s[2 * nt + 1], qa, b[2], b[3]);
        }
      }

      const int j0 = pc.j0 + i * KT;                 // the tile's first key
      const bool edge = pc.edge<KT>(i, a.window);
      // (in an edge tile) values that some rows must not see
      bool bad_v = false;
      if (edge) {
        bool mine = false;
#pragma unroll
        for (int it = 0; it < SH::TILE / (16 * kThreads); ++it) {
          const uint4 w = *reinterpret_cast<const uint4*>(kst + SH::TILE + (it * kThreads + tid) * 16);
          mine |= not_finite<T>(w.x) || not_finite<T>(w.y) || not_finite<T>(w.z) || not_finite<T>(w.w);
        }
        bad_v = __syncthreads_or(mine);              // (also: K has been read by every warp)
      }
      // Whether this thread's row sees key j; how far away it is.
      auto sees_key = [&](int j, int row, int& far) {
        const int jd = j - pc.len;
        bool see = true;
        int k_pos = j;
        if (jd >= 0) {
          if (pc.chain) {
            see = jd <= tok[row];
          } else {
            see = jd < pc.n && ((bits[row] >> (jd & 63)) & 1);
            k_pos = pc.len + s_depth[jd & 63];
          }
        }
        far = q_pos[row] - k_pos;
        return see && !(a.window > 0 && far >= a.window);
      };
      auto sees = [&](int x, int y, int& far) {      // the key of score (x, y)
        return sees_key(j0 + wk * NK + x * 8 + 2 * c + (y & 1), y >> 1, far);
      };
      if (a.cap_in != 0.f) {
        // (in units of log 2)
        const float k = a.cap_in * kCapUnit, co = a.cap_out;
        if (edge) {
          // what a row does not see must not choose how its scores are capped
#pragma unroll
          for (int x = 0; x < NK / 8; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              int far;
              if (!sees(x, y, far)) s[x][y] = 0.f;
            }
        }
        float far[2] = {0.f, 0.f};
#pragma unroll
        for (int x = 0; x < NK / 8; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y) far[y >> 1] = fmaxf(far[y >> 1], fabsf(s[x][y]));
        auto near = [&](float t) {
          const float u = t * t;
          return t * fmaf(fmaf(fmaf(kCap3 * co, u, kCap2 * co), u, kCap1 * co), u, co);
        };
        auto quotient = [&](float x) { return co * (1.f - __fdividef(2.f, ex2(x * a.cap_in) + 1.f)); };
        if (__all_sync(0xffffffffu, fmaxf(far[0], far[1]) * k <= kCapNear)) {
#pragma unroll
          for (int x = 0; x < NK / 8; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) s[x][y] = near(s[x][y] * k);
        } else {
          float reach[2];
          bool none = true;                          // no row near (padding rows have no say)
#pragma unroll
          for (int row = 0; row < 2; ++row) {
            far[row] = fmaxf(far[row], __shfl_xor_sync(0xffffffffu, far[row], 1));
            far[row] = fmaxf(far[row], __shfl_xor_sync(0xffffffffu, far[row], 2));
            reach[row] = cap_polynomial_reach(far[row] * k, co);
            none = none && (tok[row] < 0 || reach[row] < 0.f);
          }
          if (__all_sync(0xffffffffu, none)) {
#pragma unroll
            for (int x = 0; x < NK / 8; ++x)
#pragma unroll
              for (int y = 0; y < 4; ++y) s[x][y] = quotient(s[x][y]);
          } else {
#pragma unroll
            for (int x = 0; x < NK / 8; ++x)
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const float t = s[x][y] * k;
                s[x][y] = fabsf(t) <= reach[y >> 1] ? near(t) : quotient(s[x][y]);
              }
          }
        }
      } else {
#pragma unroll
        for (int x = 0; x < NK / 8; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y) s[x][y] *= a.score_log2;
      }
      if (edge || a.slopes) {
#pragma unroll
        for (int x = 0; x < NK / 8; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            int far;
            const bool see = sees(x, y, far);
            s[x][y] = see ? s[x][y] - slope[y >> 1] * (float)far : -INFINITY;
          }
      }
      float corr[2];
#pragma unroll
      for (int row = 0; row < 2; ++row) {
        float top = -INFINITY;
#pragma unroll
        for (int x = 0; x < NK / 8; ++x) top = fmaxf(top, fmaxf(s[x][2 * row], s[x][2 * row + 1]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float now = fmaxf(m[row], top);
        const float use = now == -INFINITY ? 0.f : now;   // nothing visible so far
        corr[row] = ex2(m[row] - use);
        m[row] = now;
        float sum = 0.f;
        const float shift = HALF ? use - kHalfShift : use;
#pragma unroll
        for (int x = 0; x < NK / 8; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float p = ex2(s[x][2 * row + y] - shift);
            s[x][2 * row + y] = p;
            sum += p;
          }
        l[row] = l[row] * corr[row] + sum;
      }
      // (mostly no row of the warp has a new maximum)
      if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
        for (int x = 0; x < D / 8; ++x) {
          acc[x][0] *= corr[0];
          acc[x][1] *= corr[0];
          acc[x][2] *= corr[1];
          acc[x][3] *= corr[1];
        }
      }
      if (!bad_v) {
#pragma unroll
        for (int kk = 0; kk < NK / 16; ++kk) {
          uint32_t p[4];
          p[0] = pack<T>(s[2 * kk][0], s[2 * kk][1]);
          p[1] = pack<T>(s[2 * kk][2], s[2 * kk][3]);
          p[2] = pack<T>(s[2 * kk + 1][0], s[2 * kk + 1][1]);
          p[3] = pack<T>(s[2 * kk + 1][2], s[2 * kk + 1][3]);
          const int row = wk * NK + kk * 16 + (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
          for (int dt = 0; dt < D / 16; ++dt) {
            const int ch = dt * 2 + (lane >> 4);
            uint32_t b[4];
            ldsm4_t(va + row * (D * 2) + ((ch ^ (row & 7)) << 4), b);
            mma<T>(acc[2 * dt], p, b[0], b[1]);
            mma<T>(acc[2 * dt + 1], p, b[2], b[3]);
          }
        }
      } else {
        // Some value of V is not finite, and 0 times it would be NaN in rows
        // that do not see it: this tile's products one by one, for the keys
        // that the row sees.  P lies over the K tile, which is done with.
        uint32_t* pp = reinterpret_cast<uint32_t*>(kst);  // [MT][KT / 2]
#pragma unroll
        for (int x = 0; x < NK / 8; ++x)
#pragma unroll
          for (int row = 0; row < 2; ++row)
            pp[(wm * 16 + g + 8 * row) * (KT / 2) + (wk * NK + x * 8) / 2 + c] =
                pack<T>(s[x][2 * row], s[x][2 * row + 1]);
        __syncwarp();                                 // a warp reads what it wrote itself
        for (int j = wk * NK; j < (wk + 1) * NK; ++j) {
          float p[2];
          bool see[2];
#pragma unroll
          for (int row = 0; row < 2; ++row) {
            int far;
            see[row] = sees_key(j0 + j, row, far);
            const float2 w = unpack<T>(pp[(wm * 16 + g + 8 * row) * (KT / 2) + j / 2]);
            p[row] = j & 1 ? w.y : w.x;
          }
#pragma unroll
          for (int x = 0; x < D / 8; ++x) {
            const float2 w = unpack<T>(*reinterpret_cast<const uint32_t*>(
                kst + SH::TILE + j * (D * 2) + ((x ^ (j & 7)) << 4) + c * 4));
#pragma unroll
            for (int row = 0; row < 2; ++row)
              if (see[row]) {
                acc[x][2 * row] += p[row] * w.x;
                acc[x][2 * row + 1] += p[row] * w.y;
              }
          }
        }
      }
    }

    // Join the warps that share rows, then write the result or a partial.
    cp_wait<0>();
#pragma unroll
    for (int row = 0; row < 2; ++row) {
      l[row] += __shfl_xor_sync(0xffffffffu, l[row], 1);
      l[row] += __shfl_xor_sync(0xffffffffu, l[row], 2);
      if (c == 0) {
        s_m[wk][wm * 16 + g + 8 * row] = m[row];
        s_l[wk][wm * 16 + g + 8 * row] = l[row];
      }
    }
    __syncthreads();                                 // the stages are free
    float* s_o = reinterpret_cast<float*>(smem);     // [WK][MT][OP]
#pragma unroll
    for (int x = 0; x < D / 8; ++x)
#pragma unroll
      for (int row = 0; row < 2; ++row)
        *reinterpret_cast<float2*>(s_o + (wk * MT + wm * 16 + g + 8 * row) * SH::OP + x * 8 + 2 * c) =
            make_float2(acc[x][2 * row], acc[x][2 * row + 1]);
    // (SHARED: what goes to the output undivided by its sum is joined later)
    const bool direct = !SHARED || (a.part == 1 && a.shared[pc.r] == 0);
    const bool whole = pc.whole && direct;
    const int slot = 2 * cta + (pc.begins ? 1 : 0);
    if (tid < rows) {
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < WK; ++w) top = fmaxf(top, s_m[w][tid]);
      const float use = top == -INFINITY ? 0.f : top;
      float f[WK];
#pragma unroll
      for (int w = 0; w < WK; ++w) {
        f[w] = ex2(s_m[w][tid] - use);
        sum += s_l[w][tid] * f[w];
      }
      const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
#pragma unroll
      for (int w = 0; w < WK; ++w) s_m[w][tid] = f[w] * inv;
      if (whole) {
        if (a.lse) {
          const int lt = tid / a.G, gg = tid - lt * a.G;
          a.lse[(long long)(pc.f + pc.tok0 + lt) * a.H * a.G + h * a.G + gg] =
              sum == 0.f ? -INFINITY
                         : (top - (HALF ? kHalfShift : 0.f)) * 0.6931471805599453f + logf(sum);
        }
      } else {
        float* ml = a.ml + ((long long)slot * MT + tid) * 2;
        if (SHARED && pc.whole) {
          const int lt = tid / a.G, gg = tid - lt * a.G;
          ml = a.rows_ml + ((long long)token_of<SHARED>(a, pc, pc.tok0 + lt) * a.H * a.G + h * a.G + gg) * 2;
        }
        *reinterpret_cast<float2*>(ml) = make_float2(top, sum);
      }
    }
    __syncthreads();
    for (int x = tid; x < rows * (D / 4); x += kThreads) {
      const int row = x / (D / 4), c4 = (x % (D / 4)) * 4;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WK; ++w) {
        const float4 y = *reinterpret_cast<const float4*>(s_o + (w * MT + row) * SH::OP + c4);
        const float f = s_m[w][row];
        o.x += y.x * f;
        o.y += y.y * f;
        o.z += y.z * f;
        o.w += y.w * f;
      }
      if (whole) {
        const int lt = row / a.G, gg = row - lt * a.G;
        const long long at_row = (long long)(pc.f + pc.tok0 + lt) * a.H * a.G + h * a.G + gg;
        *reinterpret_cast<uint2*>(a.out + (at_row * D + c4) * 2) =
            make_uint2(pack<T>(o.x, o.y), pack<T>(o.z, o.w));
      } else {
        float* part = a.partial + ((long long)slot * MT + row) * D;
        if (SHARED && pc.whole) {
          const int lt = row / a.G, gg = row - lt * a.G;
          part = a.rows + ((long long)token_of<SHARED>(a, pc, pc.tok0 + lt) * a.H * a.G + h * a.G + gg) * D;
        }
        *reinterpret_cast<float4*>(part + c4) = o;
      }
    }
    if (SHARED && pc.begins) note_unit(a, pc, cta, tid, kThreads);
    if (!whole && pc.begins) head = make_int4(pc.last - cta + 1, pc.f + pc.tok0, h, rows);
  }
  if (SHARED) griddep_wait();
  else if (tid == 0) a.head[cta] = head;
}

// Joins the partials of the units that cross CTAs.  WPR warps work on one row,
// each on every WPR-th piece.  blockIdx.x is the CTA in whose share a unit
// begins (32 of them where up to kFewUnits units are looked for), blockIdx.y a
// group of its rows.
constexpr int kMergeWarps = 8;
constexpr int kFewUnits = 4;
template <typename T, int D, int WPR>
__global__ void __launch_bounds__(kMergeWarps * 32) tree_merge_kernel(TreeArgs a, int MT) {
  constexpr int RPC = kMergeWarps / WPR;             // rows per CTA
  constexpr int VPL = D / 32;                        // values per lane
  __shared__ float s_o[kMergeWarps][D], s_sum[kMergeWarps];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = warp % WPR;
  unsigned begins = 1;
  if constexpr (WPR > 1) {
    const int look = blockIdx.x * 32 + lane;
    begins = __ballot_sync(0xffffffffu, look < a.ctas && a.head[min(look, a.ctas - 1)].x != 0);
  }
  for (; begins; begins &= begins - 1) {
    const int cta = WPR > 1 ? blockIdx.x * 32 + __ffs(begins) - 1 : blockIdx.x;
    const int4 head = a.head[cta];
    if (head.x == 0) continue;
    for (int r0 = blockIdx.y * RPC; r0 < head.w; r0 += gridDim.y * RPC) {
      const int row = r0 + warp / WPR;
      const bool have = row < head.w;
      // piece 0 is the second partial of its CTA (the unit begins there), the others the first
      auto slot = [&](int i) { return (long long)(2 * (cta + i) + (i == 0 ? 1 : 0)) * MT + row; };
      float top = -INFINITY;
      if (have)
        for (int i = lane; i < head.x; i += 32) top = fmaxf(top, a.ml[slot(i) * 2]);
#pragma unroll
      for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      const float use = top == -INFINITY ? 0.f : top;
      float o[VPL], sum = 0.f;
#pragma unroll
      for (int x = 0; x < VPL; ++x) o[x] = 0.f;
      if (have)
#pragma unroll 8
        for (int i = part; i < head.x; i += WPR) {
          const float2 ml = *reinterpret_cast<const float2*>(a.ml + slot(i) * 2);
          const float f = ex2(ml.x - use);
          sum += ml.y * f;
          const float* p = a.partial + slot(i) * D + lane * VPL;
          if constexpr (VPL >= 4) {
#pragma unroll
            for (int x = 0; x < VPL; x += 4) {
              const float4 y = *reinterpret_cast<const float4*>(p + x);
              o[x] += y.x * f;
              o[x + 1] += y.y * f;
              o[x + 2] += y.z * f;
              o[x + 3] += y.w * f;
            }
          } else {
            const float2 y = *reinterpret_cast<const float2*>(p);
            o[0] += y.x * f;
            o[1] += y.y * f;
          }
        }
      if constexpr (WPR > 1) {
#pragma unroll
        for (int x = 0; x < VPL; ++x) s_o[warp][lane * VPL + x] = o[x];
        if (lane == 0) s_sum[warp] = sum;
        __syncthreads();
        if (part == 0) {
#pragma unroll
          for (int w = 1; w < WPR; ++w) {
            sum += s_sum[warp + w];
#pragma unroll
            for (int x = 0; x < VPL; ++x) o[x] += s_o[warp + w][lane * VPL + x];
          }
        }
        __syncthreads();
      }
      if (!have || part != 0) continue;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const int lt = row / a.G, gg = row - lt * a.G;
      const long long at = (long long)(head.y + lt) * a.H * a.G + head.z * a.G + gg;
      unsigned char* dst = a.out + (at * D + lane * VPL) * 2;
#pragma unroll
      for (int x = 0; x < VPL; x += 2)
        *reinterpret_cast<uint32_t*>(dst + x * 2) = pack<T>(o[x] * inv, o[x + 1] * inv);
      if (a.lse && lane == 0) {
        constexpr float shift = std::is_same<T, __half>::value ? kHalfShift : 0.f;
        a.lse[at] = sum == 0.f ? -INFINITY : (top - shift) * 0.6931471805599453f + logf(sum);
      }
    }
  }
}

// Joins after the attention, whose m-tiles hold MT rows.
template <typename T, int D>
cudaError_t launch_merge(const TreeArgs& a, int MT, cudaStream_t st) {
  const int most = a.max_new < a.tpm ? a.max_new : a.tpm;
  const int rows = most * a.G;
  // A few units lie in up to 304 CTAs' shares: eight warps on a row (one: 16 us for 304
  // pieces), a block for 32 shares (one unit of 256 rows, 32768 tokens: 31 us the call, 80 with
  // a block for each share).
  if ((long long)a.R * a.H * (((long long)a.max_new + a.tpm - 1) / a.tpm) <= kFewUnits)
    return launch_pdl(tree_merge_kernel<T, D, kMergeWarps>, dim3((a.ctas + 31) / 32, rows),
                      dim3(kMergeWarps * 32), 0, st, a, MT);
  // Else a warp per row, in few groups: every CTA of the grid without a unit to join costs its
  // launch (304 x 32 of them 5 us), a further round of rows 1.5 us.
  const int groups = (rows + kMergeWarps - 1) / kMergeWarps;
  return launch_pdl(tree_merge_kernel<T, D, 1>, dim3(a.ctas, groups), dim3(kMergeWarps * 32), 0, st, a, MT);
}

template <typename T, int D, int WM, bool SHARED>
cudaError_t launch_one(const TreeArgs& a, int dev, cudaStream_t st) {
  using SH = Shape<T, D, WM, SHARED>;
  static SmemLimit limit;
  cudaError_t e = limit.raise(reinterpret_cast<const void*>(tree_attn_kernel<SH>), SH::SMEM, dev);
  if (e == cudaSuccess)
    e = launch_pdl(tree_attn_kernel<SH>, dim3(a.ctas), dim3(SH::THREADS), SH::SMEM, st, a);
  return e != cudaSuccess || SHARED ? e : launch_merge<T, D>(a, SH::MT, st);
}

template <int D, bool SHARED>
cudaError_t launch_width(const TreeArgs& a, int dtype, int wm, int dev, cudaStream_t st) {
  if (dtype == AVSG_BF16) {
    if (wm == 1) return launch_one<__nv_bfloat16, D, 1, SHARED>(a, dev, st);
    if (wm == 2) return launch_one<__nv_bfloat16, D, 2, SHARED>(a, dev, st);
    return launch_one<__nv_bfloat16, D, 4, SHARED>(a, dev, st);
  }
  if (wm == 1) return launch_one<__half, D, 1, SHARED>(a, dev, st);
  if (wm == 2) return launch_one<__half, D, 2, SHARED>(a, dev, st);
  return launch_one<__half, D, 4, SHARED>(a, dev, st);
}

}  // namespace tree
}  // namespace avsg
