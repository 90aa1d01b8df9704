// avsg_prefix_attention: tree attention in which the prefix that a group of
// requests shares is computed once for all of them.
//
// Softmax over a row's keys splits over any partition of them: with (m, l, o) the maximum,
// the sum of 2^(s - m) and the output not divided by it of either part,
//   out = sum_i o_i 2^(m_i - m) / sum_i l_i 2^(m_i - m),  m = max_i m_i.
// So there are two lists of units, each cut into equal shares as in
// avsg_tree_attn.cuh:
//   part 0  (group, kv-head, m-tile): the group's new tokens, listed by
//           avsg_prefix_find, as rows, its prefix as keys;
//   part 1  (request, kv-head, m-tile): a request's new tokens, its keys
//           behind the prefix (all of them where it has none, and then the output itself);
// and a kernel that joins a row's pieces of both (and looks every token with a
// prefix up in the list).  The parts are launches of
// their own: a group has many rows and a long prefix (tcgen05's work), a request often few rows
// and few keys of its own (mma.sync's).  They run side by side: part 1 does
// not wait for part 0 before it begins, only before it ends, so that what follows it follows
// both; and each part's list is cut into as many shares as its cost gives it
// SMs, the CTAs behind that leave at once.
//
// What bounds it: part 0 the tensor cores (from about 100 rows a group on), part
// 1 HBM and what the beginnings and ends of its units take; K and V of a prefix are read once for
// each 256 rows of its group.  Measured: 64 requests behind 32768 tokens, up to
// 500 tokens of their own, one new token each, 8 kv-heads of 4: 68 us (the tree
// attention, for which every request reads the prefix, 1030); one part after the other 88.  Of the 68: 4 us until
// both parts have found their shares, 50 for the parts, 2 between kernels, 5 for the join.
// 69 requests with trees of up to 16 tokens in four groups of up to 32768: 294 to 304 us.
// Where no request has a group it costs 8 to 28 us more than the tree attention (64 requests alone,
// one new token each: 42 and 32 us at 100 tokens, 59 and 44 at 500, 121 and 101 at 2000, 206 and 178 at
// 4000, 335 and 327 at 8000): the empty
// part and the join, and part 1's kernel alone takes 13% more at 2000 tokens, of which twice the
// stalls for instructions are seen, but neither its registers nor the order of its branches is the cause.
#include "avsg_tree_plan.cuh"

namespace avsg {
namespace {

constexpr int kJoinThreads = 256;

struct JoinPart {
  const int4* unit;              // see TreeArgs
  const float* rows;
  const float* rows_ml;
  const float* partial;
  const float* ml;
  int ctas, MT;
};
struct JoinArgs {
  JoinPart part[2];
  const int32_t* first;
  const int32_t* shared;         // the groups, see TreeArgs
  const int32_t* group_first;
  const int32_t* token;
  unsigned char* out;
  float* lse;
  DevErr* err;
  int R, H, G, T, places;
  unsigned checks;               // blocks that look at tokens, in front of those that join rows
};

// Whether token t, if it has a prefix, is in the list of a group with a prefix of that length.  The workspace
// may hold another call's entries: one is this call's if the place that it names lies in the group that it
// names and lists the token, as part 0 has then written the token's entries anew.
__device__ __forceinline__ bool token_listed(const JoinArgs& a, int t) {
  const int common = a.part[1].unit[(long long)t * a.H].w;
  if (common == 0) return true;
  const int4 pre = a.part[0].unit[(long long)t * a.H];
  const int lead = pre.x >> 16;
  const long long at = (long long)pre.w + pre.z;
  if (lead < 0 || lead >= a.R || at < 0 || at >= a.places) return false;
  return a.token[at] == t && a.shared[lead] == common && a.group_first[lead] <= at && at < a.group_first[lead + 1];
}

// WPR warps join the pieces of one row, each every WPR-th of them.  Two dependent chains of loads: where the pieces lie, then
// their maxima, sums and outputs side by side, up to kJoinAhead outputs before the first weight is known.
// What bounds it is how many bytes are on their way (20 000 rows of 3 pieces: 13 us; with two outputs
// ahead in 32 registers and 8 blocks an SM 16).
constexpr int kJoinAhead = 4;
constexpr int join_blocks(int D) { return D == 256 ? 3 : 5; }
template <typename T, int D, int WPR>
__global__ void __launch_bounds__(kJoinThreads, join_blocks(D)) prefix_join_kernel(JoinArgs a) {
  constexpr int VPL = D / 32, ROWS = kJoinThreads / 32 / WPR;
  __shared__ float s_o[WPR > 1 ? kJoinThreads / 32 : 1][D], s_ml[kJoinThreads / 32][2];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, heads = a.H * a.G;
  if (blockIdx.x < a.checks) {
    // (in blocks of their own: in each row's way the check cost 2.4 us of 19 for 20 000 rows)
    const long long t = (long long)blockIdx.x * kJoinThreads + threadIdx.x;
    if (load_err(a.err) == 0 && t < min(a.T, a.first[a.R]) && !token_listed(a, (int)t))
      raise_error(a.err, AVSG_ERR_BAD_SELECTION, -1, (int)t);
    return;
  }
  const int part = warp % WPR;             // of the row's warps
  const long long row = (long long)(blockIdx.x - a.checks) * ROWS + warp / WPR;
  const int t = (int)(row / heads), hg = (int)(row - (long long)t * heads), h = hg / a.G, g = hg - h * a.G;
  // A row without anything to join has no pieces.  Its warps stay for the barrier below: each reads the
  // error word for itself, and another row's warp may raise it between two reads.
  bool live = t < a.T;
  const int tokens = a.first[a.R];
  const bool latched = __any_sync(0xffffffffu, load_err(a.err) != 0);
  int4 own = make_int4(0, -1, 0, 0), pre = own;
  if (live) {
    own = a.part[1].unit[(long long)t * a.H + h];
    pre = a.part[0].unit[(long long)t * a.H + h];  // (any contents, where the token has no prefix)
  }
  // (own.y < 0: written by its part)
  live = live && !latched && t < tokens && own.y >= 0;
  if (!own.w) pre = make_int4(0, -1, 0, 0);
  pre.x &= 0xffff;                         // (see token_listed)
  auto pieces = [&](const int4& u) { return u.y < 0 ? 0 : u.y == 0 ? 1 : u.y; };
  auto fits = [&](const JoinPart& p, const int4& u) {
    return u.y <= 0 || (u.x >= 0 && u.x < p.ctas && u.y <= p.ctas - u.x && u.z >= 0 && u.z < p.MT / a.G);
  };
  if (live && ((own.w && pre.y < 0) || !fits(a.part[0], pre) || !fits(a.part[1], own))) {
    if (lane == 0) raise_error(a.err, AVSG_ERR_BAD_SELECTION, -1, t);
    live = false;
  }
  if (WPR == 1 && !live) return;
  const int n0 = pieces(pre), all = live ? n0 + pieces(own) : 0;
  const int n = (all - part + WPR - 1) / WPR;  // this warp's
  // where piece i lies among the part's partials or rows
  auto place = [&](int k, const float*& ml, const float*& o) {
    const int i = k * WPR + part;
    const bool second = i >= n0;
    const JoinPart& p = a.part[second];
    const int4 u = second ? own : pre;
    const int j = second ? i - n0 : i;
    if (u.y == 0) {
      ml = p.rows_ml + row * 2;
      o = p.rows + row * D;
    } else {
      // the first piece is the second partial of its CTA, the others the first ones of theirs
      const long long slot = (long long)(2 * (u.x + j) + (j == 0 ? 1 : 0)) * p.MT + u.z * a.G + g;
      ml = p.ml + slot * 2;
      o = p.partial + slot * D;
    }
  };
  float top = -INFINITY, sum = 0.f, o[VPL];
#pragma unroll
  for (int x = 0; x < VPL; ++x) o[x] = 0.f;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const float *ml = nullptr, *from = nullptr;
    float2 y = make_float2(-INFINITY, 0.f);
    if (i0 + lane < n) {
      place(i0 + lane, ml, from);
      y = *reinterpret_cast<const float2*>(ml);
    }
    const int most = min(32, n - i0);
    float z[kJoinAhead][VPL];
    auto fetch = [&](int j0) {
#pragma unroll
      for (int j = 0; j < kJoinAhead; ++j) {
        const float* p = reinterpret_cast<const float*>(__shfl_sync(
            0xffffffffu, reinterpret_cast<unsigned long long>(from), (j0 + j) & 31)) + lane * VPL;
        if (j0 + j < most) {
          if constexpr (VPL >= 4) {
#pragma unroll
            for (int x = 0; x < VPL; x += 4) *reinterpret_cast<float4*>(z[j] + x) = *reinterpret_cast<const float4*>(p + x);
          } else {
            *reinterpret_cast<float2*>(z[j]) = *reinterpret_cast<const float2*>(p);
          }
        }
      }
    };
    fetch(0);
    float now = y.x;
#pragma unroll
    for (int d = 16; d; d >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, d));
    now = fmaxf(now, top);
    const float use = now == -INFINITY ? 0.f : now, old = tree::ex2(top - use);
    top = now;
    const float f = tree::ex2(y.x - use);
    float add = y.y * f;
#pragma unroll
    for (int d = 16; d; d >>= 1) add += __shfl_xor_sync(0xffffffffu, add, d);
    sum = sum * old + add;
#pragma unroll
    for (int x = 0; x < VPL; ++x) o[x] *= old;
    for (int j0 = 0; j0 < most; j0 += kJoinAhead) {
      if (j0 > 0) fetch(j0);
#pragma unroll
      for (int j = 0; j < kJoinAhead; ++j) {
        const float w = __shfl_sync(0xffffffffu, f, (j0 + j) & 31);
        if (j0 + j < most)
#pragma unroll
          for (int x = 0; x < VPL; ++x) o[x] += z[j][x] * w;
      }
    }
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int x = 0; x < VPL; ++x) s_o[warp][lane * VPL + x] = o[x];
    if (lane == 0) {
      s_ml[warp][0] = top;
      s_ml[warp][1] = live ? sum : -1.f;   // (a sum is never negative)
    }
    // a barrier of the row's warps, to which all of them come (waiting for the block's other rows costs 0.8 us)
    asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / WPR), "n"(32 * WPR) : "memory");
    if (part != 0 || !live) return;
    float tops[WPR];
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      if (s_ml[warp + w][1] < 0.f) return; // a sibling saw an error: the row is written whole or not at all
      tops[w] = s_ml[warp + w][0];
      top = fmaxf(top, tops[w]);
    }
    const float use = top == -INFINITY ? 0.f : top;
    sum = 0.f;
#pragma unroll
    for (int x = 0; x < VPL; ++x) o[x] = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      const float f = tree::ex2(tops[w] - use);
      sum += s_ml[warp + w][1] * f;
#pragma unroll
      for (int x = 0; x < VPL; ++x) o[x] += s_o[warp + w][lane * VPL + x] * f;
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  unsigned char* dst = a.out + (row * D + lane * VPL) * 2;
#pragma unroll
  for (int x = 0; x < VPL; x += 2)
    *reinterpret_cast<uint32_t*>(dst + x * 2) = tree::pack<T>(o[x] * inv, o[x + 1] * inv);
  if (a.lse && lane == 0) {
    constexpr float shift = std::is_same<T, __half>::value ? tree::kHalfShift : 0.f;
    a.lse[row] = sum == 0.f ? -INFINITY : (top - shift) * 0.6931471805599453f + logf(sum);
  }
}

template <typename T, int D, int WPR>
cudaError_t launch_join_one(JoinArgs a, int dev, cudaStream_t st) {
  constexpr int ROWS = kJoinThreads / 32 / WPR;
  static SmemSplit split;
  auto kernel = prefix_join_kernel<T, D, WPR>;
  const cudaError_t e = split.ask(reinterpret_cast<const void*>(kernel), dev);
  if (e != cudaSuccess) return e;
  const long long rows = (long long)a.T * a.H * a.G;
  a.checks = ((unsigned)a.T + kJoinThreads - 1) / kJoinThreads;
  return launch_pdl(kernel, dim3((unsigned)((rows + ROWS - 1) / ROWS) + a.checks), dim3(kJoinThreads), 0, st, a);
}
template <typename T, int D>
cudaError_t launch_join_width(const JoinArgs& a, int sms, int dev, cudaStream_t st) {
  const long long rows = (long long)a.T * a.H * a.G;
  // few rows may have many pieces each: several warps a row as long as all blocks fit the SMs at once
  const long long fit = (long long)sms * join_blocks(D) * (kJoinThreads / 32);
  if (rows * 4 <= fit) return launch_join_one<T, D, 4>(a, dev, st);
  if (rows * 2 <= fit) return launch_join_one<T, D, 2>(a, dev, st);
  return launch_join_one<T, D, 1>(a, dev, st);
}
template <typename T>
cudaError_t launch_join(const JoinArgs& a, int D, int sms, int dev, cudaStream_t st) {
  return D == 64    ? launch_join_width<T, 64>(a, sms, dev, st)
         : D == 128 ? launch_join_width<T, 128>(a, sms, dev, st)
                    : launch_join_width<T, 256>(a, sms, dev, st);
}

// What a CTA takes for a unit's beginning and end, a tile, and on tcgen05 a tile of up to 128 rows,
// in hundredths of a microsecond: least squares over the CTAs of calls with a long document or draft trees,
// heads of each width, on either kernel (GB300; wm 2 between its neighbours).  Tiles are 128 keys on tcgen05, 64 with mma.sync and for heads of 256.
struct CtaCost {
  int begin, tile, small;
};
CtaCost cta_cost(const Plan& x, int D) {
  const int w = D == 64 ? 0 : D == 128 ? 1 : 2;
  static const CtaCost umma[3] = {{600, 153, 88}, {950, 158, 105}, {1040, 84, 84}};
  static const CtaCost mma[3][3] = {{{330, 85, 85}, {400, 125, 125}, {590, 170, 170}},
                                    {{400, 105, 105}, {500, 165, 165}, {650, 210, 210}},
                                    {{450, 130, 130}, {700, 212, 212}, {700, 250, 250}}};
  return x.umma ? umma[w] : mma[x.wm == 4 ? 2 : x.wm - 1][w];
}

struct PrefixWork {
  size_t unit[2], rows_ml[2], rows[2], part[2], bytes;
};
PrefixWork prefix_layout(const avsg_pages* p, int G, int max_new, int num_tokens, int sms) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t T = num_tokens, heads = (size_t)p->num_kv_heads * G;
  PrefixWork w;
  size_t at = 0;
  for (int i = 0; i < 2; ++i) {
    w.unit[i] = at;
    w.rows_ml[i] = w.unit[i] + up(T * p->num_kv_heads * sizeof(int4));
    w.rows[i] = w.rows_ml[i] + up(T * heads * 2 * sizeof(float));
    w.part[i] = w.rows[i] + up(T * heads * p->head_dim * sizeof(float));
    at = w.part[i] + up(workspace_bytes(p->head_dim, G, i == 0 ? (num_tokens < 1 ? 1 : num_tokens) : max_new, sms));
  }
  w.bytes = at;
  return w;
}

}  // namespace
}  // namespace avsg

using namespace avsg;

extern "C" int avsg_prefix_attention_workspace(const avsg_pages* p, int32_t q_per_kv, int32_t max_new,
                                               int32_t num_tokens, size_t* bytes) {
  const int rc = check_attention(p, q_per_kv, max_new);
  if (rc != AVSG_OK) return rc;
  if (!bytes || num_tokens < 0) return AVSG_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  const int rd = paged_device(p->d_k, &dev, &sms);
  if (rd != AVSG_OK) return rd;
  *bytes = prefix_layout(p, q_per_kv, max_new, num_tokens, sms).bytes;
  return AVSG_OK;
}

extern "C" int avsg_prefix_attention(const avsg_pages* p, const avsg_tree* t, const avsg_prefixes* x, void* stream) {
  if (!x || x->num_tokens < 0 || x->reserved0 != 0) return AVSG_ERR_INVALID_ARG;
  TreeArgs a{};
  int dev = 0, sms = 0;
  const int rc = tree_args(p, t, &a, &dev, &sms);
  if (rc != AVSG_OK || a.T == 0) return rc;
  if (!x->d_shared || !x->d_first || (x->num_tokens > 0 && (!x->d_token || !x->d_request)))
    return AVSG_ERR_INVALID_ARG;
  const int D = p->head_dim, G = t->q_per_kv;
  const PrefixWork w = prefix_layout(p, G, t->max_new, t->num_tokens, sms);
  if (t->work_bytes < w.bytes) return AVSG_ERR_CAPACITY;
  if ((int64_t)a.T * a.H * G / (kJoinThreads / 32) + a.T / kJoinThreads + 2 > INT32_MAX) return AVSG_ERR_CAPACITY;
  unsigned char* work = static_cast<unsigned char*>(t->d_work);
  a.places = x->num_tokens;
  a.shared = x->d_shared;
  a.group_first = x->d_first;
  a.token = x->d_token;
  a.request = x->d_request;
  a.sms = sms;
  JoinArgs j{};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Plan plans[2] = {plan_attention(p, G, t->num_tokens, sms), plan_attention(p, G, t->max_new, sms)};
  CtaCost cost[2];
  for (int i = 0; i < 2; ++i) {
    cost[i] = cta_cost(plans[i], D);
    TreeArgs::Cost& c = a.cost[i];
    c.per_sm = plans[i].ctas / sms;
    c.keys = plans[i].umma && D != 256 ? 128 : 64;
    c.tpm = plans[i].MT / G;
    // (part 1's CTAs end less evenly, 10% behind their median)
    const int num = i == 0 ? 10 : 11, den = 10 * c.per_sm;
    c.begin = cost[i].begin * num / den;
    c.tile = cost[i].tile * num / den;
    c.small = cost[i].small * num / den;
  }
  // Cutting a list into shares splits about a unit per CTA, which pays for a beginning and an end more.
  a.lead = a.cost[0].begin > a.cost[1].begin ? a.cost[0].begin - a.cost[1].begin : 0;
  for (int i = 0; i < 2; ++i) {
    const Plan& plan = plans[i];
    const Workspace l = tree_layout(plan, D);
    TreeArgs b = a;
    b.part = i;
    b.unit = reinterpret_cast<int4*>(work + w.unit[i]);
    b.rows_ml = reinterpret_cast<float*>(work + w.rows_ml[i]);
    b.rows = reinterpret_cast<float*>(work + w.rows[i]);
    b.ml = reinterpret_cast<float*>(work + w.part[i] + l.ml);
    b.partial = reinterpret_cast<float*>(work + w.part[i] + l.part);
    b.tpm = plan.MT / G;
    b.ctas = plan.ctas;
    // Places of the list: of a tile by its cost, of a unit's beginning and end in tiles.
    b.w_full = b.w_small = 1;
    if (i == 0 && plan.umma && D != 256) {
      b.w_full = D == 64 ? 5 : 3;
      b.w_small = D == 64 ? 3 : 2;
      b.small_rows = plan.MT / 2;
    }
    const int tile = i == 0 ? cost[i].tile : cost[i].small;
    b.begin = (cost[i].begin + tile / 2) / tile * b.w_full;
    b.min_tiles = 2 * b.w_full;
    j.part[i] = JoinPart{b.unit, b.rows, b.rows_ml, b.partial, b.ml, plan.ctas, plan.MT};
    const cudaError_t e = plan.umma ? launch_prefix_umma(b, p->dtype, D, dev, st)
                                    : launch_prefix_part(b, p->dtype, D, plan.wm, dev, st);
    if (e != cudaSuccess) return AVSG_ERR_CUDA;
  }
  j.first = t->d_first;
  j.shared = a.shared;
  j.group_first = a.group_first;
  j.token = a.token;
  j.places = a.places;
  j.out = a.out;
  j.lse = a.lse;
  j.err = a.err;
  j.R = a.R;
  j.H = a.H;
  j.G = G;
  j.T = a.T;
  const cudaError_t e =
      p->dtype == AVSG_BF16 ? launch_join<__nv_bfloat16>(j, D, sms, dev, st) : launch_join<__half>(j, D, sms, dev, st);
  return e == cudaSuccess ? AVSG_OK : AVSG_ERR_CUDA;
}
