// avsg_page_compact: the pages in use move to the front of the pool.
//
// With F = the free ids (the stack) and live = num_pages - |F|, the n-th id at
// or above live that is not in F moves to the n-th id of F below live (there are
// as many of one as of the other).  Both numbers come from one table, the count of
// free ids before every 32nd id: with f(x) = free ids below x, a free id x is
// hole f(x), and a live id x >= live is mover x - f(x) - (live - f(live)), which is
// live - 1 - (x - f(x)) from the last one backwards.
//
// What bounds it: the pages that move, read once and written once in every
// layer.  The bitmap, its sums, the lists of holes and movers and the check of
// all held entries come before (latency): for pools of up to 65536 pages every
// CTA builds the bitmap in its own shared memory, and no CTA needs another one;
// for larger ones it is one cluster's work, in global memory.  Everything else
// is written by the second kernel, which takes tables, shares and stack
// element by element, so that outputs may be the inputs, and pages in pieces of 4 KB by the warp.
// It goes by what every CTA of the first one found, and not by the error word, which a call on another
// stream may change between two CTAs' reads: part of the pages would move.
// Measured: 64 requests of up to 1500 tokens, a third of the pool free, 8
// layers, 0.54 GB of K and V moved: 177 us (6.1 TB/s read and written, 90% of the copy's
// rate); a pool of one layer and 150 pages 10.5 us (12.7 with the cluster's barriers).
#include <cooperative_groups.h>

#include "avsg_paged.cuh"

namespace cg = cooperative_groups;

namespace avsg {
namespace {

constexpr int kCompactThreads = 1024;
constexpr int kCompactCluster = 8;
constexpr int kPackThreads = 256;
constexpr int kPackBatch = 8;              // 16-byte chunks in flight per thread
constexpr int kPackPiece = 32 * kPackBatch;  // 16-byte chunks of a warp's piece

struct CompactArgs {
  int R, shift, max_pages, num_pages, words;
  const int32_t* len;
  const int32_t* tables;
  const int32_t* free_list;
  const int32_t* count;
  uint32_t* bits;                          // [words] bitmap of free ids
  int32_t* before;                         // [words] free ids before the word's first
  int32_t* holes;                          // [num_pages / 2 + 1]
  int32_t* movers;                         // [num_pages / 2 + 1], the last one first
  int32_t* live;                           // {live pages, free ids below that: the pages that move}
  int32_t* fine;                           // [ctas] whether the checks of a CTA of the first kernel passed
  int ctas;
  DevErr* err;
};
constexpr int kMostPlanCtas = 32;          // (a warp of the second kernel reads their words)

__device__ __forceinline__ int free_before(const uint32_t* bits, const int32_t* before, int id) {
  return __ldcg(before + (id >> 5)) + __popc(__ldcg(bits + (id >> 5)) & ((1u << (id & 31)) - 1));
}

// One word's results: free ids before it, its holes and movers.  sum: free ids before the word.
__device__ __forceinline__ void list_word(const CompactArgs& a, int live, int w, uint32_t b, int sum) {
  a.bits[w] = b;
  a.before[w] = sum;
  if (live >> 5 == w) {
    a.live[0] = live;
    a.live[1] = sum + __popc(b & ((1u << (live & 31)) - 1));
  }
  // (the ids of the word that lie in the pool)
  const uint32_t ids = a.num_pages - w * 32 >= 32 ? 0xffffffffu : (1u << (a.num_pages - w * 32)) - 1;
  if (w >= live >> 5)
    for (uint32_t u = ~b & ids; u; u &= u - 1) {
      const int x = __ffs(u) - 1, id = w * 32 + x;
      if (id >= live) a.movers[live - 1 - (id - sum - __popc(b & ((1u << x) - 1)))] = id;
    }
  for (; b; b &= b - 1, ++sum) {
    const int id = w * 32 + __ffs(b) - 1;
    if (id < live) a.holes[sum] = id;
  }
}
// What request r holds lies in the pool and is in use (a warp); *fine is 0 afterwards if it does not.
template <typename F>
__device__ __forceinline__ void check_held(const CompactArgs& a, int r, int32_t* fine, F&& is_free) {
  const int len = a.len[r];
  const long long held = ((long long)len + (1 << a.shift) - 1) >> a.shift;
  if (len < 0 || held > a.max_pages) {
    raise_error(a.err, len < 0 ? AVSG_ERR_BAD_SELECTION : AVSG_ERR_CAPACITY, r, -1);
    *fine = 0;
    return;
  }
  const int32_t* row = a.tables + (size_t)r * a.max_pages;
  int bad = -1;                            // (latched behind the loop, which then has its loads side by side)
#pragma unroll 4
  for (int x = threadIdx.x & 31; x < (int)held; x += 32) {
    const int32_t id = row[x];
    if (id < 0 || id >= a.num_pages || is_free(id)) bad = x;
  }
  if (bad >= 0) {
    raise_error(a.err, AVSG_ERR_BAD_SELECTION, r, bad);
    *fine = 0;
  }
}

__global__ void __launch_bounds__(kCompactThreads) compact_plan_kernel(CompactArgs a) {
  __shared__ long long s_warp[kCompactThreads / 32];
  __shared__ int s_sum[kCompactCluster];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  const int tid = threadIdx.x, at = rank * kCompactThreads + tid, threads = ctas * kCompactThreads;
  griddep_wait();
  bool ok = load_err(a.err) == 0;
  const int count = *a.count;
  if (count < 0 || count > a.num_pages) {
    if (ok && at == 0) raise_error(a.err, AVSG_ERR_BAD_SELECTION, -1, -1);
    ok = false;
  }
  const int live = a.num_pages - count;
  if (ok)
    for (int w = at; w < a.words; w += threads) a.bits[w] = 0;
  __threadfence();
  cluster.sync();
  if (ok)
    for (long long i = at; i < count; i += threads) {
      const int32_t id = a.free_list[i];
      if (id < 0 || id >= a.num_pages || (atomicOr(a.bits + (id >> 5), 1u << (id & 31)) >> (id & 31) & 1)) {
        raise_error(a.err, AVSG_ERR_BAD_SELECTION, -1, (int)i);
        ok = false;
      }
    }
  __threadfence();
  cluster.sync();
  ok = !__syncthreads_or(!ok || load_err(a.err) != 0);
  if (tid == 0) a.fine[rank] = ok;         // (before the barriers that what is found below comes after)
  // a range of words per CTA, of it one per thread
  const int per_cta = (a.words + ctas - 1) / ctas;
  const int c0 = min(a.words, rank * per_cta), c1 = min(a.words, c0 + per_cta);
  const int per = (c1 - c0 + kCompactThreads - 1) / kCompactThreads;
  const int w0 = min(c1, c0 + tid * per), w1 = min(c1, w0 + per);
  long long mine = 0, all;
  if (ok)
    for (int w = w0; w < w1; ++w) mine += __popc(__ldcg(a.bits + w));
  long long sum = block_exclusive(mine, s_warp, &all);
  if (tid < ctas) *cluster.map_shared_rank(&s_sum[rank], tid) = (int)all;
  cluster.sync();
  for (int c = 0; c < rank; ++c) sum += s_sum[c];
  if (ok)
    for (int w = w0; w < w1; ++w) {
      const uint32_t b = __ldcg(a.bits + w);
      list_word(a, live, w, b, (int)sum);
      sum += __popc(b);
    }
  if (ok && at == 0 && live >> 5 >= a.words) {  // every page is in use
    a.live[0] = live;
    a.live[1] = 0;
  }
  // what the requests hold lies in the pool and is in use
  if (ok)
    for (int r = at >> 5; r < a.R; r += threads >> 5)
      check_held(a, r, a.fine + rank, [&](int id) { return __ldcg(a.bits + (id >> 5)) >> (id & 31) & 1; });
  cluster.sync();                          // (no CTA ends while another may write its s_sum)
}

constexpr int kSmallPool = 65536;          // pages whose bitmap every CTA builds for itself
__global__ void __launch_bounds__(kCompactThreads) compact_plan_small_kernel(CompactArgs a) {
  __shared__ uint32_t s_bits[kSmallPool / 32];
  __shared__ int s_warp[kCompactThreads / 32];
  constexpr int kEach = kSmallPool / 32 / kCompactThreads;  // words of a thread
  const int tid = threadIdx.x;
  for (int w = tid; w < a.words; w += kCompactThreads) s_bits[w] = 0;
  griddep_wait();
  const bool latched = load_err(a.err) != 0;
  const int count = *a.count;
  const bool fits = count >= 0 && count <= a.num_pages;
  if (!fits && !latched && tid == 0 && blockIdx.x == 0) raise_error(a.err, AVSG_ERR_BAD_SELECTION, -1, -1);
  if (__syncthreads_or(latched || !fits)) {
    if (tid == 0) a.fine[blockIdx.x] = 0;
    return;
  }
  if (tid == 0) a.fine[blockIdx.x] = 1;    // (before the barrier that what is found below comes after)
  griddep_launch();
  int bad = -1;
  for (int i = tid; i < count; i += kCompactThreads) {
    const int32_t id = a.free_list[i];
    if (id < 0 || id >= a.num_pages || (atomicOr(s_bits + (id >> 5), 1u << (id & 31)) >> (id & 31) & 1)) bad = i;
  }
  if (bad >= 0 && blockIdx.x == 0) raise_error(a.err, AVSG_ERR_BAD_SELECTION, -1, bad);
  if (__syncthreads_or(bad >= 0)) {
    if (tid == 0) a.fine[blockIdx.x] = 0;
    return;
  }
  const int live = a.num_pages - count;
  if (blockIdx.x == 0) {
    const int w0 = min(a.words, tid * kEach), w1 = min(a.words, w0 + kEach);
    int mine = 0, all;
    for (int w = w0; w < w1; ++w) mine += __popc(s_bits[w]);
    int sum = block_exclusive(mine, s_warp, &all);
    for (int w = w0; w < w1; ++w) {
      list_word(a, live, w, s_bits[w], sum);
      sum += __popc(s_bits[w]);
    }
    if (tid == 0 && live >> 5 >= a.words) {  // every page is in use
      a.live[0] = live;
      a.live[1] = 0;
    }
  }
  const int warps = gridDim.x * (kCompactThreads / 32);
  for (int r = blockIdx.x * (kCompactThreads / 32) + (tid >> 5); r < a.R; r += warps)
    check_held(a, r, a.fine + blockIdx.x, [&](int id) { return s_bits[id >> 5] >> (id & 31) & 1; });
}

struct PackArgs {
  CompactArgs c;
  int num_layers;
  long long page_chunks;                   // 16-byte chunks of a page
  long long layer_bytes;
  unsigned char* k;
  unsigned char* v;
  const int32_t* shares;
  int32_t* shares_out;
  int32_t* tables_out;
  int32_t* free_out;
  int32_t* map;
};

__global__ void __launch_bounds__(kPackThreads) compact_move_kernel(PackArgs a) {
  const CompactArgs& c = a.c;
  griddep_wait();
  const int lane = threadIdx.x & 31;
  if (__any_sync(0xffffffffu, lane < c.ctas && c.fine[lane] == 0)) return;
  const long long threads = (long long)gridDim.x * kPackThreads;
  const long long at = (long long)blockIdx.x * kPackThreads + threadIdx.x;
  const int live = c.live[0], low = c.live[1], count = c.num_pages - live;
  const int kept = live - low;             // live ids that stay; as many move as there are holes
  auto target = [&](int id) {              // new id of a page in use
    return id < live ? id : c.holes[id - free_before(c.bits, c.before, id) - kept];
  };
  for (long long x = at; x < c.num_pages; x += threads) {
    const int id = (int)x;
    const bool is_free = c.bits[id >> 5] >> (id & 31) & 1;
    const int to = is_free ? -1 : target(id);
    a.map[id] = to;
    if (a.shares) {
      // a page's own thread writes its new place, and what lies behind the pages in use
      const int32_t s = a.shares[id];
      if (to >= 0) a.shares_out[to] = s;
      if (id >= live) a.shares_out[id] = 0;
    }
    if (id < count) a.free_out[id] = c.num_pages - 1 - id;
    else if (a.free_out != c.free_list) a.free_out[id] = c.free_list[id];
  }
  const long long entries = (long long)c.R * c.max_pages;
  for (long long x = at; x < entries; x += threads) {
    const int r = (int)(x / c.max_pages), col = (int)(x - (long long)r * c.max_pages);
    const int32_t id = c.tables[x];
    if (((long long)col << c.shift) < c.len[r]) a.tables_out[x] = target(id);
    else if (a.tables_out != c.tables) a.tables_out[x] = id;
  }
  // pages: a warp moves a piece of one, the n-th mover's to the n-th hole
  const long long pieces = (a.page_chunks + kPackPiece - 1) / kPackPiece;
  const long long units = (long long)low * a.num_layers * 2 * pieces;
  for (long long u = at >> 5; u < units; u += threads >> 5) {
    const long long piece = u % pieces, x = u / pieces;
    const int kv = (int)(x & 1), layer = (int)((x >> 1) % a.num_layers), n = (int)((x >> 1) / a.num_layers);
    const int from = c.movers[low - 1 - n], to = c.holes[n];
    unsigned char* base = (kv ? a.v : a.k) + layer * a.layer_bytes;
    const uint4* src = reinterpret_cast<const uint4*>(base) + from * a.page_chunks;
    uint4* dst = reinterpret_cast<uint4*>(base) + to * a.page_chunks;
    const long long i0 = piece * kPackPiece + lane;
    uint4 w[kPackBatch];
#pragma unroll
    for (int j = 0; j < kPackBatch; ++j)
      if (i0 + 32 * j < a.page_chunks) w[j] = __ldcs(src + i0 + 32 * j);
#pragma unroll
    for (int j = 0; j < kPackBatch; ++j)
      if (i0 + 32 * j < a.page_chunks) dst[i0 + 32 * j] = w[j];
  }
}

struct CompactWork {
  size_t bits, before, holes, movers, live, fine, bytes;
  int words;
};
CompactWork compact_layout(const avsg_pages* p) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  CompactWork w;
  w.words = (int)(((int64_t)p->num_pages + 31) / 32);
  w.bits = 0;
  w.before = w.bits + up((size_t)w.words * 4);
  w.holes = w.before + up((size_t)w.words * 4);
  w.movers = w.holes + up(((size_t)p->num_pages / 2 + 1) * 4);
  w.live = w.movers + up(((size_t)p->num_pages / 2 + 1) * 4);
  w.fine = w.live + 128;
  w.bytes = w.live + 256;
  static_assert(kMostPlanCtas * sizeof(int32_t) <= 128 && kCompactCluster <= kMostPlanCtas, "see fine");
  return w;
}

}  // namespace
}  // namespace avsg

using namespace avsg;

extern "C" int avsg_page_compact_workspace(const avsg_pages* p, size_t* bytes) {
  const int rc = check_pages(p);
  if (rc != AVSG_OK) return rc;
  if (!bytes) return AVSG_ERR_INVALID_ARG;
  *bytes = compact_layout(p).bytes;
  return AVSG_OK;
}

extern "C" int avsg_page_compact(const avsg_pages* p, const int32_t* d_shares, int32_t* d_shares_out,
                                 int32_t* d_tables_out, int32_t* d_free_out, int32_t* d_map, void* d_work,
                                 size_t work_bytes, void* stream) {
  int rc = check_pages(p);
  if (rc != AVSG_OK) return rc;
  if (!d_tables_out || !d_free_out || !d_map || !d_work || reinterpret_cast<uintptr_t>(d_work) % 256 ||
      (d_shares == nullptr) != (d_shares_out == nullptr))
    return AVSG_ERR_INVALID_ARG;
  if (p->max_pages > kMaxColumns) return AVSG_ERR_CAPACITY;
  const CompactWork w = compact_layout(p);
  if (work_bytes < w.bytes) return AVSG_ERR_CAPACITY;
  int dev = 0, sms = 0;
  rc = paged_device(p->d_k, &dev, &sms);
  if (rc != AVSG_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  unsigned char* work = static_cast<unsigned char*>(d_work);
  PackArgs a{};
  CompactArgs& c = a.c;
  c.R = p->num_requests;
  c.shift = page_shift_of(p->page_tokens);
  c.max_pages = p->max_pages;
  c.num_pages = p->num_pages;
  c.words = w.words;
  c.len = p->d_len;
  c.tables = p->d_tables;
  c.free_list = p->d_free;
  c.count = p->d_free_count;
  c.bits = reinterpret_cast<uint32_t*>(work + w.bits);
  c.before = reinterpret_cast<int32_t*>(work + w.before);
  c.holes = reinterpret_cast<int32_t*>(work + w.holes);
  c.movers = reinterpret_cast<int32_t*>(work + w.movers);
  c.live = reinterpret_cast<int32_t*>(work + w.live);
  c.fine = reinterpret_cast<int32_t*>(work + w.fine);
  c.err = reinterpret_cast<DevErr*>(p->d_error);
  a.num_layers = p->num_layers;
  a.page_chunks = (long long)p->num_kv_heads * p->page_tokens * p->head_dim / 8;
  a.layer_bytes = a.page_chunks * 16 * p->num_pages;
  a.k = static_cast<unsigned char*>(p->d_k);
  a.v = static_cast<unsigned char*>(p->d_v);
  a.shares = d_shares;
  a.shares_out = d_shares_out;
  a.tables_out = d_tables_out;
  a.free_out = d_free_out;
  a.map = d_map;
  // a warp for every 32 held entries, a thread for every word of the bitmap
  const int64_t most = (int64_t)c.R * c.max_pages > c.num_pages ? (int64_t)c.R * c.max_pages : c.num_pages;
  const bool small = c.num_pages <= kSmallPool;
  c.ctas = 1;
  while (c.ctas < kCompactCluster && c.ctas * kCompactThreads < most) c.ctas *= 2;
  // (a small pool: as many CTAs as the requests have warps; each reads the whole stack)
  const int rows = (c.R + kCompactThreads / 32 - 1) / (kCompactThreads / 32);
  if (small) c.ctas = rows < kMostPlanCtas ? rows : kMostPlanCtas;
  cudaError_t e =
      small ? launch_pdl(compact_plan_small_kernel, dim3(c.ctas), dim3(kCompactThreads), 0, st, c)
            : launch_pdl_cluster(c.ctas, compact_plan_kernel, dim3(c.ctas), dim3(kCompactThreads), 0, st, c);
  if (e == cudaSuccess) {
    const int64_t half = (c.num_pages + 1) / 2;            // no more pages move
    const int64_t warps = half * a.num_layers * 2 * ((a.page_chunks + kPackPiece - 1) / kPackPiece);
    const int64_t want = (warps + kPackThreads / 32 - 1) / (kPackThreads / 32);
    const int grid = want < 6 * sms ? (int)want : 6 * sms;
    e = launch_pdl(compact_move_kernel, dim3(grid), dim3(kPackThreads), 0, st, a);
  }
  return e == cudaSuccess ? AVSG_OK : AVSG_ERR_CUDA;
}
