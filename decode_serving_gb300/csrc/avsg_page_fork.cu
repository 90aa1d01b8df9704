// avsg_page_fork: requests continue as copies of others, with shared pages.
//
// Request r becomes what request q = parent[r] was: the full pages of the old
// row q are held by both, its partly filled last page (if it has one) stays
// with q or, if q goes on as something else, with the lowest of its children,
// and is copied for the others.  A request that becomes another one lets go of its old row's full
// pages (and of the last one, if nobody goes on with its row) and takes hold of q's;
// a page that both rows have in the same place changes nothing.  So
//     shares' = shares + (requests that take hold of the page) - (that let go of it)
// holders beyond the first, and the page is free when that is -1.
//
// What bounds it.  The rows of the copied pages: 2 bytes moved per byte, by
// fork_copy_kernel.  What comes before, tables and counts, is latency: one cluster of up to
// 8 CTAs whose hardware barriers part the phases
//   check      lengths, parents, ids; marks of the pages that change holders
//              cleared; rows that others still need after they are overwritten set aside
//   count      gains and losses added to each page's mark, the last request that touches it noted
//   back       pages without a holder counted, piece by piece
//   write      shares, free stack
//   write      tables, lengths
// Only requests that become others are looked at, a row and its parent's side
// by side; where their rows agree (beams and samples of one prompt, but for
// the last pages) nothing is counted, and where all of them do, the middle three are left out.
// Nothing is written before every check has passed.  Sums and maxima of whole
// numbers decide everything, so that the result does not depend on an order.
#include <cooperative_groups.h>

#include <utility>

#include "avsg_paged.cuh"

namespace cg = cooperative_groups;

namespace avsg {
namespace {

constexpr int kForkThreads = 1024;
constexpr int kForkCluster = 8;
constexpr int kItems = 8192;               // pieces of rows that the warps take in turn
constexpr int kLeastColumns = 128;         // columns of a piece, at least

struct ForkArgs {
  int R, shift, max_pages, num_pages;
  int cols, pieces;                        // columns of a piece, pieces of a row
  int32_t* len;
  const int32_t* parent;
  int32_t* tables;
  int32_t* free_list;
  int32_t* count;
  int32_t* shares;
  int32_t* delta;                          // [num_pages]
  int32_t* last;                           // [num_pages] the highest row that changes a page's count
  int32_t* aside;                          // [R][max_pages]
  int32_t* back;                           // [R * pieces] pages that a piece gives back
  int4* copies;                            // [R] {from, to, rows, 0}
  int32_t* num_copies;
  DevErr* err;
};

__global__ void __launch_bounds__(kForkThreads) page_fork_kernel(ForkArgs a) {
  extern __shared__ int32_t s_mem[];
  __shared__ long long s_warp[kForkThreads / 32];
  __shared__ int s_any[kForkCluster];
  int32_t* s_len = s_mem;                  // [R] each
  int32_t* s_parent = s_len + a.R;
  int32_t* s_times = s_parent + a.R;
  int32_t* s_heir = s_times + a.R;         // the lowest child
  int32_t* s_copy = s_heir + a.R;          // number of the request's copy, or -1
  int32_t* s_at = s_copy + a.R;            // [R * pieces] pages given back by the pieces before
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = rank * (kForkThreads / 32) + (tid >> 5), warps = ctas * (kForkThreads / 32);
  const int page_mask = (1 << a.shift) - 1;
  const int items = a.R * a.pieces;
  auto started = cluster.barrier_arrive();  // (s_any is written by other CTAs)

  for (int r = tid; r < a.R; r += kForkThreads) {
    s_times[r] = 0;
    s_heir[r] = a.R;
  }
  griddep_wait();
  bool ok = load_err(a.err) == 0;
  const int count = *a.count;
  __syncthreads();
  int bad = 0, bad_r = -1;
  for (int r = tid; r < a.R; r += kForkThreads) {
    const int len = a.len[r], q = a.parent[r];
    int code = 0;
    if (len < 0 || q < -1 || q >= a.R) code = AVSG_ERR_BAD_SELECTION;
    else if ((((long long)len + page_mask) >> a.shift) > a.max_pages) code = AVSG_ERR_CAPACITY;
    if (code && !bad) {
      bad = code;
      bad_r = r;
    }
    s_len[r] = len;
    s_parent[r] = q;
    if (!code && q >= 0) {
      atomicAdd(&s_times[q], 1);
      if (q != r) atomicMin(&s_heir[q], r);
    }
  }
  if (!bad && tid == 0 && (count < 0 || count > a.num_pages)) bad = AVSG_ERR_BAD_SELECTION;
  if (bad && rank == 0) raise_error(a.err, bad, bad_r, -1);
  ok = !__syncthreads_or(!ok || bad);
  // Which requests get a copy: those whose parent's last page stays with another one.
  const int per = (a.R + kForkThreads - 1) / kForkThreads;
  const int r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);
  auto copied = [&](int r) {
    const int q = s_parent[r];
    return q >= 0 && q != r && (s_len[q] & page_mask) != 0 && (s_parent[q] == q || s_heir[q] != r);
  };
  long long mine = 0, num;
  if (ok)
    for (int r = r0; r < r1; ++r) mine += copied(r);
  long long before = block_exclusive(mine, s_warp, &num);
  const int num_copies = (int)num;
  if (ok && num_copies > count) {
    if (rank == 0 && tid == 0) raise_error(a.err, AVSG_ERR_CAPACITY, -1, -1);
    ok = false;
  }
  if (ok)
    for (int r = r0; r < r1; ++r) s_copy[r] = copied(r) ? (int)before++ : -1;
  __syncthreads();
  auto held = [&](int q) { return (s_len[q] + page_mask) >> a.shift; };
  // end of the piece that begins at column x0 of a row with this many
  auto piece_end = [&](int x0, int columns) { return columns - x0 > a.cols ? x0 + a.cols : columns; };

  // What request r lets go of and takes hold of, in the columns of its piece.  A partly filled last
  // page is nobody else's: it changes hands, or goes with a row that nobody goes on with.
  auto each_column = [&](int i, auto&& f) {
    const int r = i / a.pieces, q = s_parent[r], x0 = (i - r * a.pieces) * a.cols;
    if (q == r) return;
    const int lose = s_times[r] == 0 ? held(r) : s_len[r] >> a.shift, gain = q < 0 ? 0 : s_len[q] >> a.shift;
    const int x1 = piece_end(x0, max(lose, gain));
    const int32_t* mine = a.tables + (size_t)r * a.max_pages;
    const int32_t* theirs = a.tables + (size_t)max(q, 0) * a.max_pages;
#pragma unroll 2
    for (int x = x0; x < x1; x += 32) {
      const int at = x + lane;
      const int32_t from = at < lose && at < x1 ? mine[at] : -1, to = at < gain && at < x1 ? theirs[at] : -1;
      f(r, at, at < lose && at < x1, from, at < gain && at < x1, to);
    }
  };
  // (request, whether it lets go): at most one of a page's marks
  auto mark = [](int r, bool loses) { return 2 * r + (loses ? 1 : 0); };

  // check
  bool any = false;
  if (ok) {
    for (int r = rank * kForkThreads + tid; r < a.R; r += ctas * kForkThreads) {
      const int q = s_parent[r];
      if (q < 0 || q == r || (s_len[q] & page_mask) == 0) continue;
      const int32_t last = a.tables[(size_t)q * a.max_pages + (s_len[q] >> a.shift)];
      if (last < 0 || last >= a.num_pages) raise_error(a.err, AVSG_ERR_BAD_SELECTION, q, s_len[q] >> a.shift);
      if (s_copy[r] >= 0) {
        const int to = a.free_list[count - 1 - s_copy[r]];
        if (to < 0 || to >= a.num_pages) raise_error(a.err, AVSG_ERR_BAD_SELECTION, -1, count - 1 - s_copy[r]);
        a.copies[s_copy[r]] = make_int4(last, to, s_len[q] & page_mask, 0);
      }
    }
    if (rank == 0 && tid == 0) *a.num_copies = num_copies;
    for (int i = warp; i < items; i += warps) {
      each_column(i, [&](int r, int x, bool loses, int32_t from, bool gains, int32_t to) {
        if (loses && (from < 0 || from >= a.num_pages)) {
          raise_error(a.err, AVSG_ERR_BAD_SELECTION, r, x);
        } else if (gains && (to < 0 || to >= a.num_pages)) {
          raise_error(a.err, AVSG_ERR_BAD_SELECTION, s_parent[r], x);
        } else if (from != to) {
          any = true;
          if (loses) {
            a.delta[from] = 0;
            a.last[from] = -1;
          }
          if (gains) {
            a.delta[to] = 0;
            a.last[to] = -1;
          }
        }
      });
      const int q = i / a.pieces;
      if (s_parent[q] == q || s_times[q] == 0) continue;
      const int x0 = (i - q * a.pieces) * a.cols, x1 = piece_end(x0, held(q));
      for (int x = x0 + lane; x < x1; x += 32)
        a.aside[(size_t)q * a.max_pages + x] = a.tables[(size_t)q * a.max_pages + x];
    }
    __threadfence();
  }
  any = __syncthreads_or(any);
  cluster.barrier_wait(std::move(started));
  if (tid < ctas) *cluster.map_shared_rank(&s_any[rank], tid) = any;
  cluster.sync();
  ok = !__syncthreads_or(!ok || load_err(a.err) != 0);
  // (every CTA sees the same words, so all go on or none; those that stop keep the barriers)
  any = false;
  for (int c = 0; c < ctas; ++c) any |= s_any[c] != 0;

  long long total = 0;
  const long long left = (long long)count - num_copies;
  if (any) {
    // count
    if (ok)
      for (int i = warp; i < items; i += warps)
        each_column(i, [&](int r, int, bool loses, int32_t from, bool gains, int32_t to) {
          if (from == to) return;
          if (loses) {
            atomicAdd(a.delta + from, -1);
            atomicMax(a.last + from, mark(r, true));
          }
          if (gains) {
            atomicAdd(a.delta + to, 1);
            atomicMax(a.last + to, mark(r, false));
          }
        });
    __threadfence();
    cluster.sync();
    // back: a page that goes is given back by the last request that held it
    if (ok)
      for (int i = warp; i < items; i += warps) {
        int n = 0;
        each_column(i, [&](int r, int, bool loses, int32_t from, bool, int32_t to) {
          n += loses && from != to && __ldcg(a.last + from) == mark(r, true) &&
               a.shares[from] + __ldcg(a.delta + from) < 0;
        });
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) a.back[i] = n;
      }
    __threadfence();
    cluster.sync();
    const int each = (items + kForkThreads - 1) / kForkThreads;
    const int i0 = min(items, tid * each), i1 = min(items, i0 + each);
    long long n = 0;
    if (ok)
      for (int i = i0; i < i1; ++i) n += __ldcg(a.back + i);
    long long at = block_exclusive(n, s_warp, &total);
    if (ok)
      for (int i = i0; i < i1; ++i) {
        s_at[i] = (int)at;
        at += __ldcg(a.back + i);
      }
    if (ok && left + total > a.num_pages) {
      if (rank == 0 && tid == 0) raise_error(a.err, AVSG_ERR_CAPACITY, -1, -1);
      ok = false;
    }
    __syncthreads();
  }
  griddep_launch();
  // write: shares and the stack (the reverse order of taking)
  if (ok && any)
    for (int i = warp; i < items; i += warps) {
      int at = s_at[i];
      each_column(i, [&](int r, int, bool loses, int32_t from, bool gains, int32_t to) {
        const bool own_to = gains && from != to && __ldcg(a.last + to) == mark(r, false);
        if (own_to) a.shares[to] += __ldcg(a.delta + to);
        const bool own = loses && from != to && __ldcg(a.last + from) == mark(r, true);
        const int now = own ? a.shares[from] + __ldcg(a.delta + from) : 0;
        const unsigned gone = __ballot_sync(0xffffffffu, own && now < 0);
        if (own) a.shares[from] = max(now, 0);
        if (own && now < 0)
          a.free_list[left + total - 1 - (at + __popc(gone & ((1u << lane) - 1)))] = from;
        at += __popc(gone);
      });
    }
  cluster.sync();
  // write: tables and lengths
  if (!ok) return;
  for (int i = warp; i < items; i += warps) {
    const int r = i / a.pieces, q = s_parent[r];
    if (q < 0 || q == r) continue;
    const int x0 = (i - r * a.pieces) * a.cols, x1 = piece_end(x0, held(q));
    const int32_t* from = (s_parent[q] == q ? a.tables : a.aside) + (size_t)q * a.max_pages;
    const int own = s_copy[r] >= 0 ? s_len[q] >> a.shift : -1;
#pragma unroll 4
    for (int x = x0 + lane; x < x1; x += 32)
      a.tables[(size_t)r * a.max_pages + x] = x == own ? __ldcg(&a.copies[s_copy[r]].y) : __ldcg(from + x);
  }
  for (int r = rank * kForkThreads + tid; r < a.R; r += ctas * kForkThreads) {
    const int q = s_parent[r];
    if (q != r) a.len[r] = q < 0 ? 0 : s_len[q];
  }
  if (rank == 0 && tid == 0) *a.count = (int)(left + total);
}

struct ForkCopyArgs {
  int H, shift, num_layers;
  int chunks;                              // 16-byte chunks of one row
  long long layer_bytes;
  unsigned char* k;
  unsigned char* v;
  const int4* copies;
  const int32_t* num_copies;
  DevErr* err;
};

constexpr int kCopyThreads = 256;
constexpr int kCopyBatch = 4;              // 16-byte chunks in flight per thread

// A warp takes the rows of one page's kv-head in one layer of K or V: they are contiguous.
__global__ void __launch_bounds__(kCopyThreads) fork_copy_kernel(ForkCopyArgs a) {
  griddep_wait();
  if (load_err(a.err) != 0) return;
  const int lane = threadIdx.x & 31;
  const long long units = (long long)*a.num_copies * a.num_layers * 2 * a.H;
  const long long head_bytes = (long long)(a.chunks * 16) << a.shift;
  const long long step = (long long)gridDim.x * (kCopyThreads / 32);
  for (long long u = (long long)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); u < units; u += step) {
    const int h = (int)(u % a.H);
    const long long x = u / a.H;
    const int kv = (int)(x & 1), layer = (int)((x >> 1) % a.num_layers), n = (int)((x >> 1) / a.num_layers);
    const int4 c = a.copies[n];
    unsigned char* base = (kv ? a.v : a.k) + layer * a.layer_bytes + h * head_bytes;
    const uint4* from = reinterpret_cast<const uint4*>(base + c.x * head_bytes * a.H);
    uint4* to = reinterpret_cast<uint4*>(base + c.y * head_bytes * a.H);
    const int end = c.z * a.chunks;
    for (int i0 = lane; i0 < end; i0 += 32 * kCopyBatch) {
      uint4 w[kCopyBatch];
#pragma unroll
      for (int j = 0; j < kCopyBatch; ++j)
        if (i0 + 32 * j < end) w[j] = __ldcs(from + i0 + 32 * j);
#pragma unroll
      for (int j = 0; j < kCopyBatch; ++j)
        if (i0 + 32 * j < end) to[i0 + 32 * j] = w[j];
    }
  }
}

struct ForkWork {
  size_t delta, last, aside, back, copies, num, bytes;
  int cols, pieces;
};
ForkWork fork_layout(const avsg_pages* p) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t R = p->num_requests;
  ForkWork w;
  // as many pieces as fit the shared memory of a CTA
  const int64_t fit = kItems / R < 1 ? 1 : kItems / (int64_t)R;
  int64_t cols = (p->max_pages + fit - 1) / fit;
  if (cols < kLeastColumns) cols = kLeastColumns;
  w.cols = (int)cols;
  w.pieces = (int)((p->max_pages + cols - 1) / cols);
  w.delta = 0;
  w.last = w.delta + up((size_t)p->num_pages * 4);
  w.aside = w.last + up((size_t)p->num_pages * 4);
  w.back = w.aside + up(R * p->max_pages * 4);
  w.copies = w.back + up(R * w.pieces * 4);
  w.num = w.copies + up(R * sizeof(int4));
  w.bytes = w.num + 256;
  return w;
}

SmemLimit g_fork_smem;

}  // namespace
}  // namespace avsg

using namespace avsg;

extern "C" int avsg_page_fork_workspace(const avsg_pages* p, size_t* bytes) {
  const int rc = check_pages(p);
  if (rc != AVSG_OK) return rc;
  if (!bytes) return AVSG_ERR_INVALID_ARG;
  if (p->max_pages > kMaxColumns) return AVSG_ERR_CAPACITY;
  *bytes = fork_layout(p).bytes;
  return AVSG_OK;
}

extern "C" int avsg_page_fork(const avsg_pages* p, const int32_t* d_parent, int32_t* d_shares, void* d_work,
                              size_t work_bytes, void* stream) {
  int rc = check_pages(p);
  if (rc != AVSG_OK) return rc;
  if (!d_parent || !d_shares || !d_work || reinterpret_cast<uintptr_t>(d_work) % 256) return AVSG_ERR_INVALID_ARG;
  if (p->max_pages > kMaxColumns) return AVSG_ERR_CAPACITY;
  const ForkWork w = fork_layout(p);
  if (work_bytes < w.bytes) return AVSG_ERR_CAPACITY;
  int dev = 0, sms = 0;
  rc = paged_device(p->d_k, &dev, &sms);
  if (rc != AVSG_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  unsigned char* work = static_cast<unsigned char*>(d_work);
  ForkArgs a{};
  a.R = p->num_requests;
  a.shift = page_shift_of(p->page_tokens);
  a.max_pages = p->max_pages;
  a.num_pages = p->num_pages;
  a.cols = w.cols;
  a.pieces = w.pieces;
  a.len = p->d_len;
  a.parent = d_parent;
  a.tables = p->d_tables;
  a.free_list = p->d_free;
  a.count = p->d_free_count;
  a.shares = d_shares;
  a.delta = reinterpret_cast<int32_t*>(work + w.delta);
  a.last = reinterpret_cast<int32_t*>(work + w.last);
  a.aside = reinterpret_cast<int32_t*>(work + w.aside);
  a.back = reinterpret_cast<int32_t*>(work + w.back);
  a.copies = reinterpret_cast<int4*>(work + w.copies);
  a.num_copies = reinterpret_cast<int32_t*>(work + w.num);
  a.err = reinterpret_cast<DevErr*>(p->d_error);
  const size_t smem = (5 * (size_t)a.R + (size_t)a.R * a.pieces) * sizeof(int32_t);
  int ctas = 1;
  while (ctas < kForkCluster && (int64_t)ctas * (kForkThreads / 32) < (int64_t)a.R * a.pieces) ctas *= 2;
  cudaError_t e = g_fork_smem.raise(reinterpret_cast<const void*>(page_fork_kernel), smem, dev);
  if (e == cudaSuccess) e = launch_pdl_cluster(ctas, page_fork_kernel, dim3(ctas), dim3(kForkThreads), smem, st, a);
  if (e == cudaSuccess && p->page_tokens > 1) {
    ForkCopyArgs c{};
    c.H = p->num_kv_heads;
    c.shift = a.shift;
    c.num_layers = p->num_layers;
    c.chunks = p->head_dim * 2 / 16;
    c.layer_bytes = (long long)p->num_pages * p->num_kv_heads * p->page_tokens * p->head_dim * 2;
    c.k = static_cast<unsigned char*>(p->d_k);
    c.v = static_cast<unsigned char*>(p->d_v);
    c.copies = a.copies;
    c.num_copies = a.num_copies;
    c.err = a.err;
    // (no more CTAs than the copies of all requests have units)
    const int64_t most = ((int64_t)a.R * c.num_layers * 2 * c.H + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
    const int grid = most < 6 * sms ? (int)most : 6 * sms;
    e = launch_pdl(fork_copy_kernel, dim3(grid), dim3(kCopyThreads), 0, st, c);
  }
  return e == cudaSuccess ? AVSG_OK : AVSG_ERR_CUDA;
}
