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
// What bounds it.  The rows of the copied pages, 2 bytes moved per byte, and the latency of what is
// decided before and beside.  Three launches:
//   fork_check_kernel  one cluster: lengths, parents and ids checked, what gets
//                      copied listed, marks of the pages that change holders
//                      cleared, rows set aside that others still need after they are overwritten;
//   fork_copy_kernel   the whole GPU: the copies;
//   fork_write_kernel  one cluster, beside the copies (it waits for them at
//                      its end, so that what follows follows both):
//     count            gains and losses added to each page's mark, the last request that touches it noted
//     back             pages without a holder counted, piece by piece
//     write            shares, free stack, then tables and lengths
// with the hardware barriers of a cluster of up to 8 CTAs between the phases.  Whether the fork
// happens is one word, written by the check, and not the error word, which a call on another stream
// may change between two CTAs' reads: a CTA that left would leave the others to write into its shared memory.
// Only requests that become others are looked at, a row and its parent's side
// by side; where their rows agree (beams and samples of one prompt, but for
// the last pages) nothing is counted.  Nothing is written before every check has passed, but the check
// of the stack's room, which only wrong shares fail.  Sums and maxima of whole
// numbers decide everything, so that the result does not depend on an order.
// Measured: 8 samples of a prompt of 1000 tokens, one layer: 11.6 us; 256 beams
// through 16 layers, 64 MB read and written: 22.3 us (29.5 with the copies
// behind the tables); 96 samples of six prompts of up to 32768 tokens: 23 us
// (46 when every row of a changed count was walked).
#include <cooperative_groups.h>

#include <utility>

#include "avsg_paged.cuh"

namespace cg = cooperative_groups;

namespace avsg {
namespace {

constexpr int kForkThreads = 1024;         // of the check
constexpr int kWriteThreads = 512;         // of the write: they fit an SM beside the CTAs of the copy
constexpr int kForkCluster = 8;
constexpr int kItems = 8192;               // pieces of rows that the warps take in turn
constexpr int kLeastColumns = 128;         // columns of a piece, at least

struct ForkArgs {
  int R, shift, max_pages, num_pages;
  int cols, pieces;                        // columns of a piece, pieces of a row
  int beside;                              // a copy runs beside the write
  int32_t* len;
  const int32_t* parent;
  int32_t* tables;
  int32_t* free_list;
  int32_t* count;
  int32_t* shares;
  int32_t* delta;                          // [num_pages]
  int32_t* last;                           // [num_pages] the highest request that changes a page's count
  int32_t* aside;                          // [R][max_pages]
  int4* request;                           // [R] {length, parent, times, number of its copy or -1}
  int4* copies;                            // [R] {from, to, rows, 0}
  int32_t* num_copies;                     // {copies, whether any page changes holders, free pages, whether to go on}
  DevErr* err;
};

// Exclusive prefix over the block's threads and the sum (s_warp: one slot per warp).
__device__ __forceinline__ int fork_scan(int v, int* s_warp, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  auto inclusive = [&](int x) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += o;
    }
    return x;
  };
  const int inc = inclusive(v);
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  const int sums = inclusive(lane < warps ? s_warp[lane] : 0);
  *total = __shfl_sync(0xffffffffu, sums, 31);
  return (warp == 0 ? 0 : __shfl_sync(0xffffffffu, sums, warp - 1)) + inc - v;
}
static_assert(kForkThreads <= 1024 && kWriteThreads <= 1024, "fork_scan sums a warp's lanes");

// The requests as both clusters see them.
struct ForkView {
  const ForkArgs& a;
  const int4* s_request;

  __device__ int parent(int r) const { return s_request[r].y; }
  __device__ int times(int r) const { return s_request[r].z; }
  __device__ int full(int r) const { return s_request[r].x >> a.shift; }
  __device__ int held(int r) const { return (s_request[r].x + (1 << a.shift) - 1) >> a.shift; }
  // end of the piece that begins at column x0 of a row with this many
  __device__ int piece_end(int x0, int columns) const { return columns - x0 > a.cols ? x0 + a.cols : columns; }

  // What request r lets go of and takes hold of, in the columns of its piece.  A partly filled last
  // page is nobody else's: it changes hands, or goes with a row that nobody goes on with.
  template <typename F>
  __device__ void each_column(int i, F&& f) const {
    const int lane = threadIdx.x & 31;
    const int r = i / a.pieces, q = parent(r), x0 = (i - r * a.pieces) * a.cols;
    if (q == r) return;
    int lose = times(r) == 0 ? held(r) : full(r), gain = q < 0 ? 0 : full(q);
    const int x1 = piece_end(x0, max(lose, gain));
    const int32_t* mine = a.tables + (size_t)r * a.max_pages;
    const int32_t* theirs = a.tables + (size_t)max(q, 0) * a.max_pages;
    lose = min(lose, x1);
    gain = min(gain, x1);
    // (128 columns of both rows on their way at once: beside the copies a load takes 2 to 3 us)
    for (int x = x0; x < x1; x += 128) {
      int32_t from[4], to[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int at = x + 32 * y + lane;
        from[y] = at < lose ? mine[at] : -1;
        to[y] = at < gain ? theirs[at] : -1;
      }
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int at = x + 32 * y + lane;
        if (x + 32 * y < x1) f(r, at, at < lose, from[y], at < gain, to[y]);
      }
    }
  }
};

__global__ void __launch_bounds__(kForkThreads) fork_check_kernel(ForkArgs a) {
  extern __shared__ int4 s_request[];      // [R], then [R] the lowest child
  __shared__ int s_warp[kForkThreads / 32], s_any[kForkCluster];
  int32_t* s_heir = reinterpret_cast<int32_t*>(s_request + a.R);
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = rank * (kForkThreads / 32) + (tid >> 5), warps = ctas * (kForkThreads / 32);
  const int page_mask = (1 << a.shift) - 1;
  const int items = a.R * a.pieces;
  auto started = cluster.barrier_arrive();  // (s_any is written by other CTAs)

  for (int r = tid; r < a.R; r += kForkThreads) {
    s_request[r].z = 0;
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
    s_request[r].x = len;
    s_request[r].y = q;
    if (!code && q >= 0) {
      atomicAdd(&s_request[q].z, 1);
      if (q != r) atomicMin(&s_heir[q], r);
    }
  }
  if (!bad && tid == 0 && (count < 0 || count > a.num_pages)) bad = AVSG_ERR_BAD_SELECTION;
  if (bad && rank == 0) raise_error(a.err, bad, bad_r, -1);
  ok = !__syncthreads_or(!ok || bad);
  griddep_launch();
  const ForkView v{a, s_request};
  // Which requests get a copy: those whose parent's last page stays with another one.
  const int per = (a.R + kForkThreads - 1) / kForkThreads;
  const int r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);
  auto copied = [&](int r) {
    const int q = v.parent(r);
    return q >= 0 && q != r && (s_request[q].x & page_mask) != 0 && (v.parent(q) == q || s_heir[q] != r);
  };
  int mine = 0, num_copies;
  if (ok)
    for (int r = r0; r < r1; ++r) mine += copied(r);
  int before = fork_scan(mine, s_warp, &num_copies);
  if (ok && num_copies > count) {
    if (rank == 0 && tid == 0) raise_error(a.err, AVSG_ERR_CAPACITY, -1, -1);
    ok = false;
  }
  if (ok)
    for (int r = r0; r < r1; ++r) s_request[r].w = copied(r) ? before++ : -1;
  __syncthreads();

  bool any = false, wrong = false;
  if (ok) {
    for (int r = rank * kForkThreads + tid; r < a.R; r += ctas * kForkThreads) {
      const int4 me = s_request[r];
      a.request[r] = me;
      const int q = me.y;
      if (q < 0 || q == r) continue;
      const int len = s_request[q].x;
      if ((len & page_mask) == 0) continue;
      const int32_t from = a.tables[(size_t)q * a.max_pages + (len >> a.shift)];
      if (from < 0 || from >= a.num_pages) {
        raise_error(a.err, AVSG_ERR_BAD_SELECTION, q, len >> a.shift);
        wrong = true;
      }
      if (me.w >= 0) {
        const int to = a.free_list[count - 1 - me.w];
        if (to < 0 || to >= a.num_pages) {
          raise_error(a.err, AVSG_ERR_BAD_SELECTION, -1, count - 1 - me.w);
          wrong = true;
        }
        a.copies[me.w] = make_int4(from, to, len & page_mask, 0);
      }
    }
    for (int i = warp; i < items; i += warps) {
      v.each_column(i, [&](int r, int x, bool loses, int32_t from, bool gains, int32_t to) {
        if (loses && (from < 0 || from >= a.num_pages)) {
          raise_error(a.err, AVSG_ERR_BAD_SELECTION, r, x);
          wrong = true;
        } else if (gains && (to < 0 || to >= a.num_pages)) {
          raise_error(a.err, AVSG_ERR_BAD_SELECTION, v.parent(r), x);
          wrong = true;
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
      if (v.parent(q) == q || v.times(q) == 0) continue;
      const int x0 = (i - q * a.pieces) * a.cols, x1 = v.piece_end(x0, v.held(q));
      for (int x = x0 + lane; x < x1; x += 32)
        a.aside[(size_t)q * a.max_pages + x] = a.tables[(size_t)q * a.max_pages + x];
    }
  }
  any = __syncthreads_or(any);
  ok = !__syncthreads_or(!ok || wrong);
  cluster.barrier_wait(std::move(started));
  if (tid == 0) *cluster.map_shared_rank(&s_any[rank], 0) = ok ? any : -1;
  cluster.sync();
  if (rank == 0 && tid == 0) {
    for (int c = 1; c < ctas; ++c) {
      any |= s_any[c] > 0;
      ok &= s_any[c] >= 0;
    }
    a.num_copies[0] = num_copies;
    a.num_copies[1] = any;
    a.num_copies[2] = count;
    a.num_copies[3] = ok;
  }
}

__global__ void __launch_bounds__(kWriteThreads, 3) fork_write_kernel(ForkArgs a) {
  extern __shared__ int4 s_request[];      // [R], then [R * pieces] pages that the pieces give back
  __shared__ int s_warp[kWriteThreads / 32];
  int32_t* s_back = reinterpret_cast<int32_t*>(s_request + a.R);
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = rank * (kWriteThreads / 32) + (tid >> 5), warps = ctas * (kWriteThreads / 32);
  const int items = a.R * a.pieces;
  // (every CTA of a copy has waited for the check before this one may begin)
  if (!a.beside) griddep_wait();
  // every CTA sees the same words: all go on or none
  const int num_copies = __ldcg(a.num_copies), count = __ldcg(a.num_copies + 2);
  const bool any = __ldcg(a.num_copies + 1) != 0;
  if (__ldcg(a.num_copies + 3) == 0) {
    griddep_wait();
    return;
  }
  for (int r = tid; r < a.R; r += kWriteThreads) s_request[r] = __ldcg(a.request + r);
  __syncthreads();
  const ForkView v{a, s_request};
  // (request, whether it lets go): at most one of a page's marks
  auto mark = [](int r, bool loses) { return 2 * r + (loses ? 1 : 0); };

  int total = 0;
  const int left = count - num_copies;
  bool ok = true;
  if (any) {
    // count
    for (int i = warp; i < items; i += warps)
      v.each_column(i, [&](int r, int, bool loses, int32_t from, bool gains, int32_t to) {
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
    for (int i = warp; i < items; i += warps) {
      int n = 0;
      v.each_column(i, [&](int r, int, bool loses, int32_t from, bool, int32_t to) {
        if (!loses || from == to) return;
        const int last = __ldcg(a.last + from), delta = __ldcg(a.delta + from), shares = a.shares[from];
        n += last == mark(r, true) && shares + delta < 0;
      });
      n = __reduce_add_sync(0xffffffffu, n);
      if (lane < ctas) *cluster.map_shared_rank(&s_back[i], lane) = n;
    }
    cluster.sync();
    const int each = (items + kWriteThreads - 1) / kWriteThreads;
    const int i0 = min(items, tid * each), i1 = min(items, i0 + each);
    int n = 0;
    for (int i = i0; i < i1; ++i) n += s_back[i];
    int at = fork_scan(n, s_warp, &total);
    for (int i = i0; i < i1; ++i) {
      const int k = s_back[i];
      s_back[i] = at;
      at += k;
    }
    if ((long long)left + total > a.num_pages) {
      if (rank == 0 && tid == 0) raise_error(a.err, AVSG_ERR_CAPACITY, -1, -1);
      ok = false;
    }
    __syncthreads();
    // write: shares and the stack (the reverse order of taking)
    if (ok)
      for (int i = warp; i < items; i += warps) {
        int at = s_back[i];
        v.each_column(i, [&](int r, int, bool loses, int32_t from, bool gains, int32_t to) {
          gains = gains && from != to;
          loses = loses && from != to;
          const int last_to = gains ? __ldcg(a.last + to) : -1, last_from = loses ? __ldcg(a.last + from) : -1;
          const int add_to = gains ? __ldcg(a.delta + to) : 0, add_from = loses ? __ldcg(a.delta + from) : 0;
          const bool own = loses && last_from == mark(r, true);
          if (gains && last_to == mark(r, false)) a.shares[to] += add_to;
          const int now = own ? a.shares[from] + add_from : 0;
          const unsigned gone = __ballot_sync(0xffffffffu, own && now < 0);
          if (own) a.shares[from] = max(now, 0);
          if (own && now < 0) a.free_list[left + total - 1 - (at + __popc(gone & ((1u << lane) - 1)))] = from;
          at += __popc(gone);
        });
      }
  }
  cluster.sync();                          // (rows are read above, and a CTA's s_back written by others)
  // write: tables and lengths
  if (ok) {
    for (int i = warp; i < items; i += warps) {
      const int r = i / a.pieces, q = v.parent(r);
      if (q < 0 || q == r) continue;
      const int x0 = (i - r * a.pieces) * a.cols, x1 = v.piece_end(x0, v.held(q));
      const int32_t* from = (v.parent(q) == q ? a.tables : a.aside) + (size_t)q * a.max_pages;
      const int own = s_request[r].w >= 0 ? v.full(q) : -1;
      int32_t* to = a.tables + (size_t)r * a.max_pages;
      for (int x = x0 + lane; x < x1; x += 128) {
        int32_t id[4];
#pragma unroll
        for (int y = 0; y < 4; ++y)
          if (x + 32 * y < x1) id[y] = __ldcg(from + x + 32 * y);
#pragma unroll
        for (int y = 0; y < 4; ++y)
          if (x + 32 * y < x1) to[x + 32 * y] = id[y];
      }
      if (own >= x0 && own < x1) {
        __syncwarp();                      // (after the parent's page in that column)
        if (lane == 0) to[own] = __ldcg(&a.copies[s_request[r].w].y);
      }
    }
    for (int r = rank * kWriteThreads + tid; r < a.R; r += ctas * kWriteThreads) {
      const int q = v.parent(r);
      if (q != r) a.len[r] = q < 0 ? 0 : s_request[q].x;
    }
    if (rank == 0 && tid == 0) *a.count = left + total;
  }
  griddep_wait();
}

struct ForkCopyArgs {
  int H, shift, num_layers;
  int chunks;                              // 16-byte chunks of one row
  long long layer_bytes;
  unsigned char* k;
  unsigned char* v;
  const int4* copies;
  const int32_t* num_copies;
};

constexpr int kCopyThreads = 256;
constexpr int kCopyBatch = 4;              // 16-byte chunks in flight per thread
constexpr int kCopyBlocks = 4;             // CTAs per SM

// A warp takes the rows of one page's kv-head in one layer of K or V: they are contiguous.
__global__ void __launch_bounds__(kCopyThreads, 6) fork_copy_kernel(ForkCopyArgs a) {
  griddep_wait();
  griddep_launch();
  if (a.num_copies[3] == 0) return;
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
  size_t delta, last, aside, request, copies, num, bytes;
  int cols, pieces;
};
ForkWork fork_layout(const avsg_pages* p) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t R = p->num_requests;
  ForkWork w;
  // (their counts lie in every CTA's shared memory)
  const int64_t fit = kItems / R < 1 ? 1 : kItems / (int64_t)R;
  int64_t cols = (p->max_pages + fit - 1) / fit;
  if (cols < kLeastColumns) cols = kLeastColumns;
  w.cols = (int)cols;
  w.pieces = (int)((p->max_pages + cols - 1) / cols);
  w.delta = 0;
  w.last = w.delta + up((size_t)p->num_pages * 4);
  w.aside = w.last + up((size_t)p->num_pages * 4);
  w.request = w.aside + up(R * p->max_pages * 4);
  w.copies = w.request + up(R * sizeof(int4));
  w.num = w.copies + up(R * sizeof(int4));
  w.bytes = w.num + 256;
  return w;
}

SmemLimit g_check_smem, g_write_smem;

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
  a.request = reinterpret_cast<int4*>(work + w.request);
  a.copies = reinterpret_cast<int4*>(work + w.copies);
  a.num_copies = reinterpret_cast<int32_t*>(work + w.num);
  a.err = reinterpret_cast<DevErr*>(p->d_error);
  a.beside = p->page_tokens > 1;
  const size_t check_smem = (size_t)a.R * (sizeof(int4) + sizeof(int32_t));
  const size_t write_smem = (size_t)a.R * (sizeof(int4) + a.pieces * sizeof(int32_t));
  int ctas = 1;
  while (ctas < kForkCluster && (int64_t)ctas * (kForkThreads / 32) < (int64_t)a.R * a.pieces) ctas *= 2;
  cudaError_t e = g_check_smem.raise(reinterpret_cast<const void*>(fork_check_kernel), check_smem, dev);
  if (e == cudaSuccess) e = g_write_smem.raise(reinterpret_cast<const void*>(fork_write_kernel), write_smem, dev);
  if (e == cudaSuccess)
    e = launch_pdl_cluster(ctas, fork_check_kernel, dim3(ctas), dim3(kForkThreads), check_smem, st, a);
  if (e == cudaSuccess && a.beside) {
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
    // (no more CTAs than the copies of all requests have units)
    const int64_t most = ((int64_t)a.R * c.num_layers * 2 * c.H + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
    const int grid = most < kCopyBlocks * sms ? (int)most : kCopyBlocks * sms;
    e = launch_pdl(fork_copy_kernel, dim3(grid), dim3(kCopyThreads), 0, st, c);
  }
  if (e == cudaSuccess)
    e = launch_pdl_cluster(ctas, fork_write_kernel, dim3(ctas), dim3(kWriteThreads), write_smem, st, a);
  return e == cudaSuccess ? AVSG_OK : AVSG_ERR_CUDA;
}
