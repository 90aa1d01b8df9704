// avsg_page_plan and avsg_tree_keep: the block tables of a paged device cache,
// built, extended and shrunk on the GPU from the requests' lengths.
//
// Plan.  Request r holds held = ceil(len / page) pages and needs
// need = ceil((len + new) / page); with base = the exclusive sum of
// need - held over the requests, its page x >= held is
// free[count - 1 - (base + x - held)]: the free list is a stack taken from the
// top in request order.  Token i of the request lies at position p = len + i,
// in slot page(p / page) * page + p % page.
// Keep.  Row len + path[i] moves to len + i in every layer; the pages past the
// new length go back on the stack in the reverse order of taking, so that a
// step whose drafts are all rejected leaves the stack as it found it.
//
// What bounds them: latency.  A plan of 8 requests moves under 200 bytes, one
// of 100 000 tokens under 2 MB.  Hence no scan kernel before them: every CTA
// scans all lengths itself (a few loads a thread that hit the L2), checks
// everything, so that all decide alike, and writes its share.  No CTA writes
// anything unless all checks pass.
// The outputs may alias the inputs.  The plan writes only one word that others
// read, the free count: its CTAs count themselves as they finish (in the error
// array's fourth word, which wraps to 0), and the last one writes it.  The
// keep also writes lengths and the stack: it is one cluster of up to 8 CTAs,
// whose hardware barriers separate reads from writes.
// Measured: a plan of 8 requests 5.5 us, in a graph too, one of 509 requests and
// 100 000 tokens 8.0 us (25 us when one cluster wrote all tokens); a keep of 4
// requests 7.4 us (two launches), of 64 requests through 16 layers 12.9 us.
// Every CTA of a plan checks every page that is taken, which grows with tokens
// times CTAs where pages hold one token.
#include <cooperative_groups.h>

#include "avsg_paged.cuh"

namespace cg = cooperative_groups;

namespace avsg {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanTokensPerCta = 2048;  // tokens per CTA: one round of 4 a thread
constexpr int kPlanCluster = 8;

// Largest r with start[r] <= x, start non-decreasing, start[0] = 0, x < start[n].
__device__ __forceinline__ int find_request(const int32_t* start, int n, int x) {
  int lo = 0, hi = n;  // start[lo] <= x < start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

struct PlanArgs {
  int R, shift, max_pages, num_pages, capacity, num_mask;
  int wide;                      // slot and pos are 16-byte aligned
  const int32_t* len;
  const int32_t* fresh;
  const unsigned long long* mask;
  int32_t* tables;
  const int32_t* free_list;
  const int32_t* count;
  int32_t* count_out;
  int32_t* first;
  int32_t* slot;
  int32_t* pos;
  DevErr* err;
};

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(PlanArgs a) {
  extern __shared__ int32_t s_req[];          // [R + 1] first token, [R] base - held, [R] len
  __shared__ long long s_warp[kPlanThreads / 32];
  int32_t* s_first = s_req;
  int32_t* s_base = s_req + a.R + 1;
  int32_t* s_len = s_base + a.R;
  const int rank = blockIdx.x, ctas = gridDim.x;
  const int tid = threadIdx.x;
  griddep_wait();
  bool ok = load_err(a.err) == 0;
  const int count = *a.count;
  const int page_mask = (1 << a.shift) - 1;
  const int per = (a.R + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);

  int bad = 0, bad_r = 0;                     // error code found by this thread
  long long tokens = 0, pages = 0;
  for (int r = r0; r < r1; ++r) {
    const long long len = a.len[r], n = a.fresh[r];
    const long long held = (len + page_mask) >> a.shift, need = (len + n + page_mask) >> a.shift;
    int code = 0;
    if (len < 0 || n < 0) code = AVSG_ERR_BAD_SELECTION;
    else if (need > a.max_pages) code = AVSG_ERR_CAPACITY;
    else if (n > 0 && (len & page_mask) != 0) {
      // the page that the first new token shares with older ones
      const int32_t id = a.tables[(size_t)r * a.max_pages + (len >> a.shift)];
      if (id < 0 || id >= a.num_pages) code = AVSG_ERR_BAD_SELECTION;
    }
    if (code && !bad) {
      bad = code;
      bad_r = r;
    }
    if (!code) {
      tokens += n;
      pages += need - held;
    }
  }
  long long total_tokens, total_pages;
  long long t_at = block_exclusive(tokens, s_warp, &total_tokens);
  long long p_at = block_exclusive(pages, s_warp, &total_pages);
  if (bad) {
    if (rank == 0) raise_error(a.err, bad, bad_r, -1);
  } else if (tid == 0 && (count < 0 || count > a.num_pages)) {
    bad = AVSG_ERR_BAD_SELECTION;
    if (rank == 0) raise_error(a.err, bad, -1, -1);
  } else if (tid == 0 && (total_pages > count || total_tokens > a.capacity || (a.mask && total_tokens > a.num_mask))) {
    bad = AVSG_ERR_CAPACITY;
    if (rank == 0) raise_error(a.err, bad, -1, -1);
  }
  ok = !__syncthreads_or(!ok || bad);
  if (ok) {
    for (int r = r0; r < r1; ++r) {
      const int len = a.len[r], n = a.fresh[r];
      const int held = (len + page_mask) >> a.shift;
      const int need = (int)(((long long)len + n + page_mask) >> a.shift);
      s_first[r] = (int)t_at;
      s_base[r] = (int)p_at - held;
      s_len[r] = len;
      t_at += n;
      p_at += need - held;
    }
    if (tid == 0) s_first[a.R] = (int)total_tokens;
    // the pages to be taken (every CTA checks all of them: they decide alike)
    for (int e = tid; e < (int)total_pages; e += kPlanThreads) {
      const int32_t id = a.free_list[count - 1 - e];
      if (id < 0 || id >= a.num_pages) {
        bad = 1;
        if (rank == 0) raise_error(a.err, AVSG_ERR_BAD_SELECTION, -1, count - 1 - e);
      }
    }
  }
  ok = !__syncthreads_or(!ok || bad);
  griddep_launch();
  // Everything that may alias the count has been read by this CTA; the last one writes it.
  if (tid == 0) {
    __threadfence();
    if (atomicInc(reinterpret_cast<unsigned*>(&a.err->aux), (unsigned)ctas - 1) == (unsigned)ctas - 1 && ok)
      *a.count_out = count - (int)total_pages;
  }
  if (!ok) return;

  for (int r = rank * kPlanThreads + tid; r <= a.R; r += ctas * kPlanThreads) a.first[r] = s_first[r];
  for (long long t4 = 4LL * (rank * kPlanThreads + tid); t4 < a.capacity; t4 += 4LL * ctas * kPlanThreads) {
    int32_t slot[4], pos[4];
    int r = t4 < total_tokens ? find_request(s_first, a.R, (int)t4) : a.R;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int t = (int)t4 + x;
      slot[x] = -1;
      pos[x] = 0;
      if (t >= (int)total_tokens) continue;
      while (t >= s_first[r + 1]) ++r;
      const int i = t - s_first[r], len = s_len[r], p = len + i;
      const int held = (len + page_mask) >> a.shift, at = p >> a.shift;
      int32_t* row = a.tables + (size_t)r * a.max_pages;
      int32_t page;
      if (at < held) {
        page = row[at];
      } else {
        page = a.free_list[count - 1 - (s_base[r] + at)];
        if ((p & page_mask) == 0) row[at] = page;
      }
      slot[x] = (page << a.shift) + (p & page_mask);
      pos[x] = p;
      if (a.mask) {
        const unsigned long long m = a.mask[t];
        // (requests of more drafts than a word has bits are chains)
        if (m && s_first[r + 1] - s_first[r] <= kMaxDrafts) pos[x] = len + __popcll(m) - 1;
      }
    }
    if (a.wide && t4 + 4 <= a.capacity) {
      *reinterpret_cast<int4*>(a.slot + t4) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      *reinterpret_cast<int4*>(a.pos + t4) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (t4 + x < a.capacity) {
          a.slot[t4 + x] = slot[x];
          a.pos[t4 + x] = pos[x];
        }
    }
  }
}

struct KeepArgs {
  int R, shift, max_pages, num_pages, num_path;
  const int32_t* first;
  const int32_t* path;
  const int32_t* keep;
  const int32_t* len;
  int32_t* len_out;
  const int32_t* tables;
  int32_t* free_list;
  const int32_t* count;
  int32_t* count_out;
  DevErr* err;
};

// Checks the kept paths, writes the new lengths and returns the pages past them.
__global__ void __launch_bounds__(kPlanThreads) keep_lengths_kernel(KeepArgs a) {
  extern __shared__ int32_t s_req[];          // [R + 1] first page given back, [R] its table index
  __shared__ long long s_warp[kPlanThreads / 32];
  int32_t* s_back = s_req;
  int32_t* s_from = s_req + a.R + 1;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  const int tid = threadIdx.x;
  griddep_wait();
  bool ok = load_err(a.err) == 0;
  const int count = *a.count;
  const int page_mask = (1 << a.shift) - 1;
  const int per = (a.R + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);

  int bad = 0, bad_r = -1, bad_i = -1;
  long long back = 0;
  for (int r = r0; r < r1; ++r) {
    const long long len = a.len[r], f = a.first[r], n = (long long)a.first[r + 1] - f;
    const long long k = a.keep[r];
    const long long need = (len + n + page_mask) >> a.shift;
    int code = 0;
    if (len < 0 || f < 0 || n < 0 || k < -1 || k > n) code = AVSG_ERR_BAD_SELECTION;
    else if (need > a.max_pages || (a.path && f + n > a.num_path)) code = AVSG_ERR_CAPACITY;
    if (code && !bad) {
      bad = code;
      bad_r = r;
    }
    if (!code) back += need - (((k < 0 ? 0 : len + k) + page_mask) >> a.shift);
  }
  long long total;
  long long at = block_exclusive(back, s_warp, &total);
  if (!bad && tid == 0 && (count < 0 || total + count > a.num_pages)) bad = AVSG_ERR_CAPACITY;
  if (bad && rank == 0) raise_error(a.err, bad, bad_r, bad_i);
  ok = !__syncthreads_or(!ok || bad);
  if (ok) {
    for (int r = r0; r < r1; ++r) {
      const long long len = a.len[r], n = a.first[r + 1] - a.first[r], k = a.keep[r];
      const int need = (int)((len + n + page_mask) >> a.shift);
      const int from = (int)(((k < 0 ? 0 : len + k) + page_mask) >> a.shift);
      s_back[r] = (int)at;
      s_from[r] = from;
      at += need - from;
    }
    if (tid == 0) s_back[a.R] = (int)total;
  }
  __syncthreads();
  // This CTA's share of the kept paths (strictly increasing, inside the
  // request), of the pages that stay and whose rows move, and of those that go
  // back (which rows may come from); a failure reaches the other CTAs through
  // the error word, read after the barrier.
  if (ok) {
    const int warp = rank * (kPlanThreads / 32) + (tid >> 5), warps = ctas * (kPlanThreads / 32);
    if (a.path)
      for (int r = warp; r < a.R; r += warps) {
        const int f = a.first[r], n = a.first[r + 1] - f, k = a.keep[r], lane = tid & 31;
        if (k <= 0) continue;
        // (whether rows move, and the pages that stay, are loaded beside the path)
        const bool moves = a.path[f + k - 1] != k - 1;
        bool bad_page = false;
        for (int x = (a.len[r] >> a.shift) + lane; x < s_from[r]; x += 32) {
          const int32_t id = a.tables[(size_t)r * a.max_pages + x];
          bad_page |= id < 0 || id >= a.num_pages;
        }
        for (int i = lane; i < k; i += 32) {
          const int x = a.path[f + i], before = i ? a.path[f + i - 1] : -1;
          if (x <= before || x < 0 || x >= n) raise_error(a.err, AVSG_ERR_BAD_SELECTION, r, i);
        }
        if (moves && bad_page) raise_error(a.err, AVSG_ERR_BAD_SELECTION, r, -1);
      }
    for (int e = rank * kPlanThreads + tid; e < (int)total; e += ctas * kPlanThreads) {
      const int r = find_request(s_back, a.R, e);
      const int32_t id = a.tables[(size_t)r * a.max_pages + s_from[r] + e - s_back[r]];
      if (id < 0 || id >= a.num_pages) raise_error(a.err, AVSG_ERR_BAD_SELECTION, r, -1);
    }
    __threadfence();
  }
  cluster.sync();
  ok = !__syncthreads_or(!ok || load_err(a.err) != 0);
  // A second barrier: no CTA writes before every CTA has read the lengths and the count.
  int new_len[(kMaxPagedRequests + kPlanThreads - 1) / kPlanThreads];
  int mine = 0;
  if (ok && rank == 0) {
#pragma unroll
    for (int j = 0; j < (kMaxPagedRequests + kPlanThreads - 1) / kPlanThreads; ++j) {
      const int r = tid + j * kPlanThreads;
      if (r < a.R) {
        const int k = a.keep[r];
        new_len[j] = k < 0 ? 0 : a.len[r] + k;
        ++mine;
      }
    }
  }
  cluster.sync();
  griddep_launch();
  if (!ok) return;
  if (rank == 0) {
#pragma unroll
    for (int j = 0; j < (kMaxPagedRequests + kPlanThreads - 1) / kPlanThreads; ++j)
      if (j < mine) a.len_out[tid + j * kPlanThreads] = new_len[j];
    if (tid == 0) *a.count_out = count + (int)total;
  }
  for (int e = rank * kPlanThreads + tid; e < (int)total; e += ctas * kPlanThreads) {
    const int r = find_request(s_back, a.R, e);
    a.free_list[count + (int)total - 1 - e] =
        a.tables[(size_t)r * a.max_pages + s_from[r] + e - s_back[r]];
  }
}

struct MoveArgs {
  int R, H, shift, max_pages, num_pages;
  int chunks;                    // 16-byte chunks of one row
  long long layer_bytes;
  unsigned char* k;
  unsigned char* v;
  const int32_t* first;
  const int32_t* path;
  const int32_t* keep;
  const int32_t* len_out;
  const int32_t* tables;
  DevErr* err;
};

constexpr int kMoveThreads = 256;
constexpr int kMoveBatch = 4;    // rows in flight per thread

// One CTA per (request, layer).  A thread owns one 16-byte column of one head
// of K or V and walks the kept rows in order: as the path is strictly
// increasing (path[i] >= i), a row is never written before it was read, and
// no thread touches another's column, so no barrier is needed.
__global__ void __launch_bounds__(kMoveThreads) keep_rows_kernel(MoveArgs a) {
  griddep_wait();
  if (__syncthreads_or(load_err(a.err) != 0)) return;  // nothing moves after a failed check
  const int r = blockIdx.x;
  const int k = a.keep[r];
  if (k <= 0) return;
  const int f = a.first[r], len = a.len_out[r] - k;
  const int32_t* path = a.path + f;
  if (path[k - 1] == k - 1) return;  // strictly increasing: the whole path stays in place
  const int32_t* row = a.tables + (size_t)r * a.max_pages;
  const int page_mask = (1 << a.shift) - 1;
  const int columns = a.H * 2 * a.chunks;
  auto offset = [&](int p, int h, int c) -> long long {
    const int32_t page = row[p >> a.shift];
    // (checked before by keep_lengths_kernel: a table that was changed since is not followed)
    if (page < 0 || page >= a.num_pages) {
      raise_error(a.err, AVSG_ERR_BAD_SELECTION, r, p);
      return -1;
    }
    return ((((long long)page * a.H + h) << a.shift) + (p & page_mask)) * (a.chunks * 16LL) + c * 16;
  };
  for (int col = threadIdx.x; col < columns; col += kMoveThreads) {
    const int c = col % a.chunks, hv = col / a.chunks, h = hv >> 1;
    unsigned char* base = (hv & 1 ? a.v : a.k) + (long long)blockIdx.y * a.layer_bytes;
    for (int i0 = 0; i0 < k; i0 += kMoveBatch) {
      uint4 x[kMoveBatch];
      long long to[kMoveBatch];
#pragma unroll
      for (int j = 0; j < kMoveBatch; ++j) {
        const int i = i0 + j;
        to[j] = -1;
        if (i >= k) continue;
        const int from_i = path[i];
        if (from_i == i) continue;
        const long long from = offset(len + from_i, h, c);
        to[j] = offset(len + i, h, c);
        if (from < 0) to[j] = -1;
        else if (to[j] >= 0) x[j] = *reinterpret_cast<const uint4*>(base + from);
      }
#pragma unroll
      for (int j = 0; j < kMoveBatch; ++j)
        if (to[j] >= 0) *reinterpret_cast<uint4*>(base + to[j]) = x[j];
    }
  }
}

int cluster_for(long long items) {
  int c = 1;
  while (c < kPlanCluster && (long long)c * kPlanTokensPerCta < items) c *= 2;
  return c;
}

SmemLimit g_plan_smem, g_keep_smem;

}  // namespace
}  // namespace avsg

using namespace avsg;

extern "C" int avsg_page_plan(const avsg_pages* p, const int32_t* d_new, const uint64_t* d_mask,
                              int32_t num_mask, int32_t capacity, int32_t* d_first, int32_t* d_slot, int32_t* d_pos,
                              int32_t* d_free_count_out, void* stream) {
  int rc = check_pages(p);
  if (rc != AVSG_OK) return rc;
  if (!d_new || !d_first || capacity < 0 || (capacity > 0 && (!d_slot || !d_pos)) ||
      !d_free_count_out || num_mask < 0)
    return AVSG_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  rc = paged_device(p->d_tables, &dev, &sms);
  if (rc != AVSG_OK) return rc;
  PlanArgs a{};
  a.R = p->num_requests;
  a.shift = page_shift_of(p->page_tokens);
  a.max_pages = p->max_pages;
  a.num_pages = p->num_pages;
  a.capacity = capacity;
  a.num_mask = num_mask;
  a.wide = (reinterpret_cast<uintptr_t>(d_slot) | reinterpret_cast<uintptr_t>(d_pos)) % 16 == 0;
  a.len = p->d_len;
  a.fresh = d_new;
  a.mask = reinterpret_cast<const unsigned long long*>(d_mask);
  a.tables = p->d_tables;
  a.free_list = p->d_free;
  a.count = p->d_free_count;
  a.count_out = d_free_count_out;
  a.first = d_first;
  a.slot = d_slot;
  a.pos = d_pos;
  a.err = reinterpret_cast<DevErr*>(p->d_error);
  const size_t smem = (3 * (size_t)a.R + 1) * sizeof(int32_t);
  // (no more CTAs than SMs: each one scans the lengths)
  const int64_t want = ((int64_t)capacity + kPlanTokensPerCta - 1) / kPlanTokensPerCta;
  const int ctas = want < 1 ? 1 : want < sms ? (int)want : sms;
  cudaError_t e = g_plan_smem.raise(reinterpret_cast<const void*>(page_plan_kernel), smem, dev);
  if (e == cudaSuccess)
    e = launch_pdl(page_plan_kernel, dim3(ctas), dim3(kPlanThreads), smem, static_cast<cudaStream_t>(stream), a);
  return e == cudaSuccess ? AVSG_OK : AVSG_ERR_CUDA;
}

extern "C" int avsg_tree_keep(const avsg_pages* p, const int32_t* d_first, const int32_t* d_path,
                              int32_t num_path, const int32_t* d_keep, int32_t* d_len_out,
                              int32_t* d_free_count_out, void* stream) {
  int rc = check_pages(p);
  if (rc != AVSG_OK) return rc;
  if (!d_first || !d_keep || !d_len_out || !d_free_count_out || num_path < 0) return AVSG_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  rc = paged_device(p->d_tables, &dev, &sms);
  if (rc != AVSG_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  KeepArgs a{};
  a.R = p->num_requests;
  a.shift = page_shift_of(p->page_tokens);
  a.max_pages = p->max_pages;
  a.num_pages = p->num_pages;
  a.num_path = num_path;
  a.first = d_first;
  a.path = d_path;
  a.keep = d_keep;
  a.len = p->d_len;
  a.len_out = d_len_out;
  a.tables = p->d_tables;
  a.free_list = p->d_free;
  a.count = p->d_free_count;
  a.count_out = d_free_count_out;
  a.err = reinterpret_cast<DevErr*>(p->d_error);
  const size_t smem = (2 * (size_t)a.R + 1) * sizeof(int32_t);
  const int ctas = cluster_for((long long)a.R * 64);  // a warp per 32 kept drafts
  cudaError_t e = g_keep_smem.raise(reinterpret_cast<const void*>(keep_lengths_kernel), smem, dev);
  if (e == cudaSuccess)
    e = launch_pdl_cluster(ctas, keep_lengths_kernel, dim3(ctas), dim3(kPlanThreads), smem, st, a);
  if (e == cudaSuccess && d_path) {
    MoveArgs m{};
    m.R = a.R;
    m.H = p->num_kv_heads;
    m.shift = a.shift;
    m.max_pages = a.max_pages;
    m.num_pages = a.num_pages;
    m.chunks = p->head_dim * 2 / 16;
    m.layer_bytes = (long long)p->num_pages * p->num_kv_heads * p->page_tokens * p->head_dim * 2;
    m.k = static_cast<unsigned char*>(p->d_k);
    m.v = static_cast<unsigned char*>(p->d_v);
    m.first = d_first;
    m.path = d_path;
    m.keep = d_keep;
    m.len_out = d_len_out;
    m.tables = p->d_tables;
    m.err = a.err;
    e = launch_pdl(keep_rows_kernel, dim3(a.R, p->num_layers), dim3(kMoveThreads), 0, st, m);
  }
  return e == cudaSuccess ? AVSG_OK : AVSG_ERR_CUDA;
}
