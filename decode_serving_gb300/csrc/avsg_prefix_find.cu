// avsg_prefix_find: which requests of a step begin with the same pages.
//
// Requests with new tokens and the same first page form a group; its leader is
// the lowest of them.  Their common prefix is the least, over the members, of the
// columns in which a member's row agrees with the leader's (any two then agree
// that far), full pages only.  Groups of one, and those whose prefix is shorter than
// min_tokens, stay alone.  A group's new tokens are listed in their order, so that
// an attention over the prefix can take them as the rows of one unit.
//
// What bounds it: latency, and for large batches the rows that are compared.
// One cluster of up to 16 CTAs; its barriers part marking first pages, choosing
// leaders, comparing and listing.  Measured: 8 requests of 4096 tokens 7 us,
// 509 requests, 480 of them in groups that share up to 65536 tokens, 15.8 us (21.5 with
// 8 CTAs: an SM has some 64 KB of rows on their way at a time).
#include <cooperative_groups.h>

#include "avsg_paged.cuh"

namespace cg = cooperative_groups;

namespace avsg {
namespace {

constexpr int kFindThreads = 1024;
constexpr int kFindCluster = 16;           // (beyond 8 a launch has to ask for it)
constexpr int kFindColumns = 512;          // columns of a row that a warp compares at a time
constexpr int kFindBatch = 8;              // of them in flight per thread

struct FindArgs {
  int R, shift, max_pages, num_pages, capacity, min_tokens, pieces;
  const int32_t* len;
  const int32_t* tables;
  const int32_t* first;
  int32_t* owner;                          // [num_pages] the lowest request that begins with a page
  int32_t* least;                          // [R] a leader's common columns
  int32_t* leader;
  int32_t* shared;
  int32_t* group_first;
  int32_t* token;
  int32_t* request;
  DevErr* err;
};

__global__ void __launch_bounds__(kFindThreads) prefix_find_kernel(FindArgs a) {
  extern __shared__ int32_t s_mem[];       // [R] each
  __shared__ int s_warp[kFindThreads / 32];
  int32_t* s_new = s_mem;
  int32_t* s_full = s_new + a.R;           // full pages; 0: not a member of anything
  int32_t* s_leader = s_full + a.R;
  int32_t* s_members = s_leader + a.R;     // then the first place of the leader's tokens
  int32_t* s_rows = s_members + a.R;       // new tokens of the leader's group
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = rank * (kFindThreads / 32) + (tid >> 5), warps = ctas * (kFindThreads / 32);
  griddep_wait();
  bool ok = load_err(a.err) == 0;
  int bad = 0, bad_r = -1;
  for (int r = tid; r < a.R; r += kFindThreads) {
    const int f = a.first[r], end = a.first[r + 1], len = a.len[r];
    const int full = len >> a.shift;
    int code = 0, page = 0;
    if (f < 0 || end < f || end > a.capacity || len < 0 || (r == 0 && f != 0)) code = AVSG_ERR_BAD_SELECTION;
    else if (full > a.max_pages) code = AVSG_ERR_CAPACITY;
    else if (full > 0 && end > f) {
      page = a.tables[(size_t)r * a.max_pages];
      if (page < 0 || page >= a.num_pages) code = AVSG_ERR_BAD_SELECTION;
    }
    if (code && !bad) {
      bad = code;
      bad_r = r;
    }
    s_new[r] = end - f;
    s_full[r] = end > f ? full : 0;
    s_leader[r] = page;                    // (its first page, up to the next phase)
    s_members[r] = s_rows[r] = 0;
    if (!code && rank == 0) {
      if (s_full[r]) a.owner[page] = a.R;
      a.least[r] = s_full[r];
    }
  }
  if (bad && rank == 0) raise_error(a.err, bad, bad_r, -1);
  ok = !__syncthreads_or(!ok || bad);
  __threadfence();
  cluster.sync();
  if (ok && rank == 0)
    for (int r = tid; r < a.R; r += kFindThreads)
      if (s_full[r]) atomicMin(a.owner + s_leader[r], r);
  __threadfence();
  cluster.sync();
  if (ok)
    for (int r = tid; r < a.R; r += kFindThreads) {
      s_leader[r] = s_full[r] ? __ldcg(a.owner + s_leader[r]) : r;
      if (s_full[r]) atomicAdd(&s_members[s_leader[r]], 1);
    }
  __syncthreads();
  // rows against their leaders'
  if (ok)
    for (int i = warp; i < a.R * a.pieces; i += warps) {
      const int r = i / a.pieces, lead = s_leader[r], x0 = (i - r * a.pieces) * kFindColumns;
      if (lead == r) continue;
      const int most = min(s_full[r], s_full[lead]);
      if (x0 == 0 && lane == 0) atomicMin(a.least + lead, most);
      if (x0 >= most || __ldcg(a.least + lead) <= x0) continue;
      const int x1 = min(most, x0 + kFindColumns);
      const int32_t* p = a.tables + (size_t)r * a.max_pages;
      const int32_t* q = a.tables + (size_t)lead * a.max_pages;
      int differs = x1;
      for (int x = x0 + lane; x < x1; x += 32 * kFindBatch) {
        int32_t u[kFindBatch], w[kFindBatch];
#pragma unroll
        for (int j = 0; j < kFindBatch; ++j) {
          u[j] = x + 32 * j < x1 ? p[x + 32 * j] : 0;
          w[j] = x + 32 * j < x1 ? q[x + 32 * j] : 0;
        }
#pragma unroll
        for (int j = kFindBatch - 1; j >= 0; --j)
          if (u[j] != w[j]) differs = min(differs, x + 32 * j);
      }
      differs = __reduce_min_sync(0xffffffffu, differs);
      if (differs < x1 && lane == 0) atomicMin(a.least + lead, differs);
    }
  __threadfence();
  cluster.sync();
  griddep_launch();
  if (!ok) return;
  for (int r = tid; r < a.R; r += kFindThreads) {
    const int lead = s_leader[r], pages = s_members[lead] > 1 ? __ldcg(a.least + lead) : 0;
    const int tokens = (pages << a.shift) >= a.min_tokens ? pages << a.shift : 0;
    // (s_full holds the shared tokens from here on)
    s_full[r] = tokens;
    if (tokens) atomicAdd(&s_rows[lead], s_new[r]);
  }
  __syncthreads();
  const int per = (a.R + kFindThreads - 1) / kFindThreads;
  const int r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);
  int mine = 0, total;
  for (int r = r0; r < r1; ++r) mine += s_rows[r];
  int at = block_exclusive(mine, s_warp, &total);
  for (int r = r0; r < r1; ++r) {
    s_members[r] = at;
    at += s_rows[r];
  }
  __syncthreads();
  if (rank == 0)
    for (int r = tid; r <= a.R; r += kFindThreads) {
      a.group_first[r] = r < a.R ? s_members[r] : total;
      if (r == a.R) break;
      a.leader[r] = s_full[r] ? s_leader[r] : r;
      a.shared[r] = s_full[r];
    }
  for (int r = warp; r < a.R; r += warps) {
    if (!s_full[r]) continue;
    const int lead = s_leader[r];
    int place = 0;                         // new tokens of the members before this one
    for (int x = lead + lane; x < r; x += 32)
      if (s_full[x] && s_leader[x] == lead) place += s_new[x];
    place = s_members[lead] + __reduce_add_sync(0xffffffffu, place);
    const int f = a.first[r];
    for (int x = lane; x < s_new[r]; x += 32) {
      a.token[place + x] = f + x;
      a.request[place + x] = r;
    }
  }
  for (int x = total + rank * kFindThreads + tid; x < a.capacity; x += ctas * kFindThreads)
    a.token[x] = a.request[x] = -1;
}

struct FindWork {
  size_t owner, least, bytes;
};
FindWork find_layout(const avsg_pages* p) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  FindWork w;
  w.owner = 0;
  w.least = up((size_t)p->num_pages * 4);
  w.bytes = w.least + up((size_t)p->num_requests * 4);
  return w;
}

SmemLimit g_find_smem;

// Whether the device runs clusters of kFindCluster CTAs with the most shared memory a call may need.
bool wide_cluster(int dev) {
  static std::mutex mu;
  static signed char known[kMaxDevicesPaged] = {};
  std::lock_guard<std::mutex> lock(mu);
  if (known[dev] == 0) {
    const void* kernel = reinterpret_cast<const void*>(prefix_find_kernel);
    const size_t most = 5 * (size_t)kMaxPagedRequests * sizeof(int32_t);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {kFindCluster, 1, 1};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kFindCluster);
    cfg.blockDim = dim3(kFindThreads);
    cfg.dynamicSmemBytes = most;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (g_find_smem.raise(kernel, most, dev) != cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    known[dev] = n > 0 ? 1 : -1;
  }
  return known[dev] > 0;
}

}  // namespace
}  // namespace avsg

using namespace avsg;

extern "C" int avsg_prefix_find_workspace(const avsg_pages* p, size_t* bytes) {
  const int rc = check_pages(p);
  if (rc != AVSG_OK) return rc;
  if (!bytes) return AVSG_ERR_INVALID_ARG;
  *bytes = find_layout(p).bytes;
  return AVSG_OK;
}

extern "C" int avsg_prefix_find(const avsg_pages* p, const int32_t* d_first, int32_t min_tokens,
                                const avsg_prefixes* x, void* d_work, size_t work_bytes, void* stream) {
  int rc = check_pages(p);
  if (rc != AVSG_OK) return rc;
  if (!d_first || min_tokens < 0 || !x || x->num_tokens < 0 || x->reserved0 != 0 || !x->d_leader || !x->d_shared ||
      !x->d_first || (x->num_tokens > 0 && (!x->d_token || !x->d_request)) || !d_work ||
      reinterpret_cast<uintptr_t>(d_work) % 256)
    return AVSG_ERR_INVALID_ARG;
  const FindWork w = find_layout(p);
  if (p->max_pages > kMaxColumns || work_bytes < w.bytes) return AVSG_ERR_CAPACITY;
  int dev = 0, sms = 0;
  rc = paged_device(p->d_k, &dev, &sms);
  if (rc != AVSG_OK) return rc;
  unsigned char* work = static_cast<unsigned char*>(d_work);
  FindArgs a{};
  a.R = p->num_requests;
  a.shift = page_shift_of(p->page_tokens);
  a.max_pages = p->max_pages;
  a.num_pages = p->num_pages;
  a.capacity = x->num_tokens;
  a.min_tokens = min_tokens;
  a.pieces = (p->max_pages + kFindColumns - 1) / kFindColumns;
  a.len = p->d_len;
  a.tables = p->d_tables;
  a.first = d_first;
  a.owner = reinterpret_cast<int32_t*>(work + w.owner);
  a.least = reinterpret_cast<int32_t*>(work + w.least);
  a.leader = x->d_leader;
  a.shared = x->d_shared;
  a.group_first = x->d_first;
  a.token = x->d_token;
  a.request = x->d_request;
  a.err = reinterpret_cast<DevErr*>(p->d_error);
  if ((int64_t)a.R * a.pieces > INT32_MAX / 2) return AVSG_ERR_CAPACITY;
  const size_t smem = 5 * (size_t)a.R * sizeof(int32_t);
  int ctas = 1;
  while (ctas < kFindCluster && (int64_t)ctas * (kFindThreads / 32) < (int64_t)a.R * a.pieces) ctas *= 2;
  cudaError_t e = g_find_smem.raise(reinterpret_cast<const void*>(prefix_find_kernel), smem, dev);
  if (e == cudaSuccess && ctas > 8 && !wide_cluster(dev)) ctas = 8;
  if (e == cudaSuccess)
    e = launch_pdl_cluster(ctas, prefix_find_kernel, dim3(ctas), dim3(kFindThreads), smem,
                           static_cast<cudaStream_t>(stream), a);
  return e == cudaSuccess ? AVSG_OK : AVSG_ERR_CUDA;
}
