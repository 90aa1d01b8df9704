// Shared by the paged-cache operators (page plan, rotary write, tree
// attention, keep): the checked form of avsg_pages and small device helpers.
#pragma once

#include <mutex>

#include "avsg_internal.cuh"

namespace avsg {

constexpr int kMaxPagedRequests = 8192;  // lengths of all requests are scanned by every CTA
constexpr int kMaxDrafts = 64;           // bits of a draft's ancestor mask
constexpr int kMaxDevicesPaged = 64;
constexpr int kMaxColumns = 1 << 30;     // table columns of the calls that walk whole rows

// Device of the current context and its SM count; d_ptr must be memory of
// that device (a tensor of another one would fault in the kernel).
int paged_device(const void* d_ptr, int* dev, int* sms);

// AVSG_OK, or the error of a bad avsg_pages (host checks only).
int check_pages(const avsg_pages* p);

inline int page_shift_of(int page_tokens) {
  int s = 0;
  while ((1 << s) < page_tokens) ++s;
  return s;
}

// The dynamic shared memory limit of a kernel, raised once per device.
struct SmemLimit {
  int done[kMaxDevicesPaged] = {};
  cudaError_t raise(const void* kernel, size_t bytes, int dev) {
    static std::mutex mu;
    std::lock_guard<std::mutex> lock(mu);
    if (done[dev] >= (int)bytes) return cudaSuccess;
    cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done[dev] = (int)bytes;
    return e;
  }
};

// Asks once per device for the shared memory split that the attention kernels have: a kernel of another
// one would wait until the SM is empty.
struct SmemSplit {
  bool done[kMaxDevicesPaged] = {};
  cudaError_t ask(const void* kernel, int dev) {
    static std::mutex mu;
    std::lock_guard<std::mutex> lock(mu);
    if (done[dev]) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                         cudaSharedmemCarveoutMaxShared);
    if (e == cudaSuccess) done[dev] = true;
    return e;
  }
};

// Exclusive prefix of v over the block's threads; *total receives the sum.
// s_warp: one slot per warp, reusable after the next __syncthreads.
template <typename T>
__device__ __forceinline__ T block_exclusive(T v, T* s_warp, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  T inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  T before = 0, all = 0;
  for (int w = 0; w < warps; ++w) {
    const T x = s_warp[w];
    if (w < warp) before += x;
    all += x;
  }
  __syncthreads();
  *total = all;
  return before + inc - v;
}

}  // namespace avsg
