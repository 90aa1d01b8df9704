// Host side of the paged-cache operators: argument checks they share, the
// device check and the rotary frequency table.
#include <math.h>

#include "avsg_paged.cuh"

namespace avsg {

int paged_device(const void* d_ptr, int* dev, int* sms) {
  static std::mutex mu;
  static int known[kMaxDevicesPaged] = {};
  int d = 0;
  if (cudaGetDevice(&d) != cudaSuccess) return AVSG_ERR_CUDA;
  if (d < 0 || d >= kMaxDevicesPaged) return AVSG_ERR_INVALID_ARG;
  cudaPointerAttributes at;
  if (cudaPointerGetAttributes(&at, d_ptr) != cudaSuccess) {
    cudaGetLastError();
    return AVSG_ERR_INVALID_ARG;
  }
  if (at.type != cudaMemoryTypeManaged && (at.type != cudaMemoryTypeDevice || at.device != d))
    return AVSG_ERR_INVALID_ARG;
  std::lock_guard<std::mutex> lock(mu);
  if (!known[d]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, d) != cudaSuccess)
      return AVSG_ERR_CUDA;
    known[d] = n;
  }
  *dev = d;
  *sms = known[d];
  return AVSG_OK;
}

int check_pages(const avsg_pages* p) {
  if (!p || p->num_requests < 1 || p->num_layers < 1 || p->num_pages < 1 || p->num_kv_heads < 1 ||
      p->page_tokens < 1 || p->head_dim < 8 || p->head_dim % 8 || p->max_pages < 1 || !p->d_k ||
      !p->d_v || !p->d_tables || !p->d_len || !p->d_free || !p->d_free_count || !p->d_error)
    return AVSG_ERR_INVALID_ARG;
  if (p->dtype != AVSG_BF16 && p->dtype != AVSG_F16) return AVSG_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(p->d_k) | reinterpret_cast<uintptr_t>(p->d_v)) % 16)
    return AVSG_ERR_INVALID_ARG;
  if ((p->page_tokens & (p->page_tokens - 1)) != 0 || p->page_tokens > 256)
    return AVSG_ERR_UNSUPPORTED;
  if (p->num_requests > kMaxPagedRequests || p->num_layers > 65535 ||
      (int64_t)p->num_pages * p->page_tokens > INT32_MAX ||
      (int64_t)p->max_pages * p->page_tokens > INT32_MAX || p->num_kv_heads > 65535 ||
      p->head_dim > 4096)
    return AVSG_ERR_CAPACITY;
  return AVSG_OK;
}

}  // namespace avsg

extern "C" int avsg_rotary_frequencies(int32_t rot_dim, double base, double factor,
                                       double low_turns, double high_turns, double original,
                                       uint64_t* out) {
  if (rot_dim < 2 || rot_dim % 2 || !(base > 1.0) || !(factor >= 1.0) || isinf(base) ||
      isinf(factor) || !(original >= 0.0) || isinf(original) || !out)
    return AVSG_ERR_INVALID_ARG;
  const bool ramp = original > 0.0;
  if (ramp && (!(low_turns >= 0.0) || !(high_turns > low_turns) || isinf(high_turns)))
    return AVSG_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925286766559;
  const int half = rot_dim / 2;
  for (int i = 0; i < half; ++i) {
    double inv = pow(base, -(double)i / half);
    if (ramp) {
      double keep = (original * inv / two_pi - low_turns) / (high_turns - low_turns);
      keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
      inv *= keep + (1.0 - keep) / factor;
    } else {
      inv /= factor;
    }
    // turns per position, below 1/6 (inv <= 1), as a 64-bit binary fraction
    out[i] = (uint64_t)(ldexp(inv / two_pi, 64) + 0.5);
  }
  return AVSG_OK;
}
