// avsg_tree_attention: host checks, the workspace's layout and the choice of
// the rows per m-tile.
#include "avsg_tree_attn.cuh"

namespace avsg {
namespace {

constexpr int kMostGroups = 64;

// Warps along the rows of an m-tile: 16 rows a warp, the fewest that hold all
// rows of a request and kv-head (up to 64); the other warps split the keys.
// At least one token's query heads have to fit.
int rows_warps(int G, int max_new) {
  const int64_t rows = (int64_t)G * max_new;
  return rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
}

int ctas_per_sm(int D) { return D == 256 ? 1 : 2; }

struct Workspace {
  size_t ml, part, bytes;  // byte offsets; the heads lie at 0
};
Workspace layout(int ctas, int MT, int D) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  Workspace w;
  w.ml = up((size_t)ctas * sizeof(int4));
  w.part = w.ml + up((size_t)2 * ctas * MT * 2 * sizeof(float));
  w.bytes = w.part + up((size_t)2 * ctas * MT * D * sizeof(float));
  return w;
}

int check_attention(const avsg_pages* p, int q_per_kv, int max_new) {
  const int rc = check_pages(p);
  if (rc != AVSG_OK) return rc;
  if (q_per_kv < 1 || max_new < 1) return AVSG_ERR_INVALID_ARG;
  if ((p->head_dim != 64 && p->head_dim != 128 && p->head_dim != 256) || q_per_kv > kMostGroups)
    return AVSG_ERR_UNSUPPORTED;
  return AVSG_OK;
}

}  // namespace
}  // namespace avsg

using namespace avsg;

extern "C" int avsg_tree_attention_workspace(const avsg_pages* p, int32_t q_per_kv, int32_t max_new,
                                             size_t* bytes) {
  const int rc = check_attention(p, q_per_kv, max_new);
  if (rc != AVSG_OK) return rc;
  if (!bytes) return AVSG_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  const int rd = paged_device(p->d_k, &dev, &sms);
  if (rd != AVSG_OK) return rd;
  *bytes = layout(sms * ctas_per_sm(p->head_dim), 16 * rows_warps(q_per_kv, max_new), p->head_dim).bytes;
  return AVSG_OK;
}

extern "C" int avsg_tree_attention(const avsg_pages* p, const avsg_tree* t, void* stream) {
  if (!t) return AVSG_ERR_INVALID_ARG;
  int rc = check_attention(p, t->q_per_kv, t->max_new);
  if (rc != AVSG_OK) return rc;
  if (t->num_tokens < 0 || t->layer < 0 || t->layer >= p->num_layers || t->window < 0 ||
      !(t->softmax_scale >= 0.f) || isinf(t->softmax_scale) || !(t->softcap >= 0.f) ||
      isinf(t->softcap) || t->reserved0 != 0)
    return AVSG_ERR_INVALID_ARG;
  if (t->num_tokens == 0) return AVSG_OK;
  const int64_t row = (int64_t)p->num_kv_heads * t->q_per_kv * p->head_dim;
  if (!t->d_q || !t->d_first || !t->d_out || !t->d_work || t->q_stride < row || t->q_stride % 2 ||
      reinterpret_cast<uintptr_t>(t->d_q) % 4 || reinterpret_cast<uintptr_t>(t->d_out) % 16 ||
      reinterpret_cast<uintptr_t>(t->d_work) % 256)
    return AVSG_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  rc = paged_device(p->d_k, &dev, &sms);
  if (rc != AVSG_OK) return rc;
  const int wm = rows_warps(t->q_per_kv, t->max_new), MT = 16 * wm, D = p->head_dim;
  const int ctas = sms * ctas_per_sm(D);
  const Workspace w = layout(ctas, MT, D);
  if (t->work_bytes < w.bytes) return AVSG_ERR_CAPACITY;
  const size_t layer = (size_t)p->num_pages * p->num_kv_heads * p->page_tokens * D * 2;
  unsigned char* work = static_cast<unsigned char*>(t->d_work);
  const float scale = t->softmax_scale > 0.f ? t->softmax_scale : 1.0f / sqrtf((float)D);
  const float log2e = 1.4426950408889634f;
  TreeArgs a{};
  a.k = static_cast<const unsigned char*>(p->d_k) + t->layer * layer;
  a.v = static_cast<const unsigned char*>(p->d_v) + t->layer * layer;
  a.tables = p->d_tables;
  a.len = p->d_len;
  a.first = t->d_first;
  a.mask = reinterpret_cast<const unsigned long long*>(t->d_mask);
  a.slopes = t->d_slopes;
  a.q = static_cast<const unsigned char*>(t->d_q);
  a.out = static_cast<unsigned char*>(t->d_out);
  a.lse = t->d_lse;
  a.head = reinterpret_cast<int4*>(work);
  a.ml = reinterpret_cast<float*>(work + w.ml);
  a.part = reinterpret_cast<float*>(work + w.part);
  a.err = reinterpret_cast<DevErr*>(p->d_error);
  a.q_stride = t->q_stride;
  a.R = p->num_requests;
  a.H = p->num_kv_heads;
  a.G = t->q_per_kv;
  a.T = t->num_tokens;
  a.shift = page_shift_of(p->page_tokens);
  a.max_pages = p->max_pages;
  a.num_pages = p->num_pages;
  a.max_new = t->max_new;
  a.tpm = MT / a.G;
  a.window = t->window;
  a.ctas = ctas;
  a.min_tiles = 2;
  a.score_log2 = scale * log2e;
  if (t->softcap > 0.f) {
    a.cap_in = 2.f * log2e * scale / t->softcap;
    a.cap_out = t->softcap * log2e;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = D == 64    ? launch_tree_d64(a, p->dtype, wm, dev, st)
                  : D == 128 ? launch_tree_d128(a, p->dtype, wm, dev, st)
                             : launch_tree_d256(a, p->dtype, wm, dev, st);
  return e == cudaSuccess ? AVSG_OK : AVSG_ERR_CUDA;
}
