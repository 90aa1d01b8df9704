// avsg_tree_attention: host checks, the workspace's layout and the choice of
// the rows per m-tile.
#include <float.h>

#include "avsg_tree_attn.cuh"

namespace avsg {
namespace {

constexpr int kMostGroups = 64;

// Which kernel a call runs and how its rows are cut.
struct Plan {
  bool umma;
  int wm;      // the other kernel's warps along the rows
  int MT;      // rows per m-tile
  int ctas;
  int begin;   // see TreeArgs
};
Plan plan_kernel(bool umma, int D, int64_t rows, int sms) {
  Plan x;
  x.umma = umma;
  // 16 rows a warp, the fewest that hold all rows (up to 64); the other warps split the keys
  x.wm = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
  x.MT = !umma ? 16 * x.wm : D == 256 ? 128 : 256;
  // Eight units of one tile take 6 us each on tcgen05, where 64 KB of K and V take 1.5 us; longer
  // with more of q and out.  About 2 us with mma.sync, where a tile does.  Eight requests of 1 to
  // 20000 tokens, 64 drafts each, heads of 128: 57 us, with 4 61, with 2 79, with 16 59; heads of
  // 256 and 1 to 32768: 113 us with 8, 129 with 6; 32 x 8 units of 300, one token: 29 us with 6, 33
  // with 4.
  x.begin = !umma ? 1 : (rows > 32 ? 6 : 4) + (D == 256 ? 2 : 0);
  x.ctas = umma || D == 256 ? sms : 2 * sms;
  return x;
}
Plan plan_attention(const avsg_pages* p, int G, int max_new, int sms) {
  const int64_t rows = (int64_t)G * max_new;
  // tcgen05 (avsg_tree_umma.cu): boxes of whole 8-row groups.  It always works on 128 rows; with
  // few rows it pays where contexts are long (8 x 8 units, one token, 16000 tokens: 91 us against
  // 99; 32 x 8 units, 32 rows, 3000 tokens: 80 against 89) and costs 4 to 10 us a call where they
  // are short (8 x 8 units, one token, 300 tokens: 17.4 against 11.6; 32 x 8 units, 32 rows, 50
  // tokens: 22 against 12).  Equal at about 4000 tokens up to 16 rows, 2000 up to 32; with 64 rows
  // it is never far behind.  Heads of 256: equal at 1000 (32 x 8 units, one token, 2000 tokens: 94
  // against 122; 50 tokens: 21 against 17).  Lengths are not known here; the pool's room per place
  // of a request stands for them, so that a large pool with few or short requests in it takes
  // tcgen05 at the cost just given.
  const int64_t room = (int64_t)p->num_pages * p->page_tokens / p->num_requests;
  const int64_t enough = p->head_dim == 256 ? 1024 : rows > 16 ? 4096 : 8192;
  const bool umma = p->page_tokens >= 8 && (rows > 32 || room >= enough);
  return plan_kernel(umma, p->head_dim, rows, sms);
}

struct Workspace {
  size_t ml, part, bytes;  // byte offsets; the heads lie at 0
};
Workspace layout(const Plan& x, int D) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  Workspace w;
  w.ml = up((size_t)x.ctas * sizeof(int4));
  w.part = w.ml + up((size_t)2 * x.ctas * x.MT * 2 * sizeof(float));
  w.bytes = w.part + up((size_t)2 * x.ctas * x.MT * D * sizeof(float));
  return w;
}

// Enough for either kernel: a workspace then serves every pool of these heads.
size_t workspace_bytes(int D, int G, int max_new, int sms) {
  const int64_t rows = (int64_t)G * max_new;
  const size_t a = layout(plan_kernel(false, D, rows, sms), D).bytes;
  const size_t b = layout(plan_kernel(true, D, rows, sms), D).bytes;
  return a > b ? a : b;
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
  *bytes = workspace_bytes(p->head_dim, q_per_kv, max_new, sms);
  return AVSG_OK;
}

extern "C" int avsg_tree_attention(const avsg_pages* p, const avsg_tree* t, void* stream) {
  if (!t) return AVSG_ERR_INVALID_ARG;
  int rc = check_attention(p, t->q_per_kv, t->max_new);
  if (rc != AVSG_OK) return rc;
  if (t->num_tokens < 0 || t->layer < 0 || t->layer >= p->num_layers || t->window < 0 ||
      !(t->softmax_scale >= 0.f) || !(t->softcap >= 0.f) || t->reserved0 != 0)
    return AVSG_ERR_INVALID_ARG;
  // The factors that scores and capped scores are multiplied by: an infinite one would make a score
  // of 0 a NaN.
  const float scale = t->softmax_scale > 0.f ? t->softmax_scale : 1.0f / sqrtf((float)p->head_dim);
  const float log2e = 1.4426950408889634f;
  const float score_log2 = scale * log2e, cap_out = t->softcap * log2e;
  float cap_in = t->softcap > 0.f ? 2.f * log2e * scale / t->softcap : 0.f;
  if (isinf(score_log2) || isinf(cap_out) || isinf(cap_in)) return AVSG_ERR_INVALID_ARG;
  // A factor below the normal range has few bits left; only products q.k beyond 2^126 come near such a cap.
  if (cap_in < FLT_MIN) cap_in = 0.f;
  if (t->num_tokens == 0) return AVSG_OK;
  const int64_t row = (int64_t)p->num_kv_heads * t->q_per_kv * p->head_dim;
  if (!t->d_q || !t->d_first || !t->d_out || !t->d_work || t->q_stride < row || t->q_stride % 2 ||
      reinterpret_cast<uintptr_t>(t->d_q) % 4 || reinterpret_cast<uintptr_t>(t->d_out) % 16 ||
      reinterpret_cast<uintptr_t>(t->d_work) % 256)
    return AVSG_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  rc = paged_device(p->d_k, &dev, &sms);
  if (rc != AVSG_OK) return rc;
  const int D = p->head_dim;
  const Plan x = plan_attention(p, t->q_per_kv, t->max_new, sms);
  const Workspace w = layout(x, D);
  if (t->work_bytes < workspace_bytes(D, t->q_per_kv, t->max_new, sms)) return AVSG_ERR_CAPACITY;
  const size_t layer = (size_t)p->num_pages * p->num_kv_heads * p->page_tokens * D * 2;
  unsigned char* work = static_cast<unsigned char*>(t->d_work);
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
  a.tpm = x.MT / a.G;
  a.window = t->window;
  a.ctas = x.ctas;
  a.min_tiles = 2;
  a.begin = x.begin;
  a.score_log2 = score_log2;
  if (cap_in != 0.f) {
    a.cap_in = cap_in;
    a.cap_out = cap_out;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = x.umma     ? launch_tree_umma(a, p->dtype, D, dev, st)
                  : D == 64  ? launch_tree_d64(a, p->dtype, x.wm, dev, st)
                  : D == 128 ? launch_tree_d128(a, p->dtype, x.wm, dev, st)
                             : launch_tree_d256(a, p->dtype, x.wm, dev, st);
  return e == cudaSuccess ? AVSG_OK : AVSG_ERR_CUDA;
}
