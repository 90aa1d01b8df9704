// avsg_tree_attention: its entry points (avsg_tree_plan.cuh has the checks and the choice of the kernel).
#include "avsg_tree_plan.cuh"

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
  TreeArgs a{};
  int dev = 0, sms = 0;
  const int rc = tree_args(p, t, &a, &dev, &sms);
  if (rc != AVSG_OK || a.T == 0) return rc;
  const int D = p->head_dim;
  const Plan x = plan_attention(p, t->q_per_kv, t->max_new, sms);
  const Workspace w = tree_layout(x, D);
  if (t->work_bytes < workspace_bytes(D, t->q_per_kv, t->max_new, sms)) return AVSG_ERR_CAPACITY;
  unsigned char* work = static_cast<unsigned char*>(t->d_work);
  a.head = reinterpret_cast<int4*>(work);
  a.ml = reinterpret_cast<float*>(work + w.ml);
  a.partial = reinterpret_cast<float*>(work + w.part);
  a.tpm = x.MT / a.G;
  a.ctas = x.ctas;
  a.begin = x.begin;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = x.umma     ? launch_tree_umma(a, p->dtype, D, dev, st)
                  : D == 64  ? launch_tree_d64(a, p->dtype, x.wm, dev, st)
                  : D == 128 ? launch_tree_d128(a, p->dtype, x.wm, dev, st)
                             : launch_tree_d256(a, p->dtype, x.wm, dev, st);
  return e == cudaSuccess ? AVSG_OK : AVSG_ERR_CUDA;
}
