// avsg_rotary_write: rotary positions of a step's q and k rows; q goes to the
// attention's input, k and v to their places in the paged cache (or, with no
// slots, to one row per token as avsg_append takes them).
//
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t) * magnitude,  t = pos * w_i
//
// The angle.  In fp32, pos * w is off by up to 2^-24 of itself: 0.06 rad at
// position 2^20.  The table holds w in turns as a 64-bit binary fraction, so
// pos * w modulo 2^64 IS the fraction of a turn: the reduction is exact and
// costs one 64-bit integer multiply.  Its upper 32 bits, as a signed number
// (at most half a turn, 2^-32 turns per unit), go to sincospif; what is left
// is the rounding to fp32, 2^-25 turns (2e-7 rad), at any position.
//
// What bounds it: bytes.  q, k and v are read once and written once; the
// angles of a token are computed once per CTA into shared memory and used by
// all its heads.  A thread owns one place of one head -- two chunks of 16
// bytes where widths and alignment allow: the two halves of pairs, or
// neighbours -- for the CTA's tokens, so that the index arithmetic is paid
// once for several loads, all in flight before the first is used.
// Measured: 16381 tokens of 32 + 8 + 8 heads of 128, half of each head turned:
// 68 us, 5.9 TB/s of the copy's 6.78 (one token per CTA 100 us, two 77, eight
// 80; 3 CTAs of 85 registers an SM 70, 4 of 64 75).  8 tokens: 2 us a call in a graph, 21 from
// Python, which is the host's work.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "avsg_paged.cuh"

namespace avsg {
namespace {

constexpr int kRotThreads = 256;  // at most
constexpr int kRotTokens = 4;    // tokens per CTA of a long call
constexpr int kMaxRot = 1024;

struct RotArgs {
  int T, Hq, H, G, D, rot, offset, interleaved, n_tok, shift, num_pages;
  int unit_heads;                // heads of q, k and v together
  int per_head;                  // places of one head: pair groups, then plain chunks
  long long q_stride, k_stride, v_stride;
  float magnitude;
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  void* kp;
  void* vp;
  const unsigned long long* freq;
  const int32_t* pos;
  const int32_t* slot;
  DevErr* err;
};

template <int BYTES> struct Chunk;
template <> struct Chunk<16> { using type = uint4; };
template <> struct Chunk<8> { using type = uint2; };
template <> struct Chunk<4> { using type = uint32_t; };
template <> struct Chunk<2> { using type = uint16_t; };

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16& y) { y = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f(float x, __half& y) { y = __float2half_rn(x); }
__device__ __forceinline__ void from_f(float x, float& y) { y = x; }

// VEC consecutive values as one access of 2 * VEC bytes (fp32: two of them).
template <typename T, int VEC>
union Vec {
  typename Chunk<2 * VEC>::type raw;
  T x[VEC];
  __device__ Vec() {}
};
template <typename TO, int VEC>
__device__ __forceinline__ void store_vec(TO* p, const float* x) {
  if constexpr (sizeof(TO) == 2) {
    Vec<TO, VEC> o;
#pragma unroll
    for (int i = 0; i < VEC; ++i) from_f(x[i], o.x[i]);
    *reinterpret_cast<typename Chunk<2 * VEC>::type*>(p) = o.raw;
  } else {
    if constexpr (VEC >= 4) {
#pragma unroll
      for (int i = 0; i < VEC; i += 4)
        *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) p[i] = x[i];
    }
  }
}

// T: type of q, k, v and the cache; TQ: type of q_out; VEC: values per chunk;
// TOK: tokens per CTA.
template <typename T, typename TQ, int VEC, int TOK>
__global__ void __launch_bounds__(kRotThreads, 3) rotary_kernel(RotArgs a) {
  extern __shared__ float2 s_cs[];            // [TOK][rot / 2] cos, sin
  const int tid = threadIdx.x, half = a.rot >> 1;
  const int t0 = blockIdx.x * TOK;
  const int groups = half / VEC, units = a.unit_heads * a.per_head;
  griddep_wait();
  const bool latched = load_err(a.err) != 0;

  // One place of one head: values d0 .. and d1 .. of it (d1 < 0: one chunk alone; d0 < 0: none).
  const T* src;
  long long stride;
  int hh, w, d0, d1;
  bool is_q, is_v, turns;
  Vec<T, VEC> x0[TOK], x1[TOK];
  auto load = [&](int u) {
    const int head = u / a.per_head;
    w = u - head * a.per_head;
    is_v = head >= a.Hq + a.H;
    is_q = head < a.Hq;
    hh = is_q ? head : is_v ? head - a.Hq - a.H : head - a.Hq;
    src = static_cast<const T*>(is_q ? a.q : is_v ? a.v : a.k);
    stride = is_q ? a.q_stride : is_v ? a.v_stride : a.k_stride;
    turns = !is_v && w < groups;
    if (turns) {
      d0 = a.offset + (a.interleaved ? 2 * w * VEC : w * VEC);
      d1 = a.interleaved ? d0 + VEC : d0 + half;
    } else {
      // neighbouring chunks of what keeps its values
      const int rot = is_v ? 0 : a.rot, c = 2 * (is_v ? w : w - groups);
      d0 = c * VEC;
      d1 = d0 + VEC < a.D - rot ? d0 + VEC : -1;
      if (d0 >= a.D - rot) d0 = -1;
      if (rot && d0 >= a.offset) d0 += rot;
      if (rot && d1 >= a.offset) d1 += rot;
    }
    if (u >= units) d0 = -1;
    if (d0 < 0) return;
#pragma unroll
    for (int j = 0; j < TOK; ++j) {
      if (t0 + j >= a.T) continue;
      const T* p = src + (t0 + j) * stride + (long long)hh * a.D;
      x0[j].raw = __ldcs(reinterpret_cast<const typename Chunk<2 * VEC>::type*>(p + d0));
      if (d1 >= 0) x1[j].raw = __ldcs(reinterpret_cast<const typename Chunk<2 * VEC>::type*>(p + d1));
    }
  };
  // The first place's rows are on their way while slots are read and angles computed (rows of
  // padding are read too, but go nowhere).
  int u = blockIdx.y * blockDim.x + tid;
  load(u);
  int slot[TOK];
#pragma unroll
  for (int j = 0; j < TOK; ++j) {
    const int t = t0 + j;
    slot[j] = t >= a.T ? -1 : a.slot ? a.slot[t] : t;
    if (slot[j] >= 0 && (slot[j] >> a.shift) >= a.num_pages) {
      if (tid == 0) raise_error(a.err, AVSG_ERR_BAD_SELECTION, -1, t);
      slot[j] = -1;
    }
  }
  for (int x = tid; x < TOK * half; x += blockDim.x) {
    const int j = x / half, i = x - j * half, t = t0 + j;
    if (t >= a.T) break;
    const unsigned long long turn = (unsigned long long)(long long)a.pos[t] * a.freq[i];
    float sn, cs;
    sincospif((float)(int)(turn >> 32) * 0x1p-31f, &sn, &cs);
    s_cs[x] = make_float2(cs * a.magnitude, sn * a.magnitude);
  }
  if (__syncthreads_or(latched)) return;
  griddep_launch();

  for (;;) {
    if (d0 >= 0) {
#pragma unroll
      for (int j = 0; j < TOK; ++j) {
        if (slot[j] < 0) continue;
        const int t = t0 + j;
        float y0[VEC], y1[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          y0[i] = to_f(x0[j].x[i]);
          y1[i] = to_f(x1[j].x[i]);
        }
        if (turns) {
          const float2* cs = s_cs + j * half + w * VEC;
          if (a.interleaved) {
            float z[2 * VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              z[i] = y0[i];
              z[VEC + i] = y1[i];
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              const float2 c = cs[i];
              const float p = z[2 * i], q = z[2 * i + 1];
              z[2 * i] = p * c.x - q * c.y;
              z[2 * i + 1] = p * c.y + q * c.x;
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              y0[i] = z[i];
              y1[i] = z[VEC + i];
            }
          } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              const float2 c = cs[i];
              const float p = y0[i], q = y1[i];
              y0[i] = p * c.x - q * c.y;
              y1[i] = p * c.y + q * c.x;
            }
          }
        }
        if (is_q) {
          long long row;                        // of the [.., G][D] block this head belongs to
          if (a.n_tok == 1) row = (long long)t * a.Hq + hh;
          else row = (((long long)(t / a.n_tok) * a.H + hh / a.G) * a.n_tok + t % a.n_tok) * a.G +
                     hh % a.G;
          TQ* o = static_cast<TQ*>(a.q_out) + row * a.D;
          store_vec<TQ, VEC>(o + d0, y0);
          if (d1 >= 0) store_vec<TQ, VEC>(o + d1, y1);
        } else {
          const long long row =
              ((((long long)(slot[j] >> a.shift) * a.H + hh) << a.shift) + (slot[j] & ((1 << a.shift) - 1)));
          T* o = static_cast<T*>(is_v ? a.vp : a.kp) + row * a.D;
          if (!turns) {                         // unchanged bits
            *reinterpret_cast<typename Chunk<2 * VEC>::type*>(o + d0) = x0[j].raw;
            if (d1 >= 0) *reinterpret_cast<typename Chunk<2 * VEC>::type*>(o + d1) = x1[j].raw;
          } else {
            store_vec<T, VEC>(o + d0, y0);
            store_vec<T, VEC>(o + d1, y1);
          }
        }
      }
    }
    u += gridDim.y * blockDim.x;
    if (u >= units) break;
    load(u);
  }
}

template <typename T, typename TQ, int VEC>
cudaError_t launch_rotary(const RotArgs& in, int sms, cudaStream_t st) {
  RotArgs a = in;
  const int qk = a.rot / 2 / VEC + ((a.D - a.rot) / VEC + 1) / 2, v = (a.D / VEC + 1) / 2;
  a.per_head = v > qk ? v : qk;
  const int units = a.unit_heads * a.per_head;
  // as many threads as share the places evenly
  const int rounds = (units + kRotThreads - 1) / kRotThreads;
  const int threads = ((units + rounds - 1) / rounds + 31) / 32 * 32;
  // Several tokens per CTA only when there are enough for every SM to hold
  // four CTAs; short calls spread a token's heads over CTAs instead.
  const bool many = a.T >= kRotTokens * 4 * sms;
  const int tok = many ? kRotTokens : 1;
  const int ctas = (a.T + tok - 1) / tok;
  int split = rounds;
  const int most = (4 * sms + ctas - 1) / ctas;
  if (split > most) split = most;
  const size_t smem = (size_t)tok * (a.rot / 2) * sizeof(float2);
  if (many) return launch_pdl(rotary_kernel<T, TQ, VEC, kRotTokens>, dim3(ctas, split), dim3(threads), smem, st, a);
  return launch_pdl(rotary_kernel<T, TQ, VEC, 1>, dim3(ctas, split), dim3(threads), smem, st, a);
}

template <typename T, typename TQ>
cudaError_t launch_rotary_vec(const RotArgs& a, int sms, cudaStream_t st) {
  // The widest chunk that every row start, the rotated part and its halves
  // are a multiple of, and that q, k, v are aligned to.
  long long bits = a.D | a.offset | (a.rot / 2) | a.q_stride | a.k_stride | a.v_stride;
  uintptr_t ptrs = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) |
                   reinterpret_cast<uintptr_t>(a.v) |
                   (reinterpret_cast<uintptr_t>(a.q_out) / (sizeof(TQ) / 2));
  bits |= (long long)(ptrs / 2);
  if (bits % 8 == 0) return launch_rotary<T, TQ, 8>(a, sms, st);
  if (bits % 4 == 0) return launch_rotary<T, TQ, 4>(a, sms, st);
  return launch_rotary<T, TQ, 1>(a, sms, st);
}

}  // namespace
}  // namespace avsg

using namespace avsg;

extern "C" int avsg_rotary_write(const avsg_pages* p, const avsg_rotary* r, void* stream) {
  int rc = check_pages(p);
  if (rc != AVSG_OK) return rc;
  if (!r || r->num_tokens < 0 || r->num_q_heads < 1 || r->num_q_heads % p->num_kv_heads ||
      r->rot_dim < 0 || r->rot_dim % 2 || r->rot_offset < 0 ||
      (int64_t)r->rot_offset + r->rot_dim > p->head_dim || r->tokens_per_request < 1 ||
      r->num_tokens % r->tokens_per_request || r->layer < 0 || r->layer >= p->num_layers ||
      !isfinite(r->magnitude) || r->reserved0 != 0)
    return AVSG_ERR_INVALID_ARG;
  if (r->rot_dim > kMaxRot || r->num_q_heads > 65535) return AVSG_ERR_CAPACITY;
  if (r->num_tokens == 0) return AVSG_OK;
  if (!r->d_q || !r->d_k || !r->d_v || !r->d_q_out || !r->d_pos || (r->rot_dim > 0 && !r->d_freq))
    return AVSG_ERR_INVALID_ARG;
  const int64_t q_row = (int64_t)r->num_q_heads * p->head_dim;
  const int64_t kv_row = (int64_t)p->num_kv_heads * p->head_dim;
  if (r->q_stride < q_row || r->k_stride < kv_row || r->v_stride < kv_row)
    return AVSG_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(r->d_q) | reinterpret_cast<uintptr_t>(r->d_k) |
       reinterpret_cast<uintptr_t>(r->d_v)) % 2 ||
      reinterpret_cast<uintptr_t>(r->d_q_out) % (r->q_f32 ? 4 : 2))
    return AVSG_ERR_INVALID_ARG;
  if (!r->d_slot && r->num_tokens > (int64_t)p->num_pages * p->page_tokens)
    return AVSG_ERR_CAPACITY;
  int dev = 0, sms = 0;
  rc = paged_device(p->d_k, &dev, &sms);
  if (rc != AVSG_OK) return rc;
  const size_t layer = (size_t)p->num_pages * p->num_kv_heads * p->page_tokens * p->head_dim * 2;
  RotArgs a{};
  a.T = r->num_tokens;
  a.Hq = r->num_q_heads;
  a.H = p->num_kv_heads;
  a.G = a.Hq / a.H;
  a.D = p->head_dim;
  a.rot = r->rot_dim;
  a.offset = r->rot_offset;
  a.interleaved = r->interleaved ? 1 : 0;
  a.n_tok = r->tokens_per_request;
  a.shift = page_shift_of(p->page_tokens);
  a.num_pages = p->num_pages;
  a.unit_heads = a.Hq + 2 * a.H;
  a.q_stride = r->q_stride;
  a.k_stride = r->k_stride;
  a.v_stride = r->v_stride;
  a.magnitude = r->magnitude;
  a.q = r->d_q;
  a.k = r->d_k;
  a.v = r->d_v;
  a.q_out = r->d_q_out;
  a.kp = static_cast<unsigned char*>(p->d_k) + r->layer * layer;
  a.vp = static_cast<unsigned char*>(p->d_v) + r->layer * layer;
  a.freq = reinterpret_cast<const unsigned long long*>(r->d_freq);
  a.pos = r->d_pos;
  a.slot = r->d_slot;
  a.err = reinterpret_cast<DevErr*>(p->d_error);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (p->dtype == AVSG_BF16)
    e = r->q_f32 ? launch_rotary_vec<__nv_bfloat16, float>(a, sms, st)
                 : launch_rotary_vec<__nv_bfloat16, __nv_bfloat16>(a, sms, st);
  else
    e = r->q_f32 ? launch_rotary_vec<__half, float>(a, sms, st)
                 : launch_rotary_vec<__half, __half>(a, sms, st);
  return e == cudaSuccess ? AVSG_OK : AVSG_ERR_CUDA;
}
