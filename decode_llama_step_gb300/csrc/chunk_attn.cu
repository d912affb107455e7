// Attention of ragged chunks of new tokens over the paged cache.
//
// Simple form: a warp per (row, query head) walks the row's keys with a
// running maximum and sum (m, l) and the unnormalised output in registers,
//   m' = max(m, s);  l = l e^(m - m') + e^(s - m');  o = o e^(m - m') + e^(s - m') v
// a lane holding the elements lane, lane + 32, ... of the head.
#include <cuda_bf16.h>
#include <math.h>

#include "../../include/dls.h"
#include "kernels.h"

namespace dls {

namespace {

struct ChunkArgs {
  const void *q, *k, *v;
  void* o;
  float* lse;
  const int32_t *page_table, *cu_q, *kv_len;
  int32_t* status;
  long long q_stride, o_stride;
  int n_tokens, n_seqs, n_heads, n_kv, head_dim;
  int page_shift, n_pages, max_pages;
  int causal, window;
  float scale;
};

__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float x, __half* y) { *y = __float2half_rn(x); }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16* y) { *y = __float2bfloat16_rn(x); }

template <typename T>
__global__ void __launch_bounds__(128) chunk_simple_kernel(const ChunkArgs a) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x, h = blockIdx.y * 4 + (threadIdx.x >> 5);
  if (h >= a.n_heads) return;
  const long long room = (long long)a.max_pages << a.page_shift;
  if (a.status && t == 0 && h == 0) {  // one warp looks the lengths over
    bool bad = a.cu_q[0] < 0 || a.cu_q[a.n_seqs] > a.n_tokens;
    for (int i = lane; i < a.n_seqs; i += 32)
      bad |= a.cu_q[i + 1] < a.cu_q[i] || a.kv_len[i] < 0 || a.kv_len[i] > room;
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.status, kBadPos);
  }
  int b = 0;
  while (b < a.n_seqs && a.cu_q[b + 1] <= t) ++b;
  if (b >= a.n_seqs) return;
  const int start = a.cu_q[b], end = a.cu_q[b + 1];
  int kl = a.kv_len[b];
  if (t < start) return;
  if (start < 0 || end > a.n_tokens || kl < 0 || kl > room) return;
  const long long pos = (long long)kl - end + t;
  const int hi = a.causal ? (int)(pos + 1 < 0 ? 0 : pos + 1) : kl;
  const int lo = a.window && pos - a.window + 1 > 0 ? (int)(pos - a.window + 1) : 0;
  const int hd = a.head_dim, kvh = h / (a.n_heads / a.n_kv);
  const T* q = static_cast<const T*>(a.q) + (size_t)t * a.q_stride + (size_t)h * hd;
  float qv[4], ov[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    qv[i] = lane + 32 * i < hd ? to_f(q[lane + 32 * i]) : 0.f;
    ov[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int key = lo; key < hi; ++key) {
    const int page = a.page_table[(size_t)b * a.max_pages + (key >> a.page_shift)];
    if (page < 0 || page >= a.n_pages) {
      if (a.status && lane == 0) atomicOr(a.status, kBadPage);
      continue;
    }
    const size_t row =
        ((((size_t)page * a.n_kv + kvh) << a.page_shift) + (key & ((1 << a.page_shift) - 1))) * (size_t)hd;
    const T *k = static_cast<const T*>(a.k) + row, *v = static_cast<const T*>(a.v) + row;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 32 * i < hd) s = fmaf(qv[i], to_f(k[lane + 32 * i]), s);
    s = warp_sum(s) * a.scale;
    const float mn = fmaxf(m, s);
    const float f = m == -INFINITY ? 0.f : expf(m - mn), p = mn == -INFINITY ? 0.f : expf(s - mn);
    l = l * f + p;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 32 * i < hd) ov[i] = ov[i] * f + p * to_f(v[lane + 32 * i]);
    m = mn;
  }
  const float inv = l > 0.f ? 1.0f / l : 0.f;
  T* o = static_cast<T*>(a.o) + (size_t)t * a.o_stride + (size_t)h * hd;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lane + 32 * i < hd) from_f(ov[i] * inv, &o[lane + 32 * i]);
  if (a.lse && lane == 0) a.lse[(size_t)t * a.n_heads + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

bool rows_ok(const void* p, long long stride, long long width) {
  return p && !(reinterpret_cast<uintptr_t>(p) & 15) && stride >= width && stride <= (1ll << 37) && stride % 8 == 0;
}

}  // namespace

}  // namespace dls

extern "C" uint64_t dls_attention_chunk_workspace_bytes(int32_t head_dim) {
  if (head_dim < 16 || head_dim > 128 || head_dim % 16) return 0;
  return 256;
}

extern "C" int dls_attention_chunk(const dls_attention_chunk_desc* d, void* cuda_stream) {
  using namespace dls;
  if (!d) return report_error(DLS_ERR_ARG, "attention_chunk: desc=NULL");
  const int hd = d->head_dim, pt = d->page_tokens;
  if (hd < 16 || hd > 128 || hd % 16) return report_error(DLS_ERR_ARG, "attention_chunk: head_dim=%d (a multiple of 16 up to 128)", hd);
  if (pt != 16 && pt != 32 && pt != 64 && pt != 128 && pt != 256)
    return report_error(DLS_ERR_ARG, "attention_chunk: page_tokens=%d (16, 32, 64, 128 or 256)", pt);
  if (d->kv_type != DLS_F16 && d->kv_type != DLS_BF16) return report_error(DLS_ERR_ARG, "attention_chunk: kv_type=%d", d->kv_type);
  if (d->n_kv_heads < 1 || d->n_heads < 1 || d->n_heads % d->n_kv_heads || d->n_heads / d->n_kv_heads > 128 || d->n_heads > 65536)
    return report_error(DLS_ERR_ARG, "attention_chunk: n_heads=%d n_kv_heads=%d (groups of at most 128)", d->n_heads, d->n_kv_heads);
  if (d->n_tokens < 0 || d->n_seqs < 0 || d->n_seqs > DLS_MAX_CHUNK_SEQS || d->n_pages < 1 || d->max_pages < 1 ||
      (long long)d->max_pages * pt > 0x7fffffff - 1024)
    return report_error(DLS_ERR_ARG, "attention_chunk: n_tokens=%d n_seqs=%d (at most %d) n_pages=%d max_pages=%d", d->n_tokens, d->n_seqs,
                        DLS_MAX_CHUNK_SEQS, d->n_pages, d->max_pages);
  if ((long long)d->n_pages * d->n_kv_heads * pt > 0x7fffffff - 1024)
    return report_error(DLS_ERR_ARG, "attention_chunk: the pool has more than 2^31 - 1024 rows (n_pages=%d n_kv_heads=%d page_tokens=%d)",
                        d->n_pages, d->n_kv_heads, pt);
  if ((d->causal != 0 && d->causal != 1) || d->window < 0 || (d->window && !d->causal))
    return report_error(DLS_ERR_ARG, "attention_chunk: causal=%d window=%d (a window needs causal = 1)", d->causal, d->window);
  if (!(d->scale >= 0.f) || !isfinite(d->scale)) return report_error(DLS_ERR_ARG, "attention_chunk: scale=%g", d->scale);
  if (d->n_tokens == 0 || d->n_seqs == 0) return DLS_OK;
  if (!rows_ok(d->q, d->q_stride, (long long)d->n_heads * hd) || !rows_ok(d->o, d->o_stride, (long long)d->n_heads * hd))
    return report_error(DLS_ERR_ARG, "attention_chunk: q and o need 16-byte aligned rows of n_heads * head_dim elements (strides %lld, %lld)",
                        (long long)d->q_stride, (long long)d->o_stride);
  if (!d->k_pages || !d->v_pages || ((reinterpret_cast<uintptr_t>(d->k_pages) | reinterpret_cast<uintptr_t>(d->v_pages)) & 15))
    return report_error(DLS_ERR_ARG, "attention_chunk: k_pages=%p v_pages=%p (16-byte aligned)", d->k_pages, d->v_pages);
  if (!d->page_table || !d->cu_q || !d->kv_len)
    return report_error(DLS_ERR_ARG, "attention_chunk: page_table=%p cu_q=%p kv_len=%p", (const void*)d->page_table, (const void*)d->cu_q,
                        (const void*)d->kv_len);
  if (!d->workspace || (reinterpret_cast<uintptr_t>(d->workspace) & 255) || d->workspace_bytes < dls_attention_chunk_workspace_bytes(hd))
    return report_error(DLS_ERR_ARG, "attention_chunk: workspace=%p bytes=%llu (256-byte aligned, at least %llu)", d->workspace,
                        (unsigned long long)d->workspace_bytes, (unsigned long long)dls_attention_chunk_workspace_bytes(hd));
  ChunkArgs a{};
  a.q = d->q, a.k = d->k_pages, a.v = d->v_pages, a.o = d->o, a.lse = d->lse;
  a.page_table = d->page_table, a.cu_q = d->cu_q, a.kv_len = d->kv_len, a.status = d->status;
  a.q_stride = d->q_stride, a.o_stride = d->o_stride;
  a.n_tokens = d->n_tokens, a.n_seqs = d->n_seqs, a.n_heads = d->n_heads, a.n_kv = d->n_kv_heads, a.head_dim = hd;
  a.page_shift = pt == 16 ? 4 : pt == 32 ? 5 : pt == 64 ? 6 : pt == 128 ? 7 : 8;
  a.n_pages = d->n_pages, a.max_pages = d->max_pages;
  a.causal = d->causal, a.window = d->window;
  a.scale = d->scale > 0.f ? d->scale : 1.0f / sqrtf((float)hd);
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e = cudaSuccess;
  if (a.status) e = cudaMemsetAsync(a.status, 0, sizeof(int32_t), s);
  if (e == cudaSuccess) {
    const dim3 grid(d->n_tokens, (d->n_heads + 3) / 4);
    if (d->kv_type == DLS_F16) chunk_simple_kernel<__half><<<grid, 128, 0, s>>>(a);
    else chunk_simple_kernel<__nv_bfloat16><<<grid, 128, 0, s>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return report_error(DLS_ERR_CUDA, "attention_chunk: cuda=%s", cudaGetErrorString(e));
  return DLS_OK;
}
