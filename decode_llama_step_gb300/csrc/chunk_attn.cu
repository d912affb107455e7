// The host side of the attention over the paged cache: checks, tensor maps and
// the launches over 16-bit pages (those over codes: chunk_attn8.cu).  The
// kernel stands in chunk_attn.cuh.
#include <mutex>

#include "chunk_attn.cuh"

namespace dls {

namespace {

// SMs of the current device, with the attributes of the kernels over 16-bit pages, or over codes, set on it; 0 on an
// error.  Each kind by itself: an attribute loads its kernel, and the 40 over codes took three quarters of the 3.2 ms
// that the first call over 16-bit pages then was.
int device_ready(bool codes, cudaError_t* err) {
  static std::mutex mu;
  static int sms[64][2];
  int dev = 0;
  if ((*err = cudaGetDevice(&dev)) != cudaSuccess) return 0;
  if (dev < 0 || dev >= 64) {
    *err = cudaErrorInvalidDevice;
    return 0;
  }
  std::lock_guard<std::mutex> g(mu);
  if (sms[dev][codes]) return sms[dev][codes];
  int n = 0;
  if ((*err = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return 0;
  if (codes) {
    if ((*err = chunk_codes_setup()) != cudaSuccess || (*err = few_codes_setup()) != cudaSuccess) return 0;
    return sms[dev][1] = n;
  }
  const ChunkFn f[2] = {chunk_kernel<__half, 128, 0>, chunk_kernel<__nv_bfloat16, 128, 0>};
  const ChunkFn h[2] = {chunk_kernel<__half, 64, 0>, chunk_kernel<__nv_bfloat16, 64, 0>};
  for (int i = 0; i < 2; ++i) {
    if ((*err = cudaFuncSetAttribute(f[i], cudaFuncAttributeMaxDynamicSharedMemorySize, chunk_smem<128, 0>())) != cudaSuccess) return 0;
    if ((*err = cudaFuncSetAttribute(h[i], cudaFuncAttributeMaxDynamicSharedMemorySize, chunk_smem<64, 0>())) != cudaSuccess) return 0;
  }
  return sms[dev][0] = n;
}

bool rows_ok(const void* p, long long stride, long long width) {
  return p && !(reinterpret_cast<uintptr_t>(p) & 15) && stride >= width && stride <= (1ll << 37) && stride % 8 == 0;
}

// Both calls; one over 16-bit pages has code_type 0.
int attend(const dls_attention_chunk8_desc* d, const char* what, void* cuda_stream) {
  const int hd = d->head_dim, pt = d->page_tokens;
  if (hd < 16 || hd > 128 || hd % 16) return report_error(DLS_ERR_ARG, "%s: head_dim=%d (a multiple of 16 up to 128)", what, hd);
  if (pt != 16 && pt != 32 && pt != 64 && pt != 128 && pt != 256)
    return report_error(DLS_ERR_ARG, "%s: page_tokens=%d (16, 32, 64, 128 or 256)", what, pt);
  if (d->q_type != DLS_F16 && d->q_type != DLS_BF16)
    return report_error(DLS_ERR_ARG, "%s: %s=%d", what, d->code_type ? "q_type" : "kv_type", d->q_type);
  const int bt = d->block_tokens;
  if (d->code_type && ((bt != 16 && bt != 32 && bt != 64 && bt != 128 && bt != 256) || bt > pt))
    return report_error(DLS_ERR_ARG, "%s: block_tokens=%d (16, 32, 64, 128 or 256, at most page_tokens=%d)", what, bt, pt);
  if (d->n_kv_heads < 1 || d->n_heads < 1 || d->n_heads % d->n_kv_heads || d->n_heads / d->n_kv_heads > 128 || d->n_heads > 65536)
    return report_error(DLS_ERR_ARG, "%s: n_heads=%d n_kv_heads=%d (groups of at most 128)", what, d->n_heads, d->n_kv_heads);
  if (d->n_tokens < 0 || d->n_tokens > 1 << 30 || d->n_seqs < 0 || d->n_seqs > DLS_MAX_CHUNK_SEQS || d->n_pages < 1 || d->max_pages < 1 ||
      (long long)d->max_pages * pt > 0x7fffffff - 1024)
    return report_error(DLS_ERR_ARG, "%s: n_tokens=%d n_seqs=%d (at most %d) n_pages=%d max_pages=%d", what, d->n_tokens, d->n_seqs,
                        DLS_MAX_CHUNK_SEQS, d->n_pages, d->max_pages);
  if ((long long)d->n_pages * d->n_kv_heads * pt > 0x7fffffff - 1024)
    return report_error(DLS_ERR_ARG, "%s: the pool has more than 2^31 - 1024 rows (n_pages=%d n_kv_heads=%d page_tokens=%d)", what,
                        d->n_pages, d->n_kv_heads, pt);
  if ((d->causal != 0 && d->causal != 1) || d->window < 0 || (d->window && !d->causal))
    return report_error(DLS_ERR_ARG, "%s: causal=%d window=%d (a window needs causal = 1)", what, d->causal, d->window);
  if (!(d->scale >= 0.f) || !isfinite(d->scale)) return report_error(DLS_ERR_ARG, "%s: scale=%g", what, d->scale);
  const int tpq = 128 / (d->n_heads / d->n_kv_heads);
  // decreasing cu_q can give every sequence all the rows: their tiles still have to fit an int
  if (((long long)d->n_tokens / (2 * tpq) + 1) * d->n_seqs > 0x7fffffff)
    return report_error(DLS_ERR_ARG, "%s: n_tokens=%d n_seqs=%d are too many", what, d->n_tokens, d->n_seqs);
  if (!aligned_to(d->status, 4) || !aligned_to(d->lse, 4))
    return report_error(DLS_ERR_ARG, "%s: lse=%p status=%p", what, (void*)d->lse, (void*)d->status);
  if (d->n_tokens == 0 || d->n_seqs == 0) return empty_call(d->status, cuda_stream, what);
  if (!rows_ok(d->q, d->q_stride, (long long)d->n_heads * hd) || !rows_ok(d->o, d->o_stride, (long long)d->n_heads * hd))
    return report_error(DLS_ERR_ARG, "%s: q and o need 16-byte aligned rows of n_heads * head_dim elements (strides %lld, %lld)", what,
                        (long long)d->q_stride, (long long)d->o_stride);
  if (d->q == d->o && d->q_stride != d->o_stride) return report_error(DLS_ERR_ARG, "%s: in place needs the same stride", what);
  if (!d->k_pages || !d->v_pages || ((reinterpret_cast<uintptr_t>(d->k_pages) | reinterpret_cast<uintptr_t>(d->v_pages)) & 15))
    return report_error(DLS_ERR_ARG, "%s: k_pages=%p v_pages=%p (16-byte aligned)", what, d->k_pages, d->v_pages);
  if (d->code_type && (!d->k_scales || !d->v_scales || !aligned_to(d->k_scales, 4) || !aligned_to(d->v_scales, 4)))
    return report_error(DLS_ERR_ARG, "%s: k_scales=%p v_scales=%p", what, (const void*)d->k_scales, (const void*)d->v_scales);
  if (!d->page_table || !d->cu_q || !d->kv_len || !aligned_to(d->page_table, 4) || !aligned_to(d->cu_q, 4) || !aligned_to(d->kv_len, 4))
    return report_error(DLS_ERR_ARG, "%s: page_table=%p cu_q=%p kv_len=%p", what, (const void*)d->page_table, (const void*)d->cu_q,
                        (const void*)d->kv_len);
  if (!d->workspace || (reinterpret_cast<uintptr_t>(d->workspace) & 255) || d->workspace_bytes < dls_attention_chunk_workspace_bytes(hd))
    return report_error(DLS_ERR_ARG, "%s: workspace=%p bytes=%llu (256-byte aligned, at least %llu)", what, d->workspace,
                        (unsigned long long)d->workspace_bytes, (unsigned long long)dls_attention_chunk_workspace_bytes(hd));
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e = cudaSuccess;
  const int sms = device_ready(d->code_type != 0, &e);
  if (e != cudaSuccess) return report_error(DLS_ERR_CUDA, "%s: cuda=%s", what, cudaGetErrorString(e));
  ChunkArgs a{};
  a.o = d->o, a.lse = d->lse;
  a.page_table = d->page_table, a.cu_q = d->cu_q, a.kv_len = d->kv_len, a.status = d->status;
  a.counters = static_cast<int*>(d->workspace);
  a.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(d->workspace) + kCounterBytes);
  a.o_stride = d->o_stride;
  a.n_tokens = d->n_tokens, a.n_seqs = d->n_seqs, a.n_kv = d->n_kv_heads, a.group = d->n_heads / d->n_kv_heads, a.head_dim = hd;
  a.page_shift = pt == 16 ? 4 : pt == 32 ? 5 : pt == 64 ? 6 : pt == 128 ? 7 : 8;
  a.n_pages = d->n_pages, a.max_pages = d->max_pages, a.pool_rows = d->n_pages * d->n_kv_heads * pt;
  a.causal = d->causal, a.window = d->window;
  a.tpq = tpq, a.tile_tokens = 2 * tpq, a.inv_group = (65536 + a.group - 1) / a.group;
  a.c = (d->scale > 0.f ? d->scale : 1.0f / sqrtf((float)hd)) * 1.4426950408889634f;
  // A lane of the planning warp walks at most 4 sequences and 8 more tiles; its sums fit 32 bits.
  // One token over 2048: 15.5 us with the warp's plan, 16.2 with the block's; 64 over up to 8192 (5301 on average) 218 and 220 us.
  a.small_plan = d->n_seqs <= 128 && d->n_tokens <= 8 * 2 * a.tpq && (long long)d->max_pages * pt <= 1 << 24;
  a.k_scales = d->k_scales, a.v_scales = d->v_scales;
  a.block_shift = bt == 16 ? 4 : bt == 32 ? 5 : bt == 64 ? 6 : bt == 128 ? 7 : 8;
  const CUtensorMapDataType dt = d->q_type == DLS_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const uint32_t pr = pt < BK ? pt : BK;
  CUtensorMap tq, tk, tv;
  // Few rows a sequence (two tiles of sixteen, on average): the kernel without
  // operands of 128 rows.  4 heads a KV head of 128 and 8 sequences over 4096: 16
  // rows 27 us (46 by the other), 32 rows 38 (47), 48 rows 52 (48); 64 over
  // 2048: 76 (152), 132 (152), 187 (155); heads of 64 alike.  The number of rows
  // alone is known here, and batches of unequal sequences are not served well
  // (32/8 heads of 128, bf16, e4m3): a long chunk taken this way reads its keys
  // once for every eight or sixteen rows (256 tokens over 16384 beside 64 single
  // ones over 2048: 471 us, 232 by the other kernel, 160 as a call for each kind;
  // 512 over 16384 among 63 sequences without rows: 752, 151 by the other), and
  // single tokens taken the other way work on tiles of 256 rows (64 over 2048
  // with 2048 over 16384: 657, 545 as two calls; with 2000 rows of padding: 130,
  // 70 this way).
  const bool few = d->code_type && a.group <= kFewRows && (long long)d->n_tokens * a.group <= 2 * kFewRows * (long long)d->n_seqs;
  if (few) {
    const int rows = (long long)d->n_tokens * a.group <= 8 * (long long)d->n_seqs && a.group <= 8 ? 8 : kFewRows;
    a.tile_tokens = rows / a.group;
    // Here the warp plans up to 128 tiles' worth of rows (its sums still fit 32 bits).  Single tokens over 2048, 32/8 heads
    // of 128: one 10.1 us (10.5 with the block's plan), 16 22.8 (23.6), 128 104.3 (104.9).  Where one sequence has
    // most of the tiles, one lane walks them all: 385 tokens beside 127 single ones 225 (217), 512 over 1000 alone 97 (81).
    a.small_plan = d->n_seqs <= 128 && d->n_tokens <= 128 * a.tile_tokens && (long long)d->max_pages * pt <= 1 << 24;
    const CUtensorMapSwizzle sw = hd == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : hd == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE;
    if (!make_tmap_2d(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, d->k_pages, hd, a.pool_rows, hd, hd, pr, sw) ||
        !make_tmap_2d(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, d->v_pages, hd, a.pool_rows, hd, hd, pr, sw))
      return report_error(DLS_ERR_CUDA, "%s: tensor map (head_dim=%d)", what, hd);
    if (a.status) e = cudaMemsetAsync(a.status, 0, sizeof(int32_t), s);
    if (e == cudaSuccess)
      e = launch_few_codes(tk, tv, a, d->q, d->q_stride, d->q_type == DLS_F16, d->code_type, sms < MAXC ? sms : MAXC, s);
    return e == cudaSuccess ? DLS_OK : report_error(DLS_ERR_CUDA, "%s: cuda=%s", what, cudaGetErrorString(e));
  }
  const uint64_t dims[3] = {(uint64_t)hd, (uint64_t)d->n_heads, (uint64_t)d->n_tokens};
  const uint64_t strides[2] = {(uint64_t)hd * 2, (uint64_t)d->q_stride * 2};
  const uint32_t box[3] = {64, (uint32_t)a.group, (uint32_t)a.tpq};
  auto pool = [&](CUtensorMap* m, const void* p) {
    if (d->code_type) return make_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, p, hd, a.pool_rows, hd, hd, pr, CU_TENSOR_MAP_SWIZZLE_NONE);
    return make_tmap_2d(m, dt, p, hd, a.pool_rows, hd * 2, 64, pr, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  if (!make_tmap_3d(&tq, dt, d->q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) || !pool(&tk, d->k_pages) || !pool(&tv, d->v_pages))
    return report_error(DLS_ERR_CUDA, "%s: tensor map (head_dim=%d n_heads=%d n_tokens=%d)", what, hd, d->n_heads, d->n_tokens);
  if (a.status) e = cudaMemsetAsync(a.status, 0, sizeof(int32_t), s);
  if (e == cudaSuccess) {
    const bool half = d->q_type == DLS_F16;
    const int ctas = sms < MAXC ? sms : MAXC;
    if (d->code_type) {
      e = launch_chunk_codes(tq, tk, tv, a, d->code_type, half, ctas, s);
    } else {
      const ChunkFn f = hd <= 64 ? (half ? chunk_kernel<__half, 64, 0> : chunk_kernel<__nv_bfloat16, 64, 0>)
                                 : (half ? chunk_kernel<__half, 128, 0> : chunk_kernel<__nv_bfloat16, 128, 0>);
      f<<<ctas, kThreads<0>, hd <= 64 ? chunk_smem<64, 0>() : chunk_smem<128, 0>(), s>>>(tq, tk, tv, a);
      e = cudaGetLastError();
    }
  }
  if (e != cudaSuccess) return report_error(DLS_ERR_CUDA, "%s: cuda=%s", what, cudaGetErrorString(e));
  return DLS_OK;
}

}  // namespace

}  // namespace dls

extern "C" int dls_attention_chunk(const dls_attention_chunk_desc* d, void* cuda_stream) {
  using namespace dls;
  if (!d) return report_error(DLS_ERR_ARG, "attention_chunk: desc=NULL");
  dls_attention_chunk8_desc c{};
  c.q = d->q, c.k_pages = d->k_pages, c.v_pages = d->v_pages;
  c.page_table = d->page_table, c.cu_q = d->cu_q, c.kv_len = d->kv_len;
  c.o = d->o, c.lse = d->lse, c.workspace = d->workspace, c.workspace_bytes = d->workspace_bytes, c.status = d->status;
  c.q_stride = d->q_stride, c.o_stride = d->o_stride;
  c.n_tokens = d->n_tokens, c.n_seqs = d->n_seqs, c.n_heads = d->n_heads, c.n_kv_heads = d->n_kv_heads, c.head_dim = d->head_dim;
  c.page_tokens = c.block_tokens = d->page_tokens, c.n_pages = d->n_pages, c.max_pages = d->max_pages;
  c.q_type = d->kv_type, c.causal = d->causal, c.window = d->window, c.scale = d->scale;
  return attend(&c, "attention_chunk", cuda_stream);
}

extern "C" int dls_attention_chunk8(const dls_attention_chunk8_desc* d, void* cuda_stream) {
  using namespace dls;
  if (!d) return report_error(DLS_ERR_ARG, "attention_chunk8: desc=NULL");
  if (d->code_type != DLS_E4M3 && d->code_type != DLS_I8) return report_error(DLS_ERR_ARG, "attention_chunk8: code_type=%d", d->code_type);
  return attend(d, "attention_chunk8", cuda_stream);
}

extern "C" uint64_t dls_attention_chunk_workspace_bytes(int32_t head_dim) {
  if (head_dim < 16 || head_dim > 128 || head_dim % 16) return 0;
  const uint64_t hdp = head_dim <= 64 ? 64 : 128;
  return dls::kCounterBytes + (uint64_t)dls::MAXC * 4 * 128 * (hdp + 2) * sizeof(float);
}
