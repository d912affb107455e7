// Append of a ragged chunk's keys and values to a paged cache held in 8 bits,
// with one scale for each block of tokens and KV head.
//
// Mathematics, per (block, head) and for K and V apart; x = the block's new rows
// (K normed and rotated as in rope_append.cu):
//   e = the least whole number with max |x| <= top 2^e   (top: 448 of e4m3, 127 of int8)
//   scale = 2^e, or the block's present scale where earlier tokens of the block
//           have one that is larger
//   code = round(x / scale); where the scale grew, earlier codes = round(code old / new)
// Scales are powers of two because a block fills token by token and may have to
// grow on the way: e4m3 codes are then moved exactly but for those that fall
// below its normal range, and whole-number codes lose half a step each time,
// a step of the last scale in all (1/2 + 1/4 + ...), however often it grows.
// With the tightest scale each new maximum would round all of them anew.  It
// costs whole-number codes up to one bit, e4m3 ones nothing.
//
// What bounds it: bytes for prompts, latency for single tokens.  A unit of work
// is a block, a head and K or V: four warps for a block with many new rows, one
// for a few.  Blocks are found by the row that begins them: a CTA looks over a
// window of `window` rows (1 to 32, about the rows of a sequence), so the grid
// follows from the number of rows alone and the lengths stay on the device.
#include "kernels.h"
#include "rope.cuh"

namespace dls {

namespace {

constexpr int ATHREADS = 128;
constexpr int AWARPS = ATHREADS / 32;

struct App8Args {
  const void *k, *v;
  long long k_stride, v_stride;
  uint8_t *k_pages, *v_pages;
  float *k_scales, *v_scales;
  const float* k_norm;
  const int32_t *page_table, *cu_q, *kv_len;
  int32_t* status;
  int n_tokens, n_seqs, n_kv, head_dim, rot_dim;
  int page_shift, block_shift, n_pages, max_pages;
  int lanes_log2;      // lanes of a row (power of two >= head_dim / 16)
  int window;          // rows that a CTA looks over
  int heads;           // heads of a CTA
  float eps, inv_hd;
  unsigned long long turn[kMaxPairs];
};

template <int CODE>
struct Coder;
template <>
struct Coder<DLS_E4M3> {
  static constexpr int kTopExp = 8;
  static constexpr unsigned kTopFrac = 0x600000u;  // 448 = 1.75 * 2^8
  static __device__ __forceinline__ uint32_t two(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
  }
  static __device__ __forceinline__ uint32_t four(float a, float b, float c, float d) { return two(a, b) | two(c, d) << 16; }
  static __device__ __forceinline__ void values(uint32_t w, float (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t h;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w >> (16 * i))));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
};
template <>
struct Coder<DLS_I8> {
  static constexpr int kTopExp = 6;
  static constexpr unsigned kTopFrac = 0x7e0000u;  // 127 = 1.984375 * 2^6
  static __device__ __forceinline__ uint32_t one(float x) {
    // to the nearest, a tie to the even one; NaN gives 0 (so the clamp is after the conversion)
    return (uint32_t)max(min(__float2int_rn(x), 127), -127) & 0xffu;
  }
  static __device__ __forceinline__ uint32_t four(float a, float b, float c, float d) {
    return one(a) | one(b) << 8 | one(c) << 16 | one(d) << 24;
  }
  static __device__ __forceinline__ void values(uint32_t w, float (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (float)(int8_t)(w >> (8 * i));
  }
};

constexpr int kLeastExp = -64, kMostExp = 64;  // of a scale

// 2^e for the largest magnitude of a block.
template <int CODE>
__device__ __forceinline__ float scale_for(float amax) {
  const unsigned b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - Coder<CODE>::kTopExp + ((b & 0x7fffffu) > Coder<CODE>::kTopFrac);
  return __uint_as_float((unsigned)(min(max(e, kLeastExp), kMostExp) + 127) << 23);
}

template <typename IN, int CODE, bool HALVES>
__global__ void __launch_bounds__(ATHREADS) append8_kernel(const __grid_constant__ App8Args a) {
  __shared__ float s_max[2][AWARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool is_v = blockIdx.y & 1;
  const int head0 = (int)(blockIdx.y >> 1) * a.heads, head1 = min(head0 + a.heads, a.n_kv);
  const int hd = a.head_dim, block = 1 << a.block_shift;

  if (a.status && blockIdx.x == 0 && blockIdx.y == 0 && warp == 0) {
    const long long room = (long long)a.max_pages << a.page_shift;
    bool bad = a.cu_q[0] < 0 || a.cu_q[a.n_seqs] > a.n_tokens;
    for (int b = lane; b < a.n_seqs; b += 32) {
      const int start = a.cu_q[b], end = a.cu_q[b + 1], kl = a.kv_len[b];
      bad |= end < start || kl < 0 || kl > room || (long long)kl < (long long)end - start;
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.status, kBadPos);
  }

  // the lane's row of the window: its sequence, position and page, and whether it begins a block
  const int w0 = blockIdx.x * a.window, row = w0 + lane;
  const int s0 = seq_of(a.cu_q, a.n_seqs, w0, lane);
  int b;
  {
    const int c = s0 + 1 + lane <= a.n_seqs ? a.cu_q[s0 + 1 + lane] : 0x7fffffff;
    b = s0;
    if (__shfl_sync(0xffffffffu, c, 31) >= w0 + a.window) {
      for (int i = 0; i < a.window; ++i) {
        const int n = __popc(__ballot_sync(0xffffffffu, c <= w0 + i));
        if (lane == i) b = s0 + n;
      }
    } else {  // many empty sequences among them
      int lo = s0, hi = a.n_seqs;  // the first sequence from s0 on that ends behind the row
      while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        if (a.cu_q[mid + 1] <= row) lo = mid + 1;
        else hi = mid;
      }
      b = lo;
    }
  }
  int pos = 0, page = -1, n_rows = 0;
  if (lane < a.window && row < a.n_tokens && b < a.n_seqs) {
    const int start = a.cu_q[b], end = a.cu_q[b + 1], kl = a.kv_len[b];
    const long long room = (long long)a.max_pages << a.page_shift;
    // as in the 16-bit append: only these keep the position inside the sequence, whatever cu_q holds
    if (row >= start && row < end && start >= 0 && end <= a.n_tokens && kl >= end - start && kl <= room) {
      pos = kl - (end - row);
      const int off = pos & (block - 1);
      if (row == start || off == 0) {
        n_rows = min(block - off, end - row);
        page = a.page_table[(size_t)b * a.max_pages + (pos >> a.page_shift)];
        if (page < 0 || page >= a.n_pages) {
          if (a.status && blockIdx.y == 0) atomicOr(a.status, kBadPage);
          n_rows = 0;
        }
      }
    }
  }
  unsigned todo = __ballot_sync(0xffffffffu, n_rows > 0);
  if (!todo) return;

  const int lph = 1 << a.lanes_log2, c = lane & (lph - 1), sub = lane >> a.lanes_log2, rps = 32 >> a.lanes_log2;
  const bool live = 16 * c < hd, rot = 16 * c < a.rot_dim && !is_v;
  const bool turns = 16 * c < a.rot_dim;
  const int ea = turns ? 8 * c : 16 * c, eb = turns ? (a.rot_dim >> 1) + 8 * c : 16 * c + 8;  // the lane's two vectors
  const IN* const src = static_cast<const IN*>(is_v ? a.v : a.k);
  const long long stride = is_v ? a.v_stride : a.k_stride;
  uint8_t* const pages = is_v ? a.v_pages : a.k_pages;
  float* const scales = is_v ? a.v_scales : a.k_scales;
  const float* const norm = is_v ? nullptr : a.k_norm;

  // values of the lane's sixteen elements: normed, rotated
  auto finish = [&](float (&xa)[8], float (&xb)[8], int at) {
    if (norm) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(xa[e], xa[e], fmaf(xb[e], xb[e], ss));
      for (int o = lph >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (live) {
        Vec8<float> na, nb;
        na.load(norm + ea);
        nb.load(norm + eb);
        float wa[8], wb[8];
        na.get(wa);
        nb.get(wb);
        const float r = rsqrtf(ss * a.inv_hd + a.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) xa[e] *= r * wa[e], xb[e] *= r * wb[e];
      }
    }
    if (rot) {
      float cs[8], sn[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int pair = HALVES ? 8 * c + e : (e < 4 ? 4 * c + e : (a.rot_dim >> 2) + 4 * c + e - 4);
        const unsigned long long f = (unsigned long long)(long long)at * a.turn[pair & (kMaxPairs - 1)];
        sincospif((float)(int)(f >> 32) * 4.656612873077393e-10f, &sn[e], &cs[e]);  // 2^-31: half turns
      }
      if (HALVES) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = xa[e], y = xb[e];
          xa[e] = x * cs[e] - y * sn[e];
          xb[e] = x * sn[e] + y * cs[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = xa[2 * e], y = xa[2 * e + 1];
          xa[2 * e] = x * cs[e] - y * sn[e];
          xa[2 * e + 1] = x * sn[e] + y * cs[e];
          x = xb[2 * e], y = xb[2 * e + 1];
          xb[2 * e] = x * cs[e + 4] - y * sn[e + 4];
          xb[2 * e + 1] = x * sn[e + 4] + y * cs[e + 4];
        }
      }
    }
  };

  // one block and head: by one warp, or by all of them (wn = 1 or AWARPS, this one the wi-th)
  auto unit = [&](auto keep, int wn, int wi, int turn_of, int row0, int pos0, int m, int pg, int head) {
    constexpr int KEEP = decltype(keep)::value;
    const int off = pos0 & (block - 1);
    const size_t first = (((size_t)pg * a.n_kv + head) << a.page_shift) + (pos0 & ((1 << a.page_shift) - 1)) - off;  // block's slot 0
    float* const scale_at = scales + (first >> a.block_shift);
    uint8_t* const out = pages + first * hd;
    float old = off ? *scale_at : 0.f;
    const int steps = (m + wn * rps - 1) / (wn * rps);
    auto index = [&](int step) { return (step * wn + wi) * rps + sub; };
    auto fetch = [&](int step, float (&xa)[8], float (&xb)[8]) {
      const int i = index(step);
#pragma unroll
      for (int e = 0; e < 8; ++e) xa[e] = xb[e] = 0.f;
      if (live && i < m) {
        const IN* const p = src + (size_t)(row0 + i) * stride + (size_t)head * hd;
        Vec8<IN> va, vb;
        va.load(p + ea);
        vb.load(p + eb);
        va.get(xa);
        vb.get(xb);
      }
    };
    float xa[KEEP][8], xb[KEEP][8];
    float amax = 0.f;
    auto most = [&](const float (&u)[8], const float (&v)[8]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fmaxf(fabsf(u[e]), fabsf(v[e])));
    };
#pragma unroll
    for (int s = 0; s < KEEP; ++s) fetch(s, xa[s], xb[s]);
#pragma unroll
    for (int s = 0; s < KEEP; ++s)
      if (s < steps) {
        finish(xa[s], xb[s], pos0 + index(s));
        most(xa[s], xb[s]);
      }
#pragma unroll 1
    for (int s = KEEP; s < steps; ++s) {
      float u[8], v[8];
      fetch(s, u, v);
      finish(u, v, pos0 + index(s));
      most(u, v);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (wn > 1) {  // (two sets of maxima: a warp may begin the next unit while another still reads these)
      if (lane == 0) s_max[turn_of & 1][warp] = amax;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < AWARPS; ++w) amax = fmaxf(amax, s_max[turn_of & 1][w]);
    }
    const float need = scale_for<CODE>(fminf(amax, 3.402823466e38f));
    float scale = need;
    if (off) {
      old = fminf(fmaxf(old, 0x1p-64f), 0x1p64f);  // (also of a scale that is none)
      scale = fmaxf(old, need);
      if (scale > old) {
        const float f = old / scale;
        for (int i = (wi * 32 + lane) * 16; i < off * hd; i += wn * 512) {
          uint4 w = *reinterpret_cast<const uint4*>(out + i);
          uint32_t* const u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float x[4];
            Coder<CODE>::values(u[k], x);
            u[k] = Coder<CODE>::four(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
          }
          *reinterpret_cast<uint4*>(out + i) = w;
        }
      }
    }
    if (wi == 0 && lane == 0) *scale_at = scale;
    const float inv = 1.f / scale;
    auto store = [&](int step, const float (&u)[8], const float (&v)[8]) {
      const int i = index(step);
      if (!live || i >= m) return;
      uint8_t* const p = out + (size_t)(off + i) * hd;
      *reinterpret_cast<uint2*>(p + ea) = make_uint2(Coder<CODE>::four(u[0] * inv, u[1] * inv, u[2] * inv, u[3] * inv),
                                                     Coder<CODE>::four(u[4] * inv, u[5] * inv, u[6] * inv, u[7] * inv));
      *reinterpret_cast<uint2*>(p + eb) = make_uint2(Coder<CODE>::four(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                                                     Coder<CODE>::four(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
    };
#pragma unroll
    for (int s = 0; s < KEEP; ++s)
      if (s < steps) store(s, xa[s], xb[s]);
#pragma unroll 1
    for (int s = KEEP; s < steps; ++s) {
      float u[8], v[8];
      fetch(s, u, v);
      finish(u, v, pos0 + index(s));
      store(s, u, v);
    }
  };

  const int few = 2 * rps;  // rows that one warp takes by itself
  int at = 0, big = 0;
  for (unsigned left = todo; left; left &= left - 1) {
    const int from = __ffs(left) - 1;
    const int row0 = w0 + from, pos0 = __shfl_sync(0xffffffffu, pos, from), m = __shfl_sync(0xffffffffu, n_rows, from);
    const int pg = __shfl_sync(0xffffffffu, page, from);
    for (int h = head0; h < head1; ++h) {
      if (m <= few) {
        if ((at++ & (AWARPS - 1)) == warp) unit(std::integral_constant<int, 2>(), 1, 0, 0, row0, pos0, m, pg, h);
      } else {
        unit(std::integral_constant<int, 4>(), AWARPS, warp, big++, row0, pos0, m, pg, h);
      }
    }
  }
}

template <typename IN, int CODE>
cudaError_t launch_append8(const App8Args& a, int pairing, dim3 grid, cudaStream_t s) {
  if (pairing == DLS_ROPE_HALVES) append8_kernel<IN, CODE, true><<<grid, ATHREADS, 0, s>>>(a);
  else append8_kernel<IN, CODE, false><<<grid, ATHREADS, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename IN>
cudaError_t launch_append8_code(const App8Args& a, int code, int pairing, dim3 grid, cudaStream_t s) {
  return code == DLS_E4M3 ? launch_append8<IN, DLS_E4M3>(a, pairing, grid, s) : launch_append8<IN, DLS_I8>(a, pairing, grid, s);
}

}  // namespace

}  // namespace dls

extern "C" int dls_kv_append8(const dls_kv_append8_desc* d, void* cuda_stream) {
  using namespace dls;
  if (!d) return report_error(DLS_ERR_ARG, "kv_append8: desc=NULL");
  if (!rope_shape_ok(d->head_dim, d->rot_dim, d->pairing, d->inv_freq, d->eps))
    return report_error(DLS_ERR_ARG, "kv_append8: head_dim=%d rot_dim=%d (multiples of 16, at most 256) pairing=%d inv_freq=%p eps=%g",
                        d->head_dim, d->rot_dim, d->pairing, (const void*)d->inv_freq, d->eps);
  if (!type_bytes(d->in_type) || (d->code_type != DLS_E4M3 && d->code_type != DLS_I8))
    return report_error(DLS_ERR_ARG, "kv_append8: in_type=%d code_type=%d", d->in_type, d->code_type);
  const int pt = d->page_tokens, bt = d->block_tokens;
  if (pt != 16 && pt != 32 && pt != 64 && pt != 128 && pt != 256)
    return report_error(DLS_ERR_ARG, "kv_append8: page_tokens=%d (16, 32, 64, 128 or 256)", pt);
  if ((bt != 16 && bt != 32 && bt != 64 && bt != 128 && bt != 256) || bt > pt)
    return report_error(DLS_ERR_ARG, "kv_append8: block_tokens=%d (16, 32, 64, 128 or 256, at most page_tokens=%d)", bt, pt);
  if (d->n_tokens < 0 || d->n_tokens > 1 << 30 || d->n_seqs < 0 || d->n_seqs > 1 << 30 || d->n_kv_heads < 1 || d->n_kv_heads > 4096 ||
      d->n_pages < 1 || d->max_pages < 1 || (long long)d->max_pages * pt > 0x7fffffff)
    return report_error(DLS_ERR_ARG, "kv_append8: n_tokens=%d n_seqs=%d n_kv_heads=%d n_pages=%d max_pages=%d", d->n_tokens, d->n_seqs,
                        d->n_kv_heads, d->n_pages, d->max_pages);
  if (!aligned_to(d->status, 4)) return report_error(DLS_ERR_ARG, "kv_append8: status=%p", (void*)d->status);
  if (d->n_tokens == 0 || d->n_seqs == 0) return empty_call(d->status, cuda_stream, "kv_append8");
  if (!d->page_table || !d->cu_q || !d->kv_len || !aligned_to(d->page_table, 4) || !aligned_to(d->cu_q, 4) || !aligned_to(d->kv_len, 4))
    return report_error(DLS_ERR_ARG, "kv_append8: page_table=%p cu_q=%p kv_len=%p", (const void*)d->page_table, (const void*)d->cu_q,
                        (const void*)d->kv_len);
  if (!aligned_to(d->k_norm, 16)) return report_error(DLS_ERR_ARG, "kv_append8: k_norm=%p (16-byte aligned)", (const void*)d->k_norm);
  if (!rows_ok(d->k, d->k_stride, d->n_kv_heads, d->head_dim, d->in_type) || !rows_ok(d->v, d->v_stride, d->n_kv_heads, d->head_dim, d->in_type))
    return report_error(DLS_ERR_ARG, "kv_append8: k and v need 16-byte aligned rows of heads * head_dim elements");
  if (!d->k_pages || !d->v_pages || !aligned_to(d->k_pages, 16) || !aligned_to(d->v_pages, 16))
    return report_error(DLS_ERR_ARG, "kv_append8: k_pages=%p v_pages=%p (16-byte aligned)", d->k_pages, d->v_pages);
  if (!d->k_scales || !d->v_scales || !aligned_to(d->k_scales, 4) || !aligned_to(d->v_scales, 4))
    return report_error(DLS_ERR_ARG, "kv_append8: k_scales=%p v_scales=%p", (void*)d->k_scales, (void*)d->v_scales);
  App8Args a{};
  a.k = d->k, a.v = d->v, a.k_stride = d->k_stride, a.v_stride = d->v_stride;
  a.k_pages = static_cast<uint8_t*>(d->k_pages), a.v_pages = static_cast<uint8_t*>(d->v_pages);
  a.k_scales = d->k_scales, a.v_scales = d->v_scales, a.k_norm = d->k_norm;
  a.page_table = d->page_table, a.cu_q = d->cu_q, a.kv_len = d->kv_len, a.status = d->status;
  a.n_tokens = d->n_tokens, a.n_seqs = d->n_seqs, a.n_kv = d->n_kv_heads, a.head_dim = d->head_dim, a.rot_dim = d->rot_dim;
  while ((16 << a.page_shift) < pt) ++a.page_shift;
  while ((16 << a.block_shift) < bt) ++a.block_shift;
  a.page_shift += 4, a.block_shift += 4;
  a.n_pages = d->n_pages, a.max_pages = d->max_pages;
  while ((16 << a.lanes_log2) < d->head_dim) ++a.lanes_log2;
  a.eps = d->eps, a.inv_hd = 1.0f / (float)d->head_dim;
  if (!set_turns(a.turn, a.rot_dim, d->inv_freq)) return report_error(DLS_ERR_ARG, "kv_append8: inv_freq is not finite");
  const int mean = d->n_tokens / d->n_seqs;  // rows of a sequence, about
  a.window = 1;
  while (a.window < 32 && a.window * 2 <= mean) a.window *= 2;
  a.heads = mean < 2 ? std::min(4, d->n_kv_heads) : 1;
  const dim3 grid((unsigned)((d->n_tokens + a.window - 1) / a.window), (unsigned)((d->n_kv_heads + a.heads - 1) / a.heads) * 2);
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e = cudaSuccess;
  if (a.status) e = cudaMemsetAsync(a.status, 0, sizeof(int32_t), s);
  if (e == cudaSuccess)
    e = d->in_type == DLS_F32   ? launch_append8_code<float>(a, d->code_type, d->pairing, grid, s)
        : d->in_type == DLS_F16 ? launch_append8_code<__half>(a, d->code_type, d->pairing, grid, s)
                                : launch_append8_code<__nv_bfloat16>(a, d->code_type, d->pairing, grid, s);
  if (e != cudaSuccess) return report_error(DLS_ERR_CUDA, "kv_append8: cuda=%s", cudaGetErrorString(e));
  return DLS_OK;
}
