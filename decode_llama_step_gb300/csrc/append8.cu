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
// What bounds it: bytes for prompts, latency for single tokens.  Blocks are
// found by the row that begins them: a CTA looks over a window of `window`
// rows (1 to 32, about the rows of a sequence), so the grid follows from the
// number of rows alone and the lengths stay on the device.  The CTA's warps
// share a block's angles (cos and sin of its rows in shared memory: worked out
// for each head they took as long as everything else).  A unit of work is a
// block, a head and K or V, and a warp takes it by itself: its rows once for
// the largest magnitude, and again (from L1 or L2) for the codes, but for the
// last few, which it still has.  The norm's factor of a row is taken into both
// at the end.  All warps on one unit, rows in registers in between: a third
// fewer instructions, half the warps, a barrier a unit, 44 us for the chunks of
// a prefill batch (9762 tokens, 8 heads of 128, bf16) against 32.
// Measured (GPU time): those 31.9 us (9.0 at the copy rate; 68% of the issue
// slots busy, instructions bound it), 64 single tokens 5.0 us.
#include "kernels.h"
#include "rope.cuh"

namespace dls {

namespace {

constexpr int ATHREADS = 256;
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
  int angle_rows;      // rows whose angles are held: a block's, or 0 where they are too many
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

__device__ __forceinline__ void scale2(float& x, float& y, f2_t f) {
  f2_t p;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(pk2(x, y)), "l"(f));
  const float2 v = upk2(p);
  x = v.x, y = v.y;
}

constexpr int kLeastExp = -64, kMostExp = 64;  // of a scale

// 2^e for the largest magnitude of a block.
template <int CODE>
__device__ __forceinline__ float scale_for(float amax) {
  const unsigned b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - Coder<CODE>::kTopExp + ((b & 0x7fffffu) > Coder<CODE>::kTopFrac);
  return __uint_as_float((unsigned)(min(max(e, kLeastExp), kMostExp) + 127) << 23);
}

template <typename IN, int CODE, bool HALVES>
__global__ void __launch_bounds__(ATHREADS, 4) append8_kernel(const __grid_constant__ App8Args a) {
  extern __shared__ float angles[];  // cos [angle_rows][rot_dim / 2], then sin
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int head0 = (int)blockIdx.y * a.heads, n_units = 2 * (min(head0 + a.heads, a.n_kv) - head0);
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

  // the frequencies, read as memory: as a constant, lanes with one each take turns
  __shared__ unsigned long long s_turn[kMaxPairs];
  {
    const unsigned long long* turn = a.turn;
    asm volatile("" : "+l"(turn));
    if (threadIdx.x < a.rot_dim >> 1) s_turn[threadIdx.x] = turn[threadIdx.x];
  }

  // the lane's row of the window: its sequence, position and page, and whether it begins a block.  32 sequences from the
  // window's first on are looked at together, their lengths with them (each load waited for is 0.4 us)
  const int w0 = blockIdx.x * a.window, row = w0 + lane;
  const int s0 = a.n_seqs <= 32 ? 0 : seq_of(a.cu_q, a.n_seqs, w0, lane);
  const bool some = s0 + lane < a.n_seqs;
  int start = some ? a.cu_q[s0 + lane] : 0, end = some ? a.cu_q[s0 + lane + 1] : 0x7fffffff, kl = some ? a.kv_len[s0 + lane] : 0, b;
  if (a.n_seqs <= 32 || __shfl_sync(0xffffffffu, end, 31) >= w0 + a.window) {
    int at = 0;  // how many of the ends are not behind the row
#pragma unroll
    for (int step = 16; step; step >>= 1)
      if (__shfl_sync(0xffffffffu, end, at + step - 1) <= row) at += step;
    at += __shfl_sync(0xffffffffu, end, at) <= row;
    b = s0 + at;  // (at = 32: behind the last sequence)
    start = __shfl_sync(0xffffffffu, start, at & 31);
    end = __shfl_sync(0xffffffffu, end, at & 31);
    kl = __shfl_sync(0xffffffffu, kl, at & 31);
  } else {  // many empty sequences among them
    int lo = s0, hi = a.n_seqs;  // the first sequence from s0 on that ends behind the row
    while (lo < hi) {
      const int mid = lo + (hi - lo) / 2;
      if (a.cu_q[mid + 1] <= row) lo = mid + 1;
      else hi = mid;
    }
    b = lo;
    if (b < a.n_seqs) start = a.cu_q[b], end = a.cu_q[b + 1], kl = a.kv_len[b];
  }
  int pos = 0, page = -1, n_rows = 0;
  if (lane < a.window && row < a.n_tokens && b < a.n_seqs) {
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
  const int pairs = a.rot_dim >> 1;
  const bool live = 16 * c < hd, turns = 16 * c < a.rot_dim;
  const int ea = turns ? 8 * c : 16 * c, eb = turns ? pairs + 8 * c : 16 * c + 8;  // the lane's two vectors
  auto turned = [&](int at, int pair, float* sine, float* cosine) {
    const unsigned long long f = (unsigned long long)(long long)at * s_turn[pair];
    sincospif((float)(int)(f >> 32) * 4.656612873077393e-10f, sine, cosine);  // 2^-31: half turns
  };

  for (; todo; todo &= todo - 1) {
    const int from = __ffs(todo) - 1;
    const int row0 = w0 + from, pos0 = __shfl_sync(0xffffffffu, pos, from), m = __shfl_sync(0xffffffffu, n_rows, from);
    const int pg = __shfl_sync(0xffffffffu, page, from), off = pos0 & (block - 1);
    if (pairs) __syncthreads();  // the frequencies are there, the last block's angles used
    if (a.angle_rows && pairs) {
      for (int pair = lane; pair < pairs; pair += 32)
#pragma unroll 2
        for (int i = warp; i < m; i += AWARPS) turned(pos0 + i, pair, &angles[(a.angle_rows + i) * pairs + pair], &angles[i * pairs + pair]);
      __syncthreads();
    }
#pragma unroll 1
    for (int index = warp; index < n_units; index += AWARPS) {
      const bool is_v = index & 1;
      const int head = head0 + (index >> 1);
      const long long stride = is_v ? a.v_stride : a.k_stride;
      const IN* const src = static_cast<const IN*>(is_v ? a.v : a.k) + (size_t)row0 * stride + (size_t)head * hd;
      const size_t first = (((size_t)pg * a.n_kv + head) << a.page_shift) + (pos0 & ((1 << a.page_shift) - 1)) - off;  // block's slot 0
      uint8_t* const out = (is_v ? a.v_pages : a.k_pages) + first * hd;
      float* const scale_at = (is_v ? a.v_scales : a.k_scales) + (first >> a.block_shift);
      float old = off ? *scale_at : 0.f;
      Vec8<IN> va, vb;
      // (lanes past the block's rows take its last one again: it changes no maximum)
      auto fetch = [&](int s) {
        const IN* const p = src + min(s + sub, m - 1) * stride;
        if (live) va.load(p + ea), vb.load(p + eb);
      };
      float xa[8], xb[8], r = 1.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) xa[e] = xb[e] = 0.f;
      // the fetched row's values but for its norm's factor r; `next`: the row fetched after it, none past the end
      auto values = [&](int s, int next) {
        if (live) {
          va.get(xa);
          vb.get(xb);
        }
        if (next < m) fetch(next);
        if (is_v) return;
        if (a.k_norm) {
          f2_t s2 = pk2(0.f, 0.f);
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const f2_t x = pk2(xa[e], xa[e + 1]), y = pk2(xb[e], xb[e + 1]);
            s2 = ffma2(x, x, ffma2(y, y, s2));
          }
          float ss = upk2(s2).x + upk2(s2).y;
          for (int o = lph >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          r = rsqrtf(ss * a.inv_hd + a.eps);
          if (live) {
            Vec8<float> na, nb;
            na.load(a.k_norm + ea);
            nb.load(a.k_norm + eb);
            float wa[8], wb[8];
            na.get(wa);
            nb.get(wb);
#pragma unroll
            for (int e = 0; e < 8; e += 2) scale2(xa[e], xa[e + 1], pk2(wa[e], wa[e + 1])), scale2(xb[e], xb[e + 1], pk2(wb[e], wb[e + 1]));
          }
        }
        if (turns) {
          // (pairs 8 c .. of the halves pairing; 4 c .. of each vector in the adjacent one)
          const int i = min(s + sub, m - 1), q0 = HALVES ? 8 * c : 4 * c, q1 = HALVES ? q0 + 4 : q0 + (pairs >> 1);
          float cs[8], sn[8];
          if (a.angle_rows) {
            const float *const cosines = angles + i * pairs, *const sines = cosines + a.angle_rows * pairs;
            *reinterpret_cast<float4*>(cs) = *reinterpret_cast<const float4*>(cosines + q0);
            *reinterpret_cast<float4*>(cs + 4) = *reinterpret_cast<const float4*>(cosines + q1);
            *reinterpret_cast<float4*>(sn) = *reinterpret_cast<const float4*>(sines + q0);
            *reinterpret_cast<float4*>(sn + 4) = *reinterpret_cast<const float4*>(sines + q1);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) turned(pos0 + i, (e < 4 ? q0 : q1 - 4) + e, &sn[e], &cs[e]);
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

      auto store = [&](int s) {
        uint8_t* const p = out + (size_t)(off + s + sub) * hd;
        *reinterpret_cast<uint2*>(p + ea) = make_uint2(Coder<CODE>::four(xa[0], xa[1], xa[2], xa[3]),
                                                       Coder<CODE>::four(xa[4], xa[5], xa[6], xa[7]));
        *reinterpret_cast<uint2*>(p + eb) = make_uint2(Coder<CODE>::four(xb[0], xb[1], xb[2], xb[3]),
                                                       Coder<CODE>::four(xb[4], xb[5], xb[6], xb[7]));
      };

      float amax = 0.f, scale = 0.f, inv = 0.f;
      const int last = (m - 1) / rps * rps;
      fetch(0);
#pragma unroll 1
      for (int turn_no = 0; turn_no < 2; ++turn_no) {
        // first all rows for the magnitude, then the codes: of the last ones, which are still there, and of those before
        if (turn_no) {
#pragma unroll
          for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          scale = scale_for<CODE>(fminf(amax, 3.402823466e38f));
          if (off) {  // earlier tokens of the block
            old = fminf(fmaxf(old, 0x1p-64f), 0x1p64f);  // (also of a scale that is none)
            scale = fmaxf(old, scale);
            if (scale > old) {
              const float f = old / scale;
#pragma unroll 1
              for (int i = lane * 16; i < off * hd; i += 512) {
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
          if (lane == 0) *scale_at = scale;
          inv = 1.f / scale;
          if (__builtin_expect((__float_as_uint(scale) & 0x7fffffu) != 0, 0)) {
            // kept from elsewhere and no power of two, so the reciprocal is rounded: divisions, by themselves, since a
            // choice between the two in the loop below costs 2% of the time
#pragma unroll 1
            for (int s = 0; s < m; s += rps) {
              fetch(s);
              values(s, m);
              if (live && s + sub < m) {
#pragma unroll
                for (int e = 0; e < 8; ++e) xa[e] = __fdiv_rn(xa[e] * r, scale), xb[e] = __fdiv_rn(xb[e] * r, scale);
                store(s);
              }
            }
            break;
          }
        }
#pragma unroll 1
        for (int s = turn_no ? last : 0;;) {
          // (the second turn goes last, 0, 1, ...)
          const int next = turn_no && s == last ? 0 : s + rps;
          if (!turn_no) {
            values(s, next);
            float most = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) most = fmaxf(most, fmaxf(fabsf(xa[e]), fabsf(xb[e])));
            amax = fmaxf(amax, most * r);
            if (s == last) break;
          } else {
            // (lanes without elements keep their zeros, which every row's sum of squares takes in, also where r is no number)
            const float f = live ? r * inv : 0.f;
            const f2_t f2 = pk2(f, f);
#pragma unroll
            for (int e = 0; e < 8; e += 2) scale2(xa[e], xa[e + 1], f2), scale2(xb[e], xb[e + 1], f2);
            if (live && s + sub < m) {
              store(s);
            }
            if (next == last) break;
            if (s == last) fetch(0);
            values(next, next + rps);
          }
          s = next;
        }
      }
    }
  }
}

template <typename IN, int CODE>
cudaError_t launch_append8(const App8Args& a, int pairing, dim3 grid, cudaStream_t s) {
  const int smem = a.angle_rows * a.rot_dim * 4;
  void (*const f)(const App8Args) = pairing == DLS_ROPE_HALVES ? append8_kernel<IN, CODE, true> : append8_kernel<IN, CODE, false>;
  if (smem > 40 * 1024) {  // beyond what a launch may ask for unannounced
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, 65536);
    if (e != cudaSuccess) return e;
  }
  f<<<grid, ATHREADS, smem, s>>>(a);
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
  a.heads = std::min(AWARPS / 2, d->n_kv_heads);  // a unit a warp
  const unsigned groups = (unsigned)((d->n_kv_heads + a.heads - 1) / a.heads);
  // smaller windows where CTAs are few: the blocks that begin in one are taken one after another
  while (a.window > 4 && (long long)(d->n_tokens / a.window) * groups < 304) a.window /= 2;
  const unsigned windows = (unsigned)((d->n_tokens + a.window - 1) / a.window);
  a.angle_rows = bt * a.rot_dim <= 16384 ? bt : 0;
  const dim3 grid(windows, groups);
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
