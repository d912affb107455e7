// Per-head RMSNorm + rotation of q and k, and the append of a ragged chunk's
// keys and values to the paged cache: one kernel, two entry points.
//
// Mathematics, per head x of a token at position p:
//   y = x * rsqrt(mean(x^2) + eps) * w
//   (a, b) -> (a cos f - b sin f, a sin f + b cos f),  f = p * inv_freq[i]
// Angles: the host turns inv_freq[i] into F[i] = round(inv_freq[i] / 2 pi *
// 2^64), a turn being 2^64.  p * F[i] in 64-bit integers wraps modulo one
// turn exactly, so the fraction of a turn has no cancellation however far
// p is; its upper 32 bits, rounded to the 24 of a float, go to sincospi.  All
// that grows with p is F's own error: the roundings of 2 pi and of the
// quotient, each 2^-53 of inv_freq at most, and 2^-65 of a turn (at position
// 2^31 less than 2^-34 of one).
//
// What bounds it: bytes (each element is read once and written once).  A
// lane owns sixteen elements of a head as two 8-element vectors whose
// rotation partners are its own (vectors 8c and rot/2 + 8c: in the halves
// pairing one holds the partners of the other, in the adjacent pairing each
// holds its own), so nothing is exchanged but the sum of squares, loads and
// stores are contiguous over a head's lanes, and in-place calls are safe.  A
// warp stays on one token and walks its heads, one pass fetched ahead, so a
// token's cos and sin serve every head of the walk; the lanes that hold the
// same pairs of different heads share the work of them.
// Measured: 8192 bf16 tokens of 72 heads of 128, normed and turned, 57.7 us
// (5.2 TB/s; 44.5 at the copy rate); an append of 9762 tokens with q, k and v
// in bf16 (32 + 2 x 8 heads of 128) 50.5 us (4.8 TB/s).  Without any arithmetic
// the same walk takes as long: what is left is the walk's thousands of
// streams, one a warp, a limit of this walk and not of the operator.  A CTA
// that walks four tokens together reaches 49 us as a bare copy, but 67 with
// the norm, whose exchanges then stand in the way; two passes fetched ahead
// cost the warps that they gain.
#include <cuda_bf16.h>
#include <math.h>

#include "../../include/dls.h"
#include "kernels.h"

namespace dls {

namespace {

constexpr int kMaxPairs = 128;   // rot_dim <= 256
constexpr int RTHREADS = 128;

struct RopeSrc {
  const void* in;
  void* out;             // token-major rows, or a page pool (paged != 0)
  const float* norm;     // fp32 [head_dim] or null
  long long in_stride, out_stride;
  int heads;
  int rotate, paged;
};

struct RopeArgs {
  RopeSrc src[3];        // q, k, v (heads = 0: absent)
  const int32_t* positions;  // qk_norm_rope; null: positions follow from cu_q / kv_len
  const int32_t *page_table, *cu_q, *kv_len;
  int32_t* status;
  int n_tokens, n_seqs, head_dim, rot_dim, pairing;
  int page_shift, n_pages, max_pages, n_kv;
  int lanes_log2;        // lanes of a head (power of two >= head_dim / 16)
  int heads_total, passes, per_warp, chunks;  // head passes of a token, passes of a warp, warps of a token
  float eps, inv_hd;
  unsigned long long turn[kMaxPairs];
};

template <typename T>
struct Vec8;
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  static __device__ __forceinline__ void put(float* p, const float (&x)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
  }
};
template <>
struct Vec8<__half> {
  uint4 v;
  __device__ __forceinline__ void load(const __half* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ void put(__half* p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec8<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void put(__nv_bfloat16* p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Number of cu_q[1..n] that are <= t, counted by the whole warp (32 probes a
// round, so two dependent loads up to 1024 sequences).  The result is in
// [0, n] whatever cu_q holds.
__device__ __forceinline__ int seq_of(const int32_t* cu_q, int n, int t, int lane) {
  int lo = 0;  // entries below lo are <= t
  while (n - lo > 32) {
    const int step = (n - lo + 31) / 32;
    const int at = lo + (lane + 1) * step;  // the last entry of lane's block (1-based)
    const unsigned hit = __ballot_sync(0xffffffffu, at <= n && cu_q[at] <= t);
    const int blocks = __popc(hit);
    const int end = min(n, lo + (blocks + 1) * step);
    lo += blocks * step;
    n = end;
  }
  const unsigned hit = __ballot_sync(0xffffffffu, lo + lane < n && cu_q[lo + lane + 1] <= t);
  return lo + __popc(hit);
}

// One warp looks every sequence's lengths over and flags what does not fit.
__device__ __noinline__ void check_lengths(const RopeArgs& a, int lane) {
  const long long room = (long long)a.max_pages << a.page_shift;
  bool bad = a.cu_q[0] < 0 || a.cu_q[a.n_seqs] > a.n_tokens;
  for (int b = lane; b < a.n_seqs; b += 32) {
    const int start = a.cu_q[b], end = a.cu_q[b + 1], kl = a.kv_len[b];
    bad |= end < start || kl < 0 || kl > room || (long long)kl < (long long)end - start;
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.status, kBadPos);
}

template <typename IN, typename OUT, bool HALVES>
__global__ void __launch_bounds__(RTHREADS, sizeof(IN) == 4 ? 5 : 6) rope_kernel(const __grid_constant__ RopeArgs a) {
  const int lane = threadIdx.x & 31;
  const unsigned w = blockIdx.x * (RTHREADS / 32) + (threadIdx.x >> 5);
  const int t = (int)(w / (unsigned)a.chunks), part = (int)(w - (unsigned)t * a.chunks);
  if (t >= a.n_tokens) return;
  const int lph = 1 << a.lanes_log2;            // lanes of a head
  const int c = lane & (lph - 1), sub = lane >> a.lanes_log2;
  const int hpw = 32 >> a.lanes_log2;           // heads of a pass
  const bool live = 16 * c < a.head_dim;
  const bool rot = 16 * c < a.rot_dim;
  const int ea = rot ? 8 * c : 16 * c;          // the lane's two vectors
  const int eb = rot ? (a.rot_dim >> 1) + 8 * c : 16 * c + 8;
  const int pass0 = part * a.per_warp, pass1 = min(a.passes, pass0 + a.per_warp);

  // where the lane's head of a pass lies; kind -1: none
  struct Item {
    int kind, head;
  };
  auto item = [&](int pass) {
    Item it;
    it.head = pass * hpw + sub;
    it.kind = 0;
    if (it.head >= a.src[0].heads) it.head -= a.src[0].heads, it.kind = 1;
    if (it.kind == 1 && it.head >= a.src[1].heads) it.head -= a.src[1].heads, it.kind = 2;
    if (!live || pass >= pass1 || (it.kind == 2 && it.head >= a.src[2].heads)) it.kind = -1;
    return it;
  };
  auto fetch = [&](const Item& it, Vec8<IN>& va, Vec8<IN>& vb) {
    if (it.kind < 0) return;
    const RopeSrc& s = a.src[it.kind];
    const IN* p = static_cast<const IN*>(s.in) + (size_t)t * s.in_stride + (size_t)it.head * a.head_dim;
    va.load(p + ea);
    vb.load(p + eb);
  };

  Item it = item(pass0);
  Vec8<IN> va, vb;
  fetch(it, va, vb);

  int pos;
  long long slot = -1;  // row of the token's first head in the pools: page * n_kv * page_tokens + offset
  if (a.positions) {
    pos = a.positions[t];
  } else {
    if (a.status && w == 0) check_lengths(a, lane);
    const int b = seq_of(a.cu_q, a.n_seqs, t, lane);
    if (b >= a.n_seqs) return;  // behind the last sequence
    const int start = a.cu_q[b], end = a.cu_q[b + 1], kl = a.kv_len[b];
    const long long room = (long long)a.max_pages << a.page_shift;
    // before the first sequence, or lengths that do not fit (check_lengths
    // flags them).  Where cu_q decreases, seq_of's count can name a sequence
    // that ends before t: only start <= t < end and end - start <= kl <= room
    // put the position into [0, kl), inside the sequence's row of the page
    // table.  A sequence whose kl does not hold its chunk is left out whole.
    if (t < start || t >= end || start < 0 || end > a.n_tokens || kl < end - start || kl > room) return;
    pos = kl - (end - t);
    const int page = a.page_table[(size_t)b * a.max_pages + (pos >> a.page_shift)];
    if (page >= 0 && page < a.n_pages)
      slot = (((long long)page * a.n_kv) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
    else if (a.status && lane == 0)
      atomicOr(a.status, kBadPage);
  }

  // cos and sin of the lane's eight pairs (elements e, e of the two vectors
  // in the halves pairing; 2e, 2e + 1 of each vector in the adjacent one)
  float cs[8], sn[8];
  auto turned = [&](int e, float* sine, float* cosine) {
    const int pair = HALVES ? 8 * c + e : (e < 4 ? 4 * c + e : (a.rot_dim >> 2) + 4 * c + e - 4);
    const unsigned long long f = (unsigned long long)(long long)pos * a.turn[pair & (kMaxPairs - 1)];
    sincospif((float)(int)(f >> 32) * 4.656612873077393e-10f, sine, cosine);  // 2^-31: half turns
  };
  if (a.lanes_log2 <= 3) {
    // four lanes at least hold the same pairs of different heads: each works out two of the eight
    float s0, s1, c0, c1;
    turned(sub & 3, &s0, &c0);
    turned((sub & 3) + 4, &s1, &c1);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int src = (e << a.lanes_log2) + c;
      sn[e] = __shfl_sync(0xffffffffu, s0, src);
      cs[e] = __shfl_sync(0xffffffffu, c0, src);
      sn[e + 4] = __shfl_sync(0xffffffffu, s1, src);
      cs[e + 4] = __shfl_sync(0xffffffffu, c1, src);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) turned(e, &sn[e], &cs[e]);
  }

  for (int pass = pass0; pass < pass1; ++pass) {
    const Item next = item(pass + 1);
    Vec8<IN> na, nb;
    fetch(next, na, nb);
    float xa[8], xb[8];
    float ss = 0.f;
    if (it.kind >= 0) {
      va.get(xa);
      vb.get(xb);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(xa[e], xa[e], fmaf(xb[e], xb[e], ss));
    }
    for (int o = lph >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (it.kind >= 0) {
      const RopeSrc& s = a.src[it.kind];
      if (s.norm) {
        // the weights come from L1 each time: kept, they cost a fifth of the warps
        Vec8<float> na8, nb8;
        na8.load(s.norm + ea);
        nb8.load(s.norm + eb);
        float wa[8], wb[8];
        na8.get(wa);
        nb8.get(wb);
        const float r = rsqrtf(ss * a.inv_hd + a.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) xa[e] *= r * wa[e], xb[e] *= r * wb[e];
      }
      if (rot && s.rotate) {
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
      OUT* p = static_cast<OUT*>(s.out);
      bool ok = true;
      if (s.paged) {
        ok = slot >= 0;
        p += (size_t)(slot + ((long long)it.head << a.page_shift)) * a.head_dim;
      } else {
        p += (size_t)t * s.out_stride + (size_t)it.head * a.head_dim;
      }
      if (ok) {
        Vec8<OUT>::put(p + ea, xa);
        Vec8<OUT>::put(p + eb, xb);
      }
    }
    it = next;
    va = na;
    vb = nb;
  }
}

template <typename IN, typename OUT>
void launch_rope_out(const RopeArgs& a, unsigned grid, cudaStream_t s) {
  if (a.pairing == DLS_ROPE_HALVES) rope_kernel<IN, OUT, true><<<grid, RTHREADS, 0, s>>>(a);
  else rope_kernel<IN, OUT, false><<<grid, RTHREADS, 0, s>>>(a);
}

template <typename IN>
cudaError_t launch_rope_in(const RopeArgs& a, int out_type, unsigned grid, cudaStream_t s) {
  switch (out_type) {
    case DLS_F32: launch_rope_out<IN, float>(a, grid, s); break;
    case DLS_F16: launch_rope_out<IN, __half>(a, grid, s); break;
    default: launch_rope_out<IN, __nv_bfloat16>(a, grid, s); break;
  }
  return cudaGetLastError();
}

int type_bytes(int t) { return t == DLS_F32 ? 4 : t == DLS_F16 || t == DLS_BF16 ? 2 : 0; }

// Rows of `heads * head_dim` elements `stride` apart that 16-byte accesses can reach.
bool rows_ok(const void* p, long long stride, int heads, int hd, int type) {
  return p && !(reinterpret_cast<uintptr_t>(p) & 15) && stride >= (long long)heads * hd &&
         stride <= (1ll << 40) && !((stride * type_bytes(type)) & 15);
}

bool set_turns(RopeArgs* a, const double* inv_freq) {
  for (int i = 0; i < a->rot_dim / 2; ++i) {
    if (!isfinite(inv_freq[i])) return false;
    // the fraction of |inv_freq|, which a double holds exactly; one of a small
    // negative frequency would lie next to 1, on steps of 2^-53 whatever it is
    double turns = fabs(inv_freq[i]) / 6.283185307179586476925286766559;
    turns -= floor(turns);
    const unsigned long long f = (unsigned long long)rint(turns * 18446744073709551616.0);  // 2^64; turns <= 1 - 2^-53
    a->turn[i] = inv_freq[i] < 0.0 ? 0ull - f : f;
  }
  return true;
}

int launch_rope(RopeArgs& a, int in_type, int out_type, const char* what, cudaStream_t s) {
  a.lanes_log2 = 0;
  while ((16 << a.lanes_log2) < a.head_dim) ++a.lanes_log2;
  a.inv_hd = 1.0f / (float)a.head_dim;
  a.heads_total = a.src[0].heads + a.src[1].heads + a.src[2].heads;
  const int hpw = 32 >> a.lanes_log2;
  a.passes = (a.heads_total + hpw - 1) / hpw;
  // Passes of a warp: few enough for three rounds of the 24 warps that an SM
  // holds with 16-bit inputs (with fp32 ones it holds 20, so the rounds are a
  // little more: 1021 tokens of 40 fp32 heads of 64 run 5105 warps of one pass
  // in 1.7 rounds, 7.7 us over a floor of 3.1).  8192 bf16 tokens of 72 heads of 128: 57.7 us with 2 warps a token (9
  // passes each), 59.9 with one (18; the last round a quarter full), 59.5 and
  // 66.5 with 3 and 4 (each repeats the token's start); 46.6 for a plain copy
  // of the bytes.
  const long long want = (long long)a.n_tokens * a.passes / (152 * 24 * 3);
  a.per_warp = (int)(want < 1 ? 1 : want > a.passes ? a.passes : want);
  a.chunks = (a.passes + a.per_warp - 1) / a.per_warp;
  a.per_warp = (a.passes + a.chunks - 1) / a.chunks;
  const long long warps = (long long)a.n_tokens * a.chunks;
  const long long grid = (warps + RTHREADS / 32 - 1) / (RTHREADS / 32);
  if (warps > 0x7fffffff - RTHREADS) return report_error(DLS_ERR_ARG, "%s: n_tokens=%d heads=%d are too many", what, a.n_tokens, a.heads_total);
  cudaError_t e = cudaSuccess;
  if (a.status) e = cudaMemsetAsync(a.status, 0, sizeof(int32_t), s);
  if (e == cudaSuccess) {
    switch (in_type) {
      case DLS_F32: e = launch_rope_in<float>(a, out_type, (unsigned)grid, s); break;
      case DLS_F16: e = launch_rope_in<__half>(a, out_type, (unsigned)grid, s); break;
      default: e = launch_rope_in<__nv_bfloat16>(a, out_type, (unsigned)grid, s); break;
    }
  }
  if (e != cudaSuccess) return report_error(DLS_ERR_CUDA, "%s: cuda=%s", what, cudaGetErrorString(e));
  return DLS_OK;
}

bool rope_shape_ok(int hd, int rot, int pairing, const double* inv_freq, float eps) {
  return hd >= 16 && hd <= 256 && hd % 16 == 0 && rot >= 0 && rot <= hd && rot % 16 == 0 &&
         (pairing == DLS_ROPE_ADJACENT || pairing == DLS_ROPE_HALVES) && (rot == 0 || inv_freq) && eps >= 0.f &&
         isfinite(eps);
}

}  // namespace

}  // namespace dls

extern "C" int dls_qk_norm_rope(const dls_qk_norm_rope_desc* d, void* cuda_stream) {
  using namespace dls;
  if (!d) return report_error(DLS_ERR_ARG, "qk_norm_rope: desc=NULL");
  if (!rope_shape_ok(d->head_dim, d->rot_dim, d->pairing, d->inv_freq, d->eps))
    return report_error(DLS_ERR_ARG, "qk_norm_rope: head_dim=%d rot_dim=%d (multiples of 16, at most 256) pairing=%d inv_freq=%p eps=%g",
                        d->head_dim, d->rot_dim, d->pairing, (const void*)d->inv_freq, d->eps);
  if (!type_bytes(d->in_type) || !type_bytes(d->out_type))
    return report_error(DLS_ERR_ARG, "qk_norm_rope: in_type=%d out_type=%d", d->in_type, d->out_type);
  if (d->n_tokens < 0 || d->n_heads < 0 || d->n_kv_heads < 0 || d->n_heads > 4096 || d->n_kv_heads > 4096)
    return report_error(DLS_ERR_ARG, "qk_norm_rope: n_tokens=%d n_heads=%d n_kv_heads=%d", d->n_tokens, d->n_heads, d->n_kv_heads);
  if (d->n_tokens == 0 || d->n_heads + d->n_kv_heads == 0) return DLS_OK;
  if (!d->positions || !aligned_to(d->positions, 4) || !aligned_to(d->q_norm, 16) || !aligned_to(d->k_norm, 16))
    return report_error(DLS_ERR_ARG, "qk_norm_rope: positions=%p q_norm=%p k_norm=%p (16-byte aligned norms)", (const void*)d->positions,
                        (const void*)d->q_norm, (const void*)d->k_norm);
  if ((d->n_heads && (!rows_ok(d->q, d->q_stride, d->n_heads, d->head_dim, d->in_type) ||
                      !rows_ok(d->q_out, d->q_out_stride, d->n_heads, d->head_dim, d->out_type))) ||
      (d->n_kv_heads && (!rows_ok(d->k, d->k_stride, d->n_kv_heads, d->head_dim, d->in_type) ||
                         !rows_ok(d->k_out, d->k_out_stride, d->n_kv_heads, d->head_dim, d->out_type))))
    return report_error(DLS_ERR_ARG, "qk_norm_rope: q, k and their outputs need 16-byte aligned rows of heads * head_dim elements");
  if ((d->n_heads && d->q == d->q_out && (d->in_type != d->out_type || d->q_stride != d->q_out_stride)) ||
      (d->n_kv_heads && d->k == d->k_out && (d->in_type != d->out_type || d->k_stride != d->k_out_stride)))
    return report_error(DLS_ERR_ARG, "qk_norm_rope: in place needs the same type and stride");
  RopeArgs a{};
  a.src[0] = {d->q, d->q_out, d->q_norm, d->q_stride, d->q_out_stride, d->n_heads, 1, 0};
  a.src[1] = {d->k, d->k_out, d->k_norm, d->k_stride, d->k_out_stride, d->n_kv_heads, 1, 0};
  a.positions = d->positions;
  a.n_tokens = d->n_tokens;
  a.head_dim = d->head_dim;
  a.rot_dim = d->rot_dim;
  a.pairing = d->pairing;
  a.eps = d->eps;
  if (!set_turns(&a, d->inv_freq)) return report_error(DLS_ERR_ARG, "qk_norm_rope: inv_freq is not finite");
  return launch_rope(a, d->in_type, d->out_type, "qk_norm_rope", static_cast<cudaStream_t>(cuda_stream));
}

extern "C" int dls_kv_append(const dls_kv_append_desc* d, void* cuda_stream) {
  using namespace dls;
  if (!d) return report_error(DLS_ERR_ARG, "kv_append: desc=NULL");
  if (!rope_shape_ok(d->head_dim, d->rot_dim, d->pairing, d->inv_freq, d->eps))
    return report_error(DLS_ERR_ARG, "kv_append: head_dim=%d rot_dim=%d (multiples of 16, at most 256) pairing=%d inv_freq=%p eps=%g",
                        d->head_dim, d->rot_dim, d->pairing, (const void*)d->inv_freq, d->eps);
  if (!type_bytes(d->in_type) || (d->kv_type != DLS_F16 && d->kv_type != DLS_BF16))
    return report_error(DLS_ERR_ARG, "kv_append: in_type=%d kv_type=%d", d->in_type, d->kv_type);
  const int pt = d->page_tokens;
  if (pt != 16 && pt != 32 && pt != 64 && pt != 128 && pt != 256)
    return report_error(DLS_ERR_ARG, "kv_append: page_tokens=%d (16, 32, 64, 128 or 256)", pt);
  if (d->n_tokens < 0 || d->n_seqs < 0 || d->n_seqs > 1 << 30 || d->n_kv_heads < 1 || d->n_kv_heads > 4096 || d->n_pages < 1 ||
      d->max_pages < 1 || (long long)d->max_pages * pt > 0x7fffffff || (d->q && (d->n_heads < 1 || d->n_heads > 4096)))
    return report_error(DLS_ERR_ARG, "kv_append: n_tokens=%d n_seqs=%d n_heads=%d n_kv_heads=%d n_pages=%d max_pages=%d", d->n_tokens,
                        d->n_seqs, d->n_heads, d->n_kv_heads, d->n_pages, d->max_pages);
  if (!aligned_to(d->status, 4)) return report_error(DLS_ERR_ARG, "kv_append: status=%p", (void*)d->status);
  if (d->n_tokens == 0 || d->n_seqs == 0) return empty_call(d->status, cuda_stream, "kv_append");
  if (!d->page_table || !d->cu_q || !d->kv_len || !aligned_to(d->page_table, 4) || !aligned_to(d->cu_q, 4) || !aligned_to(d->kv_len, 4))
    return report_error(DLS_ERR_ARG, "kv_append: page_table=%p cu_q=%p kv_len=%p", (const void*)d->page_table, (const void*)d->cu_q,
                        (const void*)d->kv_len);
  if (!aligned_to(d->q_norm, 16) || !aligned_to(d->k_norm, 16))
    return report_error(DLS_ERR_ARG, "kv_append: q_norm=%p k_norm=%p (16-byte aligned)", (const void*)d->q_norm, (const void*)d->k_norm);
  if (!rows_ok(d->k, d->k_stride, d->n_kv_heads, d->head_dim, d->in_type) ||
      !rows_ok(d->v, d->v_stride, d->n_kv_heads, d->head_dim, d->in_type) ||
      (d->q && (!rows_ok(d->q, d->q_stride, d->n_heads, d->head_dim, d->in_type) ||
                !rows_ok(d->q_out, d->q_out_stride, d->n_heads, d->head_dim, d->kv_type))))
    return report_error(DLS_ERR_ARG, "kv_append: k, v, q and q_out need 16-byte aligned rows of heads * head_dim elements");
  if (!d->k_pages || !d->v_pages || ((reinterpret_cast<uintptr_t>(d->k_pages) | reinterpret_cast<uintptr_t>(d->v_pages)) & 15))
    return report_error(DLS_ERR_ARG, "kv_append: k_pages=%p v_pages=%p (16-byte aligned)", d->k_pages, d->v_pages);
  if (d->q && d->q == d->q_out && (d->in_type != d->kv_type || d->q_stride != d->q_out_stride))
    return report_error(DLS_ERR_ARG, "kv_append: in place needs the same type and stride");
  RopeArgs a{};
  if (d->q) a.src[0] = {d->q, d->q_out, d->q_norm, d->q_stride, d->q_out_stride, d->n_heads, 1, 0};
  a.src[1] = {d->k, d->k_pages, d->k_norm, d->k_stride, 0, d->n_kv_heads, 1, 1};
  a.src[2] = {d->v, d->v_pages, nullptr, d->v_stride, 0, d->n_kv_heads, 0, 1};
  a.page_table = d->page_table;
  a.cu_q = d->cu_q;
  a.kv_len = d->kv_len;
  a.status = d->status;
  a.n_tokens = d->n_tokens;
  a.n_seqs = d->n_seqs;
  a.n_kv = d->n_kv_heads;
  a.n_pages = d->n_pages;
  a.max_pages = d->max_pages;
  a.page_shift = pt == 16 ? 4 : pt == 32 ? 5 : pt == 64 ? 6 : pt == 128 ? 7 : 8;
  a.head_dim = d->head_dim;
  a.rot_dim = d->rot_dim;
  a.pairing = d->pairing;
  a.eps = d->eps;
  if (!set_turns(&a, d->inv_freq)) return report_error(DLS_ERR_ARG, "kv_append: inv_freq is not finite");
  return launch_rope(a, d->in_type, d->kv_type, "kv_append", static_cast<cudaStream_t>(cuda_stream));
}
