// Verification of drafted tokens against the target's probabilities, from
// given random numbers.
//
// Mathematics, per sequence: its rows are the current token and the drafts;
// target row r gives p (and draft row r gives q, from which the token of row r
// + 1 was drawn).  Draft x of row r + 1 stands while u[r] q(x) < p(x).  At the
// first that does not, the token comes from w = max(p - q, 0); where all stand,
// from w = p of the last row:
//   token = the least t with  sum_{j <= t} w_j > v sum_j w_j.
// Without draft probabilities the draft was certain (q(x) = 1): x stands while
// u < p(x), and w is p without x.
//
// Which token it is must not depend on how the sums are formed: 128256
// borders, most of them of unlikely tokens, lie so close that the rounding of
// a 32-bit sum (or of p - q in 32 bits) moves the pick past some of them.  So
// p and q become whole numbers of 2^-45 (to the nearest: 2^21 of them on the
// random numbers' own 2^-24) and everything after is integer arithmetic: sums
// in any order give the same bits, and v sum w is compared exactly (its floor,
// against whole sums).  u q(x) < p(x) is exact in a double.  The conversion
// takes two additions: p + 2 holds p's first 22 bits in its mantissa, and what
// is left, added to 3 2^-23, the next 23 (units of 2^-60 by shifts: 24 us for 64
// sequences where this took 21, both with the kind of weight asked at every pair).
//
// What bounds it: the bytes of one row of p and one of q a sequence; the rows
// of drafts that stand are never read but at one token.  A cluster of CTAs
// takes a sequence, each a slice of the vocabulary: sums, exchanged through
// distributed shared memory, then the CTA whose slice holds the border finds
// the warp, the lane and the token by prefix sums of the (cached) slice.
// Measured (GPU time; 128256 tokens, fp32): one sequence 6.9 us, 64 sequences
// 16.9 us (9.8 at the copy rate), 22.7 with the rows in HBM.
#include <cuda_bf16.h>
#include <math.h>

#include <type_traits>

#include "../../include/dls.h"
#include "kernels.h"

namespace dls {

namespace {

constexpr int kMostThreadsV = 512;
constexpr int kMaxCluster = 8;
typedef unsigned long long u64_t;

struct VerifyArgs {
  const int32_t *tokens, *cu_q, *kv_len;
  const float *accept, *pick;
  const void *target, *draft;
  long long target_stride, draft_stride;
  int32_t *out_tokens, *n_accepted, *kv_len_out, *status;
  int n_tokens, n_seqs, vocab;
  int wide;  // rows of both lie alike to 16 bytes (or there is no draft)
};

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// Two probabilities in whole numbers of 2^-45, each as hi * 2^23 + lo; outside
// [0, 1] the nearer end, NaN 0.
__device__ __forceinline__ float saturated(float x) {
  float y;
  asm("add.sat.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
  return y;
}
// (as the bits of the sums: kHi and kLo more than the numbers)
constexpr int kHi = 0x40000000, kLo = 0x34c00000;
__device__ __forceinline__ void units2(float x, float y, int (&hi)[2], int (&lo)[2]) {
  const f2_t v = pk2(x, y), h = fadd2(v, pk2(2.f, 2.f));                // steps of 2^-22
  const f2_t rest = fadd2(v, ffma2(h, pk2(-1.f, -1.f), pk2(2.f, 2.f)));  // exact, at most 2^-23
  const f2_t l = fadd2(rest, pk2(0x1.8p-22f, 0x1.8p-22f));               // steps of 2^-45
  hi[0] = __float_as_int(upk2(h).x), hi[1] = __float_as_int(upk2(h).y);
  lo[0] = __float_as_int(upk2(l).x), lo[1] = __float_as_int(upk2(l).y);
}
__device__ __forceinline__ u64_t joined(int hi, int lo) { return (u64_t)((long long)hi * (1 << 23) + lo); }

// floor(v s) below s, v in [0, 1)
__device__ __forceinline__ u64_t part_of(u64_t s, float v) {
  const unsigned b = __float_as_uint(fminf(fmaxf(v, 0.f), 0x1.fffffep-1f)), e = b >> 23;
  const unsigned m = e ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
  const unsigned sh = 150u - (e ? e : 1u);  // v = m 2^-sh, 24 <= sh
  const u64_t lo = s * m, hi = __umul64hi(s, m);
  if (sh < 64) return (hi << (64 - sh)) | (lo >> sh);
  return sh < 128 ? hi >> (sh - 64) : 0;
}

// A row in pieces of V elements: piece k holds elements k V - off ..., off such
// that pieces lie at 16-byte boundaries (V = 1: single elements).  Whole
// pieces are loaded as they lie; those at the ends, element by element.
template <typename T, int V>
struct Piece16 {
  typename std::conditional<(V > 1), uint4, T>::type w;
  __device__ __forceinline__ void load(const T* row, int first) {
    if constexpr (V > 1) w = __ldg(reinterpret_cast<const uint4*>(row + first));
    else w = row[first];
  }
  __device__ __forceinline__ void get(float (&x)[V]) const {
    if constexpr (V == 1) {
      x[0] = as_float(w);
    } else {
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(u[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const unsigned short h = (unsigned short)(i & 1 ? u[i >> 1] >> 16 : u[i >> 1]);
          if constexpr (std::is_same<T, __half>::value) x[i] = __half2float(__ushort_as_half(h));
          else x[i] = __uint_as_float((uint32_t)h << 16);
        }
      }
    }
  }
};
template <typename T, int V>
__device__ __forceinline__ void ends(const T* row, int first, int vocab, float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = first + i >= 0 && first + i < vocab ? as_float(row[first + i]) : 0.f;
}

// Weight of an element: of p alone, of p without token x, or of what p has over q.
enum What { ALONE, WITHOUT, OVER };

// Sums of weights and of p alone, hi and lo apart, of few elements (hi is at
// most 2^22, lo up to that either way; unsigned: what wraps on the way is gone
// at the end).
struct Sums {
  unsigned hi, lo, p_hi, p_lo;
};
// Adds V elements; `each` is told the weight of every one.
template <int V, typename Each>
__device__ __forceinline__ void weigh(const float (&p)[V], const float (&q)[V], int first, int what, int x, Sums& s, Each&& each) {
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    const float p0 = saturated(p[i]), p1 = V > 1 ? saturated(p[i + (V > 1)]) : 0.f;
    int h[2], l[2];
    units2(p0, p1, h, l);
    constexpr unsigned n = V > 1 ? 2 : 1;
    s.p_hi += (unsigned)h[0] + (V > 1 ? (unsigned)h[1] : 0u) - n * kHi, s.p_lo += (unsigned)l[0] + (V > 1 ? (unsigned)l[1] : 0u) - n * kLo;
    int g[2] = {kHi, kHi}, k[2] = {kLo, kLo};
    bool in[2] = {true, V > 1};
    if (what == OVER) {
      const float q0 = saturated(q[i]), q1 = V > 1 ? saturated(q[i + (V > 1)]) : 0.f;
      units2(q0, q1, g, k);
      in[0] = p0 > q0, in[1] = V > 1 && p1 > q1;
    } else if (what == WITHOUT) {
      in[0] = first + i != x, in[1] = V > 1 && first + i + 1 != x;
    }
#pragma unroll
    for (int e = 0; e < (int)n; ++e) {
      if (in[e]) s.hi += (unsigned)(h[e] - g[e]), s.lo += (unsigned)(l[e] - k[e]);
      each(i + e, in[e] ? joined(h[e] - g[e], l[e] - k[e]) : 0);
    }
  }
}

__device__ __forceinline__ u64_t warp_sum64(u64_t v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T, int V>
__global__ void __launch_bounds__(kMostThreadsV, 2) verify_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ u64_t warp_sums[kMostThreadsV / 32][2];
  __shared__ __align__(16) u64_t all[kMaxCluster][2];  // each CTA's sums
  __shared__ int s_stop;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta_warps = blockDim.x >> 5;
  unsigned rank, ctas;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  const int b = blockIdx.x / ctas;
  const int start = a.cu_q[b], end = a.cu_q[b + 1];
  const bool bad = start < 0 || end < start || end > a.n_tokens;
  if (bad || start == end) {  // (the whole cluster alike)
    if (rank == 0 && tid == 0) {
      a.n_accepted[b] = 0;
      if (a.kv_len_out) a.kv_len_out[b] = a.kv_len[b];
      if (bad && a.status) atomicOr(a.status, kBadPos);
    }
    return;
  }
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const T *target = static_cast<const T*>(a.target), *draft = static_cast<const T*>(a.draft);

  // the first row whose draft does not stand, or the last row
  if (warp == 0) {
    int stop = end - 1, r = start;
    bool strange = false;
    for (; r < end - 1; r += 32) {
      const int row = r + lane;
      bool falls = false;
      if (row < end - 1) {
        const int x = a.tokens[row + 1];
        const bool in = x >= 0 && x < a.vocab;
        strange |= !in;
        double p = 0., q = 1.;
        if (in) {
          p = as_float(target[(size_t)row * a.target_stride + x]);
          if (draft) q = as_float(draft[(size_t)row * a.draft_stride + x]);
        }
        falls = !(in && (double)a.accept[row] * q < p);
      }
      const unsigned hit = __ballot_sync(0xffffffffu, falls);
      if (hit) {
        stop = r + __ffs(hit) - 1;
        break;
      }
    }
    if (lane == 0) s_stop = stop;
    if (rank == 0 && a.status)  // tokens behind the 32 that were looked at last
      for (r += 32 + lane; r < end - 1; r += 32) strange |= a.tokens[r + 1] < 0 || a.tokens[r + 1] >= a.vocab;
    if (strange && rank == 0 && a.status) atomicOr(a.status, kBadToken);
  }
  __syncthreads();
  const int stop = s_stop;
  const bool refused = stop < end - 1;
  if (rank == 0) {
    for (int r = start + tid; r < end; r += blockDim.x)
      if (r != stop) a.out_tokens[r] = r < stop ? a.tokens[r + 1] : -1;
    if (tid == 0) {
      a.n_accepted[b] = stop - start;
      if (a.kv_len_out) a.kv_len_out[b] = a.kv_len[b] - (end - 1 - stop);
    }
  }

  // sums: warp's run of pieces inside the CTA's slice of the row
  const T* const p = target + (size_t)stop * a.target_stride;
  const T* const q = draft ? draft + (size_t)stop * a.draft_stride : nullptr;
  const int what = !refused ? ALONE : draft ? OVER : WITHOUT;
  const int x = refused ? a.tokens[stop + 1] : -1;
  const int off = V > 1 ? (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T)) : 0;
  const int pieces = (a.vocab + off + V - 1) / V;
  const int per_warp = (pieces + (int)ctas * cta_warps - 1) / ((int)ctas * cta_warps);
  const int c0 = (int)min((long long)(rank * cta_warps + warp) * per_warp, (long long)pieces), c1 = min(c0 + per_warp, pieces);
  const int in0 = off ? 1 : 0, in1 = (a.vocab + off) / V;  // whole pieces
  u64_t sum = 0, plain = 0;
  constexpr int U = V == 8 ? 2 : 4;  // pieces in flight
  // (a loop for each kind: asked at every pair of elements, the kind took as many instructions as the sums)
  auto add_up = [&](auto kind) {
    constexpr int WHAT = decltype(kind)::value;
    for (int c = max(c0, in0) + lane; c < min(c1, in1); c += 32 * U) {
      Piece16<T, V> pp[U], qq[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int at = min(c + 32 * k, in1 - 1) * V - off;
        pp[k].load(p, at);
        if (WHAT == OVER) qq[k].load(q, at);
      }
      Sums s{};
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (c + 32 * k >= min(c1, in1)) continue;
        float x_p[V], x_q[V];
        pp[k].get(x_p);
        if (WHAT == OVER) qq[k].get(x_q);
        weigh<V>(x_p, x_q, (c + 32 * k) * V - off, WHAT, x, s, [](int, u64_t) {});
      }
      sum += joined((int)s.hi, (int)s.lo);  // (16 elements)
      plain += joined((int)s.p_hi, (int)s.p_lo);
    }
  };
  if (what == OVER) add_up(std::integral_constant<int, OVER>());
  else if (what == WITHOUT) add_up(std::integral_constant<int, WITHOUT>());
  else add_up(std::integral_constant<int, ALONE>());
  auto any_piece = [&](int c, int how, Sums& s, auto&& each) {
    float x_p[V], x_q[V];
    if (c >= in0 && c < in1) {
      Piece16<T, V> pp, qq;
      pp.load(p, c * V - off);
      if (how == OVER) qq.load(q, c * V - off);
      pp.get(x_p);
      if (how == OVER) qq.get(x_q);
    } else {
      ends<T, V>(p, c * V - off, a.vocab, x_p);
      if (how == OVER) ends<T, V>(q, c * V - off, a.vocab, x_q);
    }
    weigh<V>(x_p, x_q, c * V - off, how, x, s, each);
  };
  if (lane < 2) {  // the piece before the whole ones, the one behind
    const int c = lane ? in1 : 0;
    if (c >= c0 && c < c1 && (lane ? in1 >= in0 : in0 > 0)) {
      Sums s{};
      any_piece(c, what, s, [](int, u64_t) {});
      sum += joined((int)s.hi, (int)s.lo);
      plain += joined((int)s.p_hi, (int)s.p_lo);
    }
  }
  sum = warp_sum64(sum);
  plain = warp_sum64(plain);
  if (lane == 0) warp_sums[warp][0] = sum, warp_sums[warp][1] = plain;
  __syncthreads();
  if (warp == 0) {
    u64_t s = lane < cta_warps ? warp_sums[lane][0] : 0, u = lane < cta_warps ? warp_sums[lane][1] : 0;
    s = warp_sum64(s);
    u = warp_sum64(u);
    // to every CTA of the cluster (all have begun: they arrived)
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    if (lane < (int)ctas) {
      uint32_t at;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(&all[rank][0])), "r"(lane));
      asm volatile("st.shared::cluster.v2.u64 [%0], {%1, %2};" ::"r"(at), "l"(s), "l"(u) : "memory");
    }
  } else {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  u64_t total = 0, before = 0;
  int col = 0;
  for (int k = 0; k < (int)ctas; ++k) {
    if (k == (int)rank) before = total;
    total += all[k][0];
  }
  int how = what;
  if (total == 0) {  // nothing over the draft's: p itself
    col = 1, how = ALONE;
    for (int k = 0; k < (int)ctas; ++k) {
      if (k == (int)rank) before = total;
      total += all[k][1];
    }
  }
  if (total == 0) {
    if (rank == 0 && tid == 0) {
      a.out_tokens[stop] = -1;
      if (a.status) atomicOr(a.status, kBadToken);
    }
    return;
  }
  const u64_t border = part_of(total, a.pick[b]);
  // the warp whose run passes the border
  for (int w = 0; w < warp; ++w) before += warp_sums[w][col];
  if (!(before <= border && before + warp_sums[warp][col] > border)) return;
  for (int c = c0; c < c1; c += 32) {
    u64_t mine = 0, w[V];
    if (c + lane < c1) {
      Sums s{};
      any_piece(c + lane, how, s, [&](int i, u64_t x) { w[i] = x; });
      mine = joined((int)s.hi, (int)s.lo);
    }
    u64_t pre = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64_t y = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) pre += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + pre > border);
    if (hit) {
      if (lane == __ffs(hit) - 1) {
        u64_t at = before + pre - mine;
        int t = (c + lane) * V - off;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          at += w[i];
          if (at <= border) ++t;
        }
        a.out_tokens[stop] = t;
      }
      return;
    }
    before += __shfl_sync(0xffffffffu, pre, 31);
  }
}

template <typename T>
cudaError_t launch_verify(const VerifyArgs& a, unsigned ctas, cudaStream_t s) {
  cudaLaunchConfig_t c{};
  cudaLaunchAttribute at[1];
  // (many sequences: smaller blocks, four an SM, go round it evenly)
  c.gridDim = dim3(ctas * (unsigned)a.n_seqs), c.blockDim = dim3(ctas * (unsigned)a.n_seqs <= 152 ? kMostThreadsV : kMostThreadsV / 2), c.stream = s;
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas, at[0].val.clusterDim.y = 1, at[0].val.clusterDim.z = 1;
  c.attrs = at, c.numAttrs = 1;
  return a.wide ? cudaLaunchKernelEx(&c, verify_kernel<T, 16 / (int)sizeof(T)>, a) : cudaLaunchKernelEx(&c, verify_kernel<T, 1>, a);
}

}  // namespace

}  // namespace dls

extern "C" int dls_verify_draft(const dls_verify_draft_desc* d, void* cuda_stream) {
  using namespace dls;
  if (!d) return report_error(DLS_ERR_ARG, "verify_draft: desc=NULL");
  const int size = d->prob_type == DLS_F32 ? 4 : d->prob_type == DLS_F16 || d->prob_type == DLS_BF16 ? 2 : 0;
  if (!size) return report_error(DLS_ERR_ARG, "verify_draft: prob_type=%d", d->prob_type);
  if (d->n_tokens < 0 || d->n_seqs < 0 || d->n_seqs > 1 << 24 || d->vocab < 1 || d->vocab > 1 << 18)
    return report_error(DLS_ERR_ARG, "verify_draft: n_tokens=%d n_seqs=%d (at most 2^24) vocab=%d (1 to 2^18)", d->n_tokens, d->n_seqs, d->vocab);
  if (d->target_stride < d->vocab || d->target_stride > 1ll << 32 || (d->draft && (d->draft_stride < d->vocab || d->draft_stride > 1ll << 32)))
    return report_error(DLS_ERR_ARG, "verify_draft: target_stride=%lld draft_stride=%lld (vocab=%d to 2^32)", (long long)d->target_stride,
                        (long long)d->draft_stride, d->vocab);
  if (!aligned_to(d->status, 4)) return report_error(DLS_ERR_ARG, "verify_draft: status=%p", (void*)d->status);
  if (d->n_seqs == 0) return empty_call(d->status, cuda_stream, "verify_draft");
  if (!d->cu_q || !d->n_accepted || (!d->kv_len != !d->kv_len_out))
    return report_error(DLS_ERR_ARG, "verify_draft: cu_q=%p n_accepted=%p kv_len=%p kv_len_out=%p (both lengths, or neither)",
                        (const void*)d->cu_q, (void*)d->n_accepted, (const void*)d->kv_len, (void*)d->kv_len_out);
  if (d->n_tokens && (!d->tokens || !d->target || !d->accept || !d->pick || !d->out_tokens))
    return report_error(DLS_ERR_ARG, "verify_draft: tokens=%p target=%p accept=%p pick=%p out_tokens=%p", (const void*)d->tokens, d->target,
                        (const void*)d->accept, (const void*)d->pick, (void*)d->out_tokens);
  const void* words[] = {d->tokens, d->cu_q, d->accept, d->pick, d->kv_len, d->out_tokens, d->n_accepted, d->kv_len_out};
  for (const void* w : words)
    if (!aligned_to(w, 4)) return report_error(DLS_ERR_ARG, "verify_draft: %p is not aligned to its 4-byte elements", w);
  if (!aligned_to(d->target, size) || !aligned_to(d->draft, size))
    return report_error(DLS_ERR_ARG, "verify_draft: target=%p draft=%p are not aligned to their elements", d->target, d->draft);
  if (d->out_tokens && d->out_tokens == d->tokens) return report_error(DLS_ERR_ARG, "verify_draft: out_tokens cannot be tokens");
  VerifyArgs a{};
  a.tokens = d->tokens, a.cu_q = d->cu_q, a.kv_len = d->kv_len, a.accept = d->accept, a.pick = d->pick;
  a.target = d->target, a.draft = d->draft, a.target_stride = d->target_stride, a.draft_stride = d->draft_stride;
  a.out_tokens = d->out_tokens, a.n_accepted = d->n_accepted, a.kv_len_out = d->kv_len_out, a.status = d->status;
  a.n_tokens = d->n_tokens, a.n_seqs = d->n_seqs, a.vocab = d->vocab;
  // rows r of both begin at the same place of a 16-byte piece for every r
  a.wide = !d->draft || (!((reinterpret_cast<uintptr_t>(d->target) ^ reinterpret_cast<uintptr_t>(d->draft)) & 15) &&
                         !(((d->target_stride - d->draft_stride) * size) & 15));
  unsigned ctas = kMaxCluster;
  while (ctas > 1 && ((long long)ctas * d->n_seqs > 608 || d->vocab < 2048 * (int)ctas)) ctas /= 2;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e = cudaSuccess;
  if (a.status) e = cudaMemsetAsync(a.status, 0, sizeof(int32_t), s);
  if (e == cudaSuccess)
    e = d->prob_type == DLS_F32 ? launch_verify<float>(a, ctas, s) : d->prob_type == DLS_F16 ? launch_verify<__half>(a, ctas, s)
                                                                                              : launch_verify<__nv_bfloat16>(a, ctas, s);
  if (e != cudaSuccess) return report_error(DLS_ERR_CUDA, "verify_draft: cuda=%s", cudaGetErrorString(e));
  return DLS_OK;
}
