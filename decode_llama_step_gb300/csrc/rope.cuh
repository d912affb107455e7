// Pieces that the kernels around norm, rotation and the append share: vectors
// of eight elements, a row's sequence, and a frequency as a part of a turn.
#pragma once
#include <cuda_bf16.h>
#include <math.h>

#include "../../include/dls.h"
#include "common.cuh"

namespace dls {

constexpr int kMaxPairs = 128;   // rot_dim <= 256

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

inline int type_bytes(int t) { return t == DLS_F32 ? 4 : t == DLS_F16 || t == DLS_BF16 ? 2 : 0; }

// Rows of `heads * head_dim` elements `stride` apart that 16-byte accesses can reach.
inline bool rows_ok(const void* p, long long stride, int heads, int hd, int type) {
  return p && !(reinterpret_cast<uintptr_t>(p) & 15) && stride >= (long long)heads * hd &&
         stride <= (1ll << 40) && !((stride * type_bytes(type)) & 15);
}

// inv_freq[i] in parts of a turn, a turn being 2^64 (see rope_append.cu).
inline bool set_turns(unsigned long long* turn, int rot_dim, const double* inv_freq) {
  for (int i = 0; i < rot_dim / 2; ++i) {
    if (!isfinite(inv_freq[i])) return false;
    // the fraction of |inv_freq|, which a double holds exactly; one of a small
    // negative frequency would lie next to 1, on steps of 2^-53 whatever it is
    double turns = fabs(inv_freq[i]) / 6.283185307179586476925286766559;
    turns -= floor(turns);
    const unsigned long long f = (unsigned long long)rint(turns * 18446744073709551616.0);  // 2^64; turns <= 1 - 2^-53
    turn[i] = inv_freq[i] < 0.0 ? 0ull - f : f;
  }
  return true;
}

inline bool rope_shape_ok(int hd, int rot, int pairing, const double* inv_freq, float eps) {
  return hd >= 16 && hd <= 256 && hd % 16 == 0 && rot >= 0 && rot <= hd && rot % 16 == 0 &&
         (pairing == DLS_ROPE_ADJACENT || pairing == DLS_ROPE_HALVES) && (rot == 0 || inv_freq) && eps >= 0.f &&
         isfinite(eps);
}

}  // namespace dls
