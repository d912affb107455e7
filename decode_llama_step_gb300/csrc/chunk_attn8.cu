// Attention over pages of 8-bit codes: the kernels of chunk_attn.cuh over both
// kinds of codes.
#include "chunk_attn.cuh"

namespace dls {

namespace {

template <typename T, int CODE>
ChunkFn codes_fn(int hd) {
  return hd <= 64 ? chunk_kernel<T, 64, CODE> : chunk_kernel<T, 128, CODE>;
}
ChunkFn codes_fn(int hd, int code, bool half) {
  return code == DLS_E4M3 ? (half ? codes_fn<__half, DLS_E4M3>(hd) : codes_fn<__nv_bfloat16, DLS_E4M3>(hd))
                          : (half ? codes_fn<__half, DLS_I8>(hd) : codes_fn<__nv_bfloat16, DLS_I8>(hd));
}
int codes_smem(int hd) { return hd <= 64 ? chunk_smem<64, DLS_E4M3>() : chunk_smem<128, DLS_E4M3>(); }

}  // namespace

cudaError_t chunk_codes_setup() {
  for (int i = 0; i < 8; ++i) {
    const int hd = i & 1 ? 64 : 128;
    const cudaError_t e =
        cudaFuncSetAttribute(codes_fn(hd, i & 2 ? DLS_I8 : DLS_E4M3, i & 4), cudaFuncAttributeMaxDynamicSharedMemorySize, codes_smem(hd));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_chunk_codes(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const ChunkArgs& a, int code, bool half,
                               int ctas, cudaStream_t s) {
  codes_fn(a.head_dim, code, half)<<<ctas, kThreads<DLS_E4M3>, codes_smem(a.head_dim), s>>>(tq, tk, tv, a);
  return cudaGetLastError();
}

}  // namespace dls
