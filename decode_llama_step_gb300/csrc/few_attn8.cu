// Attention over pages of 8-bit codes for few rows: at most sixteen rows (new
// tokens x query heads of a KV head) a tile of work, as single tokens and
// short verify passes have them.
//
// The mathematics and the division of the work are those of chunk_attn.cuh.
// There a tile of codes is converted in shared memory for the 5th-generation
// tensor core, whose operands of 128 rows lie there: it is written by the copy,
// read and written twice as wide by the conversion and read by the product, 1536
// cycles of shared memory's 128 bytes a cycle for 128 keys of 128, as long as
// HBM takes to bring them (745 cycles a 16 KB), and the chain copy -
// conversion - product - softmax - product passes through barriers at every
// step.  Sixteen rows need no such operands.  Here a warp takes sixteen keys at
// a time for itself: codes come from memory into a ring by TMA, go to
// registers once (conflict-free through the copy's swizzle), are converted
// there and are the fragments of the warp-wide product m16n8k16 as they lie:
//   S = Q K^T  lane 4r + c holds dimensions [32 c, 32 c + 32) of key r: four
//              codes of them are its part of a k-step, q's fragments follow
//   O += P V   lane 4r + c holds dimensions [16 r, 16 r + 16) of keys 2c,
//              2c + 1, 2c + 8, 2c + 9: byte permutes pair the keys
// (head_dim 128; half of each at 64; other ones are read by words as they lie:
// k-step s is dimensions [16 s, 16 s + 16), four of them a lane, and the lane's
// dimensions of V are [32 i + 4 r, 32 i + 4 r + 4), and two of a last half).
// The scores' fragment is the weights'.
// Eight such warps work on 128 keys; each keeps its own (R, l, O), joined in
// shared memory at the end of a piece and, where a tile was cut, through the
// workspace in range order.
//
// What bounds it, measured (GPU time): 64 single tokens of 64 heads over up to
// 8192 cached (0.7 GB of codes) 121 us, 5.8 TB/s of 6.7 (272 us through the
// tensor-memory kernel): HBM, with a warp's step of 1450 cycles for 1310 of
// HBM's close behind it.  One token over 2048, 32 heads: 9.4 us, a chain of launch, plan, page table, copy,
// step and join.  Sixteen warps of 96 registers in place of eight: 202 us (their
// steps spill); copies for each warp apart, 2 KB each: 186.
#include <type_traits>

#include "chunk_attn.cuh"

namespace dls {

namespace {

constexpr int FWARPS = 8;
constexpr int FTHREADS = (FWARPS + 2) * 32;   // with one warp for the copies, one for the scales
constexpr int FK = 16;             // keys of a warp's step; FWARPS * FK = BK
static_assert(FWARPS * FK == BK, "a key tile is a round of the warps");
// What a tile of work costs beyond its key tiles, in key tiles.  1, 3, 6 and 12 of them: 64 single tokens 123.2, 123.4,
// 124.8, 128.1 us; eight verify passes 17.5, 17.5, 18.3, 21.2.
constexpr int kFewCost = 1;
constexpr int kFewSteps = 1;       // key tiles of a range at least (one token over 2048: 9.4 us, 11.8 with four)

template <int HD, bool WIDE>
struct FCfg {
  static constexpr int kRows = WIDE ? 16 : 8;
  static constexpr int kPart = BK * HD;              // bytes of a key tile's K or V
  static constexpr int kStage = 2 * kPart;
  static constexpr int NST = 131072 / kStage < 8 ? 131072 / kStage : 8;  // 128 KB in flight an SM
  static constexpr int kMergeOff = NST * kStage;
  static constexpr bool kWide16 = HD == 64 || HD == 128;      // read 16 bytes at a time, through a swizzle
  static constexpr int kRowF = kWide16 ? HD : HD + 4;         // floats of a row where shares are joined
  static constexpr int kMergeBytes = FWARPS * kRows * kRowF * 4;
  static constexpr int kEnd = kMergeOff + (kMergeBytes < MAXC * 32 * 4 ? MAXC * 32 * 4 : kMergeBytes);  // (or a join's statistics)
  static constexpr int kMiscOff = kEnd < DLS_MAX_CHUNK_SEQS * 16 ? DLS_MAX_CHUNK_SEQS * 16 : kEnd;        // (or the lengths being planned over)
};
struct FMisc {
  uint64_t full[8], empty[8], pq_full[QDEPTH], pq_empty[QDEPTH];
  Piece pq[QDEPTH];
  float scale[8][2][FWARPS];     // of a stage: K's and V's for each warp's keys
  float R[FWARPS][16], l[FWARPS][16];
  long long scan[FWARPS + 2];
  long long range0, range1, per;
  int b0, t0, off0, kvh0, start0, ql0, kl0;
  int abort, last;
};
template <int HD, bool WIDE>
constexpr int few_smem() {
  return FCfg<HD, WIDE>::kMiscOff + (int)sizeof(FMisc) + 1024;
}
static_assert(few_smem<128, true>() <= 227 * 1024, "shared memory");

struct FewArgs {
  ChunkArgs c;
  const void* q;
  long long q_stride;
  int q_bf16;
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two codes (the lower or upper half of a word) to two halves.
template <int CODE, bool UPPER>
__device__ __forceinline__ uint32_t two_halves(uint32_t w) {
  uint32_t h;
  if constexpr (CODE == DLS_E4M3) {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(UPPER ? w >> 16 : w)));
  } else {
    const uint32_t x = __byte_perm(w ^ 0x80808080u, 0x64646464u, UPPER ? 0x4342 : 0x4140), bias = 0x64806480u;  // see codes_to_half
    const __half2 p = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&bias));
    h = *reinterpret_cast<const uint32_t*>(&p);
  }
  return h;
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}

__device__ __forceinline__ bool all_warps(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)ok), "n"(FWARPS * 32)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void meet() { named_bar(1, FWARPS * 32); }

// A lane's dimensions of one row of q as halves: words 2 s and 2 s + 1 belong
// to k-step s.  A bf16 row is multiplied by a power of two that makes it
// halves (see the converting warps of chunk_attn.cuh); cq takes it back.
template <int HD>
__device__ __forceinline__ void load_q(const FewArgs& a, bool live, size_t at, uint32_t (&w)[HD / 8], float& cq) {
  const uint16_t* const row = static_cast<const uint16_t*>(a.q) + at;
  const int c = threadIdx.x & 3;
  if constexpr (HD == 64 || HD == 128) {
    const uint4* p = reinterpret_cast<const uint4*>(row + (HD / 4) * c);
#pragma unroll
    for (int i = 0; i < HD / 32; ++i) {
      const uint4 x = live ? p[i] : make_uint4(0, 0, 0, 0);
      w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int s = 0; s < HD / 16; ++s) {
      const uint2 x = live ? *reinterpret_cast<const uint2*>(row + 16 * s + 4 * c) : make_uint2(0, 0);
      w[2 * s] = x.x, w[2 * s + 1] = x.y;
    }
  }
  cq = 1.f;
  if (a.q_bf16) {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < HD / 8; ++i) most = max(most, max(w[i] << 16 & 0x7fff0000u, w[i] & 0x7fff0000u));
    most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
    most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
    const int e = most >= 0x7f800000u || !most ? 0 : min(14 - ((int)(most >> 23) - 127), 100);
    const float f = __uint_as_float((unsigned)(e + 127) << 23);
    cq = __uint_as_float((unsigned)(127 - e) << 23);
#pragma unroll
    for (int i = 0; i < HD / 8; ++i) w[i] = Kind<__half>::pack(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xffff0000u) * f);
  }
}

template <int HD, int CODE, bool WIDE>
__global__ void __launch_bounds__(FTHREADS, 1) few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                                                          const __grid_constant__ FewArgs fa) {
  using C = FCfg<HD, WIDE>;
  constexpr int NST = C::NST, HDP = HD <= 64 ? 64 : 128;  // HDP: as the workspace is laid out
  const ChunkArgs& a = fa.c;
  extern __shared__ __align__(1024) uint8_t fsm[];
  const uint32_t raw = smem_u32(fsm), pad = (1024u - (raw & 1023u)) & 1023u, base = raw + pad;
  FMisc& sh = *reinterpret_cast<FMisc*>(fsm + pad + C::kMiscOff);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int* const ab = &sh.abort;

  if (warp == 0 && lane < NST) {
    mbar_init(smem_u32(&sh.full[lane]), 1 + 2 * FWARPS);  // the copies' bytes, the scales
    mbar_init(smem_u32(&sh.empty[lane]), FWARPS);
  }
  if (warp == FWARPS && lane < QDEPTH) {
    mbar_init(smem_u32(&sh.pq_full[lane]), 1);
    mbar_init(smem_u32(&sh.pq_empty[lane]), FWARPS + 1);
  }
  if (tid == FTHREADS - 1) {
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    sh.abort = 0;
  }
  mbar_fence_init();
  if (!a.small_plan) {
    plan<FTHREADS, kFewCost, kFewSteps>(a, reinterpret_cast<int4*>(fsm + pad), sh);
    fence_async_smem();  // its scratch is overwritten by copies from here on
  }
  __syncthreads();

  if (warp == FWARPS) {
    // ---------------- the list of pieces, and their copies
    Cursor at;
    if (a.small_plan) {
      plan_warp<kFewCost, kFewSteps>(a, lane, at.pos, at.end, at.per, at.b, at.t, at.off, at.kvh, at.s);
    } else {
      at.pos = sh.range0, at.end = sh.range1, at.per = sh.per;
      at.b = sh.b0, at.t = sh.t0, at.off = sh.off0, at.kvh = sh.kvh0;
      at.s.start = sh.start0, at.s.ql = sh.ql0, at.s.kl = sh.kl0;
    }
    const int pr = min(1 << a.page_shift, BK), npc = BK / pr;  // keys of a copy, copies of a K or V tile
    bool ok = true;
    int u = 0;
    for (int k = 0; ok; ++k) {
      const Piece p = next_piece<kFewCost>(a, at);
      if (k >= QDEPTH && !(ok = __all_sync(0xffffffffu, cwait(smem_u32(&sh.pq_empty[k % QDEPTH]), ((k / QDEPTH) - 1) & 1, ab)))) break;
      if (lane == 0) {
        sh.pq[k % QDEPTH] = p;
        mbar_arrive(smem_u32(&sh.pq_full[k % QDEPTH]));
      }
      __syncwarp();
      if (p.mode == END) break;
      const int32_t* table = a.page_table + (size_t)p.b * a.max_pages;
      int entries_at = -(1 << 30), entry = -1;
#pragma unroll 1
      for (int j = p.ja; j < p.jb; ++j, ++u) {
        const int first = (j * BK) >> a.page_shift, last = ((j + 1) * BK - 1) >> a.page_shift;
        if (last >= entries_at + 32) {  // the table's entries, 32 at a time
          entries_at = first;
          const int e = entries_at + lane;
          entry = -1;
          if ((long long)e << a.page_shift < p.kl && (long long)(e + 1) << a.page_shift > p.lo) entry = table[e];
        }
        const int s = u % NST;
        if (u >= NST && !(ok = __all_sync(0xffffffffu, cwait(smem_u32(&sh.empty[s]), ((u / NST) - 1) & 1, ab)))) break;
        const uint32_t bar = smem_u32(&sh.full[s]), dst = base + s * C::kStage;
        if (lane == 0) mbar_expect_tx(bar, C::kStage);
        __syncwarp();
        {
          const int x = lane >> 1, v = lane & 1, key = j * BK + x * pr;
          const int page = __shfl_sync(0xffffffffu, entry, ((key >> a.page_shift) - entries_at) & 31);
          if (x < npc) {
            int y = a.pool_rows;  // past the end of the pool: the copy fills zeros
            if (key < p.kl && key + pr > p.lo) {
              if (page >= 0 && page < a.n_pages)
                y = ((page * a.n_kv + p.kvh) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
              else if (a.status)
                atomicOr(a.status, kBadPage);
            }
            tma_load_2d(dst + v * C::kPart + x * pr * HD, v ? &tm_v : &tm_k, 0, y, bar);
          }
        }
      }
    }
    // no copy may be in flight when the CTA ends
    __syncwarp();
    for (int x = u > NST ? u - NST : 0; x < u; ++x) cwait(smem_u32(&sh.full[x % NST]), (x / NST) & 1, ab, false);
    if (!ok && a.status && lane == 0) atomicOr(a.status, kTimeout);
    return;
  }
  if (warp == FWARPS + 1) {
    // ---------------- both scales of each warp's keys (no page: 0).  A warp of its own: with the copies' they took
    // 1250 cycles a key tile, which bounded narrow heads
    bool ok = true;
    int u = 0;
    const int w = lane & 7, v = lane >> 3 & 1;
    for (int k = 0; ok; ++k) {
      if (!(ok = __all_sync(0xffffffffu, cwait(smem_u32(&sh.pq_full[k % QDEPTH]), (k / QDEPTH) & 1, ab)))) break;
      const Piece p = sh.pq[k % QDEPTH];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.pq_empty[k % QDEPTH]));
      if (p.mode == END) break;
      const int32_t* table = a.page_table + (size_t)p.b * a.max_pages;
      const int per_page = a.page_shift - a.block_shift;
      int entries_at = -(1 << 30), entry = -1;
#pragma unroll 1
      for (int j = p.ja; j < p.jb; ++j, ++u) {
        const int first = (j * BK) >> a.page_shift, last = ((j + 1) * BK - 1) >> a.page_shift;
        if (last >= entries_at + 32) {
          entries_at = first;
          const int e = entries_at + lane;
          entry = -1;
          if ((long long)e << a.page_shift < p.kl && (long long)(e + 1) << a.page_shift > p.lo) entry = table[e];
        }
        const int s = u % NST, key = j * BK + w * FK;
        const int page = __shfl_sync(0xffffffffu, entry, ((key >> a.page_shift) - entries_at) & 31);
        const float* from = v ? a.v_scales : a.k_scales;
        int bytes = 0;
        if (key < p.kl && key + FK > p.lo && page >= 0 && page < a.n_pages) {
          from += ((size_t)(page * a.n_kv + p.kvh) << per_page) + ((key & ((1 << a.page_shift) - 1)) >> a.block_shift);
          bytes = 4;
        }
        if (u >= NST && !(ok = __all_sync(0xffffffffu, cwait(smem_u32(&sh.empty[s]), ((u / NST) - 1) & 1, ab)))) break;
        if (lane < 2 * FWARPS) {
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(&sh.scale[s][v][w])), "l"(from), "r"(bytes) : "memory");
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sh.full[s])) : "memory");
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // none in flight when the CTA ends
    return;
  }

  // ---------------- the warps' own keys
  const int r = lane >> 2, c = lane & 3, G = a.group;
  float* const merge = reinterpret_cast<float*>(fsm + pad + C::kMergeOff);
  int u0 = 0;
  bool ok = true;
  for (int k = 0;; ++k) {
    ok = ok && cwait(smem_u32(&sh.pq_full[k % QDEPTH]), (k / QDEPTH) & 1, ab);
    if (!(ok = all_warps(ok))) break;  // (and everyone has read the last piece's sums)
    const Piece p = sh.pq[k % QDEPTH];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.pq_empty[k % QDEPTH]));
    if (p.mode == END) break;
    const int n_rows = p.n * G;
    // the lane's rows: r, and r + 8 of a wide tile
    Row row[2];
    uint32_t qa[WIDE ? 2 : 1][HD / 8];
    float cq[2] = {1.f, 1.f}, R[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int h = 0; h < (WIDE ? 2 : 1); ++h) {
      const int x = r + 8 * h, tok = token_of(a, x), pos = p.pos0 + tok;
      row[h].ok = x < n_rows;
      row[h].hi = !row[h].ok ? 0x7fffffff : a.causal ? min(max(pos + 1, 0), p.kl) : p.kl;
      row[h].lo = row[h].ok && a.window && pos >= a.window ? pos - a.window + 1 : 0;
      const size_t qrow = row[h].ok ? (size_t)(p.row0 + tok) * fa.q_stride + (size_t)(p.kvh * G + x - tok * G) * HD : 0;
      load_q<HD>(fa, row[h].ok, qrow, qa[h], cq[h]);
    }
    float o[HD / 8][4];
#pragma unroll
    for (int i = 0; i < HD / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    const int n = p.jb - p.ja;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int u = u0 + i, s = u % NST, key0 = (p.ja + i) * BK + warp * FK;
      ok = __all_sync(0xffffffffu, ok && cwait(smem_u32(&sh.full[s]), (u / NST) & 1, ab));
      if (!ok) break;
      if (key0 < p.kl && key0 + FK > p.lo) {
        const uint32_t kt = base + s * C::kStage + warp * FK * HD, vt = kt + C::kPart;
        const bool ragged = __any_sync(0xffffffffu, (row[0].ok && (key0 < row[0].lo || key0 + FK > row[0].hi)) ||
                                                        (WIDE && row[1].ok && (key0 < row[1].lo || key0 + FK > row[1].hi)));
        // ---- S = Q K^T for two groups of eight keys
        float sc[2][4] = {};
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int key = 8 * t + r;
          auto product = [&](int st, uint32_t x) {
            const uint32_t qf[4] = {qa[0][2 * st], WIDE ? qa[WIDE][2 * st] : 0u, qa[0][2 * st + 1], WIDE ? qa[WIDE][2 * st + 1] : 0u};
            mma16816(sc[t], qf, two_halves<CODE, false>(x), two_halves<CODE, true>(x));
          };
          if constexpr (C::kWide16) {
#pragma unroll
            for (int h = 0; h < HD / 64; ++h) {
              const int chunk = HD == 128 ? (2 * c + h) ^ (key & 7) : c ^ (key >> 1 & 3);
              const uint4 w = lds128(kt + key * HD + chunk * 16);
              const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) product(4 * h + e, x[e]);
            }
          } else {
            uint32_t x[HD / 16];
#pragma unroll
            for (int st = 0; st < HD / 16; ++st) x[st] = lds32(kt + key * HD + 16 * st + 4 * c);
#pragma unroll
            for (int st = 0; st < HD / 16; ++st) product(st, x[st]);
          }
        }
        // V's codes: keys 2c, 2c + 1, 2c + 8, 2c + 9
        constexpr int VW = (HD + 16) / 32;  // words of a lane's dimensions, the last one a half where HD / 16 is odd
        uint32_t v[4][VW];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = 2 * c + (e & 1) + 8 * (e >> 1);
          if constexpr (HD == 128) {
            const uint4 w = lds128(vt + key * HD + ((r ^ (key & 7)) << 4));
            v[e][0] = w.x, v[e][1] = w.y, v[e][2] = w.z, v[e][3] = w.w;
          } else if constexpr (HD != 64) {
#pragma unroll
            for (int x = 0; x < HD / 32; ++x) v[e][x] = lds32(vt + key * HD + 32 * x + 4 * r);
            if constexpr (HD % 32 != 0) v[e][VW - 1] = lds16(vt + key * HD + HD - 16 + 2 * r);
          } else {
            asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                         : "=r"(v[e][0]), "=r"(v[e][1])
                         : "r"(vt + key * HD + (((r >> 1) ^ (key >> 1 & 3)) << 4) + (r & 1) * 8));
          }
        }
        const float sk = fminf(fmaxf(sh.scale[s][0][warp], 0x1p-64f), 0x1p64f), sv = fminf(fmaxf(sh.scale[s][1][warp], 0x1p-64f), 0x1p64f);
        const float lsv = log2f(sv), isv = 1.f / sv;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.empty[s]));
        if (__builtin_expect(ragged, 0)) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = key0 + 8 * t + 2 * c + (e & 1);
              const Row& w = row[WIDE ? e >> 1 : 0];
              if (key < w.lo || key >= w.hi) sc[t][e] = -INFINITY;
            }
          // rows of V that no query may see can hold anything
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0 + 2 * c + (e & 1) + 8 * (e >> 1);
            if (key >= p.kl || key < p.lo)
#pragma unroll
              for (int x = 0; x < VW; ++x) v[e][x] = 0;
          }
        }
        // ---- weights: as softmax_codes
        uint32_t pa[4] = {0, 0, 0, 0};
        float ck[2], m[2];
        bool grow = false;
#pragma unroll
        for (int h = 0; h < (WIDE ? 2 : 1); ++h) {
          ck[h] = fmaxf(fmaxf(a.c * sk, 0x1p-126f) * cq[h], 0x1p-126f);
          m[h] = fmaf(fmaxf(fmaxf(sc[0][2 * h], sc[0][2 * h + 1]), fmaxf(sc[1][2 * h], sc[1][2 * h + 1])), ck[h], lsv);
          grow |= row[h].ok && m[h] > R[h] + kGrow;
        }
        if (__builtin_expect(__any_sync(0xffffffffu, grow), 0)) {
#pragma unroll
          for (int h = 0; h < (WIDE ? 2 : 1); ++h) {
            float x = fmaxf(m[h], __shfl_xor_sync(0xffffffffu, m[h], 1));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
            if (x > R[h] + kGrow) {
              const float f = ex2(R[h] - x);
              R[h] = x;
              l[h] *= f;
#pragma unroll
              for (int e = 0; e < HD / 8; ++e) o[e][2 * h] *= f, o[e][2 * h + 1] *= f;
            }
          }
        }
#pragma unroll
        for (int h = 0; h < (WIDE ? 2 : 1); ++h) {
          const float nr = kShift + lsv - (R[h] == -INFINITY ? 0.f : R[h]);
          const float w0 = ex2(fmaf(sc[0][2 * h], ck[h], nr)), w1 = ex2(fmaf(sc[0][2 * h + 1], ck[h], nr));
          const float w2 = ex2(fmaf(sc[1][2 * h], ck[h], nr)), w3 = ex2(fmaf(sc[1][2 * h + 1], ck[h], nr));
          l[h] = fmaf((w0 + w1) + (w2 + w3), isv, l[h]);
          pa[h] = Kind<__half>::pack(w0, w1);
          pa[2 + h] = Kind<__half>::pack(w2, w3);
        }
        // ---- O += P V: eight dimensions a product
#pragma unroll
        for (int x = 0; x < VW; ++x) {
          const uint32_t lo01 = __byte_perm(v[0][x], v[1][x], 0x5140), lo23 = __byte_perm(v[2][x], v[3][x], 0x5140);
          const uint32_t hi01 = __byte_perm(v[0][x], v[1][x], 0x7362), hi23 = __byte_perm(v[2][x], v[3][x], 0x7362);
          mma16816(o[4 * x], pa, two_halves<CODE, false>(lo01), two_halves<CODE, false>(lo23));
          mma16816(o[4 * x + 1], pa, two_halves<CODE, true>(lo01), two_halves<CODE, true>(lo23));
          if (4 * x + 2 < HD / 8) {
            mma16816(o[(4 * x + 2) % (HD / 8)], pa, two_halves<CODE, false>(hi01), two_halves<CODE, false>(hi23));
            mma16816(o[(4 * x + 3) % (HD / 8)], pa, two_halves<CODE, true>(hi01), two_halves<CODE, true>(hi23));
          }
        }
      } else {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.empty[s]));
      }
    }
    u0 += n;

    // ---- the warps' shares meet.  Where codes are read 16 bytes at a time a
    // lane's HD / 4 dimensions of a row lie in 16-byte pieces, moved by its number
    // against bank conflicts; else rows are four floats longer.
    constexpr int kPieces = HD / 16, kRowF = C::kRowF;  // 16-byte pieces of a lane, floats of a row
#pragma unroll
    for (int h = 0; h < (WIDE ? 2 : 1); ++h) {
      float s = l[h];
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      if (c == 0) sh.R[warp][r + 8 * h] = R[h], sh.l[warp][r + 8 * h] = s;
      float* const to = merge + (size_t)(warp * C::kRows + r + 8 * h) * kRowF;
#pragma unroll
      for (int x = 0; x < kPieces; ++x) {
        if constexpr (C::kWide16) {
          // dimensions 4 x .. of the lane's: o[j][.] holds j and HD / 8 + j
          const int up = x >= kPieces / 2, j = 4 * x - up * (HD / 8);
          *reinterpret_cast<float4*>(to + c * (HD / 4) + ((x ^ (lane & (kPieces - 1))) << 2)) =
              make_float4(o[j][2 * h + up], o[j + 1][2 * h + up], o[j + 2][2 * h + up], o[j + 3][2 * h + up]);
        } else if (x < HD / 32 * 2) {
          // eight dimensions from 32 i + 8 c on: o[4 i + e][.] holds e and 4 + e of them
          const int up = x & 1, j = 4 * (x >> 1);
          *reinterpret_cast<float4*>(to + 32 * (x >> 1) + 8 * c + 4 * up) =
              make_float4(o[j][2 * h + up], o[j + 1][2 * h + up], o[(j + 2) % (HD / 8)][2 * h + up], o[(j + 3) % (HD / 8)][2 * h + up]);
        } else {
          // four of the last sixteen: o[j][.] holds 0 and 2, o[j + 1][.] 1 and 3
          const int j = HD / 8 - 2;
          *reinterpret_cast<float4*>(to + HD - 16 + 4 * c) = make_float4(o[j][2 * h], o[j + 1][2 * h], o[j][2 * h + 1], o[j + 1][2 * h + 1]);
        }
      }
    }
    meet();
    constexpr int C4 = HD / 4;  // 16-byte pieces of a row
    float* const part = p.np > 1 ? partial_at<HDP>(a, blockIdx.x, p.idx == 0, 0) : nullptr;
    auto put = [&](int x, int d, const float4& y) {
      const int tok = token_of(a, x), head = p.kvh * G + x - tok * G;
      const size_t at = (size_t)(p.row0 + tok) * a.o_stride + (size_t)head * HD + 4 * d;
      uint2 w;
      if (fa.q_bf16) w = make_uint2(Kind<__nv_bfloat16>::pack(y.x, y.y), Kind<__nv_bfloat16>::pack(y.z, y.w));
      else w = make_uint2(Kind<__half>::pack(y.x, y.y), Kind<__half>::pack(y.z, y.w));
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + at) = w;
    };
    auto put_lse = [&](int x, float M, float L) {
      const int tok = token_of(a, x);
      a.lse[(size_t)(p.row0 + tok) * (a.n_kv * G) + p.kvh * G + x - tok * G] = lse_of(M, L);
    };
    for (int it = tid; it < n_rows * C4; it += FWARPS * 32) {
      const int x = it / C4, d = it - x * C4;
      int from = 4 * d;
      if constexpr (C::kWide16) {
        const int q = d / kPieces, piece = d - q * kPieces;
        from = q * (HD / 4) + ((piece ^ ((4 * (x & 7) + q) & (kPieces - 1))) << 2);
      }
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int w = 0; w < FWARPS; ++w) M = fmaxf(M, sh.R[w][x]);
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < FWARPS; ++w) {
        const float f = weight(sh.R[w][x], M);
        const float4 z = *reinterpret_cast<const float4*>(merge + (size_t)(w * C::kRows + x) * kRowF + from);
        L = fmaf(f, sh.l[w][x], L);
        y.x = fmaf(f, z.x, y.x), y.y = fmaf(f, z.y, y.y), y.z = fmaf(f, z.z, y.z), y.w = fmaf(f, z.w, y.w);
      }
      if (part) {
        __stcg(reinterpret_cast<float4*>(part + 256) + it, y);
        if (d == 0) __stcg(part + x, M), __stcg(part + 128 + x, L);
      } else {
        const float inv = L > 0.f ? 1.f / L : 0.f;
        put(x, d, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
        if (d == 0 && a.lse) put_lse(x, M, L);
      }
    }
    if (part) {
      // the last piece of the tile to arrive joins them all
      meet();
      if (tid == 0) {
        int* cnt = a.counters + p.c0 * 2;
        int seen;
        asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(seen) : "l"(cnt) : "memory");
        const bool last = seen == p.np - 1;
        if (last) *cnt = 0;  // ready for the next call
        sh.last = last;
      }
      meet();
      if (sh.last) {
        float *sw = merge, *sl = merge + MAXC * 16;
        for (int x = tid; x < p.np * n_rows; x += FWARPS * 32) {
          const int i = x / n_rows;
          const float* from = partial_at<HDP>(a, p.c0 + i, i == 0, 0) + (x - i * n_rows);
          sw[x] = __ldcg(from);
          sl[x] = __ldcg(from + 128);
        }
        meet();
        for (int it = tid; it < n_rows * C4; it += FWARPS * 32) {
          const int x = it / C4, d = it - x * C4;
          float M = -INFINITY, L = 0.f;
#pragma unroll 4
          for (int i = 0; i < p.np; ++i) M = fmaxf(M, sw[i * n_rows + x]);
          float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
          for (int i = 0; i < p.np; ++i) {
            const float4 z = __ldcg(reinterpret_cast<const float4*>(partial_at<HDP>(a, p.c0 + i, i == 0, 0) + 256) + it);
            const float f = weight(sw[i * n_rows + x], M);
            L = fmaf(f, sl[i * n_rows + x], L);
            y.x = fmaf(f, z.x, y.x), y.y = fmaf(f, z.y, y.y), y.z = fmaf(f, z.z, y.z), y.w = fmaf(f, z.w, y.w);
          }
          const float inv = L > 0.f ? 1.f / L : 0.f;
          put(x, d, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
          if (d == 0 && a.lse) put_lse(x, M, L);
        }
      }
    }
  }
  if (!ok && a.status && lane == 0) atomicOr(a.status, kTimeout);
}

using FewFn = void (*)(const CUtensorMap, const CUtensorMap, const FewArgs);

struct Few {
  FewFn f;
  int smem;
};
template <int HD, int CODE>
Few few_of(bool wide) {
  if (wide) return {few_kernel<HD, CODE, true>, few_smem<HD, true>()};
  return {few_kernel<HD, CODE, false>, few_smem<HD, false>()};
}
template <int CODE>
Few few_of(int hd, bool wide) {
  switch (hd) {
    case 16: return few_of<16, CODE>(wide);
    case 32: return few_of<32, CODE>(wide);
    case 48: return few_of<48, CODE>(wide);
    case 64: return few_of<64, CODE>(wide);
    case 80: return few_of<80, CODE>(wide);
    case 96: return few_of<96, CODE>(wide);
    case 112: return few_of<112, CODE>(wide);
    default: return few_of<128, CODE>(wide);
  }
}
Few few_of(int hd, int code, bool wide) { return code == DLS_E4M3 ? few_of<DLS_E4M3>(hd, wide) : few_of<DLS_I8>(hd, wide); }

}  // namespace

cudaError_t few_codes_setup() {
  for (int i = 0; i < 32; ++i) {
    const Few k = few_of(16 + (i >> 2) * 16, i & 2 ? DLS_I8 : DLS_E4M3, i & 1);
    const cudaError_t e = cudaFuncSetAttribute(k.f, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_few_codes(const CUtensorMap& tk, const CUtensorMap& tv, const ChunkArgs& c, const void* q, long long q_stride, bool half,
                             int code, int ctas, cudaStream_t s) {
  FewArgs a{c, q, q_stride, !half};
  const bool wide = a.c.tile_tokens * a.c.group > 8;
  const Few k = few_of(a.c.head_dim, code, wide);
  k.f<<<ctas, FTHREADS, k.smem, s>>>(tk, tv, a);
  return cudaGetLastError();
}

}  // namespace dls
