// Attention of ragged chunks of new tokens over the paged cache, on the
// 5th-generation tensor cores.
//
// Mathematics: for a query row with raw scores s_k = q . K[k] over its keys,
// c = scale * log2(e) and any reference R, with p_k = 2^(c s_k - R):
//   o = sum_k p_k V[k] / sum_k p_k,   lse = R ln 2 + ln sum_k p_k
// One pass over the keys in tiles of 128 keeps (R, l = sum p, O = sum p V);
// R follows the running maximum, but only when it falls more than 2^8
// behind, because moving R costs a pass over O (O *= 2^(R - R'), l likewise).
// Ranges of keys done by different CTAs are joined by the same formula.
//
// A tile of work is a KV head and up to 2 * (128 / G) consecutive new tokens
// of a sequence: two 128-row MMA operands ("slots"), row = token * G + query
// head of the group, so one K/V tile from the pages serves 256 rows:
//   S = Q K^T   tcgen05.mma M = 128, N = 128 keys, K = head_dim (fp32 in TMEM)
//   P = 2^(...) softmax warps, thread = row, written over S as 16-bit TMEM operand
//   O += P V    M = 128, N = head_dim, K = 128 keys (A from TMEM, V MN-major)
// While one slot's softmax runs, the tensor core works for the other.  Tiles
// with rows for one slot only (few new tokens: single tokens, verify passes,
// the ends of chunks) give both slots the same Q and every second key tile
// ("split"), joined in the epilogue.
//
// Work is divided by key tiles, not by sequences: the key tiles of all
// (KV head, sequence, token tile) in a row, each tile of work led by what it
// costs besides (kTileCost), are cut into one equal range per CTA, whatever
// the mix of prompts and single tokens; a tile cut by a range border leaves
// partial (R, l, O) in the workspace and the last CTA to arrive joins them in
// range order.  Each CTA finds its range itself from the device-side lengths,
// so a call is one launch and a captured graph follows the lengths.
//
// What bounds it, measured on one GB300 (8B and 70B head counts, head_dim
// 128, bf16, GPU time):
//  - prompts: 8192 tokens of 32 heads 395 us (1394 TFLOP/s), 2048 tokens of
//    64 heads over 32768 1480 us (1440 TFLOP/s; cuBLAS reaches 1919 in a burst,
//    1698 under the power cap).  The MMA warp: the tensor pipe takes about two
//    products ahead, and its barrier waits (about 100 cycles each) show
//    between them; QK^T also reads 128 bytes a cycle of shared memory, all
//    there is.  Slower in this place: a warp per slot (the slots fall into
//    step and their softmaxes collide: 1540 us on the second case), asking
//    barriers between the halves of a product (1530), a third score buffer
//    for narrow heads, softmax in rolled chunks (1573).  Moving R at every new
//    maximum (kGrow = 0): 475 and 1600 us.
//  - single tokens: 64 of 64 heads over up to 8192 cached (5301 on average,
//    1.39 GB) 222 us, 6.3 TB/s (a plain copy moves 6.8): the cache is read once.
//  - small calls: latencies in a row (lengths, page table, first tiles,
//    epilogue, arrival, join): one token over 2048 cached 15.7 us (16.9 with
//    the cache in HBM).  The split-K kernel of dls_attention_decode, which
//    takes one fp32 row a sequence, has a shorter chain: 10.6 (11.8) there.
//
// Over pages of 8-bit codes (CODE) eight more warps turn codes into halves in
// shared memory, and everything after is the same but for the scales, which the
// softmax takes in (softmax_codes).  The last 2048 tokens of 16384, 32 heads,
// bf16, e4m3: 472 us (1.09 PFLOP/s).  What bounds it there: a key tile is written by the
// copy, read, written as halves and read by the products, 2560 cycles of shared
// memory's rate beside 2048 of the tensor core's, and the conversion gets what
// the products leave.
//
// Warps: 0 copies (TMA), 1 MMA, 2 the CTA's piece list, 4-7 / 8-11 softmax of
// slot 0 / 1, 12-19 conversion.  Every wait is bounded (2 s) and sets an abort flag.
#pragma once
#include <cuda_bf16.h>
#include <math.h>

#include <type_traits>

#include "../../include/dls.h"
#include "kernels.h"
#include "tc.cuh"

namespace dls {

struct ChunkArgs {
  void* o;
  float* lse;
  const int32_t *page_table, *cu_q, *kv_len;
  int32_t* status;
  int* counters;
  float* partials;
  long long o_stride;
  int n_tokens, n_seqs, n_kv, group, head_dim;
  int page_shift, n_pages, max_pages, pool_rows;
  int causal, window;
  int tpq;      // tokens of a slot: 128 / group
  int tile_tokens;  // tokens of a tile of work: both slots', or a few (few_attn8.cu)
  unsigned inv_group;  // ceil(2^16 / group): r / group = r * inv_group >> 16 for r < 128
  float c;      // scale * log2(e)
  int small_plan;  // few sequences and tiles: one warp plans
  const float *k_scales, *v_scales;  // of codes: [n_pages][n_kv][page / block]
  int block_shift;
};

namespace {

constexpr int BK = 128;          // keys per tile
constexpr int MAXC = 152;        // CTAs at most (one per SM)
// Threads of a CTA: copies, products and the list (4 warps), softmax (8) and,
// over codes, what makes them operands (8).
template <int CODE>
constexpr int kThreads = CODE ? 640 : 384;
constexpr int kMostWarps = kThreads<DLS_E4M3> / 32;
constexpr int QDEPTH = 4;        // pieces the list runs ahead
// Units of a range at least: a key tile per slot of a split tile.  One token
// over 2048: 15.3 us with two, 15.7 with one (on twice the SMs, but twice the
// partials to join), 16.3 with four; the larger calls do not notice.
constexpr int kMinSteps = 2;
// What a tile of work costs beyond its key tiles (Q, first product, epilogue,
// join), in key tiles: one value for both head widths.  0, 2, 3 and 5 of them:
// prompt of 8192 458, 399, 398, 406 us; of 2048 80, 61, 62, 64; eight verify
// passes 37.8, 34.3, 33.3, 35.3; mixed batch of narrow heads 96, 96, 96, 97.
constexpr int kTileCost = 3;
constexpr float kGrow = 8.f;     // log2 the maximum may exceed the reference by
constexpr float kShift = 7.f;    // weights are kept as 2^(c s - R + 7): at most 2^15 in fp16, with 7 more binades below
constexpr uint64_t kWaitNsC = 2000000000ull;
constexpr int kPCol = 64;         // the weights' columns in a slot's S (packed: 64 of them)
constexpr int kJoinCap = 1024;     // (piece, row) statistics of a slot that a join keeps in shared memory
constexpr int kCounterBytes = 4096;  // int [MAXC][2], at the start of the workspace

enum Mode { PAIR = 0, SPLIT = 1, END = 2 };

// Token of a slot's row r (0..127).
__device__ __forceinline__ int token_of(const ChunkArgs& a, int r) { return (int)((unsigned)r * a.inv_group >> 16); }

// What a CTA does at a time: key tiles [ja, jb) of one tile of work.
struct Piece {
  int mode, b, kvh;
  int row0, n;        // first row (token) in q / o, tokens
  int pos0, kl, lo;   // position of the first token, cached keys, first key any row may see
  int ja, jb;
  int np, idx, c0;    // pieces of the tile, which one this is, CTA of its first one
};

// CODE: 0 for 16-bit pages, else the codes' type (dls_dtype).
template <int HDP, int CODE>
struct CCfg {
  static constexpr int KA = HDP / 64;        // 64-wide swizzle atoms along the head dimension
  static constexpr int kQ = 128 * HDP * 2;   // one slot's Q
  static constexpr int kKV = BK * HDP * 2;   // one K or V tile
  // Stages of 32 KB: a K or a V tile, or both of a narrow head's key tile.
  // There one barrier serves both: apart, the MMA warp's waits (about 100
  // cycles each) took as long as its products.  13 ragged chunks of 32 heads of
  // 64: 98 us, 100 with K and V in stages of their own.
  static constexpr bool kTogether = HDP == 64;
  static constexpr int kUses = kTogether ? 1 : 2;  // ring uses of a key tile
  static constexpr int kStage = kTogether ? 2 * kKV : kKV;
  // Codes arrive in a ring of their own, half the size a use.  Three stages of
  // operands: with two (and five of wide heads' codes) the next K waits for the
  // last product with this one, 609 us against 521 (2048 tokens over 16384, 32 heads of 128).
  static constexpr int NST = !CODE ? 4 : 3;
  static constexpr int kRaw = CODE ? kStage / 2 : 0;
  static constexpr int NRAW = kTogether ? 5 : 3;
  static constexpr int kKVOff = 2 * kQ;
  static constexpr int kXOff = kKVOff + NST * kStage;  // 8 KB a slot: its output rows on their way out, or statistics being joined
  static constexpr int kRawOff = kXOff + 2 * 8192;
  static constexpr int kMiscOff = kRawOff + (CODE ? NRAW * kRaw : 0);
};
constexpr int kScaleRing = 4;  // key tiles whose scales are held: those whose softmax may be under way (see the converting warps)

struct CMisc {
  uint64_t full[4], empty[4], s_full[2], p_full[2][2], o_full[2], o_free[2], q_full, q_empty, x_full, pq_full[QDEPTH], pq_empty[QDEPTH];
  Piece pq[QDEPTH];
  float xm[128], xl[128];        // slot 1's statistics for slot 0 (split)
  long long scan[kMostWarps];
  long long range0, range1, per;
  int b0, t0, off0, kvh0;
  int start0, ql0, kl0;          // sequence b0
  uint32_t tmem;
  int abort, last[2];
};
struct CodeMisc : CMisc {
  uint64_t raw_full[5], raw_empty[5], q_ready;
  int8_t q_exp[2][2][128];                        // powers of two that a piece's rows were multiplied by (bf16 q), pieces in turn
  float raw_scale[5][2][8];                       // of a raw stage with keys: of K and of V, for 16 keys each
  __align__(16) float scale[kScaleRing][3][8];     // c * K's, log2 of V's, 1 / V's
};
template <int CODE>
struct MiscOf {
  using type = CodeMisc;
};
template <>
struct MiscOf<0> {
  using type = CMisc;
};

// 16-bit pages: with room to begin at a multiple of 1024.  (Codes take all there
// is; their kernel's shared memory is declared aligned and looked at.)
template <int HDP, int CODE>
constexpr int chunk_smem() {
  return CCfg<HDP, CODE>::kMiscOff + (int)sizeof(typename MiscOf<CODE>::type) + (CODE ? 0 : 1024);
}
static_assert(2 * kJoinCap * 4 <= 8192, "join area");
static_assert(chunk_smem<128, 0>() <= 227 * 1024 && chunk_smem<64, 0>() <= 227 * 1024, "shared memory");
static_assert(chunk_smem<128, DLS_I8>() <= 227 * 1024 && chunk_smem<64, DLS_I8>() <= 227 * 1024, "shared memory");
// a CTA allocates all of tensor memory: a second one must not fit on the SM
static_assert(2 * chunk_smem<64, 0>() > 227 * 1024 && 2 * chunk_smem<64, DLS_I8>() > 227 * 1024, "one CTA per SM");
// the lengths being planned over lie in the Q and K/V area before its first use
static_assert(DLS_MAX_CHUNK_SEQS * 16 <= CCfg<64, 0>::kXOff, "plan scratch");

__device__ __forceinline__ bool cwait(uint32_t bar, uint32_t parity, int* abort_flag, bool heed_abort = true) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i) {
    if (i & 63) continue;
    if (heed_abort && *(volatile int*)abort_flag) return false;
    const uint64_t t = global_ns();
    if (!t0) t0 = t;
    if (t - t0 > kWaitNsC) {
      *(volatile int*)abort_flag = 1;
      return false;
    }
  }
  return true;
}

// A value that is the same in every lane, as one the compiler knows to be.
__device__ __forceinline__ int uniform(int x) { return (int)__reduce_max_sync(0xffffffffu, (unsigned)x); }

// The four warps of a softmax group meet; with a vote, all learn whether all
// are well.  A plain hardware barrier: a warp whose wait ran out goes on to
// the end of its piece without waiting, so that nobody is left here, and the
// group stops together at the vote that begins the next piece.
__device__ __forceinline__ void wg_sync(int slot) { named_bar(1 + slot, 128); }
__device__ __forceinline__ bool wg_all(int slot, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)ok), "r"(1 + slot)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
struct Kind;
template <>
struct Kind<__half> {
  static constexpr uint32_t kIdesc = 0;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
  }
};
template <>
struct Kind<__nv_bfloat16> {
  static constexpr uint32_t kIdesc = (1u << 7) | (1u << 10);  // A and B bf16
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
  }
};

// ---- division of the work -----------------------------------------------------------------

struct Seq {
  int start, ql, kl;
  bool bad;
};

// Sequence b's rows and lengths; ql = 0 where they do not fit.
__device__ __forceinline__ Seq seq_get(const ChunkArgs& a, int b) {
  Seq s;
  s.start = a.cu_q[b];
  const int end = a.cu_q[b + 1];
  s.kl = a.kv_len[b];
  s.bad = s.start < 0 || end < s.start || end > a.n_tokens || s.kl < 0 || s.kl > ((long long)a.max_pages << a.page_shift);
  s.ql = s.bad ? 0 : end - s.start;
  return s;
}

struct Tile {
  int mode, n, pos0, lo, j0, keys, units;  // keys: key tiles to do; units: kTileCost and the key tiles (one at least)
};

template <int COST>
__device__ __forceinline__ Tile tile_of(const ChunkArgs& a, int ql, int kl, int t) {
  Tile x;
  const int i0 = t * a.tile_tokens;
  x.n = min(a.tile_tokens, ql - i0);
  x.mode = x.n > a.tpq ? PAIR : SPLIT;
  x.pos0 = kl - ql + i0;
  const int hi = a.causal ? min(max(x.pos0 + x.n, 0), kl) : kl;
  x.lo = a.window && x.pos0 >= a.window ? min(x.pos0 - a.window + 1, hi) : 0;
  x.j0 = x.lo / BK;
  x.keys = hi > x.lo ? (hi + BK - 1) / BK - x.j0 : 0;
  x.units = COST + max(x.keys, 1);
  return x;
}

template <int WARPS>
__device__ __forceinline__ long long block_scan(long long v, long long* sums, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  long long pre = 0, tot = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) pre += sums[w];
    tot += sums[w];
  }
  __syncthreads();
  *total = tot;
  return pre + x - v;
}

// Quotient of non-negative values, out of line (64-bit division is long).
__device__ __noinline__ long long quotient(long long x, long long y) {
  return (x | y) >> 32 ? x / y : (long long)((unsigned)x / (unsigned)y);
}

// The CTA's range of key tiles and where it begins (all threads).  Short
// loops, not unrolled: every CTA runs this once, and what it costs is
// instruction fetches and latencies.
template <int THREADS, int COST, int MIN, typename Misc>
__device__ __noinline__ void plan(const ChunkArgs& a, int4* info, Misc& sh) {
  const int tid = threadIdx.x, tp = a.tile_tokens;
  const int per_s = (a.n_seqs + THREADS - 1) / THREADS;
  const int s0 = min(tid * per_s, a.n_seqs), s1 = min(s0 + per_s, a.n_seqs);
  long long mine = 0, total;
  bool bad = false;
#pragma unroll 1
  for (int b = s0; b < s1; ++b) {
    const Seq s = seq_get(a, b);
    bad |= s.bad;
    info[b] = make_int4((int)mine, s.ql, s.kl, s.start);
    mine += (s.ql + tp - 1) / tp;
  }
  if (bad && blockIdx.x == 0 && a.status) atomicOr(a.status, kBadPos);
  const int before = (int)block_scan<THREADS / 32>(mine, sh.scan, &total);
#pragma unroll 1
  for (int b = s0; b < s1; ++b) info[b].x += before;  // the first tile of the sequence
  __syncthreads();
  const int n_tiles = (int)total;
  const int per_t = (n_tiles + THREADS - 1) / THREADS;
  const int t0 = min(tid * per_t, n_tiles), t1 = min(t0 + per_t, n_tiles);
  int lo = 0, hi = t0 < t1 ? a.n_seqs : 1;
#pragma unroll 1
  while (hi - lo > 1) {  // the last sequence whose first tile is not behind t0
    const int mid = (lo + hi) >> 1;
    if (info[mid].x <= t0) lo = mid;
    else hi = mid;
  }
  // first pass: the steps of tiles t0 .. t1 - 1; second: the tile that holds
  // the range's first step, in the thread whose tiles do
  long long pre = 0, stop = -1, r0 = 0, head = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    long long sum = 0;
    int b = lo;
#pragma unroll 1
    for (int t = t0; t < t1; ++t) {
#pragma unroll 1
      while (b + 1 < a.n_seqs && info[b + 1].x <= t) ++b;
      const int4 f = info[b];
      const int st = tile_of<COST>(a, f.y, f.z, t - f.x).units;
      if (stop >= 0 && sum + st > stop) {
        sh.off0 = (int)(stop - sum);
        sh.b0 = b;
        sh.t0 = t - f.x;
        sh.kvh0 = (int)head;
        sh.start0 = f.w;
        sh.ql0 = f.y;
        sh.kl0 = f.z;
        break;
      }
      sum += st;
    }
    if (pass) break;
    pre = block_scan<THREADS / 32>(sum, sh.scan, &total);
    const long long all = total * a.n_kv, per = max(quotient(all + gridDim.x - 1, gridDim.x), (long long)MIN);
    r0 = min(per * blockIdx.x, all);
    const long long r1 = min(r0 + per, all);
    if (tid == 0) {
      sh.range0 = r0;
      sh.range1 = r1;
      sh.per = per;
    }
    if (r0 >= r1) break;  // (uniform)
    head = quotient(r0, total);
    const long long at = r0 - head * total;
    if (at < pre || at >= pre + sum) break;  // another thread's
    stop = at - pre;
  }
  __syncthreads();
}

// The same by one warp, without a barrier, for few sequences and tiles: the
// other warps are at their posts meanwhile.  A lane takes consecutive
// sequences.  Returns the range; where it begins goes to the last arguments.
template <int COST, int MIN>
__device__ __forceinline__ void plan_warp(const ChunkArgs& a, int lane, long long& r0, long long& r1, long long& per, int& b0, int& t0,
                                          int& off0, int& kvh0, Seq& seq0) {
  const int per_s = (a.n_seqs + 31) / 32, tp = a.tile_tokens;
  const int s0 = min(lane * per_s, a.n_seqs), s1 = min(s0 + per_s, a.n_seqs);
  unsigned pre = 0, total = 0, stop = 0;
  bool seek = false;
  int from = 0;
  b0 = t0 = off0 = kvh0 = 0;
  seq0 = {};
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    unsigned sum = 0;
    bool bad = false, found = false;
#pragma unroll 1
    for (int b = s0; b < s1 && !found; ++b) {
      const Seq s = seq_get(a, b);
      bad |= s.bad;
#pragma unroll 1
      for (int t = 0; t * tp < s.ql; ++t) {
        const unsigned st = tile_of<COST>(a, s.ql, s.kl, t).units;
        if (seek && sum + st > stop) {
          b0 = b, t0 = t, off0 = (int)(stop - sum), seq0 = s;
          found = true;
          break;
        }
        sum += st;
      }
    }
    if (pass) break;
    if (bad && blockIdx.x == 0 && a.status) atomicOr(a.status, kBadPos);
    pre = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) pre += y;
    }
    total = __shfl_sync(0xffffffffu, pre, 31);
    pre -= sum;
    const long long all = (long long)total * a.n_kv;
    per = max(quotient(all + gridDim.x - 1, gridDim.x), (long long)MIN);
    r0 = min(per * blockIdx.x, all);
    r1 = min(r0 + per, all);
    if (r0 >= r1) return;
    kvh0 = (int)quotient(r0, total);
    stop = (unsigned)(r0 - (long long)kvh0 * total);
    seek = stop >= pre && stop - pre < sum;
    stop -= pre;
    from = __ffs(__ballot_sync(0xffffffffu, seek)) - 1;
    if (!seek) break;
  }
  __syncwarp();
  b0 = __shfl_sync(0xffffffffu, b0, from);
  t0 = __shfl_sync(0xffffffffu, t0, from);
  off0 = __shfl_sync(0xffffffffu, off0, from);
  seq0.start = __shfl_sync(0xffffffffu, seq0.start, from);
  seq0.ql = __shfl_sync(0xffffffffu, seq0.ql, from);
  seq0.kl = __shfl_sync(0xffffffffu, seq0.kl, from);
}

// Where a CTA stands in its range.
struct Cursor {
  long long pos, end, per;
  int b, t, off, kvh;
  Seq s;
};
// The next piece of the range (mode END: none), by a whole warp alike.
template <int COST>
__device__ __forceinline__ Piece next_piece(const ChunkArgs& a, Cursor& c) {
  Piece p;
  p.mode = END;
  while (c.pos < c.end) {
    const Tile x = tile_of<COST>(a, c.s.ql, c.s.kl, c.t);
    const int take = (int)min((long long)(x.units - c.off), c.end - c.pos);
    const int u0 = max(c.off - COST, 0), u1 = c.off + take - COST;  // key tiles of it here
    const long long first = c.pos - c.off + COST;                   // position of the tile's first key tile
    if (u1 > u0) {
      p.mode = x.mode;
      p.b = c.b;
      p.kvh = c.kvh;
      p.row0 = c.s.start + c.t * a.tile_tokens;
      p.n = x.n;
      p.pos0 = x.pos0;
      p.kl = c.s.kl;
      p.lo = x.lo;
      p.ja = x.j0 + u0;
      p.jb = x.keys ? x.j0 + u1 : p.ja;
      p.c0 = (int)quotient(first, c.per);
      p.np = (int)quotient(first + (x.units - COST) - 1, c.per) - p.c0 + 1;
      p.idx = (int)blockIdx.x - p.c0;
    }
    c.pos += take;
    c.off += take;
    if (c.off == x.units) {
      c.off = 0;
      if (++c.t * a.tile_tokens >= c.s.ql && c.pos < c.end) {
        c.t = 0;
#pragma unroll 1
        do {
          if (++c.b == a.n_seqs) c.b = 0, ++c.kvh;
          c.s = seq_get(a, c.b);
        } while (c.s.ql == 0);
      }
    }
    if (u1 > u0) break;
  }
  return p;
}

// Key tiles of a slot inside a piece: first, first + stride, ... (count of them).
struct Steps {
  int first, count, stride;
};
__device__ __forceinline__ Steps slot_steps(const ChunkArgs& a, const Piece& p, int slot) {
  Steps s;
  if (p.mode != PAIR) {
    s.first = p.ja + slot;
    s.stride = 2;
    s.count = (p.jb - p.ja - slot + 1) >> 1;
    return s;
  }
  const int n = min(p.n - slot * a.tpq, a.tpq), pos0 = p.pos0 + slot * a.tpq;
  const int hi = a.causal ? min(max(pos0 + n, 0), p.kl) : p.kl;
  const int lo = a.window && pos0 >= a.window ? min(pos0 - a.window + 1, hi) : 0;
  s.first = max(p.ja, lo / BK);
  s.stride = 1;
  s.count = hi > lo ? max(min(p.jb, (hi + BK - 1) / BK) - s.first, 0) : 0;
  return s;
}

// Order of a piece's n key tiles in the ring: pair K0 V0 K1 V1 ..., else K0 K1 V0 K2 V1 K3 V2 ...
__device__ __forceinline__ int ring_v(int mode, int i, int n) { return mode == PAIR ? 2 * i + 1 : n == 1 ? 1 : 2 + i + min(i, n - 2); }
struct RingUse {
  int tile;
  bool is_v;
};
__device__ __forceinline__ RingUse ring_use(int mode, int x, int n) {  // the inverse of ring_k and ring_v
  if (mode == PAIR || n == 1) return {x >> 1, (x & 1) != 0};
  if (x < 2) return {x, false};
  if (x < 2 * n - 2) return {(x & 1) ? (x >> 1) + 1 : (x >> 1) - 1, !(x & 1)};
  return {x - n, true};
}
__device__ __forceinline__ int ring_k(int mode, int i) { return mode == PAIR ? 2 * i : i < 2 ? i : 2 * i - 1; }

// ---- codes as 16-bit operands ---------------------------------------------------------------

// Sixteen codes to sixteen halves, exactly.  Both kinds of codes fit a half,
// so products over codes are in fp16 whatever q's type is (q in bf16: see the
// converting warps), and the weights keep a half's eleven bits.
template <int CODE>
__device__ __forceinline__ void codes_to_half(const uint4& w, uint4 (&e)[2]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (CODE == DLS_E4M3) {
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[2 * i]) : "h"((uint16_t)u[i]));
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[2 * i + 1]) : "h"((uint16_t)(u[i] >> 16)));
    } else {
      // byte b + 128 under 0x64 is the half 1024 + 128 + b
      const uint32_t c = u[i] ^ 0x80808080u, bias = 0x64806480u;  // 1152
      const uint32_t x = __byte_perm(c, 0x64646464u, 0x4140), y = __byte_perm(c, 0x64646464u, 0x4342);
      const __half2 b = *reinterpret_cast<const __half2*>(&bias);
      const __half2 p = __hsub2(*reinterpret_cast<const __half2*>(&x), b), q = __hsub2(*reinterpret_cast<const __half2*>(&y), b);
      h[2 * i] = *reinterpret_cast<const uint32_t*>(&p);
      h[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&q);
    }
  }
  e[0] = make_uint4(h[0], h[1], h[2], h[3]);
  e[1] = make_uint4(h[4], h[5], h[6], h[7]);
}

// ---- the kernel ----------------------------------------------------------------------------

struct Row {
  int lo, hi;       // keys of the row
  bool ok;          // a row of the batch (others are padding of the operand)
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Scores of keys key0 .. key0 + N - 1 outside the row's range become -inf.
template <int N>
__device__ __forceinline__ void mask_keys(uint32_t (&v)[N], int key0, const Row& row) {
  const int lo = row.lo - key0, hi = row.hi - key0;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i < lo || i >= hi) v[i] = 0xff800000u;
}

template <int N>
__device__ __forceinline__ float max_of(const uint32_t (&v)[N], float m) {
  float m4[4] = {m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < N; i += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k) m4[k] = max3(m4[k], __uint_as_float(v[i + 2 * k]), __uint_as_float(v[i + 2 * k + 1]));
  return fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
}

// Move the row's reference to mc (= c * new maximum) where that is more than
// 2^kGrow above it; O and l follow.  The S tile being there means that every
// product before it is complete, so O is at rest until the weights are handed
// over.
__device__ __forceinline__ void follow_max(float mc, const Row& row, bool first, uint32_t tO, int hd, float& R, float& l) {
  const bool grow = mc > R + kGrow;  // R = -inf before the row's first key
  if (__builtin_expect(!first && __any_sync(0xffffffffu, grow && row.ok), 0)) {
    const float f = grow ? ex2(R - mc) : 1.f;
    l *= f;
#pragma unroll 1
    for (int d = 0; d < hd; d += 16) {
      uint32_t w[16];
      tmem_read(tO + d, w);
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * f);
      tmem_st16(tO + d, w);
    }
  }
  if (grow) R = mc;
}

// The warp's weights stored so far are visible to the tensor core.
__device__ __forceinline__ void hand_over(uint32_t bar, int lane) {
  tmem_wait_st();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// Weights of scores v[at .. at + 31] and their sum.  The weights are rounded to
// 16 bits because a product with 16-bit V takes nothing wider (a second one
// for the remainders would add half to the tensor work); their sum takes them
// unrounded, so the roundings stay independent errors of half a step.
template <typename T, int N>
__device__ __forceinline__ void weights32(const uint32_t (&v)[N], int at, f2_t c2, f2_t r2, uint32_t (&w)[16], f2_t (&sum)[2]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 x = upk2(ffma2(pk2(__uint_as_float(v[at + 2 * i]), __uint_as_float(v[at + 2 * i + 1])), c2, r2));
    const float a = ex2(x.x), b = ex2(x.y);
    sum[i & 1] = fadd2(sum[i & 1], pk2(a, b));
    w[i] = Kind<T>::pack(a, b);
  }
}

// One key tile's softmax for the thread's row: 128 score columns at tS, the
// weights to the packed operand at tS + kPCol, over scores that are in
// registers by then.
template <typename T, bool HALVES>
__device__ __forceinline__ void softmax_tile(uint32_t tS, uint32_t tO, int key0, const Row& row, float c, bool first, int hd, float& R,
                                             float& l, uint32_t p_half, int lane) {
  const bool ragged = __any_sync(0xffffffffu, row.ok && (key0 < row.lo || key0 + BK > row.hi));
  uint32_t v[128];
  tmem_read(tS, v);
  if (__builtin_expect(ragged, 0)) mask_keys(v, key0, row);
  follow_max(max_of(v, -INFINITY) * c, row, first, tO, hd, R, l);
  const float nr = kShift - (R == -INFINITY ? 0.f : R);
  const f2_t c2 = pk2(c, c), r2 = pk2(nr, nr);
  f2_t sum[2] = {pk2(0.f, 0.f), pk2(0.f, 0.f)};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t w[16];
    weights32<T>(v, 32 * k, c2, r2, w, sum);
    tmem_st16(tS + kPCol + 16 * k, w);
    if (HALVES && k == 1) hand_over(p_half, lane);
  }
  const float2 s2 = upk2(fadd2(sum[0], sum[1]));
  l += s2.x + s2.y;
}

// The same over codes: sc = c * K's scale, log2 of V's scale, 1 / V's scale
// for 16 keys each.  With the score c s = sc[0] * (q . codes) the weight
// handed to the product is p * V's scale = 2^(c s + log2 V's scale - R), whose
// largest is what the reference follows, so it keeps its bits in 16 whatever
// the scales are; l takes p back from it.  cq: what the row's q was multiplied
// by, taken back.
template <bool HALVES>
__device__ __forceinline__ void softmax_codes(uint32_t tS, uint32_t tO, int key0, const Row& row, const float (&sc)[3][8], float cq, bool first,
                                              int hd, float& R, float& l, uint32_t p_half, int lane) {
  const bool ragged = __any_sync(0xffffffffu, row.ok && (key0 < row.lo || key0 + BK > row.hi));
  uint32_t v[128];
  tmem_read_by_32(tS, v);
  if (__builtin_expect(ragged, 0)) mask_keys(v, key0, row);
  float m = -INFINITY;
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    float x = __uint_as_float(v[16 * g]), y = __uint_as_float(v[16 * g + 1]);
#pragma unroll
    for (int i = 2; i < 14; i += 4) {
      x = max3(x, __uint_as_float(v[16 * g + i]), __uint_as_float(v[16 * g + i + 1]));
      y = max3(y, __uint_as_float(v[16 * g + i + 2]), __uint_as_float(v[16 * g + i + 3]));
    }
    x = max3(x, __uint_as_float(v[16 * g + 14]), __uint_as_float(v[16 * g + 15]));
    m = fmaxf(m, fmaf(fmaxf(x, y), fmaxf(sc[0][g] * cq, 0x1p-126f), sc[1][g]));
  }
  follow_max(m, row, first, tO, hd, R, l);
  const float nr = kShift - (R == -INFINITY ? 0.f : R);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t w[16];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int g = 2 * k + h;
      const float c = fmaxf(sc[0][g] * cq, 0x1p-126f), r = nr + sc[1][g];
      const f2_t c2 = pk2(c, c), r2 = pk2(r, r);
      f2_t sum = pk2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 x = upk2(ffma2(pk2(__uint_as_float(v[16 * g + 2 * i]), __uint_as_float(v[16 * g + 2 * i + 1])), c2, r2));
        const float a = ex2(x.x), b = ex2(x.y);
        sum = fadd2(sum, pk2(a, b));
        w[8 * h + i] = Kind<__half>::pack(a, b);
      }
      const float2 s = upk2(sum);
      l = fmaf(s.x + s.y, sc[2][g], l);
    }
    tmem_st16(tS + kPCol + 16 * k, w);
    if (HALVES && k == 1) hand_over(p_half, lane);
  }
}

__device__ __forceinline__ float weight(float R, float M) { return R == -INFINITY ? 0.f : ex2(R - M); }

template <int HDP>  // (the same with codes: a workspace serves both)
__device__ __forceinline__ float* partial_at(const ChunkArgs& a, int cta, int which, int slot) {
  return a.partials + (size_t)((cta * 2 + which) * 2 + slot) * (128 * (HDP + 2));  // R [128], l [128], O [HDP / 4][128][4]
}

__device__ __forceinline__ float lse_of(float R, float l) {
  return l > 0.f ? fmaf(R - kShift, 0.6931471805599453f, logf(l)) : -INFINITY;
}

// Join the partials of a tile's slot (rows 0..nrows-1; the slot's 128
// threads).  The statistics of all pieces go to shared memory first, so that
// the long loop has nothing but independent loads of O, which lie row by row
// for four columns at a time: lanes read neighbours.
template <typename T, int HDP>
__device__ __noinline__ void join(const ChunkArgs& a, int c0, int np, int kvh, int row0, int slot, int nrows, int tw, float* area) {
  float *sw = area, *sl = area + kJoinCap;
  const bool fits = np * nrows <= kJoinCap;
  const int c8 = a.head_dim / 8;
  const bool few = nrows * c8 <= 128;  // a value or none per thread
  float4 y0[8], y1[8];                 // then the first pieces' values are fetched along with the statistics
  int few_r = 0, few_d = 0;
  if (few) {
    few_d = min(tw, nrows * c8 - 1) / nrows, few_r = min(tw, nrows * c8 - 1) - few_d * nrows;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4* q = reinterpret_cast<const float4*>(partial_at<HDP>(a, c0 + min(i, np - 1), min(i, np - 1) == 0, slot) + 256) +
                        2 * few_d * 128 + few_r;
      y0[i] = __ldcg(q), y1[i] = __ldcg(q + 128);
    }
  }
  const unsigned inv_rows = ((1u << 20) + nrows - 1) / nrows;  // x / nrows = x * inv_rows >> 20 for x < 2048 (nrows <= 128)
  if (fits) {
#pragma unroll 2
    for (int x = tw; x < np * nrows; x += 128) {
      const int i = (int)((unsigned)x * inv_rows >> 20);
      const float* q = partial_at<HDP>(a, c0 + i, i == 0, slot) + (x - i * nrows);
      sw[x] = __ldcg(q);
      sl[x] = __ldcg(q + 128);
    }
    wg_sync(slot);
  }
  if (fits && tw < nrows) {
    const int r = tw;
    float M = -INFINITY, L = 0.f;
#pragma unroll 2
    for (int i = 0; i < np; ++i) M = fmaxf(M, sw[i * nrows + r]);
#pragma unroll 2
    for (int i = 0; i < np; ++i) {
      const float w = weight(sw[i * nrows + r], M);
      L = fmaf(w, sl[i * nrows + r], L);
      sw[i * nrows + r] = w;
    }
    sl[r] = L > 0.f ? 1.f / L : 0.f;
    if (a.lse) {
      const int tok = token_of(a, r);
      a.lse[((size_t)row0 + tok) * (a.n_kv * a.group) + kvh * a.group + r - tok * a.group] = lse_of(M, L);
    }
  }
  if (fits) wg_sync(slot);
  auto put = [&](int r, int d, const float4& u, const float4& v, float inv) {
    const int tok = token_of(a, r), head = kvh * a.group + r - tok * a.group;
    *reinterpret_cast<uint4*>(static_cast<T*>(a.o) + ((size_t)row0 + tok) * a.o_stride + (size_t)head * a.head_dim + 8 * d) =
        make_uint4(Kind<T>::pack(u.x * inv, u.y * inv), Kind<T>::pack(u.z * inv, u.w * inv), Kind<T>::pack(v.x * inv, v.y * inv),
                   Kind<T>::pack(v.z * inv, v.w * inv));
  };
  auto add = [](float4& u, float w, const float4& y) {
    u.x = fmaf(w, y.x, u.x), u.y = fmaf(w, y.y, u.y), u.z = fmaf(w, y.z, u.z), u.w = fmaf(w, y.w, u.w);
  };
  const int total = nrows * c8;  // at most 2048
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  if (!fits) {  // many pieces of many rows: statistics again for every value
#pragma unroll 1
    for (int x = tw; x < total; x += 128) {
      const int d = x / nrows, r = x - d * nrows;
      float M = -INFINITY, L = 0.f;
#pragma unroll 4
      for (int i = 0; i < np; ++i) M = fmaxf(M, __ldcg(partial_at<HDP>(a, c0 + i, i == 0, slot) + r));
      float4 u = zero, v = zero;
#pragma unroll 2
      for (int i = 0; i < np; ++i) {
        const float* q = partial_at<HDP>(a, c0 + i, i == 0, slot);
        const float w = weight(__ldcg(q + r), M);
        L = fmaf(w, __ldcg(q + 128 + r), L);
        add(u, w, __ldcg(reinterpret_cast<const float4*>(q + 256) + 2 * d * 128 + r));
        add(v, w, __ldcg(reinterpret_cast<const float4*>(q + 256) + (2 * d + 1) * 128 + r));
      }
      put(r, d, u, v, L > 0.f ? 1.f / L : 0.f);
      if (a.lse && d == 0) {
        const int tok = token_of(a, r);
        a.lse[((size_t)row0 + tok) * (a.n_kv * a.group) + kvh * a.group + r - tok * a.group] = lse_of(M, L);
      }
    }
    return;
  }
  // the time is the latency of the loads: eight values of eight columns in
  // flight (a thread's items are 128 apart), or four pieces of one
  if (total > 128) {
#pragma unroll 1
    for (int x0 = tw; x0 < total; x0 += 128 * 8) {
      int at[8];
      float4 u[8], v[8];
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        const int x = min(x0 + 128 * y, total - 1), d = (int)((unsigned)x * inv_rows >> 20);
        at[y] = 2 * d * 128 + x - d * nrows;  // (d, row)
        u[y] = v[y] = zero;
      }
#pragma unroll 1
      for (int i = 0; i < np; ++i) {
        const float4* q = reinterpret_cast<const float4*>(partial_at<HDP>(a, c0 + i, i == 0, slot) + 256);
#pragma unroll
        for (int y = 0; y < 8; ++y) y0[y] = __ldcg(q + at[y]), y1[y] = __ldcg(q + at[y] + 128);
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          const float w = sw[i * nrows + (at[y] & 127)];
          add(u[y], w, y0[y]);
          add(v[y], w, y1[y]);
        }
      }
#pragma unroll
      for (int y = 0; y < 8; ++y)
        if (x0 + 128 * y < total) put(at[y] & 127, at[y] >> 8, u[y], v[y], sl[at[y] & 127]);
    }
  } else if (tw < total) {
    float4 u = zero, v = zero;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float w = i < np ? sw[i * nrows + few_r] : 0.f;
      add(u, w, y0[i]);
      add(v, w, y1[i]);
    }
#pragma unroll 4
    for (int i = 8; i < np; ++i) {
      const float4* q = reinterpret_cast<const float4*>(partial_at<HDP>(a, c0 + i, false, slot) + 256) + 2 * few_d * 128 + few_r;
      const float w = sw[i * nrows + few_r];
      add(u, w, __ldcg(q));
      add(v, w, __ldcg(q + 128));
    }
    put(few_r, few_d, u, v, sl[few_r]);
  }
}

template <typename T, int HDP, int CODE>
__global__ void __launch_bounds__(kThreads<CODE>, 1) chunk_kernel(const __grid_constant__ CUtensorMap tm_q,
                                                            const __grid_constant__ CUtensorMap tm_k,
                                                            const __grid_constant__ CUtensorMap tm_v,
                                                            const __grid_constant__ ChunkArgs a) {
  using C = CCfg<HDP, CODE>;
  using W = typename std::conditional<CODE != 0, __half, T>::type;  // of the products' operands
  constexpr bool kTurnQ = !std::is_same<W, T>::value;
  using Misc = typename MiscOf<CODE>::type;
  constexpr int NST = C::NST;
  // The compiler is not to know where the parts lie: with their addresses known
  // to it the last 2048 tokens of 32768, 64 heads of 128, cost 1577 us instead of
  // 1487 over 16-bit pages, and codes (2048 of 16384, 32 heads) 477 instead of 472.
  extern __shared__ uint8_t csm_any[];
  extern __shared__ __align__(1024) uint8_t csm_aligned[];
  uint8_t* const csm = CODE ? csm_aligned : csm_any;
  const uint32_t raw = smem_u32(csm);
  uint32_t pad = CODE ? 0u : (1024u - (raw & 1023u)) & 1023u;
  if (CODE) asm volatile("" : "+r"(pad));
  if (CODE && (raw & 1023u)) {  // (no room was asked for to align it)
    if (a.status && threadIdx.x == 0) atomicOr(a.status, kTimeout);
    return;
  }
  const uint32_t qbase = raw + pad, kvbase = qbase + C::kKVOff;
  Misc& sh = *reinterpret_cast<Misc*>(csm + pad + C::kMiscOff);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // set up by warps 1 and 2 while the others begin on the plan
  if (tid == 64) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(smem_u32(&sh.full[i]), CODE ? 8 : 1);  // the copy, or the converting warps
      mbar_init(smem_u32(&sh.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.s_full[i]), 1);
      mbar_init(smem_u32(&sh.p_full[i][0]), 4);
      mbar_init(smem_u32(&sh.p_full[i][1]), 4);
      mbar_init(smem_u32(&sh.o_full[i]), 1);
      mbar_init(smem_u32(&sh.o_free[i]), 4);
    }
    mbar_init(smem_u32(&sh.q_full), 1);
    mbar_init(smem_u32(&sh.q_empty), 1);
    mbar_init(smem_u32(&sh.x_full), 4);
    for (int i = 0; i < QDEPTH; ++i) {
      mbar_init(smem_u32(&sh.pq_full[i]), 1);
      mbar_init(smem_u32(&sh.pq_empty[i]), CODE ? 18 : 10);
    }
    if constexpr (CODE != 0) {
      for (int i = 0; i < C::NRAW; ++i) {
        mbar_init(smem_u32(&sh.raw_full[i]), 33);  // the copy's bytes, and each lane's scales
        mbar_init(smem_u32(&sh.raw_empty[i]), 8);
      }
      mbar_init(smem_u32(&sh.q_ready), 8);
    }
    sh.abort = 0;
    mbar_fence_init();
  }
  if (tid == 96) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sh.tmem), 512);
    tmem_relinquish();
  }
  if (!a.small_plan) {
    plan<kThreads<CODE>, kTileCost, kMinSteps>(a, reinterpret_cast<int4*>(csm + pad), sh);
    // its scratch (generic proxy) is overwritten by TMA from here on
    fence_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  int* const ab = &sh.abort;

  if (warp < 4) {
    // (what the block was launched with, 168 or 96 a thread, is shared out anew)
    if constexpr (CODE != 0) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 0) {
      // ---------------- copies: Q tiles, and K/V tiles piece by piece of a page
      const int pr = min(1 << a.page_shift, BK);  // keys of a copy
      const int npc = BK / pr;
      const uint32_t qbytes = 128u * a.group * a.tpq * C::KA;
      int u = 0, nq = 0;
      bool ok = true, q_out = false;
      for (int k = 0; ok; ++k) {
        if (!(ok = __all_sync(0xffffffffu, cwait(smem_u32(&sh.pq_full[k % QDEPTH]), (k / QDEPTH) & 1, ab)))) break;
        const Piece p = sh.pq[k % QDEPTH];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.pq_empty[k % QDEPTH]));
        if (p.mode == END) break;
        const int n = p.jb - p.ja;
        if (n == 0) continue;
        if (nq > 0 && !(ok = __all_sync(0xffffffffu, cwait(smem_u32(&sh.q_empty), (nq - 1) & 1, ab)))) break;
        if (lane == 0) {
          const uint32_t bar = smem_u32(&sh.q_full);
          mbar_expect_tx(bar, p.mode == PAIR ? 2 * qbytes : qbytes);
          const int h0 = p.kvh * a.group;
          for (int at = 0; at < C::KA; ++at) {
            const uint32_t d = qbase + at * (128 * 128);
            tma_load_3d(d, &tm_q, at * 64, h0, p.row0, bar);
            if (p.mode == PAIR) tma_load_3d(d + C::kQ, &tm_q, at * 64, h0, p.row0 + a.tpq, bar);
          }
        }
        ++nq;
        q_out = true;
        const int32_t* table = a.page_table + (size_t)p.b * a.max_pages;
        [[maybe_unused]] int entries_at = -(1 << 30), entry = -1;
        // ring use: key tile j's K, its V, or both
        auto coded_tile = [&](int j, bool is_v) {
          if constexpr (CODE != 0) {
            constexpr int NRAW = C::NRAW;
            const int s = u % NRAW;
            if (u >= NRAW && !(ok = __all_sync(0xffffffffu, cwait(smem_u32(&sh.raw_empty[s]), ((u / NRAW) - 1) & 1, ab)))) return;
            const uint32_t bar = smem_u32(&sh.raw_full[s]), row = a.head_dim;  // bytes of a key
            uint32_t dst = qbase + C::kRawOff + s * C::kRaw;
            if (lane == 0) mbar_expect_tx(bar, (C::kTogether ? 2 : 1) * BK * row);
            __syncwarp();
            // the table's entries, 32 at a time (a load of its own for every tile would stand before its copies)
            const int first = (j * BK) >> a.page_shift, last = ((j + 1) * BK - 1) >> a.page_shift;
            if (first < entries_at || last >= entries_at + 32) {
              entries_at = first - (last - first + 1);  // V of the tile before is still to come
              const int e = entries_at + lane;
              entry = -1;
              if (e >= 0 && (long long)e << a.page_shift < p.kl && (long long)(e + 1) << a.page_shift > p.lo) entry = table[e];
            }
            constexpr int kPer = C::kTogether ? 2 : 1;
            {
              const int x = lane / kPer;
              const bool v = C::kTogether ? lane % kPer : is_v;
              const int key = j * BK + x * pr;
              const int page = __shfl_sync(0xffffffffu, entry, ((key >> a.page_shift) - entries_at) & 31);
              if (lane < npc * kPer) {
                int y = a.pool_rows;  // past the end of the pool: the copy fills zeros
                if (key < p.kl && key + pr > p.lo) {
                  if (page >= 0 && page < a.n_pages)
                    y = ((page * a.n_kv + p.kvh) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
                  else if (a.status)
                    atomicOr(a.status, kBadPage);
                }
                tma_load_2d(dst + (C::kTogether && v ? BK * row : 0) + x * pr * row, v ? &tm_v : &tm_k, 0, y, bar);
              }
            }
            if (C::kTogether || !is_v) {  // with the keys: both scales of every 16 of them (no page: 0)
              const int key = j * BK + (lane & 7) * 16;
              const int page = __shfl_sync(0xffffffffu, entry, ((key >> a.page_shift) - entries_at) & 31);
              const float* from = lane < 8 ? a.k_scales : a.v_scales;
              int bytes = 0;
              if (key < p.kl && key + 16 > p.lo && page >= 0 && page < a.n_pages) {
                from += ((size_t)((page * a.n_kv + p.kvh)) << (a.page_shift - a.block_shift)) + ((key & ((1 << a.page_shift) - 1)) >> a.block_shift);
                bytes = 4;
              }
              if (lane < 16)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(&sh.raw_scale[s][lane >> 3][lane & 7])), "l"(from), "r"(bytes)
                             : "memory");
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
            ++u;
          }
        };
        auto tile = [&](int j, bool is_v) {
          if constexpr (CODE != 0) return coded_tile(j, is_v);
          const int s = u % NST;
          if (u >= NST && !(ok = __all_sync(0xffffffffu, cwait(smem_u32(&sh.empty[s]), ((u / NST) - 1) & 1, ab)))) return;
          const uint32_t bar = smem_u32(&sh.full[s]);
          uint32_t dst = kvbase + s * C::kStage;
          if (lane == 0) mbar_expect_tx(bar, C::kStage);
          __syncwarp();
          constexpr int kPer = C::kTogether ? 2 : C::KA;  // copies of a page's piece: K and V, or the halves of a row
          if (lane < npc * kPer) {
            const int x = lane / kPer, which = lane % kPer, at = C::kTogether ? 0 : which;
            if (C::kTogether) is_v = which, dst += which * C::kKV;
            const int key = j * BK + x * pr;
            int y = a.pool_rows;  // past the end of the pool: the copy fills zeros
            if (key < p.kl && key + pr > p.lo) {
              const int page = table[key >> a.page_shift];
              if (page >= 0 && page < a.n_pages)
                y = ((page * a.n_kv + p.kvh) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
              else if (a.status)
                atomicOr(a.status, kBadPage);
            }
            tma_load_2d(dst + at * (BK * 128) + x * pr * 128, is_v ? &tm_v : &tm_k, at * 64, y, bar);
          }
          ++u;
        };
#pragma unroll 1
        for (int x = 0; ok && x < C::kUses * n; ++x) {
          const RingUse r = C::kTogether ? RingUse{x, false} : ring_use(p.mode, x, n);
          tile(p.ja + r.tile, r.is_v);
        }
      }
      // no copy may be in flight when the CTA ends
      __syncwarp();
      if constexpr (CODE != 0) {
        for (int x = u > C::NRAW ? u - C::NRAW : 0; x < u; ++x) cwait(smem_u32(&sh.raw_full[x % C::NRAW]), (x / C::NRAW) & 1, ab, false);
      } else {
        for (int x = u > NST ? u - NST : 0; x < u; ++x) cwait(smem_u32(&sh.full[x % NST]), (x / NST) & 1, ab, false);
      }
      if (q_out) cwait(smem_u32(&sh.q_full), (nq - 1) & 1, ab, false);
      __syncwarp();
    } else if (warp == 1) {
      // ---------------- MMA issue (the whole warp, converged: see umma_f16_warp)
      const uint32_t id_s = umma_idesc_f16(128, BK) | Kind<W>::kIdesc;
      const uint32_t id_o = umma_idesc_f16_bmn(128, a.head_dim) | Kind<W>::kIdesc;
      const int ksteps = a.head_dim / 16;
      constexpr bool T2 = C::kTogether;
      int u0 = 0, nq = 0;        // ring position of the piece, Q tiles seen
      int np0 = 0, np1 = 0;      // weights consumed, per slot
      bool ok = true;
      auto wait = [&](uint64_t& bar, int phase) { return __all_sync(0xffffffffu, cwait(smem_u32(&bar), phase & 1, ab)) != 0; };
      auto wait_full = [&](int u) { return wait(sh.full[u % NST], u / NST); };
      auto release = [&](int u) { umma_commit_warp(smem_u32(&sh.empty[u % NST])); };
      auto qk = [&](int slot, uint32_t q, int u) {
        const uint32_t kt = kvbase + (u % NST) * C::kStage;
        tc_fence_after();
        const uint64_t qd = umma_desc_k128(q), kd = umma_desc_k128(kt);
        int ks = 0;
#pragma unroll 1
        for (; ks + 4 <= ksteps; ks += 4) umma_f16_warp4(tmem + slot * 128, qd + ks * 256, kd + ks * 256, id_s, ks != 0);
#pragma unroll 1
        for (; ks < ksteps; ++ks) {
          const uint32_t off = (ks >> 2) * 1024 + (ks & 3) * 2;
          umma_f16_warp(tmem + slot * 128, qd + off, kd + off, id_s, ks != 0);
        }
        umma_commit_warp(smem_u32(&sh.s_full[slot]));
      };
      // the weights arrive in two halves (64 keys each); the first product of
      // a piece waits until the slot's last O has been read (of: a bit per
      // slot whether there is one, and the parity of their number four bits
      // up.  Only pieces with products of the slot have a phase of o_free: a
      // slot without keys waits for nothing, and its warps may be pieces ahead)
      uint32_t of = 0;
      auto pv = [&](int slot, int phase, int u, bool first) {
        if (!T2 && !wait(sh.p_full[slot][0], phase)) return false;
        if (T2 && !wait(sh.p_full[slot][1], phase)) return false;
        if (first) {
          if ((of >> slot & 1) && !wait(sh.o_free[slot], 1 ^ (of >> (4 + slot) & 1))) return false;
          of = (of | 1u << slot) ^ 16u << slot;
        }
        tc_fence_after();
        const uint32_t vt = kvbase + (u % NST) * C::kStage + (T2 ? C::kKV : 0), tp = tmem + slot * 128 + kPCol, to = tmem + 256 + slot * HDP;
        const uint64_t vd = umma_desc_mn128(vt, BK * 128, 1024);
        umma_f16_ta_warp4(to, tp, vd, id_o, !first);
        if (!T2 && !wait(sh.p_full[slot][1], phase)) return false;
        tc_fence_after();
        umma_f16_ta_warp4(to, tp + 32, vd + 512, id_o, true);
        return true;
      };
      for (int k = 0; ok; ++k) {
        if (!(ok = wait(sh.pq_full[k % QDEPTH], k / QDEPTH))) break;
        const Piece& p = sh.pq[k % QDEPTH];
        const int mode = uniform(p.mode);
        if (mode == END) break;
        const int n = uniform(p.jb - p.ja);
        const Steps s0 = slot_steps(a, p, 0), s1 = slot_steps(a, p, 1);
        const int f0 = uniform(s0.first - p.ja), f1 = uniform(s1.first - p.ja), c0 = uniform(s0.count), c1 = uniform(s1.count);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.pq_empty[k % QDEPTH]));
        __syncwarp();
        if (n > 0) {
          if constexpr (kTurnQ) ok = wait(sh.q_ready, nq);
          else ok = wait(sh.q_full, nq);
          if (!ok) break;
          ++nq;
          const int u = u0;
          u0 += C::kUses * n;
          if (mode == PAIR) {
            const int e0 = f0 + c0, e1 = f1 + c1;  // slot s works on key tiles f .. e - 1
            if (!(ok = wait_full(u))) break;
            if (f0 == 0 && c0) qk(0, qbase, u);
            if (f1 == 0 && c1) qk(1, qbase + C::kQ, u);
            if (!T2) release(u);
            if (n == 1) umma_commit_warp(smem_u32(&sh.q_empty));
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
              const int uv = u + (T2 ? i : 2 * i + 1), uk = uv + 1;
              const bool more = i + 1 < n;
              if (!T2 && !(ok = wait_full(uv))) break;
              if (i >= f0 && i < e0) {
                if (!(ok = pv(0, np0++, uv, i == f0))) break;
                if (i + 1 == e0) umma_commit_warp(smem_u32(&sh.o_full[0]));
              }
              if (more) {
                if (!(ok = wait_full(uk))) break;
                if (i + 1 >= f0 && i + 1 < e0) qk(0, qbase, uk);
              }
              if (i >= f1 && i < e1) {
                if (!(ok = pv(1, np1++, uv, i == f1))) break;
                if (i + 1 == e1) umma_commit_warp(smem_u32(&sh.o_full[1]));
              }
              release(uv);
              if (more) {
                if (i + 1 >= f1 && i + 1 < e1) qk(1, qbase + C::kQ, uk);
                if (!T2) release(uk);
                if (i + 2 == n) umma_commit_warp(smem_u32(&sh.q_empty));
              }
            }
          } else {
            // two key tiles (one per slot) a turn
#pragma unroll 1
            for (int i = 0; i < 2 && i < n; ++i) {
              if (!(ok = wait_full(u + i))) break;
              qk(i, qbase, u + i);
              if (!T2) release(u + i);
              if (i == n - 1) umma_commit_warp(smem_u32(&sh.q_empty));
            }
#pragma unroll 1
            for (int i = 0; ok && i < n; ++i) {
              const int slot = i & 1, uv = u + (T2 ? i : ring_v(mode, i, n));
              if (!T2 && !(ok = wait_full(uv))) break;
              if (!(ok = pv(slot, slot ? np1++ : np0++, uv, i < 2))) break;
              release(uv);
              if (i + 2 >= n) umma_commit_warp(smem_u32(&sh.o_full[slot]));
              if (i + 2 < n) {
                const int uk = u + (T2 ? i + 2 : ring_k(mode, i + 2));
                if (!(ok = wait_full(uk))) break;
                qk(slot, qbase, uk);
                if (!T2) release(uk);
                if (i + 2 == n - 1) umma_commit_warp(smem_u32(&sh.q_empty));
              }
            }
          }
        }
      }
      __syncwarp();
    } else if (warp == 2) {
      // ---------------- the CTA's pieces
      Cursor at;
      if (a.small_plan) {
        plan_warp<kTileCost, kMinSteps>(a, lane, at.pos, at.end, at.per, at.b, at.t, at.off, at.kvh, at.s);
      } else {
        at.pos = sh.range0, at.end = sh.range1, at.per = sh.per;
        at.b = sh.b0, at.t = sh.t0, at.off = sh.off0, at.kvh = sh.kvh0;
        at.s.start = sh.start0, at.s.ql = sh.ql0, at.s.kl = sh.kl0;
      }
      bool ok = true;
      int k = 0;
      for (;;) {
        const Piece p = next_piece<kTileCost>(a, at);
        if (k >= QDEPTH && !(ok = __all_sync(0xffffffffu, cwait(smem_u32(&sh.pq_empty[k % QDEPTH]), ((k / QDEPTH) - 1) & 1, ab)))) break;
        if (lane == 0) {
          sh.pq[k % QDEPTH] = p;
          mbar_arrive(smem_u32(&sh.pq_full[k % QDEPTH]));
        }
        __syncwarp();
        ++k;
        if (p.mode == END) break;
      }
    }
  } else if (CODE != 0 && warp >= 12) {
    if constexpr (CODE != 0) {
      // ---------------- codes to halves (exact), in the layout that the copies of 16-bit pages have
      asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
      constexpr int NRAW = C::NRAW;
      const int ct = tid - 12 * 32;
      const int nc = a.head_dim / 16;  // 16-byte pieces of a key
      const unsigned inv_nc = (65536 + nc - 1) / nc;        // x / nc = x * inv_nc >> 16 for x < 1024
      const bool even = (nc & (nc - 1)) == 0;
      // where the thread's column begins in an operand tile (even): see put
      const int own_c = ct & (nc - 1), own_row = (int)((unsigned)ct * inv_nc >> 16);
      const uint32_t own_at = (own_c >> 2) * (BK * 128) + own_row * 128 + ((2 * own_c & 7 ^ (own_row & 7)) << 4);
      const uint32_t own_step = C::kTogether ? 256 / nc * 128 : 4096;
      static_assert(!C::kTogether || C::kKV == BK * 128, "V's rows follow K's");
      int u = 0, nt = 0, nq = 0;                            // ring uses, key tiles, Q tiles seen
      bool ok = true;
      for (int k = 0; ok; ++k) {
        if (!(ok = __all_sync(0xffffffffu, cwait(smem_u32(&sh.pq_full[k % QDEPTH]), (k / QDEPTH) & 1, ab)))) break;
        const Piece& q = sh.pq[k % QDEPTH];
        const int mode = q.mode, n = q.jb - q.ja, ja = q.ja, kl = q.kl, lo = q.lo, tokens = q.n;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.pq_empty[k % QDEPTH]));
        if (mode == END) break;
        if (kTurnQ && n > 0) {
          // q in bf16: a row times the power of two that puts its largest
          // value next to 2^15 is a row of halves, exactly but for what lies
          // 2^38 below that value; the softmax takes the power back
          if (!(ok = __all_sync(0xffffffffu, cwait(smem_u32(&sh.q_full), nq & 1, ab)))) break;
          const int s = ct >> 7, qr = ct & 127, rows = min(mode == PAIR ? tokens - s * a.tpq : tokens, a.tpq) * a.group;
          if (qr < rows && (mode == PAIR || s == 0)) {
            const uint32_t at = qbase + s * C::kQ + qr * 128;
            uint32_t most = 0;
            for (int j = 0; j < a.head_dim / 8; ++j) {
              const uint4 w = lds128(at + (j >> 3) * (128 * 128) + (((j & 7) ^ (qr & 7)) << 4));
              const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) most = max(most, max(x[i] << 16 & 0x7fff0000u, x[i] & 0x7fff0000u));
            }
            const int e = most >= 0x7f800000u || !most ? 0 : min(14 - ((int)(most >> 23) - 127), 100);
            const float f = __uint_as_float((unsigned)(e + 127) << 23);
            for (int j = 0; j < a.head_dim / 8; ++j) {
              const uint32_t y = at + (j >> 3) * (128 * 128) + (((j & 7) ^ (qr & 7)) << 4);
              const uint4 w = lds128(y);
              auto two = [&](uint32_t x) { return Kind<__half>::pack(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xffff0000u) * f); };
              sts128(y, make_uint4(two(w.x), two(w.y), two(w.z), two(w.w)));
            }
            sh.q_exp[nq & 1][s][qr] = (int8_t)e;
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.q_ready));
          ++nq;
        }
#pragma unroll 1
        for (int x = 0; x < C::kUses * n; ++x, ++u) {
          const RingUse r = C::kTogether ? RingUse{x, false} : ring_use(mode, x, n);
          const int rs = u % NRAW, key0 = (ja + r.tile) * BK;
          if (!(ok = __all_sync(0xffffffffu, cwait(smem_u32(&sh.raw_full[rs]), (u / NRAW) & 1, ab)))) break;
          const uint32_t from = qbase + C::kRawOff + rs * C::kRaw, to = kvbase + (u % NST) * C::kStage;
          auto stage_free = [&] { return u < NST || cwait(smem_u32(&sh.empty[u % NST]), ((u / NST) - 1) & 1, ab); };
          // (read before the stage is handed back)
          const bool keys = C::kTogether || !r.is_v;
          float sk = 0.f, sv = 0.f;
          if (keys && ct < 8) sk = sh.raw_scale[rs][0][ct], sv = sh.raw_scale[rs][1][ct];
          auto scales = [&] {
            // The operand stage being free, all key tiles but the last three
            // have had their second product, and so their softmax: this place
            // of the ring is free.
            if (keys && ct < 8) {
              sk = fminf(fmaxf(sk, 0x1p-64f), 0x1p64f);
              sv = fminf(fmaxf(sv, 0x1p-64f), 0x1p64f);
              float(&to)[3][8] = sh.scale[nt % kScaleRing];
              to[0][ct] = fmaxf(a.c * sk, 0x1p-126f);  // (never 0: a masked score is -infinity times it)
              to[1][ct] = log2f(sv);
              to[2][ct] = 1.f / sv;
            }
            nt += keys;
          };
          // 16-byte chunk j of a row lies at j ^ (row & 7) of its 128 bytes.  (A row of 128 meets four bank groups twice;
          // storing the upper half's chunks in the other order, without conflicts, costs four selects a piece and 6 us of 484.)
          auto put = [&](uint32_t dst, int row, int c, const uint4& w, bool zero) {
            uint4 e[2];
            codes_to_half<CODE>(w, e);
            if (zero) e[0] = e[1] = make_uint4(0, 0, 0, 0);
            const uint32_t at = dst + (c >> 2) * (BK * 128) + row * 128 + ((2 * c & 7 ^ (row & 7)) << 4);
            sts128(at, e[0]);
            sts128(at ^ 16, e[1]);
          };
          // rows of V that no query may see can hold anything: 0 * NaN would reach every row through the product
          const bool ragged = (C::kTogether || r.is_v) && (key0 + BK > kl || key0 < lo);
          auto hidden = [&](int row) { return key0 + row >= kl || key0 + row < lo; };
          bool freed = false;
          if (even && !ragged) {
            // a thread's pieces (K's and V's, one behind the other, or of wide heads one of them) lie in one column, the
            // same distance apart in both forms (V's rows follow K's there too): addresses are sums
            uint4 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!C::kTogether || i < nc) w[i] = lds128(from + ct * 16 + i * 4096);
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.raw_empty[rs]));
            freed = true;
            if (!(ok = __all_sync(0xffffffffu, stage_free()))) break;
            const uint32_t at = to + own_at;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (C::kTogether && i >= nc) continue;
              uint4 e[2];
              codes_to_half<CODE>(w[i], e);
              sts128(at + i * own_step, e[0]);
              sts128((at ^ 16) + i * own_step, e[1]);
            }
            scales();
          } else {
            if (!(ok = __all_sync(0xffffffffu, stage_free()))) break;
            scales();
            const int total = (C::kTogether ? 2 : 1) * BK * nc;
#pragma unroll 1
            for (int i = ct; i < total; i += 256) {
              const bool second = i >= BK * nc;
              const int at = second ? i - BK * nc : i, row = (int)((unsigned)at * inv_nc >> 16);
              const bool v = C::kTogether ? second : r.is_v;
              put(to + (second ? C::kKV : 0), row, at - row * nc, lds128(from + i * 16), v && ragged && hidden(row));
            }
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (!freed) mbar_arrive(smem_u32(&sh.raw_empty[rs]));
            mbar_arrive(smem_u32(&sh.full[u % NST]));
          }
        }
      }
      __syncwarp();
    }
  } else {
    // ---------------- softmax and epilogue: slot = warpgroup, thread = row (TMEM lane)
    if constexpr (CODE != 0) asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int slot = (warp >> 2) - 1, quarter = warp & 3, tw = tid & 127;
    const uint32_t tl = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + tl + slot * 128, tO = tmem + tl + 256 + slot * HDP;
    const int hd = a.head_dim, G = a.group;
    int u0 = 0, ns = 0, nx = 0, tiles = 0, pieces = 0;
    int no[2] = {0, 0};  // phases of o_full passed
    bool ok = true;
    for (int k = 0;; ++k) {
      ok = ok && cwait(smem_u32(&sh.pq_full[k % QDEPTH]), (k / QDEPTH) & 1, ab);
      if (!(ok = wg_all(slot, ok))) break;
      // read where it lies (registers are short here); handed back at the end of the piece
      const Piece& p = sh.pq[k % QDEPTH];
      if (p.mode == END) break;
      const int n = p.jb - p.ja, u = u0;
      [[maybe_unused]] const int nt0 = tiles, nq = pieces;  // key tiles and Q tiles before this piece's
      u0 += C::kUses * n;
      tiles += n;
      pieces += n > 0;
      const Steps st = slot_steps(a, p, slot);
      const int tok0 = p.mode == PAIR ? slot * a.tpq : 0;
      const int ntok = p.mode == PAIR ? min(p.n - tok0, a.tpq) : p.n;
      const int tok = token_of(a, tw), hg = tw - tok * G;
      const bool busy = quarter * 32 < ntok * G;  // the warp has rows of the batch
      Row row;
      row.ok = tok < ntok;
      row.lo = 0;
      row.hi = 0x7fffffff;  // padding rows: never a reason to mask
      if (row.ok) {
        const int pos = p.pos0 + tok0 + tok;
        row.hi = a.causal ? min(max(pos + 1, 0), p.kl) : p.kl;
        row.lo = a.window && pos >= a.window ? pos - a.window + 1 : 0;
      }
      float R = -INFINITY, l = 0.f;
      [[maybe_unused]] float cq = 1.f;
      for (int i = 0; i < st.count; ++i) {
        const int j = st.first + i * st.stride;
        ok = __all_sync(0xffffffffu, ok && cwait(smem_u32(&sh.s_full[slot]), ns & 1, ab));
        ++ns;
        tc_fence_after();
        if (!CODE && __builtin_expect((j + 1) * BK > p.kl || j * BK < p.lo, 0)) {  // (codes: the converting warps see to it)
          // rows of V that no query may see can hold anything: 0 * NaN would
          // reach every row through the product.  (This wait comes after
          // s_full: the MMA warp has then consumed the stage's previous
          // tile, so the barrier is at most one phase behind.)
          const int uv = u + (C::kTogether ? j - p.ja : ring_v(p.mode, j - p.ja, n));
          ok = __all_sync(0xffffffffu, ok && cwait(smem_u32(&sh.full[uv % NST]), (uv / NST) & 1, ab));
          const int key = j * BK + tw;
          if (key >= p.kl || key < p.lo) {
            const uint32_t v = kvbase + (uv % NST) * C::kStage + (C::kTogether ? C::kKV : 0) + tw * 128;
            for (int at = 0; at < C::KA; ++at)
              for (int x = 0; x < 8; ++x) sts128(v + at * (BK * 128) + x * 16, make_uint4(0, 0, 0, 0));
          }
          fence_async_smem();
        }
        const uint32_t h0 = smem_u32(&sh.p_full[slot][0]), h1 = smem_u32(&sh.p_full[slot][1]);
        if (busy) {
          if constexpr (kTurnQ)
            if (i == 0) cq = __uint_as_float((unsigned)(127 - sh.q_exp[nq & 1][p.mode == PAIR ? slot : 0][tw]) << 23);
          if constexpr (CODE != 0)
            softmax_codes<!C::kTogether>(tS, tO, j * BK, row, sh.scale[(nt0 + j - p.ja) % kScaleRing], cq, i == 0, hd, R, l, h0, lane);
          else
            softmax_tile<T, !C::kTogether>(tS, tO, j * BK, row, a.c, i == 0, hd, R, l, h0, lane);
          hand_over(h1, lane);
        } else {
          // (after s_full, so that no warp arrives for two tiles in one phase)
          tc_fence_before();
          __syncwarp();
          if (!C::kTogether && lane == 0) mbar_arrive(h0);
          if (lane == 0) mbar_arrive(h1);
        }
      }
      if (st.count) {
        ok = __all_sync(0xffffffffu, ok && cwait(smem_u32(&sh.o_full[slot]), no[slot] & 1, ab));
        ++no[slot];
      }
      const int nrows = ntok * G;
      float* const part = p.np > 1 ? partial_at<HDP>(a, blockIdx.x, p.idx == 0, p.mode == PAIR ? slot : 0) : nullptr;
      const size_t t = (size_t)p.row0 + tok0 + tok;
      const int head = p.kvh * G + hg;
      bool use0 = st.count > 0, use1 = false;
      float w0 = 1.f, w1 = 0.f;
      const int count1 = slot == 1 ? 0 : slot_steps(a, p, 1).count;
      if (p.mode != PAIR) {
        // slot 0 takes slot 1's share
        if (slot == 1) {
          // (the last statistics have been read: this piece's P V waited for o_free of the piece before)
          if (st.count) {
            sh.xm[tw] = R, sh.xl[tw] = l;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.x_full));
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.pq_empty[k % QDEPTH]));
          continue;
        }
        if (count1) {
          ok = __all_sync(0xffffffffu, ok && cwait(smem_u32(&sh.x_full), nx & 1, ab) && cwait(smem_u32(&sh.o_full[1]), no[1] & 1, ab));
          ++nx;
          use1 = true;
          const float R1 = sh.xm[tw], l1 = sh.xl[tw], M = fmaxf(R, R1);
          w0 = weight(R, M);
          w1 = weight(R1, M);
          l = w0 * l + w1 * l1;
          R = M;
        }
      }
      if (count1) ++no[1];
      tc_fence_after();
      const uint32_t tO1 = tO + HDP;  // slot 1's O
      float inv = 1.f;
      if (!part) inv = l > 0.f ? 1.f / l : 0.f;
      w0 *= inv;
      w1 *= inv;
      // 64 bytes of each row at a time through shared memory, so that a store
      // covers 8 rows x 64 bytes (a lane storing its own row: 32 rows x 16,
      // 32 cycles a store); partials lie column by column and need none
      const uint32_t stage = qbase + C::kXOff + slot * 8192 + quarter * 2048;
      // the four rows that this lane stores a 16-byte chunk of, and where
      T* to[4];
      bool mine[4];
      const int ch = lane & 3;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rr = quarter * 32 + 8 * i + (lane >> 2), tk = token_of(a, rr);
        mine[i] = tk < ntok;
        to[i] = static_cast<T*>(a.o) + ((size_t)p.row0 + tok0 + tk) * a.o_stride + (size_t)(p.kvh * G + rr - tk * G) * hd + 8 * ch;
      }
      const uint32_t put = stage + lane * 64, get = stage + (lane >> 2) * 64;
      const int swz = lane >> 1 & 3;                 // of the row lane and, for every i, of row 8 i + lane / 4: (lane >> 3 & 3)
      const uint32_t got = get + ((ch ^ (lane >> 3 & 3)) << 4);
#pragma unroll 1
      for (int d = 0; busy && d < hd; d += 32) {
        if (use0 && !use1 && !part) {  // the common case: one slot's whole tile
          uint32_t v[32];
          tmem_read(tO + d, v);
          const f2_t w2 = pk2(w0, w0), none = pk2(-0.f, -0.f);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 g = upk2(ffma2(pk2(__uint_as_float(v[8 * i + 2 * e]), __uint_as_float(v[8 * i + 2 * e + 1])), w2, none));
              y[e] = Kind<T>::pack(g.x, g.y);
            }
            sts128(put + ((i ^ swz) << 4), make_uint4(y[0], y[1], y[2], y[3]));
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 y = lds128(got + i * 512);
            if (mine[i] && d + 8 * ch < hd) *reinterpret_cast<uint4*>(to[i] + d) = y;
          }
          __syncwarp();
          continue;
        }
        float f[32];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t v[16] = {}, w[16] = {};
          if (use0) tmem_read(tO + d + 16 * h, v);  // (a column past head_dim is allocated, and not stored)
          if (use1) tmem_read(tO1 + d + 16 * h, w);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            f[16 * h + i] = use0 ? __uint_as_float(v[i]) * w0 : 0.f;
            if (use1) f[16 * h + i] = fmaf(__uint_as_float(w[i]), w1, f[16 * h + i]);
          }
        }
        if (part) {
          if (row.ok)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (d + 4 * i < hd)
                __stcg(reinterpret_cast<float4*>(part + 256) + (d / 4 + i) * 128 + tw,
                       make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            sts128(put + ((i ^ swz) << 4),
                   make_uint4(Kind<T>::pack(f[8 * i], f[8 * i + 1]), Kind<T>::pack(f[8 * i + 2], f[8 * i + 3]),
                              Kind<T>::pack(f[8 * i + 4], f[8 * i + 5]), Kind<T>::pack(f[8 * i + 6], f[8 * i + 7])));
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 y = lds128(got + i * 512);
            if (mine[i] && d + 8 * ch < hd) *reinterpret_cast<uint4*>(to[i] + d) = y;
          }
          __syncwarp();
        }
      }
      // O is read: the next piece may overwrite it
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (use0) mbar_arrive(smem_u32(&sh.o_free[slot]));
        if (use1) mbar_arrive(smem_u32(&sh.o_free[1]));
      }
      if (row.ok) {
        if (part) {
          __stcg(part + tw, R);
          __stcg(part + 128 + tw, l);
        } else if (a.lse) {
          a.lse[t * (a.n_kv * G) + head] = lse_of(R, l);
        }
      }
      if (part) {
        // the last piece of the tile to arrive joins them all
        // (one thread's acquire-release orders the group's accesses: the group meets around it)
        wg_sync(slot);
        if (tw == 0) {
          int* cnt = a.counters + p.c0 * 2 + slot;
          int seen;
          asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(seen) : "l"(cnt) : "memory");
          const bool last = seen == p.np - 1;
          if (last) *cnt = 0;  // ready for the next call
          sh.last[slot] = last;
        }
        wg_sync(slot);
        if (sh.last[slot]) {
          float* area = reinterpret_cast<float*>(csm + pad + C::kXOff + slot * 8192);
          join<T, HDP>(a, p.c0, p.np, p.kvh, p.row0 + tok0, slot, nrows, tw, area);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.pq_empty[k % QDEPTH]));
    }
    if (!ok && a.status && lane == 0) atomicOr(a.status, kTimeout);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

using ChunkFn = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const ChunkArgs);

// Over codes (chunk_attn8.cu): attributes of the kernels on the current device, and a launch.
cudaError_t chunk_codes_setup();
cudaError_t launch_chunk_codes(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const ChunkArgs& a, int code, bool half,
                               int ctas, cudaStream_t s);

// The same for tiles of few rows (few_attn8.cu): at most 16 rows a tile, c's tile_tokens.
constexpr int kFewRows = 16;
cudaError_t few_codes_setup();
cudaError_t launch_few_codes(const CUtensorMap& tk, const CUtensorMap& tv, const ChunkArgs& c, const void* q, long long q_stride, bool half,
                             int code, int ctas, cudaStream_t s);

}  // namespace dls
