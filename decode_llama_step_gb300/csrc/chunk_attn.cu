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
// Warps: 0 copies (TMA), 1 MMA, 2 the CTA's piece list, 4-7 / 8-11 softmax of
// slot 0 / 1.  Every wait is bounded (2 s) and sets an abort flag.
#include <cuda_bf16.h>
#include <math.h>

#include <mutex>

#include "../../include/dls.h"
#include "kernels.h"
#include "tc.cuh"

namespace dls {

namespace {

constexpr int BK = 128;          // keys per tile
constexpr int MAXC = 152;        // CTAs at most (one per SM)
constexpr int CTHREADS = 384;
constexpr int CWARPS = CTHREADS / 32;
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
  unsigned inv_group;  // ceil(2^16 / group): r / group = r * inv_group >> 16 for r < 128
  float c;      // scale * log2(e)
  int small_plan;  // few sequences and tiles: one warp plans
};

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

template <int HDP>
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
  static constexpr int NST = 4;
  static constexpr int kKVOff = 2 * kQ;
  static constexpr int kXOff = kKVOff + NST * kStage;  // 8 KB a slot: its output rows on their way out, or statistics being joined
  static constexpr int kMiscOff = kXOff + 2 * 8192;
};

struct CMisc {
  uint64_t full[4], empty[4], s_full[2], p_full[2][2], o_full[2], o_free[2], q_full, q_empty, x_full, pq_full[QDEPTH], pq_empty[QDEPTH];
  Piece pq[QDEPTH];
  float xm[128], xl[128];        // slot 1's statistics for slot 0 (split)
  long long scan[CWARPS];
  long long range0, range1, per;
  int b0, t0, off0, kvh0;
  int start0, ql0, kl0;          // sequence b0
  uint32_t tmem;
  int abort, last[2];
};

template <int HDP>
constexpr int chunk_smem() {
  return CCfg<HDP>::kMiscOff + (int)sizeof(CMisc) + 1024;
}
static_assert(2 * kJoinCap * 4 <= 8192, "join area");
static_assert(chunk_smem<128>() <= 227 * 1024 && chunk_smem<64>() <= 227 * 1024, "shared memory");
// a CTA allocates all of tensor memory: a second one must not fit on the SM
static_assert(2 * chunk_smem<64>() > 227 * 1024, "one CTA per SM");
// the lengths being planned over lie in the Q and K/V area before its first use
static_assert(DLS_MAX_CHUNK_SEQS * 16 <= CCfg<64>::kXOff, "plan scratch");

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

__device__ __forceinline__ Tile tile_of(const ChunkArgs& a, int ql, int kl, int t) {
  Tile x;
  const int i0 = t * 2 * a.tpq;
  x.n = min(2 * a.tpq, ql - i0);
  x.mode = x.n > a.tpq ? PAIR : SPLIT;
  x.pos0 = kl - ql + i0;
  const int hi = a.causal ? min(max(x.pos0 + x.n, 0), kl) : kl;
  x.lo = a.window && x.pos0 >= a.window ? min(x.pos0 - a.window + 1, hi) : 0;
  x.j0 = x.lo / BK;
  x.keys = hi > x.lo ? (hi + BK - 1) / BK - x.j0 : 0;
  x.units = kTileCost + max(x.keys, 1);
  return x;
}

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
  for (int w = 0; w < CWARPS; ++w) {
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
__device__ __noinline__ void plan(const ChunkArgs& a, int4* info, CMisc& sh) {
  const int tid = threadIdx.x, tp = 2 * a.tpq;
  const int per_s = (a.n_seqs + CTHREADS - 1) / CTHREADS;
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
  const int before = (int)block_scan(mine, sh.scan, &total);
#pragma unroll 1
  for (int b = s0; b < s1; ++b) info[b].x += before;  // the first tile of the sequence
  __syncthreads();
  const int n_tiles = (int)total;
  const int per_t = (n_tiles + CTHREADS - 1) / CTHREADS;
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
      const int st = tile_of(a, f.y, f.z, t - f.x).units;
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
    pre = block_scan(sum, sh.scan, &total);
    const long long all = total * a.n_kv, per = max(quotient(all + gridDim.x - 1, gridDim.x), (long long)kMinSteps);
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
__device__ __forceinline__ void plan_warp(const ChunkArgs& a, int lane, long long& r0, long long& r1, long long& per, int& b0, int& t0,
                                          int& off0, int& kvh0, Seq& seq0) {
  const int per_s = (a.n_seqs + 31) / 32, tp = 2 * a.tpq;
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
        const unsigned st = tile_of(a, s.ql, s.kl, t).units;
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
    per = max(quotient(all + gridDim.x - 1, gridDim.x), (long long)kMinSteps);
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

__device__ __forceinline__ float weight(float R, float M) { return R == -INFINITY ? 0.f : ex2(R - M); }

template <int HDP>
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

template <typename T, int HDP>
__global__ void __launch_bounds__(CTHREADS, 1) chunk_kernel(const __grid_constant__ CUtensorMap tm_q,
                                                            const __grid_constant__ CUtensorMap tm_k,
                                                            const __grid_constant__ CUtensorMap tm_v,
                                                            const __grid_constant__ ChunkArgs a) {
  using C = CCfg<HDP>;
  constexpr int NST = C::NST;
  extern __shared__ uint8_t csm[];
  const uint32_t raw = smem_u32(csm);
  const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
  const uint32_t qbase = raw + pad, kvbase = qbase + C::kKVOff;
  CMisc& sh = *reinterpret_cast<CMisc*>(csm + pad + C::kMiscOff);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // set up by warps 1 and 2 while the others begin on the plan
  if (tid == 64) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(smem_u32(&sh.full[i]), 1);
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
      mbar_init(smem_u32(&sh.pq_empty[i]), 10);
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
    plan(a, reinterpret_cast<int4*>(csm + pad), sh);
    // its scratch (generic proxy) is overwritten by TMA from here on
    fence_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  int* const ab = &sh.abort;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
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
        // ring use: key tile j's K, its V, or both
        auto tile = [&](int j, bool is_v) {
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
      for (int x = u > NST ? u - NST : 0; x < u; ++x) cwait(smem_u32(&sh.full[x % NST]), (x / NST) & 1, ab, false);
      if (q_out) cwait(smem_u32(&sh.q_full), (nq - 1) & 1, ab, false);
      __syncwarp();
    } else if (warp == 1) {
      // ---------------- MMA issue (the whole warp, converged: see umma_f16_warp)
      const uint32_t id_s = umma_idesc_f16(128, BK) | Kind<T>::kIdesc;
      const uint32_t id_o = umma_idesc_f16_bmn(128, a.head_dim) | Kind<T>::kIdesc;
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
          if (!(ok = wait(sh.q_full, nq))) break;
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
      long long pos, end, per;
      int b, t, off, kvh;
      Seq s;
      if (a.small_plan) {
        plan_warp(a, lane, pos, end, per, b, t, off, kvh, s);
      } else {
        pos = sh.range0, end = sh.range1, per = sh.per;
        b = sh.b0, t = sh.t0, off = sh.off0, kvh = sh.kvh0;
        s.start = sh.start0, s.ql = sh.ql0, s.kl = sh.kl0;
      }
      bool ok = true;
      int k = 0;
      for (;;) {
        Piece p;
        p.mode = END;
        while (pos < end) {
          const Tile x = tile_of(a, s.ql, s.kl, t);
          const int take = (int)min((long long)(x.units - off), end - pos);
          const int u0 = max(off - kTileCost, 0), u1 = off + take - kTileCost;  // key tiles of it here
          const long long first = pos - off + kTileCost;                       // position of the tile's first key tile
          if (u1 > u0) {
            p.mode = x.mode;
            p.b = b;
            p.kvh = kvh;
            p.row0 = s.start + t * 2 * a.tpq;
            p.n = x.n;
            p.pos0 = x.pos0;
            p.kl = s.kl;
            p.lo = x.lo;
            p.ja = x.j0 + u0;
            p.jb = x.keys ? x.j0 + u1 : p.ja;
            p.c0 = (int)quotient(first, per);
            p.np = (int)quotient(first + (x.units - kTileCost) - 1, per) - p.c0 + 1;
            p.idx = (int)blockIdx.x - p.c0;
          }
          pos += take;
          off += take;
          if (off == x.units) {
            off = 0;
            if (++t * 2 * a.tpq >= s.ql && pos < end) {
              t = 0;
#pragma unroll 1
              do {
                if (++b == a.n_seqs) b = 0, ++kvh;
                s = seq_get(a, b);
              } while (s.ql == 0);
            }
          }
          if (u1 > u0) break;
        }
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
  } else {
    // ---------------- softmax and epilogue: slot = warpgroup, thread = row (TMEM lane)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int slot = (warp >> 2) - 1, quarter = warp & 3, tw = tid & 127;
    const uint32_t tl = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + tl + slot * 128, tO = tmem + tl + 256 + slot * HDP;
    const int hd = a.head_dim, G = a.group;
    int u0 = 0, ns = 0, nx = 0;
    int no[2] = {0, 0};  // phases of o_full passed
    bool ok = true;
    for (int k = 0;; ++k) {
      ok = ok && cwait(smem_u32(&sh.pq_full[k % QDEPTH]), (k / QDEPTH) & 1, ab);
      if (!(ok = wg_all(slot, ok))) break;
      // read where it lies (registers are short here); handed back at the end of the piece
      const Piece& p = sh.pq[k % QDEPTH];
      if (p.mode == END) break;
      const int n = p.jb - p.ja, u = u0;
      u0 += C::kUses * n;
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
      for (int i = 0; i < st.count; ++i) {
        const int j = st.first + i * st.stride;
        ok = __all_sync(0xffffffffu, ok && cwait(smem_u32(&sh.s_full[slot]), ns & 1, ab));
        ++ns;
        tc_fence_after();
        if (__builtin_expect((j + 1) * BK > p.kl || j * BK < p.lo, 0)) {
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

using ChunkFn = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const ChunkArgs);

// SMs of the current device, with the kernels' attributes set on it; 0 on an error.
int device_ready(cudaError_t* err) {
  static std::mutex mu;
  static int sms[64];
  int dev = 0;
  if ((*err = cudaGetDevice(&dev)) != cudaSuccess) return 0;
  if (dev < 0 || dev >= 64) {
    *err = cudaErrorInvalidDevice;
    return 0;
  }
  std::lock_guard<std::mutex> g(mu);
  if (sms[dev]) return sms[dev];
  int n = 0;
  if ((*err = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return 0;
  const ChunkFn f[2] = {chunk_kernel<__half, 128>, chunk_kernel<__nv_bfloat16, 128>};
  const ChunkFn h[2] = {chunk_kernel<__half, 64>, chunk_kernel<__nv_bfloat16, 64>};
  for (int i = 0; i < 2; ++i) {
    if ((*err = cudaFuncSetAttribute(f[i], cudaFuncAttributeMaxDynamicSharedMemorySize, chunk_smem<128>())) != cudaSuccess) return 0;
    if ((*err = cudaFuncSetAttribute(h[i], cudaFuncAttributeMaxDynamicSharedMemorySize, chunk_smem<64>())) != cudaSuccess) return 0;
  }
  return sms[dev] = n;
}

bool rows_ok(const void* p, long long stride, long long width) {
  return p && !(reinterpret_cast<uintptr_t>(p) & 15) && stride >= width && stride <= (1ll << 37) && stride % 8 == 0;
}

}  // namespace

}  // namespace dls

extern "C" uint64_t dls_attention_chunk_workspace_bytes(int32_t head_dim) {
  if (head_dim < 16 || head_dim > 128 || head_dim % 16) return 0;
  const uint64_t hdp = head_dim <= 64 ? 64 : 128;
  return dls::kCounterBytes + (uint64_t)dls::MAXC * 4 * 128 * (hdp + 2) * sizeof(float);
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
  if (d->n_tokens < 0 || d->n_tokens > 1 << 30 || d->n_seqs < 0 || d->n_seqs > DLS_MAX_CHUNK_SEQS || d->n_pages < 1 || d->max_pages < 1 ||
      (long long)d->max_pages * pt > 0x7fffffff - 1024)
    return report_error(DLS_ERR_ARG, "attention_chunk: n_tokens=%d n_seqs=%d (at most %d) n_pages=%d max_pages=%d", d->n_tokens, d->n_seqs,
                        DLS_MAX_CHUNK_SEQS, d->n_pages, d->max_pages);
  if ((long long)d->n_pages * d->n_kv_heads * pt > 0x7fffffff - 1024)
    return report_error(DLS_ERR_ARG, "attention_chunk: the pool has more than 2^31 - 1024 rows (n_pages=%d n_kv_heads=%d page_tokens=%d)",
                        d->n_pages, d->n_kv_heads, pt);
  if ((d->causal != 0 && d->causal != 1) || d->window < 0 || (d->window && !d->causal))
    return report_error(DLS_ERR_ARG, "attention_chunk: causal=%d window=%d (a window needs causal = 1)", d->causal, d->window);
  if (!(d->scale >= 0.f) || !isfinite(d->scale)) return report_error(DLS_ERR_ARG, "attention_chunk: scale=%g", d->scale);
  const int tpq = 128 / (d->n_heads / d->n_kv_heads);
  // decreasing cu_q can give every sequence all the rows: their tiles still have to fit an int
  if (((long long)d->n_tokens / (2 * tpq) + 1) * d->n_seqs > 0x7fffffff)
    return report_error(DLS_ERR_ARG, "attention_chunk: n_tokens=%d n_seqs=%d are too many", d->n_tokens, d->n_seqs);
  if (!aligned_to(d->status, 4) || !aligned_to(d->lse, 4))
    return report_error(DLS_ERR_ARG, "attention_chunk: lse=%p status=%p", (void*)d->lse, (void*)d->status);
  if (d->n_tokens == 0 || d->n_seqs == 0) return empty_call(d->status, cuda_stream, "attention_chunk");
  if (!rows_ok(d->q, d->q_stride, (long long)d->n_heads * hd) || !rows_ok(d->o, d->o_stride, (long long)d->n_heads * hd))
    return report_error(DLS_ERR_ARG, "attention_chunk: q and o need 16-byte aligned rows of n_heads * head_dim elements (strides %lld, %lld)",
                        (long long)d->q_stride, (long long)d->o_stride);
  if (d->q == d->o && d->q_stride != d->o_stride) return report_error(DLS_ERR_ARG, "attention_chunk: in place needs the same stride");
  if (!d->k_pages || !d->v_pages || ((reinterpret_cast<uintptr_t>(d->k_pages) | reinterpret_cast<uintptr_t>(d->v_pages)) & 15))
    return report_error(DLS_ERR_ARG, "attention_chunk: k_pages=%p v_pages=%p (16-byte aligned)", d->k_pages, d->v_pages);
  if (!d->page_table || !d->cu_q || !d->kv_len || !aligned_to(d->page_table, 4) || !aligned_to(d->cu_q, 4) || !aligned_to(d->kv_len, 4))
    return report_error(DLS_ERR_ARG, "attention_chunk: page_table=%p cu_q=%p kv_len=%p", (const void*)d->page_table, (const void*)d->cu_q,
                        (const void*)d->kv_len);
  if (!d->workspace || (reinterpret_cast<uintptr_t>(d->workspace) & 255) || d->workspace_bytes < dls_attention_chunk_workspace_bytes(hd))
    return report_error(DLS_ERR_ARG, "attention_chunk: workspace=%p bytes=%llu (256-byte aligned, at least %llu)", d->workspace,
                        (unsigned long long)d->workspace_bytes, (unsigned long long)dls_attention_chunk_workspace_bytes(hd));
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e = cudaSuccess;
  const int sms = device_ready(&e);
  if (e != cudaSuccess) return report_error(DLS_ERR_CUDA, "attention_chunk: cuda=%s", cudaGetErrorString(e));
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
  a.tpq = tpq, a.inv_group = (65536 + a.group - 1) / a.group;
  a.c = (d->scale > 0.f ? d->scale : 1.0f / sqrtf((float)hd)) * 1.4426950408889634f;
  // a lane of the planning warp walks at most 4 sequences and 8 more tiles; its sums fit 32 bits.
  // One token over 2048: 15.5 us with the warp's plan, 16.2 with the block's; 64 over up to 8192 (5301 on average) 218 and 220 us.
  a.small_plan = d->n_seqs <= 128 && d->n_tokens <= 8 * 2 * a.tpq && (long long)d->max_pages * pt <= 1 << 24;
  const CUtensorMapDataType dt = d->kv_type == DLS_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const uint32_t pr = pt < BK ? pt : BK;
  CUtensorMap tq, tk, tv;
  const uint64_t dims[3] = {(uint64_t)hd, (uint64_t)d->n_heads, (uint64_t)d->n_tokens};
  const uint64_t strides[2] = {(uint64_t)hd * 2, (uint64_t)d->q_stride * 2};
  const uint32_t box[3] = {64, (uint32_t)a.group, (uint32_t)a.tpq};
  if (!make_tmap_3d(&tq, dt, d->q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_2d(&tk, dt, d->k_pages, hd, a.pool_rows, hd * 2, 64, pr, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_2d(&tv, dt, d->v_pages, hd, a.pool_rows, hd * 2, 64, pr, CU_TENSOR_MAP_SWIZZLE_128B))
    return report_error(DLS_ERR_CUDA, "attention_chunk: tensor map (head_dim=%d n_heads=%d n_tokens=%d)", hd, d->n_heads, d->n_tokens);
  if (a.status) e = cudaMemsetAsync(a.status, 0, sizeof(int32_t), s);
  if (e == cudaSuccess) {
    const bool half = d->kv_type == DLS_F16;
    const ChunkFn f = hd <= 64 ? (half ? chunk_kernel<__half, 64> : chunk_kernel<__nv_bfloat16, 64>)
                               : (half ? chunk_kernel<__half, 128> : chunk_kernel<__nv_bfloat16, 128>);
    f<<<sms < MAXC ? sms : MAXC, CTHREADS, hd <= 64 ? chunk_smem<64>() : chunk_smem<128>(), s>>>(tq, tk, tv, a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return report_error(DLS_ERR_CUDA, "attention_chunk: cuda=%s", cudaGetErrorString(e));
  return DLS_OK;
}
