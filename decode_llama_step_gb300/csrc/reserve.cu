// Pages reserved and rows laid out for a batch of requests, from their lengths
// on the device.
//
// Mathematics (b = sequence, in order; page = page_tokens):
//   give_b = held_b where the request is over; its pages go on the stack
//   need_b = max(0, ceil((kv_b + new_b) / page) - held_b)
//   pages are granted where the inclusive prefix sum of need fits the stack,
//   rows where the inclusive prefix sum of new (of those granted) fits
//   max_rows; page i of b's fresh ones is stack[avail - 1 - (exclusive need + i)].
// Both prefix sums only grow, so what does not fit leaves out a tail of the
// sequences that need something, and the sums of those granted need no second
// round.
//
// What bounds it: latency.  A batch is a few kilobytes; the chain is lengths,
// two block scans, the stack's (or the table's) page, the row's stores.  One
// launch: every CTA of the cluster reads the lengths and scans them all by
// itself, the cluster meets once (the state may be written only after all have
// read it, the stack read only after the pages that come back are on it), then
// each takes its share of the rows.
// Measured (GPU time): 64 single tokens 5.0 us, 211 prompts of 300 thousand rows
// together 14.0 us (16 CTAs; 17.4 with eight).
#include <type_traits>

#include "../../include/dls.h"
#include "kernels.h"

namespace dls {

namespace {

constexpr int kMostThreads = 1024;
constexpr int kPerThread = DLS_MAX_CHUNK_SEQS / kMostThreads;  // sequences of a thread at most
// Sums stop here, above every bound that they are held to (2^27 pages, 2^30 rows): sums cut off so stay a prefix sum,
// and those that matter are exact.
constexpr unsigned kCap = (1u << 30) + 1;

struct ReserveArgs {
  const int32_t *new_len, *kv_len, *held, *free_count;
  int32_t *page_table, *free_pages, *kv_len_out, *held_out, *free_count_out, *cu_q;
  int32_t *positions, *slots, *seq_ids, *status;
  int n_seqs, max_rows, page_shift, n_pages, max_pages;
};

// A sequence as the row pass needs it.
struct SeqRow {
  int kv, held, pop;  // cached tokens, pages held, stack index of its first fresh page (ended: where its pages go)
};

__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ unsigned cluster_size() {
  unsigned r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ unsigned capped(unsigned a, unsigned b) { return min(a + b, kCap); }  // (both at most kCap)

// Inclusive prefix sums of two values over the warp.
__device__ __forceinline__ void warp_scan2(unsigned& x, unsigned& y, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned ux = __shfl_up_sync(0xffffffffu, x, o), uy = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) x = capped(x, ux), y = capped(y, uy);
  }
}
// Of two values a thread: the sums of the threads before, and of all.
__device__ __forceinline__ void block_scan2(unsigned x, unsigned y, uint2& before, uint2& total, uint2* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned ix = x, iy = y;
  warp_scan2(ix, iy, lane);
  if (lane == 31) sums[warp] = make_uint2(ix, iy);
  const unsigned px = __shfl_up_sync(0xffffffffu, ix, 1), py = __shfl_up_sync(0xffffffffu, iy, 1);
  __syncthreads();
  // every warp scans the warps' sums by itself
  const uint2 w = lane < (int)(blockDim.x >> 5) ? sums[lane] : make_uint2(0, 0);
  unsigned wx = w.x, wy = w.y;
  warp_scan2(wx, wy, lane);
  total = make_uint2(__shfl_sync(0xffffffffu, wx, 31), __shfl_sync(0xffffffffu, wy, 31));
  const unsigned bx = __shfl_sync(0xffffffffu, wx, (warp + 31) & 31), by = __shfl_sync(0xffffffffu, wy, (warp + 31) & 31);
  before = make_uint2(capped(warp ? bx : 0, lane ? px : 0), capped(warp ? by : 0, lane ? py : 0));
}

__global__ void __launch_bounds__(kMostThreads, 1) reserve_kernel(const __grid_constant__ ReserveArgs a) {
  extern __shared__ __align__(16) uint8_t rsm[];
  __shared__ uint2 sums[2][32];
  __shared__ int s_flags, s_used, s_end;
  int* const cu = reinterpret_cast<int*>(rsm);                       // [n_seqs + 1]
  SeqRow* const rows = reinterpret_cast<SeqRow*>(cu + a.n_seqs + 1);  // [n_seqs]
  const int tid = threadIdx.x, lane = tid & 31, threads = blockDim.x;
  const unsigned rank = cluster_rank(), ctas = cluster_size();
  const int page = 1 << a.page_shift;
  const long long room = (long long)a.max_pages << a.page_shift;
  const int per = (a.n_seqs + threads - 1) / threads, b0 = min(tid * per, a.n_seqs), b1 = min(b0 + per, a.n_seqs);

  int fresh[kPerThread], kv[kPerThread], held[kPerThread], need[kPerThread];
  bool grant[kPerThread], lost[kPerThread];  // lost: over, in a state that cannot be
  int flags = 0;
  if (tid == 0) s_flags = s_used = s_end = 0;
  const int count_in = *a.free_count;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    fresh[i] = kv[i] = held[i] = 0;
    if (b0 + i < b1) fresh[i] = a.new_len[b0 + i], kv[i] = a.kv_len[b0 + i], held[i] = a.held[b0 + i];
  }
  const int count = min(max(count_in, 0), a.n_pages);
  if (count != count_in) flags |= kBadPos;
  unsigned give_sum = 0, need_sum = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    // a state that cannot be: the request is left out, its pages are not given back
    const bool bad = kv[i] < 0 || kv[i] > room || held[i] < 0 || held[i] > a.max_pages || ((long long)held[i] << a.page_shift) < kv[i];
    const bool far = fresh[i] > 0 && (long long)kv[i] + fresh[i] > room;
    if (bad || far) flags |= kBadPos;
    grant[i] = !bad && !far && fresh[i] > 0;
    need[i] = grant[i] ? max(0, (int)(((long long)kv[i] + fresh[i] + page - 1) >> a.page_shift) - held[i]) : 0;
    lost[i] = bad && fresh[i] < 0;
    if (lost[i]) held[i] = 0;
    if (fresh[i] < 0) give_sum = capped(give_sum, held[i]);
    need_sum = capped(need_sum, need[i]);
  }
  uint2 before, total;
  block_scan2(give_sum, need_sum, before, total, sums[0]);
  const unsigned give_before = before.x, need_before = before.y;
  if (capped(count, total.x) > (unsigned)a.n_pages) flags |= kBadPos;  // (more pages than the pool has: the rest is dropped)
  const unsigned avail = min(capped(count, total.x), (unsigned)a.n_pages);
  // pages
  unsigned row_sum = 0, at = need_before;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    at = capped(at, need[i]);
    if (grant[i] && need[i] && at > avail) grant[i] = false, flags |= kNoRoom;
    if (grant[i]) row_sum = capped(row_sum, min((unsigned)fresh[i], kCap));
  }
  block_scan2(row_sum, 0, before, total, sums[1]);
  // rows, and what is left of both
  unsigned pop = need_before, give = give_before;
  int used = 0, end = 0;
  at = before.x;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    if (b0 + i >= b1) continue;
    if (grant[i]) at = capped(at, min((unsigned)fresh[i], kCap));
    const bool fits = at <= (unsigned)a.max_rows;
    if (grant[i] && !fits) grant[i] = false, flags |= kNoRoom;
    if (fits) end = (int)at;
    SeqRow r;
    r.kv = kv[i], r.held = held[i];
    r.pop = fresh[i] < 0 ? (int)min(capped(count, give), (unsigned)a.n_pages) : pop < avail ? (int)(avail - 1 - pop) : -1;
    rows[b0 + i] = r;
    cu[b0 + i + 1] = fits ? (int)at : -1;  // (-1: where the last rows that fit end)
    if (fresh[i] < 0) give = capped(give, held[i]);
    pop = capped(pop, need[i]);
    if (!grant[i]) need[i] = 0;
    used += need[i];
  }
  used = (int)__reduce_add_sync(0xffffffffu, (unsigned)used);
  end = (int)__reduce_max_sync(0xffffffffu, (unsigned)end);
  flags = (int)__reduce_or_sync(0xffffffffu, (unsigned)flags);
  if (lane == 0) {
    atomicMax(&s_end, end);
    if (used) atomicAdd(&s_used, used);
    if (flags) atomicOr(&s_flags, flags);
  }
  if (tid == 0) cu[0] = 0;
  const bool gives = __syncthreads_or(give_sum != 0);
  const int all = s_end;
  for (int b = b0; b < b1; ++b)
    if (cu[b + 1] < 0) cu[b + 1] = all;

  // pages of ended requests go on the stack: 32 sequences a look, a warp for each of theirs
  const int warps = ctas * (threads >> 5), warp = rank * (threads >> 5) + (tid >> 5);
  for (int b = warp * 32; gives && b < a.n_seqs; b += warps * 32) {
    const bool over = b + lane < a.n_seqs && a.new_len[b + lane] < 0 && rows[b + lane].held > 0;
    unsigned todo = __ballot_sync(0xffffffffu, over);
    while (todo) {
      const int s = b + __ffs(todo) - 1;
      todo &= todo - 1;
      const SeqRow r = rows[s];
      const int n = min(r.held, a.n_pages - r.pop);
      for (int j = lane; j < n; j += 32) a.free_pages[r.pop + j] = a.page_table[(size_t)s * a.max_pages + j];
    }
  }
  // (the state is read, the stack is whole; a cluster of one takes 2000 cycles for its barrier, a block 30)
  if (ctas > 1) cluster_meet();
  else __syncthreads();

  if (rank == 0) {
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int b = b0 + i;
      if (b >= b1) continue;
      const bool over = fresh[i] < 0;
      // (in place, what is there is the only record of pages that were not given back: it stays)
      if (!lost[i] || a.kv_len_out != a.kv_len) a.kv_len_out[b] = over ? 0 : kv[i] + cu[b + 1] - cu[b];
      if (!lost[i] || a.held_out != a.held) a.held_out[b] = over ? 0 : held[i] + need[i];
      a.cu_q[b + 1] = cu[b + 1];
    }
    if (tid == 0) {
      a.cu_q[0] = 0;
      *a.free_count_out = (int)avail - s_used;
      if (a.status) atomicOr(a.status, s_flags);
    }
  }

  // Rows: a warp takes a run of them, a lane one at a time or, where there are
  // many, four neighbours, which then as a rule are of one sequence and one page.
  // (16-byte stores where the arrays allow.)
  bool bad_page = false;
  auto seq_from = [&](int lo, int row) {  // the sequence from lo on that holds the row: the last that begins there or before
    if (cu[lo + 1] > row) return lo;
    int hi = a.n_seqs;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cu[mid] <= row) lo = mid;
      else hi = mid;
    }
    return lo;
  };
  auto page_of = [&](int s, const SeqRow& q, int j, bool first) {  // first: the row that enters a fresh page in the table
    if (j < q.held) return a.page_table[(size_t)s * a.max_pages + j];
    const int x = q.pop - (j - q.held), p = x >= 0 ? a.free_pages[x] : -1;
    if (first) a.page_table[(size_t)s * a.max_pages + j] = p;
    return p;
  };
  auto run = [&](auto lane_rows) {
    constexpr int kRowsLane = decltype(lane_rows)::value, kTurn = 32 * kRowsLane;
    const int share = ((all + warps - 1) / warps + kRowsLane - 1) / kRowsLane * kRowsLane;
    const int r0 = (int)min((long long)share * warp, (long long)all), r1 = min(r0 + share, all);
    int s = 0;
    for (int r = r0 + lane * kRowsLane; r < r1; r += kTurn) {
      int pos[kRowsLane], slot[kRowsLane], id[kRowsLane];
      s = seq_from(s, r);
      const int n = min(kRowsLane, r1 - r);
      SeqRow q = rows[s];
      int begin = cu[s], end_s = cu[s + 1], x = s, last = -1, p = -1;
#pragma unroll
      for (int i = 0; i < kRowsLane; ++i) {
        if (i >= n) continue;
        if (r + i >= end_s) {
          x = seq_from(x, r + i);
          q = rows[x], begin = cu[x], end_s = cu[x + 1], last = -1;
        }
        const int at_pos = q.kv + r + i - begin, j = at_pos >> a.page_shift, off = at_pos & (page - 1);
        if (j != last || off == 0) p = page_of(x, q, j, off == 0), last = j;
        const bool ok = p >= 0 && p < a.n_pages;
        bad_page |= !ok;
        pos[i] = at_pos, slot[i] = ok ? (p << a.page_shift) + off : -1, id[i] = x;
      }
      auto put = [&](int32_t* to, const int (&v)[kRowsLane]) {
        if (!to) return;
        if (kRowsLane == 4 && n == 4 && !(reinterpret_cast<uintptr_t>(to) & 15)) {
          *reinterpret_cast<int4*>(to + r) = make_int4(v[0], v[kRowsLane > 1], v[kRowsLane / 2], v[kRowsLane - 1]);
        } else {
#pragma unroll
          for (int i = 0; i < kRowsLane; ++i)
            if (i < n) to[r + i] = v[i];
        }
      };
      put(a.positions, pos);
      put(a.slots, slot);
      put(a.seq_ids, id);
    }
  };
  if (all > warps * 32) run(std::integral_constant<int, 4>());
  else run(std::integral_constant<int, 1>());
  if (a.status && bad_page) atomicOr(a.status, kBadPage);
}

}  // namespace

}  // namespace dls

extern "C" int dls_kv_reserve(const dls_kv_reserve_desc* d, void* cuda_stream) {
  using namespace dls;
  if (!d) return report_error(DLS_ERR_ARG, "kv_reserve: desc=NULL");
  const int pt = d->page_tokens;
  if (pt != 16 && pt != 32 && pt != 64 && pt != 128 && pt != 256)
    return report_error(DLS_ERR_ARG, "kv_reserve: page_tokens=%d (16, 32, 64, 128 or 256)", pt);
  if (d->n_seqs < 0 || d->n_seqs > DLS_MAX_CHUNK_SEQS || d->max_rows < 0 || d->max_rows > 1 << 30 || d->n_pages < 1 || d->max_pages < 1 ||
      (long long)d->max_pages * pt > 0x7fffffff || (long long)d->n_pages * pt > 0x7fffffff)
    return report_error(DLS_ERR_ARG, "kv_reserve: n_seqs=%d (at most %d) max_rows=%d (at most 2^30) n_pages=%d max_pages=%d (times page_tokens below 2^31)",
                        d->n_seqs, DLS_MAX_CHUNK_SEQS, d->max_rows, d->n_pages, d->max_pages);
  if (!d->cu_q || !d->free_count || !d->free_count_out || !d->free_pages)
    return report_error(DLS_ERR_ARG, "kv_reserve: cu_q=%p free_count=%p free_count_out=%p free_pages=%p", (void*)d->cu_q,
                        (const void*)d->free_count, (void*)d->free_count_out, (void*)d->free_pages);
  if (d->n_seqs && (!d->new_len || !d->kv_len || !d->held || !d->page_table || !d->kv_len_out || !d->held_out))
    return report_error(DLS_ERR_ARG, "kv_reserve: new_len=%p kv_len=%p held=%p page_table=%p kv_len_out=%p held_out=%p",
                        (const void*)d->new_len, (const void*)d->kv_len, (const void*)d->held, (void*)d->page_table, (void*)d->kv_len_out,
                        (void*)d->held_out);
  const void* all[] = {d->new_len, d->kv_len, d->held, d->page_table, d->free_pages, d->free_count, d->kv_len_out, d->held_out,
                       d->free_count_out, d->cu_q, d->positions, d->slots, d->seq_ids, d->status};
  for (const void* p : all)
    if (!aligned_to(p, 4)) return report_error(DLS_ERR_ARG, "kv_reserve: %p is not aligned to its int32 elements", p);
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  ReserveArgs a{};
  a.new_len = d->new_len, a.kv_len = d->kv_len, a.held = d->held, a.free_count = d->free_count;
  a.page_table = d->page_table, a.free_pages = d->free_pages;
  a.kv_len_out = d->kv_len_out, a.held_out = d->held_out, a.free_count_out = d->free_count_out, a.cu_q = d->cu_q;
  a.positions = d->positions, a.slots = d->slots, a.seq_ids = d->seq_ids, a.status = d->status;
  a.n_seqs = d->n_seqs, a.max_rows = d->max_rows, a.n_pages = d->n_pages, a.max_pages = d->max_pages;
  a.page_shift = pt == 16 ? 4 : pt == 32 ? 5 : pt == 64 ? 6 : pt == 128 ? 7 : 8;
  cudaError_t e = cudaSuccess;
  if (a.status) e = cudaMemsetAsync(a.status, 0, sizeof(int32_t), s);
  const int smem = (a.n_seqs + 1) * 4 + a.n_seqs * (int)sizeof(SeqRow);
  if (e == cudaSuccess && a.max_rows > 131072)  // a cluster of 16
    e = cudaFuncSetAttribute(reserve_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && smem > 40 * 1024)  // beyond what a launch may ask for unannounced (48 KB, the static part with it)
    e = cudaFuncSetAttribute(reserve_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (DLS_MAX_CHUNK_SEQS + 1) * 4 + DLS_MAX_CHUNK_SEQS * (int)sizeof(SeqRow));
  if (e == cudaSuccess) {
    cudaLaunchConfig_t c{};
    cudaLaunchAttribute at[1];
    const unsigned ctas = a.max_rows <= 4096 ? 1 : a.max_rows <= 16384 ? 2 : a.max_rows <= 65536 ? 4 : a.max_rows <= 131072 ? 8 : 16;
    const int wanted = std::max(a.n_seqs, a.max_rows / 4);
    int threads = 128;
    while (threads < kMostThreads && threads < wanted) threads *= 2;
    c.gridDim = dim3(ctas), c.blockDim = dim3(threads), c.dynamicSmemBytes = smem, c.stream = s;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ctas, at[0].val.clusterDim.y = 1, at[0].val.clusterDim.z = 1;
    c.attrs = at, c.numAttrs = 1;
    e = cudaLaunchKernelEx(&c, reserve_kernel, a);
  }
  if (e != cudaSuccess) return report_error(DLS_ERR_CUDA, "kv_reserve: cuda=%s", cudaGetErrorString(e));
  return DLS_OK;
}
