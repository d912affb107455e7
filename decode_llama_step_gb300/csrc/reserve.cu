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
#include <math.h>

#include "../../include/dls.h"
#include "kernels.h"

namespace dls {

namespace {

constexpr int RSV_THREADS = 1024;
constexpr int RSV_WARPS = RSV_THREADS / 32;
constexpr int kPerThread = DLS_MAX_CHUNK_SEQS / RSV_THREADS;  // sequences of a thread at most

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

// Exclusive prefix sums of two values over the block; the totals too.
__device__ __forceinline__ void block_scan2(long long& x, long long& y, long long& tx, long long& ty, longlong2* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long ix = x, iy = y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long ux = __shfl_up_sync(0xffffffffu, ix, o), uy = __shfl_up_sync(0xffffffffu, iy, o);
    if (lane >= o) ix += ux, iy += uy;
  }
  __syncthreads();  // the sums' last readers are through
  if (lane == 31) sums[warp] = make_longlong2(ix, iy);
  __syncthreads();
  // every warp scans the warps' sums by itself
  longlong2 w = sums[lane];
  const longlong2 mine = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long ux = __shfl_up_sync(0xffffffffu, w.x, o), uy = __shfl_up_sync(0xffffffffu, w.y, o);
    if (lane >= o) w.x += ux, w.y += uy;
  }
  tx = __shfl_sync(0xffffffffu, w.x, 31);
  ty = __shfl_sync(0xffffffffu, w.y, 31);
  const long long px = __shfl_sync(0xffffffffu, w.x - mine.x, warp), py = __shfl_sync(0xffffffffu, w.y - mine.y, warp);
  x = px + ix - x;
  y = py + iy - y;
}
static_assert(RSV_WARPS == 32, "block_scan2 gives each warp's sum to a lane");

__global__ void __launch_bounds__(RSV_THREADS, 1) reserve_kernel(const __grid_constant__ ReserveArgs a) {
  extern __shared__ uint8_t rsm[];
  __shared__ longlong2 sums[32];
  int* const cu = reinterpret_cast<int*>(rsm);                       // [n_seqs + 1]
  SeqRow* const rows = reinterpret_cast<SeqRow*>(cu + a.n_seqs + 1);  // [n_seqs]
  const int tid = threadIdx.x, lane = tid & 31;
  const unsigned rank = cluster_rank(), ctas = cluster_size();
  const int page = 1 << a.page_shift;
  const long long room = (long long)a.max_pages << a.page_shift;
  const int per = (a.n_seqs + RSV_THREADS - 1) / RSV_THREADS, b0 = min(tid * per, a.n_seqs), b1 = min(b0 + per, a.n_seqs);

  int fresh[kPerThread], kv[kPerThread], held[kPerThread], need[kPerThread];
  bool grant[kPerThread];
  int flags = 0;
  const int count_in = *a.free_count, count = min(max(count_in, 0), a.n_pages);
  if (count != count_in) flags |= kBadPos;
  long long give_sum = 0, need_sum = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    fresh[i] = kv[i] = held[i] = need[i] = 0;
    grant[i] = false;
    if (b0 + i >= b1) continue;
    fresh[i] = a.new_len[b0 + i], kv[i] = a.kv_len[b0 + i], held[i] = a.held[b0 + i];
    // a state that cannot be: the request is left out, its pages are not given back
    const bool bad = kv[i] < 0 || kv[i] > room || held[i] < 0 || held[i] > a.max_pages || ((long long)held[i] << a.page_shift) < kv[i];
    const bool far = fresh[i] > 0 && (long long)kv[i] + fresh[i] > room;
    if (bad || far) flags |= kBadPos;
    grant[i] = !bad && !far && fresh[i] > 0;
    if (grant[i]) need[i] = max(0, (int)(((long long)kv[i] + fresh[i] + page - 1) >> a.page_shift) - held[i]);
    if (fresh[i] < 0 && !bad) give_sum += held[i];
    else if (fresh[i] < 0) held[i] = 0;
    need_sum += need[i];
  }
  long long give_at = give_sum, need_at = need_sum, give_total, need_total;
  block_scan2(give_at, need_at, give_total, need_total, sums);
  if (count + give_total > a.n_pages) flags |= kBadPos;  // (more pages than the pool has: the rest is dropped)
  const int avail = (int)min(count + give_total, (long long)a.n_pages);
  // pages
  long long row_sum = 0;
  {
    long long at = need_at;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      at += need[i];
      if (grant[i] && need[i] && at > avail) grant[i] = false, flags |= kNoRoom;
      if (grant[i]) row_sum += fresh[i];
    }
  }
  long long row_at = row_sum, zero = 0, row_total, none;
  block_scan2(row_at, zero, row_total, none, sums);
  // rows, and what is left of both
  long long used = 0;
  int last = 0;  // one past the thread's last row
  {
    long long at = row_at, pop = need_at, give = give_at;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      if (b0 + i >= b1) continue;
      const bool asked = grant[i];
      if (asked) at += fresh[i];
      if (asked && at > a.max_rows) grant[i] = false, flags |= kNoRoom;
      SeqRow r;
      r.kv = kv[i], r.held = held[i];
      r.pop = fresh[i] < 0 ? (int)min(count + give, (long long)a.n_pages) : (int)max(avail - 1 - pop, -1ll);
      rows[b0 + i] = r;
      cu[b0 + i + 1] = grant[i] ? (int)at : -1;  // where it ends; settled below
      if (fresh[i] < 0) give += held[i];
      pop += need[i];
      if (grant[i]) used += need[i], last = (int)at;
      else need[i] = 0;
    }
  }
  // totals of what was granted: pages used, and the end of the rows
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    used += __shfl_xor_sync(0xffffffffu, used, o);
    last = max(last, __shfl_xor_sync(0xffffffffu, last, o));
    flags |= __shfl_xor_sync(0xffffffffu, flags, o);
  }
  __shared__ int w_last[RSV_WARPS], w_flags[RSV_WARPS];
  __shared__ long long w_used[RSV_WARPS];
  if (lane == 0) w_last[tid >> 5] = last, w_used[tid >> 5] = used, w_flags[tid >> 5] = flags;
  // a sequence without rows ends where the one before it does
  __syncthreads();
  int end = 0;  // the end of the rows before this thread's sequences
  for (int w = 0; w < (tid >> 5); ++w) end = max(end, w_last[w]);
  {
    int mine = 0;
    for (int b = b0; b < b1; ++b) mine = max(mine, cu[b + 1]);
    int pre = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) pre = max(pre, u);
    }
    const int before = __shfl_up_sync(0xffffffffu, pre, 1);
    if (lane) end = max(end, before);
    for (int b = b0; b < b1; ++b) cu[b + 1] = end = max(end, cu[b + 1]);
  }
  int total = 0;
  used = 0;
  for (int w = 0; w < RSV_WARPS; ++w) total = max(total, w_last[w]), used += w_used[w], flags |= w_flags[w];
  if (tid == 0) cu[0] = 0;
  __syncthreads();

  // pages of ended requests go on the stack: 32 sequences a look, a warp for each of theirs
  const int warps = ctas * RSV_WARPS, warp = rank * RSV_WARPS + (tid >> 5);
  for (int b = warp * 32; b < a.n_seqs; b += warps * 32) {
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
  cluster_meet();  // (the state is read, the stack is whole)

  if (rank == 0) {
    for (int i = 0; b0 + i < b1; ++i) {
      const int b = b0 + i;
      const bool over = fresh[i] < 0;
      a.kv_len_out[b] = over ? 0 : kv[i] + cu[b + 1] - cu[b];
      a.held_out[b] = over ? 0 : held[i] + need[i];
      a.cu_q[b + 1] = cu[b + 1];
    }
    if (tid == 0) {
      a.cu_q[0] = 0;
      *a.free_count_out = avail - (int)used;
      if (a.status) atomicOr(a.status, flags);
    }
  }

  // rows: a warp takes a run of them, 32 at a time
  const long long share = ((long long)total + warps - 1) / warps;
  const int r0 = (int)min(share * warp, (long long)total), r1 = (int)min((long long)r0 + share, (long long)total);
  bool bad_page = false;
  int s = 0;
  if (r0 < r1) {
    int lo = 0, hi = a.n_seqs;  // the last sequence that begins at r0 or before and is not empty
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cu[mid] <= r0) lo = mid;
      else hi = mid;
    }
    s = lo;
  }
  for (int r = r0; r < r1; r += 32) {
    const int row = r + lane;
    if (row < r1) {
      if (cu[s + 1] <= row) {
        int lo = s, hi = a.n_seqs;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (cu[mid] <= row) lo = mid;
          else hi = mid;
        }
        s = lo;
      }
      const SeqRow q = rows[s];
      const int pos = q.kv + row - cu[s], j = pos >> a.page_shift, off = pos & (page - 1);
      int p;
      if (j >= q.held) {
        const int at = q.pop - (j - q.held);
        p = at >= 0 ? a.free_pages[at] : -1;
        if (off == 0) a.page_table[(size_t)s * a.max_pages + j] = p;
      } else {
        p = a.page_table[(size_t)s * a.max_pages + j];
      }
      const bool ok = p >= 0 && p < a.n_pages;
      bad_page |= !ok;
      if (a.positions) a.positions[row] = pos;
      if (a.slots) a.slots[row] = ok ? (p << a.page_shift) + off : -1;
      if (a.seq_ids) a.seq_ids[row] = s;
    }
  }
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
  if (e == cudaSuccess && smem > 40 * 1024)  // beyond what a launch may ask for unannounced (48 KB, the static part with it)
    e = cudaFuncSetAttribute(reserve_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (DLS_MAX_CHUNK_SEQS + 1) * 4 + DLS_MAX_CHUNK_SEQS * (int)sizeof(SeqRow));
  if (e == cudaSuccess) {
    cudaLaunchConfig_t c{};
    cudaLaunchAttribute at[1];
    const unsigned ctas = a.max_rows <= 4096 ? 1 : a.max_rows <= 16384 ? 2 : a.max_rows <= 65536 ? 4 : 8;
    c.gridDim = dim3(ctas), c.blockDim = dim3(RSV_THREADS), c.dynamicSmemBytes = smem, c.stream = s;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ctas, at[0].val.clusterDim.y = 1, at[0].val.clusterDim.z = 1;
    c.attrs = at, c.numAttrs = 1;
    e = cudaLaunchKernelEx(&c, reserve_kernel, a);
  }
  if (e != cudaSuccess) return report_error(DLS_ERR_CUDA, "kv_reserve: cuda=%s", cudaGetErrorString(e));
  return DLS_OK;
}
