// tables.cu -- page tables and slot maps built on the device from request
// lengths.
//
// A batch is admitted (whole prompts) or stepped (a few rows a sequence) by
// the lengths alone: sequence b holds ctx_b rows and gets new_b more, packed
// one sequence after the other into a token buffer.  With ps rows to a page,
//   start_b   = new_0 + .. + new_{b-1}
//   entries   ceil(ctx_b / ps) .. ceil((ctx_b + new_b) / ps) - 1 of its table
//             row that are -1 pop the stack of free pages, in (b, entry) order
//   slot(start_b + i) = table[b][(ctx_b + i) / ps] * ps + (ctx_b + i) % ps
// Integer work of a few bytes a row (8 of slot, 4 of position), so what bounds
// it is latency: the prefix sums over the sequences, then one table read and
// one store a row.
//
// fused_kernel, one launch (out of place, up to kFusedBatch sequences and
// kFusedEntries table entries in use, which max_rows bounds): every CTA works out
// the same plan in shared memory -- lengths, prefix sums, the entries in use, the
// popped ids: four dependent loads -- and then writes its share of the table and
// of the slots, whose look-ups are all in shared memory.
// Else two launches.  tables_kernel: one thread-block cluster; CTA r owns a
// contiguous range of sequences (one warp per sequence), counts the entries
// that need a page, scans rows and counts over its range, reads the other
// CTAs' totals over distributed shared memory, and writes its table rows.
// slots_kernel: the whole device, one thread per pair of token rows (one
// 16-byte store of two slots), the row's sequence found by bisection of the
// starts, which sit in shared memory up to kStartsMax sequences.
// Measured: 32 prompts (results of 4.5 MB) 13.2 us in one launch (14.3 in two), a
// step of 256 sequences 7.4 us; both are launch, dependent loads and one round of
// stores, 0.3 TB/s at most.
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace tidar {

namespace cg = cooperative_groups;

namespace {

constexpr int kTThreads = 1024;
constexpr int kTWarps = kTThreads / 32;
constexpr int kTMaxCluster = 8;           // portable
constexpr int kFThreads = 512;
constexpr int kFWarps = kFThreads / 32;
constexpr int kFusedBatch = 1024;
constexpr int kFusedEntries = 16384;
constexpr int kTablesMaxBatch = 65536;
constexpr int kSThreads = 256;
constexpr int kStartsMax = 8192;

struct TablesArgs {
  int B, ps, num_pages, max_pages, max_rows, capacity;
  const int32_t* table_in;
  const int32_t* ctx;
  const int32_t* newl;
  const int32_t* free_pages;
  const int32_t* free_count;
  int32_t* table_out;
  int32_t* count_out;
  int32_t* starts;
  int64_t* slots;
  int32_t* positions;
  unsigned int* err;
};

// One owned sequence: rows it adds (0 when its lengths are invalid), the pages
// it needs (0 when it is skipped), both then replaced by exclusive sums.
struct TabRec {
  long long rows, need;
  int ok;
};

__global__ void __launch_bounds__(kTThreads) tables_kernel(TablesArgs a, int per) {
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  extern __shared__ __align__(16) unsigned char s_raw[];
  TabRec* rec = reinterpret_cast<TabRec*>(s_raw);
  __shared__ long long s_rows, s_need, w_rows[kTWarps], w_need[kTWarps];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int b0 = rank * per, nown = max(0, min(a.B, b0 + per) - b0);
  const int ps = a.ps;
  pdl_wait();
  pdl_trigger();

  const int count = *a.free_count;
  // 1. validate and count, one warp per sequence; the row is copied on the way
  //    (an update in place has nothing to copy: only the entries it needs are
  //    read), eight entries a lane in flight
  for (int i = wid; i < nown; i += kTWarps) {
    const int b = b0 + i;
    const int c = a.ctx[b], m = a.newl[b];
    const int32_t* src = a.table_in + (size_t)b * a.max_pages;
    int32_t* dst = a.table_out + (size_t)b * a.max_pages;
    const bool copy = src != dst;
    const bool len_ok = c >= 0 && m >= 0 && (long long)c + m <= (long long)a.max_pages * ps;
    if (!len_ok && lane == 0) raise_error(a.err, TIDAR_DEVERR_BAD_LEN);
    const bool rows = len_ok && m > 0;
    const int lo = rows ? c / ps : 0, first = rows ? (int)(((long long)c + ps - 1) / ps) : 0;
    const int last = rows ? (int)(((long long)c + m + ps - 1) / ps) : 0;
    int need = 0;
    bool bad = false;
    for (int e0 = copy ? 0 : lo; e0 < (copy ? a.max_pages : last); e0 += 256) {
      int id[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int e = e0 + 32 * u + lane;
        id[u] = e < (copy ? a.max_pages : last) ? src[e] : 0;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int e = e0 + 32 * u + lane;
        if (copy && e < a.max_pages) dst[e] = id[u];
        const bool in = e >= lo && e < last, want = in && e >= first && id[u] == -1;
        bad = bad || (in && !want && (id[u] < 0 || id[u] >= a.num_pages));
        need += __popc(__ballot_sync(0xffffffffu, want));
      }
    }
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
      if (bad) raise_error(a.err, TIDAR_DEVERR_BAD_PAGE);
      TabRec r;
      r.rows = m > 0 ? m : 0;
      r.ok = len_ok && !bad;
      r.need = r.ok ? need : 0;
      rec[i] = r;
    }
  }
  __syncthreads();
  // 2. exclusive sums over this CTA's range: a contiguous run per thread, then
  //    over the threads
  {
    const int run = (nown + kTThreads - 1) / kTThreads;
    const int i0 = min(nown, (int)threadIdx.x * run), i1 = min(nown, i0 + run);
    long long rows = 0, need = 0;
    for (int i = i0; i < i1; ++i) rows += rec[i].rows, need += rec[i].need;
    long long xr = rows, xn = need;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long yr = __shfl_up_sync(0xffffffffu, xr, o), yn = __shfl_up_sync(0xffffffffu, xn, o);
      if (lane >= o) xr += yr, xn += yn;
    }
    if (lane == 31) w_rows[wid] = xr, w_need[wid] = xn;
    __syncthreads();
    long long br = 0, bn = 0;
    for (int w = 0; w < wid; ++w) br += w_rows[w], bn += w_need[w];
    xr += br - rows;
    xn += bn - need;
    for (int i = i0; i < i1; ++i) {
      const long long r = rec[i].rows, q = rec[i].need;
      rec[i].rows = xr;
      rec[i].need = xn;
      xr += r;
      xn += q;
    }
    if (threadIdx.x == kTThreads - 1) s_rows = xr, s_need = xn;
  }
  // 3. bases across the cluster
  cl.sync();
  long long base_r = 0, all_r = 0, base_n = 0, all_n = 0;
  for (int r = 0; r < C; ++r) {
    const long long x = *cl.map_shared_rank(&s_rows, r), y = *cl.map_shared_rank(&s_need, r);
    if (r < rank) base_r += x, base_n += y;
    all_r += x;
    all_n += y;
  }
  const bool pool_ok = count >= 0 && count <= a.capacity && all_n <= count;
  const bool ok = pool_ok && all_r <= a.max_rows;
  cl.sync();                     // no CTA leaves, or rewrites the count, while a peer reads
  if (rank == 0 && threadIdx.x == 0) {
    if (!pool_ok) raise_error(a.err, TIDAR_DEVERR_POOL);
    if (all_r > a.max_rows) raise_error(a.err, TIDAR_DEVERR_BAD_COUNT);
    *a.count_out = ok ? count - (int)all_n : count;
    a.starts[a.B] = (int32_t)min(all_r, (long long)a.max_rows);
  }
  // 4. the starts (one past the token buffer is its end) and the popped pages
  for (int i = wid; i < nown; i += kTWarps) {
    const int b = b0 + i;
    const TabRec r = rec[i];
    if (lane == 0) a.starts[b] = (int32_t)min(base_r + r.rows, (long long)a.max_rows);
    const long long pages = (i + 1 < nown ? rec[i + 1].need : s_need) - r.need;
    if (!ok || pages == 0) continue;
    const int c = a.ctx[b], m = a.newl[b];
    const int32_t* src = a.table_in + (size_t)b * a.max_pages;
    int32_t* dst = a.table_out + (size_t)b * a.max_pages;
    const int first = (int)(((long long)c + ps - 1) / ps), last = (int)(((long long)c + m + ps - 1) / ps);
    long long pop = base_n + r.need;              // pages popped before this entry
    for (int e0 = first; e0 < last; e0 += 256) {
      int id[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int e = e0 + 32 * u + lane;
        id[u] = e < last ? src[e] : 0;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const bool want = id[u] == -1;            // 0 past the end
        const unsigned m32 = __ballot_sync(0xffffffffu, want);
        if (want) dst[e0 + 32 * u + lane] = a.free_pages[count - 1 - (pop + __popc(m32 & ((1u << lane) - 1u)))];
        pop += __popc(m32);
      }
    }
  }
}

__global__ void __launch_bounds__(kSThreads) slots_kernel(TablesArgs a) {
  extern __shared__ __align__(16) unsigned char s_raw[];
  int32_t* s_starts = reinterpret_cast<int32_t*>(s_raw);
  const bool local = a.B <= kStartsMax;
  pdl_wait();
  pdl_trigger();
  if (local) {
    for (int i = threadIdx.x; i <= a.B; i += kSThreads) s_starts[i] = a.starts[i];
    __syncthreads();
  }
  const int32_t* starts = local ? s_starts : a.starts;
  const int total = starts[a.B];
  bool bad = false;
  for (long long r0 = 2 * ((long long)blockIdx.x * kSThreads + threadIdx.x); r0 < a.max_rows;
       r0 += 2LL * gridDim.x * kSThreads) {
    long long slot[2] = {-1, -1};
    int pos[2] = {-1, -1};
    int b = 0;
    if (r0 < total) {
      // the last sequence that starts at or before the row (empty ones before it share its start)
      int lo = 0, hi = a.B - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (starts[mid] <= r0) lo = mid;
        else hi = mid - 1;
      }
      b = lo;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const long long r = r0 + u;
      if (r >= total) continue;
      while (b + 1 < a.B && starts[b + 1] <= r) ++b;
      const int c = a.ctx[b];
      const long long p = (long long)c + (r - starts[b]);
      if (c < 0 || p >= (long long)a.max_pages * a.ps) continue;       // reported by tables_kernel
      pos[u] = (int)p;
      const int page = a.table_out[(size_t)b * a.max_pages + p / a.ps];
      if (page < 0 || page >= a.num_pages) bad = true;
      else slot[u] = (long long)page * a.ps + p % a.ps;
    }
    if (r0 + 1 < a.max_rows) {
      *reinterpret_cast<longlong2*>(a.slots + r0) = make_longlong2(slot[0], slot[1]);
      if (a.positions) *reinterpret_cast<int2*>(a.positions + r0) = make_int2(pos[0], pos[1]);
    } else {
      a.slots[r0] = slot[0];
      if (a.positions) a.positions[r0] = pos[0];
    }
  }
  if (bad) raise_error(a.err, TIDAR_DEVERR_BAD_PAGE);
}

// Inclusive sum of one value a thread over the block (kFThreads threads); total in
// `total`.  ws: kFWarps values of shared memory, free again after the next barrier.
__device__ __forceinline__ long long block_scan(long long v, long long* ws, long long& total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) ws[wid] = v;
  __syncthreads();
  long long before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kFWarps; ++w) {
    const long long x = ws[w];
    if (w < wid) before += x;
    total += x;
  }
  __syncthreads();
  return v + before;
}

// Index in lo .. hi of the last of non-decreasing values that is <= x
// (values[lo] <= x).
__device__ __forceinline__ int last_at_most(const int* values, int lo, int hi, int x) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (values[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Shared memory: [B] first entry in use, [B] first entry that may be popped (-1:
// the sequence is skipped), [B + 1] offsets of the sequences' entries, [B + 1]
// row starts, [B] ctx, a word per 32 entries (which of them need a page) and the
// number of those before it, then the entries.
__global__ void __launch_bounds__(kFThreads) fused_kernel(TablesArgs a, int entry_cap) {
  extern __shared__ __align__(16) unsigned char s_raw[];
  __shared__ long long ws[kFWarps];
  int* s_lo = reinterpret_cast<int*>(s_raw);
  int* s_first = s_lo + a.B;
  int* s_off = s_first + a.B;
  int* s_start = s_off + a.B + 1;
  int* s_ctx = s_start + a.B + 1;
  const int words = (entry_cap + 31) / 32;
  unsigned* s_mask = reinterpret_cast<unsigned*>(s_ctx + a.B);
  int* s_pre = reinterpret_cast<int*>(s_mask + words);
  int* s_ent = s_pre + words;
  __shared__ int s_bad;
  const int lps = 31 - __clz(a.ps), t = threadIdx.x;
  const bool lead = blockIdx.x == 0;
  pdl_wait();
  pdl_trigger();
  const int count = *a.free_count, lane = t & 31;
  if (t == 0) s_bad = 0;
  // 1. lengths: rows and entries in use of up to two sequences a thread
  constexpr int kPer = kFusedBatch / kFThreads;
  long long rows[kPer], used[kPer], rsum = 0, usum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = t * kPer + i;
    rows[i] = used[i] = 0;
    if (b < a.B) {
      const int c = a.ctx[b], m = a.newl[b];
      const bool ok = c >= 0 && m >= 0 && (long long)c + m <= (long long)a.max_pages << lps;
      if (!ok && lead) raise_error(a.err, TIDAR_DEVERR_BAD_LEN);
      rows[i] = m > 0 ? m : 0;
      const int lo = ok ? c >> lps : 0, last = ok && m > 0 ? (int)(((long long)c + m + a.ps - 1) >> lps) : lo;
      used[i] = last - lo;
      s_lo[b] = lo;
      s_first[b] = ok ? (int)(((long long)c + a.ps - 1) >> lps) : -1;
      s_ctx[b] = c;
    }
    rsum += rows[i];
    usum += used[i];
  }
  long long all_r, all_u;
  long long r0 = block_scan(rsum, ws, all_r) - rsum, u0 = block_scan(usum, ws, all_u) - usum;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = t * kPer + i;
    if (b < a.B) {
      s_start[b] = (int)min(r0, (long long)a.max_rows);
      s_off[b] = (int)min(u0, (long long)entry_cap);
    }
    r0 += rows[i];
    u0 += used[i];
  }
  const bool fits = all_r <= a.max_rows;          // then all_u <= entry_cap
  const int total = (int)min(all_r, (long long)a.max_rows), ents = (int)min(all_u, (long long)entry_cap);
  if (t == 0) s_start[a.B] = total, s_off[a.B] = ents;
  __syncthreads();
  // 2. the entries in use, and which need a page; a bad one skips its sequence
  const int rounds = (ents + kFThreads - 1) / kFThreads;
  constexpr int kU = 4;                                    // rounds whose loads are in flight together
  for (int j0 = 0; j0 < rounds; j0 += kU) {
    int seq[kU], at[kU], id[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int e = (j0 + u) * kFThreads + t;
      id[u] = 0;
      if (e < ents) {
        seq[u] = last_at_most(s_off, 0, a.B - 1, e);
        at[u] = s_lo[seq[u]] + e - s_off[seq[u]];
        id[u] = a.table_in[(size_t)seq[u] * a.max_pages + at[u]];
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int e = (j0 + u) * kFThreads + t;
      bool want = false;
      if (e < ents) {
        s_ent[e] = id[u];
        want = id[u] == -1 && at[u] >= s_first[seq[u]];
        if (!want && (id[u] < 0 || id[u] >= a.num_pages)) {
          s_first[seq[u]] = 0x7fffffff;                    // every thread that writes it writes this
          s_bad = 1;
          if (lead) raise_error(a.err, TIDAR_DEVERR_BAD_PAGE);
        }
      }
      const unsigned m = __ballot_sync(0xffffffffu, want);
      if (lane == 0 && e < ents) s_mask[e >> 5] = m;
    }
  }
  __syncthreads();
  if (s_bad) {                                             // the skipped sequences' entries need none
    for (int j = 0; j < rounds; ++j) {
      const int e = j * kFThreads + t;
      bool want = false;
      if (e < ents) {
        const int b = last_at_most(s_off, 0, a.B - 1, e);
        want = s_ent[e] == -1 && s_lo[b] + e - s_off[b] >= s_first[b];
      }
      const unsigned m = __ballot_sync(0xffffffffu, want);
      if (lane == 0 && e < ents) s_mask[e >> 5] = m;
    }
    __syncthreads();
  }
  // 3. rank of every entry that needs a page, then the page
  const int nw = (ents + 31) / 32;
  static_assert(kFusedEntries / 32 <= kFThreads, "one word a thread");
  const int mine = t < nw ? __popc(s_mask[t]) : 0;
  long long all_n;
  const long long before = block_scan(mine, ws, all_n) - mine;
  if (t < nw) s_pre[t] = (int)before;
  __syncthreads();
  const bool pool_ok = count >= 0 && count <= a.capacity && all_n <= count, ok = pool_ok && fits;
  if (ok) {
#pragma unroll 4
    for (int e = t; e < ents; e += kFThreads) {
      const unsigned m = s_mask[e >> 5];
      if ((m >> lane) & 1u) s_ent[e] = a.free_pages[count - 1 - (s_pre[e >> 5] + __popc(m & ((1u << lane) - 1u)))];
    }
  }
  if (lead) {
    if (t == 0) {
      if (!pool_ok) raise_error(a.err, TIDAR_DEVERR_POOL);
      if (!fits) raise_error(a.err, TIDAR_DEVERR_BAD_COUNT);
      *a.count_out = ok ? count - (int)all_n : count;
    }
    for (int b = t; b <= a.B; b += kFThreads) a.starts[b] = s_start[b];
  }
  __syncthreads();
  // 4. this CTA's share of the table ...
  const int gt = blockIdx.x * kFThreads + t, gn = gridDim.x * kFThreads;
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    const int lo = s_lo[b], off = s_off[b], n = s_off[b + 1] - off;
    const size_t row = (size_t)b * a.max_pages;
    for (int e = t; e < a.max_pages; e += kFThreads)
      a.table_out[row + e] = e >= lo && e - lo < n ? s_ent[off + e - lo] : a.table_in[row + e];
  }
  // ... and of the slots, two rows a thread
  bool bad = false;
  for (long long rw = 2LL * (gt - lane); rw < a.max_rows; rw += 2LL * gn) {
    // the warp's 64 rows lie on sequences b0 .. b1, mostly one
    int b = 0;
    if (rw < total) {
      const int b0 = last_at_most(s_start, 0, a.B - 1, (int)rw);
      const int end = (int)min(rw + 63, (long long)total - 1);
      const int b1 = s_start[b0 + 1] > end ? b0 : last_at_most(s_start, b0, a.B - 1, end);
      b = b0 == b1 ? b0 : last_at_most(s_start, b0, b1, (int)min(rw + 2 * lane, (long long)end));
    }
    const long long r2 = rw + 2 * lane;
    if (r2 >= a.max_rows) continue;
    long long slot[2] = {-1, -1};
    int pos[2] = {-1, -1};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const long long r = r2 + u;
      if (r >= total) continue;
      while (b + 1 < a.B && s_start[b + 1] <= r) ++b;
      const int c = s_ctx[b];
      const long long p = (long long)c + (r - s_start[b]);
      if (c < 0 || p >= (long long)a.max_pages << lps) continue;
      pos[u] = (int)p;
      const int e = (int)(p >> lps) - s_lo[b];
      const int page = e < s_off[b + 1] - s_off[b] ? s_ent[s_off[b] + e] : a.table_in[(size_t)b * a.max_pages + (p >> lps)];
      if (page < 0 || page >= a.num_pages) bad = true;
      else slot[u] = ((long long)page << lps) + (p & (a.ps - 1));
    }
    if (r2 + 1 < a.max_rows) {
      *reinterpret_cast<longlong2*>(a.slots + r2) = make_longlong2(slot[0], slot[1]);
      if (a.positions) *reinterpret_cast<int2*>(a.positions + r2) = make_int2(pos[0], pos[1]);
    } else {
      a.slots[r2] = slot[0];
      if (a.positions) a.positions[r2] = pos[0];
    }
  }
  if (bad) raise_error(a.err, TIDAR_DEVERR_BAD_PAGE);
}

// Shared memory of a call, in bytes, and the most that any call takes.
constexpr size_t fused_smem(long long B, long long entries) {
  return (5 * (size_t)B + 2 + (size_t)entries + 2 * (((size_t)entries + 31) / 32)) * sizeof(int);
}
constexpr size_t tables_smem(int per) { return (size_t)per * sizeof(TabRec); }
constexpr size_t kFusedSmemMax = fused_smem(kFusedBatch, kFusedEntries);
constexpr size_t kTablesSmemMax = tables_smem(kTablesMaxBatch / kTMaxCluster);
static_assert(kFusedSmemMax + 1024 <= 232448 && kTablesSmemMax + 1024 <= 232448, "shared memory budget");

// A kernel's opt-in is the function's, shared by all host threads and captured
// calls: set to the most once per device, never to one call's size.
cudaError_t smem_attr() {
  static bool set[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorNotSupported;
  if (!set[dev]) {
    e = cudaFuncSetAttribute(fused_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kFusedSmemMax);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTablesSmemMax);
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  return cudaSuccess;
}

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace tidar

extern "C" tidar_status tidar_build_tables(const tidar_tables_desc* d, const int32_t* page_table,
                                           const int32_t* ctx_lens, const int32_t* new_lens,
                                           const tidar_page_pool* pool, int32_t* page_table_out,
                                           int32_t* free_count_out, int32_t* row_starts, int64_t* slots,
                                           int32_t* positions, tidar_stream_t stream) {
  using namespace tidar;
  if (!d) return TIDAR_ERR_INVALID_ARG;
  if (d->batch < 0 || d->max_pages_per_seq <= 0 || d->num_pages <= 0 || d->max_rows < 0 || d->page_size <= 0)
    return TIDAR_ERR_INVALID_ARG;
  if (d->page_size != 16 && d->page_size != 32 && d->page_size != 64 && d->page_size != 128)
    return TIDAR_ERR_UNSUPPORTED;
  if (d->batch > kTablesMaxBatch || (long long)d->max_pages_per_seq * d->page_size > 0x7fffffffLL)
    return TIDAR_ERR_UNSUPPORTED;
  if (d->batch == 0) return TIDAR_OK;
  if (!page_table || !ctx_lens || !new_lens || !page_table_out || !free_count_out || !row_starts ||
      (d->max_rows > 0 && !slots))
    return TIDAR_ERR_INVALID_ARG;
  if (!pool || !pool->free_count || pool->capacity < 0 || (pool->capacity > 0 && !pool->free_pages))
    return TIDAR_ERR_INVALID_ARG;
  if (!aligned(slots, 16) || !aligned(positions, 8)) return TIDAR_ERR_INVALID_ARG;
  TablesArgs a{};
  a.B = d->batch; a.ps = d->page_size; a.num_pages = d->num_pages; a.max_pages = d->max_pages_per_seq;
  a.max_rows = d->max_rows; a.capacity = pool->capacity;
  a.table_in = page_table; a.ctx = ctx_lens; a.newl = new_lens; a.free_pages = pool->free_pages;
  a.free_count = pool->free_count; a.table_out = page_table_out; a.count_out = free_count_out;
  a.starts = row_starts; a.slots = slots; a.positions = positions;
  const tidar_status st = error_word_status(&a.err);
  if (st != TIDAR_OK) return st;
  if (const cudaError_t e = smem_attr(); e != cudaSuccess) return cuda_status(e);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // Entries in use: a sequence of m > 0 rows uses at most m / ps + 2.  In place the
  // CTAs of one launch would read what others have already written.
  const long long entries = a.max_rows / a.ps + 2LL * a.B;
  if (a.B <= kFusedBatch && entries <= kFusedEntries && a.table_in != a.table_out && a.free_count != a.count_out) {
    const size_t smem = fused_smem(a.B, entries);
    // a CTA per 1024 rows or per table row, up to one an SM
    const long long want = std::max<long long>(((long long)a.max_rows + 2 * kFThreads - 1) / (2 * kFThreads), a.B);
    const cudaError_t e = launch_pdl(fused_kernel, dim3((unsigned)std::min<long long>(std::max<long long>(want, 1), 148)),
                                     kFThreads, smem, s, a, (int)entries);
    return e == cudaSuccess ? TIDAR_OK : cuda_status(e);
  }
  // one warp per sequence, up to the portable cluster
  const int C = std::min(kTMaxCluster, (a.B + kTWarps - 1) / kTWarps);
  const int per = (a.B + C - 1) / C;
  cudaError_t e = launch_cluster(tables_kernel, C, 1, kTThreads, tables_smem(per), s, a, per);
  if (e != cudaSuccess) return cuda_status(e);
  if (a.max_rows > 0) {
    const long long pairs = ((long long)a.max_rows + 1) / 2;
    const int grid = (int)std::min<long long>((pairs + kSThreads - 1) / kSThreads, 148 * 8);
    e = launch_pdl(slots_kernel, dim3(grid), kSThreads, a.B <= kStartsMax ? (size_t)(a.B + 1) * 4 : 0, s, a);
    if (e != cudaSuccess) return cuda_status(e);
  }
  return TIDAR_OK;
}
