// Blocks of a paged cache: forking, reserving (with copy on write), trimming and compacting
// the block table and its reference counts on the device, and copying blocks' rows.
//
// The state is a table [B][C] of pool blocks (-1: none) and a count of holders per block; a
// block is free when its count is 0, so the counts are the whole allocator: the free blocks of
// lowest id come out of a prefix sum over them, and results do not depend on thread order.
#include <algorithm>

#include "decode_common.cuh"

namespace mla {
namespace blocks {

constexpr int kBT = MLA_BLOCK_TOKENS;
constexpr int kThreads = 1024;        // the single-CTA kernels
constexpr int kTile = kThreads * 32;  // ids per step of a pass over the counts: a 32-bit word per thread
constexpr int kMaxBlocks = 1 << 24;   // 2^31 token rows, the most a cache may hold
constexpr int kShortRow = 8;          // columns a thread walks by itself; longer runs go to a warp

struct Table {
  const int32_t* in;
  int32_t* out;
  int32_t* refs;      // updated in place (the output counts)
  int32_t B, C, n_blocks;
  int32_t* status;
};

__device__ __forceinline__ void flag(int32_t* status, int32_t bit) { atomicOr(status + 1, bit); }

// A table entry's block, or -1 for none (an entry outside the pool counts as none).
__device__ __forceinline__ int entry(const Table& t, int32_t e) {
  if (e >= 0 && e < t.n_blocks) return e;
  if (e != -1) flag(t.status, MLA_DEVERR_BLOCK);
  return -1;
}

__device__ __forceinline__ bool length_ok(const Table& t, int L) { return L >= 0 && (long long)L <= (long long)t.C * kBT; }

// The pair that writes row r (the first i with dst[i] == r), or -1: none, or a pair to skip.
// Whole warp; flags what is skipped.
__device__ __forceinline__ int pair_of(const int32_t* __restrict__ src, const int32_t* __restrict__ dst, int n, int r,
                                       int rows, int32_t* status) {
  const int lane = threadIdx.x & 31;
  int first = INT_MAX, count = 0;
  for (int i = lane; i < n; i += 32)
    if (dst[i] == r) {
      first = min(first, i);
      ++count;
    }
  first = __reduce_min_sync(0xffffffffu, first);
  if (first == INT_MAX) return -1;
  count = __reduce_add_sync(0xffffffffu, count);
  const int s = src[first];
  bool bad = s < 0 || s >= rows;
  if (!bad && s != r) {   // a source that another pair rewrites
    bool written = false;
    for (int j = lane; j < n; j += 32) written |= dst[j] == s && src[j] != s;
    bad = __any_sync(0xffffffffu, written);
  }
  if ((bad || count > 1) && lane == 0) flag(status, MLA_DEVERR_ROW);
  return bad ? -1 : first;
}

// Destinations outside the table (no row looks for them); the whole grid takes part.
__device__ void check_rows(const int32_t* __restrict__ dst, int n, int rows, int32_t* status, int thread, int threads) {
  for (int i = thread; i < n; i += threads)
    if (dst[i] < 0 || dst[i] >= rows) flag(status, MLA_DEVERR_ROW);
}

// ------------------------------------------------------------------ clusters
// The bookkeeping kernels run as one cluster of 8 CTAs: enough threads for tables and counts
// of some hundred thousand entries, with a barrier in hardware between the phases (the counts
// are copied before any thread changes one, say), so that a call is a single launch.
constexpr int kCluster = 8;
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void copy_ints(int32_t* out, const int32_t* in, long long n, int thread, int threads) {
  if (out == in) return;
  if ((((uintptr_t)out | (uintptr_t)in) & 15) == 0) {
    const long long n4 = n / 4;
    for (long long i = thread; i < n4; i += threads)
      reinterpret_cast<int4*>(out)[i] = __ldg(reinterpret_cast<const int4*>(in) + i);
    for (long long i = 4 * n4 + thread; i < n; i += threads) out[i] = __ldg(in + i);
  } else {
    for (long long i = thread; i < n; i += threads) out[i] = __ldg(in + i);
  }
}

// ------------------------------------------------------------------ fork
// A warp per table row.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
fork_kernel(Table t, const int32_t* refs_in, const int32_t* __restrict__ src, const int32_t* __restrict__ dst, int n,
            const int32_t* __restrict__ seq_lens) {
  pdl_wait();
  pdl_trigger();
  const int thread = blockIdx.x * kThreads + threadIdx.x, lane = threadIdx.x & 31;
  copy_ints(t.refs, refs_in, t.n_blocks, thread, kCluster * kThreads);
  check_rows(dst, n, t.B, t.status, thread, kCluster * kThreads);
  cluster_sync();
  for (int r = thread / 32; r < t.B; r += kCluster * kThreads / 32) {
    int i = pair_of(src, dst, n, r, t.B, t.status), cols = 0, s = 0;
    if (i >= 0) {
      s = src[i];
      const int L = seq_lens[s];
      if (!length_ok(t, L)) {
        if (lane == 0) flag(t.status, MLA_DEVERR_SEQ_LEN);
        i = -1;
      }
      cols = (int)(((long long)L + kBT - 1) / kBT);
    }
    if (i < 0 && t.out == t.in) continue;
    const int32_t* row = t.in + (size_t)r * t.C;
    const int32_t* from = t.in + (size_t)s * t.C;
    int32_t* out = t.out + (size_t)r * t.C;
    for (int j = lane; j < t.C; j += 32) {
      int32_t now = row[j];
      if (i >= 0) {
        const int was = entry(t, now);
        now = j < cols ? entry(t, from[j]) : -1;
        if (was != now) {   // (a row cut to its own length keeps most of its blocks)
          if (was >= 0) atomicSub(t.refs + was, 1);
          if (now >= 0) atomicAdd(t.refs + now, 1);
        }
      }
      out[j] = now;
    }
  }
}

// ------------------------------------------------------------------ trim
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
trim_kernel(Table t, const int32_t* refs_in, const int32_t* __restrict__ seq_lens, int n_sink, int window) {
  pdl_wait();
  pdl_trigger();
  const int thread = blockIdx.x * kThreads + threadIdx.x;
  copy_ints(t.refs, refs_in, t.n_blocks, thread, kCluster * kThreads);
  cluster_sync();
  const int n = t.B * t.C;   // at most 2^30
  constexpr int kBatch = 8;  // entries and lengths in flight
  for (int i0 = thread; i0 < n; i0 += kBatch * kCluster * kThreads) {
    int32_t e[kBatch], len[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = min(i0 + k * kCluster * kThreads, n - 1);
      e[k] = t.in[i];
      len[k] = __ldg(seq_lens + i / t.C);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kCluster * kThreads;
      if (i >= n) break;
      const long long t0 = (long long)(i % t.C) * kBT, L = len[k];
      if (!length_ok(t, len[k])) {
        flag(t.status, MLA_DEVERR_SEQ_LEN);
      } else {
        const int id = entry(t, e[k]);
        const bool keep = t0 < min((long long)n_sink, L) || (window > 0 && t0 < L && t0 + kBT > L - window);
        if (!keep) {
          if (id >= 0) atomicSub(t.refs + id, 1);
          e[k] = -1;
        }
      }
      t.out[i] = e[k];
    }
  }
}

// ------------------------------------------------------------------ passes over the counts
// Bit i of the returned word: `pick(count)` of id = base + 32 * threadIdx.x + i (false past
// the pool).  Warp w reads its 1024 ids in 32 coalesced loads; lane k keeps the k-th ballot.
template <typename F>
__device__ __forceinline__ uint32_t count_word(const int32_t* refs, int n_blocks, int base, F pick) {
  const int lane = threadIdx.x & 31, w0 = base + (threadIdx.x >> 5) * 1024;
  uint32_t word = 0;
  if (w0 >= n_blocks) return 0;
#pragma unroll 1
  for (int k0 = 0; k0 < 32 && w0 + 32 * k0 < n_blocks; k0 += 16) {
    int32_t c[16];   // 16 loads in flight
#pragma unroll
    for (int k = 0; k < 16; ++k) c[k] = __ldcg(refs + min(w0 + 32 * (k0 + k) + lane, n_blocks - 1));
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const uint32_t m = __ballot_sync(0xffffffffu, w0 + 32 * (k0 + k) + lane < n_blocks && pick(c[k]));
      if (lane == k0 + k) word = m;
    }
  }
  return word;
}

// Writes the ids of `word`'s set bits to list[first ...], those below `limit` only.
__device__ __forceinline__ void list_bits(uint32_t word, int id0, int32_t* list, int first, int limit) {
  while (word && first < limit) {
    list[first++] = id0 + __ffs(word) - 1;
    word &= word - 1;
  }
}

// ------------------------------------------------------------------ reserve
struct ReserveWs {
  int32_t* need;    // [B] new blocks of earlier rows
  int32_t* copy;    // [B] index of the row's copy in the list, -1: none
  int32_t* writers; // [n_blocks] rows that write into a shared block ...
  int32_t* last;    // [n_blocks] ... and the last of them (valid at shared blocks only; more than kThreads rows)
  int32_t* free_ids;  // [n_blocks]
  int32_t* given_up;  // [n_blocks] the block that the k-th new one replaces, -1: none
};
constexpr int kSharedIds = 4096;   // new ids kept in shared memory (more of them: in the workspace)

// One row: its columns [c0, c1) that tokens [L, N) start, and the shared block that they write
// into (-1: none).  A row with bad lengths is an empty one.
struct Row {
  int L, c0, c1, shared;
};
__device__ __forceinline__ Row row_of(const Table& t, const int32_t* refs, const int32_t* seq_lens,
                                      const int32_t* new_lens, int b, bool report) {
  Row r{seq_lens[b], 0, 0, -1};
  const int N = new_lens[b];
  if (!length_ok(t, r.L) || !length_ok(t, N) || N < r.L) {
    if (report) flag(t.status, MLA_DEVERR_SEQ_LEN);
    r.L = 0;
    return r;
  }
  r.c0 = (int)(((long long)r.L + kBT - 1) / kBT);
  r.c1 = (int)(((long long)N + kBT - 1) / kBT);
  if (N > r.L && r.L % kBT) {
    const int32_t e = t.in[(size_t)b * t.C + r.L / kBT];
    if (e < 0 || e >= t.n_blocks) {
      if (report) flag(t.status, MLA_DEVERR_BLOCK);
    } else if (refs[e] > 1) {
      r.shared = e;
    }
  }
  return r;
}

// A column that tokens start gets a new block where it has none, and where others hold its block
// too: a sequence that went back to a shorter length still names the blocks behind it, and what
// it writes there must not reach a fork's.
__device__ __forceinline__ bool held_too(const int32_t* refs, int e) { return __ldcg(refs + e) > 1; }

// Latency bound (5 to 6 us on 16 to 160 rows, 11 us with 65536 blocks).  CTA 0 decides while the
// others copy the table and the counts (calls that are not in place); after the cluster's barrier
// CTA 0 writes what changes.  Decisions read the input only.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
reserve_kernel(Table t, const int32_t* refs_in, const int32_t* __restrict__ seq_lens,
               const int32_t* __restrict__ new_lens, ReserveWs ws, int32_t* copies) {
  __shared__ int s_warp[32];
  __shared__ __align__(16) int32_t s_ids[kSharedIds];   // the writers' shared blocks, then the new ids
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x != 0) {
    const int thread = (blockIdx.x - 1) * kThreads + tid, threads = (kCluster - 1) * kThreads;
    copy_ints(t.refs, refs_in, t.n_blocks, thread, threads);
    copy_ints(t.out, t.in, (long long)t.B * t.C, thread, threads);
    cluster_sync();
    return;
  }
  // the first kThreads rows stay in registers, one per thread
  Row mine{0, 0, 0, -1};
  if (tid < t.B) mine = row_of(t, refs_in, seq_lens, new_lens, tid, true);
  auto row = [&](int b) { return b == tid ? mine : row_of(t, refs_in, seq_lens, new_lens, b, false); };
  // 1. A writer of a shared block copies while another holder is left: every writer when there
  // are other holders, else all but the last one.
  bool my_copy = false;
  if (t.B <= kThreads) {   // compared in shared memory
    s_ids[tid] = mine.shared;
    __syncthreads();
    if (mine.shared >= 0) {
      int writers = 0, later = 0;
      for (int j = 0; j < t.B; j += 4) {   // entries past B are -1
        const int4 v = *reinterpret_cast<const int4*>(s_ids + j);
        const int w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          writers += w[k] == mine.shared;
          later += w[k] == mine.shared && j + k > tid;
        }
      }
      my_copy = refs_in[mine.shared] > writers || later > 0;
    }
  } else {                 // counted in the workspace
    for (int b = tid; b < t.B; b += kThreads) {
      const Row r = b == tid ? mine : row_of(t, refs_in, seq_lens, new_lens, b, true);
      if (r.shared >= 0) { ws.writers[r.shared] = 0; ws.last[r.shared] = -1; }
    }
    __syncthreads();
    for (int b = tid; b < t.B; b += kThreads) {
      const Row r = row(b);
      if (r.shared >= 0) { atomicAdd(ws.writers + r.shared, 1); atomicMax(ws.last + r.shared, b); }
    }
  }
  __syncthreads();
  auto copies_block = [&](const Row& r, int b) {
    if (t.B <= kThreads) return my_copy;
    return r.shared >= 0 && (refs_in[r.shared] > __ldcg(ws.writers + r.shared) || __ldcg(ws.last + r.shared) != b);
  };
  // 2. new blocks per row (long runs of columns: a warp per row), then their prefix sums
  bool any_long = false, any_back = false;   // back: some column's block is held by others
  auto wants = [&](int b, int j) {
    const int e = entry(t, t.in[(size_t)b * t.C + j]);
    const bool back = e >= 0 && held_too(refs_in, e);
    any_back |= back;
    return e < 0 || back ? 1 : 0;
  };
  for (int b = tid; b < t.B; b += kThreads) {
    const Row r = row(b);
    int need = copies_block(r, b) ? 1 : 0;
    ws.copy[b] = need;
    if (r.c1 - r.c0 <= kShortRow)
      for (int j = r.c0; j < r.c1; ++j) need += wants(b, j);
    else
      any_long = true;
    ws.need[b] = need;
  }
  if (__syncthreads_or(any_long || any_back)) {   // (neither in a step of single tokens)
    for (int b = warp; b < t.B; b += kThreads / 32) {
      const Row r = row_of(t, refs_in, seq_lens, new_lens, b, false);
      if (r.c1 - r.c0 <= kShortRow) continue;
      int n = 0;
      for (int j = r.c0 + lane; j < r.c1; j += 32) n += wants(b, j);
      n = __reduce_add_sync(0xffffffffu, n);
      if (lane == 0) ws.need[b] += n;
    }
    any_long = __syncthreads_or(any_long);
    any_back = __syncthreads_or(any_back);
  }
  int total = 0, n_copies = 0;
  for (int base = 0; base < t.B; base += kThreads) {
    const int b = base + tid;
    const int need = b < t.B ? ws.need[b] : 0, cp = b < t.B ? ws.copy[b] : 0;
    int tot_n, tot_c;
    const int ex_n = block_exscan(need, &tot_n, s_warp), ex_c = block_exscan(cp, &tot_c, s_warp);
    if (b < t.B) {
      ws.need[b] = total + ex_n;
      ws.copy[b] = cp ? n_copies + ex_c : -1;
    }
    total += tot_n;
    n_copies += tot_c;
  }
  // 3. the free blocks of lowest id
  const int want = min(total, t.n_blocks);
  int32_t* ids = want <= kSharedIds ? s_ids : ws.free_ids;
  int n_free = 0;
  for (int base = 0; base < t.n_blocks; base += kTile) {
    const uint32_t word = count_word(refs_in, t.n_blocks, base, [](int32_t c) { return c <= 0; });
    int tot;
    const int ex = block_exscan(__popc(word), &tot, s_warp);
    list_bits(word, base + 32 * tid, ids, n_free + ex, want);
    n_free += tot;
  }
  const bool ok = total <= n_free;
  if (tid == 0) {
    t.status[0] = ok ? n_copies : 0;
    t.status[2] = t.n_blocks - n_free + (ok ? total : 0);
    t.status[3] = ok ? total : 0;
    if (!ok) flag(t.status, MLA_DEVERR_POOL);
  }
  cluster_sync();   // the output holds the input's values, and the ids are listed
  if (!ok) return;
  // 4. table and copy list, and the new blocks' counts.  Rows are independent: row b's new ids are
  // ids[need[b] ...].  Where counts decide (any_back) none changes yet (but a new block's, which was
  // 0 at most): what is given up is noted and loses its holders after the last row.
  for (int b = tid; b < t.B; b += kThreads) {
    // (not row_of: copy[] and need[] carry what was decided)
    int at = ws.need[b];
    const int L = seq_lens[b], N = new_lens[b];
    auto take = [&](int32_t* e) {
      const int old = *e, id = ids[at];
      if (any_back) ws.given_up[at] = old >= 0 && old < t.n_blocks ? old : -1;
      ++at;
      *e = id;
      t.refs[id] = 1;
      return id;
    };
    if (ws.copy[b] >= 0) {
      int32_t* e = t.out + (size_t)b * t.C + L / kBT;
      int32_t* c = copies + 3 * (size_t)ws.copy[b];
      c[0] = *e;
      if (!any_back) atomicSub(t.refs + *e, 1);
      c[1] = take(e);
      c[2] = L % kBT;
    }
    if (!length_ok(t, L) || !length_ok(t, N) || N < L) continue;
    const int c0 = (int)(((long long)L + kBT - 1) / kBT), c1 = (int)(((long long)N + kBT - 1) / kBT);
    if (c1 - c0 > kShortRow) continue;
    for (int j = c0; j < c1; ++j) {
      int32_t* e = t.out + (size_t)b * t.C + j;
      if (*e < 0 || *e >= t.n_blocks || (any_back && held_too(t.refs, *e))) take(e);
    }
  }
  for (int b = warp; any_long && b < t.B; b += kThreads / 32) {
    const int L = seq_lens[b], N = new_lens[b];
    const int c0 = (int)(((long long)L + kBT - 1) / kBT), c1 = (int)(((long long)N + kBT - 1) / kBT);
    if (c1 - c0 <= kShortRow || !length_ok(t, L) || !length_ok(t, N)) continue;
    int at = ws.need[b] + (ws.copy[b] >= 0 ? 1 : 0);
    for (int j0 = c0; j0 < c1; j0 += 32) {
      const int j = j0 + lane;
      int32_t* e = t.out + (size_t)b * t.C + min(j, c1 - 1);
      const int old = *e;
      const bool none = old < 0 || old >= t.n_blocks, want = j < c1 && (none || (any_back && held_too(t.refs, old)));
      const uint32_t m = __ballot_sync(0xffffffffu, want);
      if (want) {
        const int k = at + __popc(m & ((1u << lane) - 1)), id = ids[k];
        if (any_back) ws.given_up[k] = none ? -1 : old;
        *e = id;
        t.refs[id] = 1;
      }
      at += __popc(m);
    }
  }
  // 5. what was given up loses a holder (and is free where every holder went back)
  if (!any_back) return;
  __syncthreads();
  for (int k = tid; k < total; k += kThreads) {
    const int old = ws.given_up[k];
    if (old >= 0 && atomicSub(t.refs + old, 1) == 1) atomicSub(t.status + 2, 1);
  }
}

// ------------------------------------------------------------------ compact
struct CompactWs {
  int32_t* remap;   // [n_blocks] new id of every block in use
  int32_t* holes;   // [n_blocks / 2] free ids below the number of blocks in use, ascending
  int32_t* movers;  // [n_blocks / 2] ids in use from there on, ascending
};

// CTA 0 lists the moves while the others copy the counts (a call that is not in place) and set
// every other block's new id; after the cluster's barrier CTA 0 moves the counts, and after
// another one the table entries follow their blocks.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
compact_kernel(Table t, const int32_t* refs_in, CompactWs ws, int32_t* copies) {
  __shared__ int s_warp[32];
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  int n_movers = 0;
  if (blockIdx.x != 0) {
    const int thread = (blockIdx.x - 1) * kThreads + tid, threads = (kCluster - 1) * kThreads;
    copy_ints(t.refs, refs_in, t.n_blocks, thread, threads);
    for (int i = thread; i < t.n_blocks; i += threads) ws.remap[i] = i;
  } else {
    auto in_use = [](int32_t c) { return c > 0; };
    const uint32_t first = count_word(refs_in, t.n_blocks, 0, in_use);
    int live = 0;
    for (int base = 0; base < t.n_blocks; base += kTile) {
      int tot;
      block_exscan(__popc(base ? count_word(refs_in, t.n_blocks, base, in_use) : first), &tot, s_warp);
      live += tot;
    }
    int n_holes = 0;
    for (int base = 0; base < t.n_blocks; base += kTile) {
      const uint32_t used = base ? count_word(refs_in, t.n_blocks, base, in_use) : first;
      const int id0 = base + 32 * tid;
      // bits below the border: ids id0 .. live - 1 (all of them in the pool)
      const int below = max(0, min(32, live - id0));
      const uint32_t lo = below == 32 ? 0xffffffffu : (1u << below) - 1u;
      const uint32_t hole = ~used & lo, mover = used & ~lo;
      int tot_h, tot_m;
      const int ex_h = block_exscan(__popc(hole), &tot_h, s_warp), ex_m = block_exscan(__popc(mover), &tot_m, s_warp);
      list_bits(hole, id0, ws.holes, n_holes + ex_h, t.n_blocks / 2);
      list_bits(mover, id0, ws.movers, n_movers + ex_m, t.n_blocks / 2);
      n_holes += tot_h;
      n_movers += tot_m;
    }
    if (tid == 0) {   // as many blocks in use behind the border as free ones before it
      t.status[0] = n_movers;
      t.status[2] = live;
      t.status[3] = n_movers;
    }
  }
  cluster_sync();
  if (blockIdx.x == 0) {
    for (int k = tid; k < n_movers; k += kThreads) {
      const int from = ws.movers[k], to = ws.holes[k];
      ws.remap[from] = to;
      t.refs[to] = __ldcg(t.refs + from);
      t.refs[from] = 0;
      copies[3 * (size_t)k] = from; copies[3 * (size_t)k + 1] = to; copies[3 * (size_t)k + 2] = kBT;
    }
  }
  cluster_sync();
  const int n = t.B * t.C;   // at most 2^30
  for (int i = blockIdx.x * kThreads + tid; i < n; i += kCluster * kThreads) {
    const int id = entry(t, t.in[i]);
    t.out[i] = id >= 0 ? __ldcg(ws.remap + id) : -1;
  }
}

// ------------------------------------------------------------------ copies
struct CopyArgs {
  const int32_t* copies;
  int32_t max_copies, n_blocks;
  int32_t* status;
  char* base[3];        // c_kv, c_scales, k_rope (null: none)
  uint32_t row[3];      // bytes per token row
  uint32_t chunks[3];   // steps per block
};
constexpr int kCopyThreads = 256, kCopyCtas = 8;             // threads, CTAs per SM
constexpr int kCopyVec = 4;                                  // 16-byte loads a thread has in flight
constexpr uint32_t kChunk = kCopyThreads * kCopyVec * 16;    // bytes per CTA step: 16 KB

// Work items: (copy, array, chunk); a block's rows are contiguous in each array.  Bound by HBM:
// 134 MB moved in 47 us, 88% of the measured copy rate
// (32 KB steps of 4 CTAs 48 us; one warp with 16 KB bulk copies through a ring in shared memory
// 46 to 49, depending on how much is in flight).
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(CopyArgs a) {
  pdl_wait();
  pdl_trigger();
  const int n = min(__ldcg(a.status), a.max_copies);
  const uint32_t per = a.chunks[0] + a.chunks[1] + a.chunks[2];
  const long long items = (long long)n * per;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int32_t* c = a.copies + 3 * (it / per);
    uint32_t chunk = (uint32_t)(it % per);
    int k = 0;
    while (chunk >= a.chunks[k]) chunk -= a.chunks[k++];
    const int src = c[0], dst = c[1], rows = c[2];
    if (src < 0 || src >= a.n_blocks || dst < 0 || dst >= a.n_blocks || rows < 0 || rows > kBT) {
      if (threadIdx.x == 0) flag(a.status, MLA_DEVERR_BLOCK);
      continue;
    }
    const size_t block = (size_t)a.row[k] * kBT;
    const uint32_t bytes = a.row[k] * rows, o0 = chunk * kChunk;
    if (o0 >= bytes) continue;
    const uint32_t o1 = min(bytes, o0 + kChunk), v1 = o1 & ~15u;
    const char* s = a.base[k] + block * src;
    char* d = a.base[k] + block * dst;
    const uint32_t o = o0 + 16 * threadIdx.x;
    uint4 v[kCopyVec];
#pragma unroll
    for (int j = 0; j < kCopyVec; ++j)
      if (o + j * 16 * kCopyThreads < v1) v[j] = __ldcs(reinterpret_cast<const uint4*>(s + o + j * 16 * kCopyThreads));
#pragma unroll
    for (int j = 0; j < kCopyVec; ++j)
      if (o + j * 16 * kCopyThreads < v1) __stcs(reinterpret_cast<uint4*>(d + o + j * 16 * kCopyThreads), v[j]);
    // the end of the last row, where rows are not whole 16-byte units (fewer than 16 bytes)
    if (v1 + threadIdx.x < o1) d[v1 + threadIdx.x] = s[v1 + threadIdx.x];
  }
}

// ------------------------------------------------------------------ residual ring
// A CTA per ring.  With the lengths, slots that hold a token behind the source's length are
// empty in the destination: appends only raise a slot's position, so one of a later token would
// keep the sequence's own token out.
__global__ void __launch_bounds__(256) ring_kernel(mla_cache_t c, uint32_t row_bytes, const int32_t* __restrict__ src,
                                                   const int32_t* __restrict__ dst, int n,
                                                   const int32_t* __restrict__ seq_lens, int32_t* status) {
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x;
  if (r == 0) check_rows(dst, n, c.B, status, threadIdx.x, blockDim.x);
  __shared__ int s_pair;
  if (threadIdx.x < 32) {
    int i = pair_of(src, dst, n, r, c.B, status);
    if (i >= 0 && seq_lens && (unsigned)seq_lens[src[i]] > (unsigned)c.T_cap) {   // the fork skips the pair too
      if (threadIdx.x == 0) flag(status, MLA_DEVERR_SEQ_LEN);
      i = -1;
    }
    if (threadIdx.x == 0) s_pair = i;
  }
  __syncthreads();
  const int i = s_pair;
  if (i < 0) return;
  const int from = src[i], L = seq_lens ? seq_lens[from] : INT_MAX;
  // (a row that is cut while others copy from it: they see a position before or after, and
  // leave it out either way)
  for (int o = threadIdx.x; o < MLA_RESID_WINDOW; o += blockDim.x) {
    const int p = c.resid_pos[(size_t)from * MLA_RESID_WINDOW + o];
    c.resid_pos[(size_t)r * MLA_RESID_WINDOW + o] = p < L ? p : -1;
  }
  if (from == r) return;
  const size_t bytes = (size_t)row_bytes * MLA_RESID_WINDOW;   // a multiple of 16: 128 rows
  const uint4* s = reinterpret_cast<const uint4*>((const char*)c.c_resid + bytes * from);
  uint4* d = reinterpret_cast<uint4*>((char*)c.c_resid + bytes * r);
  for (size_t o = threadIdx.x; o < bytes / 16; o += blockDim.x) d[o] = s[o];
}

// ------------------------------------------------------------------ host side
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

// True when [a, a + n) and [b, b + n) share bytes without being the same range.
bool overlap(const void* a, const void* b, size_t n) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x != y && x < y + n && y < x + n;
}

bool sizes_ok(int32_t B, int32_t C, int32_t n_blocks) {
  return B > 0 && C > 0 && n_blocks > 0 && C <= kMaxBlocks && n_blocks <= kMaxBlocks && (long long)B * C <= (1 << 30);
}

mla_status_t check_table(const int32_t* table, const int32_t* refs, int32_t B, int32_t C, int32_t n_blocks,
                         const int32_t* table_out, const int32_t* refs_out, const int32_t* status) {
  if (!table || !refs || !table_out || !refs_out || !status || !sizes_ok(B, C, n_blocks)) return MLA_ERR_INVALID_ARG;
  if (!aligned4(table) || !aligned4(refs) || !aligned4(table_out) || !aligned4(refs_out) || !aligned4(status))
    return MLA_ERR_ALIGNMENT;
  if (overlap(table, table_out, (size_t)B * C * 4) || overlap(refs, refs_out, (size_t)n_blocks * 4))
    return MLA_ERR_INVALID_ARG;
  return MLA_OK;
}

mla_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA; }

// Workspace: two ints per row and four per block (reserve), two per block (compact).
size_t workspace_ints(int32_t B, int32_t n_blocks) { return 2 * (size_t)B + 4 * (size_t)n_blocks; }

}  // namespace blocks
}  // namespace mla

using namespace mla::blocks;

extern "C" {

size_t mla_blocks_workspace_bytes(int32_t B, int32_t n_cols, int32_t n_blocks) {
  return sizes_ok(B, n_cols, n_blocks) ? (workspace_ints(B, n_blocks) * 4 + 255) & ~(size_t)255 : 0;
}

mla_status_t mla_blocks_fork(const int32_t* table, const int32_t* refs, int32_t B, int32_t n_cols, int32_t n_blocks,
                             const int32_t* src, const int32_t* dst, int32_t n, const int32_t* seq_lens,
                             int32_t* table_out, int32_t* refs_out, int32_t* status, void* stream) {
  const mla_status_t st = check_table(table, refs, B, n_cols, n_blocks, table_out, refs_out, status);
  if (st != MLA_OK) return st;
  if (!src || !dst || !seq_lens || n <= 0) return MLA_ERR_INVALID_ARG;
  if (!aligned4(src) || !aligned4(dst) || !aligned4(seq_lens)) return MLA_ERR_ALIGNMENT;
  const cudaStream_t s = (cudaStream_t)stream;
  const Table t{table, table_out, refs_out, B, n_cols, n_blocks, status};
  return cuda_status(mla_launch_kernel(fork_kernel, dim3(kCluster), dim3(kThreads), 0, s, true, t, refs, src, dst, n, seq_lens));
}

mla_status_t mla_blocks_reserve(const int32_t* table, const int32_t* refs, int32_t B, int32_t n_cols, int32_t n_blocks,
                                const int32_t* seq_lens, const int32_t* new_lens, int32_t* table_out,
                                int32_t* refs_out, int32_t* copies, int32_t max_copies, int32_t* status,
                                void* workspace, size_t ws_bytes, void* stream) {
  const mla_status_t st = check_table(table, refs, B, n_cols, n_blocks, table_out, refs_out, status);
  if (st != MLA_OK) return st;
  if (!seq_lens || !new_lens || !copies || !workspace || max_copies < B) return MLA_ERR_INVALID_ARG;
  if (!aligned4(seq_lens) || !aligned4(new_lens) || !aligned4(copies) || ((uintptr_t)workspace & 15)) return MLA_ERR_ALIGNMENT;
  if (ws_bytes < mla_blocks_workspace_bytes(B, n_cols, n_blocks)) return MLA_ERR_WORKSPACE_TOO_SMALL;
  const cudaStream_t s = (cudaStream_t)stream;
  int32_t* w = (int32_t*)workspace;
  ReserveWs ws;
  ws.need = w; ws.copy = w + B;
  ws.writers = w + 2 * (size_t)B; ws.last = ws.writers + n_blocks; ws.free_ids = ws.last + n_blocks;
  ws.given_up = ws.free_ids + n_blocks;
  const Table t{table, table_out, refs_out, B, n_cols, n_blocks, status};
  return cuda_status(mla_launch_kernel(reserve_kernel, dim3(kCluster), dim3(kThreads), 0, s, true, t, refs, seq_lens,
                                       new_lens, ws, copies));
}

mla_status_t mla_blocks_trim(const int32_t* table, const int32_t* refs, int32_t B, int32_t n_cols, int32_t n_blocks,
                             const int32_t* seq_lens, int32_t n_sink, int32_t window, int32_t* table_out,
                             int32_t* refs_out, int32_t* status, void* stream) {
  const mla_status_t st = check_table(table, refs, B, n_cols, n_blocks, table_out, refs_out, status);
  if (st != MLA_OK) return st;
  if (!seq_lens || n_sink < 0 || window < 0) return MLA_ERR_INVALID_ARG;
  if (!aligned4(seq_lens)) return MLA_ERR_ALIGNMENT;
  const cudaStream_t s = (cudaStream_t)stream;
  const Table t{table, table_out, refs_out, B, n_cols, n_blocks, status};
  return cuda_status(mla_launch_kernel(trim_kernel, dim3(kCluster), dim3(kThreads), 0, s, true, t, refs, seq_lens, n_sink, window));
}

mla_status_t mla_blocks_compact(const int32_t* table, const int32_t* refs, int32_t B, int32_t n_cols, int32_t n_blocks,
                                int32_t* table_out, int32_t* refs_out, int32_t* copies, int32_t max_copies,
                                int32_t* status, void* workspace, size_t ws_bytes, void* stream) {
  const mla_status_t st = check_table(table, refs, B, n_cols, n_blocks, table_out, refs_out, status);
  if (st != MLA_OK) return st;
  if (!copies || !workspace || max_copies < n_blocks / 2) return MLA_ERR_INVALID_ARG;
  if (!aligned4(copies) || ((uintptr_t)workspace & 15)) return MLA_ERR_ALIGNMENT;
  if (ws_bytes < mla_blocks_workspace_bytes(B, n_cols, n_blocks)) return MLA_ERR_WORKSPACE_TOO_SMALL;
  const cudaStream_t s = (cudaStream_t)stream;
  int32_t* w = (int32_t*)workspace;
  CompactWs ws{w, w + n_blocks, w + n_blocks + n_blocks / 2};
  const Table t{table, table_out, refs_out, B, n_cols, n_blocks, status};
  return cuda_status(mla_launch_kernel(compact_kernel, dim3(kCluster), dim3(kThreads), 0, s, true, t, refs, ws, copies));
}

mla_status_t mla_blocks_copy(const mla_config_t* cfg, const mla_cache_t* cache, const int32_t* copies,
                             int32_t max_copies, int32_t* status, void* stream) {
  mla_status_t st = mla_validate_config(cfg);
  if (st != MLA_OK) return st;
  if ((st = mla_validate_cache(*cfg, cache)) != MLA_OK) return st;
  if (!cache->block_table || !copies || !status || max_copies <= 0) return MLA_ERR_INVALID_ARG;
  if (!aligned4(copies) || !aligned4(status)) return MLA_ERR_ALIGNMENT;
  const bool quant = mla_kind_quant(cfg->cache_kind);
  const uint32_t eb = cfg->dtype == MLA_F32 ? 4 : 2;
  CopyArgs a;
  a.copies = copies; a.max_copies = max_copies; a.n_blocks = cache->n_blocks; a.status = status;
  a.base[0] = (char*)cache->c_kv;
  a.row[0] = quant ? (uint32_t)(cfg->d_c * mla_quant_bits(cfg->cache_kind) / 8) : (uint32_t)cfg->d_c * eb;
  a.base[1] = quant ? (char*)cache->c_scales : nullptr;
  a.row[1] = quant ? (uint32_t)(cfg->d_c / 32 * 2) : 0;
  a.base[2] = cfg->r_pairs > 0 ? (char*)cache->k_rope : nullptr;
  a.row[2] = (uint32_t)(cfg->n_kv_heads * 2 * cfg->r_pairs) * eb;
  long long items = 0;   // no CTAs without work where the list is short
  for (int k = 0; k < 3; ++k) {
    a.chunks[k] = a.base[k] ? (a.row[k] * kBT + kChunk - 1) / kChunk : 0;
    items += (long long)a.chunks[k] * max_copies;
  }
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MLA_ERR_CUDA;
  return cuda_status(mla_launch_kernel(copy_kernel, dim3((unsigned)std::min<long long>(items, kCopyCtas * sms)), dim3(kCopyThreads), 0, (cudaStream_t)stream, true, a));
}

mla_status_t mla_ring_copy(const mla_config_t* cfg, const mla_cache_t* cache, const int32_t* src, const int32_t* dst,
                           int32_t n, const int32_t* seq_lens, int32_t* status, void* stream) {
  mla_status_t st = mla_validate_config(cfg);
  if (st != MLA_OK) return st;
  if ((st = mla_validate_cache(*cfg, cache)) != MLA_OK) return st;
  if (!cache->c_resid || !src || !dst || !status || n <= 0) return MLA_ERR_INVALID_ARG;
  if (!aligned4(src) || !aligned4(dst) || !aligned4(status) || !aligned4(seq_lens)) return MLA_ERR_ALIGNMENT;
  return cuda_status(mla_launch_kernel(ring_kernel, dim3(cache->B), dim3(256), 0, (cudaStream_t)stream, true, *cache,
                                       (uint32_t)cfg->d_c * 2, src, dst, n, seq_lens, status));
}

}  // extern "C"
