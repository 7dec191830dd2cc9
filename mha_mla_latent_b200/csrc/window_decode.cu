// Windowed decode attention over the latent cache (split over the visible tokens), for up to 32
// query heads: one new query per sequence against the sinks and the newest tokens.
//
// Paper notes "MHA2MLA" (ACL 2025), §关键设计: the absorbed query of every head scores against
// the one shared latent, the partial-RoPE term is added, the softmax weights the latent.
// Tokens are the rows of both products, so a softmax thread owns a token and holds one score
// per head: its mask is one bit, the heads' sums are kept apart in registers, and nothing but
// the running maximum is shared between threads.  Per tile of 128 tokens:
//     S[t][h]    = sum_c C[t][c] Q_lat[h][c] + sum_j KR[t][j] Q_rope[h][j]    M = 128, N = heads
//     O[c][h]   += sum_t C[t][c] P[t][h],   P = 2^(S - m[h])                   M = 128 (twice for d_c > 128)
// Q_rope is block-diagonal over the KV heads; a box of 64 key columns (8 KV heads) is multiplied
// with the 16 (or all) heads it concerns only.  (The operand's zeros times a key that is not
// finite are NaN for the heads of the box's other KV heads: rows that come out NaN are computed
// once more, head by head, when they are merged.)  O^T needs 32 columns per 128 latent columns, so
// two streams of tiles (even and odd, one softmax group each) keep an accumulator of their own
// and the chain load -> S -> softmax -> O of one overlaps the other's.  The streams' results are
// merged in tensor memory when a piece (part of one sequence) ends.
//
// What bounds it is HBM: the cached rows of the visible tokens, read once (ncu: 1.01 times their
// bytes; the tensor pipe is active for 7.6% of the kernel's time at d_c = 256).
// B200, whole calls: 32 sequences, 4160 visible tokens, 32 heads, d_c = 256: 45 us for 136 MB, of
// which tiles flow for about 28 (4.9 TB/s); the rest is the hand-over between the three launches,
// the first tiles and the last tile's chain.  64 sequences, 4005 tokens, 4-bit d_c = 128: 56 us.
//
// The running maximum is raised lazily: a thread that sees a score above m[h] + kTau reports it
// in the group's per-tile barrier (an OR over its 128 threads) and the group then takes the
// tile's maxima, rescales its accumulator and goes on.  Between raises P stays below 2^kTau.
//
// Roles: warp 0 TMA producer, warp 1 MMA issuer, warps 4-7 and 8-11 the softmax groups,
// warps 12-15 dequantise a quantised latent.  Every wait is bounded; a group leaves its loop only
// where all of it does (the barrier carries the failure too).
#include <cuda.h>

#include <algorithm>
#include <type_traits>

#include "decode_common.cuh"
#include "sm100.cuh"
#include "warp_mma.cuh"

namespace mla {
namespace wdec {

using namespace sm100;

constexpr int kUnit = 64;                 // tokens of a schedule tile and of a TMA box
constexpr int kT = 128;                   // tokens per product tile: two units
constexpr uint32_t kHalf = kUnit * 128;   // bytes of a box: 64 rows x 128 B
constexpr uint32_t kSlot = 2 * kHalf;     // ring slot: 128 tokens x 64 columns
// Threads: four warpgroups with a quantised latent (the last one dequantises), else three.
template <int QB> constexpr int kThreadsOf = QB ? 512 : 384;
constexpr float kTau = 8.0f;              // lazy-rescale threshold, log2 units
constexpr int kSBufs = 4;                 // S tiles in tensor memory: keys go ahead of their tile's latent
constexpr uint32_t kCols = 256, kSCol = 0, kOCol = 128;   // S: 4 x 32 columns, O: 2 streams x 2 blocks x 32
constexpr uint32_t kSmemMax = 232448;
constexpr int kMaxC = 4, kMaxK = 8, kMaxRaw = 3;
constexpr int kPieces = 64;               // pieces of a worker kept in shared memory

struct Args {
  int H, G, d_c, dcp, R, P, T_cap;
  int n_cbox, n_kbox, kr_rows;            // boxes per token row; heads a key box is multiplied with
  int n_blk;                              // parts of a latent tile: blocks of 128 columns
  int NC, NK, NRAW;                       // latent tiles, key boxes, code tiles in the rings
  int B, workers, cost;                   // cost of a piece, in units (see seq_units)
  int skip_tile;                          // testing only: 1-based tile whose latent is not copied (0 = none)
  MlaWindow win;
  int4* pieces;                           // [P] by slot: the pieces past the first kPieces of a worker
  const int32_t* seq_lens;
  const float* qrope;                     // [B][H][8], rotated, scaled
  float* opart;                           // [P][H][d_c]
  float* mlpart;                          // [H][P][2]
  const __half* scales;
  uint32_t code_row;
  mla_cache_t cache;
  int32_t* err;
  uint64_t wait_ns;
  uint32_t off_q, off_qr, off_p, off_c, off_k, off_raw, raw_stage, off_red, off_list, off_bar;
};

enum {
  kCFull = 0, kCEmpty = kCFull + 2 * kMaxC, kKFull = kCEmpty + 2 * kMaxC, kKEmpty = kKFull + kMaxK, kRFull = kKEmpty + kMaxK,
  kREmpty = kRFull + kMaxRaw, kSFull = kREmpty + kMaxRaw, kSEmpty = kSFull + kSBufs, kPFull = kSEmpty + kSBufs, kODone = kPFull + 2,
  kOEmpty = kODone + 2, kQFull, kQEmpty, kMeet, kDone, kBars
};
// Exchange area, floats: per group the tile maxima of its warps [2][4][32] (first row also the
// scores of a stream's first visible token); by piece parity the sums of all warps
// [2][2][4][32] and the groups' maxima [2][2][32]; per group the merge weights [2][2][32].
constexpr uint32_t kRedBytes = (2 * 4 * 32 + 2 * 2 * 4 * 32 + 2 * 2 * 32 + 2 * 2 * 32) * 4;

__device__ __forceinline__ uint32_t sw128(int r, int c) { return (uint32_t)r * 128u + (uint32_t)(((c ^ r) & 7) << 4); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Walk over a worker's pieces in tiles: x is the tile's first token in the sequence's span.  A
// piece is (sequence, first token, end, the sequence's length); its slot is slot0 + its number.
struct Walk {
  const Args* a;
  const int4* list;   // the first kPieces pieces; the others at their slots, which are consecutive
  int pc, end, slot0, b, x, x0, x1, len;
  Span span;
  __device__ void init(const Args* args, const int4* pieces, int n, int first_slot) {
    a = args;
    list = pieces;
    slot0 = first_slot;
    pc = 0;
    end = n;
    if (pc < end) load();
  }
  __device__ void load() {
    const int4 p = pc < kPieces ? list[pc] : a->pieces[slot0 + pc];
    b = p.x; x0 = p.y; x1 = p.z; len = p.w; x = x0;
    span = unit_span(len, 1, kUnit, a->win);
  }
  __device__ bool valid() const { return pc < end; }
  __device__ bool first() const { return x == x0; }
  __device__ bool last() const { return x + kT >= x1; }
  __device__ int rows() const { return min(kT, x1 - x); }
  __device__ int slot() const { return slot0 + pc; }
  __device__ int units() const { return x1 - x > kUnit ? 2 : 1; }
  __device__ int token(int unit) const { return span.token(x + unit * kUnit); }
  // Every row of the tile holds a visible token.
  __device__ bool whole() const {
    if (x1 - x < kT) return false;
    const int t0 = token(0), t1 = token(1);
    return (t0 >= span.lo || t0 + kUnit <= a->win.n_sink) && (t1 >= span.lo || t1 + kUnit <= a->win.n_sink);
  }
  __device__ bool visible(int r) const {
    const int t = token(r >> 6) + (r & 63);
    return r < x1 - x && (t >= span.lo || t < a->win.n_sink);
  }
  __device__ void next() {
    x += kT;
    if (x >= x1) { ++pc; if (pc < end) load(); }
  }
};

// The same walk where only the pieces' ends count.
struct Tiles {
  const Walk* w;      // pieces, as of the walk's start
  int pc, left, n;    // left: tiles of the piece, with this one; n: tiles gone by
  bool first;
  __device__ void init(const Walk& walk) { w = &walk; pc = 0; n = 0; load(); }
  __device__ bool valid() const { return pc < w->end; }
  __device__ void load() {
    if (!valid()) return;
    const int4 p = pc < kPieces ? w->list[pc] : w->a->pieces[w->slot0 + pc];
    left = (p.z - p.y + kT - 1) / kT;
    first = true;
  }
  __device__ bool last() const { return left == 1; }
  __device__ void next() {
    ++n;
    first = false;
    if (--left == 0) { ++pc; load(); }
  }
};

// Reduction over the lanes of x[h] for every h: lane h (mod N) receives column h's.
template <int N, typename F>
__device__ __forceinline__ float columns(float (&x)[N], int lane, F op) {
  if (N == 16) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = op(x[i], __shfl_xor_sync(0xffffffffu, x[i], 16));
  }
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float give = up ? x[i] : x[i + o], keep = up ? x[i + o] : x[i];
      x[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
  return x[0];
}

// The larger of two streams' maxima, NaN if one is: scores that are not numbers must not pass
// for a stream without a tile (-inf).
__device__ __forceinline__ float top_of(float a, float b) { return a != a ? a : b != b ? b : fmaxf(a, b); }

// Barrier of 128 threads that returns the OR of their predicates.
__device__ __forceinline__ bool group_or(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"((uint32_t)p), "r"(id)
      : "memory");
  return r != 0;
}

template <int N> __device__ __forceinline__ void tmem_ld(uint32_t ta, uint32_t (&v)[N]);
template <> __device__ __forceinline__ void tmem_ld<16>(uint32_t ta, uint32_t (&v)[16]) { tmem_ld16(ta, v); }
template <> __device__ __forceinline__ void tmem_ld<32>(uint32_t ta, uint32_t (&v)[32]) { tmem_ld32(ta, v); }

// The worker's pieces: list[0 .. min(n, kPieces)), the others in the workspace; returns n.  Whole
// CTA.  Reads the lengths, which were complete before the kernel ahead of this one started.
__device__ __forceinline__ int worker_pieces(const Args& a, int w, int4* list, int* slot0, int* s_warp, int* s_misc) {
  const int tid = threadIdx.x, nt = blockDim.x;
  if (tid == 0) { s_misc[0] = INT_MAX; s_misc[1] = 0; }
  int total = 0;
  SeqUnits mine;
  int my_ex = 0;
  for (int base = 0; base < a.B; base += nt) {
    mine = seq_units(a.seq_lens, base + tid, a.B, a.T_cap, kUnit, a.cost, a.win);
    int tot;
    my_ex = block_exscan(mine.n, &tot, s_warp);
    total += tot;
  }
  const int busy = busy_workers(total, a.workers);
  if (w >= busy) return 0;
  const int w0 = (int)worker_begin(w, total, busy), w1 = (int)worker_begin(w + 1, total, busy);
  int c_carry = 0, ne_carry = 0;
  for (int base = 0; base < a.B; base += nt) {
    if (a.B > nt) {   // more sequences than threads: their units once more
      mine = seq_units(a.seq_lens, base + tid, a.B, a.T_cap, kUnit, a.cost, a.win);
      int tot;
      my_ex = block_exscan(mine.n, &tot, s_warp);
      my_ex += c_carry;
      c_carry += tot;
    }
    int tot_ne;
    const int ne = ne_carry + block_exscan(mine.n > 0 ? 1 : 0, &tot_ne, s_warp);
    ne_carry += tot_ne;
    const int first = my_ex + a.cost;   // where the sequence's own units begin
    const bool in = mine.n > 0 && first < w1 && my_ex + mine.n > w0;
    if (in) atomicMin(s_misc, ne);   // the worker's first sequence
    __syncthreads();
    if (in) {
      const int k = ne - s_misc[0];
      const int4 p = make_int4(base + tid, max(0, w0 - first) * kUnit, min(mine.len, (w1 - first) * kUnit), mine.L);
      if (k < kPieces) list[k] = p;
      else a.pieces[w + ne] = p;
      atomicMax(s_misc + 1, k + 1);
    }
  }
  __syncthreads();
  *slot0 = w + s_misc[0];
  return s_misc[1];
}

// The same for up to kWarpSeqs sequences, by one warp, while the others set the CTA up; n and
// slot0 go to s_misc.  (Most CTAs can start only when the absorption's have left their SMs, so
// what they do before their first copy counts: barriers of the whole CTA here cost 1 us.)
constexpr int kWarpSeqs = 128;
__device__ __forceinline__ void warp_pieces(const Args& a, int w, int4* list, int* s_misc) {
  constexpr int K = kWarpSeqs / 32;
  const int lane = threadIdx.x & 31;
  int L[K], ex[K], total = 0;
  SeqUnits u[K];
#pragma unroll
  for (int k = 0; k < K; ++k) L[k] = 32 * k + lane < a.B ? __ldg(a.seq_lens + 32 * k + lane) : 0;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    u[k] = units_of(L[k], a.T_cap, kUnit, a.cost, a.win);
    ex[k] = total;
    if (32 * k >= a.B) continue;
    int x = u[k].n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    ex[k] += x - u[k].n;
    total += __shfl_sync(0xffffffffu, x, 31);
  }
  const int busy = busy_workers(total, a.workers);
  int slot0 = 0, n = 0;
  if (w < busy) {
    const int w0 = (int)worker_begin(w, total, busy), w1 = (int)worker_begin(w + 1, total, busy);
    int ne0 = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (32 * k >= a.B) continue;
      const uint32_t some = __ballot_sync(0xffffffffu, u[k].n > 0);
      const int ne = ne0 + __popc(some & ((1u << lane) - 1)), first = ex[k] + a.cost;   // where the sequence's own units begin
      const bool in = u[k].n > 0 && first < w1 && ex[k] + u[k].n > w0;
      const uint32_t mine = __ballot_sync(0xffffffffu, in);
      if (mine && n == 0) slot0 = w + __shfl_sync(0xffffffffu, ne, __ffs(mine) - 1);
      if (in) {
        const int4 p = make_int4(32 * k + lane, max(0, w0 - first) * kUnit, min(u[k].len, (w1 - first) * kUnit), L[k]);
        const int i = w + ne - slot0;
        if (i < kPieces) list[i] = p;
        else a.pieces[w + ne] = p;
      }
      n += __popc(mine);
      ne0 += __popc(some);
    }
  }
  __threadfence_block();
  if (lane == 0) { s_misc[0] = slot0; s_misc[1] = n; }
}

// N: heads padded to 16 or 32; QB: code width of a quantised latent (4 or 2), 0 for bf16.
template <int N, int QB>
__global__ void __launch_bounds__(kThreadsOf<QB>, 1)
window_decode_kernel(const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_kr,
                     const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ Args a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t sb = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sb - smem_u32(smem_raw));
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  auto bar = [&](int i) { return sb + a.off_bar + 8u * (uint32_t)i; };
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + a.off_bar + 8 * kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(s_tmem + 1);
  const uint64_t lim = a.wait_ns;
  constexpr uint32_t kPRow = N * 2;                     // bytes of a P row
  constexpr uint32_t kPBytes = kT * kPRow;
  constexpr uint32_t kPLayout = N == 32 ? (uint32_t)kLayoutSW64 : 6u;   // 64- or 32-byte swizzle
  const int NC = a.NC, NK = a.NK, NRAW = a.NRAW;

  __shared__ int s_warp[32], s_misc[2];
  int4* list = reinterpret_cast<int4*>(smem + a.off_list);
  const bool by_warp = a.B <= kWarpSeqs;
  // The kernel ahead is this call's absorption, which started once everything before it was
  // done: lengths and block table can be read now.
  if (warp == 0) {
    if (by_warp) warp_pieces(a, blockIdx.x, list, s_misc);
    if (lane == 0) {
      *abort_flag = 0;
      tma_prefetch_desc(&tm_c);
      tma_prefetch_desc(&tm_kr);
      tma_prefetch_desc(&tm_q);
    }
  } else if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), kCols);
    tmem_relinquish();
  } else if (warp == 2) {
    for (int i = lane; i < kBars; i += 32) {
      int n = 1;
      if (i >= kCFull && i < kCEmpty && QB) n = 4;      // the dequantising warps
      if (i >= kREmpty && i < kSFull) n = 4;
      if (i >= kSEmpty && i < kODone) n = 4;            // a softmax group's warps (S read, P written)
      if (i == kOEmpty || i == kMeet) n = 8;            // both groups
      if (i == kQFull) n = 2;                           // Q_lat bytes, the RoPE rows
      mbar_init(bar(i), n);
    }
    fence_mbar_init();
  } else {
    // query rows past the last head and the zero blocks of the RoPE operand stay zero
    for (uint32_t i = threadIdx.x - 96; i < (a.off_p - a.off_q) / 16; i += kThreadsOf<QB> - 96)
      reinterpret_cast<uint4*>(smem + a.off_q)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const uint32_t c_bytes = (uint32_t)a.n_cbox * kSlot;
  int slot0 = s_misc[0], n_pieces = s_misc[1];
  if (!by_warp) n_pieces = worker_pieces(a, blockIdx.x, list, &slot0, s_warp, s_misc);
  // Registers with a quantised latent: 512 threads x 128 = 65536 = 128 x (88 + 168 + 168 + 88).
  if (warp < 4) {
    if (QB) setmaxnreg_dec<88>();
    if (warp == 0) {
      // ============================================================ TMA producer (converged warp, elected lane)
      // Cursors: latent (or code) tiles, key boxes, queries, whose places free up at different
      // times.  The cache rows of a tile's units are looked up when the cursor reaches it, not
      // when its place is free.  Nothing is copied before the absorption is done: copies started
      // ahead of it slow its few loads down by more than they gain (Llama-shaped layers, us: 47.9
      // against 47.0 at d_c = 256, 25.5 against 23.8 at d_c = 64).
      auto ready = [&](int i, int parity) { return __all_sync(0xffffffffu, mbar_test(bar(i), parity)) != 0; };
      Walk wc, wk, wq;
      wc.init(&a, list, n_pieces, slot0);
      wk = wc;
      wq = wc;
      // Cache rows of the next 32 units of a walk's piece, one per lane (a unit lies in one block),
      // and the two of its tile: one look into the block table per 32 units.
      struct Rows { int unit0, lane_row, row[2]; } c_at, k_at;
      auto rows_at = [&](const Walk& it, Rows& o) {
        const int unit = (it.x - it.x0) / kUnit;
        if (it.first() || unit + 1 - o.unit0 >= 32) {
          o.unit0 = unit;
          const int ux = it.x + lane * kUnit;
          o.lane_row = 0;
          if (ux < it.x1) {
            const MlaLoc lc = mla_loc(a.cache, it.b, it.span.token(ux), a.err);
            o.lane_row = (int)(lc.pb * lc.cap + lc.pt);
          }
        }
        o.row[0] = __shfl_sync(0xffffffffu, o.lane_row, unit - o.unit0);
        o.row[1] = __shfl_sync(0xffffffffu, o.lane_row, unit - o.unit0 + 1);
      };
      if (wc.valid()) rows_at(wc, c_at);
      k_at = c_at;
      int nc = 0, pc = 0, nk = 0, kb = 0, u = 0;   // pc: parts of latent tile nc copied; u: query loads issued
      RingPos rc, rk;
      const int c_ring = QB ? NRAW : NC;
      int looks = 0;
      uint64_t idle = 0;
      auto load_q = [&]() {
        if (elect_one()) {
          mbar_expect_tx(bar(kQFull), (uint32_t)a.n_cbox * a.H * 128u);
          for (int k = 0; k < a.n_cbox; ++k) tma_load_2d(sb + a.off_q + k * N * 128, &tm_q, bar(kQFull), k * 64, wq.b * a.H);
        }
        __syncwarp();
        ++u;
        if (++wq.pc < wq.end) wq.load();
      };
      bool ok = true;
      if (wq.valid()) {
        pdl_wait();
        load_q();   // ahead of the first tile: behind it, ragged Llama-shaped sequences take 21.3 us instead of 20.3
      }
      while (ok && (wc.valid() || wk.valid() || wq.valid())) {
        bool progress = false;
        if (wc.valid()) {
          const int s = rc.slot;
          if (nc < c_ring || ready(QB ? kREmpty + s : kCEmpty + 2 * s + pc, rc.parity ^ 1)) {
            const int units = wc.units(), k1 = min(2 * pc + 2, a.n_cbox);
            if (nc + 1 != a.skip_tile && elect_one()) {
              if (QB) {
                const uint32_t dst = sb + a.off_raw + s * a.raw_stage;
                mbar_expect_tx(bar(kRFull + s), (uint32_t)units * kUnit * a.code_row);
                tma_load_2d(dst, &tm_c, bar(kRFull + s), 0, c_at.row[0]);
                if (units > 1) tma_load_2d(dst + kUnit * a.code_row, &tm_c, bar(kRFull + s), 0, c_at.row[1]);
              } else {
                const uint32_t dst = sb + a.off_c + s * c_bytes;
                const uint32_t full = bar(kCFull + 2 * s + pc);
                mbar_expect_tx(full, (uint32_t)(units * (k1 - 2 * pc)) * kHalf);
                for (int k = 2 * pc; k < k1; ++k) {
                  tma_load_2d(dst + k * kSlot, &tm_c, full, k * 64, c_at.row[0]);
                  if (units > 1) tma_load_2d(dst + k * kSlot + kHalf, &tm_c, full, k * 64, c_at.row[1]);
                }
              }
            }
            __syncwarp();
            if (QB || ++pc == a.n_blk) {
              pc = 0;
              wc.next();
              rc.next(c_ring);
              ++nc;
              if (wc.valid()) rows_at(wc, c_at);
            }
            progress = true;
          }
        }
        while (wk.valid()) {
          const int s = rk.slot;
          if (!(nk < NK || ready(kKEmpty + s, rk.parity ^ 1))) break;
          const int units = wk.units();
          if (elect_one()) {
            mbar_expect_tx(bar(kKFull + s), (uint32_t)units * kHalf);
            tma_load_2d(sb + a.off_k + s * kSlot, &tm_kr, bar(kKFull + s), kb * 64, k_at.row[0]);
            if (units > 1) tma_load_2d(sb + a.off_k + s * kSlot + kHalf, &tm_kr, bar(kKFull + s), kb * 64, k_at.row[1]);
          }
          __syncwarp();
          rk.next(NK);
          ++nk;
          if (++kb == a.n_kbox) {
            kb = 0;
            wk.next();
            if (wk.valid()) rows_at(wk, k_at);
          }
          progress = true;
        }
        if (wq.valid() && ready(kQEmpty, (u - 1) & 1)) {
          load_q();
          progress = true;
        }
        if (progress) {
          looks = 0;
        } else if ((++looks & 63) == 0) {
          const uint64_t now = globaltimer();
          if (looks == 64) idle = now;
          if (*abort_flag || now - idle > lim) { *abort_flag = 1; ok = false; }
          ok = __all_sync(0xffffffffu, ok) != 0;
        }
      }
      // every issued copy lands before the CTA exits
      volatile int never = 0;
      auto drain = [&](int first, int ring, int issued) {
        for (int i = max(0, issued - ring); i < issued; ++i) mbar_spin(bar(first + i % ring), (i / ring) & 1, &never, lim);
      };
      if (QB) drain(kRFull, NRAW, nc);
      for (int i = max(0, nc - NC); !QB && i < nc + (pc > 0); ++i)
        for (int m = 0; m < (i < nc ? a.n_blk : pc); ++m) mbar_spin(bar(kCFull + 2 * (i % NC) + m), (i / NC) & 1, &never, lim);
      drain(kKFull, NK, nk);
      if (*abort_flag && u > 0) {   // the queries' copy (its barrier may still miss the RoPE rows: wait a moment instead)
        const uint64_t t0 = globaltimer();
        while (!mbar_test(bar(kQFull), (u - 1) & 1) && globaltimer() - t0 < 1000000ull) {}
      }
    } else if (warp == 1) {
      // ============================================================ MMA issuer (converged warp, elected lane)
      const uint32_t id_s = idesc_bf16_f32(kT, N, false, false), id_k = idesc_bf16_f32(kT, a.kr_rows, false, false);
      const uint32_t id_o = idesc_bf16_f32(kT, N, true, true);
      const uint64_t desc_q = smem_desc(sb + a.off_q, 16, 1024, kLayoutSW128);
      const uint64_t desc_qr = smem_desc(sb + a.off_qr, 16, 1024, kLayoutSW128);
      auto ready = [&](int i, int parity) { return __all_sync(0xffffffffu, mbar_test(bar(i), parity)) != 0; };
      Walk i2;                // the tile whose O is issued next
      i2.init(&a, list, n_pieces, slot0);
      const Walk start = i2;
      Tiles ik, i1;           // the tiles whose key product, and whose latent product, is issued next
      ik.init(start);
      i1.init(start);
      // S is the sum of the key product, which goes first, and the latent product.  The keys of a
      // tile wait for its place in tensor memory only and so leave their ring early, most of them
      // while the tile's latent is still being copied.
      int kb = 0, m1 = 0, uk = 0, n2 = 0, u2 = 0;   // key boxes of ik, latent parts of i1 issued; pieces begun, finished
      RingPos r1, r2, rk;                           // latent tiles of S and of O, key boxes
      bool ok = true;
      int looks = 0;
      uint64_t idle = 0;
      while (ok && i2.valid()) {
        bool progress = false;
        // O(n2): its P, and for a stream's first tile of a piece the accumulators read out
        if (n2 < i1.n && ready(kPFull + (n2 & 1), (n2 >> 1) & 1)) {
          const bool fresh = i2.x - i2.x0 < 2 * kT;   // the piece's first or second tile: its stream starts
          if (!fresh || u2 == 0 || ready(kOEmpty, (u2 - 1) & 1)) {
            tc_fence_after();
            const int s = n2 & 1;
            if (elect_one()) {
              const uint64_t dp = smem_desc(sb + a.off_p + s * kPBytes, 16, 8 * kPRow, kPLayout);
              const uint64_t dc = smem_desc(sb + a.off_c + r2.slot * c_bytes, kSlot, 1024, kLayoutSW128);
              const int steps = (i2.rows() + 15) / 16;
              for (int m = 0; m < a.n_blk; ++m) {
                const uint32_t d = tmem + kOCol + s * 64 + m * 32;
                const uint64_t dm = dc + (uint32_t)m * (2 * kSlot >> 4);
                if (steps == kT / 16) {
                  tc_mma_bf16(d, dm, dp, id_o, !fresh);
  #pragma unroll
                  for (int k = 1; k < kT / 16; ++k) tc_mma_bf16(d, dm + 128 * k, dp + k * (16 * kPRow >> 4), id_o, 1);
                } else {
                  for (int k = 0; k < steps; ++k)
                    tc_mma_bf16(d, dm + 128u * k, dp + (uint32_t)k * (16 * kPRow >> 4), id_o, !fresh || k > 0);
                }
                tc_commit(bar(kCEmpty + 2 * r2.slot + m));
              }
              tc_commit(bar(kODone + s));
            }
            __syncwarp();
            if (i2.last()) ++u2;
            i2.next();
            r2.next(NC);
            ++n2;
            progress = true;
          }
        }
        // latent parts of S(i1)
        if (i1.n < ik.n && ready(kCFull + 2 * r1.slot + m1, r1.parity)) {
          tc_fence_after();
          const int s = i1.n & (kSBufs - 1);
          const bool done = m1 + 1 == a.n_blk;
          if (elect_one()) {
            const uint32_t d = tmem + kSCol + s * 32;
            uint64_t da = smem_desc(sb + a.off_c + r1.slot * c_bytes + m1 * 2 * kSlot, 16, 1024, kLayoutSW128);
            uint64_t db = desc_q + (uint32_t)m1 * (2 * N * 128 >> 4);
            for (int k = 2 * m1; k < min(2 * m1 + 2, a.n_cbox); ++k) {   // a box of 64 columns is four steps
              tc_mma_bf16(d, da, db, id_s, 1);
              tc_mma_bf16(d, da + 2, db + 2, id_s, 1);
              tc_mma_bf16(d, da + 4, db + 4, id_s, 1);
              tc_mma_bf16(d, da + 6, db + 6, id_s, 1);
              da += kSlot >> 4;
              db += (N * 128) >> 4;
            }
            if (done) {
              tc_commit(bar(kSFull + s));
              if (i1.last()) tc_commit(bar(kQEmpty));
            }
          }
          __syncwarp();
          if (done) {
            m1 = 0;
            r1.next(NC);
            i1.next();
          } else {
            ++m1;
          }
          progress = true;
        }
        // key boxes of S(ik), as many as are there
        if (ik.valid() && (kb > 0 || ((ik.n < kSBufs || ready(kSEmpty + (ik.n & (kSBufs - 1)), (ik.n / kSBufs - 1) & 1)) &&
                                      (!ik.first || ready(kQFull, uk & 1))))) {
          int take = 0;
          RingPos rt = rk;
          while (take < a.n_kbox - kb && ready(kKFull + rt.slot, rt.parity)) {
            ++take;
            rt.next(NK);
          }
          if (take > 0) {
            tc_fence_after();
            if (elect_one()) {
              const uint32_t d0 = tmem + kSCol + (ik.n & (kSBufs - 1)) * 32;
              for (int j = 0; j < take; ++j, ++kb) {
                // KV heads 8 kb .. 8 kb + 7: query heads from col on
                const uint32_t col = a.kr_rows == N ? 0 : (kb * 8 * a.G) & ~15;
                const bool more = a.kr_rows == N ? kb > 0 : kb > 0 && col == (uint32_t)(((kb - 1) * 8 * a.G) & ~15);   // columns begun
                const uint64_t da = smem_desc(sb + a.off_k + rk.slot * kSlot, 16, 1024, kLayoutSW128);
                const uint64_t db = desc_qr + (uint32_t)kb * (a.kr_rows * 128u >> 4);
                const int steps = min(4, (a.R - kb * 64 + 15) / 16);
                tc_mma_bf16(d0 + col, da, db, id_k, more);
                if (steps > 1) tc_mma_bf16(d0 + col, da + 2, db + 2, id_k, 1);
                if (steps > 2) tc_mma_bf16(d0 + col, da + 4, db + 4, id_k, 1);
                if (steps > 3) tc_mma_bf16(d0 + col, da + 6, db + 6, id_k, 1);
                tc_commit(bar(kKEmpty + rk.slot));
                rk.next(NK);
              }
              kb -= take;
            }
            __syncwarp();
            rk = rt;
            kb += take;
            if (kb == a.n_kbox) {
              kb = 0;
              if (ik.first) ++uk;
              ik.next();
            }
            progress = true;
          }
        }
        if (progress) {
          looks = 0;
        } else if ((++looks & 63) == 0) {
          const uint64_t now = globaltimer();
          if (looks == 64) idle = now;
          if (*abort_flag || now - idle > lim) { *abort_flag = 1; ok = false; }
          ok = __all_sync(0xffffffffu, ok) != 0;
        }
      }
      if (elect_one()) tc_commit(bar(kDone));   // whatever was issued has finished before tensor memory is freed
      __syncwarp();
      volatile int never = 0;
      mbar_spin(bar(kDone), 0, &never, lim);
    }   // (warps 2 and 3 idle)
  } else if (QB != 0 && warp >= 12) {
    // ============================================================ dequantisation (a token row per thread)
    if (QB) setmaxnreg_dec<88>();
    const int r = (warp - 12) * 32 + lane;
    Walk it;
    it.init(&a, list, n_pieces, slot0);
    // Where a row's values come from is asked for ahead of its tile, so that no load is waited
    // for in the loop: the cache row (a look into the block table) two tiles, the group scales
    // and the ring tag a tile ahead.
    struct Src {
      bool live = false;
      int tag = -1, pos = 0;            // ring: the position its slot holds, the token's own
      size_t slot = 0;
      unsigned short sc[8];             // fp16 scales
    };
    Walk w1 = it, w2 = it;              // one and two tiles ahead
    auto cache_row = [&](const Walk& t) -> long long {
      if (!t.valid() || !t.visible(r)) return -1;
      const MlaLoc lc = mla_loc(a.cache, t.b, t.token(r >> 6), a.err);
      return (long long)lc.pb * lc.cap + lc.pt + (r & 63);
    };
    auto source = [&](const Walk& t, long long row, Src& o) {
      o.live = row >= 0;
      o.tag = -1;
      if (!o.live) return;
      const unsigned short* sp = reinterpret_cast<const unsigned short*>(a.scales) + (size_t)row * (a.d_c / 32);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < a.d_c / 32) o.sc[k] = __ldg(sp + k);
      if (a.cache.c_resid) {
        o.pos = t.token(r >> 6) + (r & 63);
        if (o.pos >= t.len - MLA_RESID_WINDOW) {
          o.slot = (size_t)t.b * MLA_RESID_WINDOW + (o.pos & (MLA_RESID_WINDOW - 1));
          o.tag = __ldg(a.cache.resid_pos + o.slot);
        }
      }
    };
    Src cur, nxt;
    source(it, cache_row(it), cur);
    if (w1.valid()) w1.next();
    long long row1 = cache_row(w1);
    w2 = w1;
    bool ok = true;
    RingPos rr, rc;   // code tiles, latent tiles
    for (int n = 0; ok && it.valid(); ++n, it.next(), rr.next(NRAW), rc.next(NC)) {
      const int rs = rr.slot, cs = rc.slot;
      source(w1, row1, nxt);
      if (w2.valid()) w2.next();
      const long long row2 = cache_row(w2);
      ok = __all_sync(0xffffffffu, mbar_wait(bar(kRFull + rs), rr.parity, abort_flag, lim));
      if (!ok) break;
      uint8_t* C = smem + a.off_c + cs * c_bytes;
      auto put = [&](int chunk, uint4 v) { *reinterpret_cast<uint4*>(C + (chunk >> 3) * kSlot + sw128(r, chunk)) = v; };
      const bool kept = cur.live && cur.tag >= 0 && cur.tag == cur.pos;   // one of the window's unquantised tokens
      const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.cache.c_resid) + cur.slot * a.d_c);
      const uint8_t* codes = smem + a.off_raw + rs * a.raw_stage + r * a.code_row;
      uint32_t scw[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) scw[k] = cur.sc[2 * k] | (uint32_t)cur.sc[2 * k + 1] << 16;
#pragma unroll 1
      for (int m = 0; m < a.n_blk; ++m) {   // a part: 128 columns
        if (n >= NC) ok = __all_sync(0xffffffffu, mbar_wait(bar(kCEmpty + 2 * cs + m), rc.parity ^ 1, abort_flag, lim));
        if (!ok) break;
        const int g1 = min(4 * m + 4, a.d_c / 32);
        if (kept) {
          for (int c = 16 * m; c < 4 * g1; ++c) put(c, __ldg(src + c));
        } else if (cur.live) {
          // (rolled loops, eight values a time: with more code per pass the roles no longer fit the
          // instruction caches; 4-bit Llama-shaped case, us: 57.5 so, 61.1 with 32 values a pass)
#pragma unroll 1
          for (int g = 4 * m; g < g1; ++g) {
            const float sv = __half2float(__ushort_as_half((unsigned short)scw[0]));
#pragma unroll
            for (int k = 0; k < 4; ++k) scw[k] = __funnelshift_r(scw[k], k < 3 ? scw[k + 1] : 0u, 16);   // the next group's scale
            uint32_t wd[4];
            if (QB == 4) {
              const uint4 cw = *reinterpret_cast<const uint4*>(codes + g * 16);
              wd[0] = cw.x; wd[1] = cw.y; wd[2] = cw.z; wd[3] = cw.w;
            } else {
              const uint2 cw = *reinterpret_cast<const uint2*>(codes + g * 8);
              wd[0] = cw.x; wd[1] = cw.x >> 16; wd[2] = cw.y; wd[3] = cw.y >> 16;
            }
#pragma unroll 1
            for (int ch = 0; ch < 4; ++ch) {
              put(4 * g + ch, dequant8<QB ? QB : 4>(wd[0], sv));
              wd[0] = wd[1]; wd[1] = wd[2]; wd[2] = wd[3];
            }
          }
        } else {
          for (int c = 16 * m; c < 4 * g1; ++c) put(c, make_uint4(0, 0, 0, 0));
        }
        for (int c = max(16 * m, a.d_c / 8); c < min(16 * m + 16, a.dcp / 8); ++c) put(c, make_uint4(0, 0, 0, 0));   // padding columns
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kCFull + 2 * cs + m));
      }
      if (!ok) break;
      if (lane == 0) mbar_arrive(bar(kREmpty + rs));
      cur = nxt;
      w1 = w2;
      row1 = row2;
    }
  } else {
    // ============================================================ softmax groups
    if (QB) setmaxnreg_inc<168>();
    const int s = warp >= 8;                 // stream
    const int q = warp & 3, r = 32 * q + lane;
    const uint32_t lane0 = tmem + ((uint32_t)(32 * q) << 16);
    float* red = reinterpret_cast<float*>(smem + a.off_red) + s * 4 * 32;
    float* sums = reinterpret_cast<float*>(smem + a.off_red) + 2 * 4 * 32;   // [parity][stream][warp][32]
    float* tops = sums + 2 * 2 * 4 * 32;                                     // [parity][stream][32]
    float* wts = tops + 2 * 2 * 32 + s * 2 * 32;                             // merge weights [stream][32]
    pdl_wait();   // the RoPE queries, and the partials this kernel writes
    pdl_trigger();
    auto warp_wait = [&](int i, int parity) { return __all_sync(0xffffffffu, mbar_wait(bar(i), parity, abort_flag, lim)) != 0; };
    auto arrive = [&](int i) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(i));
    };
    Walk it;
    it.init(&a, list, n_pieces, slot0);
    int n = 0, u = 0;                        // tiles and pieces of the CTA
    RingPos rc;                              // latent tiles
    float m[N], l[N];
    bool some = false;                       // this stream had a tile in the piece
    bool fail = false;
    while (it.valid()) {   // left only where the whole group leaves: after group_or
      const bool last = it.last();
      if (it.first()) {
        some = false;
#pragma unroll
        for (int h = 0; h < N; ++h) { m[h] = -INFINITY; l[h] = 0.f; }
        if (warp == 4) {   // the RoPE query rows, once S of the previous piece has read its own
          fail = u > 0 && !warp_wait(kQEmpty, (u - 1) & 1);
          if (!fail && lane < a.H) {
            const float4* src = reinterpret_cast<const float4*>(a.qrope + ((size_t)it.b * a.H + lane) * 8);
            const float4 x = __ldcg(src), y = __ldcg(src + 1);
            const int g = lane / a.G, kb = g >> 3;
            const int col = a.kr_rows == N ? 0 : (kb * 8 * a.G) & ~15;
            *reinterpret_cast<uint4*>(smem + a.off_qr + kb * a.kr_rows * 128 + sw128(lane - col, g & 7)) =
                make_uint4(pack2(x.x, x.y), pack2(x.z, x.w), pack2(y.x, y.y), pack2(y.z, y.w));
          }
          fence_proxy_async_smem();
          if (!fail) arrive(kQFull);
        }
      }
      if ((n & 1) == s) {
        const int k = n >> 1;
        const int buf = n & (kSBufs - 1);
        if (!fail) fail = !warp_wait(kSFull + buf, (n / kSBufs) & 1);
        float x[N];
        {
          uint32_t raw[N];
          tc_fence_after();
          tmem_ld<N>(lane0 + kSCol + buf * 32, raw);
          tmem_wait_ld();
          const bool vis = it.visible(r);
#pragma unroll
          for (int h = 0; h < N; ++h) {
            asm volatile("" : "+r"(raw[h]));   // the values exist only after the wait
            x[h] = vis ? __uint_as_float(raw[h]) : -INFINITY;
          }
        }
        tc_fence_before();
        arrive(kSEmpty + buf);
        if (!some) {
          // the stream starts from the scores of its first visible token plus kTau: a raise (a
          // reduction over the tile, microseconds with its code cold) is then needed only for
          // scores 2 kTau above that token's, and the sums stay as exact with a maximum that is
          // up to kTau too high
          const int t0 = it.token(0);
          const int first = t0 >= it.span.lo || t0 < a.win.n_sink ? 0 : it.span.lo - t0;
          if (r == first) {
#pragma unroll
            for (int h = 0; h < N; ++h) red[h] = x[h];
          }
          (void)group_or(1 + s, false);
#pragma unroll
          for (int h = 0; h < N; ++h) m[h] = red[h] + kTau;
        }
        bool raise = false;
#pragma unroll
        for (int h = 0; h < N; ++h) raise |= x[h] > m[h] + kTau;
        // P's buffer and the accumulator are free once the stream's previous tile is in O
        if (!fail && k > 0) fail = !warp_wait(kODone + s, (k - 1) & 1);
        if (group_or(1 + s, raise || fail)) {
          float y[N];
#pragma unroll
          for (int h = 0; h < N; ++h) y[h] = x[h];
          const float top = columns<N>(y, lane, [](float p, float o) { return fmaxf(p, o); });
          if (lane < N) red[q * 32 + lane] = top;
          if (group_or(1 + s, fail)) break;   // the whole group leaves here
          tc_fence_after();
          float al[N];
#pragma unroll
          for (int h = 0; h < N; ++h) {
            const float t = fmaxf(fmaxf(red[h], red[32 + h]), fmaxf(red[64 + h], red[96 + h]));
            const bool up = t > m[h] + kTau;
            al[h] = up ? ex2_approx(m[h] - t) : 1.f;   // m = -inf: 0
            m[h] = up ? t : m[h];
            l[h] *= al[h];
          }
          if (some) {
            for (int blk = 0; blk < a.n_blk; ++blk) {
#pragma unroll
              for (int h0 = 0; h0 < N; h0 += 8) {
                uint32_t o[8];
                tmem_ld8(lane0 + kOCol + s * 64 + blk * 32 + h0, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al[h0 + e]);
                tmem_st8(lane0 + kOCol + s * 64 + blk * 32 + h0, o);
              }
            }
            tmem_wait_st();
          }
        }
        some = true;
        // P row of this token, rounded to bf16: both operands of a product have the latent's type.
        // Tokens' errors are independent: 0.0012 of the output's norm over few visible tokens, 0.0005
        // over thousands, where the output's own rounding makes 0.0017; P in two halves would double
        // O's products and P's buffers.  The sum takes P as it was: rounding to nearest has no bias
        // to make up for.
        uint32_t pk[N / 2];
#pragma unroll
        for (int h = 0; h < N; h += 2) {
          const float m0 = m[h] == -INFINITY ? 0.f : m[h], m1 = m[h + 1] == -INFINITY ? 0.f : m[h + 1];
          const float p0 = ex2_approx(x[h] - m0), p1 = ex2_approx(x[h + 1] - m1);
          l[h] += p0;
          l[h + 1] += p1;
          pk[h / 2] = pack2(p0, p1);
        }
        uint8_t* prow = smem + a.off_p + s * kPBytes + r * kPRow;
#pragma unroll
        for (int c = 0; c < N / 8; ++c) {
          const int at = N == 32 ? (c ^ (r >> 1)) & 3 : (c ^ (r >> 2)) & 1;
          *reinterpret_cast<uint4*>(prow + at * 16) = make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        }
        if (!QB && !it.whole()) {
          // rows without a visible token (stale or hidden, possibly not finite) are zeroed
          // before O's product multiplies them by P = 0; S of this tile has been read
          uint8_t* C = smem + a.off_c + rc.slot * c_bytes;
          auto zero_rows = [&](int from, int to) {   // consecutive threads, consecutive 16-byte chunks
            for (int i = from * 8 + r; i < to * 8; i += 128)
              for (int b = 0; b < a.n_cbox; ++b) *reinterpret_cast<uint4*>(C + b * kSlot + i * 16) = make_uint4(0, 0, 0, 0);
          };
          const int rows = it.rows();
          for (int j = 0; j < it.units(); ++j) {
            const int t0 = it.token(j), end = min(64, rows - 64 * j);
            zero_rows(64 * j + min(end, max(0, a.win.n_sink - t0)), 64 * j + min(end, it.span.lo - t0));
          }
          zero_rows(rows, (rows + 15) & ~15);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        arrive(kPFull + s);
      }
      if (last) {
        // ---------------- the piece's partial (m, l, O): both streams merged
        const int par = u & 1;
        {
          float y[N];
#pragma unroll
          for (int h = 0; h < N; ++h) y[h] = l[h];
          const float sum = columns<N>(y, lane, [](float p, float o) { return p + o; });
          if (lane < N) sums[((par * 2 + s) * 4 + q) * 32 + lane] = sum;
          if (r == 0) {
#pragma unroll
            for (int h = 0; h < N; ++h) tops[(par * 2 + s) * 32 + h] = m[h];
          }
        }
        // both streams' last tiles are in O when their counters stand at the piece's end
        const int done0 = (n + 2) >> 1, done1 = (n + 1) >> 1;   // tiles of each stream so far
        arrive(kMeet);
        if (!fail) fail = !warp_wait(kMeet, u & 1);
        const float* t0 = tops + par * 2 * 32;
        if (r < N) {   // a stream without a tile in this piece weighs nothing
          const float m0 = t0[r], m1 = t0[32 + r], M = top_of(m0, m1);
          wts[r] = m0 == -INFINITY ? 0.f : ex2_approx(m0 - M);
          wts[32 + r] = m1 == -INFINITY ? 0.f : ex2_approx(m1 - M);
        }
        if (!fail && done0 > 0) fail = !warp_wait(kODone, (done0 - 1) & 1);
        if (!fail && done1 > 0) fail = !warp_wait(kODone + 1, (done1 - 1) & 1);
        if (group_or(1 + s, fail)) break;
        tc_fence_after();
        // this group writes heads [N/2 s, N/2 s + N/2): lane = latent column
        const float* l0 = sums + par * 2 * 4 * 32;
        constexpr int HN = N / 2;
        float w0[HN], w1[HN];   // weight 0: the stream's columns may be stale
#pragma unroll
        for (int e = 0; e < HN; ++e) { w0[e] = wts[HN * s + e]; w1[e] = wts[32 + HN * s + e]; }
        float* dst = a.opart + ((size_t)it.slot() * a.H + HN * s) * a.d_c + r;
#pragma unroll 1
        for (int blk = 0; blk < a.n_blk; ++blk, dst += 128) {
          uint32_t o0[HN], o1[HN];
#pragma unroll
          for (int e = 0; e < HN; e += 8) {
            tmem_ld8(lane0 + kOCol + blk * 32 + HN * s + e, *reinterpret_cast<uint32_t(*)[8]>(o0 + e));
            tmem_ld8(lane0 + kOCol + 64 + blk * 32 + HN * s + e, *reinterpret_cast<uint32_t(*)[8]>(o1 + e));
          }
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < HN; ++e) {
            asm volatile("" : "+r"(o0[e]), "+r"(o1[e]));
            const float v = (w0[e] != 0.f ? w0[e] * __uint_as_float(o0[e]) : 0.f) + (w1[e] != 0.f ? w1[e] * __uint_as_float(o1[e]) : 0.f);
            if (HN * s + e < a.H && blk * 128 + r < a.d_c) dst[(size_t)e * a.d_c] = v;
          }
        }
        if (s == 0 && r < a.H) {
          const float M = top_of(t0[r], t0[32 + r]);
          float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            sum0 += l0[k * 32 + r];
            sum1 += l0[(4 + k) * 32 + r];
          }
          *reinterpret_cast<float2*>(a.mlpart + ((size_t)r * a.P + it.slot()) * 2) = make_float2(M, wts[r] * sum0 + wts[32 + r] * sum1);
        }
        tc_fence_before();
        arrive(kOEmpty);
        ++u;
      }
      it.next();
      rc.next(NC);
      ++n;
    }
  }
  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
  if (threadIdx.x == 0 && *abort_flag) raise_error(a.err, MLA_DEVERR_TIMEOUT);
}

// ------------------------------------------------------------------ absorption
// q_lat[row][c] = scale x log2(e) x sum_d q[row][d] W_ukF[g][d][c] (summed in float32, rounded once
// to bf16, the type of the latents that it meets in the attention's product, which makes 0.0016 of
// the output's norm; in two halves it would double S's products) for 32 rows (sequence, query head
// of KV head g) and 64 latent columns per CTA, and the kept pairs of the rows, rotated at L - 1.
// Latency bound: the W_uk slice and the frequencies come from the plan and are fetched before the
// kernel ahead is waited for; what follows the wait is one round trip for queries and lengths.
constexpr int kARows = 32, kACols = 64, kAThreads = 256;
struct AbsorbArgs {
  int B, H, G, n_kv, d_h, d_c, T_cap;
  float scale;
  const __nv_bfloat16* q;       // [B][H][d_h]
  const __nv_bfloat16* W_ukF;   // [n_kv][d_h][d_c]
  const int32_t* seq_lens;
  const int32_t* rope_pair;     // [n_kv][4]
  const double* theta;
  __nv_bfloat16* qlat;          // [B][H][d_c]
  float* qrope;                 // [B][H][8]
};

__global__ void __launch_bounds__(kAThreads) window_absorb_kernel(AbsorbArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  using bf16 = __nv_bfloat16;
  constexpr int WLD = kACols + 8;
  const int KP = (a.d_h + 15) & ~15, QLD = KP + 8;
  bf16* sw = reinterpret_cast<bf16*>(smem);   // [KP][WLD]
  bf16* sq = sw + KP * WLD;                   // [32][QLD]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rows_g = a.B * a.G, n_rb = (rows_g + kARows - 1) / kARows;
  const int g = blockIdx.x % a.n_kv, rb = (blockIdx.x / a.n_kv) % n_rb, cc = blockIdx.x / (a.n_kv * n_rb);
  const int row0 = rb * kARows, c0 = cc * kACols;
  const bf16* W = a.W_ukF + (size_t)g * a.d_h * a.d_c;
  auto index = [&](int row) { return (size_t)(row / a.G) * a.H + g * a.G + row % a.G; };
  for (int v = tid; v < KP * (kACols / 8); v += kAThreads) {   // zeros past the matrix edges
    const int d = v / (kACols / 8), c = (v % (kACols / 8)) * 8;
    const bool ok = d < a.d_h && c0 + c < a.d_c;   // whole chunks: d_c is a multiple of 32
    cp_async16(smem_u32(sw + d * WLD + c), ok ? (const void*)(W + (size_t)d * a.d_c + c0 + c) : a.W_ukF, ok ? 16u : 0u);
  }
  // RoPE (first column chunk): a thread per row and kept pair
  const int rr = row0 + tid / 4;
  const bool rot = cc == 0 && tid < 4 * kARows && rr < rows_g;
  const int pair = rot ? __ldg(a.rope_pair + g * 4 + (tid & 3)) : 0;
  const double th = rot ? __ldg(a.theta + pair) : 0.0;
  pdl_wait();
  pdl_trigger();
  for (int v = tid; v < kARows * (KP / 8); v += kAThreads) {
    const int r = v / (KP / 8), d = (v % (KP / 8)) * 8;
    const bool ok = row0 + r < rows_g && d < a.d_h;   // whole chunks: d_h is a multiple of 8
    cp_async16(smem_u32(sq + r * QLD + d), ok ? (const void*)(a.q + index(row0 + r) * a.d_h + d) : a.q, ok ? 16u : 0u);
  }
  cp_async_commit();
  if (rot) {
    const size_t o = index(rr);
    const int L = __ldg(a.seq_lens + rr / a.G);
    const uint32_t xy = __ldg(reinterpret_cast<const uint32_t*>(a.q + o * a.d_h) + pair);
    const float x = __uint_as_float(xy << 16), y = __uint_as_float(xy & 0xFFFF0000u);
    // the special-function unit's sine and cosine of an angle reduced to [-pi, pi]: about 5e-7
    // off, against the 2^-8 of the rounding to bf16 that the attention applies
    float sn, cs;
    __sincosf(rope_angle(L >= 1 && L <= a.T_cap ? L - 1 : 0, th), &sn, &cs);
    *reinterpret_cast<float2*>(a.qrope + o * 8 + 2 * (tid & 3)) = make_float2((x * cs - y * sn) * a.scale, (x * sn + y * cs) * a.scale);
  }
  cp_async_wait_all();
  __syncthreads();
  const int m0 = 16 * (warp & 1), n0 = 16 * (warp >> 1);
  if (row0 + m0 >= rows_g) return;
  float acc[2][4] = {};
#pragma unroll 4
  for (int k0 = 0; k0 < KP; k0 += 16) {
    uint32_t fa[4], fb[4];
    wmma16::load_a(fa, sq, QLD, m0, k0, lane);
    wmma16::load_b2(fb, sw, WLD, k0, n0, lane);
    wmma16::mma_16816(acc[0], fa, fb[0], fb[1]);
    wmma16::mma_16816(acc[1], fa, fb[2], fb[3]);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int row = row0 + m0 + (lane >> 2) + 8 * j;
    if (row >= rows_g) continue;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      const int c = c0 + n0 + 8 * nt + 2 * (lane & 3);
      if (c < a.d_c)
        *reinterpret_cast<__nv_bfloat162*>(a.qlat + index(row) * a.d_c + c) =
            __floats2bfloat162_rn(acc[nt][2 * j] * a.scale, acc[nt][2 * j + 1] * a.scale);
    }
  }
}

// ------------------------------------------------------------------ merge of the pieces, W_uv
// out[row][d] = sum_c (sum_j 2^(m_j - M) O_j[c] / sum_j 2^(m_j - M) l_j) W_uv[g][c][d] for 16 rows
// (sequence, query head of KV head g) and 64 columns per CTA.  Latency bound: the W_uv chunk is
// fetched and the pieces' slots are counted before the attention kernel is waited for, and a
// warp, which merges one row, has eight 16-byte loads per lane in flight: 4, 8 or 16 pieces of
// up to 256, 128 or 64 columns (CP quads of columns; with twice the loads only one CTA fits an
// SM, and 32 sequences at d_c = 256 take 2 us more).  The merged latent goes into the warp
// products as two bf16 halves, so its rounding does not count.
constexpr int kMRows = 16, kMCols = 64, kMThreads = 512, kMSlots = 8;
struct MergeArgs {
  int B, H, G, n_kv, d_c, d_h, P, workers, T_cap, cost;
  int kind;                    // cache kind
  MlaWindow win;
  mla_cache_t cache;
  const int32_t* seq_lens;
  const __nv_bfloat16* qlat;   // [B][H][d_c], scaled
  const float* qrope;          // [B][H][8], rotated, scaled
  const float* opart;
  const float* mlpart;
  const __nv_bfloat16* W_uv;   // [n_kv][d_c][d_h]
  __nv_bfloat16* out;          // [B][H][d_h]
  int32_t* err;
};

// Latent columns c .. c + 7 of token t (cache row `row`) of sequence b, of length L.
__device__ __forceinline__ void latent8(const MergeArgs& a, int b, int L, int t, size_t row, int c, float (&v)[8]) {
  const __nv_bfloat16* kept = nullptr;
  if (a.kind == MLA_CACHE_SAME) {
    kept = reinterpret_cast<const __nv_bfloat16*>(a.cache.c_kv) + row * a.d_c + c;
  } else if (a.cache.c_resid && t >= L - MLA_RESID_WINDOW) {
    const size_t slot = (size_t)b * MLA_RESID_WINDOW + (t & (MLA_RESID_WINDOW - 1));
    if (__ldg(a.cache.resid_pos + slot) == t) kept = reinterpret_cast<const __nv_bfloat16*>(a.cache.c_resid) + slot * a.d_c + c;
  }
  uint4 u;
  if (kept) {
    u = __ldg(reinterpret_cast<const uint4*>(kept));
  } else {
    const float scale = __half2float(__ldg(reinterpret_cast<const __half*>(a.cache.c_scales) + row * (a.d_c / 32) + c / 32));
    const uint8_t* codes = reinterpret_cast<const uint8_t*>(a.cache.c_kv);
    u = mla_kind_int4(a.kind) ? dequant8<4>(__ldg(reinterpret_cast<const uint32_t*>(codes + (row * a.d_c + c) / 2)), scale)
                              : dequant8<2>(__ldg(reinterpret_cast<const unsigned short*>(codes + (row * a.d_c + c) / 4)), scale);
  }
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = __uint_as_float(w[e] << 16);
    v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}

// One row's merged latent once more, from the cache and its own KV head's keys only, a lane per 8
// columns (whole warp; a token at a time, 3.5 ms for 4096: for rows that came out NaN).  Rows that
// the definition makes NaN end at the first such score.  (The test and this code cost the
// Llama-shaped calls 1.2 us at d_c = 256 and 0.6 with 4-bit latents, whether inlined or not; a test
// of the scores in the attention kernel, whose softmax has no registers for it, 1.0 and 3.)
__device__ __forceinline__ void exact_row(const MergeArgs& a, int b, int h, __nv_bfloat16* hi, __nv_bfloat16* lo) {
  const int lane = threadIdx.x & 31, c = 8 * lane, L = __ldg(a.seq_lens + b);   // a valid length: the row has pieces
  const bool mine = c < a.d_c;
  const size_t qi = (size_t)b * a.H + h;
  float q[8] = {}, o[8] = {}, m = -INFINITY, l = 0.f;
  if (mine) {
    const uint4 u = __ldcg(reinterpret_cast<const uint4*>(a.qlat + qi * a.d_c + c));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      q[2 * e] = __uint_as_float(w[e] << 16);
      q[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
  }
  const float qr = lane < 8 ? __bfloat162float(__float2bfloat16_rn(__ldcg(a.qrope + qi * 8 + lane))) : 0.f;
  const int from = max(0, L - a.win.window), sinks = min(a.win.n_sink, from);
#pragma unroll 1
  for (int i = 0; i < sinks + L - from; ++i) {
    const int t = i < sinks ? i : from + i - sinks;
    const MlaLoc lc = mla_loc(a.cache, b, t, a.err);
    const size_t row = (size_t)lc.pb * lc.cap + lc.pt;
    float v[8] = {}, s = 0.f;
    if (mine) latent8(a, b, L, t, row, c, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) s += q[e] * v[e];
    if (lane < 8) s += qr * __bfloat162float(__ldg(reinterpret_cast<const __nv_bfloat16*>(a.cache.k_rope) + (row * a.n_kv + h / a.G) * 8 + lane));
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    const float top = fmaxf(m, s), base = top == -INFINITY ? 0.f : top, al = exp2f(m - base), p = exp2f(s - base);
    m = top;
    l = l * al + p;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = o[e] * al + p * v[e];
    if (l != l) break;
  }
  if (!mine) return;
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float x = o[e] / l, y = o[e + 1] / l;
    const uint32_t w = pack2(x, y);
    *reinterpret_cast<uint32_t*>(hi + c + e) = w;
    *reinterpret_cast<uint32_t*>(lo + c + e) = pack2(x - __uint_as_float(w << 16), y - __uint_as_float(w & 0xFFFF0000u));
  }
}

template <int CP>
__global__ void __launch_bounds__(kMThreads, 2) window_merge_kernel(const __grid_constant__ MergeArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  using bf16 = __nv_bfloat16;
  constexpr int WLD = kMCols + 8;
  const int ALD = a.d_c + 8;
  bf16* sw = reinterpret_cast<bf16*>(smem);            // [d_c][WLD]
  bf16* shi = sw + a.d_c * WLD;                        // [16][ALD]
  bf16* slo = shi + kMRows * ALD;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rows_g = a.B * a.G, n_rb = (rows_g + kMRows - 1) / kMRows;
  const int g = blockIdx.x % a.n_kv, rb = (blockIdx.x / a.n_kv) % n_rb, cc = blockIdx.x / (a.n_kv * n_rb);
  const int row0 = rb * kMRows, d0 = cc * kMCols;
  const bf16* W = a.W_uv + (size_t)g * a.d_c * a.d_h;
  for (int v = tid; v < a.d_c * (kMCols / 8); v += kMThreads) {
    const int c = v / (kMCols / 8), d = (v % (kMCols / 8)) * 8;
    const bool ok = d0 + d < a.d_h;   // whole chunks: d_h is a multiple of 8
    cp_async16(smem_u32(sw + c * WLD + d), ok ? (const void*)(W + (size_t)c * a.d_h + d0 + d) : a.W_uv, ok ? 16u : 0u);
  }
  cp_async_commit();
  // Each warp finds its row's sequence among the units by itself: the last CTAs start when the
  // attention's have left their SMs, so barriers here cost time.
  const int r = warp, row = row0 + r, b = row / a.G;
  int total = 0, before = 0, units = 0, ne = 0;   // units of all, of the sequences before b, of b; non-empty ones before b
  for (int base = 0; base < a.B; base += 128) {
    int L[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int v = base + 32 * k + lane;
      L[k] = v < a.B ? __ldg(a.seq_lens + v) : 0;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int v = base + 32 * k + lane, n = units_of(L[k], a.T_cap, kUnit, a.cost, a.win).n;
      if (base + 32 * k >= a.B) continue;
      if (blockIdx.x == 0 && warp == 0 && (unsigned)L[k] > (unsigned)a.T_cap) raise_error(a.err, MLA_DEVERR_SEQ_LEN);   // treated as empty
      total += __reduce_add_sync(0xffffffffu, n);
      before += __reduce_add_sync(0xffffffffu, v < b ? n : 0);
      units += __reduce_add_sync(0xffffffffu, v == b ? n : 0);
      ne += __popc(__ballot_sync(0xffffffffu, v < b && n > 0));
    }
  }
  const int busy = busy_workers(total, a.workers);
  pdl_wait();   // the partials
  pdl_trigger();
  bool sound_row = true;   // whole warp
  {   // a row per warp
    constexpr int kBatch = kMSlots * 32 / CP;         // pieces per batch
    constexpr int kAcc = CP > 32 ? 2 : 1;             // quads of columns per lane
    const int quad = lane % CP, sub = lane / CP;      // (CP = 16: two pieces side by side)
    float4 acc[kAcc];
#pragma unroll
    for (int e = 0; e < kAcc; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < rows_g) {
      const int h = g * a.G + row % a.G;
      int first = 0, np = 0;
      if (units > 0) {
        const int w0 = worker_of(before + a.cost, total, busy), w1 = worker_of(before + units - 1, total, busy);
        first = w0 + ne;
        np = w1 - w0 + 1;
      }
      const float2* ml = reinterpret_cast<const float2*>(a.mlpart) + (size_t)h * a.P + first;
      const float* op = a.opart + ((size_t)first * a.H + h) * a.d_c + 4 * quad;
      const size_t step = (size_t)a.H * a.d_c;
      float4 v[kMSlots];
      // slot s of the batch from piece k on: its piece, and the lane's quad of columns there
      auto piece = [&](int k, int s) { return k + (CP > 32 ? s / 2 : CP == 32 ? s : 2 * s + sub); };
      auto fetch = [&](int k) {
#pragma unroll
        for (int s = 0; s < kMSlots; ++s) {
          const int c = 128 * (s % kAcc);
          v[s] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (piece(k, s) < np && 4 * quad + c < a.d_c) v[s] = __ldcg(reinterpret_cast<const float4*>(op + piece(k, s) * step + c));
        }
      };
      fetch(0);   // in the same round trip as the maxima
      float2 mine = lane < np ? __ldcg(ml + lane) : make_float2(-INFINITY, 0.f);
      float M = mine.x;
      for (int k = lane + 32; k < np; k += 32) M = fmaxf(M, __ldcg(ml + k).x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      float wt = 0.f, den = 0.f;
#pragma unroll 1
      for (int k = 0; k < np; k += kBatch) {
        if ((k & 31) == 0) {   // the weights of pieces k .. k + 31, one per lane
          if (k > 0) mine = k + lane < np ? __ldcg(ml + k + lane) : make_float2(-INFINITY, 0.f);
          wt = mine.x == -INFINITY ? 0.f : exp2f(mine.x - M);
          den += wt * mine.y;
        }
        if (k > 0) fetch(k);
#pragma unroll
        for (int s = 0; s < kMSlots; ++s) {
          const float wk = __shfl_sync(0xffffffffu, wt, piece(k, s) & 31);   // 0 past the last piece
          float4& x = acc[s % kAcc];
          x.x += wk * v[s].x; x.y += wk * v[s].y; x.z += wk * v[s].z; x.w += wk * v[s].w;
        }
      }
      if (CP == 16) {
        acc[0].x += __shfl_xor_sync(0xffffffffu, acc[0].x, 16); acc[0].y += __shfl_xor_sync(0xffffffffu, acc[0].y, 16);
        acc[0].z += __shfl_xor_sync(0xffffffffu, acc[0].z, 16); acc[0].w += __shfl_xor_sync(0xffffffffu, acc[0].w, 16);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
      sound_row = units == 0 || den > 0.f;                // a score that is no number makes the sum one as well
      const float inv = units > 0 ? 1.f / den : 0.f;
#pragma unroll
      for (int e = 0; e < kAcc; ++e) { acc[e].x *= inv; acc[e].y *= inv; acc[e].z *= inv; acc[e].w *= inv; }
    }
#pragma unroll
    for (int e = 0; e < kAcc; ++e) {
      const int c = 128 * e + 4 * quad;
      if (c >= a.d_c || sub > 0) continue;
      const uint32_t h0 = pack2(acc[e].x, acc[e].y), h1 = pack2(acc[e].z, acc[e].w);
      const uint32_t l0 = pack2(acc[e].x - __uint_as_float(h0 << 16), acc[e].y - __uint_as_float(h0 & 0xFFFF0000u));
      const uint32_t l1 = pack2(acc[e].z - __uint_as_float(h1 << 16), acc[e].w - __uint_as_float(h1 & 0xFFFF0000u));
      *reinterpret_cast<uint2*>(shi + r * ALD + c) = make_uint2(h0, h1);
      *reinterpret_cast<uint2*>(slo + r * ALD + c) = make_uint2(l0, l1);
    }
  }
  cp_async_wait_all();
  if (!sound_row) {   // (off the way of the usual case)
    __syncwarp();   // other lanes write over what was stored
    exact_row(a, b, g * a.G + row % a.G, shi + r * ALD, slo + r * ALD);
  }
  __syncthreads();
  if (warp >= kMCols / 8) return;
  const int n0 = 8 * warp;   // this warp's columns
  float ahi[4] = {}, alo[4] = {};
#pragma unroll 2
  for (int k0 = 0; k0 < a.d_c; k0 += 32) {
    uint32_t bw[4], fh[4], fl[4];
    // four 8 x 8 blocks down the columns: B fragments of two steps of 16
    wmma16::ldsm_x4_t(smem_u32(sw + (k0 + lane) * WLD + n0), bw[0], bw[1], bw[2], bw[3]);
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      wmma16::load_a(fh, shi, ALD, 0, k0 + 16 * st, lane);
      wmma16::load_a(fl, slo, ALD, 0, k0 + 16 * st, lane);
      wmma16::mma_16816(ahi, fh, bw[2 * st], bw[2 * st + 1]);
      wmma16::mma_16816(alo, fl, bw[2 * st], bw[2 * st + 1]);
    }
  }
  const int d = d0 + n0 + 2 * (lane & 3);
  if (d >= a.d_h) return;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int row = row0 + (lane >> 2) + 8 * j;
    if (row >= rows_g) continue;
    const size_t o = ((size_t)(row / a.G) * a.H + g * a.G + row % a.G) * a.d_h + d;
    *reinterpret_cast<__nv_bfloat162*>(a.out + o) = __floats2bfloat162_rn(ahi[2 * j] + alo[2 * j], ahi[2 * j + 1] + alo[2 * j + 1]);
  }
}

// ------------------------------------------------------------------ host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = []() -> EncodeTiledFn {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &qr) == cudaSuccess &&
        qr == cudaDriverEntryPointSuccess)
      return (EncodeTiledFn)p;
    return nullptr;
  }();
  return fn;
}

// 2-D map: bf16 boxes of 64 columns with the 128-byte swizzle, or plain byte rows (codes).
static bool map_2d(CUtensorMap* m, bool bytes, const void* base, uint64_t cols, uint64_t rows, uint32_t box_cols,
                   uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t gdim[2] = {cols, rows};
  cuuint64_t gstride[1] = {cols * (bytes ? 1 : 2)};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t es[2] = {1, 1};
  return fn(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), gdim,
            gstride, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, bytes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Layout {
  int N, NC, NK, NRAW, n_cbox, n_kbox, kr_rows;
  uint32_t off_q, off_qr, off_p, off_c, off_k, off_raw, raw_stage, off_red, off_list, off_bar, total;
};

// [Q_lat boxes][RoPE query boxes][P of two streams][latent ring][key-box ring][code ring]
// [exchange][pieces][barriers].  Of the slots left (16 KB: 128 tokens x 64 columns) a tile's key boxes
// come first, the others hold latent tiles, at least two (one per stream).  Dequantised latents
// are not in flight: two tiles of them, three of codes, and key boxes in all the rest.
static bool layout(const mla_config_t& c, int R, Layout* out) {
  Layout L{};
  const int G = c.n_heads / c.n_kv_heads, qbits = mla_kind_quant(c.cache_kind) ? mla_quant_bits(c.cache_kind) : 0;
  L.N = c.n_heads <= 16 ? 16 : 32;
  L.n_cbox = (c.d_c + 63) / 64;
  L.n_kbox = (R + 63) / 64;
  L.kr_rows = L.n_kbox == 1 || G > 2 ? L.N : 16;
  L.NRAW = qbits ? 3 : 0;
  L.raw_stage = (uint32_t)(kT * c.d_c * qbits / 8);
  L.off_qr = (uint32_t)(L.n_cbox * L.N) * 128;
  L.off_p = L.off_qr + (uint32_t)(L.n_kbox * L.kr_rows) * 128;
  L.off_c = L.off_p + 2u * kT * L.N * 2;
  const uint32_t tail = kRedBytes + kPieces * 16 + 8 * kBars + 16 + 1024 + 1024;   // alignment, static part
  const uint32_t fixed = L.off_c + L.NRAW * L.raw_stage + tail;
  if (fixed > kSmemMax) return false;
  const int slots = (int)((kSmemMax - fixed) / kSlot);
  L.NC = qbits ? 2 : std::max(2, std::min(kMaxC, (slots - L.n_kbox) / L.n_cbox));
  L.NK = std::min(kMaxK, slots - L.NC * L.n_cbox);
  if (L.NK < 1) return false;
  L.off_k = L.off_c + (uint32_t)(L.NC * L.n_cbox) * kSlot;
  L.off_raw = L.off_k + (uint32_t)L.NK * kSlot;
  L.off_red = L.off_raw + L.NRAW * L.raw_stage;
  L.off_list = L.off_red + kRedBytes;
  L.off_bar = L.off_list + kPieces * 16;
  L.total = L.off_bar + 8 * kBars + 16 + 1024;
  *out = L;
  return true;
}

}  // namespace wdec
}  // namespace mla

// Shapes: bf16 with r = 4 kept pairs per KV head, up to 32 query heads and 32 KV heads, d_c a
// multiple of 32 up to 256, head dim a multiple of 8, code rows of whole 16 bytes.
bool mla_window_decode_capable(const mla_plan& p) {
  const mla_config_t& c = p.cfg;
  if (c.dtype != MLA_BF16 || c.r_pairs != 4 || c.n_heads > 32 || c.head_dim % 8 != 0 || c.d_c % 32 != 0 || c.d_c > 256) return false;
  if (mla_kind_quant(c.cache_kind) && c.d_c * mla_quant_bits(c.cache_kind) / 8 % 16 != 0) return false;
  mla::wdec::Layout L;
  return mla::wdec::layout(c, p.R, &L);
}

cudaError_t mla_launch_window_decode(const mla_plan& p, const mla_cache_t& c, const int32_t* seq_lens, const void* q,
                                     int B, void* out, void* ws, const DecodeLayout& D, MlaWindow win, cudaStream_t s) {
  using namespace mla::wdec;
  const mla_config_t& cfg = p.cfg;
  char* base = (char*)ws;
  const int qbits = mla_kind_quant(cfg.cache_kind) ? mla_quant_bits(cfg.cache_kind) : 0;
  Layout L;
  if (!layout(cfg, p.R, &L)) return cudaErrorInvalidValue;
  Args a;
  a.H = cfg.n_heads; a.G = a.H / cfg.n_kv_heads; a.d_c = cfg.d_c; a.dcp = L.n_cbox * 64; a.R = p.R; a.P = D.P;
  a.T_cap = c.T_cap; a.n_cbox = L.n_cbox; a.n_kbox = L.n_kbox; a.kr_rows = L.kr_rows;
  a.NC = L.NC; a.NK = L.NK; a.NRAW = L.NRAW;
  a.n_blk = (L.n_cbox + 1) / 2;
  a.B = B; a.workers = D.G; a.win = win; a.skip_tile = p.opt_skip_tile;
  // about 5 us, the time a CTA takes for 220 KB; a unit of short rows is bound by latency instead
  a.cost = std::max(2, std::min(8, (int)(3400 / mla_cache_bytes_per_token(&cfg))));
  a.pieces = (int4*)(base + D.off_piece_b);
  a.seq_lens = seq_lens; a.qrope = (const float*)(base + D.off_qrope);
  a.opart = (float*)(base + D.off_opart); a.mlpart = (float*)(base + D.off_mlpart);
  a.scales = (const __half*)c.c_scales; a.code_row = (uint32_t)(cfg.d_c * qbits / 8); a.cache = c; a.err = p.err;
  a.wait_ns = (uint64_t)p.opt_wait_us * 1000u;
  a.off_q = L.off_q; a.off_qr = L.off_qr; a.off_p = L.off_p; a.off_c = L.off_c; a.off_k = L.off_k; a.off_raw = L.off_raw;
  a.raw_stage = L.raw_stage; a.off_red = L.off_red; a.off_list = L.off_list; a.off_bar = L.off_bar;
  const uint64_t rows = mla_cache_rows(c);
  CUtensorMap tm_c, tm_kr, tm_q;
  bool ok = map_2d(&tm_kr, false, c.k_rope, p.R, rows, 64, kUnit) &&
            map_2d(&tm_q, false, base + D.off_qlat, cfg.d_c, (uint64_t)B * a.H, 64, a.H);
  ok = ok && (qbits ? map_2d(&tm_c, true, c.c_kv, a.code_row, rows, a.code_row, kUnit)
                    : map_2d(&tm_c, false, c.c_kv, cfg.d_c, rows, 64, kUnit));
  if (!ok) return cudaErrorInvalidValue;
  auto pick = [&](auto n) {
    constexpr int N = decltype(n)::value;
    return qbits == 4 ? window_decode_kernel<N, 4> : qbits == 2 ? window_decode_kernel<N, 2> : window_decode_kernel<N, 0>;
  };
  const auto kern = L.N == 16 ? pick(std::integral_constant<int, 16>()) : pick(std::integral_constant<int, 32>());
  AbsorbArgs b;
  b.B = B; b.H = a.H; b.G = a.G; b.n_kv = cfg.n_kv_heads; b.d_h = cfg.head_dim; b.d_c = cfg.d_c; b.T_cap = c.T_cap;
  b.scale = mla::kLog2e * (cfg.softmax_scale > 0.0f ? cfg.softmax_scale : (float)(1.0 / sqrt((double)cfg.head_dim)));
  b.q = (const __nv_bfloat16*)q; b.W_ukF = (const __nv_bfloat16*)p.W_ukF; b.seq_lens = seq_lens;
  b.rope_pair = p.rope_pair; b.theta = p.theta;
  b.qlat = (__nv_bfloat16*)(base + D.off_qlat); b.qrope = (float*)(base + D.off_qrope);
  const int KP = (cfg.head_dim + 15) & ~15;
  const size_t smem_b = sizeof(__nv_bfloat16) * ((size_t)KP * (kACols + 8) + (size_t)kARows * (KP + 8));
  const int n_rba = (B * a.G + kARows - 1) / kARows, n_cca = (cfg.d_c + kACols - 1) / kACols;
  cudaError_t e = mla_smem_limit(p, (const void*)window_absorb_kernel, smem_b);
  if (e == cudaSuccess) e = mla_profile_event(p, kProfAbsorb, false, s);
  if (e == cudaSuccess)
    e = mla_launch_kernel(window_absorb_kernel, dim3(cfg.n_kv_heads * n_rba * n_cca), dim3(kAThreads), smem_b, s, p.opt_pdl, b);
  if (e == cudaSuccess) e = mla_profile_event(p, kProfAbsorb, true, s);
  if (e == cudaSuccess) e = mla_smem_limit(p, (const void*)kern, L.total);
  if (e == cudaSuccess) e = mla_profile_event(p, kProfAttention, false, s);
  if (e == cudaSuccess)
    e = mla_launch_kernel(kern, dim3(D.G), dim3(qbits ? kThreadsOf<4> : kThreadsOf<0>), L.total, s, p.opt_pdl, tm_c, tm_kr, tm_q, a);
  if (e == cudaSuccess) e = mla_profile_event(p, kProfAttention, true, s);
  if (e != cudaSuccess) return e;
  MergeArgs m;
  m.B = B; m.H = a.H; m.G = a.G; m.n_kv = cfg.n_kv_heads; m.d_c = cfg.d_c; m.d_h = cfg.head_dim; m.P = D.P;
  m.workers = D.G; m.cost = a.cost; m.T_cap = c.T_cap; m.win = win; m.seq_lens = seq_lens; m.opart = a.opart; m.mlpart = a.mlpart;
  m.W_uv = (const __nv_bfloat16*)p.W_uv; m.out = (__nv_bfloat16*)out; m.err = p.err;
  m.kind = cfg.cache_kind; m.cache = c; m.qlat = b.qlat; m.qrope = a.qrope;
  const size_t smem = sizeof(__nv_bfloat16) * ((size_t)cfg.d_c * (kMCols + 8) + 2 * (size_t)kMRows * (cfg.d_c + 8));
  const int n_rb = (B * a.G + kMRows - 1) / kMRows, n_cc = (cfg.head_dim + kMCols - 1) / kMCols;
  const auto merge = cfg.d_c <= 64 ? window_merge_kernel<16> : cfg.d_c <= 128 ? window_merge_kernel<32> : window_merge_kernel<64>;
  e = mla_smem_limit(p, (const void*)merge, smem);
  if (e == cudaSuccess) e = mla_profile_event(p, kProfCombine, false, s);
  if (e == cudaSuccess)
    e = mla_launch_kernel(merge, dim3(cfg.n_kv_heads * n_rb * n_cc), dim3(kMThreads), smem, s, p.opt_pdl, m);
  if (e == cudaSuccess) e = mla_profile_event(p, kProfCombine, true, s);
  return e;
}
